"""attn_key_weights against the fp64 oracle.

Tolerance. A score is a sum of D products of bf16 pairs, exact each, added in the tensor core
with at least 24 bits below the largest partial sum: off by at most D 2^-23 sum|q k|, and by
2^-22 of it in practice; the products with scale and log2 e, the distance term, the soft-cap
(2^-22 cap) and the subtraction of the LSE add a few 2^-24 of their sizes. In all the exponent is
within E = 2^-17 (sum|q k| scale + |LSE| + |distance term| + cap) for D <= 128, so a part p is
within p (E + 2^-21) (ex2.approx: 2 ulp). The sum of n parts adds n 2^-24 of it, the previous
weight and the last addition 2^-23. The oracle returns sum p (1 + sizes); 2^-16 times it covers
all of these for n <= 2048 rows."""
import ctypes

import numpy as np
import pytest
import torch

from oracle.long_context import cached_rows, key_weights, row_scores, slopes, visible
from tests.helpers import check_canaries, guarded_empty

FILL = 7.0


class Case:
    def __init__(self, lens, Hq=4, Hkv=2, Sq=1, D=64, page=16, extra=3, seed=0, window=0,
                 softcap=0.0, alibi=False, causal=True, paged=True, scale=0.0, qscale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.lens = torch.tensor(lens, dtype=torch.int32)
        B, self.page, self.paged = len(lens), page, paged
        self.kw = dict(window=window, softcap=softcap, scale=scale)
        self.alibi, self.causal, self.shape = alibi, causal, (B, Hq, Hkv, Sq, D)
        most = max(max(lens), 1)
        self.L = most + extra
        self.q = (torch.randn(B, Hq, Sq, D, generator=g) * qscale).to(torch.bfloat16)
        if paged:
            n = (self.lens + page - 1) // page
            self.table = torch.full((B, -(-self.L // page)), -1, dtype=torch.int32)
            used = torch.arange(self.table.shape[1])[None] < n[:, None]
            perm = torch.randperm(int(n.sum()) + 2, generator=g).to(torch.int32)
            self.table[used] = perm[:int(n.sum())]
            self.k = torch.randn(len(perm), Hkv, page, D, generator=g).to(torch.bfloat16)
        else:
            self.table = None
            self.k = torch.randn(B, Hkv, most, D, generator=g).to(torch.bfloat16)
        self.previous = torch.rand(B, Hkv, self.L, generator=g)
        self.lse = self.oracle_lse()

    def rows(self, b, head):
        n, k = int(self.lens[b]), self.k.double().numpy()
        if self.table is None:
            return k[b, head, :n]
        return cached_rows(k, self.table.numpy(), b, n, head, self.page)

    def each(self):
        B, Hq, Hkv, Sq, D = self.shape
        return ((b, h, r) for b in range(B) for h in range(Hq) for r in range(Sq))

    def oracle_lse(self):
        B, Hq, Hkv, Sq, D = self.shape
        out = np.full((B, Hq, Sq), -np.inf)
        q = self.q.double().numpy()
        for b, h, r in self.each():
            n = int(self.lens[b])
            see = visible(n, n - Sq + r, self.causal, self.kw["window"])
            if see.any():
                s = row_scores(q[b, h, r], self.rows(b, h * Hkv // Hq), n - Sq + r,
                               self.kw["scale"] or D ** -0.5,
                               slopes(Hq)[h] if self.alibi else None, self.kw["softcap"])[see]
                out[b, h, r] = s.max() + np.log(np.exp(s - s.max()).sum())
        return torch.from_numpy(out).float()

    def variant(self):
        import masked_attention_gb300 as M
        return ((M.MASK_CAUSAL if self.causal else 0) | (M.MASK_WINDOW if self.kw["window"] else 0)
                | (M.SCORE_SOFTCAP if self.kw["softcap"] else 0)
                | (M.SCORE_ALIBI if self.alibi else 0))

    def run(self, previous="apart", decay=0.5, **extra):
        import masked_attention_gb300 as M
        B, Hq, Hkv, Sq, D = self.shape
        w = guarded_empty((B, Hkv, self.L if self.paged else max(self.L, self.k.shape[2])),
                          torch.float32)
        w.fill_(FILL)
        prev = {"apart": self.previous.cuda(), "same": w, "none": None}[previous]
        if previous == "same":
            w[:, :, :self.L] = self.previous.cuda()
        kw = dict(self.kw, previous=prev, decay=decay, seq_lens=self.lens.cuda())
        if self.paged:
            kw.update(page_table=self.table.cuda(), page_size=self.page)
        M.attn_key_weights(self.q.cuda(), self.k.cuda(), self.lse.cuda(), w, self.variant(),
                           **{**kw, **extra})
        assert M.attn_check_status() == M.ATTN_OK
        check_canaries()
        return w

    def check(self, previous="apart", decay=0.5, **extra):
        B, Hq, Hkv, Sq, D = self.shape
        w = self.run(previous, decay, **extra).double().cpu().numpy()
        prev = None if previous == "none" else self.previous.double().numpy()
        before = (prev if previous == "same" else np.full(w.shape, FILL))
        kw = {k: v for k, v in self.kw.items() if k != "scale"}
        ref, size = key_weights(self.q.double().numpy(), self.rows, self.lse.double().numpy(),
                                prev, decay, self.lens, before, causal=self.causal,
                                alibi=slopes(Hq) if self.alibi else None,
                                scale=self.kw["scale"] or None, **kw)
        tol = 2.0 ** -16 * size + 2.0 ** -23 * np.abs(ref)
        bad = ~(np.abs(w - ref) <= tol)
        for b in range(B):
            bad[b, :, int(self.lens[b]):] = (w != before)[b, :, int(self.lens[b]):]
        assert not bad.any(), (np.argwhere(bad)[:4], w[bad][:4], ref[bad][:4], tol[bad][:4])
        return w


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("Hq,Hkv,Sq", [(1, 1, 1), (4, 2, 1), (14, 2, 3), (8, 8, 2), (16, 1, 16)])
def test_pages_heads_and_rows(Hq, Hkv, Sq, page, D):
    Case([1, 0, 127, 128, 129, 300], Hq, Hkv, Sq, D, page).check()


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,Sq", [(2, 1, 120), (4, 1, 64), (6, 2, 86), (4, 1, 65), (3, 1, 257),
                                       (2, 1, 400)])
def test_many_rows(Hq, Hkv, Sq, D):
    """Up to 256 rows of a head in one product, and blocks of them; tiles in pairs and alone."""
    Case([0, 40, 400, 513, 640], Hq, Hkv, Sq, D, 32, seed=2).check()


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kw", [dict(alibi=True), dict(softcap=20.0), dict(softcap=2.0, alibi=True),
                                dict(window=1), dict(window=50), dict(window=129, softcap=30.0),
                                dict(window=300, alibi=True, Sq=70), dict(causal=False, Sq=5),
                                dict(causal=False, window=40, Sq=3), dict(scale=0.3),
                                dict(softcap=1e6, Sq=90), dict(qscale=12.0, softcap=50.0)])
def test_variants(kw, D):
    Case([5, 700, 0, 256, 383], D=D, seed=3, **kw).check()


@pytest.mark.gpu
@pytest.mark.parametrize("Sq", [1, 9, 150])
def test_contiguous_keys(Sq):
    Case([200, 3, 131], Sq=Sq, paged=False, D=128).check()
    Case([200, 200, 200], Sq=Sq, paged=False).check(seq_lens=None)


@pytest.mark.gpu
def test_previous_weights():
    """Apart, in place, none; a decay of 0 does not read them."""
    c = Case([150, 40])
    c.check("same", 1.0)
    c.check("same", 0.9)
    c.check("none")
    c.previous[:] = float("nan")
    c.check("none", 0.0)
    a = c.run("none")
    b = c.run("apart", decay=0.0)
    assert torch.equal(a[0, :, :150], b[0, :, :150]) and torch.equal(a[1, :, :40], b[1, :, :40])
    c = Case([150, 400], window=30)
    c.check("same", 0.75)     # keys before the window only decay
    c.check("none")


@pytest.mark.gpu
def test_sum_over_keys_counts_the_rows():
    c = Case([700, 61, 1], Hq=6, Hkv=2, Sq=3)
    w = c.run("none")
    for b, n in enumerate([700, 61, 1]):
        seen = sum(1 for r in range(3) if n - 3 + r >= 0) * 3
        assert (w[b, :, :n].double().sum(-1) - seen).abs().max() < 1e-4


@pytest.mark.gpu
def test_what_no_row_sees_changes_nothing():
    """NaN in the rest of the last page, in foreign pages, behind the window, and LSE -inf."""
    c = Case([70, 3, 200], Hq=4, Hkv=2, Sq=4, window=40, page=32)
    a = c.run("none")
    for b, n in enumerate([70, 3, 200]):
        for j in [j for j in range(200) if j >= n or j <= n - 4 - 40]:
            at = int(c.table[b, j // 32]) if j // 32 < c.table.shape[1] else -1
            if at >= 0:
                c.k[at, :, j % 32] = float("nan") if j % 2 else float("inf")
    b = c.run("none")
    assert torch.equal(a, b) and torch.isfinite(a).all()
    assert (c.lse[1, :, 0] == -np.inf).all()     # a row before the sequence's start


@pytest.mark.gpu
@pytest.mark.parametrize("Sq,Hq,Hkv", [(1, 4, 2), (3, 4, 2), (16, 8, 2), (40, 16, 2)])
@pytest.mark.parametrize("kw", [dict(), dict(softcap=20.0), dict(alibi=True), dict(window=100)])
def test_rows_without_an_lse_add_nothing(kw, Sq, Hq, Hkv):
    """Places of a batch that hold no row: LSE -inf, and whatever their queries were left with."""
    c = Case([700, 300, 129], Hq, Hkv, Sq, seed=8, **kw)
    gone = torch.zeros(c.lse.shape, dtype=torch.bool)
    gone[0, 1], gone[0, 0, -1], gone[1] = True, True, True
    c.lse[gone] = -float("inf")
    c.q[gone] = float("nan")
    c.q[0, 1, 0, 3], c.q[1, 0] = float("inf"), -float("inf")
    c.check()

@pytest.mark.gpu
def test_many_sequences():
    """More sequences than threads, most of a tile or less, empty ones among them."""
    lens = np.random.default_rng(6).integers(0, 30, 3000)
    lens[[5, 1500, 2999]] = 300, 129, 128
    Case(lens.tolist(), Hq=2, Hkv=1, Sq=2).check()


@pytest.mark.gpu
def test_nan_of_a_visible_key_shows_there():
    c = Case([40, 150], Hq=4, Hkv=2)
    at = int(c.table[1, 5])
    c.k[at, 1, 3] = float("nan")
    w = c.run("none").cpu()
    hit = torch.isnan(w)
    assert hit[1, 1, 83] and int(hit.sum()) == 1
    c.lse[0, 2] = float("nan")                   # an LSE that is NaN: its head's keys
    hit = torch.isnan(c.run("none").cpu())
    assert hit[0, 1, :40].all() and not hit[0, 0].any() and int(hit.sum()) == 41


@pytest.mark.gpu
@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kw", [dict(), dict(softcap=20.0), dict(alibi=True), dict(window=690)])
@pytest.mark.parametrize("Sq,Hq,Hkv", [(1, 1, 1), (1, 8, 2), (5, 8, 2), (37, 7, 1), (16, 16, 1)])
def test_infinite_visible_keys(Sq, Hq, Hkv, kw, D, paged):
    """Keys with a channel of -infinity or +infinity, all queries positive there, in whole tiles and
    in the last one: their score is that infinity (with a soft-cap -cap or cap), so their weight is
    0 or infinity (sum of exp(+-cap - LSE)), wherever they lie and however many rows a head has;
    other keys keep their bits."""
    c = Case([700, 640], Hq, Hkv, Sq, D, 32, seed=9, paged=paged, **kw)
    c.q[..., 3] = 0.25 + c.q[..., 3].abs()
    c.lse = c.oracle_lse()
    ref = c.run("same", 0.5)
    low, high = (12, 300, 530, 645), (77, 310, 650)
    for j in low + high:
        x = -np.inf if j in low else np.inf
        for b, n in enumerate(c.lens.tolist()):
            if j >= n:
                continue
            if paged:
                c.k[int(c.table[b, j // 32]), :, j % 32, 3] = x
            else:
                c.k[b, :, j, 3] = x
    w = c.run("same", 0.5)
    lse = c.lse.double().numpy()
    old = 0.5 * c.previous.double().numpy()
    hit = torch.zeros(w.shape, dtype=torch.bool, device="cuda")
    for j in low + high:
        for b, n in enumerate(c.lens.tolist()):
            for h in range(Hkv if j < n else 0):
                hit[b, h, j] = True
                got = float(w[b, h, j])
                # rows of the head that see the key: positions i with j <= i, i - j < window
                i = n - Sq + np.arange(Sq)
                see = (j <= i) & ((i - j < c.kw["window"]) | (c.kw["window"] == 0))
                L = lse[b, h * (Hq // Hkv):(h + 1) * (Hq // Hkv)][:, see]
                if c.kw["softcap"]:
                    s = -20.0 if j in low else 20.0
                    # E of the module's tolerance without the product, which the cap swallows
                    tol = np.exp(s - L).sum() * 2.0 ** -16 * (1 + 5 * 20 + np.abs(L).max(initial=0))
                    assert abs(got - old[b, h, j] - np.exp(s - L).sum()) <= tol + 2.0 ** -23 * got, (b, h, j)
                elif j in low or not L.size:
                    assert got == np.float32(old[b, h, j]), (b, h, j, got)
                else:
                    assert got == np.inf, (b, h, j, got)
    assert torch.equal(w[~hit], ref[~hit])


@pytest.mark.gpu
def test_pages_outside_the_pool_and_lengths_outside_the_bound():
    c = Case([100, 90, 30])
    c.table[0, 2], c.table[1, 0], c.table[2, 1] = -5, len(c.k), 2 ** 31 - 1
    c.lse = c.oracle_lse()
    c.check()
    c = Case([60, 0, 70], extra=0, page=16)
    w = c.run("none")
    far = c.lens.clone()
    far[1], far[2] = -9, 10 ** 9                 # 0 and the weights' row length
    assert torch.equal(c.run("none", seq_lens=far.cuda())[1:], w[1:])


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """A pool of more than 4 GiB whose pages lie at its end."""
    c = Case([90, 33], Hkv=2, D=128, page=128, Hq=2)
    w = c.run("none")
    pages = (1 << 32) // (2 * 2 * 128 * 128) + len(c.k)
    pool = torch.empty(pages, 2, 128, 128, dtype=torch.bfloat16, device="cuda")
    pool[-len(c.k):] = c.k.cuda()
    import masked_attention_gb300 as M
    out = torch.full_like(w, FILL)
    table = torch.where(c.table >= 0, c.table + pages - len(c.k), -1).to(torch.int32)
    M.attn_key_weights(c.q.cuda(), pool, c.lse.cuda(), out, c.variant(), page_table=table.cuda(),
                       page_size=128, seq_lens=c.lens.cuda())
    assert torch.equal(out, w)


@pytest.mark.gpu
def test_reproducible_captured_and_on_another_stream():
    import masked_attention_gb300 as M
    c = Case([900, 0, 77, 1300], Hq=8, Hkv=4, Sq=2, D=128, page=64)
    w = c.run("none")
    q, k, lse, table, lens = (t.cuda() for t in (c.q, c.k, c.lse, c.table, c.lens))
    outs = [torch.full_like(w, FILL) for _ in range(2)]

    def call(i):
        M.attn_key_weights(q, k, lse, outs[i], c.variant(), page_table=table, page_size=64,
                           seq_lens=lens)

    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):                # the current stream is followed
        call(0)
        call(0)
    side.synchronize()
    assert torch.equal(outs[0], w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(1)
    lens.copy_(torch.tensor([0, 0, 5, 0], dtype=torch.int32))
    graph.replay()                               # new lengths: only what they reach is written
    torch.cuda.synchronize()
    assert (outs[1][0] == FILL).all() and (outs[1][2, :, 5:] == FILL).all()
    lens.copy_(c.lens)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[1], w)


@pytest.mark.gpu
def test_a_wait_that_runs_out_is_reported():
    """No copy is issued: the bounded waits end, the status tells, the context goes on."""
    import masked_attention_gb300 as M
    c = Case([900, 300], Hq=8, Hkv=4, Sq=2)
    w = torch.zeros(2, 4, c.L, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(page_table=c.table.cuda(), page_size=16, seq_lens=c.lens.cuda())
    M.attn_key_weights(c.q.cuda(), c.k.cuda(), c.lse.cuda(), w, c.variant(), status=status,
                       timeout_ns=20_000_000, fault_inject=M.FAULT_NO_LOADS, **kw)
    assert M.attn_check_status(status) == M.ATTN_ERR_TIMEOUT
    assert M.attn_check_status(status) == M.ATTN_OK
    c.check()


def test_oracle_weights_against_a_softmax():
    rng = np.random.default_rng(0)
    q, K = rng.normal(size=(1, 2, 3, 8)), rng.normal(size=(9, 8))
    s = np.einsum("hrd,jd->hrj", q[0], K) * 8 ** -0.5
    s[:, np.arange(9)[None] > (9 - 3 + np.arange(3))[:, None]] = -np.inf
    lse = np.log(np.exp(s).sum(-1))
    got, _ = key_weights(q, lambda b, h: K, lse[None], np.ones((1, 1, 9)), 0.5, [9],
                         np.zeros((1, 1, 9)))
    p = np.exp(s) / np.exp(s).sum(-1, keepdims=True)
    assert np.allclose(got[0, 0], 0.5 + p.sum((0, 1)), rtol=0, atol=1e-12)


def test_refusals():
    import masked_attention_gb300 as M
    L = M.lib()

    def call(B=2, Hq=4, Hkv=2, Sq=1, max_len=100, D=64, stride=100, variant=M.MASK_CAUSAL,
             q=0x1000, k=0x2000, lse=0x3000, prev=None, w=0x4000, decay=1.0, lens=0x5000, **kw):
        p = M.attn_params(M.BF16)
        p.page_table, p.page_size, p.pages_per_seq, p.num_pages = 0x6000, 16, 7, 50
        for n, v in kw.items():
            setattr(p, n, v)
        return L.attn_key_weights(q, k, lse, prev, decay, w, B, Hq, Hkv, Sq, max_len, D, stride,
                                  variant, ctypes.byref(p), lens, None)

    inv, uns, mis = M.ATTN_ERR_INVALID_ARG, M.ATTN_ERR_UNSUPPORTED, M.ATTN_ERR_MISALIGNED
    assert call(B=-1) == call(Hq=5) == call(Sq=0) == call(max_len=-1) == call(stride=99) == inv
    assert call(decay=float("nan")) == call(decay=float("inf")) == inv
    assert call(D=96) == call(dtype=M.F32) == call(page_size=48) == uns
    assert call(variant=M.MASK_DOCUMENT) == call(variant=M.SCORE_RELBIAS) == uns
    assert call(variant=1 << 20) == inv
    assert call(variant=M.MASK_WINDOW) == call(variant=M.SCORE_SOFTCAP) == inv
    assert call(variant=M.SCORE_SOFTCAP, softcap=float("inf")) == inv
    assert call(scale=-1.0) == call(scale=float("nan")) == inv
    assert call(q_offset=1) == call(kv_offset=1) == uns
    assert call(pages_per_seq=6) == call(num_pages=0) == inv
    assert call(num_pages=2 ** 30) == uns
    assert call(B=40000) == call(Sq=2 ** 23) == uns
    assert call(max_len=2 ** 31 - 200, stride=2 ** 31 - 1, pages_per_seq=2 ** 28) == uns
    assert call(q=None) == call(k=None) == call(lse=None) == call(w=None) == inv
    assert call(q=0x1008) == call(k=0x2008) == call(lse=0x3002) == call(w=0x4001) == mis
    assert call(lens=0x5002) == call(page_table=0x6001) == call(alibi_slopes=0x7001) == mis
    assert call(prev=0x4004) == call(prev=0x4000 - 4) == call(prev=0x4000 + 4 * 399) == inv
    assert call(B=0) == call(max_len=0) == M.ATTN_OK
    t = torch.zeros(1, 1, 1, 64)
    with pytest.raises(ValueError):
        M.attn_key_weights(t, t, t, t)
