"""attn_cache_evict against the oracle's key-by-key eviction: indices, lengths, pages and copies
of weights and rows, so everything is equal bit by bit."""
import ctypes

import numpy as np
import pytest
import torch

from oracle.long_context import evict
from tests.helpers import check_canaries, guarded_empty

NAMES = ("weights_out", "kept", "new_lens", "freed", "info", "k", "v")


class Case:
    def __init__(self, lens, keep, recent=0, sink=0, starts=None, Hkv=2, D=64, page=16, extra=5,
                 seed=0, copy=False, kind="spread", L=None):
        rng = np.random.default_rng(seed)
        B = len(lens)
        self.lens, self.keep, self.recent, self.sink = np.asarray(lens, np.int32), keep, recent, sink
        self.starts = None if starts is None else np.asarray(starts, np.int32)
        self.page, self.D = page, D
        most = max(max(lens), 1)
        self.L = most + extra if L is None else L
        per = -(-self.L // page)
        shape = (B, Hkv, self.L)
        w = np.exp(3 * rng.normal(size=shape)).astype(np.float32)
        self.weights = {"spread": w, "zeros": np.where(rng.random(shape) < 0.6, 0, w),
                        "equal": np.zeros(shape), "signed": rng.normal(size=shape),
                        "few": rng.integers(0, 3, shape) - 1.0,
                        "close": 1 + rng.integers(0, 9, shape) * 2.0 ** -23}[kind].astype(np.float32)
        n = np.minimum(-(-np.maximum(self.lens, 0) // page), per)
        s = self.sequence_starts()
        hold = np.minimum(np.maximum(self.lens, 0), s + keep)
        new_per = -(-int(hold.max()) // page) + 1
        pages = int(n.sum()) + 3 + (B * new_per if copy else 0)
        perm = rng.permutation(pages).astype(np.int32)
        self.table = np.full((B, per), -7, np.int32)
        at = 0
        for b in range(B):
            self.table[b, :n[b]] = perm[at:at + n[b]]
            at += n[b]
        self.new_table = None
        if copy:
            self.new_table = np.full((B, new_per), -9, np.int32)
            for b in range(B):
                m = -(-int(hold[b]) // page)
                self.new_table[b, :m] = perm[at:at + m]
                at += m
                same = int(s[b]) // page          # pages before the first key that may go
                self.new_table[b, :same] = self.table[b, :same]
        self.k, self.v = (torch.from_numpy(rng.normal(size=(pages, Hkv, page, D))).to(torch.bfloat16)
                          for _ in (0, 1))
        self.max_freed = int(n.sum()) + 2

    def sequence_starts(self):
        s = np.full(len(self.lens), self.sink) if self.starts is None else self.starts
        return np.clip(s, 0, np.maximum(self.lens, 0))

    def run(self, in_place_weights=False, **extra):
        import masked_attention_gb300 as M
        B, Hkv, L = self.weights.shape
        i32 = torch.int32
        out = {"kept": guarded_empty((B, Hkv, self.keep), i32), "new_lens": guarded_empty((B,), i32),
               "freed": guarded_empty((self.max_freed,), i32), "info": guarded_empty((2,), i32),
               "k": guarded_empty(self.k.shape, torch.bfloat16),
               "v": guarded_empty(self.v.shape, torch.bfloat16),
               "weights_out": guarded_empty((B, Hkv, L), torch.float32)}
        out["freed"].fill_(-3)
        out["k"].copy_(self.k)
        out["v"].copy_(self.v)
        out["weights_out"].fill_(7.0)
        w = torch.from_numpy(self.weights).cuda()
        if in_place_weights:
            w = out["weights_out"].copy_(w)
        M.attn_cache_evict(w, torch.from_numpy(self.lens).cuda(), out["k"], out["v"],
                           torch.from_numpy(self.table).cuda(), out["weights_out"], out["kept"],
                           out["new_lens"], out["freed"], out["info"], page_size=self.page,
                           recent=self.recent, sink=self.sink,
                           starts=None if self.starts is None else torch.from_numpy(self.starts).cuda(),
                           new_table=None if self.new_table is None
                           else torch.from_numpy(self.new_table).cuda(), **extra)
        check_canaries()
        return out

    def check(self, in_place_weights=False):
        out = self.run(in_place_weights)
        before = self.weights if in_place_weights else np.full(self.weights.shape, 7, np.float32)
        bits = [t.view(torch.int16).numpy() for t in (self.k, self.v)]
        s = (np.full(len(self.lens), self.sink) if self.starts is None else self.starts)
        ref = evict(self.weights, self.lens, s, self.keep, self.recent, *bits, self.table, self.page,
                    self.new_table, before, np.full(self.max_freed, -3, np.int32))
        for name, r in zip(NAMES, ref):
            got = out[name].cpu()
            got = got.view(torch.int16) if name in "kv" else got
            got = got.numpy()
            if got.dtype == np.float32:
                got, r = got.view(np.int32), r.astype(np.float32).view(np.int32)
            assert np.array_equal(got, r), (name, np.argwhere(got != r)[:5])
        return out


@pytest.mark.gpu
@pytest.mark.parametrize("copy", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("keep,recent,sink", [(1, 0, 0), (1, 1, 0), (40, 8, 4), (100, 100, 0),
                                              (64, 0, 40), (127, 1, 130)])
def test_lengths_pages_and_budgets(keep, recent, sink, page, D, copy):
    Case([0, 1, keep + sink, keep + sink + 1, 300, 129, 5], keep, recent, sink, D=D, page=page,
         copy=copy).check()


@pytest.mark.gpu
@pytest.mark.parametrize("copy", [False, True])
@pytest.mark.parametrize("kind", ["zeros", "equal", "signed", "few", "close"])
def test_weights_that_tie(kind, copy):
    for seed in range(3):
        Case([400, 77, 1030], 50, 7, 3, kind=kind, seed=seed, copy=copy).check()


@pytest.mark.gpu
@pytest.mark.parametrize("copy", [False, True])
def test_infinities_nan_and_signed_zeros(copy):
    c = Case([200, 90], 20, 4, 2, copy=copy)
    c.weights[0, 0, 10:40:3] = np.inf
    c.weights[0, 1, 5:60:7] = np.nan
    c.weights[0, 1, 6] = np.inf
    c.weights[0, 1, 9] = -np.nan
    c.weights[1, 0] = np.where(np.arange(c.L) % 2, 0.0, -0.0)
    c.weights[1, 1] = -np.inf
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("copy", [False, True])
def test_starts_of_their_own(copy):
    c = Case([200, 150, 90, 64, 0, 30], 30, 5, starts=[100, 0, 200, -4, 9, 16], page=16, copy=copy)
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("seed", [0, 1])
@pytest.mark.parametrize("lens,keep,recent,Hkv", [([5000, 3000], 2500, 100, 2), ([9000], 8999, 0, 1),
                                                  ([3000] * 9, 700, 64, 4), ([4100], 1, 0, 3)])
def test_many_batches_in_place(lens, keep, recent, Hkv, seed):
    """Rows that move by one place and by thousands; weights in place and apart."""
    c = Case(lens, keep, recent, 4, Hkv=Hkv, seed=seed)
    c.check(in_place_weights=seed == 0)
    c = Case(lens, keep, recent, 4, Hkv=Hkv, seed=seed, copy=True, D=128)
    c.check(in_place_weights=seed == 1)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["spread", "equal"])
def test_more_weights_than_are_staged(kind):
    c = Case([70000, 49153, 20], 33333 if kind == "spread" else 300, 17, 1, Hkv=1, kind=kind, seed=4)
    c.check(in_place_weights=True)


@pytest.mark.gpu
def test_bad_pages_and_lengths():
    """Pages outside the pool read as zeros and are not written; lengths are cut to the bounds."""
    for copy in (False, True):
        c = Case([100, 60, 80], 30, 3, 2, copy=copy, L=100)
        c.table[0, 5], c.table[1, 0], c.table[2, 1] = len(c.k), -1, 2 ** 31 - 1
        if copy:
            c.new_table[0, 1] = -1
            c.new_table[2, 0] = 2 ** 30
        c.check()
        c.lens[:] = [-5, 10 ** 9, 80]
        c.check()


@pytest.mark.gpu
def test_rows_past_the_new_table_and_a_short_list():
    c = Case([100, 60], 50, 3, 2, copy=True)
    c.new_table = np.ascontiguousarray(c.new_table[:, :2])
    c.max_freed = 4
    c.check()
    c.max_freed = 0
    c.check()


@pytest.mark.gpu
def test_shared_first_pages_stay():
    """Two sequences hold the same first pages: with those before `starts` neither moves them."""
    c = Case([120, 140], 40, 8, starts=[32, 32], page=16)
    c.table[1, :2] = c.table[0, :2]
    c.check()


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """A pool of more than 4 GiB whose pages lie at its end."""
    import masked_attention_gb300 as M
    c = Case([700], 300, 10, 4, Hkv=2, D=128, page=128)
    ref = c.run()
    pages = (1 << 32) // (2 * 2 * 128 * 128) + len(c.k)
    pools = [torch.zeros(pages, 2, 128, 128, dtype=torch.bfloat16, device="cuda") for _ in (0, 1)]
    for pool, x in zip(pools, (c.k, c.v)):
        pool[-len(c.k):] = x.cuda()
    table = torch.from_numpy(np.where(c.table >= 0, c.table + pages - len(c.k), -1).astype(np.int32))
    out = {n: torch.empty_like(ref[n]) for n in ("weights_out", "kept", "new_lens", "freed", "info")}
    M.attn_cache_evict(torch.from_numpy(c.weights).cuda(), torch.from_numpy(c.lens).cuda(), *pools,
                       table.cuda(), *out.values(), page_size=128, recent=10, sink=4)
    assert torch.equal(out["kept"], ref["kept"])
    for pool, name in zip(pools, "kv"):
        assert torch.equal(pool[-len(c.k):], ref[name]) and not pool[:-len(c.k)].any()


@pytest.mark.gpu
def test_captured_and_on_another_stream():
    import masked_attention_gb300 as M
    c = Case([900, 40, 700], 200, 20, 4, page=32, copy=True)
    ref = c.run()
    t = {n: torch.from_numpy(getattr(c, n)).cuda() for n in ("weights", "lens", "table", "new_table")}
    k, v = c.k.cuda(), c.v.cuda()
    out = {n: torch.zeros_like(ref[n]) for n in ("weights_out", "kept", "new_lens", "freed", "info")}

    def call():
        M.attn_cache_evict(t["weights"], t["lens"], k, v, t["table"], *out.values(), page_size=32,
                           recent=20, sink=4, new_table=t["new_table"])

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(2):
        k.copy_(c.k)
        v.copy_(c.v)
        out["weights_out"].fill_(7.0)
        out["freed"].fill_(-3)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n in out:
            assert torch.equal(out[n], ref[n]), n
        assert torch.equal(k, ref["k"]) and torch.equal(v, ref["v"])
    side = torch.cuda.Stream()
    k.copy_(c.k)
    v.copy_(c.v)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    assert torch.equal(k, ref["k"]) and torch.equal(out["kept"], ref["kept"])


def test_oracle_by_hand():
    w = np.array([[[9, 1, 5, 5, 0, 7, 5, 3]]], np.float32)
    k = np.arange(32).reshape(2, 1, 16, 1).astype(np.int16)
    out, kept, lens, freed, info, k2, _ = evict(w, [8], [1], 4, 1, k, k, np.array([[1]]), 16, None,
                                                w, np.full(3, -1, np.int32))
    assert kept.tolist() == [[[2, 3, 5, 7]]] and lens.tolist() == [5] and info.tolist() == [0, 1]
    assert out.tolist() == [[[9, 5, 5, 7, 3, 0, 0, 0]]]
    assert k2[1, 0, :5, 0].tolist() == [16, 18, 19, 21, 23]
    _, _, _, freed, info, k3, _ = evict(w, [8], [1], 4, 1, k, k, np.array([[1]]), 16,
                                        np.array([[0]]), w, np.full(3, -1, np.int32))
    assert freed.tolist() == [1, -1, -1] and k3[0, 0, :5, 0].tolist() == [16, 18, 19, 21, 23]
    assert np.array_equal(k3[1], k[1])


def test_refusals():
    import masked_attention_gb300 as M
    L = M.lib()

    def call(B=2, Hkv=2, max_len=100, D=64, stride=100, sink=4, keep=50, recent=8, w=0x100000,
             wo=0x200000, lens=0x10000, starts=None, k=0x1000000, v=0x2000000, pages=40, ps=16,
             table=0x20000, per=7, new=None, new_per=0, kept=0x30000, nl=0x40000, freed=0x50000,
             n=20, info=0x60000):
        return L.attn_cache_evict(w, wo, stride, lens, starts, sink, keep, recent, k, v, pages, ps,
                                  table, per, new, new_per, B, Hkv, max_len, D, kept, nl, freed, n,
                                  info, None)

    inv, uns, mis = M.ATTN_ERR_INVALID_ARG, M.ATTN_ERR_UNSUPPORTED, M.ATTN_ERR_MISALIGNED
    assert call(B=-1) == call(Hkv=0) == call(max_len=-1) == call(sink=-1) == call(keep=0) == inv
    assert call(recent=-1) == call(recent=51) == call(stride=99) == call(pages=0) == inv
    assert call(per=0) == call(per=6) == call(n=-1) == call(new=0x70000) == inv
    assert call(D=96) == call(ps=48) == call(B=20000) == call(B=9000, Hkv=8) == uns
    assert call(keep=2 ** 31 - 1) == uns
    for name in ("w", "wo", "lens", "k", "v", "table", "kept", "nl", "freed", "info"):
        assert call(**{name: None}) == inv, name
    assert call(freed=None, n=0, B=0) == M.ATTN_OK
    assert call(k=0x1000008) == call(v=0x2000008) == mis
    for name in ("w", "wo", "lens", "table", "kept", "nl", "freed", "info", "starts", "new"):
        assert call(**{name: 0x70002, "new_per": 4}) == mis, name
    # what is written overlaps nothing else; the weights may stay in place
    assert call(wo=0x100004) == call(wo=0x100000 - 4 * 399) == inv
    assert call(kept=0x20000) == call(nl=0x10004) == call(info=0x50000 + 76) == inv
    assert call(v=0x1000000) == call(v=0x1000000 + 40 * 2 * 16 * 128 - 16) == inv
    assert call(starts=0x40004) == call(new=0x30000, new_per=3) == call(wo=0x1000000) == inv
    t = torch.zeros(1, 1, 4)
    with pytest.raises(ValueError):
        M.attn_cache_evict(t, t, t, t, t, t, t, t, t, t, page_size=16, recent=0)


def test_refuses_more_rows_than_are_counted():
    """Pool rows are numbered in 32 bits; empty batches show the check alone."""
    import masked_attention_gb300 as M

    def call(pages, Hkv=2, ps=128):
        return M.lib().attn_cache_evict(None, None, 100, None, None, 4, 50, 8, None, None, pages, ps,
                                        None, 7, None, 0, 0, Hkv, 100, 64, None, None, None, 0, None,
                                        None)

    assert call(2 ** 24 - 1) == M.ATTN_OK                      # 2^32 - 256 rows
    assert call(2 ** 24) == call(2 ** 31 - 1) == M.ATTN_ERR_UNSUPPORTED
    assert call(2 ** 27 - 1, 2, 16) == M.ATTN_OK and call(2 ** 27, 2, 16) == M.ATTN_ERR_UNSUPPORTED


@pytest.mark.gpu
@pytest.mark.parametrize("copy", [False, True])
@pytest.mark.parametrize("Hkv,D", [(1, 64), (3, 128), (40, 64)])
def test_blocks_that_share_a_pair(Hkv, D, copy):
    """From one pair, whose keys several blocks select from and move, to 120; a sequence that is cut
    beside one that is not, and slices of unlike lengths."""
    c = Case([17001, 30, 8193], 4097, 33, 5, Hkv=Hkv, D=D, page=32, copy=copy, seed=Hkv)
    c.check(in_place_weights=not copy)
    c = Case([20011], 6000, 6000, 0, Hkv=Hkv, D=D, kind="few", copy=copy, seed=Hkv)
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("copy", [False, True])
def test_most_sequences(copy):
    """As many sequences as a call takes."""
    lens = np.random.default_rng(5).integers(0, 40, 16384)
    Case(lens.tolist(), 12, 3, 2, Hkv=1, copy=copy, kind="few").check()


def pages_of(c, b, n):
    """Entries of sequence b's table row that hold its first n keys."""
    return -(-n // c.page)


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 64, 128])
def test_pages_that_the_new_table_keeps_are_not_freed(page):
    """A sequence that is not cut and keeps its pages, one whose first held keys stay where they
    are, and one whose new table names an old page that it no longer reaches."""
    c = Case([300, 1000, 900, 0, 700], 500, 40, 3, page=page, copy=True, seed=11)
    c.weights[1] = c.weights[2] = c.weights[4] = -np.arange(c.L)  # the first keys are the heaviest
    # 0: not cut, every page is kept. 1: pages of the keys that stay in front are kept
    c.new_table[0, :pages_of(c, 0, 300)] = c.table[0, :pages_of(c, 0, 300)]
    same = (3 + 500 - 40) // page
    c.new_table[1, :same] = c.table[1, :same]
    # 2: names the page behind the last one that its 503 keys reach
    at = pages_of(c, 2, 503)
    c.new_table[2, at] = c.table[2, at]
    out = c.check()
    gone = set(out["freed"].cpu().tolist()[:int(out["info"][0])])
    assert not gone & set(c.table[0, :pages_of(c, 0, 300)].tolist() + c.table[1, :same].tolist())
    assert c.table[2, at] in gone and set(c.table[4, :pages_of(c, 4, 700)].tolist()) <= gone
    c.check(in_place_weights=True)
    # all of it in a short list, and a new table that ends before its sequences do
    c.max_freed = 7
    c.check()
    c.new_table = np.ascontiguousarray(c.new_table[:, :2])
    c.check()


@pytest.mark.gpu
def test_old_table_as_the_new_one():
    """Nothing is cut and both tables are equal: nothing moves, nothing is freed, also where
    entries name no page."""
    c = Case([100, 31, 0, 64], 200, 10, 2, copy=True)
    c.new_table = c.table.copy()
    c.new_table[0, 3] = c.table[0, 3] = -1
    out = c.check()
    assert out["info"].tolist() == [0, 0] and (out["freed"] == -3).all()
    assert torch.equal(out["k"].cpu(), c.k) and torch.equal(out["v"].cpu(), c.v)


@pytest.mark.gpu
def test_kept_pages_of_many_sequences():
    """More sequences than threads: some keep all, some a part, some no page."""
    rng = np.random.default_rng(12)
    c = Case(rng.integers(0, 150, 1500).tolist(), 60, 9, 20, Hkv=1, copy=True, kind="few", seed=12)
    c.weights[:] = -np.arange(c.L)
    for b, n in enumerate(c.lens.tolist()):
        held = min(n, 20 + 60)
        stay = pages_of(c, b, n) if n <= 80 else (20 + 60 - 9) // 16
        same = int(rng.integers(0, stay + 1)) if b % 3 else stay
        c.new_table[b, :same] = c.table[b, :same]
        assert pages_of(c, b, held) <= c.new_table.shape[1]
    out = c.check()
    assert 0 < int(out["info"][0]) < int((-(-c.lens // 16)).sum())


def test_oracle_keeps_pages_that_the_new_table_names():
    w = np.arange(48, 0, -1, dtype=np.float32).reshape(1, 1, 48)
    k = np.arange(6 * 16).reshape(6, 1, 16, 1).astype(np.int16)
    args = w, [40], [0], 20, 2, k, k, np.array([[1, 2, 3]]), 16
    free = np.full(4, -1, np.int32)
    # the first page stays: keys 0 to 15 are held and do not move
    _, _, lens, freed, info, k2, _ = evict(*args, np.array([[1, 4]]), w, free)
    assert lens.tolist() == [20] and freed.tolist() == [2, 3, -1, -1] and info.tolist() == [2, 1]
    assert k2[4, 0, :4, 0].tolist() == [32, 33, 54, 55] and np.array_equal(k2[1], k[1])
    # an old page behind the last one in use is freed wherever it is named
    _, _, _, freed, info, _, _ = evict(*args, np.array([[4, 5, 3]]), w, free)
    assert freed.tolist() == [1, 2, 3, -1] and info.tolist() == [3, 1]
