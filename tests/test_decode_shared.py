"""attn_decode_shared against the fp64 oracle, which attends sequence by sequence.

Tolerances. A score's exponent is off by E = 2^-17 of what it is made of (sum|q k| scale and the
distance term; five times that with a soft-cap), as derived in tests/test_key_weights.py. The LSE
is then within E + 2^-20 (1 + |LSE|): logarithm, joins of parts, fp32 sums. A probability
carries a factor e^(+-2E), the sum's rounding (2^-18 covers it for these lengths and the joins)
and its own rounding to bf16, 2^-8; O sums p v, so it is within (2^-8 + 2^-18 + 4 E) sum p |v|,
and rounds once itself, 2^-8 |O|."""
import ctypes

import numpy as np
import pytest
import torch

from oracle.long_context import cached_rows, decode_rows, slopes
from tests.helpers import check_canaries, guarded_empty


class Case:
    """groups: (number of sequences, shared keys); own: keys of each sequence behind those."""

    def __init__(self, groups, own, Hq=4, Hkv=2, Sq=1, D=64, page=16, seed=0, window=0, softcap=0.0,
                 alibi=False, causal=True, scale=0.0, qscale=1.0, spare=0):
        g = torch.Generator().manual_seed(seed)
        B = sum(n for n, _ in groups)
        assert len(own) == B
        self.shape, self.page, self.alibi, self.causal = (B, Hq, Hkv, Sq, D), page, alibi, causal
        self.kw = dict(window=window, softcap=softcap, scale=scale)
        self.shared = torch.tensor([s for _, s in groups], dtype=torch.int32)
        self.starts = torch.tensor(np.cumsum([0] + [n for n, _ in groups]), dtype=torch.int32)
        self.group = np.repeat(np.arange(len(groups)), [n for n, _ in groups])
        # own < 0: the sequence ends that many keys before its group's shared ones do
        self.lens = torch.tensor([max(0, int(self.shared[self.group[b]]) + own[b])
                                  for b in range(B)], dtype=torch.int32)
        per = -(-int(max(int(self.lens.max()), int(self.shared.max()), 1)) // page) + spare
        self.table = torch.full((B, per), -1, dtype=torch.int32)
        ids = iter(torch.randperm(B * per + 3, generator=g).tolist())
        for b in range(B):
            first = int(self.starts[self.group[b]])
            # pages that the sequence shares hold whole or begun shared runs
            same = -(-int(self.shared[self.group[b]]) // page)
            for l in range(-(-max(int(self.lens[b]), int(self.shared[self.group[b]])) // page)):
                take = b != first and (l < same - 1 or (l < same and self.whole(b)))
                self.table[b, l] = self.table[first, l] if take else next(ids)
        pages = B * per + 3
        self.q = (torch.randn(B, Hq, Sq, D, generator=g) * qscale).to(torch.bfloat16)
        self.k, self.v = (torch.randn(pages, Hkv, page, D, generator=g).to(torch.bfloat16)
                          for _ in (0, 1))
        self.share_begun_pages()

    def share_begun_pages(self):
        """The rows of a page that is begun shared, equal in every sequence's copy of it."""
        for b, g in enumerate(self.group):
            s, first = int(self.shared[g]), int(self.starts[g])
            if s % self.page and b != first:
                for pool in (self.k, self.v):
                    pool[int(self.table[b, s // self.page]), :, :s % self.page] = \
                        pool[int(self.table[first, s // self.page]), :, :s % self.page]

    def whole(self, b):
        return int(self.shared[self.group[b]]) % self.page == 0

    def rows(self, b, h):
        B, Hq, Hkv, Sq, D = self.shape
        return tuple(cached_rows(x, self.table.numpy(), b, int(self.lens[b]), h * Hkv // Hq, self.page)
                     for x in (self.k64, self.v64))

    def variant(self):
        import masked_attention_gb300 as M
        return ((M.MASK_CAUSAL if self.causal else 0) | (M.MASK_WINDOW if self.kw["window"] else 0)
                | (M.SCORE_SOFTCAP if self.kw["softcap"] else 0)
                | (M.SCORE_ALIBI if self.alibi else 0))

    def run(self, **extra):
        import masked_attention_gb300 as M
        B, Hq, Hkv, Sq, D = self.shape
        o = guarded_empty((B, Hq, Sq, D), torch.bfloat16)
        lse = guarded_empty((B, Hq, Sq), torch.float32)
        ws = guarded_empty((M.attn_decode_shared_workspace_bytes(
            B, Hq, Hkv, Sq, len(self.shared), self.table.shape[1] * self.page, D),), torch.uint8)
        ws.fill_(0xff)                         # its contents need not be kept
        kw = dict(self.kw, page_table=self.table.cuda(), page_size=self.page, workspace=ws,
                  seq_lens=self.lens.cuda(), group_starts=self.starts.cuda(),
                  shared_lens=self.shared.cuda())
        M.attn_decode_shared(self.q.cuda(), self.k.cuda(), self.v.cuda(), o, lse, self.variant(),
                             **{**kw, **extra})
        assert M.attn_check_status() == M.ATTN_OK
        check_canaries()
        return o, lse

    def check(self, **extra):
        B, Hq, Hkv, Sq, D = self.shape
        o, lse = (t.double().cpu().numpy() for t in self.run(**extra))
        self.k64, self.v64 = self.k.double().numpy(), self.v.double().numpy()
        kw = {k: v for k, v in self.kw.items() if k != "scale"}
        O, L, A, size = decode_rows(self.q.double().numpy(), self.rows, self.lens, causal=self.causal,
                                    alibi=slopes(Hq) if self.alibi else None,
                                    scale=self.kw["scale"] or None, **kw)
        none = np.isneginf(L)
        assert np.array_equal(np.isneginf(lse), none) and (o[none] == 0).all()
        E = 2.0 ** -17 * size
        with np.errstate(invalid="ignore"):
            bad = ~none & ~(np.abs(lse - L) <= E + 2.0 ** -20 * (1 + np.abs(L)))
        assert not bad.any(), (np.argwhere(bad)[:4], lse[bad][:4], L[bad][:4])
        tol = 2.0 ** -8 * np.abs(O) + (2.0 ** -8 + 2.0 ** -18 + 4 * E[..., None]) * A
        bad = ~(np.abs(o - O) <= tol)
        assert not bad.any(), (np.argwhere(bad)[:4], o[bad][:4], O[bad][:4], tol[bad][:4])
        return o, lse


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("Hq,Hkv,Sq", [(1, 1, 1), (4, 2, 1), (14, 2, 2), (8, 8, 2), (16, 1, 1),
                                       (5, 1, 3)])
def test_pages_heads_and_rows(Hq, Hkv, Sq, page, D):
    Case([(3, 256), (1, 200), (5, 128), (2, 0)], [1, 17, 300, 5, 60, 128, 129, 1, 127, 40, 0],
         Hq, Hkv, Sq, D, page).check()


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,Sq,n", [(4, 1, 1, 33), (16, 2, 2, 20), (3, 1, 3, 40), (2, 2, 1, 300),
                                         (6, 1, 2, 11)])
def test_more_rows_than_a_block(Hq, Hkv, Sq, n, D):
    """Several row blocks of a group, and chunks of its keys side by side."""
    own = [(7 * b) % 50 + 1 for b in range(n)]
    Case([(n, 700)], own, Hq, Hkv, Sq, D, 32, seed=1).check()
    Case([(1, 100), (n, 1333), (2, 500)], [9] + own + [3, 300], Hq, Hkv, Sq, D, 64, seed=2).check()


@pytest.mark.gpu
def test_lengths_of_all_kinds():
    """Sequences that end inside the shared keys, empty ones, groups of one, of none, and shared
    lengths around the tile and page sizes."""
    for s in (127, 128, 129, 130, 143, 255, 256, 257, 400):
        Case([(3, s), (2, 0), (1, 300)], [1, -s, 40, 0, 1, 3], seed=s).check()
        Case([(4, s)], [-1, -100, 2, -s + 1], page=32, seed=s, Sq=2).check()
    Case([(1, 0)], [1]).check()
    Case([(1, 0)], [0]).check()
    Case([(2, 300)], [-300, -300]).check()


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kw", [dict(alibi=True), dict(softcap=20.0), dict(softcap=2.0, alibi=True),
                                dict(window=1), dict(window=50), dict(window=129, softcap=30.0),
                                dict(window=300, alibi=True, Sq=3), dict(causal=False, Sq=3),
                                dict(causal=False, window=40, Sq=2), dict(scale=0.3),
                                dict(softcap=1e6, Sq=2), dict(qscale=12.0, softcap=50.0),
                                dict(qscale=30.0), dict(window=900, Sq=4)])
def test_variants(kw, D):
    Case([(5, 640), (3, 200), (1, 0)], [5, 300, -20, 1, 64, 90, 0, 700, 33], D=D, seed=3, **kw).check()


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_references_that_move(D):
    """Scores that grow, fall and jump along the keys: the reference moves late, early, often."""
    for shape in ("up", "down", "jump"):
        c = Case([(4, 1000)], [3, 200, 90, 1], D=D, page=64, seed=4)
        for b in range(4):
            for l in range(c.table.shape[1]):
                if c.table[b, l] < 0:
                    continue
                f = {"up": l / 4, "down": (20 - l) / 4, "jump": 6.0 * (l % 5 == 2)}[shape]
                c.k[int(c.table[b, l])] = (torch.randn(c.k.shape[1:], generator=torch.Generator().
                                           manual_seed(int(c.table[b, l]))) + f).to(torch.bfloat16)
        c.share_begun_pages()   # each sequence's copy of the last shared page was filled apart
        c.q = c.q.abs()
        c.check()


@pytest.mark.gpu
def test_no_groups_is_a_ragged_decode():
    c = Case([(1, 0)] * 5, [1, 700, 0, 129, 64], Sq=2, D=128)
    c.check()
    a = c.run()
    b = c.run(group_starts=None, shared_lens=None)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.gpu
def test_sharing_does_not_change_the_result():
    """The same attention with and without the groups, within both sides' bounds."""
    c = Case([(7, 900), (30, 300)], [5 + b for b in range(37)], Hq=8, Hkv=2, D=128, page=64)
    a, la = c.check()
    c.shared[:] = 0
    b, lb = c.check()
    with np.errstate(invalid="ignore"):
        assert np.abs(la - lb).max() < 1e-4
    assert np.abs(a - b).max() < 2.0 ** -6 * np.abs(a).max()


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(), dict(window=40), dict(Sq=3)])
def test_what_no_row_sees_changes_nothing(kw):
    """NaN and infinities behind the sequences' ends, before the window, in other pages."""
    c = Case([(3, 200), (2, 0)], [30, 100, -60, 70, 5], page=32, seed=5, **kw)
    a, la = c.check()
    B, Hq, Hkv, Sq, D = c.shape
    seen = set()
    for b in range(B):
        n = int(c.lens[b])
        low = max(0, n - Sq - c.kw["window"] + 1) if c.kw["window"] else 0
        seen |= {(int(c.table[b, j // 32]), j % 32) for j in range(low, n)}
    g = int(c.shared[0])
    low = min(max(0, int(n) - Sq - c.kw["window"] + 1) if c.kw["window"] else 0 for n in c.lens[:3])
    for l in range(low, g):                    # keys that some row of the group sees stay finite
        seen.add((int(c.table[0, l // 32]), l % 32))
    for at in range(len(c.k)):
        for r in range(32):
            if (at, r) not in seen:
                c.k[at, :, r] = float("nan") if r % 2 else float("inf")
                c.v[at, :, r] = float("inf") if r % 3 else float("nan")
    o, lse = c.run()
    assert np.array_equal(o.double().cpu().numpy(), a)
    assert np.array_equal(lse.double().cpu().numpy(), la)


@pytest.mark.gpu
def test_nan_of_a_visible_key_shows():
    c = Case([(3, 256)], [10, 20, 30])
    c.k[int(c.table[1, 16]), 1, 2] = float("nan")        # a key of sequence 1, head pair 1
    o, lse = c.run()
    hit = torch.isnan(lse.cpu())
    assert hit[1, 2:].all() and int(hit.sum()) == 2 and torch.isnan(o.cpu())[hit].all()
    c = Case([(3, 256)], [10, 20, 30])
    c.v[int(c.table[0, 3]), 0, 5, 7] = float("nan")      # a shared value channel: all sequences
    o, lse = c.run()
    bad = torch.isnan(o.cpu())
    assert bad[:, :2, :, 7].all() and int(bad.sum()) == 6 and not torch.isnan(lse.cpu()).any()


@pytest.mark.gpu
def test_bad_pages_lengths_and_groups():
    c = Case([(3, 200), (2, 300)], [30, 100, 7, 70, 5], page=32, spare=1)
    for b in range(3):
        c.table[b, 2] = -3                               # the group's third page: zeros
    c.table[1, 8], c.table[3, 10] = len(c.k), 2 ** 31 - 1
    c.check()
    c = Case([(3, 200), (2, 300)], [30, 100, 7, 70, 5], page=32)
    ref = c.run()
    for starts in ([0, 3, 5], [-7, 3, 99]):
        o, lse = c.run(group_starts=torch.tensor(starts, dtype=torch.int32).cuda())
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])
    # entries that fall back and shared lengths outside [0, len]: bounded by the lengths
    for starts, shared in (([3, 0, 5], [200, 300]), ([0, 0, 0], [1, 2]), ([0, 2, 1], [10 ** 9, -4])):
        c.check(group_starts=torch.tensor(starts, dtype=torch.int32).cuda(),
                shared_lens=torch.tensor([s if g else 0 for g, s in enumerate(shared)],
                                         dtype=torch.int32).cuda())
    far = c.lens.clone()
    far[1], far[4] = -9, 10 ** 9
    bound = c.table.shape[1] * 32
    c.lens[1], c.lens[4] = 0, bound
    c.shared[:] = 0
    c.table[4] = torch.where(c.table[4] < 0, 1, c.table[4])
    c.check(seq_lens=far.cuda())


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Pools of more than 4 GiB whose pages lie at their ends."""
    import masked_attention_gb300 as M
    c = Case([(3, 256)], [90, 33, 5], Hkv=2, D=128, page=128)
    o, lse = c.run()
    pages = (1 << 32) // (2 * 2 * 128 * 128) + len(c.k)
    pools = [torch.empty(pages, 2, 128, 128, dtype=torch.bfloat16, device="cuda") for _ in (0, 1)]
    for pool, x in zip(pools, (c.k, c.v)):
        pool[-len(c.k):] = x.cuda()
    table = torch.where(c.table >= 0, c.table + pages - len(c.k), -1).to(torch.int32).cuda()
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    ws = torch.empty(M.attn_decode_shared_workspace_bytes(3, 4, 2, 1, 1, table.shape[1] * 128, 128),
                     dtype=torch.uint8, device="cuda")
    M.attn_decode_shared(c.q.cuda(), *pools, o2, lse2, c.variant(), page_table=table, page_size=128,
                         seq_lens=c.lens.cuda(), group_starts=c.starts.cuda(),
                         shared_lens=c.shared.cuda(), workspace=ws)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("Hq,Hkv,Sq", [(1, 1, 1), (14, 2, 2), (16, 1, 1), (5, 1, 3)])
def test_long_shared_runs(Hq, Hkv, Sq, page, D):
    """Runs long enough to be read once, beside one that each sequence reads itself."""
    Case([(3, 640), (2, 512), (2, 200), (3, 1100)], [1, 17, 300, 5, 60, 128, 129, 1, 127, -50],
         Hq, Hkv, Sq, D, page, seed=6).check()


@pytest.mark.gpu
def test_ends_of_long_shared_runs():
    """Shared lengths around the tile and page sizes and around what is read once; sequences that
    end inside the shared keys, and empty ones."""
    for s in (511, 512, 513, 527, 528, 575, 576, 577, 639, 641):
        Case([(3, s), (2, 0), (1, 300)], [1, -s, 40, 0, 1, 3], seed=s).check()
        Case([(4, s)], [-1, -100, 2, -s + 1], page=32, seed=s, Sq=2).check()
    Case([(2, 600)], [-600, -600]).check()       # nobody is there
    Case([(3, 600)], [-100, -90, -520]).check()  # the longest ends at 510: below what is read once


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(), dict(window=40), dict(window=400), dict(Sq=3),
                                dict(softcap=20.0)])
def test_what_no_row_sees_changes_nothing_behind_a_long_run(kw):
    """NaN and infinities behind the sequences' ends, before the window, in other pages."""
    c = Case([(3, 600), (2, 0)], [30, 100, -60, 70, 5], page=32, seed=5, **kw)
    a, la = c.check()
    Sq, window = c.shape[3], c.kw["window"]
    low = [max(0, int(n) - Sq - window + 1) if window else 0 for n in c.lens]
    seen = {(int(c.table[b, j // 32]), j % 32) for b in range(5) for j in range(low[b], int(c.lens[b]))}
    # keys that some row of the group sees stay finite
    seen |= {(int(c.table[0, j // 32]), j % 32) for j in range(min(low[:3]), 600)}
    for at in range(len(c.k)):
        for r in range(32):
            if (at, r) not in seen:
                c.k[at, :, r] = float("nan") if r % 2 else float("inf")
                c.v[at, :, r] = float("inf") if r % 3 else float("nan")
    o, lse = c.run()
    assert np.array_equal(o.double().cpu().numpy(), a)
    assert np.array_equal(lse.double().cpu().numpy(), la)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 128])
@pytest.mark.parametrize("groups,own,kw", [
    ([(3, 600), (2, 0)], [30, 100, -60, 70, 5], dict(window=40)),
    ([(3, 600)], [30, 100, -60], dict(window=40, Sq=3, causal=False)),
    # holes of whole tiles, one of them from a tile's start; a sequence that is empty
    ([(4, 1216)], [-576, 5, -100, -1216], dict(window=64)),
    ([(4, 1216)], [-577, 40, -130, -300], dict(window=1, softcap=20.0)),
    # several row blocks: what one of them sees the other does not
    ([(1, 100), (21, 900)], [9] + [-40 * b for b in range(21)], dict(window=7, Hq=16, Hkv=1)),
    ([(40, 700)], [3 * b - 90 for b in range(40)], dict(window=2, Hq=8, Hkv=2, alibi=True)),
    # the sequences of each row block see one run, the blocks' runs lie apart
    ([(16, 900)], [-400 - b for b in range(8)] + [5 - 5 * b for b in range(8)],
     dict(window=40, Hq=16, Hkv=1)),
])
def test_shared_keys_between_the_windows_change_nothing(groups, own, kw, page, D):
    """Sequences of a group that end apart, each with a window: NaN and infinities in every key
    that none of them sees, between their windows too."""
    c = Case(groups, own, page=page, D=D, seed=7, **kw)
    a, la = c.check()
    Sq, window = c.shape[3], c.kw["window"]
    seen = set()
    for b, n in enumerate(c.lens.tolist()):
        g = int(c.group[b])
        for j in range(max(0, n - Sq - window + 1), n):
            # a shared key is read from the first sequence's pages
            of = {b, int(c.starts[g])} if j < int(c.shared[g]) else {b}
            seen |= {(int(c.table[x, j // page]), j % page) for x in of}
    for at in range(len(c.k)):
        for r in range(page):
            if (at, r) not in seen:
                c.k[at, :, r] = float("nan") if r % 2 else float("inf")
                c.v[at, :, r] = float("inf") if r % 3 else float("nan")
    o, lse = c.run()
    assert np.array_equal(o.double().cpu().numpy(), a)
    assert np.array_equal(lse.double().cpu().numpy(), la)


@pytest.mark.gpu
def test_nan_of_a_key_that_is_read_once_shows():
    c = Case([(3, 576)], [10, 20, 30])
    c.k[int(c.table[0, 3]), 1, 2] = float("nan")         # a shared key of head pair 1
    o, lse = c.run()
    assert torch.isnan(lse.cpu())[:, 2:].all() and not torch.isnan(lse.cpu())[:, :2].any()
    assert torch.isnan(o.cpu())[:, 2:].all() and not torch.isnan(o.cpu())[:, :2].any()
    c = Case([(3, 576)], [10, 20, 30])
    c.v[int(c.table[0, 3]), 0, 5, 7] = float("nan")      # a shared value channel
    o, lse = c.run()
    bad = torch.isnan(o.cpu())
    assert bad[:, :2, :, 7].all() and int(bad.sum()) == 6 and not torch.isnan(lse.cpu()).any()


@pytest.mark.gpu
def test_bad_pages_and_groups_of_long_runs():
    c = Case([(3, 600), (2, 700)], [30, 100, 7, 70, 5], page=32, spare=1)
    for b in range(3):
        c.table[b, 2] = -3                               # the group's third page: zeros
    c.table[1, 20], c.table[3, 23] = len(c.k), 2 ** 31 - 1
    c.check()
    c = Case([(3, 600), (2, 700)], [30, 100, 7, 70, 5], page=32)
    ref = c.run()
    o, lse = c.run(group_starts=torch.tensor([-7, 3, 99], dtype=torch.int32).cuda())
    assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])
    for starts, shared in (([3, 0, 5], [0, 700]), ([0, 0, 0], [600, 600]), ([0, 3, 1], [600, 9])):
        c.check(group_starts=torch.tensor(starts, dtype=torch.int32).cuda(),
                shared_lens=torch.tensor(shared, dtype=torch.int32).cuda())


@pytest.mark.gpu
def test_far_pages_of_a_long_run():
    """Shared keys in pages past 4 GiB."""
    import masked_attention_gb300 as M
    c = Case([(3, 640)], [90, 33, 5], Hkv=2, D=128, page=128)
    o, lse = c.run()
    pages = (1 << 32) // (2 * 2 * 128 * 128) + len(c.k)
    pools = [torch.empty(pages, 2, 128, 128, dtype=torch.bfloat16, device="cuda") for _ in (0, 1)]
    for pool, x in zip(pools, (c.k, c.v)):
        pool[-len(c.k):] = x.cuda()
    table = torch.where(c.table >= 0, c.table + pages - len(c.k), -1).to(torch.int32).cuda()
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    ws = torch.empty(M.attn_decode_shared_workspace_bytes(3, 4, 2, 1, 1, table.shape[1] * 128, 128),
                     dtype=torch.uint8, device="cuda")
    M.attn_decode_shared(c.q.cuda(), *pools, o2, lse2, c.variant(), page_table=table, page_size=128,
                         seq_lens=c.lens.cuda(), group_starts=c.starts.cuda(),
                         shared_lens=c.shared.cuda(), workspace=ws)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.gpu
@pytest.mark.parametrize("G", [0, 2048, 4096])
def test_most_sequences_and_groups(G):
    """As many sequences and groups as a call takes, one of them with keys that are read once; the
    reference gathers the rows and computes in fp64 on the device."""
    import masked_attention_gb300 as M
    B, Hq, Hkv, D, page, n, long = 4096, 4, 2, 64, 16, 48, 640
    g = torch.Generator(device="cuda").manual_seed(9)
    lens = torch.randint(0, n + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    table = torch.full((B, long // page + 3), -1, dtype=torch.int32, device="cuda")
    table[:, :3] = torch.randperm(3 * B, generator=g, device="cuda").view(B, 3).to(torch.int32)
    # the last two sequences share `long` keys, in pages of their own, and have 40 more each
    shared_pages = 3 * B + torch.arange(long // page, device="cuda", dtype=torch.int32)
    table[-2:, long // page:] = table[-2:, :3].clone()
    table[-2:, :long // page] = shared_pages
    lens[-2:] = long + 40
    k, v = (torch.randn(3 * B + long // page, Hkv, page, D, generator=g, device="cuda")
            .to(torch.bfloat16) for _ in (0, 1))
    q = torch.randn(B, Hq, 1, D, generator=g, device="cuda").to(torch.bfloat16)
    starts = torch.arange(G + 1, device="cuda", dtype=torch.int32) * (B // max(G, 1))
    if G == 4096:                                # groups of one, and the last of two
        starts[-2] = B - 2
        starts[-3] = B - 2
    shared = torch.zeros(G, device="cuda", dtype=torch.int32)
    shared[-1:] = long
    o, lse = guarded_empty((B, Hq, 1, D), torch.bfloat16), guarded_empty((B, Hq, 1), torch.float32)
    ws = guarded_empty((M.attn_decode_shared_workspace_bytes(B, Hq, Hkv, 1, G, table.shape[1] * page,
                                                             D),), torch.uint8)
    groups = dict(group_starts=starts, shared_lens=shared) if G else {}
    M.attn_decode_shared(q, k, v, o, lse, M.MASK_CAUSAL, page_table=table, page_size=page,
                         seq_lens=lens, workspace=ws, **groups)
    assert M.attn_check_status() == M.ATTN_OK
    check_canaries()
    for part, most in ((slice(0, B - 2), n), (slice(B - 2, B), long + 40)):
        at = table[part, :-(-most // page)].long().clamp(min=0)
        K, V = (x[at].transpose(1, 2).reshape(at.shape[0], Hkv, -1, D).double()
                .repeat_interleave(Hq // Hkv, 1) for x in (k, v))
        there = torch.arange(K.shape[2], device="cuda")[None] < lens[part, None]
        s = torch.einsum("bhd,bhjd->bhj", q[part, :, 0].double(), K) * D ** -0.5
        size = torch.einsum("bhd,bhjd->bhj", q[part, :, 0].double().abs(), K.abs()) * D ** -0.5
        s = s.masked_fill(~there[:, None], -np.inf)
        L = torch.logsumexp(s, -1)
        p = torch.exp(s - torch.where(torch.isinf(L), 0, L)[..., None])
        O, A = (torch.einsum("bhj,bhjd->bhd", p, x) for x in (V, V.abs()))
        E = 2.0 ** -17 * size.masked_fill(~there[:, None], 0).amax(-1)
        none = torch.isinf(L)
        got_o, got_l = o[part, :, 0].double(), lse[part, :, 0].double()
        assert torch.equal(torch.isinf(got_l), none) and (got_o[none] == 0).all()
        assert (none | ((got_l - L).abs() <= E + 2.0 ** -20 * (1 + L.abs()))).all()
        tol = 2.0 ** -8 * O.abs() + (2.0 ** -8 + 2.0 ** -18 + 4 * E[..., None]) * A
        assert ((got_o - O).abs() <= tol).all()


@pytest.mark.gpu
def test_reproducible_captured_and_on_another_stream():
    """Equal bits again, on a side stream and in two graphs that share a workspace; a graph
    follows lengths and groups that change under it."""
    import masked_attention_gb300 as M
    c = Case([(20, 900), (3, 128)], [5 + 3 * b for b in range(23)], Hq=8, Hkv=2, D=128, page=64)
    ref = c.run()
    t = [x.cuda() for x in (c.q, c.k, c.v, c.table, c.lens, c.starts, c.shared)]
    outs = [[torch.empty_like(x) for x in ref] for _ in range(3)]
    ws = torch.empty(M.attn_decode_shared_workspace_bytes(23, 8, 2, 1, 2, c.table.shape[1] * 64, 128),
                     dtype=torch.uint8, device="cuda")

    def call(i):
        M.attn_decode_shared(*t[:3], *outs[i], c.variant(), page_table=t[3], page_size=64,
                             seq_lens=t[4], group_starts=t[5], shared_lens=t[6], workspace=ws)

    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call(0)
        call(0)
    side.synchronize()
    graphs = []
    for i in (1, 2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call(i)
    t[6].zero_()
    t[4].fill_(3)
    for g in graphs:
        g.replay()
    t[6].copy_(c.shared)
    t[4].copy_(c.lens)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    for out in outs:
        assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1])


@pytest.mark.gpu
def test_a_wait_that_runs_out_is_reported():
    import masked_attention_gb300 as M
    c = Case([(9, 900)], [50] * 9, Hq=8, Hkv=2, D=128, page=64)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = torch.empty(9, 8, 1, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(
        9, 8, 1, device="cuda")
    ws = torch.empty(M.attn_decode_shared_workspace_bytes(9, 8, 2, 1, 1, c.table.shape[1] * 64, 128),
                     dtype=torch.uint8, device="cuda")
    M.attn_decode_shared(c.q.cuda(), c.k.cuda(), c.v.cuda(), o, lse, c.variant(),
                         page_table=c.table.cuda(), page_size=64, seq_lens=c.lens.cuda(),
                         group_starts=c.starts.cuda(), shared_lens=c.shared.cuda(), workspace=ws,
                         status=status, timeout_ns=20_000_000, fault_inject=M.FAULT_NO_LOADS)
    assert M.attn_check_status(status) == M.ATTN_ERR_TIMEOUT
    assert M.attn_check_status(status) == M.ATTN_OK
    c.check()


def test_oracle_against_a_softmax():
    rng = np.random.default_rng(0)
    q, K, V = rng.normal(size=(1, 2, 3, 8)), rng.normal(size=(9, 8)), rng.normal(size=(9, 8))
    s = np.einsum("hrd,jd->hrj", q[0], K) * 8 ** -0.5
    s[:, np.arange(9)[None] > (9 - 3 + np.arange(3))[:, None]] = -np.inf
    p = np.exp(s)
    O, L, _, _ = decode_rows(q, lambda b, h: (K, V), [9])
    assert np.allclose(O[0], p @ V / p.sum(-1, keepdims=True), rtol=0, atol=1e-12)
    assert np.allclose(L[0], np.log(p.sum(-1)), rtol=0, atol=1e-12)


def test_refusals():
    import masked_attention_gb300 as M
    L = M.lib()

    def call(B=2, Hq=4, Hkv=2, Sq=1, max_len=100, D=64, variant=M.MASK_CAUSAL, q=0x1000, k=0x2000,
             v=0x3000, o=0x4000, lse=0x5000, lens=0x6000, gs=0x7000, sl=0x8000, G=1, ws=0x100000,
             n=1 << 40, **kw):
        p = M.attn_params(M.BF16)
        p.page_table, p.page_size, p.pages_per_seq, p.num_pages = 0x9000, 16, 7, 50
        for name, x in kw.items():
            setattr(p, name, x)
        return L.attn_decode_shared(q, k, v, o, lse, B, Hq, Hkv, Sq, max_len, D, variant,
                                    ctypes.byref(p), lens, gs, sl, G, ws, n, None)

    inv, uns, mis = M.ATTN_ERR_INVALID_ARG, M.ATTN_ERR_UNSUPPORTED, M.ATTN_ERR_MISALIGNED
    assert call(B=-1) == call(Hq=5) == call(Sq=-1) == call(max_len=-1) == call(G=-1) == inv
    assert call(D=96) == call(dtype=M.F32) == call(page_size=48) == uns
    assert call(variant=M.MASK_DOCUMENT) == call(variant=M.MASK_PREFIX) == uns
    assert call(variant=M.SCORE_RELBIAS) == uns and call(variant=1 << 20) == inv
    assert call(variant=M.MASK_WINDOW) == call(variant=M.SCORE_SOFTCAP) == inv
    assert call(scale=-1.0) == call(scale=float("nan")) == inv
    assert call(q_offset=1) == call(kv_offset=1) == uns
    assert call(page_table=None) == call(pages_per_seq=6) == call(num_pages=0) == inv
    assert call(num_pages=2 ** 30) == call(max_len=2 ** 31 - 1, pages_per_seq=2 ** 27) == uns
    assert call(Hq=34) == call(Sq=9) == call(B=4097, Hkv=2) == call(G=4097) == uns
    assert call(B=4096, Hq=32, Hkv=16) == uns                      # B * Hkv > 65535
    for name in ("q", "k", "v", "o", "lse", "lens", "gs", "sl", "ws"):
        assert call(**{name: None}) == inv, name
    for name in ("q", "k", "v", "o"):
        assert call(**{name: 0x1008}) == mis, name
    for name in ("lse", "lens", "gs", "sl", "page_table", "alibi_slopes"):
        assert call(**{name: 0x9002}) == mis, name
    assert call(ws=0x100080) == mis
    need = M.attn_decode_shared_workspace_bytes(2, 4, 2, 1, 1, 100, 64)
    assert need > 0 and call(n=need - 1) == M.ATTN_ERR_WORKSPACE_TOO_SMALL
    assert call(B=0) == call(Sq=0) == M.ATTN_OK
    for bad in ((0, 4, 2, 1, 1, 9, 64), (1, 4, 3, 1, 1, 9, 64), (1, 34, 2, 1, 1, 9, 64),
                (1, 4, 2, 1, -1, 9, 64), (1, 4, 2, 1, 1, 9, 96)):
        assert M.attn_decode_shared_workspace_bytes(*bad) == 0
    t = torch.zeros(1, 1, 1, 64)
    with pytest.raises(ValueError):
        M.attn_decode_shared(t, t, t, t, t, page_table=t, page_size=16, seq_lens=t, workspace=t)
