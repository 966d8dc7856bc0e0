"""attn_decode_q4 against the fp64 oracle on the same records.

Tolerances, per output row. Scores: the products of q with codes are exact, a
group's 32 products and its offset 136 sum(q) are added in fp32 (34 additions,
each within 2^-23 of the running sum, at most 144 sum|q|), so a score is off by
at most eps_s = sum over groups of 2^-18 * 144 sum|q| * max scale * softmax
scale, and 2^-20 of its own size for the fp32 steps after (soft-cap and ALiBi
included). A weight is then off by a factor e^(2 eps_s) (its own and the
normalising sum's score), plus 2^-11 for its rounding to fp16 and 2^-18 for the
exponentials and merges; fp16's smallest step adds at most 2^-30 of the largest
weighted scale per key. O is rounded once to bf16 (2^-8)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle.serving import bf16_value, decode_q4, q4_bytes, q4_row, q4_write
from tests.helpers import check_canaries, guarded_empty


def bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)


class Cache:
    """Random records for sequences of the given lengths; every place that no
    sequence holds has codes 0xFF and NaN scales."""

    def __init__(self, lens, Hkv, D, page, seed=0, per=None, kscale=1.0, vscale=1.0, spare=2):
        rng = np.random.default_rng(seed)
        self.lens, self.Hkv, self.D, self.page = np.asarray(lens, np.int32), Hkv, D, page
        need = -(-self.lens // page)
        per = max(1, int(need.max())) if per is None else per
        pages = int(need.sum()) + spare
        self.pool = np.full((pages, Hkv, q4_bytes(page, D)), 0xFF, np.uint8)
        self.table = np.full((len(lens), per), -1, np.int32)
        ids = rng.permutation(pages)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        for b, n in enumerate(self.lens):
            for j in range(n):
                slot = self.table[b, j // page] * page + j % page
                for h in range(Hkv):
                    k, v = rng.normal(size=(2, D))
                    q4_write(self.pool, slot, h, k * kscale, v * vscale * (1 + 3 * rng.random()),
                             page)

    def set_scales(self, b, j, which, value_bits):
        """Overwrites the K (0) or V (1) scales of key j of sequence b."""
        w = self.D // 32 * 2
        at = self.page * self.D + which * self.page * w + j % self.page * w
        rec = self.pool[self.table[b, j // self.page]]
        rec[:, at:at + w] = np.tile(np.array([value_bits], np.uint16).view(np.uint8), w // 2)


def run(c, q, variant, ws=None, pool=None, **kw):
    import masked_attention_gb300 as M
    o = guarded_empty(q.shape, torch.bfloat16)
    lse = guarded_empty(q.shape[:3], torch.float32)
    o.fill_(9.0)
    lse.fill_(9.0)
    B, Hq, Sq, D = q.shape
    n = {"full": M.attn_decode_q4_workspace_bytes(B, Hq, c.Hkv, Sq, c.table.shape[1] * c.page, D),
         "none": 0}.get(ws, ws)
    work = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    M.attn_decode_q4(q.cuda(), torch.from_numpy(c.pool).cuda() if pool is None else pool, o, lse,
                     variant, page_table=torch.from_numpy(c.table).cuda(), page_size=c.page,
                     seq_lens=torch.from_numpy(c.lens).cuda(), workspace=work, **kw)
    check_canaries()
    return o.double().cpu().numpy(), lse.double().cpu().numpy()


def check(c, q, ws="full", causal=True, window=0, sink=0, softcap=0.0, alibi=False, slopes=None,
          scale=0.0):
    import masked_attention_gb300 as M
    variant = ((M.MASK_CAUSAL if causal else 0) | (M.MASK_WINDOW if window else 0) |
               (M.SCORE_SOFTCAP if softcap else 0) | (M.SCORE_ALIBI if alibi else 0))
    B, Hq, Sq, D = q.shape
    dev = None if slopes is None else torch.from_numpy(slopes).cuda()
    o, lse = run(c, q, variant, ws, window=window, sink=sink, softcap=softcap, alibi_slopes=dev,
                 scale=scale)
    al = None
    if alibi:
        al = 2.0 ** (-8.0 * np.arange(1, Hq + 1) / Hq) if slopes is None else slopes
    qn = q.double().numpy()
    sc = scale or D ** -0.5
    with np.errstate(invalid="ignore"):
        O, L, A = decode_q4(qn, c.pool, c.table, c.lens, c.page, causal=causal, window=window,
                            sink=sink, softcap=softcap, alibi=al, scale=sc)
    w = D // 32 * 2
    sk, sv = (bf16_value(np.ascontiguousarray(
        c.pool[:, :, c.page * D + i * c.page * w:c.page * D + (i + 1) * c.page * w]).view(np.uint16))
        for i in (0, 1))
    top = [float(np.abs(s[np.isfinite(s)]).max()) if np.isfinite(s).any() else 0.0
           for s in (sk, sv)]
    big = np.abs(qn).sum(-1) * 8 * top[0] * sc + (0 if al is None else
                                                  al[None, :, None] * c.lens.max())
    eps = 2.0 ** -18 * 144 * np.abs(qn).sum(-1) * top[0] * sc + 2.0 ** -20 * big
    empty = ~np.isfinite(L)
    assert np.array_equal(np.isneginf(lse), np.isneginf(L))
    assert (o[empty & ~np.isnan(L)] == 0).all()
    tol_l = 2 * eps + 2.0 ** -20 * (1 + np.abs(np.where(empty, 0, L)))
    assert (np.abs(lse[~empty] - L[~empty]) <= tol_l[~empty]).all()
    f = (np.expm1(2 * eps) + 2.0 ** -11 + 2.0 ** -18)[..., None]
    tol = 2.0 ** -8 * np.abs(O) + f * A * (1 + 2.0 ** -8) + c.lens.max() * 2.0 ** -30 * 8 * top[1]
    assert (np.abs(o - O) <= tol)[~empty].all(), float((np.abs(o - O) / tol)[~empty].max())
    return o, lse


def queries(B, Hq, Sq, D, seed=5, size=1.0):
    return bf16(np.random.default_rng(seed).normal(size=(B, Hq, Sq, D)) * size)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("heads", [(1, 1, 1), (4, 2, 1), (8, 1, 1), (6, 2, 3), (16, 1, 1),
                                   (10, 2, 2), (2, 1, 8)])
def test_lengths(D, page, heads):
    Hq, Hkv, Sq = heads
    c = Cache([0, 1, Sq, 31, 32, 33, 130], Hkv, D, page, seed=page + D)
    check(c, queries(7, Hq, Sq, D))


@pytest.mark.gpu
@pytest.mark.parametrize("D,heads", [(64, (4, 2, 2)), (128, (8, 1, 1)), (128, (12, 1, 1))])
@pytest.mark.parametrize("ws", ["full", "none", "third", 256])
def test_long_and_split(D, heads, ws):
    """Keys shared by many CTAs, by none, and by as many as a small workspace allows."""
    import masked_attention_gb300 as M
    Hq, Hkv, Sq = heads
    c = Cache([1500, 7, 0, 900], Hkv, D, 32, seed=3)
    if ws == "third":
        full = M.attn_decode_q4_workspace_bytes(4, Hq, Hkv, Sq, c.table.shape[1] * 32, D)
        ws = full // 3 + 17
    check(c, queries(4, Hq, Sq, D), ws)


@pytest.mark.gpu
@pytest.mark.parametrize("D,heads", [(64, (4, 1, 1)), (128, (5, 1, 3))])
@pytest.mark.parametrize("lens", [[4800], [5003, 3], [1700], [0, 1700, 40]])
def test_one_long_sequence(D, heads, lens):
    """Few pairs cut into many parts."""
    Hq, Hkv, Sq = heads
    c = Cache(lens, Hkv, D, 32, seed=4)
    check(c, queries(len(lens), Hq, Sq, D))
    check(c, queries(len(lens), Hq, Sq, D), window=4500, sink=40)


@pytest.mark.gpu
@pytest.mark.parametrize("D,heads,seed", [(64, (2, 1, 1), 0), (128, (4, 2, 2), 1), (64, (9, 1, 1), 2)])
def test_large_ragged_batches(D, heads, seed):
    """Hundreds of sequences, many of them empty or short, one long: the dealing
    out over CTAs has runs of sequences per thread and segments of every kind."""
    Hq, Hkv, Sq = heads
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, 40, 331) * (rng.random(331) < 0.7)
    lens[rng.integers(0, 331, 4)] = [700, 1300, 260, 129]
    lens[:7] = 0
    lens[-5:] = 0
    c = Cache(lens, Hkv, D, 16, seed=seed, per=90)
    check(c, queries(331, Hq, Sq, D), "full")
    c.lens[:] = 0    # no sequence at all
    o, lse = run(c, queries(331, Hq, Sq, D), 1, "full")
    assert (o == 0).all() and np.isneginf(lse).all()


MASKS = [dict(window=1), dict(window=20), dict(window=20, sink=1), dict(window=33, sink=40),
         dict(window=64, sink=4), dict(window=500, sink=4), dict(window=5, sink=1000),
         dict(causal=False), dict(causal=False, window=50, sink=3)]


@pytest.mark.gpu
@pytest.mark.parametrize("D,heads", [(64, (4, 2, 1)), (128, (6, 2, 3)), (128, (16, 1, 1))])
@pytest.mark.parametrize("mask", MASKS)
def test_windows_and_sinks(D, heads, mask):
    Hq, Hkv, Sq = heads
    c = Cache([0, 2, 21, 64, 97, 400], Hkv, D, 16, seed=11)
    for ws in ("full", "none"):
        check(c, queries(6, Hq, Sq, D), ws, **mask)


@pytest.mark.gpu
@pytest.mark.parametrize("mask", [dict(window=1400, sink=4), dict(window=1300, sink=100),
                                  dict(window=2500), dict(window=1400, sink=4, alibi=True)])
@pytest.mark.parametrize("ws", ["full", "none"])
def test_long_windows(mask, ws):
    """Windows long enough to be shared by several CTAs."""
    c = Cache([2900, 1500, 0, 50], 1, 64, 32, seed=24)
    check(c, queries(4, 4, 2, 64), ws, **mask)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads", [(8, 2, 2), (12, 1, 1)])
@pytest.mark.parametrize("kw", [dict(softcap=30.0), dict(softcap=1.5), dict(alibi=True),
                                dict(alibi=True, softcap=20.0, window=90, sink=5),
                                dict(scale=0.5)])
def test_scores(D, heads, kw):
    Hq, Hkv, Sq = heads
    c = Cache([3, 250, 77], Hkv, D, 64, seed=12)
    check(c, queries(3, Hq, Sq, D), **kw)
    if "alibi" in kw:
        sl = np.random.default_rng(1).random(Hq).astype(np.float32)
        check(c, queries(3, Hq, Sq, D), slopes=sl, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("cap", [6.0, 40.0, 1e6, 1e30, 3e38])
@pytest.mark.parametrize("heads", [(8, 2, 2), (12, 1, 1)])
def test_caps_far_above_the_scores(cap, heads):
    """A cap that the scores do not come near leaves them as they are: its
    rounding has to count against the score, not against the cap."""
    Hq, Hkv, Sq = heads
    c = Cache([130, 33], Hkv, 128, 16, seed=22)
    check(c, queries(2, Hq, Sq, 128), softcap=cap)
    check(c, queries(2, Hq, Sq, 128, size=1e-3), softcap=cap)


def test_caps_that_fp32_cannot_hold_are_refused():
    import masked_attention_gb300 as M
    p = M.attn_params()
    p.dtype, p.page_table, p.page_size, p.pages_per_seq, p.num_pages = 0, 0x6000, 16, 7, 9
    for cap in (float("inf"), float("nan"), 0.0, -1.0, 1e-39):
        p.softcap = cap
        assert M.lib().attn_decode_q4(0x1000, 0x2000, 0x3000, 0x4000, 1, 4, 2, 1, 100, 64,
                                      M.SCORE_SOFTCAP, ctypes.byref(p), 0x5000, 0, None, 0,
                                      None) == M.ATTN_ERR_INVALID_ARG, cap


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_scores_that_jump(D):
    """Scores of several hundred, the largest late in the key order: the
    running reference has to follow."""
    c = Cache([600], 1, D, 16, seed=13, kscale=2.0)
    check(c, queries(1, 8, 1, D, size=6.0))
    for where in (0, 300, 599):
        k = np.zeros(D)
        k[:] = 14.0
        q4_write(c.pool, c.table[0, where // 16] * 16 + where % 16, 0, k, k, 16)
        check(c, queries(1, 8, 1, D, size=1.0))


@pytest.mark.gpu
@pytest.mark.parametrize("vscale", [1e-20, 1e-6, 1e6, 1e30])
def test_sizes_of_values(vscale):
    """V far from 1: weights carry the scale through fp16."""
    c = Cache([200, 40], 2, 128, 32, seed=14, vscale=vscale)
    check(c, queries(2, 8, 1, 128))


@pytest.mark.gpu
def test_groups_of_unlike_size():
    """Channel groups of one value row that differ by 2^12, and keys that do."""
    c = Cache([150], 1, 128, 16, seed=15)
    rng = np.random.default_rng(3)
    for j in range(150):
        k, v = rng.normal(size=(2, 128))
        v = v * np.repeat([1.0, 2.0 ** -12, 2.0 ** 6, 1.0], 32) * 2.0 ** rng.integers(-8, 9)
        q4_write(c.pool, c.table[0, j // 16] * 16 + j % 16, 0, k, v, 16)
    check(c, queries(1, 4, 1, 128))


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_masked_records_change_nothing(D):
    """Infinities and NaN in the records of masked keys: same bits as with
    ordinary ones, for causal (drafted tokens), window and sinks."""
    for kw in (dict(window=0, sink=0), dict(window=30, sink=3)):
        c = Cache([120, 50], 2, D, 16, seed=16)
        q = queries(2, 4, 3, D)
        import masked_attention_gb300 as M
        variant = M.MASK_CAUSAL | (M.MASK_WINDOW if kw["window"] else 0)
        ref = run(c, q, variant, "full", **kw)
        # the last row sees the last two keys; rows 0 and 1 do not see all of them
        for bits in (0x7fff, 0x7f80, 0xff80):
            for which in (0, 1):
                d = Cache([120, 50], 2, D, 16, seed=16)
                d.set_scales(0, 119, which, bits)
                d.set_scales(1, 49, which, bits)
                if kw["window"]:
                    for j in range(3, 80):
                        d.set_scales(0, j, which, bits)
                got = run(d, q, variant, "full", **kw)
                for x, y in zip(got, ref):
                    assert np.array_equal(x[:, :, :2], y[:, :, :2])


@pytest.mark.gpu
def test_nan_in_a_visible_record_shows():
    c = Cache([60, 60], 1, 64, 16, seed=17)
    c.set_scales(0, 20, 0, 0x7fff)
    import masked_attention_gb300 as M
    o, lse = run(c, queries(2, 2, 1, 64), M.MASK_CAUSAL, "full")
    assert np.isnan(o[0]).all() and np.isnan(lse[0]).all() and np.isfinite(o[1]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ws", ["full", "none"])
def test_infinities_and_nan_in_queries(D, ws):
    """Such a row is NaN, as its scores are; the others keep their bits. Channels
    far apart in size, and the largest finite ones, are ordinary."""
    import masked_attention_gb300 as M
    c = Cache([400, 3], 2, D, 16, seed=23)
    q = queries(2, 4, 2, D)
    ref = run(c, q, M.MASK_CAUSAL, ws)
    bad = q.clone()
    bad[0, 1, 0, 5] = float("inf")
    bad[1, 3, 1, D - 1] = float("nan")
    bad[0, 2, 1, :2] = torch.tensor([float("inf"), -float("inf")])
    o, lse = run(c, bad, M.MASK_CAUSAL, ws)
    hit = torch.zeros(2, 4, 2, dtype=torch.bool)
    hit[0, 1, 0] = hit[1, 3, 1] = hit[0, 2, 1] = True
    hit = hit.numpy()
    assert np.isnan(o[hit]).all() and np.isnan(lse[hit]).all()
    assert np.array_equal(o[~hit], ref[0][~hit]) and np.array_equal(lse[~hit], ref[1][~hit])
    q[0, 0] *= torch.logspace(-12, 0, D, base=10.0)
    q[0, 1] = 0
    q[1, 2] *= 1e-30
    check(c, q, ws)


@pytest.mark.gpu
@pytest.mark.parametrize("D,Hkv", [(64, 8), (128, 4)])
def test_pool_past_32_bits(D, Hkv):
    """The same records beyond 4 GiB of a larger pool: the same bits."""
    import masked_attention_gb300 as M
    c = Cache([1500, 70], Hkv, D, 128, seed=31)
    q = queries(2, 2 * Hkv, 1, D)
    o, lse = check(c, q)
    small = c.pool
    first = (1 << 32) // small[0].size + 3
    pool = torch.zeros(first + len(small), *small.shape[1:], dtype=torch.uint8, device="cuda")
    pool[first:] = torch.from_numpy(small).cuda()
    c.table = np.where(c.table < 0, -1, c.table + first).astype(np.int32)
    o2, lse2 = run(c, q, M.MASK_CAUSAL, "full", pool=pool)
    assert np.array_equal(o, o2) and np.array_equal(lse, lse2)


@pytest.mark.gpu
def test_pages_outside_the_pool_read_zeros():
    """Bad table entries: their keys have K = V = 0 (as attn_decode reads them)."""
    c = Cache([100, 64], 2, 64, 16, seed=18)
    c.table[0, 2] = -5
    c.table[0, 4] = len(c.pool)
    c.table[1, 0] = 2 ** 31 - 1
    t = c.table.copy()
    good = np.where((t >= 0) & (t < len(c.pool)), t, -1)
    q = queries(2, 4, 1, 64)
    import masked_attention_gb300 as M
    o, lse = run(c, q, M.MASK_CAUSAL, "full")
    O, L, _ = decode_q4(q.double().numpy(), c.pool, good, c.lens, 16)
    assert np.abs(lse - L).max() < 1e-3 and np.abs(o - O).max() < 2e-2


@pytest.mark.gpu
def test_lengths_outside_the_bound():
    """seq_lens past max_len or negative count as the bounds."""
    import masked_attention_gb300 as M
    c = Cache([90, 64, 64], 1, 64, 32, seed=19)
    q = queries(3, 2, 1, 64)
    c.lens = np.array([90, 64, 0], np.int32)
    ref = run(c, q, M.MASK_CAUSAL, "full")
    c.lens = np.array([2 ** 31 - 1, 64, -3], np.int32)
    got = run(c, q, M.MASK_CAUSAL, "full", max_len=90)
    for x, y in zip(got, ref):
        assert np.array_equal(x, y)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_matches_the_bf16_decode(D):
    """The bf16 cache holding the same values (codes times power-of-two scales
    are exact in bf16): two implementations of one attention."""
    import masked_attention_gb300 as M
    B, Hq, Hkv, page, n = 2, 8, 2, 32, 700
    c = Cache([n, n], Hkv, D, page, seed=20)
    w = D // 32 * 2
    at = page * D
    bits = np.random.default_rng(1).choice(np.array([0x3e80, 0x3f00, 0x3e00], np.uint16),
                                           size=(len(c.pool), Hkv, 2 * page * D // 32))
    c.pool[:, :, at:at + 2 * page * w] = bits.view(np.uint8).reshape(len(c.pool), Hkv, -1)
    k, v = np.zeros((2, len(c.pool), Hkv, page, D))
    for pg in range(len(c.pool)):
        for h in range(Hkv):
            for r in range(page):
                k[pg, h, r], v[pg, h, r] = q4_row(c.pool, pg * page + r, h, page, D)
    q = queries(B, Hq, 1, D)
    o4, l4 = run(c, q, M.MASK_CAUSAL | M.MASK_WINDOW, "full", window=300)
    o = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(q.shape[:3], device="cuda")
    M.attn_decode(q.cuda(), bf16(k).cuda(), bf16(v).cuda(), o, lse,
                  M.MASK_CAUSAL | M.MASK_WINDOW, Skv=n, window=300,
                  page_table=torch.from_numpy(c.table).cuda(), page_size=page, q_offset=n - 1)
    assert np.abs(lse.double().cpu().numpy() - l4).max() < 2e-3
    assert np.abs(o.double().cpu().numpy() - o4).max() < 1e-2


@pytest.mark.gpu
def test_graphs_streams_and_a_shared_workspace():
    """Two captured graphs on one workspace, replayed in turn and again; then
    calls on a side stream: same bits as eager calls."""
    import masked_attention_gb300 as M
    cs = [Cache([800, 30, 0], 2, 128, 16, seed=21, per=100),
          Cache([33, 700, 1], 2, 128, 16, seed=22, per=100)]
    q = queries(3, 8, 1, 128).cuda()
    refs = [run(c, q.cpu(), M.MASK_CAUSAL, "full") for c in cs]
    n = max(M.attn_decode_q4_workspace_bytes(3, 8, 2, 1, c.table.shape[1] * 16, 128) for c in cs)
    assert n > 0   # the tables are wide enough that the keys are shared out
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    outs = [(torch.empty_like(q), torch.empty(3, 8, 1, device="cuda")) for _ in cs]
    dev = [(torch.from_numpy(c.pool).cuda(), torch.from_numpy(c.table).cuda(),
            torch.from_numpy(c.lens).cuda()) for c in cs]

    def call(i):
        M.attn_decode_q4(q, dev[i][0], *outs[i], M.MASK_CAUSAL, page_table=dev[i][1],
                         page_size=16, seq_lens=dev[i][2], workspace=ws)

    graphs = []
    for i in (0, 1):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(i)
        graphs.append(g)

    def same(i):
        return all(np.array_equal(x.double().cpu().numpy(), y) for x, y in zip(outs[i], refs[i]))

    for i in (0, 1, 0, 0, 1):
        for t in outs[i]:
            t.fill_(4.0)
        ws.fill_(0xff)
        graphs[i].replay()
        torch.cuda.synchronize()
        assert same(i)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(0)
    s.synchronize()
    assert same(0)


def test_refusals():
    import masked_attention_gb300 as M
    L = M.lib()

    def dec(variant=0, B=1, Hq=4, Hkv=2, Sq=1, max_len=100, D=64, sink=0, q=0x1000, pool=0x2000,
            o=0x3000, lse=0x4000, lens=0x5000, ws=None, n=0, **kw):
        p = M.attn_params()
        p.dtype, p.page_table, p.page_size, p.pages_per_seq, p.num_pages = 0, 0x6000, 16, 7, 9
        for name, v in kw.items():
            setattr(p, name, v)
        return L.attn_decode_q4(q, pool, o, lse, B, Hq, Hkv, Sq, max_len, D, variant,
                                ctypes.byref(p), lens, sink, ws, n, None)

    inv, uns, mis = M.ATTN_ERR_INVALID_ARG, M.ATTN_ERR_UNSUPPORTED, M.ATTN_ERR_MISALIGNED
    assert dec(D=96) == dec(dtype=1) == dec(page_size=8) == dec(page_size=48) == uns
    assert dec(Hq=3) == dec(B=-1) == dec(Sq=-1) == dec(max_len=-1) == dec(sink=-1) == inv
    assert dec(Hq=34) == dec(Hq=8, Sq=5) == dec(B=40000) == uns       # rows, grid
    for bit in (M.MASK_DOCUMENT, M.MASK_PREFIX, M.SCORE_RELBIAS):
        assert dec(bit) == uns
    assert dec(1 << 5) == inv
    assert dec(M.MASK_WINDOW) == dec(M.SCORE_SOFTCAP) == dec(scale=float("inf")) == inv
    assert dec(q_offset=3) == dec(kv_offset=3) == uns
    assert dec(max_len=2 ** 31 - 1, pages_per_seq=2 ** 27) == uns
    assert dec(max_len=113) == dec(num_pages=0) == dec(pages_per_seq=0) == inv
    for n in ("q", "pool", "o", "lse", "lens"):
        assert dec(**{n: None}) == inv and dec(**{n: 0x1002}) == mis, n
    assert dec(page_table=None) == inv and dec(page_table=0x6001) == mis
    assert dec(q=0x1008) == dec(ws=0x100010, n=4096) == dec(alibi_slopes=0x5001) == mis
    assert dec(B=0) == dec(Sq=0) == M.ATTN_OK
    assert M.attn_decode_q4_workspace_bytes(1, 4, 2, 1, 0, 64) == 0


def group_factors(pattern, j, n, G):
    """Sizes of the G channel groups of value row j of n."""
    f = np.ones(G)
    if pattern == "steady":
        f = np.array([1.0, 2.0 ** -24, 2.0 ** -60, 2.0 ** 6])[:G]
    elif pattern == "far":
        f = np.array([2.0 ** -50, 2.0 ** 40, 1.0, 2.0 ** 10])[:G]
    elif pattern == "first half":      # keys are processed from the last one
        f[1] = 2.0 ** 30 if j < n // 2 else 1.0
    elif pattern == "second half":
        f[1] = 2.0 ** 30 if j >= n // 2 else 1.0
    elif pattern == "in turn":
        f[j % G] = 2.0 ** 24
    elif pattern == "a zero group":
        f[1] = 0.0
    elif pattern == "zero in most keys":
        f[1] = 2.0 ** -30 if j % 7 == 0 else 0.0
    elif pattern == "zero in late keys":
        f[0] = 2.0 ** -30 if j < n // 2 else 0.0
    elif pattern == "tiny":
        f[:] = 2.0 ** -112
    elif pattern == "tiny in late keys":
        f[:] = 1.0 if j < n // 2 else 2.0 ** -112
    return f


GROUP_PATTERNS = ["steady", "far", "first half", "second half", "in turn", "a zero group",
                  "zero in most keys", "zero in late keys", "tiny", "tiny in late keys"]


def check_groups(c, q, ws="full", window=0, sink=0):
    """Like check(), each channel group held to its own size. A weight is rounded to fp16 times
    its group's scale, which is at least 2^-8 of the key's largest, and 2^8 is the largest such
    product of a row: what a subnormal loses, half a step of 2^-24, is at most 2^-25 of the
    group's largest product for each key (a quantised group's largest code is 7 of at most 8)."""
    import masked_attention_gb300 as M
    o, lse = run(c, q, M.MASK_CAUSAL | (M.MASK_WINDOW if window else 0), ws, window=window, sink=sink)
    B, Hq, Sq, D = q.shape
    qn = q.double().numpy()
    O, L, A = decode_q4(qn, c.pool, c.table, c.lens, c.page, window=window, sink=sink)
    w = D // 32 * 2
    sk = bf16_value(np.ascontiguousarray(c.pool[:, :, c.page * D:c.page * (D + w)]).view(np.uint16))
    top = float(np.abs(sk[np.isfinite(sk)]).max())
    eps = (2.0 ** -18 * 144 + 2.0 ** -20 * 8) * np.abs(qn).sum(-1) * top * D ** -0.5
    f = (np.expm1(2 * eps) + 2.0 ** -11 + 2.0 ** -18)[..., None]
    size = np.repeat(A.reshape(B, Hq, Sq, D // 32, 32).max(-1), 32, -1)
    tol = (2.0 ** -8 * np.abs(O) + f * A * (1 + 2.0 ** -8) + c.lens.max() * 2.0 ** -25 * 8 / 7 * size
           + 2.0 ** -134)   # and half of bf16's smallest step
    assert (np.abs(lse - L) <= 2 * eps + 2.0 ** -20 * (1 + np.abs(L))).all()
    with np.errstate(invalid="ignore", divide="ignore"):
        assert (np.abs(o - O) <= tol).all(), float(np.nanmax(np.abs(o - O) / tol))


@pytest.mark.gpu
@pytest.mark.parametrize("pattern", GROUP_PATTERNS)
@pytest.mark.parametrize("D,heads,n", [(64, (4, 1, 1), 150), (128, (4, 1, 1), 150),
                                       (128, (6, 1, 2), 97), (64, (4, 1, 1), 1500)])
def test_groups_keep_their_own_precision(pattern, D, heads, n):
    """Channel groups of unlike size, in all keys, in some, and without values: each one's
    outputs are as precise as if it were alone."""
    Hq, Hkv, Sq = heads
    page = 16
    c = Cache([n], Hkv, D, page, seed=33)
    rng = np.random.default_rng(7)
    for j in range(n):
        k, v = rng.normal(size=(2, D))
        v = v * np.repeat(group_factors(pattern, j, n, D // 32), 32)
        q4_write(c.pool, c.table[0, j // page] * page + j % page, 0, k, v, page)
    check_groups(c, queries(1, Hq, Sq, D))
    check_groups(c, queries(1, Hq, Sq, D), window=70, sink=5)


@pytest.mark.gpu
@pytest.mark.parametrize("where", [3, 60, 99])
def test_a_heavy_key_without_values(where):
    """A key that takes nearly all of the weight (it scores 85, the others about 0) and whose
    values are zero: the others' share of about 2^-122 is what O is."""
    D, n, page = 64, 100, 16
    c = Cache([n], 1, D, page, seed=34)
    q4_write(c.pool, c.table[0, where // page] * page + where % page, 0, np.full(D, 10.6),
             np.zeros(D), page)
    check_groups(c, bf16(np.full((1, 2, 1, D), 1.0)))


@pytest.mark.gpu
@pytest.mark.parametrize("heavy,j", [(20, 5), (36, 33), (36, 5), (20, 38)])
def test_nan_values_of_a_visible_key_without_weight(heavy, j):
    """The weight of a key that scores 1600 below the largest is 0, and NaN times it is NaN,
    in a tile whose keys are all visible (keys 0 to 31) as in one that ends the sequence."""
    import masked_attention_gb300 as M
    D, n, page = 64, 40, 16
    c = Cache([n], 1, D, page, seed=35)
    for at in range(n):
        q4_write(c.pool, c.table[0, at // page] * page + at % page, 0,
                 np.full(D, 100.0 if at == heavy else -100.0), np.ones(D), page)
    c.set_scales(0, j, 1, 0x7fff)
    o, lse = run(c, bf16(np.full((1, 2, 1, D), 1.0)), M.MASK_CAUSAL, "none")
    assert np.isnan(o).all() and np.isfinite(lse).all()


def shared(lens, Hkv, D, page=16, **kw):
    """A cache whose table is wide enough that the keys are shared out over CTAs."""
    return Cache(lens, Hkv, D, page, per=max(-(-max(lens) // page), 1300 // page + 1), **kw)


def shares_out(c, q):
    import masked_attention_gb300 as M
    B, Hq, Sq, D = q.shape
    return M.attn_decode_q4_workspace_bytes(B, Hq, c.Hkv, Sq, c.table.shape[1] * c.page, D) > 0


SHARED_SCORES = [dict(softcap=30.0), dict(softcap=1.5), dict(alibi=True),
                 dict(alibi=True, softcap=20.0), dict(alibi=True, softcap=20.0, window=1450, sink=5),
                 dict(scale=0.5, causal=False), dict(softcap=1e6)]


@pytest.mark.gpu
@pytest.mark.parametrize("kw", SHARED_SCORES)
@pytest.mark.parametrize("D,heads", [(64, (4, 1, 2)), (128, (12, 1, 1))])
def test_scores_of_shared_keys(D, heads, kw):
    """Score modifications where a pair's keys are cut over many CTAs."""
    Hq, Hkv, Sq = heads
    c = shared([1700, 3, 0, 260], Hkv, D, seed=41)
    q = queries(4, Hq, Sq, D)
    assert shares_out(c, q)
    check(c, q, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("D,heads", [(64, (4, 1, 3)), (128, (16, 1, 1))])
def test_edges_of_shared_keys(D, heads):
    """NaN and infinite queries, NaN in visible and in masked records, pages outside the pool
    and lengths outside the bound, with the results of cut pairs joined from the workspace."""
    import masked_attention_gb300 as M
    Hq, Hkv, Sq = heads
    lens = [1600, 90, 1300]
    c = shared(lens, Hkv, D, seed=42)
    q = queries(3, Hq, Sq, D)
    assert shares_out(c, q)
    ref = check(c, q)
    bad = q.clone()   # such rows are NaN, the others keep their bits
    bad[0, 1, 0, 5] = float("inf")
    bad[2, Hq - 1, Sq - 1, D - 1] = float("nan")
    hit = np.zeros((3, Hq, Sq), bool)
    hit[0, 1, 0] = hit[2, Hq - 1, Sq - 1] = True
    got = run(c, bad, M.MASK_CAUSAL, "full")
    for x, y in zip(got, ref):
        assert np.isnan(x[hit]).all() and np.array_equal(x[~hit], y[~hit])
    if Sq > 1:        # the last key is masked for the first rows
        for bits in (0x7fff, 0xff80):
            d = shared(lens, Hkv, D, seed=42)
            d.set_scales(0, 1599, 0, bits)
            d.set_scales(2, 1299, 1, bits)
            for x, y in zip(run(d, q, M.MASK_CAUSAL, "full"), ref):
                assert np.array_equal(x[:, :, :Sq - 1], y[:, :, :Sq - 1])
    d = shared(lens, Hkv, D, seed=42)      # a NaN key in a part of its own
    d.set_scales(0, 40, 0, 0x7fff)
    o, lse = run(d, q, M.MASK_CAUSAL, "full")
    assert np.isnan(o[0]).all() and np.isnan(lse[0]).all()
    assert np.array_equal(o[1:], ref[0][1:]) and np.array_equal(lse[1:], ref[1][1:])
    d = shared(lens, Hkv, D, seed=42)      # pages that are not there read as zeros
    d.table[0, 2:60] = -5
    d.table[2, 7] = len(d.pool)
    t = np.where((d.table >= 0) & (d.table < len(d.pool)), d.table, -1)
    o, lse = run(d, q, M.MASK_CAUSAL, "full")
    O, L, _ = decode_q4(q.double().numpy(), d.pool, t, d.lens, 16)
    assert np.abs(lse - L).max() < 1e-3 and np.abs(o - O).max() < 2e-2
    d = shared(lens, Hkv, D, seed=42)      # lengths count as the nearest bound
    d.lens = np.array([2 ** 31 - 1, 90, -7], np.int32)
    got = run(d, q, M.MASK_CAUSAL, "full", max_len=1600)
    d.lens = np.array([1600, 90, 0], np.int32)
    for x, y in zip(got, run(d, q, M.MASK_CAUSAL, "full", max_len=1600)):
        assert np.array_equal(x, y)


@pytest.mark.gpu
@pytest.mark.parametrize("D,heads", [(64, (2, 1, 3)), (128, (12, 3, 4))])
@pytest.mark.parametrize("kw", [dict(), dict(softcap=20.0), dict(alibi=True), dict(window=2)])
def test_rows_without_a_key_take_any_query(D, heads, kw):
    """Rows before a sequence's first token (places of a padded batch) are 0 with LSE -inf
    whatever their queries hold, alone and where keys are shared out."""
    import masked_attention_gb300 as M
    Hq, Hkv, Sq = heads
    for make in (Cache, shared):
        c = make([1, 0, 2, 1400 if make is shared else 40], Hkv, D, 16, seed=51)
        q = queries(4, Hq, Sq, D)
        ref = check(c, q, **kw)
        bad = q.clone()
        for b, n in enumerate(c.lens):
            for r in range(max(0, Sq - int(n))):
                bad[b, :, r, r::3] = float("nan") if r % 2 == 0 else float("inf")
        variant = (M.MASK_CAUSAL | (M.MASK_WINDOW if "window" in kw else 0) |
                   (M.SCORE_SOFTCAP if "softcap" in kw else 0) | (M.SCORE_ALIBI if "alibi" in kw else 0))
        kw2 = {k: v for k, v in kw.items() if k != "alibi"}
        for x, y in zip(run(c, bad, variant, "full", **kw2), ref):
            assert np.array_equal(x, y)
