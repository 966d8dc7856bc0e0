"""attn_page_plan: page tables, slot maps and lengths of a serving step built
on the device, against the oracle's token-by-token plan (whole numbers: equal)."""
import numpy as np
import pytest
import torch

from oracle.serving import page_plan

NAMES = ("seq_lens", "cu_new", "slots", "positions", "seq_ids", "page_table", "info")


def make(cached, new, page, per, spare=0, seed=0):
    """A consistent state: distinct pages for what is cached, then a free list."""
    rng = np.random.default_rng(seed)
    cached, new = np.asarray(cached, np.int32), np.asarray(new, np.int32)
    c = np.maximum(cached, 0)
    have = np.minimum(-(-c // page), per)
    need = np.minimum(-(-(c + np.maximum(new, 0)) // page), per)
    n_free = int((need - have).sum()) + spare
    ids = rng.permutation(int(have.sum()) + max(n_free, 0) + 5).astype(np.int32)
    table = np.full((len(cached), per), -7, np.int32)   # what is not entered stays
    at = 0
    for b in range(len(cached)):
        table[b, :have[b]] = ids[at:at + have[b]]
        at += have[b]
    return cached, new, table, ids[at:at + max(n_free, 0)]


def run(cached, new, table, free, page, cap):
    import masked_attention_gb300 as M
    from tests.helpers import check_canaries, guarded_empty
    B = len(cached)
    dev = {n: guarded_empty(s, torch.int64 if n == "slots" else torch.int32)
           for n, s in (("seq_lens", (B,)), ("cu_new", (B + 1,)), ("slots", (cap,)),
                        ("positions", (cap,)), ("seq_ids", (cap,)),
                        ("page_table", table.shape), ("info", (4,)))}
    dev["page_table"].copy_(torch.from_numpy(table))
    M.attn_page_plan(*(torch.from_numpy(x).cuda() for x in (cached, new)), dev["page_table"],
                     torch.from_numpy(np.ascontiguousarray(free)).cuda(), dev["seq_lens"],
                     dev["cu_new"], dev["slots"], dev["positions"], dev["seq_ids"], dev["info"],
                     page_size=page)
    check_canaries()
    return [dev[n].cpu().numpy() for n in NAMES]


def check(cached, new, table, free, page, cap):
    got = run(cached, new, table, free, page, cap)
    for name, g, r in zip(NAMES, got, page_plan(cached, new, table, free, page, cap)):
        assert np.array_equal(g, r), name


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("cached,new", [
    ([0], [1]), ([5], [0]), ([0, 0, 0], [0, 0, 0]), ([15, 16, 17, 0, 127, 128], [1, 1, 1, 1, 1, 1]),
    ([3, 0, 700, 64], [300, 129, 0, 1]), ([-4, 9], [2, -3])])
def test_small_plans(page, cached, new):
    s = make(cached, new, page, per=max(1, 1000 // page + 1), spare=2)
    total = int(np.maximum(new, 0).sum())
    for cap in {max(total, 1), total + 9, max(total - 1, 1)}:   # exact, padded, one too short
        check(*s, page, cap)


@pytest.mark.gpu
def test_no_token_places():
    check(*make([40, 3], [4, 2], 16, 8), 16, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("B,most_new,seed", [(1, 5000, 0), (31, 400, 1), (257, 90, 2),
                                             (1000, 7, 3), (4099, 3, 4)])
def test_random_plans(B, most_new, seed):
    rng = np.random.default_rng(seed)
    page = int(rng.choice([16, 32, 64, 128]))
    cached, new = rng.integers(0, 500, B), rng.integers(0, most_new + 1, B)
    s = make(cached, new, page, per=-(-(500 + most_new) // page), seed=seed)
    check(*s, page, int(new.sum()) + 100)


@pytest.mark.gpu
def test_largest_batch():
    rng = np.random.default_rng(9)
    B = 16384
    s = make(rng.integers(0, 40, B), rng.integers(0, 2, B), 16, per=3)
    check(*s, 16, B)


@pytest.mark.gpu
@pytest.mark.parametrize("spare", [-1, -3, -100])
def test_free_list_runs_short(spare):
    """Pages that the free list cannot give are -1, and so are their tokens' slots."""
    s = make([10, 30, 0, 64], [40, 20, 33, 64], 16, per=12, spare=spare)
    check(*s, 16, 200)
    assert run(*s, 16, 200)[-1][2] > 0


@pytest.mark.gpu
def test_requests_longer_than_their_table():
    s = make([60, 10, 200], [10, 2, 5], 16, per=4, spare=3)
    check(*s, 16, 17)
    assert run(*s, 16, 17)[-1][3] == 2


@pytest.mark.gpu
def test_twice_and_in_a_graph():
    """Run again on its own output (the entries are there already) and as a
    captured graph that replays with new lengths."""
    import masked_attention_gb300 as M
    cached, new, table, free = make([15, 0, 33], [2, 17, 31], 16, per=8)
    d = [torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in (cached, new, table, free)]
    cap = 64
    outs = [torch.empty(n, dtype=dt, device="cuda") for n, dt in
            ((3, torch.int32), (4, torch.int32), (cap, torch.int64), (cap, torch.int32),
             (cap, torch.int32), (4, torch.int32))]

    def call():
        M.attn_page_plan(*d, *outs, page_size=16)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
        call()
    torch.cuda.current_stream().wait_stream(s)
    ref = page_plan(cached, new, table, free, 16, cap)
    assert np.array_equal(outs[2].cpu().numpy(), ref[2])
    assert np.array_equal(d[2].cpu().numpy(), ref[5])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for new2 in ([1, 1, 1], [0, 20, 3]):
        d[1].copy_(torch.tensor(new2, dtype=torch.int32))
        d[2].copy_(torch.from_numpy(table))
        g.replay()
        torch.cuda.synchronize()
        ref = page_plan(cached, np.array(new2), table, free, 16, cap)
        for got, r in zip(outs, (ref[0], ref[1], ref[2], ref[3], ref[4], ref[6])):
            assert np.array_equal(got.cpu().numpy(), r)


def test_oracle_plan_by_hand():
    """Two requests, 4-token pages written out."""
    table = np.array([[8, -7, -7], [5, 6, -7]], np.int32)
    lens, cu, slots, pos, ids, tab, info = page_plan([3, 7], [3, 2], table, [2, 9], 4, 6)
    assert lens.tolist() == [6, 9] and cu.tolist() == [0, 3, 5]
    assert slots.tolist() == [8 * 4 + 3, 2 * 4, 2 * 4 + 1, 6 * 4 + 3, 9 * 4, -1]
    assert pos.tolist() == [3, 4, 5, 7, 8, -1] and ids.tolist() == [0, 0, 0, 1, 1, -1]
    assert tab.tolist() == [[8, 2, -7], [5, 6, 9]] and info.tolist() == [5, 2, 0, 0]


@pytest.mark.gpu
def test_empty_arguments_overlap_nothing():
    """An empty free list may begin anywhere, inside an output too."""
    import masked_attention_gb300 as M
    d = {n: torch.zeros(64, dtype=torch.int32, device="cuda")
         for n in ("cached", "new", "table", "lens", "cu", "slots", "pos", "ids", "info")}
    d["cached"][:2] = torch.tensor([3, 5])
    d["new"][:2] = 1
    d["table"][[0, 4]] = torch.tensor([7, 2], dtype=torch.int32, device="cuda")
    a = {n: t.data_ptr() for n, t in d.items()}
    stream = torch.cuda.current_stream().cuda_stream
    assert M.lib().attn_page_plan(a["cached"], a["new"], 2, a["table"], 4, 16, a["lens"] + 4, 0,
                                  a["lens"], a["cu"], a["slots"], a["pos"], a["ids"], 2, a["info"],
                                  stream) == M.ATTN_OK
    assert d["lens"][:2].tolist() == [4, 6] and d["info"][:4].tolist() == [2, 0, 0, 0]
    assert d["slots"].view(torch.int64)[:2].tolist() == [7 * 16 + 3, 2 * 16 + 5]


def test_overlapping_arguments_are_refused():
    """The lengths in place, the natural mistake, and neighbours that run into
    one another."""
    import masked_attention_gb300 as M
    names = ("cached", "new", "table", "free", "lens", "cu", "slots", "pos", "ids", "info")
    size = dict(cached=8, new=8, table=32, free=12, lens=8, cu=12, slots=64, pos=32, ids=32, info=16)

    def plan(**kw):
        a = {n: 0x1000 * (i + 1) for i, n in enumerate(names)}
        a.update(kw)
        return M.lib().attn_page_plan(a["cached"], a["new"], 2, a["table"], 4, 16, a["free"], 3,
                                      a["lens"], a["cu"], a["slots"], a["pos"], a["ids"], 8,
                                      a["info"], None)

    for out in ("table", "lens", "cu", "slots", "pos", "ids", "info"):
        for i, other in enumerate(names):
            if other == out:
                continue
            at = 0x1000 * (i + 1)
            assert plan(**{out: at}) == M.ATTN_ERR_INVALID_ARG, (out, other)
            last = at + (size[other] - 1) // 8 * 8      # inside it, aligned for all types
            assert plan(**{out: last}) == M.ATTN_ERR_INVALID_ARG, (out, other)


def test_refusals():
    import masked_attention_gb300 as M
    L = M.lib()

    def plan(B=2, per=4, page=16, n_free=3, cap=8, **kw):
        a = dict(cached=0x1000, new=0x2000, table=0x3000, free=0x4000, lens=0x5000, cu=0x6000,
                 slots=0x7000, pos=0x8000, ids=0x9000, info=0xa000)
        a.update(kw)
        return L.attn_page_plan(a["cached"], a["new"], B, a["table"], per, page, a["free"], n_free,
                                a["lens"], a["cu"], a["slots"], a["pos"], a["ids"], cap, a["info"],
                                None)

    assert plan(B=0) == plan(per=0) == plan(n_free=-1) == plan(cap=-1) == M.ATTN_ERR_INVALID_ARG
    assert plan(page=24) == plan(page=8) == plan(page=256) == M.ATTN_ERR_UNSUPPORTED
    assert plan(B=16385) == M.ATTN_ERR_UNSUPPORTED
    for n in ("cached", "new", "table", "free", "lens", "cu", "slots", "pos", "ids", "info"):
        assert plan(**{n: None}) == M.ATTN_ERR_INVALID_ARG, n
        assert plan(**{n: 0x1002}) == M.ATTN_ERR_MISALIGNED, n
    assert plan(slots=0x1004) == M.ATTN_ERR_MISALIGNED
    # the binding refuses what it would pass on wrongly
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):   # CPU tensors
        M.attn_page_plan(i, i, torch.zeros(4, 2, dtype=torch.int32), i, i,
                         torch.zeros(5, dtype=torch.int32), torch.zeros(3, dtype=torch.int64),
                         i[:3], i[:3], i, page_size=16)


@pytest.mark.gpu
def test_the_largest_token_budget():
    """2^31 - 1 token places: the last ones are -1, and the work is spread over the GPU as it
    is for a few places less (the count of blocks must not overflow)."""
    import masked_attention_gb300 as M
    most = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 60 * 2 ** 30:
        pytest.skip("needs 34 GB for the outputs")
    cached, new, table, free = (torch.from_numpy(np.ascontiguousarray(x)).cuda()
                                for x in make([3, 40], [5, 700], 16, 50))
    outs = [torch.zeros(n, dtype=torch.int32, device="cuda") for n in (2, 3)]
    slots = torch.zeros(most, dtype=torch.int64, device="cuda")
    pos, ids = (torch.zeros(most, dtype=torch.int32, device="cuda") for _ in (0, 1))
    info = torch.zeros(4, dtype=torch.int32, device="cuda")
    ref = page_plan([3, 40], [5, 700], table.cpu().numpy(), free.cpu().numpy(), 16, 800)

    def call(n):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in (0, 1))
        a.record()
        M.attn_page_plan(cached, new, table, free, *outs, slots[:n], pos[:n], ids[:n], info,
                         page_size=16)
        b.record()
        b.synchronize()
        return a.elapsed_time(b)

    few = min(call(most - 1000) for _ in range(3))
    slots[-1000:] = 7
    assert min(call(most) for _ in range(2)) < 8 * few
    for got, r in zip((slots, pos, ids), ref[2:5]):
        assert np.array_equal(got[:800].cpu().numpy(), r)
        assert (got[-2000:] == -1).all()
    assert np.array_equal(info.cpu().numpy(), ref[6])
