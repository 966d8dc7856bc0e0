"""The operators around the cache as a server runs them together: the plan from
the requests' lengths, norm and rotation at the plan's positions, the cache's
write at the plan's slots, then attention over the cache; prompts attend
through a read of the cache and attn_fwd on the packed batch. Every stage is
checked against the fp64 oracle on the stage's own inputs."""
import numpy as np
import pytest
import torch

from oracle.serving import decode_q4, norm_rope, page_plan, q4_write

HQ, HKV, D, PAGE, WINDOW, SINK = 4, 2, 64, 16, 40, 4


def table(n):
    f = 10000.0 ** (-np.arange(D // 2) / (D // 2))
    a = np.arange(n)[:, None] * f
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


class Server:
    """Buffers of a fixed batch of 3 requests and 64 tokens a step."""

    B, CAP, PAGES, PER = 3, 64, 30, 8

    def __init__(self):
        i32 = dict(dtype=torch.int32, device="cuda")
        from oracle.serving import q4_bytes
        self.table = torch.full((self.B, self.PER), -1, **i32)
        self.free = torch.from_numpy(np.random.default_rng(0).permutation(self.PAGES)
                                     .astype(np.int32)).cuda()
        self.cached, self.new = torch.zeros(self.B, **i32), torch.zeros(self.B, **i32)
        self.lens, self.cu, self.info = (torch.zeros(n, **i32) for n in (self.B, self.B + 1, 4))
        self.slots = torch.zeros(self.CAP, dtype=torch.int64, device="cuda")
        self.pos, self.ids = (torch.zeros(self.CAP, **i32) for _ in (0, 1))
        self.pool = torch.zeros(self.PAGES, HKV, q4_bytes(PAGE, D), dtype=torch.uint8,
                                device="cuda")
        self.cos_sin = torch.from_numpy(table(self.PER * PAGE)).cuda()
        self.w = [torch.linspace(0.5, 1.5, D, device="cuda"), torch.linspace(1.5, 0.5, D,
                                                                             device="cuda")]
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.qkv = torch.zeros(1, self.CAP, HQ + 2 * HKV, D, **bf)
        self.q, self.k = (torch.zeros(1, n, self.CAP, D, **bf) for n in (HQ, HKV))

    def parts(self):
        x = self.qkv.transpose(1, 2)
        return x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:]

    def write(self):
        """Plan, norm and rotation, cache write of the step's tokens."""
        import masked_attention_gb300 as M
        M.attn_page_plan(self.cached, self.new, self.table, self.free, self.lens, self.cu,
                         self.slots, self.pos, self.ids, self.info, page_size=PAGE)
        q, k, v = self.parts()
        M.attn_qk_norm_rope(q, k, self.q, self.k, q_weight=self.w[0], k_weight=self.w[1],
                            cos_sin=self.cos_sin, positions=self.pos)
        M.attn_cache_store_q4(self.k, v, self.slots, self.pool, page_size=PAGE)

    def advance(self):
        self.free = self.free[int(self.info[1]):].contiguous()
        self.cached.copy_(self.lens)


def feed(s, seed, lens):
    """The step's projection output and lengths; places past the last token hold NaN."""
    n = sum(lens)
    x = torch.randn(n, HQ + 2 * HKV, D, generator=torch.Generator().manual_seed(seed))
    s.qkv.fill_(float("nan"))
    s.qkv[0, :n] = x.to(torch.bfloat16).cuda()
    s.new.copy_(torch.tensor(lens, dtype=torch.int32))
    return n


def check_write(s, mirror, before, lens):
    """Plan equal, rows within their rounding, records equal byte by byte."""
    cached, tab, free = before
    ref = page_plan(cached, lens, tab, free, PAGE, s.CAP)
    got = (s.lens, s.cu, s.slots, s.pos, s.ids, s.table, s.info)
    for g, r in zip(got, ref):
        assert np.array_equal(g.cpu().numpy(), r)
    n = sum(lens)
    q, k, v = (t[:, :, :n].double().cpu().numpy() for t in s.parts())
    cs = s.cos_sin.double().cpu().numpy()
    for x, w, out in ((q, s.w[0], s.q), (k, s.w[1], s.k)):
        r = norm_rope(x, w.double().cpu().numpy(), 1e-6, cs, ref[3][None, :n], False)
        o = out[:, :, :n].double().cpu().numpy()
        assert (np.abs(o - r) <= 2.0 ** -8 * np.abs(r) + 2.0 ** -18 * np.abs(r).max()).all()
    kk = s.k.double().cpu().numpy()
    for t in range(n):
        for h in range(HKV):
            q4_write(mirror, int(ref[2][t]), h, kk[0, h, t], v[0, h, t], PAGE)
    assert np.array_equal(s.pool.cpu().numpy(), mirror)


def attend(s, o, lse, ws):
    """One new token of each request, window and sinks."""
    import masked_attention_gb300 as M
    q = s.q[0, :, :s.B].transpose(0, 1).unsqueeze(2).contiguous()   # [B, Hq, 1, D]
    M.attn_decode_q4(q, s.pool, o, lse, M.MASK_CAUSAL | M.MASK_WINDOW, page_table=s.table,
                     page_size=PAGE, seq_lens=s.lens, window=WINDOW, sink=SINK, workspace=ws)
    return q


@pytest.mark.gpu
@pytest.mark.parametrize("captured", [False, True])
def test_prompts_then_tokens(captured):
    import masked_attention_gb300 as M
    s = Server()
    mirror = np.zeros(s.pool.shape, np.uint8)
    o = torch.empty(s.B, HQ, 1, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(s.B, HQ, 1, device="cuda")
    ws = torch.empty(max(1, M.attn_decode_q4_workspace_bytes(s.B, HQ, HKV, 1, s.PER * PAGE, D)),
                     dtype=torch.uint8, device="cuda")

    def before():
        return tuple(t.cpu().numpy().copy() for t in (s.cached, s.table, s.free))

    # prompts, in two chunks of unlike sizes
    for seed, lens in ((1, [30, 0, 17]), (2, [15, 40, 3])):
        b = before()
        n = feed(s, seed, lens)
        s.write()
        check_write(s, mirror, b, lens)
        s.advance()
    # the second chunk's attention over everything cached: read the sequences
    # back packed, attend within documents, newest tokens of each
    total = int(s.lens.sum())
    own = [np.arange(x) for x in s.lens.cpu().numpy()]
    tab = s.table.cpu().numpy()
    slots = np.concatenate([tab[b, j // PAGE] * PAGE + j % PAGE for b, j in enumerate(own)])
    ks, vs = (torch.empty(1, HKV, total, D, dtype=torch.bfloat16, device="cuda") for _ in (0, 1))
    M.attn_cache_load_q4(s.pool, torch.from_numpy(slots.astype(np.int64)).cuda(), ks, vs,
                         page_size=PAGE)
    last = np.cumsum([len(x) for x in own]) - 1
    qp = torch.zeros(1, HQ, total, D, dtype=torch.bfloat16, device="cuda")
    ends = np.cumsum([15, 40, 3]) - 1     # each request's newest token in the step
    qp[:, :, last] = s.q[:, :, ends]
    of, lf = torch.empty_like(qp), torch.empty(1, HQ, total, device="cuda")
    cu = torch.from_numpy(np.concatenate([[0], last + 1]).astype(np.int32)).cuda()
    M.attn_fwd(qp, ks, vs, of, lf, M.MASK_CAUSAL | M.MASK_DOCUMENT,
               doc_id=M.doc_ids_from_seqlens(cu, total))
    q3 = s.q[0, :, ends].transpose(0, 1).unsqueeze(2).contiguous()
    M.attn_decode_q4(q3, s.pool, o, lse, M.MASK_CAUSAL, page_table=s.table, page_size=PAGE,
                     seq_lens=s.lens, workspace=ws)
    # the same attention two ways: K and V of the packed one are rounded to bf16
    assert float((of[0, :, last].transpose(0, 1).float() - o[:, :, 0].float()).abs().max()) < 3e-2
    assert float((lf[0, :, last].T - lse[:, :, 0]).abs().max()) < 3e-2

    # tokens one by one, eager or as one captured graph
    def step():
        s.write()
        attend(s, o, lse, ws)

    graph = None
    for i in range(4):
        b = before()
        feed(s, 10 + i, [1, 1, 1])
        if captured and i == 1:
            graph = torch.cuda.CUDAGraph()
            keep = s.free
            with torch.cuda.graph(graph):
                step()
            graph.replay()
        elif graph is not None:
            s.free = keep   # the graph reads this list
            graph.replay()
        else:
            step()
        check_write(s, mirror, b, [1, 1, 1])
        q = s.q[0, :, :s.B].transpose(0, 1).unsqueeze(2).double().cpu().numpy()
        O, L, A = decode_q4(q, mirror, s.table.cpu().numpy(), s.lens.cpu().numpy(), PAGE,
                            window=WINDOW, sink=SINK)
        assert np.abs(lse.double().cpu().numpy() - L).max() < 1e-3
        assert (np.abs(o.double().cpu().numpy() - O) <= 2.0 ** -8 * np.abs(O) + 2e-3 * A).all()
        if captured:   # keep the list's address for the graph: shift it in place
            used = int(s.info[1])
            s.free.copy_(torch.roll(s.free, -used))
            s.cached.copy_(s.lens)
        else:
            s.advance()


def test_chain_sizes():
    """The window and the sinks bite in the chain: lengths pass both."""
    assert 45 + 4 > WINDOW + SINK and Server.PER * PAGE >= 45 + 4
