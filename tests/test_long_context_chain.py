"""The operators for long contexts as a server runs them together: requests behind one prompt
whose pages they share, the plan of a step, norm and rotation by positions on several axes, rows
written to the bf16 paged cache, decode with the shared keys read once, the weights that the keys
received added up, eviction of the lightest behind the shared prompt, and decode from what stayed.
Every stage is checked against its fp64 oracle on the stage's own inputs; tolerances are those of
the stages' own tests (test_norm_rope, test_decode_shared, test_key_weights: derived there)."""
import numpy as np
import pytest
import torch

from oracle.long_context import (axes_rows, cached_rows, decode_rows, evict, key_weights)
from oracle.serving import norm_rope, page_plan

HQ, HKV, D, PAGE = 4, 2, 64, 16
SHARED, KEEP, RECENT, DECAY = 528, 20, 6, 0.75    # 33 whole pages, read once
AXES = bytes([0] * 10 + [1] * 12 + [2] * 10)
FAR = 1000


def table():
    f = 10000.0 ** (-np.arange(D // 2) / (D // 2))
    a = np.arange(FAR)[:, None] * f
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def f64(t):
    return t.double().cpu().numpy()


class Server:
    """Four requests, the first three behind one prompt; 560 tokens a step at most."""

    B, CAP, PAGES, PER = 4, 560, 64, 38

    def __init__(self):
        import masked_attention_gb300 as M
        i32 = dict(dtype=torch.int32, device="cuda")
        bf = dict(dtype=torch.bfloat16, device="cuda")
        B, n = self.B, self.CAP
        self.table = torch.full((B, self.PER), -1, **i32)
        self.free = torch.from_numpy(np.random.default_rng(0).permutation(self.PAGES)
                                     .astype(np.int32)).cuda()
        self.cached, self.new, self.lens = (torch.zeros(B, **i32) for _ in range(3))
        self.cu, self.info = torch.zeros(B + 1, **i32), torch.zeros(4, **i32)
        self.slots = torch.zeros(n, dtype=torch.int64, device="cuda")
        self.places, self.ids = (torch.zeros(n, **i32) for _ in (0, 1))
        self.positions = torch.full((3, 1, n), -1, **i32)   # the tokens' own, (time, height, width)
        self.k_pool, self.v_pool = (torch.full((self.PAGES, HKV, PAGE, D), float("nan"), **bf)
                                    for _ in (0, 1))        # rows that nobody wrote
        self.cos_sin = torch.from_numpy(table()).cuda()
        self.w = [torch.linspace(0.5, 1.5, D, device="cuda"),
                  torch.linspace(1.5, 0.5, D, device="cuda")]
        self.qkv = torch.zeros(1, n, HQ + 2 * HKV, D, **bf)
        self.q, self.k = (torch.zeros(1, h, n, D, **bf) for h in (HQ, HKV))
        self.starts, self.shared = torch.tensor([0, 3], **i32), torch.tensor([SHARED], **i32)
        self.o = torch.empty(B, HQ, 1, D, **bf)
        self.lse = torch.empty(B, HQ, 1, device="cuda")
        self.weights = torch.zeros(B, HKV, self.PER * PAGE, device="cuda")
        self.ws = torch.empty(M.attn_decode_shared_workspace_bytes(B, HQ, HKV, 1, 1,
                                                                   self.PER * PAGE, D),
                              dtype=torch.uint8, device="cuda")
        self.first = torch.tensor([SHARED] * 3 + [0], **i32)    # keys that eviction leaves alone
        self.kept = torch.zeros(B, HKV, KEEP, **i32)
        self.held, self.cut = torch.zeros(B, **i32), torch.zeros(2, **i32)
        self.freed = torch.full((B * self.PER,), -1, **i32)

    def parts(self):
        x = self.qkv.transpose(1, 2)
        return x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:]

    def write(self, n):
        """Plan, norm and rotation, and the rows of the step's n tokens into their slots."""
        import masked_attention_gb300 as M
        M.attn_page_plan(self.cached, self.new, self.table, self.free, self.lens, self.cu,
                         self.slots, self.places, self.ids, self.info, page_size=PAGE)
        q, k, v = self.parts()
        M.attn_qk_norm_rope_axes(q, k, self.q, self.k, q_weight=self.w[0], k_weight=self.w[1],
                                 cos_sin=self.cos_sin, positions=self.positions, axes=AXES)
        page, row = self.slots[:n] // PAGE, self.slots[:n] % PAGE
        self.k_pool[page, :, row] = self.k[0, :, :n].transpose(0, 1)
        self.v_pool[page, :, row] = v[0, :, :n].transpose(0, 1)

    def token(self):
        """One new token of each request: write, attend, add up the weights."""
        import masked_attention_gb300 as M
        self.write(self.B)
        self.query = self.q[0, :, :self.B].transpose(0, 1).unsqueeze(2).contiguous()
        cache = dict(page_table=self.table, page_size=PAGE, seq_lens=self.lens)
        M.attn_decode_shared(self.query, self.k_pool, self.v_pool, self.o, self.lse, M.MASK_CAUSAL,
                             workspace=self.ws, group_starts=self.starts, shared_lens=self.shared,
                             **cache)
        M.attn_key_weights(self.query, self.k_pool, self.lse, self.weights, M.MASK_CAUSAL,
                           previous=self.weights, decay=DECAY, **cache)

    def evict(self):
        import masked_attention_gb300 as M
        M.attn_cache_evict(self.weights, self.lens, self.k_pool, self.v_pool, self.table,
                           self.weights, self.kept, self.held, self.freed, self.cut,
                           page_size=PAGE, recent=RECENT, starts=self.first)

    def advance(self, lens):
        """The pages taken leave the free list, kept at its address; `lens` are cached now."""
        self.free.copy_(torch.roll(self.free, -int(self.info[1])))
        self.cached.copy_(lens)


def feed(s, seed, lens, positions):
    """The step's projection output, lengths and positions; the rest holds NaN and no position."""
    n = sum(lens)
    g = torch.Generator().manual_seed(seed)
    s.qkv.fill_(float("nan"))
    s.qkv[0, :n] = torch.randn(n, HQ + 2 * HKV, D, generator=g).to(torch.bfloat16).cuda()
    s.new.copy_(torch.tensor(lens, dtype=torch.int32))
    s.positions.fill_(-1)
    s.positions[:, 0, :n] = torch.from_numpy(np.asarray(positions, np.int32)).cuda()
    return n


def snapshot(s):
    return {name: getattr(s, name).cpu().clone() for name in
            ("cached", "table", "free", "k_pool", "v_pool", "weights")}


def bits(t):
    return t.cpu().view(torch.int16).numpy()


def check_write(s, b, lens):
    ref = page_plan(b["cached"].numpy(), lens, b["table"].numpy(), b["free"].numpy(), PAGE, s.CAP)
    for got, r in zip((s.lens, s.cu, s.slots, s.places, s.ids, s.table, s.info), ref):
        assert np.array_equal(got.cpu().numpy(), r)
    n = sum(lens)
    q, k, v = (f64(t[:, :, :n]) for t in s.parts())
    rows = axes_rows(f64(s.cos_sin), s.positions[:, :, :n].cpu().numpy(), AXES)
    for x, w, out in ((q, s.w[0], s.q), (k, s.w[1], s.k)):
        r = norm_rope(x, f64(w), 1e-6, rows, np.arange(n)[None], False)
        o = f64(out[:, :, :n])
        # half a step, and 2^-19 of the row's largest before the rotation, which passes that of the
        # rotated row by a factor of sqrt(2) at most
        assert (np.abs(o - r) <= 2.0 ** -8 * np.abs(r)
                + 2.0 ** -18 * np.abs(r).max(-1, keepdims=True)).all()
    # the pools: the new rows, and every other row as it was
    for pool, was, new in ((s.k_pool, b["k_pool"], s.k), (s.v_pool, b["v_pool"], s.parts()[2])):
        want = was.clone()
        for t in range(n):
            slot = int(ref[2][t])
            want[slot // PAGE, :, slot % PAGE] = new[0, :, t].cpu()
        assert np.array_equal(bits(pool), bits(want))


def check_token(s, b):
    lens, tab, q = s.lens.cpu().numpy(), s.table.cpu().numpy(), f64(s.query)
    K, V = f64(s.k_pool), f64(s.v_pool)

    def rows(pool, i, head):
        return cached_rows(pool, tab, i, int(lens[i]), head, PAGE)

    O, L, A, size = decode_rows(q, lambda i, h: (rows(K, i, h * HKV // HQ), rows(V, i, h * HKV // HQ)),
                                lens)
    E = 2.0 ** -17 * size
    assert (np.abs(f64(s.lse) - L) <= E + 2.0 ** -20 * (1 + np.abs(L))).all()
    tol = 2.0 ** -8 * np.abs(O) + (2.0 ** -8 + 2.0 ** -18 + 4 * E[..., None]) * A
    assert (np.abs(f64(s.o) - O) <= tol).all()
    ref, size = key_weights(q, lambda i, hk: rows(K, i, hk), f64(s.lse), b["weights"].double().numpy(),
                            DECAY, lens, b["weights"].double().numpy())
    assert (np.abs(f64(s.weights) - ref) <= 2.0 ** -16 * size + 2.0 ** -23 * np.abs(ref)).all()


def check_evict(s, b):
    ref = evict(b["weights"].numpy(), s.lens.cpu().numpy(), s.first.cpu().numpy(), KEEP, RECENT,
                bits(b["k_pool"]), bits(b["v_pool"]), b["table"].numpy(), PAGE, None,
                b["weights"].numpy(), np.full(len(s.freed), -1, np.int32))
    out, kept, held, freed, cut, k, v = ref
    for got, r in ((s.kept, kept), (s.held, held), (s.freed, freed), (s.cut, cut)):
        assert np.array_equal(got.cpu().numpy(), r)
    assert np.array_equal(s.weights.cpu().numpy(), out.astype(np.float32))
    assert np.array_equal(bits(s.k_pool), k) and np.array_equal(bits(s.v_pool), v)
    shared = b["table"][0, :SHARED // PAGE].long()     # nobody's rows of the prompt moved
    assert np.array_equal(bits(s.k_pool[shared.cuda()]), bits(b["k_pool"][shared]))


def image(n, start):
    """Positions of n tokens of an image of 7 columns behind `start` tokens."""
    t = np.arange(n)
    return [np.full(n, start), start + t // 7, start + t % 7]


@pytest.mark.gpu
@pytest.mark.parametrize("captured", [False, True])
def test_prompt_tokens_eviction_tokens(captured):
    import masked_attention_gb300 as M
    s = Server()
    # the shared prompt (text and an image) by the first request, and the last one's own
    text = np.arange(SHARED - 28)
    first = [np.concatenate(x) for x in zip([text] * 3, image(28, len(text)), [np.arange(9)] * 3)]
    lens = [SHARED, 0, 0, 9]
    b = snapshot(s)
    s.write(feed(s, 1, lens, first))
    check_write(s, b, lens)
    s.advance(s.lens)
    # the others hold the prompt's pages from here on; each request's own question
    s.table[1:3, :SHARED // PAGE] = s.table[0, :SHARED // PAGE]
    s.cached[1:3] = SHARED
    lens = [30, 17, 3, 11]
    at = np.concatenate([SHARED + np.arange(x) for x in lens])
    b = snapshot(s)
    s.write(feed(s, 2, lens, [at] * 3))
    check_write(s, b, lens)
    s.advance(s.lens)
    assert s.cached.tolist() == [SHARED + 30, SHARED + 17, SHARED + 3, 20]

    clock = 600     # positions of new tokens are the caller's to count, past what is evicted too
    graphs = {}

    def run(name, work):
        if not captured:
            return work()
        if name not in graphs:
            torch.cuda.synchronize()
            graphs[name] = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graphs[name]):
                work()
        graphs[name].replay()
        torch.cuda.synchronize()

    def tokens(seeds):
        nonlocal clock
        for seed in seeds:
            feed(s, seed, [1] * s.B, [[clock] * s.B] * 3)
            b = snapshot(s)
            run("token", s.token)
            assert M.attn_check_status() == M.ATTN_OK
            check_write(s, b, [1] * s.B)
            check_token(s, b)
            s.advance(s.lens)
            clock += 1

    tokens(range(10, 13))
    for turn in range(2):
        b = snapshot(s)
        s.freed.fill_(-1)
        run("evict", s.evict)
        check_evict(s, b)
        # the first request is cut (33 own keys to 20), as are the last and, later, the others
        assert int(s.cut[1]) >= 1 and (s.held <= s.first + KEEP).all()
        # the pages given up are the free list's last ones
        gone = int(s.cut[0])
        s.info.zero_()
        if gone:
            s.free[-gone:] = s.freed[:gone]
        s.advance(s.held)
        tokens(range(20 + 10 * turn, 24 + 10 * turn))


@pytest.mark.gpu
def test_two_calls_at_once():
    """Two caches of their own on two streams: equal bits to the same calls one after the other."""
    import masked_attention_gb300 as M

    def made(seed):
        from tests.test_decode_shared import Case
        c = Case([(6, 900), (3, 0)], [9 * b + 1 + seed for b in range(9)], Hq=8, Hkv=2, D=128, page=64,
                 seed=seed)
        t = {n: getattr(c, n).cuda() for n in ("q", "k", "v", "table", "lens", "starts", "shared")}
        n = c.table.shape[1] * 64
        t["ws"] = torch.empty(M.attn_decode_shared_workspace_bytes(9, 8, 2, 1, 2, n, 128),
                              dtype=torch.uint8, device="cuda")
        t["first"] = torch.tensor([896] * 6 + [0] * 3, dtype=torch.int32, device="cuda")
        return t, n

    def run(t, n, turns=1):
        i32 = dict(dtype=torch.int32, device="cuda")
        for _ in range(turns):
            k, v = t["k"].clone(), t["v"].clone()
            o, lse = torch.empty_like(t["q"]), torch.empty(9, 8, 1, device="cuda")
            w = torch.zeros(9, 2, n, device="cuda")
            kept, held = torch.zeros(9, 2, 20, **i32), torch.zeros(9, **i32)
            freed, info = torch.full((99,), -1, **i32), torch.zeros(2, **i32)
            cache = dict(page_table=t["table"], page_size=64, seq_lens=t["lens"])
            M.attn_decode_shared(t["q"], k, v, o, lse, M.MASK_CAUSAL, group_starts=t["starts"],
                                 shared_lens=t["shared"], workspace=t["ws"], **cache)
            M.attn_key_weights(t["q"], k, lse, w, M.MASK_CAUSAL, previous=w, **cache)
            M.attn_cache_evict(w, t["lens"], k, v, t["table"], w, kept, held, freed, info, page_size=64,
                               recent=3, starts=t["first"])
        return o, lse, w, kept, held, freed, info, k, v

    both = [made(1), made(2)]
    refs = [run(*x) for x in both]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in both], []
    for s, x in zip(streams, both):
        with torch.cuda.stream(s):
            outs.append(run(*x, turns=8))
    torch.cuda.synchronize()
    assert M.attn_check_status() == M.ATTN_OK
    for ref, out in zip(refs, outs):
        for a, b in zip(ref, out):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_chain_sizes():
    """Whole pages are shared, and own keys pass what eviction keeps: a page is given up."""
    own = [30 + 3, 17 + 3, 3 + 3]
    assert SHARED % PAGE == 0 and max(own) > KEEP > RECENT
    assert -(-(SHARED + own[0]) // PAGE) > -(-(SHARED + KEEP) // PAGE)
    assert SHARED + own[0] + 8 <= Server.PER * PAGE and len(AXES) == D // 2
