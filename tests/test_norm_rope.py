"""attn_qk_norm_rope and its gradient against the fp64 oracle.

Tolerances. An output is rounded once: half a step of its type, 2^-8 |ref| for
bf16 and 2^-24 |ref| for fp32. Before that, fp32 arithmetic: the mean of
squares (a tree over D <= 128 channels) and rsqrt leave the row's factor within
8 * 2^-24, the products and the rotation (two products, one sum) add 4 * 2^-24
of |y| + |y'|, in all below 2^-20 (|y| + |y'|) <= 2^-19 max|y| of the row. The
gradient's row term is a difference of dn and n mean(dn n), each within
2^-20 of its size: 2^-18 r (max|dn| + max|n| mean|dn n|) covers both and the
rotation before. A weight's gradient is a sum of n terms dy x r: in any order
its error is at most n 2^-24 sum|term|, and each term is within 16 * 2^-24 of its
size. That size is not |dy x r|: dy = a cos + b sin is a sum of two rounded
products, fl(fl(a cos) + fl(b sin)) = dy + e with |e| <= 2^-24 (|a cos| + |b sin| +
|dy|) (1 + 2^-24), which where the products cancel is far above 2^-24 |dy|. So the size
is (|a cos| + |b sin|) |x r| >= |term|."""
import numpy as np
import pytest
import torch

from oracle.serving import norm_rope, norm_rope_backward, rotate
from tests.helpers import check_canaries, guarded_empty

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def table(max_pos, rot, base=10000.0):
    f = base ** (-np.arange(rot // 2) / (rot // 2))
    a = np.arange(max_pos)[:, None] * f
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


class Case:
    """Seeded inputs; q, k are slices of one fused tensor when asked for."""

    def __init__(self, B=2, S=5, Hq=4, Hkv=2, D=128, rot=None, inter=False, dtype=torch.bfloat16,
                 norm=True, fused=True, eps=1e-6, pos="random", max_pos=1000, seed=0, scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.shape, self.dtype, self.inter, self.eps = (B, Hq, Hkv, S, D), dtype, inter, eps
        qkv = (torch.randn(B, S, Hq + 2 * Hkv, D, generator=g) * scale).to(dtype)
        self.q, self.k = (t.transpose(1, 2) for t in (qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv]))
        dev = qkv.cuda()
        self.dq, self.dk = (t.transpose(1, 2) for t in (dev[:, :, :Hq], dev[:, :, Hq:Hq + Hkv]))
        if not fused:
            self.dq, self.dk = self.dq.contiguous(), self.dk.contiguous()
        self.gq, self.gk = (torch.randn(B, H, S, D, generator=g).to(dtype) for H in (Hq, Hkv))
        self.w = [(1 + 0.3 * torch.randn(D, generator=g)) if norm else None for _ in (0, 1)]
        rot = D if rot is None else rot
        self.table = table(max_pos, rot) if rot else None
        if pos == "random":
            self.pos = torch.randint(0, max_pos, (B, S), generator=g, dtype=torch.int32)
        elif pos == "none":
            self.pos = None
        else:
            self.pos = torch.tensor(pos, dtype=torch.int32).view(B, S)

    @property
    def live(self):
        B, _, _, S, _ = self.shape
        if self.table is None or self.pos is None:
            return np.ones((B, S), bool)
        p = self.pos.numpy()
        return (p >= 0) & (p < len(self.table))

    def kwargs(self):
        return dict(q_weight=None if self.w[0] is None else self.w[0].cuda(),
                    k_weight=None if self.w[1] is None else self.w[1].cuda(), eps=self.eps,
                    cos_sin=None if self.table is None else torch.from_numpy(self.table).cuda(),
                    positions=None if self.pos is None else self.pos.cuda(),
                    interleaved=self.inter)

    def ref_pos(self):
        B, _, _, S, _ = self.shape
        p = np.broadcast_to(np.arange(S), (B, S)) if self.pos is None else self.pos.numpy()
        return np.where(self.live, p, 0)


def turned_size(dz, c):
    """|a cos| + |b sin| of every channel of the rotated-back dz."""
    if c.table is None:
        return np.abs(dz)
    tab = np.abs(c.table.astype(np.float64))
    half = tab.shape[1] // 2
    tab[:, half:] *= -1   # rotating forward by -|sin| and back by it both add
    a = rotate(np.abs(dz), tab, c.ref_pos()[:, None], c.inter)
    b = rotate(np.abs(dz), tab, c.ref_pos()[:, None], c.inter, back=True)
    return np.maximum(a, b)


def f64(t):
    return t.double().numpy()


def check_forward(c, **extra):
    import masked_attention_gb300 as M
    outs = [guarded_empty(t.shape, c.dtype) for t in (c.q, c.k)]
    for o in outs:
        o.fill_(7.0)
    M.attn_qk_norm_rope(c.dq, c.dk, *outs, **{**c.kwargs(), **extra})
    check_canaries()
    for x, w, o in zip((c.q, c.k), c.w, outs):
        w = None if w is None else f64(w)
        tab = None if c.table is None else c.table.astype(np.float64)
        ref = norm_rope(f64(x), w, c.eps, tab, c.ref_pos(), c.inter)
        y = norm_rope(f64(x), w, c.eps, None, None, c.inter)
        got = f64(o.cpu())
        tol = HALF[c.dtype] * np.abs(ref) + 2.0 ** -19 * np.abs(y).max(-1, keepdims=True)
        live = c.live[:, None, :, None]
        assert (np.abs(got - ref) <= tol)[np.broadcast_to(live, ref.shape)].all()
        assert (got == 7.0)[np.broadcast_to(~live, ref.shape)].all()   # left as they were
    return outs


def check_backward(c):
    import masked_attention_gb300 as M
    B, Hq, Hkv, S, D = c.shape
    outs = [guarded_empty((B, S, H, D), c.dtype).transpose(1, 2) for H in (Hq, Hkv)]
    for o in outs:
        o.fill_(7.0)
    dws = [None if w is None else guarded_empty((D,), torch.float32) for w in c.w]
    ws = torch.empty(M.attn_qk_norm_rope_bwd_workspace_bytes(D), dtype=torch.uint8, device="cuda")
    M.attn_qk_norm_rope_bwd(c.dq, c.dk, c.gq.cuda(), c.gk.cuda(), *outs, dq_weight=dws[0],
                            dk_weight=dws[1], workspace=ws, **c.kwargs())
    check_canaries()
    tab = None if c.table is None else c.table.astype(np.float64)
    live = c.live[:, None, :, None]
    for x, dz, w, o, dw in zip((c.q, c.k), (c.gq, c.gk), c.w, outs, dws):
        w = None if w is None else f64(w)
        dz = f64(dz) * live
        ref, dw_ref = norm_rope_backward(f64(x), dz, w, c.eps, tab, c.ref_pos(), c.inter)
        got = f64(o.cpu())
        dn = dz if tab is None else rotate(dz, tab, c.ref_pos()[:, None], c.inter, back=True)
        if w is None:
            tol = HALF[c.dtype] * np.abs(ref) + 2.0 ** -19 * np.abs(dn).max(-1, keepdims=True)
        else:
            r = 1 / np.sqrt((f64(x) ** 2).mean(-1, keepdims=True) + c.eps)
            n = f64(x) * r
            terms = turned_size(dz, c) * np.abs(n)
            tol_w = (terms[..., 0].size + 16) * 2.0 ** -24 * terms.sum((0, 1, 2))
            assert (np.abs(f64(dw.cpu()) - dw_ref) <= tol_w).all()
            dn = dn * w
            size = np.abs(dn).max(-1, keepdims=True) + (
                np.abs(n).max(-1, keepdims=True) * np.abs(dn * n).mean(-1, keepdims=True))
            tol = HALF[c.dtype] * np.abs(ref) + 2.0 ** -18 * r * size
        m = np.broadcast_to(live, ref.shape)
        assert (np.abs(got - ref) <= tol)[m].all()
        assert (got == 7.0)[~m].all()
    return outs, dws


SHAPES = [dict(B=1, S=1, Hq=1, Hkv=1), dict(B=3, S=7, Hq=5, Hkv=1), dict(B=1, S=33, Hq=14, Hkv=2),
          dict(B=65, S=1, Hq=8, Hkv=8), dict(B=2, S=300, Hq=12, Hkv=4)]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
def test_forward_and_backward(shape, D, dtype, inter):
    for i, rot in enumerate((D, D // 2, 16, 48)):
        c = Case(D=D, dtype=dtype, inter=inter, rot=rot, fused=i % 2 == 0, seed=i, **shape)
        check_forward(c)
        check_backward(c)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kw", [dict(norm=False), dict(rot=0), dict(pos="none"),
                                dict(pos="none", rot=32, norm=False), dict(eps=0.0),
                                dict(scale=1e-4), dict(scale=100.0)])
def test_without_parts(dtype, kw):
    c = Case(dtype=dtype, B=2, S=9, Hq=6, Hkv=3, **kw)
    check_forward(c)
    check_backward(c)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Batch elements 4 GiB apart, in and out: the bits of a compact call."""
    import masked_attention_gb300 as M
    B, H, S, D = 2, 3, 5, 128
    c = Case(B, S, H, H, D, fused=False)

    def far(x=None):
        t = torch.empty((1 << 31) + H * S * D, dtype=c.dtype, device="cuda").as_strided(
            (B, H, S, D), (1 << 31, S * D, D, 1))
        return t if x is None else t.copy_(x)

    outs = check_forward(c)
    o = far()
    M.attn_qk_norm_rope(far(c.dq), None, o, None, **c.kwargs())
    assert torch.equal(o, outs[0])
    (gq, _), _ = check_backward(c)
    dx, dw = far(), torch.empty(D, device="cuda")
    ws = torch.empty(M.attn_qk_norm_rope_bwd_workspace_bytes(D), dtype=torch.uint8, device="cuda")
    M.attn_qk_norm_rope_bwd(far(c.dq), None, far(c.gq.cuda()), None, dx, None, dq_weight=dw,
                            workspace=ws, **c.kwargs())
    assert torch.equal(dx, gq)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_outside_the_table(dtype):
    """Padded places (position -1 or past the table): not written, no share in
    the weights' gradients."""
    for pos in ([0, 5, -1, 999, 1000, 2 ** 31 - 1], [-1] * 6):
        c = Case(B=2, S=3, Hq=3, Hkv=1, dtype=dtype, pos=pos)
        check_forward(c)
        check_backward(c)


@pytest.mark.gpu
def test_zero_rows():
    """x = 0: y = 0 with eps > 0; the gradient of such a row is dn / sqrt(eps)."""
    c = Case(B=1, S=4, Hq=2, Hkv=1, eps=1e-2)
    c.q[:, :, 1] = 0
    c.dq[:, :, 1] = 0
    check_forward(c)
    check_backward(c)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_in_place_and_queries_alone(dtype):
    import masked_attention_gb300 as M
    c = Case(B=2, S=40, Hq=6, Hkv=2, dtype=dtype)
    outs = check_forward(c)
    q, k = c.dq.clone(memory_format=torch.preserve_format), c.dk.clone()
    M.attn_qk_norm_rope(q, k, q, k, **c.kwargs())
    assert torch.equal(q, outs[0]) and torch.equal(k, outs[1])
    o = torch.empty_like(outs[0])
    M.attn_qk_norm_rope(c.dq, None, o, None, **c.kwargs())
    assert torch.equal(o, outs[0])
    (dq, _), (dwq, _) = check_backward(c)
    g, dw = c.gq.cuda(), torch.empty_like(dwq)
    ws = torch.empty(M.attn_qk_norm_rope_bwd_workspace_bytes(128), dtype=torch.uint8,
                     device="cuda")
    M.attn_qk_norm_rope_bwd(c.dq, None, g, None, g, None, dq_weight=dw, workspace=ws, **c.kwargs())
    assert torch.equal(g, dq)
    # another order of the sum than with the keys' rows: the sum's own bound
    assert float((dw - dwq).abs().max()) <= 2 * 480 * 2.0 ** -24 * float(dwq.abs().sum() + 480 * 8)


@pytest.mark.gpu
def test_shared_head_broadcast_input():
    """A stride of 0 (one key head read as several) is an input like any other."""
    import masked_attention_gb300 as M
    c = Case(B=2, S=6, Hq=4, Hkv=1)
    k4 = c.dk.expand(2, 4, 6, 128)
    a, b = (torch.empty(2, 4, 6, 128, dtype=c.dtype, device="cuda") for _ in (0, 1))
    M.attn_qk_norm_rope(c.dq, k4, a, b, **c.kwargs())
    _, one = check_forward(c)
    assert torch.equal(b, one.expand(2, 4, 6, 128))


@pytest.mark.gpu
def test_gradient_is_reproducible_and_captures():
    """Bitwise equal runs; a captured graph replays on another stream's inputs."""
    import masked_attention_gb300 as M
    c = Case(B=4, S=500, Hq=8, Hkv=4)
    (dq, dk), (dwq, dwk) = check_backward(c)
    outs = [torch.empty_like(t) for t in (dq, dk, dwq, dwk)]
    ws = torch.empty(M.attn_qk_norm_rope_bwd_workspace_bytes(128), dtype=torch.uint8,
                     device="cuda")
    gq, gk, kw = c.gq.cuda(), c.gk.cuda(), c.kwargs()

    def call():
        M.attn_qk_norm_rope_bwd(c.dq, c.dk, gq, gk, outs[0], outs[1], dq_weight=outs[2],
                                dk_weight=outs[3], workspace=ws, **kw)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(2):
        for t in outs:
            t.fill_(3.0)
        ws.fill_(0xff)   # its contents need not be kept
        g.replay()
        torch.cuda.synchronize()
        for got, ref in zip(outs, (dq, dk, dwq, dwk)):
            assert torch.equal(got, ref)


@pytest.mark.gpu
def test_empty_calls():
    import masked_attention_gb300 as M
    e = torch.empty(2, 3, 0, 64, dtype=torch.bfloat16, device="cuda")
    M.attn_qk_norm_rope(e, e, e, e)
    w, dw = torch.ones(64, device="cuda"), torch.full((64,), 5.0, device="cuda")
    ws = torch.empty(M.attn_qk_norm_rope_bwd_workspace_bytes(64), dtype=torch.uint8, device="cuda")
    M.attn_qk_norm_rope_bwd(e, e, e, e, e, e, q_weight=w, dq_weight=dw, workspace=ws)
    assert (dw == 0).all()   # a sum over no rows


def test_oracle_gradient_against_differences():
    """Central differences of the oracle's forward, every input and weight."""
    rng = np.random.default_rng(1)
    x, dz, w = rng.normal(size=(1, 2, 2, 64)), rng.normal(size=(1, 2, 2, 64)), rng.normal(size=64)
    tab, pos = table(50, 32).astype(np.float64), np.array([[3, 41]])
    for inter in (False, True):
        f = lambda x, w: float((dz * norm_rope(x, w, 1e-3, tab, pos, inter)).sum())  # noqa: E731
        dx, dw = norm_rope_backward(x, dz, w, 1e-3, tab, pos, inter)
        h = 1e-6
        for idx in [(0, 0, 0, 0), (0, 1, 1, 17), (0, 0, 1, 40), (0, 1, 0, 63)]:
            e = np.zeros_like(x)
            e[idx] = h
            assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - dx[idx]) < 1e-7
        for i in (0, 5, 33, 63):
            e = np.zeros(64)
            e[i] = h
            assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - dw[i]) < 1e-7


def test_oracle_rotation_keeps_relative_position():
    """Scores of rotated rows depend on the distance alone."""
    rng = np.random.default_rng(2)
    q, k = rng.normal(size=(2, 1, 1, 1, 64))
    tab = table(200, 64).astype(np.float64)
    for inter in (False, True):
        s = [float((norm_rope(q, None, 0, tab, np.array([[p + 7]]), inter) *
                    norm_rope(k, None, 0, tab, np.array([[p]]), inter)).sum()) for p in (0, 90)]
        assert abs(s[0] - s[1]) < 1e-5 * abs(q).sum()   # the table itself is fp32


def test_outputs_whose_rows_share_a_place_are_refused():
    """A broadcast tensor is an input only, and an output that starts where its
    input does has its strides."""
    import ctypes
    import masked_attention_gb300 as M
    L = M.lib()
    good, other = (4096, 1024, 128), (8192, 1024, 128)

    def call(fn, out, x=good, data=0x100000, B=2, H=4):
        p = M.attn_rope_params(M.BF16, 1e-6, None, None, 0x9000, 64, 128, 0, None)
        i, o = ctypes.byref(M.attn_view(0x1000, *x)), ctypes.byref(M.attn_view(data, *out))
        if fn == "fwd":
            return L.attn_qk_norm_rope(i, None, o, None, B, H, 0, 8, 128, ctypes.byref(p), None)
        return L.attn_qk_norm_rope_bwd(None, None, i, None, o, None, None, None, 0x200000,
                                       M.attn_qk_norm_rope_bwd_workspace_bytes(128), B, H, 0, 8,
                                       128, ctypes.byref(p), None)

    for fn in ("fwd", "bwd"):
        for out in ((0, 1024, 128), (4096, 0, 128), (4096, 1024, 0)):
            assert call(fn, out) == M.ATTN_ERR_INVALID_ARG, (fn, out)
        assert call(fn, other, data=0x1000) == M.ATTN_ERR_INVALID_ARG
        assert call(fn, good, x=(0, 1024, 128), data=0x1000) == M.ATTN_ERR_INVALID_ARG


def test_refusals():
    import ctypes
    import masked_attention_gb300 as M
    L = M.lib()

    def params(**kw):
        p = M.attn_rope_params()
        p.dtype, p.eps, p.cos_sin, p.max_pos, p.rot_dim = M.BF16, 1e-6, 0x9000, 64, 128
        for n, v in kw.items():
            setattr(p, n, v)
        return p

    def fwd(D=128, B=1, Hq=2, Hkv=1, S=8, data=0x1000, strides=(4096, 1024, 128), **kw):
        v = ctypes.byref(M.attn_view(data, *strides))
        return L.attn_qk_norm_rope(v, v, v, v, B, Hq, Hkv, S, D, ctypes.byref(params(**kw)), None)

    inv, uns, mis = M.ATTN_ERR_INVALID_ARG, M.ATTN_ERR_UNSUPPORTED, M.ATTN_ERR_MISALIGNED
    assert fwd(D=96) == fwd(dtype=7) == fwd(rot_dim=8) == fwd(rot_dim=144) == fwd(rot_dim=24) == uns
    assert fwd(B=-1) == fwd(Hq=-1) == fwd(S=-1) == fwd(eps=float("nan")) == fwd(eps=-1.0) == inv
    assert fwd(max_pos=0) == fwd(max_pos=7) == inv        # fewer rows than the default positions
    assert fwd(data=None) == fwd(strides=(4096, -128, 128)) == inv
    assert fwd(data=0x1008) == fwd(strides=(4096, 1024, 132)) == fwd(strides=(0, 1004, 128)) == mis
    assert fwd(cos_sin=0x9008) == fwd(q_weight=0x2002) == fwd(positions=0x2001) == mis
    assert fwd(B=0) == fwd(S=0) == M.ATTN_OK              # nothing to do, nothing launched

    def bwd(ws=0x100000, n=None, dqw=0x8000, dkw=None, **kw):
        v = ctypes.byref(M.attn_view(0x1000, 4096, 1024, 128))
        n = M.attn_qk_norm_rope_bwd_workspace_bytes(128) if n is None else n
        kw = {"q_weight": 0x7000, **kw}
        return L.attn_qk_norm_rope_bwd(v, v, v, v, v, v, dqw, dkw, ws, n, 1, 2, 1, 8, 128,
                                       ctypes.byref(params(**kw)), None)

    assert bwd(ws=None) == inv and bwd(ws=0x100010) == mis
    assert bwd(n=8) == M.ATTN_ERR_WORKSPACE_TOO_SMALL
    assert bwd(dkw=0x8000) == inv                         # a gradient of no weight
    assert bwd(dqw=0x8001) == mis
    assert M.attn_qk_norm_rope_bwd_workspace_bytes(96) == 0
    t = torch.zeros(1, 1, 1, 64)
    with pytest.raises(ValueError):
        M.attn_qk_norm_rope(t, t, t, t)                   # not on a GPU
    with pytest.raises(ValueError):
        M.attn_qk_norm_rope(t.half(), t, t, t)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("without", ["keys", "queries"])
def test_weight_gradient_of_a_side_without_heads(without, dtype, D):
    """A sum over no rows is 0, whatever the workspace held."""
    import masked_attention_gb300 as M
    c = Case(B=2, S=70, Hq=3, Hkv=3, D=D, dtype=dtype)
    (dq, dk), (dwq, dwk) = check_backward(c)
    ws = torch.full((M.attn_qk_norm_rope_bwd_workspace_bytes(D),), 0xff, dtype=torch.uint8,
                    device="cuda")
    dws = [torch.full((D,), 5.0, device="cuda") for _ in (0, 1)]
    gq, gk, kw = c.gq.cuda(), c.gk.cuda(), c.kwargs()
    kw.update(dq_weight=dws[0], dk_weight=dws[1], workspace=ws)
    if without == "keys":
        out = torch.empty_like(dq)
        M.attn_qk_norm_rope_bwd(c.dq, None, gq, None, out, None, **kw)
        assert torch.equal(out, dq) and (dws[1] == 0).all()
        size = turned_size(f64(c.gq), c) * np.abs(f64(c.q)) / np.sqrt(
            (f64(c.q) ** 2).mean(-1, keepdims=True))
        # another order of the sum than with the keys' rows: twice the sum's own bound
        tol = 2 * (size[..., 0].size + 16) * 2.0 ** -24 * size.sum((0, 1, 2))
        assert (np.abs(f64(dws[0].cpu()) - f64(dwq.cpu())) <= tol).all()
    else:
        none, out = c.dq[:, :0], torch.empty_like(dk)
        M.attn_qk_norm_rope_bwd(none, c.dk, gq[:, :0], gk, none, out, **kw)
        assert torch.equal(out, dk) and (dws[0] == 0).all() and torch.isfinite(dws[1]).all()


def same_kind(got, ref, tol):
    """Equal infinities and NaN; elsewhere within tol."""
    f = np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.array_equal(np.isposinf(got), np.isposinf(ref))
    assert np.array_equal(np.isneginf(got), np.isneginf(ref))
    assert (np.abs(got - ref)[f] <= np.broadcast_to(tol, ref.shape)[f]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [0, 16, 48])
@pytest.mark.parametrize("norm", [False, True])
def test_infinities_and_nan_stay_in_their_channels(norm, rot, inter, dtype, D):
    """A channel that is not rotated passes by itself: what a neighbour of it holds, in the
    input or the gradient, does not reach it. With a norm an infinite channel makes the row's
    others 0, a NaN all of them NaN."""
    import masked_attention_gb300 as M
    c = Case(B=1, S=12, Hq=3, Hkv=1, D=D, dtype=dtype, norm=norm, rot=rot, inter=inter, fused=False,
             pos=list(range(1, 13)))
    tab = None if c.table is None else c.table.astype(np.float64)
    bad = [float("inf"), -float("inf"), float("nan")]
    places = [(s, (7 * s + 5 * h) % D, bad[(s + h) % 3]) for h in range(3) for s in range(12)]
    q, g = c.q.clone(), c.gq.clone()
    for i, (s, ch, x) in enumerate(places):
        if s % 4:    # some rows stay finite
            q[0, i // 12, s, ch] = x
            g[0, i // 12, s, (ch + 3) % D] = x
    o = torch.empty(q.shape, dtype=dtype, device="cuda")
    kw = c.kwargs()
    w = None if c.w[0] is None else f64(c.w[0])
    with np.errstate(invalid="ignore", over="ignore"):
        M.attn_qk_norm_rope(q.cuda(), None, o, None, **kw)
        ref = norm_rope(f64(q), w, c.eps, tab, c.ref_pos(), inter)
        y = np.nan_to_num(norm_rope(f64(q), w, c.eps, None, None, inter), nan=0, posinf=0, neginf=0)
        size = 2.0 ** -19 * np.abs(y).max(-1, keepdims=True)
        same_kind(f64(o.cpu()), ref, HALF[dtype] * np.abs(ref) + size)
        if norm:    # finite inputs, gradients that are not: which outputs stay finite
            q = c.q
        dx, dw = torch.empty_like(o), torch.empty(D, device="cuda")
        ws = torch.empty(M.attn_qk_norm_rope_bwd_workspace_bytes(D), dtype=torch.uint8, device="cuda")
        M.attn_qk_norm_rope_bwd(q.cuda(), None, g.cuda(), None, dx, None, workspace=ws,
                                dq_weight=dw if norm else None, **kw)
        ref, dw_ref = norm_rope_backward(f64(q), f64(g), w, c.eps, tab, c.ref_pos(), inter)
        if norm:
            assert np.array_equal(np.isfinite(f64(dx.cpu())), np.isfinite(ref))
            assert np.array_equal(np.isfinite(f64(dw.cpu())), np.isfinite(dw_ref))
        else:
            size = 2.0 ** -19 * np.abs(np.nan_to_num(f64(g), nan=0, posinf=0, neginf=0)).max(
                -1, keepdims=True)
            same_kind(f64(dx.cpu()), ref, HALF[dtype] * np.abs(ref) + size)


LONG = [dict(B=3, S=1667, Hq=20, Hkv=7, D=128), dict(B=1667, S=3, Hq=9, Hkv=2, D=64, rot=32),
        dict(B=2, S=2501, Hq=5, Hkv=5, D=64, inter=True), dict(B=2, S=2499, Hq=1, Hkv=14, D=128, rot=48),
        dict(B=5, S=1001, Hq=6, Hkv=1, D=128, dtype=torch.float32),
        dict(B=411, S=13, Hq=10, Hkv=3, D=64, dtype=torch.float32, inter=True, rot=16)]


@pytest.mark.gpu
@pytest.mark.parametrize("kw", LONG)
def test_blocks_with_many_items(kw):
    """Thousands of tokens: a block goes through several items of several tokens, over the
    sequences' ends, with rows outside the table on its way."""
    c = Case(seed=9, **kw)
    gone = torch.rand(c.pos.shape, generator=torch.Generator().manual_seed(1)) < 0.2
    c.pos[gone] = torch.where(torch.arange(int(gone.sum())) % 2 == 0, -1, len(c.table)).to(torch.int32)
    check_forward(c)
    check_backward(c)
