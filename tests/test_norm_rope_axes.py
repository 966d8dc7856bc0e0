"""attn_qk_norm_rope_axes and its gradient: positions on several axes.

The reference is the one-axis oracle with a table row of its own for every token (its
channel pairs picked from the rows of their axes), and the checks and tolerances are those
of tests/test_norm_rope.py, whose arithmetic the calls share."""
import ctypes

import numpy as np
import pytest
import torch

from oracle.long_context import axes_rows
from oracle.serving import norm_rope, norm_rope_backward
from tests.test_norm_rope import Case, check_backward, check_forward, f64, table


class AxesCase(Case):
    def __init__(self, axes, A=None, hole=(), **kw):
        super().__init__(**kw)
        B, _, _, S, D = self.shape
        A = max(axes) + 1 if A is None else A
        g = torch.Generator().manual_seed(77)
        self.source = self.table
        self.axes = bytes(axes)
        self.positions = torch.randint(0, len(self.source), (A, B, S), generator=g,
                                       dtype=torch.int32)
        for a, b, s, p in hole:
            self.positions[a, b, s] = p
        self.table = axes_rows(self.source, self.positions.numpy(), axes)

    @property
    def live(self):
        p = self.positions.numpy()
        return ((p >= 0) & (p < len(self.source))).all(0)

    def ref_pos(self):
        B, _, _, S, _ = self.shape
        return np.arange(B * S).reshape(B, S)

    def kwargs(self):
        return {**super().kwargs(), "cos_sin": torch.from_numpy(self.source).cuda(),
                "positions": self.positions.cuda(), "axes": self.axes}


@pytest.fixture
def axes_calls(monkeypatch):
    """The shared checks call the several-axes functions."""
    import masked_attention_gb300 as M
    monkeypatch.setattr(M, "attn_qk_norm_rope", M.attn_qk_norm_rope_axes)
    monkeypatch.setattr(M, "attn_qk_norm_rope_bwd", M.attn_qk_norm_rope_axes_bwd)


def runs(*n):
    return [a for a, k in enumerate(n) for _ in range(k)]


def cyclic(A, n):
    return [i % A for i in range(n)]


# rot, axis of every pair: runs on and off multiples of 4, pairs dealt out, one axis, four
LAYOUTS = [(128, runs(16, 24, 24)), (128, cyclic(3, 64)), (128, runs(1, 62, 1)),
           (64, runs(13, 19)), (64, cyclic(4, 32)), (64, runs(32)), (16, runs(3, 5)),
           (48, cyclic(2, 24)), (48, runs(5, 6, 6, 7))]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot,axes", LAYOUTS)
def test_forward_and_backward(rot, axes, inter, dtype, axes_calls):
    for i, shape in enumerate([dict(B=1, S=1, Hq=1, Hkv=1), dict(B=3, S=7, Hq=5, Hkv=1),
                               dict(B=65, S=1, Hq=8, Hkv=8), dict(B=2, S=190, Hq=6, Hkv=2)]):
        for D in {128, max(64, rot)}:
            c = AxesCase(axes, D=D, rot=rot, inter=inter, dtype=dtype, fused=i % 2 == 0, seed=i,
                         norm=i != 1, **shape)
            check_forward(c)
            check_backward(c)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
def test_equal_positions_give_the_bits_of_one_axis(inter, dtype):
    import masked_attention_gb300 as M
    for rot, axes in LAYOUTS[:5]:
        c = Case(B=2, S=150, Hq=6, Hkv=2, D=128, rot=rot, inter=inter, dtype=dtype)
        one = [torch.empty_like(t) for t in (c.dq, c.dk)]
        more = [torch.empty_like(t) for t in (c.dq, c.dk)]
        kw = c.kwargs()
        M.attn_qk_norm_rope(c.dq, c.dk, *one, **kw)
        kw["positions"] = kw["positions"].expand(4, 2, 150).contiguous()
        M.attn_qk_norm_rope_axes(c.dq, c.dk, *more, axes=axes, **kw)
        assert all(torch.equal(a, b) for a, b in zip(one, more))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bad", [-1, 1000, 2 ** 31 - 1, -2 ** 31])
def test_rows_outside_the_table_on_any_axis(bad, dtype, axes_calls):
    """Not written and without a share in the weights' gradients, whichever axis leaves the
    table, one that no channel pair uses among them."""
    hole = [(0, 0, 1, bad), (1, 0, 2, bad), (2, 1, 0, bad), (3, 1, 2, bad)]
    c = AxesCase(runs(16, 24, 24), A=4, hole=hole, B=2, S=4, Hq=3, Hkv=1, dtype=dtype)
    assert c.live.sum() == 4
    check_forward(c)
    check_backward(c)


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(B=3, S=1667, Hq=20, Hkv=7, D=128),
                                dict(B=1667, S=3, Hq=9, Hkv=2, D=64, rot=32),
                                dict(B=2, S=2501, Hq=5, Hkv=5, D=64, inter=True),
                                dict(B=5, S=1001, Hq=6, Hkv=1, D=128, dtype=torch.float32)])
def test_blocks_with_many_items(kw, axes_calls):
    rot = kw.get("rot", kw["D"])
    B, S = kw["B"], kw["S"]
    hole = [(i % 3, i * 7 % B, i * 11 % S, (-1, 1000)[i % 2]) for i in range(B * S // 9)]
    c = AxesCase(cyclic(3, rot // 2), hole=hole, seed=9, **{"rot": rot, **kw})
    check_forward(c)
    check_backward(c)


@pytest.mark.gpu
def test_infinities_and_nan_stay_in_their_channels():
    """Without a norm a pair that holds an infinity or NaN keeps it to itself."""
    import masked_attention_gb300 as M
    axes = runs(3, 5)
    c = AxesCase(axes, B=1, S=12, Hq=3, Hkv=1, D=64, rot=16, norm=False, fused=False)
    q = c.q.clone()
    for i in range(36):
        q[0, i // 12, i % 12, (7 * i) % 64] = (float("inf"), -float("inf"), float("nan"))[i % 3]
    o = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    M.attn_qk_norm_rope_axes(q.cuda(), None, o, None, **c.kwargs())
    with np.errstate(invalid="ignore"):
        ref = norm_rope(f64(q), None, c.eps, c.table.astype(np.float64), c.ref_pos(), False)
    got = f64(o.cpu())
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.array_equal(np.isinf(got), np.isinf(ref))


@pytest.mark.gpu
def test_in_place_other_stream_and_captured(axes_calls):
    """In place with equal bits; a captured forward and gradient replay on new contents."""
    import masked_attention_gb300 as M
    c = AxesCase(runs(16, 24, 24), B=4, S=100, Hq=8, Hkv=4)
    outs = check_forward(c)
    (dq, dk), (dwq, dwk) = check_backward(c)
    q, k = c.dq.clone(), c.dk.clone()
    keep = q.clone(), k.clone()
    grads = [torch.empty_like(t) for t in (dq, dk, dwq, dwk)]
    ws = torch.empty(M.attn_qk_norm_rope_bwd_workspace_bytes(128), dtype=torch.uint8, device="cuda")
    kw, g0, g1 = c.kwargs(), c.gq.cuda(), c.gk.cuda()

    def call():
        M.attn_qk_norm_rope_axes_bwd(q, k, g0, g1, grads[0], grads[1], dq_weight=grads[2],
                                     dk_weight=grads[3], workspace=ws, **kw)
        M.attn_qk_norm_rope_axes(q, k, q, k, **kw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for _ in range(2):
        q.copy_(keep[0])
        k.copy_(keep[1])
        ws.fill_(0xff)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(q, outs[0]) and torch.equal(k, outs[1])
        assert all(torch.equal(a, b) for a, b in zip(grads, (dq, dk, dwq, dwk)))


def test_oracle_gradient_against_differences():
    rng = np.random.default_rng(1)
    x, dz, w = rng.normal(size=(1, 2, 2, 64)), rng.normal(size=(1, 2, 2, 64)), rng.normal(size=64)
    pos = rng.integers(0, 50, (3, 1, 2))
    rows = axes_rows(table(50, 32).astype(np.float64), pos, cyclic(3, 16))
    at = np.arange(2)[None]
    for inter in (False, True):
        f = lambda x, w: float((dz * norm_rope(x, w, 1e-3, rows, at, inter)).sum())  # noqa: E731
        dx, dw = norm_rope_backward(x, dz, w, 1e-3, rows, at, inter)
        for idx in [(0, 0, 0, 0), (0, 1, 1, 17), (0, 0, 1, 40), (0, 1, 0, 63)]:
            e = np.zeros_like(x)
            e[idx] = 1e-6
            assert abs((f(x + e, w) - f(x - e, w)) / 2e-6 - dx[idx]) < 1e-7
        for i in (0, 5, 33):
            e = np.zeros(64)
            e[i] = 1e-6
            assert abs((f(x, w + e) - f(x, w - e)) / 2e-6 - dw[i]) < 1e-7


def test_oracle_rows_by_hand():
    tab = np.arange(40.0).reshape(10, 4)          # two pairs
    rows = axes_rows(tab, np.array([[[3, 9]], [[5, 0]]]), [1, 0])
    assert rows.tolist() == [[20, 13, 22, 15], [0, 37, 2, 39]]


def test_refusals():
    import masked_attention_gb300 as M
    L = M.lib()

    def fwd(axes=3, pairs=bytes(64), bwd=False, **kw):
        p = M.attn_rope_params(M.BF16, 1e-6, None, None, 0x9000, 64, 128, 0, 0xa000)
        for n, v in kw.items():
            setattr(p, n, v)
        v = ctypes.byref(M.attn_view(0x1000, 4096, 1024, 128))
        if bwd:
            return L.attn_qk_norm_rope_axes_bwd(
                v, v, v, v, v, v, None, None, 0x100000,
                M.attn_qk_norm_rope_bwd_workspace_bytes(128), 1, 2, 1, 8, 128, ctypes.byref(p),
                axes, pairs, None)
        return L.attn_qk_norm_rope_axes(v, v, v, v, 1, 2, 1, 8, 128, ctypes.byref(p), axes, pairs,
                                        None)

    inv = M.ATTN_ERR_INVALID_ARG
    for bwd in (False, True):
        assert fwd(axes=0, bwd=bwd) == fwd(axes=5, bwd=bwd) == fwd(axes=-1, bwd=bwd) == inv
        assert fwd(pairs=None, bwd=bwd) == fwd(pairs=bytes(63) + b"\x03", bwd=bwd) == inv
        assert fwd(cos_sin=None, bwd=bwd) == fwd(positions=None, bwd=bwd) == inv
        assert fwd(rot_dim=24, bwd=bwd) == M.ATTN_ERR_UNSUPPORTED
        assert fwd(positions=0xa002, bwd=bwd) == M.ATTN_ERR_MISALIGNED
    t = torch.zeros(1, 1, 1, 64)
    with pytest.raises(ValueError):
        M.attn_qk_norm_rope_axes(t, t, t, t, cos_sin=t, positions=t, axes=[0])   # not on a GPU


@pytest.mark.gpu
def test_refusals_of_tensors():
    import masked_attention_gb300 as M
    c = AxesCase(runs(16, 24, 24), B=2, S=3, Hq=2, Hkv=1)
    kw = c.kwargs()

    def refused(**bad):
        with pytest.raises((ValueError, M.AttnError)):
            M.attn_qk_norm_rope_axes(c.dq, c.dk, torch.empty_like(c.dq), torch.empty_like(c.dk),
                                     **{**kw, **bad})

    refused(positions=kw["positions"][0])
    refused(positions=kw["positions"][:, :, :2].contiguous())
    refused(positions=kw["positions"].long())
    refused(positions=kw["positions"].transpose(1, 2))
    refused(positions=torch.zeros(5, 2, 3, dtype=torch.int32, device="cuda"))
    refused(axes=c.axes[:-1])
    refused(axes=[3] * 64)
    refused(cos_sin=kw["cos_sin"][:, :64].contiguous())
    refused(positions=None)
