"""The operators around the paged key/value cache, each as a measured case: the page plan built
from request lengths, the per-head norm with the position rotation (forward and backward), the
4-bit cache's write and read, and decode attention over that cache.

``run`` computes a case with elementary torch operations when ``own`` is false and through the
framework's public calls when it is true. ``exact`` gives the same outputs from the definitions
in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
GROUP = 32  # channels that share one scale in the 4-bit cache
WORKSPACE = 1 << 28  # bytes of the one workspace that a program keeps for its largest call


def _case(name, op, **kw):
    return dict(name=name, op=op, **kw)


def listed():
    return [
        # a serving step of 64 requests: every one gets one more token, a few need a new page
        _case("plan step 64", "plan", B=64, ps=16, cached=8000, new=1, cap=64),
        # chunked prompts of 500 requests scheduled together, ragged, into a fixed token budget
        _case("plan prompts 500", "plan", B=500, ps=16, cached=3000, new=256, cap=65536),
        # queries and keys of one new token for 32 requests, from a fused projection
        _case("rope step 32", "rope", B=32, S=1, Hq=32, Hkv=8, D=128, rot=128, f32=False,
              inter=False, norm=True, fused=True, far=32768, pad=0),
        # a packed prompt of 16384 tokens, from a fused projection into the attention's layout
        _case("rope prompt 16384", "rope", B=1, S=16384, Hq=32, Hkv=8, D=128, rot=128, f32=False,
              inter=False, norm=True, fused=True, far=131072, pad=0),
        # a training step's backward at the training workload's shape
        _case("rope backward train", "rope_bwd", B=8, S=4096, Hq=16, Hkv=16, D=128, rot=128,
              f32=False, inter=False, norm=True, fused=False, far=4096, pad=0),
        # a small fp32 backward: odd length, grouped heads, half of the channels rotated
        _case("rope backward f32 odd", "rope_bwd", B=2, S=333, Hq=8, Hkv=2, D=64, rot=32,
              f32=True, inter=True, norm=True, fused=True, far=2048, pad=7),
        # a prompt chunk is written to the cache and read back for the chunk's own attention
        _case("cache prompt 16384", "cache", T=16384, Hkv=8, D=128, ps=64, pad=0),
        # the new tokens of 47 requests in a batch padded to 48
        _case("cache step 48", "cache", T=48, Hkv=8, D=64, ps=16, pad=1),
        # one short conversation, one new token
        _case("decode 1 x 700", "decode", B=1, Hq=16, Hkv=2, Sq=1, D=64, ps=16, longest=700,
              ragged=False, window=0, sink=0, softcap=0.0, alibi=False),
        # the decode workload: 16 sequences of a 32768-token cache, one new token each
        _case("decode 16 x 32768", "decode", B=16, Hq=32, Hkv=8, Sq=1, D=128, ps=64,
              longest=32768, ragged=False, window=0, sink=0, softcap=0.0, alibi=False),
        # a mixed batch of 61 requests (some slots of the batch empty), two drafted tokens each
        _case("decode 61 ragged", "decode", B=61, Hq=32, Hkv=8, Sq=2, D=128, ps=16,
              longest=15001, ragged=True, window=0, sink=0, softcap=50.0, alibi=False),
        # the decode workload with a window of 4096 and four first tokens that stay visible
        _case("decode window 4096 sink 4", "decode", B=16, Hq=32, Hkv=8, Sq=1, D=128, ps=64,
              longest=32768, ragged=False, window=4096, sink=4, softcap=0.0, alibi=False),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "rope", "rope_bwd", "cache", "decode", "decode"])
    if op == "plan":
        B = _log(rng, 1, 1500)
        return dict(op=op, B=B, ps=rng.choice([16, 32, 64, 128]), cached=_log(rng, 1, 16000),
                    new=_log(rng, 1, 300), cap=_log(rng, max(1, B // 2), 100000))
    if op in ("rope", "rope_bwd"):
        D, group, Hkv = rng.choice([64, 128]), rng.choice([1, 2, 4, 7, 8]), _log(rng, 1, 16)
        f32, B = rng.random() < 0.25, _log(rng, 1, 64)
        most = 800_000_000 // (B * Hkv * (group + 1) * D * (4 if f32 else 2) *
                               (2 if op == "rope" else 3))
        S = 1 if op == "rope" and rng.random() < 0.3 else _log(rng, 1, max(1, min(20000, most)))
        return dict(op=op, B=B, S=S, Hq=Hkv * group, Hkv=Hkv, D=D,
                    rot=rng.choice([D, D, D // 2, 16]), f32=f32, inter=rng.random() < 0.4,
                    norm=rng.random() < 0.8, fused=rng.random() < 0.5,
                    far=max(S, _log(rng, 64, 131072)), pad=rng.choice([0, 0, _log(rng, 1, 9)]))
    if op == "cache":
        D, Hkv = rng.choice([64, 128]), _log(rng, 1, 16)
        return dict(op=op, T=_log(rng, 1, 100_000_000 // (Hkv * D)), Hkv=Hkv, D=D,
                    ps=rng.choice([16, 32, 64, 128]), pad=rng.choice([0, 0, _log(rng, 1, 9)]))
    D, Hkv, B = rng.choice([64, 128]), _log(rng, 1, 16), _log(rng, 1, 80)
    Sq = rng.choice([1, 1, 1, 2, 3, 4])
    group = rng.choice([g for g in (1, 2, 3, 4, 5, 8, 16) if g * Sq <= 16])
    longest = _log(rng, 1, max(1, min(60000, 500_000_000 // (B * Hkv * D))))
    window = rng.choice([0, 0, _log(rng, 1, 8192)])
    return dict(op=op, B=B, Hq=Hkv * group, Hkv=Hkv, Sq=Sq, D=D, ps=rng.choice([16, 32, 64, 128]),
                longest=longest, ragged=rng.random() < 0.6, window=window,
                sink=rng.choice([0, 1, 4, 40]) if window else 0,
                softcap=rng.choice([0.0, 0.0, 30.0]), alibi=rng.random() < 0.2)


# ---------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------
def _row_bytes(D):
    """Bytes of one token of one head in the cache: K and V codes, then their scales."""
    return D + 4 * (D // GROUP)


def _quantise(x):
    """Codes 0..15 (8 stands for 0) and bf16 scales of x [..., D], one scale for 32 channels."""
    g = x.float().unflatten(-1, (-1, GROUP))
    s = (g.abs().amax(-1) / 7).to(torch.bfloat16)
    n = torch.where(s[..., None] > 0, torch.round(g / s[..., None].float()), 0.0)
    return (n.clamp(-8, 7) + 8).to(torch.uint8).flatten(-2), s


def _records(k, v):
    """The page records [pages, Hkv, bytes] that hold k and v [pages, Hkv, page, D]."""
    codes, scales = [], []
    for x in (k, v):
        n, s = _quantise(x)
        codes.append((n[..., 0::2] | (n[..., 1::2] << 4)).flatten(-2))
        scales.append(s.contiguous().view(torch.uint8).flatten(-2))
    return torch.cat(codes + scales, dim=-1)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    h = torch.Generator().manual_seed(seed)  # small host-side choices

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)

    def ints(lo, hi, n):
        return torch.randint(lo, hi + 1, (n,), generator=h, dtype=torch.int32)

    st, op = dict(case), case["op"]
    if op == "plan":
        B, ps, cap = case["B"], case["ps"], case["cap"]
        cached, new = ints(0, case["cached"], B), ints(1, case["new"], B)
        new[ints(0, B - 1, max(1, B // 8)).long()] = 0  # slots of the batch without a request
        pages = -(-(case["cached"] + case["new"]) // ps)
        have = (cached + ps - 1) // ps
        need = int(((cached + new + ps - 1) // ps - have).sum())
        perm = torch.randperm(int(have.sum()) + need + 8, generator=h).to(torch.int32)
        table = torch.full((B, pages), -1, dtype=torch.int32)
        table[torch.arange(pages)[None] < have[:, None]] = perm[:int(have.sum())]
        st.update(cached_lens=cached.to(DEV), new_lens=new.to(DEV), page_table=table.to(DEV),
                  free_pages=perm[int(have.sum()):].to(DEV),
                  seq_lens=torch.zeros(B, dtype=torch.int32, device=DEV),
                  cu_new=torch.zeros(B + 1, dtype=torch.int32, device=DEV),
                  slots=torch.zeros(cap, dtype=torch.int64, device=DEV),
                  positions=torch.zeros(cap, dtype=torch.int32, device=DEV),
                  seq_ids=torch.zeros(cap, dtype=torch.int32, device=DEV),
                  info=torch.zeros(4, dtype=torch.int32, device=DEV))
    elif op in ("rope", "rope_bwd"):
        B, S, Hq, Hkv, D = (case[n] for n in ("B", "S", "Hq", "Hkv", "D"))
        dt = torch.float32 if case["f32"] else torch.bfloat16
        if case["fused"]:  # one projection's output [B, S, (Hq + 2 Hkv) * D]
            qkv = normal(B, S, Hq + 2 * Hkv, D, dtype=dt)
            q, k = (qkv[:, :, a:b].transpose(1, 2) for a, b in ((0, Hq), (Hq, Hq + Hkv)))
        else:
            q, k = (normal(B, S, n, D, dtype=dt).transpose(1, 2) for n in (Hq, Hkv))
        half = case["rot"] // 2
        freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)
        angle = torch.arange(case["far"], dtype=torch.float64, device=DEV)[:, None] * freq
        start = ints(0, case["far"] - S, B)
        pos = start[:, None] + torch.arange(S, dtype=torch.int32)
        pos.view(-1)[B * S - min(case["pad"], B * S - 1):] = -1  # rows that hold no token
        w = [1 + 0.1 * normal(D, dtype=torch.float32) if case["norm"] else None for _ in (0, 1)]
        st.update(q=q, k=k, cos_sin=torch.cat([angle.cos(), angle.sin()], 1).float(),
                  positions=pos.to(DEV), q_weight=w[0], k_weight=w[1], eps=1e-6,
                  q_out=torch.zeros(B, Hq, S, D, dtype=dt, device=DEV),
                  k_out=torch.zeros(B, Hkv, S, D, dtype=dt, device=DEV))
        if op == "rope_bwd":
            st.update(dq_out=normal(B, Hq, S, D, dtype=dt), dk_out=normal(B, Hkv, S, D, dtype=dt),
                      dqw=torch.zeros(D, device=DEV), dkw=torch.zeros(D, device=DEV),
                      workspace=torch.empty(WORKSPACE, dtype=torch.uint8, device=DEV))
            st["dq"], st["dk"] = (torch.zeros(B, S, n, D, dtype=dt, device=DEV).transpose(1, 2)
                                  for n in (Hq, Hkv))
    elif op == "cache":
        T, Hkv, D, ps = (case[n] for n in ("T", "Hkv", "D", "ps"))
        pages = -(-T // ps) + 3
        slots = torch.randperm(pages, generator=g, device=DEV)[:, None] * ps
        slots = (slots + torch.arange(ps, device=DEV)).view(-1)[:T].contiguous()
        if case["pad"]:
            slots[max(1, T - case["pad"]):] = -1
        k, v = (normal(T, Hkv, D).transpose(0, 1)[None] for _ in (0, 1))
        # key channels differ in size, a few of them by much
        k = (k * (1 + 4 * torch.rand(D, generator=g, device=DEV) ** 8)).to(torch.bfloat16)
        st.update(k=k, v=v, slots=slots,
                  pool=torch.zeros(pages, Hkv, ps * _row_bytes(D), dtype=torch.uint8, device=DEV),
                  k_out=torch.zeros(1, Hkv, T, D, dtype=torch.bfloat16, device=DEV),
                  v_out=torch.zeros(1, Hkv, T, D, dtype=torch.bfloat16, device=DEV))
    else:
        B, Hq, Hkv, Sq, D, ps = (case[n] for n in ("B", "Hq", "Hkv", "Sq", "D", "ps"))
        lens = torch.full((B,), case["longest"], dtype=torch.int32)
        if case["ragged"]:
            lens = ints(1, case["longest"], B)
            lens[B // 2] = 0  # an empty slot of the batch
            lens[0] = case["longest"]
        per = -(-case["longest"] // ps)
        pages = int(((lens + ps - 1) // ps).sum()) + 2
        perm = torch.randperm(pages, generator=h).to(torch.int32)
        table = torch.full((B, per), -1, dtype=torch.int32)
        used = torch.arange(per)[None] < ((lens + ps - 1) // ps)[:, None]
        table[used] = perm[:int(used.sum())]
        st.update(q=normal(B, Hq, Sq, D), pool=_records(normal(pages, Hkv, ps, D),
                                                        normal(pages, Hkv, ps, D)),
                  page_table=table.to(DEV), seq_lens=lens.to(DEV),
                  o=torch.empty(B, Hq, Sq, D, dtype=torch.bfloat16, device=DEV),
                  lse=torch.empty(B, Hq, Sq, device=DEV),
                  workspace=torch.empty(WORKSPACE, dtype=torch.uint8, device=DEV))
    return st


# ---------------------------------------------------------------------------
# Plain forms: elementary operations in 32 bits, rounded once.
# ---------------------------------------------------------------------------
def _plain_plan(s):
    ps, cap, free = s["ps"], s["cap"], s["free_pages"]
    cached, new = s["cached_lens"].long(), s["new_lens"].long()
    B, per = s["page_table"].shape
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)])
    have, need = ((x + ps - 1).div(ps, rounding_mode="floor").clamp(max=per)
                  for x in (cached, cached + new))
    first = torch.cat([need.new_zeros(1), (need - have).cumsum(0)])
    lp = torch.arange(per, device=DEV)[None]
    at = first[:-1, None] + lp - have[:, None]
    fresh = (lp >= have[:, None]) & (lp < need[:, None])
    got = torch.where(at < free.numel(), free[at.clamp(0, free.numel() - 1)], -1)
    table = torch.where(fresh, got, s["page_table"])
    t = torch.arange(cap, device=DEV)
    b = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=B - 1)
    live = t < cu[-1]
    pos = cached[b] + t - cu[b]
    page = torch.where(pos < per * ps, table[b, (pos // ps).clamp(max=per - 1)], -1).long()
    slots = torch.where(live & (page >= 0), page * ps + pos % ps, -1)
    taken = first[-1].clamp(max=free.numel())
    info = torch.stack([cu[-1], taken, first[-1] - taken, (cached + new > per * ps).sum()])
    i32 = torch.int32
    return ((cached + new).to(i32), cu.to(i32), slots, torch.where(live, pos, -1).to(i32),
            torch.where(live, b, -1).to(i32), table, info.to(i32))


def _rotate(y, s, sign):
    """y [B, H, S, D] turned by the angles of its positions (sign -1: back)."""
    rot, half = s["rot"], s["rot"] // 2
    cs = s["cos_sin"][s["positions"].clamp(min=0).long()][:, None]
    c, d = cs[..., :half], cs[..., half:] * sign
    if s["inter"]:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        z = torch.stack([a * c - b * d, b * c + a * d], -1).flatten(-2)
    else:
        a, b = y[..., :half], y[..., half:rot]
        z = torch.cat([a * c - b * d, b * c + a * d], -1)
    return torch.cat([z, y[..., rot:]], -1)


def _plain_rope(s):
    live = (s["positions"] >= 0)[:, None, :, None]
    out = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + s["eps"]) * w
        out.append(torch.where(live, _rotate(y, s, 1.0), 0.0).to(x.dtype))
    return tuple(out)


def _plain_rope_bwd(s):
    live = (s["positions"] >= 0)[:, None, :, None]
    out, dws = [], []
    for x, dz, w in ((s["q"], s["dq_out"], s["q_weight"]), (s["k"], s["dk_out"], s["k_weight"])):
        dy = torch.where(live, _rotate(dz.float(), s, -1.0), 0.0)
        if w is not None:
            xf = x.float()
            r = torch.rsqrt(xf.square().mean(-1, keepdim=True) + s["eps"])
            n = xf * r
            dws.append((dy * n).sum((0, 1, 2)))
            dn = dy * w
            dy = r * (dn - n * (dn * n).mean(-1, keepdim=True))
        out.append(dy.to(x.dtype))
    return tuple(out + dws)


def _plain_cache(s):
    out = []
    for x in (s["k"], s["v"]):
        n, sc = _quantise(x)
        y = (n.float() - 8) * sc.float().repeat_interleave(GROUP, -1)
        out.append(torch.where((s["slots"] >= 0)[:, None], y, 0.0).to(torch.bfloat16))
    return tuple(out)


def _unpack(s, wide=torch.float32):
    """K and V [B, Hkv, L, D] of the batch from the page records, L = pages * page size."""
    Hkv, D, ps = s["Hkv"], s["D"], s["ps"]
    rec = s["pool"][s["page_table"].clamp(min=0).long()]       # [B, pages, Hkv, bytes]
    at, out = 0, []
    codes = []
    for _ in (0, 1):
        c = rec[..., at:at + ps * D // 2].unflatten(-1, (ps, D // 2))
        codes.append(torch.stack([c & 15, c >> 4], -1).flatten(-2))
        at += ps * D // 2
    for c in codes:
        b = ps * (D // GROUP) * 2
        sc = rec[..., at:at + b].contiguous().view(torch.bfloat16).unflatten(-1, (ps, D // GROUP))
        x = (c.to(wide) - 8) * sc.to(wide).repeat_interleave(GROUP, -1)
        out.append(x.transpose(1, 2).flatten(2, 3))
        at += b
    return out


def _slopes(Hq, dtype=torch.float32):
    return torch.exp2(-8.0 * torch.arange(1, Hq + 1, device=DEV, dtype=dtype) / Hq)


def _plain_decode(s):
    B, Hq, Hkv, Sq, D = (s[n] for n in ("B", "Hq", "Hkv", "Sq", "D"))
    k, v = _unpack(s)
    L = k.shape[2]
    q = s["q"].float().view(B, Hkv, -1, D)                     # rows (head of the group, token)
    x = (q @ k.transpose(-1, -2)).view(B, Hq, Sq, L) / math.sqrt(D)
    j = torch.arange(L, device=DEV)
    lens = s["seq_lens"][:, None, None, None]
    i = lens - Sq + torch.arange(Sq, device=DEV)[:, None]      # absolute position of the row
    if s["alibi"]:
        x = x - _slopes(Hq)[:, None, None] * (i - j)
    if s["softcap"]:
        x = s["softcap"] * torch.tanh(x / s["softcap"])
    keep = (j < lens) & (j <= i)
    if s["window"]:
        keep = keep & ((i - j < s["window"]) | (j < s["sink"]))
    x = torch.where(keep, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(m.isinf(), 0.0, m))
    l = e.sum(-1, keepdim=True)
    o = (e.view(B, Hkv, -1, L) @ v).view(B, Hq, Sq, D) / torch.where(l > 0, l, 1.0)
    return o.to(torch.bfloat16), (m + torch.log(l)).squeeze(-1)


PLAIN = {"plan": _plain_plan, "rope": _plain_rope, "rope_bwd": _plain_rope_bwd,
         "cache": _plain_cache, "decode": _plain_decode}


# ---------------------------------------------------------------------------
# The framework's calls.
# ---------------------------------------------------------------------------
def _own(s):
    import masked_attention_gb300 as M
    op = s["op"]
    if op == "plan":
        M.attn_page_plan(s["cached_lens"], s["new_lens"], s["page_table"], s["free_pages"],
                         s["seq_lens"], s["cu_new"], s["slots"], s["positions"], s["seq_ids"],
                         s["info"], page_size=s["ps"])
        return tuple(s[n] for n in ("seq_lens", "cu_new", "slots", "positions", "seq_ids",
                                    "page_table", "info"))
    if op == "rope":
        M.attn_qk_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], q_weight=s["q_weight"],
                            k_weight=s["k_weight"], eps=s["eps"], cos_sin=s["cos_sin"],
                            positions=s["positions"], interleaved=s["inter"])
        return s["q_out"], s["k_out"]
    if op == "rope_bwd":
        M.attn_qk_norm_rope_bwd(s["q"], s["k"], s["dq_out"], s["dk_out"], s["dq"], s["dk"],
                                q_weight=s["q_weight"], k_weight=s["k_weight"],
                                dq_weight=s["dqw"] if s["norm"] else None,
                                dk_weight=s["dkw"] if s["norm"] else None,
                                workspace=s["workspace"], eps=s["eps"], cos_sin=s["cos_sin"],
                                positions=s["positions"], interleaved=s["inter"])
        return (s["dq"], s["dk"]) + ((s["dqw"], s["dkw"]) if s["norm"] else ())
    if op == "cache":
        M.attn_cache_store_q4(s["k"], s["v"], s["slots"], s["pool"], page_size=s["ps"])
        M.attn_cache_load_q4(s["pool"], s["slots"], s["k_out"], s["v_out"], page_size=s["ps"])
        return s["k_out"], s["v_out"]
    variant = (M.MASK_CAUSAL | (M.MASK_WINDOW if s["window"] else 0) |
               (M.SCORE_SOFTCAP if s["softcap"] else 0) | (M.SCORE_ALIBI if s["alibi"] else 0))
    M.attn_decode_q4(s["q"], s["pool"], s["o"], s["lse"], variant, page_table=s["page_table"],
                     page_size=s["ps"], seq_lens=s["seq_lens"], max_len=s["longest"],
                     window=s["window"], sink=s["sink"], softcap=s["softcap"],
                     workspace=s["workspace"])
    return s["o"], s["lse"]


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# ---------------------------------------------------------------------------
# Work that no implementation can do without.
# ---------------------------------------------------------------------------
def _expected_keys(case):
    """Keys of one sequence that some of its rows see, on the average over the drawn lengths."""
    L = case["longest"]
    lens = [L] if not case["ragged"] else [max(1, round(L * (n + 0.5) / 64)) for n in range(64)]
    seen = [min(n, case["window"] + case["Sq"] - 1 + case["sink"]) if case["window"] else n
            for n in lens]
    return sum(seen) / len(seen)


def work(case):
    op = case["op"]
    if op == "plan":
        B, tokens = case["B"], case["cap"]
        return dict(bytes=4 * B * 4 + 16 * tokens + 8 * B * (case["new"] / case["ps"]), flops=0)
    if op in ("rope", "rope_bwd"):
        rows = case["B"] * case["S"] * (case["Hq"] + case["Hkv"])
        es, passes = (4 if case["f32"] else 2), (2 if op == "rope" else 3)
        table = min(case["far"], case["B"] * case["S"]) * case["rot"] * 4
        return dict(bytes=rows * case["D"] * es * passes + table + 4 * case["B"] * case["S"],
                    flops=rows * case["D"] * (8 if op == "rope" else 16))
    if op == "cache":
        rows = case["T"] * case["Hkv"]  # bf16 K and V in, records out, records in, bf16 out
        return dict(bytes=rows * (8 * case["D"] + 2 * _row_bytes(case["D"])) + 8 * case["T"],
                    flops=rows * case["D"] * 8)
    keys, D = _expected_keys(case), case["D"]
    rows = case["B"] * case["Hq"] * case["Sq"]
    return dict(bytes=case["B"] * case["Hkv"] * keys * _row_bytes(D) + rows * (4 * D + 4),
                flops=4 * D * rows * keys)


# ---------------------------------------------------------------------------
# The definitions in 64 bits.
# ---------------------------------------------------------------------------
def _exact_rope(s):
    f64 = torch.float64
    D, rot, half = s["D"], s["rot"], s["rot"] // 2
    # the rotation as index and factor tables: z[c] = C[c] y[c] + E[c] y[P[c]]
    c = torch.arange(D, device=DEV)
    if s["inter"]:
        mate, which, first = c ^ 1, c // 2, c % 2 == 0
    else:
        first = c < half
        mate, which = torch.where(first, c + half, c - half), torch.where(first, c, c - half)
    mate, which = torch.where(c < rot, mate, c), torch.where(c < rot, which, 0)
    cs = s["cos_sin"].to(f64)[s["positions"].clamp(min=0).long()]      # [B, S, rot]
    C = torch.where(c < rot, cs[..., which], 1.0)[:, None]
    E = torch.where(c < rot, cs[..., half + which], 0.0)[:, None]
    E = torch.where(first, -E, E)
    live = (s["positions"] >= 0)[:, None, :, None].to(f64)
    fwd, bwd, dws = [], [], []
    for name in ("q", "k"):
        x, w = s[name].to(f64), s[name + "_weight"]
        rho = (x.pow(2).sum(-1, keepdim=True) / D + s["eps"]).pow(-0.5) if w is not None else 1.0
        gain = w.to(f64) if w is not None else 1.0
        if s["op"] == "rope":
            y = x * rho * gain
            fwd.append(live * (C * y + E * y[..., mate]))
            continue
        dz = s["d" + name + "_out"].to(f64) * live
        dy = C * dz + (E * dz)[..., mate]
        if w is not None:
            dws.append((dy * x * rho).sum(dim=(0, 1, 2)))
            dy = gain * dy
            dy = rho * dy - x * rho.pow(3) * (dy * x).sum(-1, keepdim=True) / D
        bwd.append(dy)
    return tuple(fwd or bwd + dws)


def _exact_cache(s):
    out = []
    for x in (s["k"], s["v"]):
        g = x.double().reshape(1, s["Hkv"], s["T"], -1, GROUP)
        step = (g.abs().max(-1, keepdim=True).values / 7).to(torch.bfloat16).double()
        y = (g / step.clamp(min=1e-300)).round().clamp(-8, 7) * step
        out.append(y.reshape(x.shape) * (s["slots"] >= 0).double()[:, None])
    return tuple(out)


def _exact_decode(s):
    f64 = torch.float64
    B, Hq, Hkv, Sq, D, ps = (s[n] for n in ("B", "Hq", "Hkv", "Sq", "D", "ps"))
    o = torch.zeros(B, Hq, Sq, D, dtype=f64, device=DEV)
    lse = torch.full((B, Hq, Sq), -math.inf, dtype=f64, device=DEV)
    group, half, ng = Hq // Hkv, D // 2, D // GROUP
    sl = _slopes(Hq, f64)
    for b, n in enumerate(s["seq_lens"].tolist()):
        if n == 0:
            continue
        j = torch.arange(n, device=DEV)
        rec = s["pool"][s["page_table"][b, j // ps].long()]            # [n, Hkv, bytes]
        row = (j % ps)[:, None, None]

        def take(base, width):
            at = base + row * width + torch.arange(width, device=DEV)
            return torch.gather(rec, 2, at.expand(-1, Hkv, -1))        # [n, Hkv, width]

        kv = []
        for which in (0, 1):
            c = take(which * ps * half, half).to(torch.int32)
            x = torch.stack([c.remainder(16), c.div(16, rounding_mode="floor")], -1) - 8
            t = take(2 * ps * half + which * ps * ng * 2, ng * 2).contiguous().view(torch.bfloat16)
            x = x.reshape(n, Hkv, ng, GROUP).to(f64) * t.to(f64)[..., None]
            kv.append(x.reshape(n, Hkv, D))
        for r in range(Sq):
            i = n - Sq + r
            if i < 0:
                continue
            see = j <= i
            if s["window"]:
                see = see & ((j > i - s["window"]) | (j < s["sink"]))
            at = see.nonzero()[:, 0]
            K, V = kv[0][at], kv[1][at]
            q = s["q"][b, :, r].to(f64).view(Hkv, group, D)
            x = torch.einsum("hgd,nhd->hgn", q, K).reshape(Hq, -1) * D ** -0.5
            if s["alibi"]:
                x = x - sl[:, None] * (i - at)
            if s["softcap"]:
                x = (x / s["softcap"]).tanh() * s["softcap"]
            lse[b, :, r] = torch.logsumexp(x, -1)
            p = torch.softmax(x, -1).view(Hkv, group, -1)
            o[b, :, r] = torch.einsum("hgn,nhd->hgd", p, V).reshape(Hq, D)
    return o, lse


def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    if case["op"] == "decode":
        return _exact_decode(s)
    return _exact_cache(s) if case["op"] == "cache" else _exact_rope(s)
