"""The operators for long contexts on the bf16 paged cache, each as a measured case: the norm and
rotation of queries and keys with positions on several axes (forward and backward), decode
attention for sequences that share prefixes, the attention weight that each cached key received,
and the eviction of the keys that received least.

``run`` computes a case with elementary torch operations when ``own`` is false and through the
framework's public calls when it is true. ``exact`` gives the same outputs from the definitions
in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"


def _case(name, op, **kw):
    return dict(name=name, op=op, **kw)


def listed():
    return [
        # queries and keys of one new token for 48 requests, positions (time, height, width)
        _case("axes step 48", "axes", B=48, S=1, Hq=32, Hkv=8, D=128, rot=128, f32=False,
              inter=False, norm=True, fused=True, far=32768, pad=0, axes="16+24+24"),
        # a packed prompt of text and images, from a fused projection into the attention's layout
        _case("axes prompt 16384", "axes", B=1, S=16384, Hq=32, Hkv=8, D=128, rot=128, f32=False,
              inter=False, norm=True, fused=True, far=131072, pad=0, axes="16+24+24"),
        # a training step's backward at the training workload's shape, pairs dealt to the axes
        _case("axes backward train", "axes_bwd", B=8, S=4096, Hq=16, Hkv=16, D=128, rot=128,
              f32=False, inter=False, norm=True, fused=False, far=4096, pad=0, axes="cyclic 3"),
        # a small fp32 backward of image patches: two axes, odd length, half of the channels
        _case("axes backward f32 odd", "axes_bwd", B=2, S=333, Hq=8, Hkv=2, D=64, rot=32,
              f32=True, inter=True, norm=True, fused=True, far=2048, pad=7, axes="8+8"),
        # four questions about one short document
        _case("shared 4 x 1000", "shared", B=4, G=1, Hq=16, Hkv=2, Sq=1, D=64, ps=16, prefix=1000,
              suffix=60, ragged=False, window=0, softcap=0.0, alibi=False),
        # 64 requests behind one long prompt, one new token each
        _case("shared 64 x 32768", "shared", B=64, G=1, Hq=32, Hkv=8, Sq=1, D=128, ps=64,
              prefix=32768, suffix=700, ragged=False, window=0, softcap=0.0, alibi=False),
        # a mixed batch of 61 requests behind 7 prompts of unlike lengths (an empty slot among
        # them), two drafted tokens each
        _case("shared 61 ragged", "shared", B=61, G=7, Hq=32, Hkv=8, Sq=2, D=128, ps=16,
              prefix=15001, suffix=1500, ragged=True, window=0, softcap=50.0, alibi=False),
        # one short conversation, one new token
        _case("weights 1 x 700", "weights", B=1, Hq=16, Hkv=2, Sq=1, D=64, ps=16, longest=700,
              ragged=False, window=0, softcap=0.0, alibi=False),
        # the decode workload: 16 sequences of a 32768-token cache, weights added up step by step
        _case("weights 16 x 32768", "weights", B=16, Hq=32, Hkv=8, Sq=1, D=128, ps=64,
              longest=32768, ragged=False, window=0, softcap=0.0, alibi=False),
        # after a prefill of two long prompts: what the last 64 tokens looked at
        _case("weights last 64 of 40000", "weights", B=2, Hq=32, Hkv=8, Sq=64, D=128, ps=64,
              longest=40000, ragged=True, window=0, softcap=0.0, alibi=False),
        # three short conversations are cut down
        _case("evict 3 x 1500", "evict", B=3, Hkv=2, D=64, ps=16, longest=1500, keep=1000,
              recent=64, sink=4, ragged=True),
        # long prompts are cut to a quarter after the prefill
        _case("evict 8 x 32768", "evict", B=8, Hkv=8, D=128, ps=64, longest=32768, keep=8192,
              recent=1024, sink=4, ragged=False),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["axes", "axes_bwd", "shared", "shared", "weights", "weights", "evict"])
    D = rng.choice([64, 128])
    if op in ("axes", "axes_bwd"):
        group, Hkv = rng.choice([1, 2, 4, 7, 8]), _log(rng, 1, 16)
        f32, B = rng.random() < 0.25, _log(rng, 1, 64)
        most = 800_000_000 // (B * Hkv * (group + 1) * D * (4 if f32 else 2) *
                               (2 if op == "axes" else 3))
        S = 1 if op == "axes" and rng.random() < 0.3 else _log(rng, 1, max(1, min(20000, most)))
        rot = rng.choice([D, D, D // 2, 16])
        a = rng.randint(1, rot // 2 - 2)
        b = rng.randint(1, rot // 2 - a - 1)
        axes = rng.choice([f"{a}+{b}+{rot // 2 - a - b}", f"{a}+{rot // 2 - a}", "cyclic 3",
                           "cyclic 2", "cyclic 4"])
        return dict(op=op, B=B, S=S, Hq=Hkv * group, Hkv=Hkv, D=D, rot=rot, f32=f32,
                    inter=rng.random() < 0.4, norm=rng.random() < 0.8, fused=rng.random() < 0.5,
                    far=max(S, _log(rng, 64, 131072)), pad=rng.choice([0, 0, _log(rng, 1, 9)]),
                    axes=axes)
    Hkv, ps = _log(rng, 1, 16), rng.choice([16, 32, 64, 128])
    scores = dict(window=rng.choice([0, 0, 0, _log(rng, 1, 8192)]),
                  softcap=rng.choice([0.0, 0.0, 30.0]), alibi=rng.random() < 0.2)
    if op == "shared":
        B, Sq = _log(rng, 1, 96), rng.choice([1, 1, 1, 2, 3, 4])
        group = rng.choice([g for g in (1, 2, 3, 4, 5, 8, 16) if g * Sq <= 16])
        # bounded by the largest listed case's products and bytes
        most = min(8_000_000_000 // (D * B * Hkv * group * Sq), 130_000_000 // (Hkv * D * 2))
        prefix = _log(rng, 1, max(1, min(40000, most)))
        return dict(op=op, B=B, G=rng.randint(1, max(1, B // 4)), Hq=Hkv * group, Hkv=Hkv, Sq=Sq,
                    D=D, ps=ps, prefix=prefix,
                    suffix=_log(rng, Sq, max(Sq, min(3000, most // B))),
                    ragged=rng.random() < 0.6, **scores)
    if op == "weights":
        B, Sq = _log(rng, 1, 32), rng.choice([1, 1, 1, 2, _log(rng, 3, 200)])
        group = rng.choice([1, 2, 3, 4, 8])
        most = min(20_000_000_000 // (D * B * Hkv * group * Sq), 500_000_000 // (B * Hkv * D))
        return dict(op=op, B=B, Hq=Hkv * group, Hkv=Hkv, Sq=Sq, D=D, ps=ps,
                    longest=_log(rng, 1, max(1, min(60000, most))), ragged=rng.random() < 0.6,
                    **scores)
    B = _log(rng, 1, 48)
    longest = _log(rng, 8, max(8, min(60000, 250_000_000 // (B * Hkv * D))))
    keep = _log(rng, 1, longest)
    return dict(op=op, B=B, Hkv=Hkv, D=D, ps=ps, longest=longest, keep=keep,
                recent=rng.randint(0, keep), sink=rng.choice([0, 1, 4, 40]),
                ragged=rng.random() < 0.6)


# ---------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------
def _pair_axes(case):
    """The axis of each rotated channel pair, from "16+24+24" (runs) or "cyclic 3"."""
    n = case["rot"] // 2
    if case["axes"].startswith("cyclic"):
        return bytes(i % int(case["axes"].split()[1]) for i in range(n))
    return b"".join(bytes([a]) * int(x) for a, x in enumerate(case["axes"].split("+")))


def _cos_sin(far, rot):
    half = rot // 2
    freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)
    angle = torch.arange(far, dtype=torch.float64, device=DEV)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _slopes(Hq, dtype=torch.float32):
    return torch.exp2(-8.0 * torch.arange(1, Hq + 1, device=DEV, dtype=dtype) / Hq)


def _paged(g, pages, Hkv, ps, D):
    """A pool of normal rows, made page by page in pieces (fp32 needs twice the room)."""
    pool = torch.empty(pages, Hkv, ps, D, dtype=torch.bfloat16, device=DEV)
    step = max(1, (1 << 26) // (Hkv * ps * D))
    for at in range(0, pages, step):
        pool[at:at + step] = torch.randn(pool[at:at + step].shape, generator=g, device=DEV)
    return pool


def _table(h, lens, per, ps, start=0):
    """A table [B, per] with distinct pages from `start` on for lens [B], in a random order."""
    n = (lens + ps - 1) // ps
    table = torch.full((len(lens), per), -1, dtype=torch.int32)
    used = torch.arange(per)[None] < n[:, None]
    table[used] = start + torch.randperm(int(n.sum()), generator=h).to(torch.int32)
    return table


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    h = torch.Generator().manual_seed(seed)  # small host-side choices

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)

    def ints(lo, hi, n):
        return torch.randint(lo, hi + 1, (n,), generator=h, dtype=torch.int32)

    def lengths(longest, B):
        lens = torch.full((B,), longest, dtype=torch.int32)
        if case["ragged"]:
            lens = ints(1, longest, B)
            lens[B // 2] = 0  # an empty slot of the batch
            lens[0] = longest
        return lens

    st, op = dict(case), case["op"]
    if op in ("axes", "axes_bwd"):
        B, S, Hq, Hkv, D = (case[n] for n in ("B", "S", "Hq", "Hkv", "D"))
        dt = torch.float32 if case["f32"] else torch.bfloat16
        if case["fused"]:  # one projection's output [B, S, (Hq + 2 Hkv) * D]
            qkv = normal(B, S, Hq + 2 * Hkv, D, dtype=dt)
            q, k = (qkv[:, :, a:b].transpose(1, 2) for a, b in ((0, Hq), (Hq, Hq + Hkv)))
        else:
            q, k = (normal(B, S, n, D, dtype=dt).transpose(1, 2) for n in (Hq, Hkv))
        # text, then an image of about half of the tokens (its rows and columns count from the
        # text's end), then text that goes on behind the image's largest position
        axes = _pair_axes(case)
        A, t = max(axes) + 1, torch.arange(S)
        text, side = S // 4, max(1, math.isqrt(S // 2))
        cell = (t - text).clamp(min=0)
        image = (t >= text) & (cell < side * side)
        grid = [torch.zeros_like(t), cell // side, cell % side, cell % 2]
        tail = torch.where(t < text, t, t - side * side + side)
        pos = torch.stack([torch.where(image, text + grid[a], tail) for a in range(A)])
        start = ints(0, case["far"] - S, B)
        pos = (start[:, None] + pos[:, None].clamp(0, S - 1)).to(torch.int32)    # [A, B, S]
        pos.view(A, -1)[:, B * S - min(case["pad"], B * S - 1):] = -1  # rows that hold no token
        w = [1 + 0.1 * normal(D, dtype=torch.float32) if case["norm"] else None for _ in (0, 1)]
        st.update(q=q, k=k, cos_sin=_cos_sin(case["far"], case["rot"]), positions=pos.to(DEV),
                  pair_axes=axes, q_weight=w[0], k_weight=w[1], eps=1e-6,
                  q_out=torch.zeros(B, Hq, S, D, dtype=dt, device=DEV),
                  k_out=torch.zeros(B, Hkv, S, D, dtype=dt, device=DEV))
        st["axis_of"] = torch.tensor(list(axes), device=DEV)
        if op == "axes_bwd":
            st.update(dq_out=normal(B, Hq, S, D, dtype=dt), dk_out=normal(B, Hkv, S, D, dtype=dt),
                      dqw=torch.zeros(D, device=DEV), dkw=torch.zeros(D, device=DEV),
                      workspace=torch.empty(1 << 24, dtype=torch.uint8, device=DEV))
            st["dq"], st["dk"] = (torch.zeros(B, S, n, D, dtype=dt, device=DEV).transpose(1, 2)
                                  for n in (Hq, Hkv))
        return st

    B, Hkv, D, ps = (case[n] for n in ("B", "Hkv", "D", "ps"))
    if op == "shared":
        Hq, Sq, G = case["Hq"], case["Sq"], min(case["G"], case["B"])
        cuts = (torch.randperm(B - 1, generator=h)[:G - 1] + 1).sort().values
        starts = torch.cat([torch.zeros(1), cuts, torch.full((1,), B)]).to(torch.int32)
        shared = torch.full((G,), case["prefix"], dtype=torch.int32)
        own_lens = torch.full((B,), case["suffix"], dtype=torch.int32)
        if case["ragged"]:
            shared = ints(0, case["prefix"], G)
            shared[0] = case["prefix"]
            own_lens = ints(Sq, case["suffix"], B)
        shared = shared // ps * ps  # whole pages are shared
        group = torch.repeat_interleave(torch.arange(G), (starts[1:] - starts[:-1]).long())
        lens = shared[group] + own_lens
        if case["ragged"] and B > 2:
            lens[B // 2] = 0
        longest = case["prefix"] + case["suffix"]
        per = -(-longest // ps)
        lead = _table(h, shared, per, ps)
        table = _table(h, own_lens, per, ps, start=int(((shared + ps - 1) // ps).sum()))
        pages = int(table.max()) + 3
        for b in range(B):  # the group's pages, then the sequence's own
            n = int(shared[group[b]]) // ps
            table[b] = torch.cat([lead[group[b], :n], table[b, :per - n]])
        st.update(q=normal(B, Hq, Sq, D), k=_paged(g, pages, Hkv, ps, D),
                  v=_paged(g, pages, Hkv, ps, D), page_table=table.to(DEV), seq_lens=lens.to(DEV),
                  group_starts=starts.to(DEV), shared_lens=shared.to(DEV), max_len=longest,
                  o=torch.empty(B, Hq, Sq, D, dtype=torch.bfloat16, device=DEV),
                  lse=torch.empty(B, Hq, Sq, device=DEV),
                  workspace=torch.empty(1 << 28, dtype=torch.uint8, device=DEV))
        return st

    lens = lengths(case["longest"], B)
    per = -(-case["longest"] // ps)
    table = _table(h, lens, per, ps)
    if op == "weights":
        Hq, Sq = case["Hq"], case["Sq"]
        pages = int(((lens + ps - 1) // ps).sum()) + 2
        st.update(q=normal(B, Hq, Sq, D), k=_paged(g, pages, Hkv, ps, D),
                  page_table=table.to(DEV), seq_lens=lens.to(DEV), decay=0.9375,
                  previous=torch.rand(B, Hkv, case["longest"], generator=g, device=DEV) ** 8,
                  weights=torch.zeros(B, Hkv, case["longest"], device=DEV))
        st["lse"] = torch.stack([torch.logsumexp(_scores(st, b), -1) for b in range(B)])
        return st
    # weights of a few keys are large, many are equal (no row looked at them)
    w = torch.randn(B, Hkv, case["longest"], generator=g, device=DEV)
    w = torch.where(torch.rand(w.shape, generator=g, device=DEV) < 0.2, 0.0, (3 * w).exp())
    keep_per = -(-(case["sink"] + case["keep"]) // ps)
    pages = B * per
    held = torch.minimum(lens, torch.tensor(case["sink"] + case["keep"]))
    new_table = _table(h, held, keep_per, ps, start=pages)
    for b in range(B):  # pages wholly before the first key that may go stay
        n = min(case["sink"], int(lens[b])) // ps
        new_table[b, :n] = table[b, :n]
    pages += B * keep_per
    st.update(weights=w, seq_lens=lens.to(DEV), k=_paged(g, pages, Hkv, ps, D),
              v=_paged(g, pages, Hkv, ps, D), page_table=table.to(DEV),
              new_table=new_table.to(DEV), weights_out=torch.zeros_like(w),
              kept=torch.zeros(B, Hkv, case["keep"], dtype=torch.int32, device=DEV),
              new_lens=torch.zeros(B, dtype=torch.int32, device=DEV),
              freed=torch.zeros(B * per, dtype=torch.int32, device=DEV),
              info=torch.zeros(2, dtype=torch.int32, device=DEV))
    return st


# ---------------------------------------------------------------------------
# Plain forms: elementary operations in 32 bits, rounded once.
# ---------------------------------------------------------------------------
def _rotate(y, s, sign):
    """y [B, H, S, D] turned by the angles of its positions (sign -1: back)."""
    rot, half = s["rot"], s["rot"] // 2
    pos = s["positions"].clamp(min=0).long()[s["axis_of"]]             # [pairs, B, S]
    i = torch.arange(half, device=DEV)[:, None, None]
    c, d = (s["cos_sin"][pos, i + at].permute(1, 2, 0)[:, None] for at in (0, half))
    d = d * sign
    if s["inter"]:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        z = torch.stack([a * c - b * d, b * c + a * d], -1).flatten(-2)
    else:
        a, b = y[..., :half], y[..., half:rot]
        z = torch.cat([a * c - b * d, b * c + a * d], -1)
    return torch.cat([z, y[..., rot:]], -1)


def _plain_axes(s):
    live = (s["positions"] >= 0).all(0)[:, None, :, None]
    out = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + s["eps"]) * w
        out.append(torch.where(live, _rotate(y, s, 1.0), 0.0).to(x.dtype))
    return tuple(out)


def _plain_axes_bwd(s):
    live = (s["positions"] >= 0).all(0)[:, None, :, None]
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


def _rows(s, name, b):
    """Rows [Hkv, L, D] of sequence b, L = all that its table can hold."""
    rec = s[name][s["page_table"][b].clamp(min=0).long()]              # [pages, Hkv, ps, D]
    return rec.float().transpose(0, 1).flatten(1, 2)


def _scores(s, b):
    """Masked scores [Hq, Sq, L] of sequence b."""
    Hq, Hkv, Sq, D = (s[n] for n in ("Hq", "Hkv", "Sq", "D"))
    k = _rows(s, "k", b)
    L = k.shape[1]
    q = s["q"][b].float().view(Hkv, -1, D)                             # rows (head, token)
    x = (q @ k.transpose(-1, -2)).view(Hq, Sq, L) / math.sqrt(D)
    j = torch.arange(L, device=DEV)
    i = s["seq_lens"][b] - Sq + torch.arange(Sq, device=DEV)[:, None]  # the row's position
    if s["alibi"]:
        x = x - _slopes(Hq)[:, None, None] * (i - j)
    if s["softcap"]:
        x = s["softcap"] * torch.tanh(x / s["softcap"])
    keep = j <= i
    if s["window"]:
        keep = keep & (i - j < s["window"])
    return torch.where(keep, x, -math.inf)


def _plain_shared(s):
    out, lses = [], []
    for b in range(s["B"]):
        x = _scores(s, b)
        m = x.amax(-1, keepdim=True)
        e = torch.exp(x - torch.where(m.isinf(), 0.0, m))
        l = e.sum(-1, keepdim=True)
        o = (e.view(s["Hkv"], -1, x.shape[-1]) @ _rows(s, "v", b)).view(s["Hq"], s["Sq"], s["D"])
        out.append(o / torch.where(l > 0, l, 1.0))
        lses.append((m + torch.log(l)).squeeze(-1))
    return torch.stack(out).to(torch.bfloat16), torch.stack(lses)


def _plain_weights(s):
    out = []
    for b in range(s["B"]):
        lse = s["lse"][b][..., None]
        p = torch.exp(_scores(s, b) - torch.where(lse.isinf(), 0.0, lse))
        out.append(p.view(s["Hkv"], -1, p.shape[-1]).sum(1)[:, :s["longest"]])
    here = torch.arange(s["longest"], device=DEV) < s["seq_lens"][:, None, None]
    return torch.where(here, s["decay"] * s["previous"] + torch.stack(out), s["weights"])


def _plain_evict(s):
    B, Hkv, ps, keep = (s[n] for n in ("B", "Hkv", "ps", "keep"))
    L, lens = s["longest"], s["seq_lens"].long()[:, None, None]
    j = torch.arange(L, device=DEV).expand(B, Hkv, L)
    first = lens.clamp(max=s["sink"])
    cut = lens - first > keep
    last = j >= lens - s["recent"]
    rank = torch.sort(torch.where((j >= first) & (j < lens) & ~last, s["weights"], -math.inf),
                      dim=-1, descending=True, stable=True).indices.argsort(-1)
    held = (j < lens) & (~cut | (j < first) | last | (rank < keep - s["recent"]))
    at = held.long().cumsum(-1) - 1                                    # new position of a held key
    new = torch.where(cut, first + keep, lens)
    b, hd, src = held.nonzero(as_tuple=True)
    dst = at[b, hd, src]
    kept = torch.full((B, Hkv, keep), -1, dtype=torch.int32, device=DEV)
    pick = dst >= first[b, 0, 0]
    kept[b[pick], hd[pick], (dst - first[b, 0, 0])[pick]] = src[pick].to(torch.int32)
    w = torch.where(j < lens, 0.0, s["weights_out"])
    w[b, hd, dst] = s["weights"][b, hd, src]
    from_page = s["page_table"][b, src // ps].long()
    to_page = s["new_table"][b, dst // ps].long()
    for pool in (s["k"], s["v"]):
        pool[to_page, hd, dst % ps] = pool[from_page, hd, src % ps]
    have, stay = (lens + ps - 1) // ps, first // ps
    p = torch.arange(s["page_table"].shape[1], device=DEV)[None]
    gone = s["page_table"][(p >= stay[:, 0]) & (p < have[:, 0])]
    freed = torch.cat([gone, s["freed"][gone.numel():]])
    info = torch.stack([(have - stay).sum(), cut.sum()]).to(torch.int32)
    return (kept, new.view(-1).to(torch.int32), w, freed, info, s["k"], s["v"])


PLAIN = {"axes": _plain_axes, "axes_bwd": _plain_axes_bwd, "shared": _plain_shared,
         "weights": _plain_weights, "evict": _plain_evict}


# ---------------------------------------------------------------------------
# The framework's calls.
# ---------------------------------------------------------------------------
def _own(s):
    import masked_attention_gb300 as M
    op = s["op"]
    if op == "axes":
        M.attn_qk_norm_rope_axes(s["q"], s["k"], s["q_out"], s["k_out"], cos_sin=s["cos_sin"],
                                 positions=s["positions"], axes=s["pair_axes"],
                                 q_weight=s["q_weight"], k_weight=s["k_weight"], eps=s["eps"],
                                 interleaved=s["inter"])
        return s["q_out"], s["k_out"]
    if op == "axes_bwd":
        M.attn_qk_norm_rope_axes_bwd(s["q"], s["k"], s["dq_out"], s["dk_out"], s["dq"], s["dk"],
                                     cos_sin=s["cos_sin"], positions=s["positions"],
                                     axes=s["pair_axes"], q_weight=s["q_weight"],
                                     k_weight=s["k_weight"],
                                     dq_weight=s["dqw"] if s["norm"] else None,
                                     dk_weight=s["dkw"] if s["norm"] else None,
                                     workspace=s["workspace"], eps=s["eps"],
                                     interleaved=s["inter"])
        return (s["dq"], s["dk"]) + ((s["dqw"], s["dkw"]) if s["norm"] else ())
    if op == "evict":
        M.attn_cache_evict(s["weights"], s["seq_lens"], s["k"], s["v"], s["page_table"],
                           s["weights_out"], s["kept"], s["new_lens"], s["freed"], s["info"],
                           page_size=s["ps"], recent=s["recent"], sink=s["sink"],
                           new_table=s["new_table"])
        return tuple(s[n] for n in ("kept", "new_lens", "weights_out", "freed", "info", "k", "v"))
    variant = (M.MASK_CAUSAL | (M.MASK_WINDOW if s["window"] else 0) |
               (M.SCORE_SOFTCAP if s["softcap"] else 0) | (M.SCORE_ALIBI if s["alibi"] else 0))
    if op == "weights":
        M.attn_key_weights(s["q"], s["k"], s["lse"], s["weights"], variant,
                           previous=s["previous"], decay=s["decay"], page_table=s["page_table"],
                           page_size=s["ps"], seq_lens=s["seq_lens"], window=s["window"],
                           softcap=s["softcap"])
        return s["weights"]
    M.attn_decode_shared(s["q"], s["k"], s["v"], s["o"], s["lse"], variant,
                         page_table=s["page_table"], page_size=s["ps"], seq_lens=s["seq_lens"],
                         group_starts=s["group_starts"], shared_lens=s["shared_lens"],
                         max_len=s["max_len"], window=s["window"], softcap=s["softcap"],
                         workspace=s["workspace"])
    return s["o"], s["lse"]


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# ---------------------------------------------------------------------------
# Work that no implementation can do without.
# ---------------------------------------------------------------------------
def _mean_length(case, longest):
    return longest / 2 if case["ragged"] else longest


def work(case):
    op = case["op"]
    if op in ("axes", "axes_bwd"):
        rows = case["B"] * case["S"] * (case["Hq"] + case["Hkv"])
        es, passes = (4 if case["f32"] else 2), (2 if op == "axes" else 3)
        table = min(case["far"], case["B"] * case["S"]) * case["rot"] * 4
        return dict(bytes=rows * case["D"] * es * passes + table +
                    4 * case["B"] * case["S"] * (max(_pair_axes(case)) + 1),
                    flops=rows * case["D"] * (8 if op == "axes" else 16))
    B, Hkv, D = case["B"], case["Hkv"], case["D"]
    if op == "evict":
        n = _mean_length(case, case["longest"])
        held = B * Hkv * min(n, case["sink"] + case["keep"])
        return dict(bytes=B * Hkv * n * 8 + held * (4 + 8 * D), flops=0)
    rows = B * case["Hq"] * case["Sq"]
    if op == "weights":
        n = _mean_length(case, case["longest"])
        seen = min(n, case["window"] + case["Sq"] - 1) if case["window"] else n
        return dict(bytes=B * Hkv * (seen * 2 * D + 8 * n) + rows * (2 * D + 4),
                    flops=2 * D * rows * seen)
    prefix, suffix = (_mean_length(case, case[n]) for n in ("prefix", "suffix"))
    seen = [prefix, suffix]
    if case["window"]:
        reach = case["window"] + case["Sq"] - 1
        seen = [min(prefix, max(0, reach - suffix)), min(suffix, reach)]
    G = min(case["G"], B)
    return dict(bytes=(G * seen[0] + B * seen[1]) * Hkv * 4 * D + rows * (4 * D + 4),
                flops=4 * D * rows * sum(seen))


# ---------------------------------------------------------------------------
# The definitions in 64 bits.
# ---------------------------------------------------------------------------
def _exact_axes(s):
    f64 = torch.float64
    D, rot, half = s["D"], s["rot"], s["rot"] // 2
    B, S = s["B"], s["S"]
    # every channel's factors: z[c] = C[c] y[c] + E[c] y[mate[c]]
    C = torch.ones(B, S, D, dtype=f64, device=DEV)
    E = torch.zeros(B, S, D, dtype=f64, device=DEV)
    mate = torch.arange(D, device=DEV)
    table = s["cos_sin"].to(f64)
    for i, a in enumerate(s["pair_axes"]):
        lo, hi = (2 * i, 2 * i + 1) if s["inter"] else (i, i + half)
        at = s["positions"][a].long().clamp(min=0)
        C[..., lo] = C[..., hi] = table[:, i][at]
        E[..., hi] = table[:, half + i][at]
        E[..., lo] = -E[..., hi]
        mate[lo], mate[hi] = hi, lo
    C, E = C[:, None], E[:, None]
    live = (s["positions"].amin(0) >= 0)[:, None, :, None].to(f64)
    fwd, bwd, dws = [], [], []
    for name in ("q", "k"):
        x, w = s[name].to(f64), s[name + "_weight"]
        rho = (x.pow(2).sum(-1, keepdim=True) / D + s["eps"]).pow(-0.5) if w is not None else 1.0
        gain = w.to(f64) if w is not None else 1.0
        if s["op"] == "axes":
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


def _exact_attention(s):
    """Outputs of "shared" (O, LSE) or "weights", sequence by sequence, row by row."""
    f64 = torch.float64
    B, Hq, Hkv, Sq, D, ps = (s[n] for n in ("B", "Hq", "Hkv", "Sq", "D", "ps"))
    group = Hq // Hkv
    o = torch.zeros(B, Hq, Sq, D, dtype=f64, device=DEV)
    lse = torch.full((B, Hq, Sq), -math.inf, dtype=f64, device=DEV)
    weights = s["weights"].to(f64).clone() if s["op"] == "weights" else None
    for b, n in enumerate(s["seq_lens"].tolist()):
        if n == 0:
            continue
        j = torch.arange(n, device=DEV)
        page, line = s["page_table"][b, j // ps].long(), j % ps
        K = s["k"][page, :, line].to(f64)                              # [n, Hkv, D]
        V = s["v"][page, :, line].to(f64) if weights is None else None
        if weights is not None:
            weights[b, :, :n] = s["previous"][b, :, :n].to(f64) * s["decay"]
        for r in range(Sq):
            i = n - Sq + r
            if i < 0:
                continue
            lo, hi = max(0, i - s["window"] + 1) if s["window"] else 0, i + 1
            q = s["q"][b, :, r].to(f64).view(Hkv, group, D)
            x = torch.einsum("hgd,nhd->hgn", q, K[lo:hi]).reshape(Hq, -1) * D ** -0.5
            if s["alibi"]:
                x = x - _slopes(Hq, f64)[:, None] * (i - j[lo:hi])
            if s["softcap"]:
                x = (x / s["softcap"]).tanh() * s["softcap"]
            if weights is not None:
                p = (x - s["lse"][b, :, r, None].to(f64)).exp()
                weights[b, :, lo:hi] += p.view(Hkv, group, -1).sum(1)
                continue
            lse[b, :, r] = torch.logsumexp(x, -1)
            p = torch.softmax(x, -1).view(Hkv, group, -1)
            o[b, :, r] = torch.einsum("hgn,nhd->hgd", p, V[lo:hi]).reshape(Hq, D)
    return weights if weights is not None else (o, lse)


def _exact_evict(s):
    """Key by key lists, one (sequence, head) after the other; values are copies."""
    B, Hkv, ps, keep, recent = (s[n] for n in ("B", "Hkv", "ps", "keep", "recent"))
    f64 = torch.float64
    kept, w = torch.full_like(s["kept"], -1), s["weights_out"].to(f64).clone()
    K, V = s["k"].to(f64), s["v"].to(f64)
    new_lens, gone, cut = [], [], 0
    for b, n in enumerate(s["seq_lens"].tolist()):
        first = min(n, s["sink"])
        fits = n - first <= keep
        cut += not fits
        new_lens.append(n if fits else first + keep)
        gone.append(s["page_table"][b, first // ps:-(-n // ps)])
        w[b, :, :n] = 0
        for h in range(Hkv):
            old = torch.arange(first, n, device=DEV)
            if not fits:
                old = old[:n - first - recent]
                heavy = s["weights"][b, h, old].sort(descending=True, stable=True).indices
                old = torch.cat([old[heavy[:keep - recent].sort().values],
                                 torch.arange(n - recent, n, device=DEV)])
            kept[b, h, :len(old)] = old.to(torch.int32)
            old = torch.cat([torch.arange(first, device=DEV), old])
            new = torch.arange(len(old), device=DEV)
            w[b, h, new] = s["weights"][b, h, old].to(f64)
            src, dst = s["page_table"][b, old // ps].long(), s["new_table"][b, new // ps].long()
            for pool, out in ((s["k"], K), (s["v"], V)):
                out[dst, h, new % ps] = pool[src, h, old % ps].to(f64)
    gone = torch.cat(gone)
    freed = torch.cat([gone, s["freed"][len(gone):]])
    i32 = dict(dtype=torch.int32, device=DEV)
    return (kept, torch.tensor(new_lens, **i32), w, freed,
            torch.tensor([len(gone), cut], **i32), K, V)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "evict":
        return _exact_evict(s)
    return _exact_axes(s) if case["op"].startswith("axes") else _exact_attention(s)
