"""CPU oracle (fp64, numpy) of the operators around the paged cache. TEST
INFRASTRUCTURE ONLY, as ``oracle/attention.py``; shares no code with the
library.

* ``page_plan``: page tables and slot maps, request by request, token by token;
* ``norm_rope``, ``norm_rope_backward``: per-head RMS norm and rotation, the
  backward as the analytic gradient (pinned by central differences);
* ``q4_quantise``, ``q4_pack``, ``q4_row``: the 4-bit cache's codes, records
  and reads;
* ``decode_q4``: attention of the last rows of each sequence over its cached
  rows, one query row at a time.
"""
from __future__ import annotations

import math

import numpy as np

GROUP = 32


def page_plan(cached, new, table, free, page, cap):
    """Returns seq_lens, cu, slots, positions, seq_ids, table, info."""
    B, per = table.shape
    table = table.copy()
    slots, pos, ids = [], [], []
    cu, taken, lacking, over = [0], 0, 0, 0
    for b in range(B):
        c, n = max(int(cached[b]), 0), max(int(new[b]), 0)
        have, need = min(-(-c // page), per), min(-(-(c + n) // page), per)
        for lp in range(have, need):
            if taken < len(free):
                table[b, lp] = free[taken]
                taken += 1
            else:
                table[b, lp] = -1
                lacking += 1
        over += c + n > per * page
        for t in range(c, c + n):
            pg = int(table[b, t // page]) if t // page < per else -1
            slots.append(pg * page + t % page if pg >= 0 else -1)
            pos.append(t)
            ids.append(b)
        cu.append(cu[-1] + n)
    total = cu[-1]

    def out(x, dt):
        return np.array((x + [-1] * cap)[:cap], dt)

    lens = [max(int(c), 0) + max(int(n), 0) for c, n in zip(cached, new)]
    return (np.array(lens, np.int32), np.array(cu, np.int32), out(slots, np.int64),
            out(pos, np.int32), out(ids, np.int32), table,
            np.array([total, taken, lacking, over], np.int32))


def _pairs(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(y, table, pos, interleaved, back=False):
    """y [..., S, D] (pos [..., S] broadcastable) turned by the table's angles."""
    rot = table.shape[1]
    a, b = _pairs(rot, interleaved)
    cs = table[pos]
    c, s = cs[..., :rot // 2], cs[..., rot // 2:] * (-1.0 if back else 1.0)
    z = y.copy()
    z[..., a] = y[..., a] * c - y[..., b] * s
    z[..., b] = y[..., b] * c + y[..., a] * s
    return z


def norm_rope(x, weight, eps, table, pos, interleaved):
    """x [B, H, S, D], pos [B, S] (all inside the table) or table None."""
    y = np.asarray(x, np.float64)
    if weight is not None:
        y = y / np.sqrt((y ** 2).mean(-1, keepdims=True) + eps) * weight
    return y if table is None else rotate(y, table, pos[:, None], interleaved)


def norm_rope_backward(x, dz, weight, eps, table, pos, interleaved):
    """(dx, dweight or None) of sum(dz * norm_rope(x))."""
    dy = np.asarray(dz, np.float64)
    if table is not None:
        dy = rotate(dy, table, pos[:, None], interleaved, back=True)
    if weight is None:
        return dy, None
    x = np.asarray(x, np.float64)
    r = 1.0 / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    n = x * r
    dn = dy * weight
    return r * (dn - n * (dn * n).mean(-1, keepdims=True)), (dy * n).sum((0, 1, 2))


def bf16_bits(x):
    """fp64 -> bf16 bits, to nearest even (in one rounding), NaN -> 0x7fff."""
    x = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        a = np.abs(x)
        e = np.maximum(np.floor(np.log2(np.where(a > 0, a, 1.0))), -126.0)
        step = 2.0 ** (e - 7)
        r = np.rint(a / step) * step
        r32 = np.where(a > 0, r, 0.0).astype(np.float32)
    bits = (r32.view(np.uint32) >> 16).astype(np.uint16)
    bits = np.where(np.signbit(x), bits | 0x8000, bits)
    return np.where(np.isnan(x), np.uint16(0x7fff), bits).astype(np.uint16)


def bf16_value(bits):
    return (np.asarray(bits).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def q4_quantise(x):
    """Codes uint8 [..., D] and scale bits uint16 [..., D / 32] of x."""
    g = np.asarray(x, np.float64).reshape(*x.shape[:-1], -1, GROUP)
    a = np.abs(g).max(-1)
    bits = np.where(np.isfinite(a), bf16_bits(np.where(np.isfinite(a), a, 0.0) / 7.0),
                    np.uint16(0x7fff)).astype(np.uint16)
    s = bf16_value(bits)[..., None]
    with np.errstate(invalid="ignore", divide="ignore"):
        n = np.where(s > 0, np.clip(np.rint(g / s), -8, 7), 0.0) + 8
    return n.astype(np.uint8).reshape(x.shape), bits


def q4_bytes(page, D):
    return page * (D + D // GROUP * 4)


def q4_write(pool, slot, head, k, v, page):
    """Writes one token's K and V row [D] into pool [pages, Hkv, bytes]."""
    D = k.shape[-1]
    rec, row = pool[slot // page, head], slot % page
    for i, x in enumerate((k, v)):
        codes, bits = q4_quantise(x)
        at = i * page * (D // 2) + row * (D // 2)
        rec[at:at + D // 2] = codes[0::2] | (codes[1::2] << 4)
        w = D // GROUP * 2
        at = page * D + i * page * w + row * w
        rec[at:at + w] = bits.view(np.uint8)


def q4_row(pool, slot, head, page, D):
    """(K row, V row) fp64 [D] at a slot; zeros outside the pool."""
    if slot < 0 or slot // page >= pool.shape[0]:
        return np.zeros(D), np.zeros(D)
    rec, row, out = pool[slot // page, head], slot % page, []
    for i in range(2):
        at = i * page * (D // 2) + row * (D // 2)
        b = rec[at:at + D // 2]
        n = np.stack([b & 15, b >> 4], -1).reshape(D).astype(np.float64) - 8
        w = D // GROUP * 2
        at = page * D + i * page * w + row * w
        s = bf16_value(rec[at:at + w].copy().view(np.uint16))
        out.append(n * np.repeat(s, GROUP))
    return out[0], out[1]


def decode_q4(q, pool, table, lens, page, *, causal=True, window=0, sink=0, softcap=0.0,
              alibi=None, scale=None):
    """O [B, Hq, Sq, D], LSE [B, Hq, Sq], and per row sum_j p_j |v_j| [.., D]
    and the largest score magnitude that a tolerance needs."""
    B, Hq, Sq, D = q.shape
    Hkv = pool.shape[1]
    O, L = np.zeros(q.shape), np.full(q.shape[:3], -np.inf)
    A = np.zeros(q.shape)
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    for b in range(B):
        n = int(lens[b])
        for hk in range(Hkv):
            kv = [q4_row(pool, int(table[b, j // page]) * page + j % page
                         if table[b, j // page] >= 0 else -1, hk, page, D) for j in range(n)]
            if not n:
                continue
            K, V = np.stack([x[0] for x in kv]), np.stack([x[1] for x in kv])
            for h in range(hk * (Hq // Hkv), (hk + 1) * (Hq // Hkv)):
                for r in range(Sq):
                    i = n - Sq + r
                    j = np.arange(n)
                    see = np.full(n, i >= 0)
                    if causal:
                        see &= j <= i
                    if window:
                        see &= (i - j < window) | (j < sink)
                    at = np.nonzero(see)[0]
                    if not len(at):
                        continue
                    s = K[at] @ q[b, h, r].astype(np.float64) * scale
                    if alibi is not None:
                        s = s - alibi[h] * (i - at)
                    if softcap:
                        s = softcap * np.tanh(s / softcap)
                    m = s.max()
                    p = np.exp(s - m)
                    L[b, h, r] = m + np.log(p.sum())
                    p /= p.sum()
                    O[b, h, r] = p @ V[at]
                    A[b, h, r] = p @ np.abs(V[at])
    return O, L, A
