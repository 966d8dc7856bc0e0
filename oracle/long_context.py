"""fp64 definitions of the operators for long contexts on the bf16 paged cache, written out
plainly (test infrastructure: nothing in the package imports it)."""
import numpy as np


def axes_rows(table, pos, axes):
    """The table [B * S, rot] whose row b * S + s holds the cosines and sines of token (b, s):
    channel pair i from row pos[axes[i], b, s] of `table`. With it a rotation by positions on
    several axes is the one-axis rotation at positions 0 .. B * S - 1."""
    half = table.shape[1] // 2
    out = np.zeros((pos[0].size, table.shape[1]), table.dtype)
    for i, a in enumerate(axes):
        for t, p in enumerate(np.asarray(pos[a]).ravel()):
            if 0 <= p < len(table):
                out[t, i], out[t, half + i] = table[p, i], table[p, half + i]
    return out


def cached_rows(pool, table, b, n, head, page):
    """Rows [n, D] of a head of sequence b; a page outside the pool reads as zeros."""
    out = np.zeros((n, pool.shape[-1]))
    for j in range(n):
        at = int(table[b, j // page])
        if 0 <= at < len(pool):
            out[j] = pool[at, head, j % page]
    return out


def visible(n, i, causal, window):
    """Truth of every key below n for a row at position i."""
    j = np.arange(n)
    see = np.full(n, i >= 0)
    if causal:
        see &= j <= i
    if window:
        see &= i - j < window
    return see


def row_scores(q, K, i, scale, slope=None, softcap=0.0):
    """Modified scores of one query row at position i against keys 0 .. len(K) - 1."""
    with np.errstate(invalid="ignore", over="ignore"):
        s = K @ q * scale
    if slope is not None:
        s = s - slope * (i - np.arange(len(K)))
    return softcap * np.tanh(s / softcap) if softcap else s


def slopes(Hq):
    return 2.0 ** (-8.0 * np.arange(1, Hq + 1) / Hq)


def key_weights(q, rows, lse, previous, decay, lens, weights, *, causal=True, window=0,
                softcap=0.0, alibi=None, scale=None):
    """weights [B, Hkv, L] after the call, and the sum of the new parts times (1 + the size of
    what their exponent was made of), which a tolerance needs. rows(b, head): keys [n, D]."""
    B, Hq, Sq, D = q.shape
    Hkv = weights.shape[1]
    out, size = np.array(weights, np.float64), np.zeros(weights.shape)
    scale = D ** -0.5 if scale is None else scale
    for b in range(B):
        n = int(lens[b])
        for hk in range(Hkv):
            K = rows(b, hk)
            new = np.zeros(n)
            for h in range(hk * (Hq // Hkv), (hk + 1) * (Hq // Hkv)):
                for r in range(Sq):
                    i = n - Sq + r
                    see = visible(n, i, causal, window)
                    if lse[b, h, r] == -np.inf or not see.any():
                        continue
                    slope = None if alibi is None else alibi[h]
                    s = row_scores(q[b, h, r], K, i, scale, slope, softcap)
                    p = np.where(see, np.exp(np.where(see, s, 0) - lse[b, h, r]), 0)
                    new += p
                    with np.errstate(invalid="ignore"):
                        parts = np.abs(K) @ np.abs(q[b, h, r]) * scale
                    # the cap's own error: nothing below a quarter of it, above it cap <= 4 |s|
                    parts = parts * (5 if softcap else 1) + np.abs(lse[b, h, r])
                    if slope is not None:
                        parts = parts + slope * np.abs(i - np.arange(n)) * (5 if softcap else 1)
                    size[b, hk, :n] += p * (1 + np.where(see, parts, 0))
            old = 0 if previous is None else decay * previous[b, hk, :n]
            out[b, hk, :n] = old + new
    return out, size
