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


def evict(weights, lens, starts, keep, recent, k, v, table, page, new_table, weights_out, freed):
    """(weights_out, kept, new_lens, freed, info, k, v) after the eviction, key by key."""
    B, Hkv, L = weights.shape
    k, v, out, freed = k.copy(), v.copy(), weights_out.copy(), freed.copy()
    kept = np.full((B, Hkv, keep), -1, np.int32)
    new_lens, cut, gone = np.zeros(B, np.int32), 0, []
    old = k.copy(), v.copy()
    most = min(L, table.shape[1] * page)
    for b in range(B):
        n = min(max(int(lens[b]), 0), most)
        first = min(max(int(starts[b]), 0), n)
        fits = n - first <= keep
        cut += not fits
        new_lens[b] = n if fits else first + keep
        dest = table if new_table is None else new_table
        begin = first if new_table is None else first // page * page
        have = -(-n // page)
        used = -(-int(new_lens[b]) // page)
        for p in range(used if new_table is None else first // page, have):
            # a page that the new table names in the same place, among those it uses, is kept
            if new_table is None or p >= min(used, new_table.shape[1]) or new_table[b, p] != table[b, p]:
                gone.append(int(table[b, p]))
        for h in range(Hkv):
            hold = list(range(first, n))
            if not fits:
                # NaN above all; equal weights by index
                order = sorted(range(first, n - recent), key=lambda j: (
                    -np.inf if np.isnan(weights[b, h, j]) else -weights[b, h, j],
                    not np.isnan(weights[b, h, j]), j))
                hold = sorted(order[:keep - recent]) + list(range(n - recent, n))
            kept[b, h, :len(hold)] = hold
            hold = list(range(first)) + hold
            w = [weights[b, h, j] for j in hold]
            out[b, h, :n] = 0
            out[b, h, :len(w)] = w
            for m, j in enumerate(hold):
                if m < begin or (new_table is None and m == j):
                    continue
                src = int(table[b, j // page])
                dst = int(dest[b, m // page]) if m // page < dest.shape[1] else -1
                if not 0 <= dst < len(k) or (dst == src and m % page == j % page):
                    continue
                for pool, was in zip((k, v), old):
                    row = was[src, h, j % page] if 0 <= src < len(k) else 0
                    pool[dst, h, m % page] = row
    n = min(len(gone), len(freed))
    freed[:n] = gone[:n]
    return out, kept, new_lens, freed, np.array([len(gone), cut], np.int32), k, v


def decode_rows(q, rows, lens, *, causal=True, window=0, softcap=0.0, alibi=None, scale=None):
    """O [B, Hq, Sq, D], LSE [B, Hq, Sq], per row sum_j p_j |v_j| [.., D] and the size of what
    the scores were made of, which a tolerance needs. rows(b, h): keys and values [n, D] as
    head h of sequence b sees them."""
    B, Hq, Sq, D = q.shape
    O, A = np.zeros(q.shape), np.zeros(q.shape)
    L, size = np.full(q.shape[:3], -np.inf), np.zeros(q.shape[:3])
    scale = D ** -0.5 if scale is None else scale
    for b in range(B):
        n = int(lens[b])
        if not n:
            continue
        for h in range(Hq):
            K, V = rows(b, h)
            for r in range(Sq):
                i = n - Sq + r
                see = visible(n, i, causal, window)
                if not see.any():
                    continue
                slope = None if alibi is None else alibi[h]
                s = row_scores(q[b, h, r], K, i, scale, slope, softcap)[see]
                m = s.max()
                p = np.exp(s - m)
                L[b, h, r] = m + np.log(p.sum())
                p /= p.sum()
                O[b, h, r], A[b, h, r] = p @ V[see], p @ np.abs(V[see])
                parts = np.abs(K[see]) @ np.abs(q[b, h, r]) * scale
                if slope is not None:
                    parts = parts + slope * np.abs(i - np.arange(n))[see]
                size[b, h, r] = parts.max() * (5 if softcap else 1)
    return O, L, A, size
