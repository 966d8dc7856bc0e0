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
