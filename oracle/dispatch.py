"""Token dispatch by expert and SwiGLU, with their gradients, in float64 (oracle).

TEST INFRASTRUCTURE ONLY -- see the package docstring.

    xp[row(t, j)] = x[t];           dx[t] = sum_j dxp[row(t, j)]
    y[t] = sum_j p[t, j] o[row(t, j)];   do[row(t, j)] = p[t, j] dy[t],  dp[t, j] = <dy[t], o[row(t, j)]>
    a = gate s up, s = 1 / (1 + e^-gate);
    dgate = da up s (1 + gate (1 - s)),  dup = da gate s

Nothing is rounded here: the caller rounds where the call under test does.
"""

import numpy as np


def maps(topk_idx, E, row_align=1):
    """(offsets, row_map, src_row): experts in order, an expert's slots in
    flat order, padding after each; ids outside [0, E) take no row (-1)."""
    T, k = topk_idx.shape
    offsets, row_map, src = [0], np.full((T, k), -1, dtype=np.int64), []
    for e in range(E):
        for t, j in np.argwhere(topk_idx == e):
            row_map[t, j] = len(src)
            src.append(t)
        src += [-1] * (-len(src) % row_align)
        offsets.append(len(src))
    return np.array(offsets), row_map, np.array(src, dtype=np.int64)


def permute(x, row_map, rows):
    xp = np.zeros((rows, x.shape[1]))
    for t, j in np.argwhere(row_map >= 0):
        xp[row_map[t, j]] = x[t]
    return xp


def gather_sum(src, row_map, w=None):
    """(sum, sum of magnitudes) over a token's dispatched slots."""
    out, mag = np.zeros((row_map.shape[0], src.shape[1])), np.zeros((row_map.shape[0], src.shape[1]))
    for j in range(row_map.shape[1]):
        here = row_map[:, j] >= 0
        v = src[row_map[here, j]] * (1.0 if w is None else w[here, j, None])
        out[here] += v
        mag[here] += np.abs(v)
    return out, mag


def unpermute_bwd(dy, o, row_map, w):
    """(do, dp, sum of the magnitudes of dp's products)."""
    do, dp, mag = np.zeros_like(o), np.zeros(row_map.shape), np.zeros(row_map.shape)
    for j in range(row_map.shape[1]):
        here = row_map[:, j] >= 0
        r = row_map[here, j]
        do[r] = w[here, j, None] * dy[here]
        dp[here, j] = np.sum(dy[here] * o[r], axis=1)
        mag[here, j] = np.sum(np.abs(dy[here] * o[r]), axis=1)
    return do, dp, mag


def sigmoid(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-g))


def swiglu(h):
    gate, up = np.split(h, 2, axis=1)
    return gate * sigmoid(gate) * up


def swiglu_bwd(da, h):
    gate, up = np.split(h, 2, axis=1)
    s = sigmoid(gate)
    return np.concatenate((da * up * s * (1.0 + gate * (1.0 - s)), da * gate * s), axis=1)
