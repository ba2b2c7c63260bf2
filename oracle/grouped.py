"""Products of rows grouped by expert and their gradients, in float64.

Expert e owns the rows offsets[e] .. offsets[e + 1] - 1; rows that no expert owns give
zero rows, experts without rows zero weight gradients. The derivative is that of
y[p, n] = sum_k x[p, k] w[e(p), n, k].
"""
import numpy as np


def expert_of_rows(offsets, S):
    """Expert of every row, -1 for rows that none owns."""
    e = np.full(S, -1, np.int64)
    for i in range(len(offsets) - 1):
        e[offsets[i]:offsets[i + 1]] = i
    return e


def grouped_gemm(x, w, offsets):
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    y = np.zeros((x.shape[0], w.shape[1]))
    for e in range(w.shape[0]):
        a, b = offsets[e], offsets[e + 1]
        y[a:b] = x[a:b] @ w[e].T
    return y


def grouped_gemm_backward(x, w, offsets, d_y):
    x, w, d_y = (np.asarray(v, np.float64) for v in (x, w, d_y))
    d_x, d_w = np.zeros(x.shape), np.zeros(w.shape)
    for e in range(w.shape[0]):
        a, b = offsets[e], offsets[e + 1]
        d_x[a:b] = d_y[a:b] @ w[e]
        d_w[e] = d_y[a:b].T @ x[a:b]
    return d_x, d_w
