"""Rows in expert order and back, and the gradients, in float64, slot by slot.

reverse[p] is the slot t k + j of sorted row p; the first n rows have an expert. Slots without a row add nothing.
"""
import numpy as np


def gather(hidden, reverse, n, k):
    return np.asarray(hidden, np.float64)[np.asarray(reverse[:n]) // k]


def gather_backward(d_x, reverse, n, T, k):
    d = np.zeros((T, d_x.shape[1]))
    for p in range(n):
        d[reverse[p] // k] += np.asarray(d_x[p], np.float64)
    return d


def combine(y, weights, reverse, n):
    T, k = weights.shape
    out = np.zeros((T, y.shape[1]))
    for p in range(n):
        t, j = divmod(int(reverse[p]), k)
        out[t] += float(weights[t, j]) * np.asarray(y[p], np.float64)
    return out


def combine_backward(d_out, y, weights, reverse, n):
    """(d_y of the first n rows, d_weights)."""
    k = weights.shape[1]
    d_out, y = np.asarray(d_out, np.float64), np.asarray(y, np.float64)
    d_y, d_w = np.zeros((n, y.shape[1])), np.zeros(weights.shape)
    for p in range(n):
        t, j = divmod(int(reverse[p]), k)
        d_y[p] = float(weights[t, j]) * d_out[t]
        d_w[t, j] = d_out[t] @ y[p]
    return d_y, d_w
