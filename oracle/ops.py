"""The operators without a context in fp64 (oracle): MXFP4 conversion, pairs
grouped by expert, ragged products and the weighted sum of expert rows.

MXFP4 follows OCP MX v1.0 with the shared exponent floor(log2 max) - 2; the
products and the sum are the layer's own arithmetic (snackonai, "The Code,
Annotated": grouped evaluation, then the exact merge) on caller-held operands.
"""
from __future__ import annotations

import numpy as np

from .expert import _E2M1, mxfp4_matrix, silu  # noqa: F401


def mx_quantize(x: np.ndarray):
    """x [R, C] (exact in fp64) -> (codes uint8 [R, C/2], scales uint8 [R, C/32])."""
    x = np.asarray(x, np.float64)
    R, C = x.shape
    v = x.reshape(R, C // 32, 32)
    with np.errstate(invalid="ignore", over="ignore"):
        amax = np.abs(v).max(axis=2)
        bad = ~np.isfinite(v).all(axis=2)
        _, e = np.frexp(np.where(bad, 1.0, amax))
        e = np.where(bad | (amax == 0), 0, np.clip(e - 3, -127, 127))
        q = np.where(bad[:, :, None], 0.0, v) * np.exp2(-e.astype(np.float64))[:, :, None]
    # nearest magnitude of the grid; of two equally near ones the even code
    grid = _E2M1[:8]
    dist = np.abs(np.abs(q)[..., None] - grid)
    near = dist == dist.min(axis=-1, keepdims=True)
    even = np.arange(8) % 2 == 0
    code = np.where(near.sum(-1) == 2, np.argmax(near & even, axis=-1), np.argmax(near, axis=-1))
    code = np.where((q < 0) & (code > 0), code | 8, code).astype(np.uint8).reshape(R, C)
    scales = np.where(bad, 255, e + 127).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), scales


def mx_values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    return mxfp4_matrix(codes, scales, codes.shape[0], codes.shape[1] * 2)


def group_pairs(ids: np.ndarray, E: int):
    """(offsets [E+1], perm [T*k]): pairs by (expert, pair index), those of no expert last as -1."""
    flat = np.asarray(ids).reshape(-1)
    by = [np.flatnonzero(flat == e) for e in range(E)]
    offsets = np.concatenate([[0], np.cumsum([len(b) for b in by])]).astype(np.int32)
    perm = np.full(flat.size, -1, np.int32)
    if offsets[-1]:
        perm[:offsets[-1]] = np.concatenate(by)
    return offsets, perm


def grouped_rows(x, w_of, offsets, n_rows, N, x_index=None, div=1, glu=False):
    """Rows by position and their error scale.  w_of(e) -> [N, K] fp64; returns
    (rows [n_rows, N or N/2], bound [same]): bound is the magnitude sum of each
    output's terms (for glu a bound of the output's sensitivity to the
    relative error of the two sums)."""
    x = np.asarray(x, np.float64)
    out_n = N // 2 if glu else N
    rows = np.full((n_rows, out_n), np.nan)
    size = np.zeros((n_rows, out_n))
    for e in range(len(offsets) - 1):
        p = np.arange(offsets[e], offsets[e + 1])
        if not len(p):
            continue
        if x_index is None:
            a = x[p]
        else:
            i = np.asarray(x_index)[p]
            ok = (i >= 0) & (i // div < len(x))
            a = np.where(ok[:, None], x[np.where(ok, i // div, 0)], 0.0)
        w = w_of(e)
        z, m = a @ w.T, np.abs(a) @ np.abs(w).T
        if glu:
            g, u, mg, mu = z[:, :out_n], z[:, out_n:], m[:, :out_n], m[:, out_n:]
            rows[p] = silu(g) * u
            # |silu'| <= 1.1
            size[p] = 1.1 * mg * np.abs(u) + np.abs(silu(g)) * mu + 1e-3 * mg * mu
        else:
            rows[p], size[p] = z, m
    return rows, size


def combine(p, w, ids=None, E=0):
    """(y [T, H], magnitude sums)."""
    w = np.asarray(w, np.float64)
    T, k = w.shape
    p = np.asarray(p, np.float64).reshape(T, k, -1)
    if ids is not None:
        ok = (np.asarray(ids) >= 0) & (np.asarray(ids) < E)
        p = np.where(ok[:, :, None], p, 0.0)
        w = np.where(ok, w, 0.0)
    t = w[:, :, None] * p
    return t.sum(1), np.abs(t).sum(1)
