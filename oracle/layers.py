"""float64 references of the serving operators: router, row grouping, the experts of a
mixture-of-experts layer and low-rank adapters, each with the bound its arithmetic gives.

Written from the definitions in ``include/fp8gemm_layers.h`` with plain loops over
tokens, experts and adapters; pinned by ``tests/test_oracle_layers.py``.
"""
from __future__ import annotations

import numpy as np

from .formats import unpack_fp4
from .gemm import ACT_LIPSCHITZ, activation, dequantize, output_ulp

FP32_EPS = 2.0 ** -24                    # half a step of binary32, relative
SPLIT_EPS = 2.0 ** -17                   # a value kept as two bf16 (8 + 8 bits, RNE)


# ---- router -------------------------------------------------------------------
def route_reference(logits, k: int, scoring: str, renormalize: bool, scale: float = 1.0):
    """(ids int32 [T, k], weights float64 [T, k]) of float64-exact logits [T, E]."""
    l = np.array(logits, dtype=np.float64)
    l[np.isnan(l)] = -np.inf
    T, E = l.shape
    ids = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        order = sorted((e for e in range(E) if l[t, e] > -np.inf), key=lambda e: (-l[t, e], e))
        chosen = order[:k]
        if not chosen:
            continue
        top = l[t, chosen[0]]
        if scoring == "softmax" or (renormalize and top < -60):     # e^l / sum: the same ratios
            p = {e: 1.0 if l[t, e] == top else float(np.exp(l[t, e] - top)) for e in order}
            total = sum(p[e] for e in (chosen if renormalize else order))
        else:
            p = {e: float(1.0 / (1.0 + np.exp(-l[t, e]))) for e in chosen}
            total = sum(p.values()) if renormalize else 1.0
        for j, e in enumerate(chosen):
            ids[t, j] = e
            w[t, j] = scale * p[e] / total
    return ids, w


def route_tolerance(logits, weights, k: int):
    """|w| times: the exponent's rounding (|l - max| half steps of binary32, and |l| for a
    sigmoid's), two ulp of each exponential, the sums of E terms and two divisions."""
    l = np.array(logits, dtype=np.float64)
    l[~np.isfinite(l)] = 0.0
    spread = np.abs(l).max(axis=1, keepdims=True) * 2
    return np.abs(weights) * (spread + l.shape[1] + k + 16) * 2 * FP32_EPS + 2.0 ** -120


# ---- grouping -----------------------------------------------------------------
def group_reference(ids, groups: int):
    """(order int32 [n], offsets int32 [groups + 1])."""
    flat = np.asarray(ids).reshape(-1)
    runs = [[i for i, g in enumerate(flat) if g == want] for want in range(groups)]
    rest = [i for i, g in enumerate(flat) if not 0 <= g < groups]
    offsets = np.cumsum([0] + [len(r) for r in runs]).astype(np.int32)
    return np.array([i for r in runs + [rest] for i in r], np.int32), offsets


# ---- experts ------------------------------------------------------------------
def _expert(q, s, mode, fmt, e):
    codes = unpack_fp4(q[e]) if fmt == "e2m1" else q[e]
    rows = codes.shape[0]
    scale = np.asarray(s).reshape(-1)[e] if mode == "tensor" else \
        np.asarray(s).reshape(-1, rows)[e] if mode == "rowwise" else s[e]
    return dequantize(codes, scale, mode, fmt)


def moe_reference(x, ids, weights, q13, s13, q2, s2, mode: str, fmt: str, act: str, out: str):
    """(out float64 [T, H], bound): the bound carries the fp32 sums over H and I (one half
    step per term), the activation's Lipschitz constant, h's two-bf16 form, the sum over
    slots and the output's rounding."""
    x = np.asarray(x, np.float64)
    E = q13.shape[0]
    T, H = x.shape
    y = np.zeros((T, H))
    tol = np.zeros((T, H))
    size = np.zeros((T, H))
    for e in range(E):
        rows, slots = np.nonzero(np.asarray(ids) == e)
        if not rows.size:
            continue
        w13, w2 = _expert(q13, s13, mode, fmt, e), _expert(q2, s2, mode, fmt, e)
        inner = w2.shape[1]
        xe = x[rows]
        gu = xe @ w13.T
        dgu = (np.abs(xe) @ np.abs(w13).T) * (H + 8) * FP32_EPS
        g, u, dg, du = gu[:, :inner], gu[:, inner:], dgu[:, :inner], dgu[:, inner:]
        a = activation(g, act)
        h = a * u
        da = ACT_LIPSCHITZ[act] * dg + 2.0 ** -20 * (np.abs(a) + np.abs(g))
        dh = da * (np.abs(u) + du) + np.abs(a) * du + (2 * FP32_EPS + SPLIT_EPS) * np.abs(h)
        wt = np.asarray(weights, np.float64)[rows, slots][:, None]
        np.add.at(y, rows, wt * (h @ w2.T))
        mag = np.abs(wt) * (np.abs(h) @ np.abs(w2).T)
        np.add.at(size, rows, mag)
        np.add.at(tol, rows, np.abs(wt) * (dh @ np.abs(w2).T) + mag * (2 * inner + 16) * FP32_EPS)
    tol = tol + size * ids.shape[1] * 2 * FP32_EPS
    return y, tol + 0.5 * output_ulp(np.abs(y) + tol, out)


# ---- adapters -----------------------------------------------------------------
def lora_reference(x, base, a, b, groups_of_rows, scales, act: str, out: str):
    """(out float64 [M, N], bound); groups_of_rows [M]: a row's adapter, or none outside
    [0, G).  v is kept in two 16-bit values: within 2^-17 of each entry for bf16, within
    2^-21 of a row's largest for f16."""
    x, base = np.asarray(x, np.float64), np.asarray(base, np.float64)
    a, b = np.asarray(a, np.float64), np.asarray(b, np.float64)
    G, rank, K = a.shape
    y, tol = base.copy(), np.abs(base) * 2 * FP32_EPS
    for m, g in enumerate(np.asarray(groups_of_rows).reshape(-1)):
        if not 0 <= g < G:
            continue
        s = 1.0 if scales is None else float(scales[g])
        v = a[g] @ x[m]
        dv = (np.abs(a[g]) @ np.abs(x[m])) * (K + 8) * FP32_EPS
        split = SPLIT_EPS * np.abs(v) if out == "bf16" else 2.0 ** -21 * np.abs(v).max()
        y[m] += s * (b[g] @ v)
        mag = np.abs(s) * (np.abs(b[g]) @ np.abs(v))
        tol[m] += np.abs(s) * (np.abs(b[g]) @ (dv + split)) + mag * (2 * rank + 8) * FP32_EPS
        tol[m] += 2 * FP32_EPS * np.abs(y[m])
    z = activation(y, act)
    tol = ACT_LIPSCHITZ[act] * tol
    if act != "none":
        tol = tol + 2.0 ** -20 * (np.abs(z) + np.abs(y))
    return z, tol + 0.5 * output_ulp(np.abs(z) + tol, out)
