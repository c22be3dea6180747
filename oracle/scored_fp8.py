"""Plain float64 definitions of the scored router, its gradient, the combine's
backward, FP8 rows and the FP8 expert products (test infrastructure only).

Written from include/moeq.h; shares no code with the CUDA library. Selections
are full sorts, e4m3 is a table of 256 values, products are matrix products
in float64 of the values the bytes stand for.
"""

from __future__ import annotations

import math

import numpy as np

__all__ = ["scored_scores", "route_scored", "route_scored_bwd", "combine_bwd", "e4m3_values",
           "e4m3_nearest", "block_exponents", "quantize_rows", "rows_values", "weight_values",
           "fp8_gemm", "swiglu", "swiglu_bwd"]


# ----------------------------------------------------------------------------- router

def scored_scores(logits, score: str):
    """Scores [T, E]; NaN and -inf logits are masked and score 0."""
    x = np.asarray(logits, np.float64)
    out = np.zeros_like(x)
    for t in range(x.shape[0]):
        live = np.array([not math.isnan(v) and v != -math.inf for v in x[t]])
        if not live.any():
            continue
        v = x[t][live]
        if score == "sigmoid":
            with np.errstate(over="ignore"):
                out[t][live] = 1.0 / (1.0 + np.exp(-v))
        else:
            m = v.max()
            z = np.where(v == m, 1.0, np.exp(np.where(v == m, 0.0, v - m)))
            out[t][live] = z / z.sum()
    return out


def route_scored(logits, k, score="softmax", groups=1, topk_groups=1, group_top=1, renorm=True,
                 scale=1.0, bias=None):
    """(topk_idx [T, k], gates [T, k]): sort of (masked last, key descending, id ascending)."""
    x = np.asarray(logits, np.float64)
    T, E = x.shape
    s = scored_scores(logits, score)
    idx = np.zeros((T, k), np.int32)
    gates = np.zeros((T, k))
    n = E // groups
    for t in range(T):
        key = s[t].copy()
        if bias is None:
            # the logits order the scores, also where the scores round to equal numbers
            key = x[t].copy()
        else:
            key = key + np.asarray(bias, np.float64)
        masked = np.isnan(x[t]) | (x[t] == -np.inf) | np.isnan(key) | (key == -np.inf)
        add = s[t] if bias is None else key         # what a group sums
        best = []
        for g in range(groups):
            live = [e for e in range(g * n, (g + 1) * n) if not masked[e]]
            live.sort(key=lambda e: (-key[e], e))
            if not live:
                best.append(-math.inf)
            elif group_top == 1:
                best.append(key[live[0]])
            else:
                best.append(sum(add[e] for e in live[:2]))
        kept = sorted(range(groups), key=lambda g: (-best[g], g))[:topk_groups]
        cand = [e for g in kept for e in range(g * n, (g + 1) * n)]
        cand.sort(key=lambda e: (bool(masked[e]), 0.0 if masked[e] else -key[e], e))
        idx[t] = cand[:k]
        w = np.array([0.0 if masked[e] else s[t, e] for e in idx[t]])
        if renorm:
            w = w / w.sum() if w.sum() > 0 else np.zeros(k)
        gates[t] = scale * w
    return idx, gates


def route_scored_bwd(d_gates, logits, topk, score="softmax", renorm=True, scale=1.0, gates=None):
    """gates (if given): slots whose gate is 0 are masked and contribute nothing."""
    d = np.asarray(d_gates, np.float64)
    s = scored_scores(logits, score)
    T, E = s.shape
    out = np.zeros((T, E))
    for t in range(T):
        sel = [int(e) for e in topk[t]]
        w = np.array([s[t, e] for e in sel])
        if gates is not None:
            w = np.where(np.asarray(gates)[t] == 0, 0.0, w)
        dw = scale * np.where(w > 0, d[t], 0.0)
        if renorm:
            S = w.sum()
            ds = (dw - (dw * w).sum() / S) / S if S > 0 else np.zeros(len(sel))
        else:
            ds = dw
        full = np.zeros(E)
        full[sel] = np.where(w > 0, ds, 0.0)          # a masked expert's gate is the constant 0
        if score == "sigmoid":
            out[t] = full * s[t] * (1.0 - s[t])
        else:
            out[t] = s[t] * (full - (full * s[t]).sum())
    return out


def combine_bwd(dy, rows, inv_perm, gates, k):
    """(d_rows, d_gates) without rounding d_rows to BF16."""
    dy, rows = np.asarray(dy, np.float64), np.asarray(rows, np.float64)
    T = dy.shape[0]
    d_rows = np.zeros_like(rows)
    d_gates = np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            p = int(inv_perm[t * k + j])
            d_gates[t, j] = float(dy[t] @ rows[p])
            d_rows[p] = (1.0 if gates is None else float(gates[t, j])) * dy[t]
    return d_rows, d_gates


# ----------------------------------------------------------------------------- e4m3

def e4m3_values():
    """Value of each of the 256 codes: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f and 0xff are NaN."""
    out = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = math.nan if (c & 0x7F) == 0x7F else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        out[c] = -v if c & 0x80 else v
    return out


_GRID = e4m3_values()[:127]                      # 0 .. 448, ascending


def e4m3_nearest(v):
    """Codes of the nearest e4m3 values, ties to the even code, magnitudes above 448 saturated, non-finite to NaN."""
    v = np.asarray(v, np.float64)
    a = np.minimum(np.abs(np.where(np.isfinite(v), v, 0.0)), 448.0)
    hi = np.clip(np.searchsorted(_GRID, a, side="left"), 1, 126)
    lo = hi - 1
    dl, dh = a - _GRID[lo], _GRID[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(np.isfinite(v), code, 0x7F)
    return (code | np.where(np.signbit(v) & np.isfinite(v), 0x80, 0)).astype(np.uint8)


def block_exponents(v, block):
    """Smallest e >= -126 with amax <= 448 * 2^e over the finite values of each block; 0 for blocks of zeros."""
    v = np.asarray(v, np.float64)
    M, K = v.shape
    nb = -(-K // block)
    out = np.zeros((M, nb), np.int64)
    for b in range(nb):
        c = v[:, b * block:(b + 1) * block]
        amax = np.abs(np.where(np.isfinite(c), c, 0.0)).max(1)
        for m in range(M):
            if amax[m] == 0.0:
                continue
            e = int(np.frexp(amax[m])[1]) - 10
            while amax[m] > 448.0 * 2.0 ** e:
                e += 1
            out[m, b] = max(e, -126)
    return out


def quantize_rows(v, block=128):
    """(codes uint8 [M, K], exponents [M, blocks])."""
    v = np.asarray(v, np.float64)
    e = block_exponents(v, block)
    s = np.repeat(2.0 ** e.astype(np.float64), block, 1)[:, :v.shape[1]]
    return e4m3_nearest(v / s), e


def rows_values(codes, scales, block):
    """codes [M, K], scales [M, blocks] (numbers) -> values."""
    s = np.repeat(np.asarray(scales, np.float64), block, 1)[:, :codes.shape[1]]
    return e4m3_values()[codes] * s


def weight_values(codes, scales):
    E, N, K = codes.shape
    s = np.repeat(np.repeat(np.asarray(scales, np.float64), 128, 1)[:, :N], 128, 2)[:, :, :K]
    return e4m3_values()[codes] * s


# ----------------------------------------------------------------------------- products

def fp8_gemm(a, w, offsets, bwd=False):
    """(out, mag): rows a [M, R] times their expert's weights, and the same product of magnitudes."""
    E = w.shape[0]
    F = w.shape[2] if bwd else w.shape[1]
    out, mag = np.zeros((a.shape[0], F)), np.zeros((a.shape[0], F))
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            m = w[e] if bwd else w[e].T
            out[lo:hi] = a[lo:hi] @ m
            mag[lo:hi] = np.abs(a[lo:hi]) @ np.abs(m)
    return out, mag


def swiglu(gu):
    f = gu.shape[1] // 2
    g, u = gu[:, :f], gu[:, f:]
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def swiglu_bwd(dh, gu):
    f = gu.shape[1] // 2
    g, u = gu[:, :f], gu[:, f:]
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-g))
    return np.concatenate([dh * u * s * (1.0 + g * (1.0 - s)), dh * g * s], 1)
