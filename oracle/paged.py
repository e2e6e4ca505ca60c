"""Paged latent cache, its append and the attention over it, and the residual
RMS norm (oracle).

Position p of sequence b is entry p % page_size of page table[b][p // page_size];
a position past the table, or whose table value is no page, holds no entry.
The new tokens of sequence b are rows [cu[b], cu[b + 1]) at its last positions.
Norm: y = s / sqrt(mean(s^2) + eps) * weight with s = x + residual.  Append:
norm, rotation of the last 64 channels, then the cache-entry encoding.
Attention: row at position p sees positions [0, p], with a window (p - w, p].
All in float64.
"""
from __future__ import annotations

import numpy as np

from .quant import fp4_dequant_rows, fp8_window_dequant_rows


def rms_norm(x, eps, weight=None, residual=None):
    """(sum, normed) in float64."""
    s = np.asarray(x, dtype=np.float64)
    if residual is not None:
        s = s + np.asarray(residual, dtype=np.float64)
    y = s / np.sqrt((s * s).mean(axis=1, keepdims=True) + float(np.float32(eps)))
    return s, y if weight is None else y * np.asarray(weight, dtype=np.float64)


def entry_of(table, page_size, n_pages, b, p):
    """(page, entry in page) of position p of sequence b, or None."""
    if p < 0 or p // page_size >= table.shape[1]:
        return None
    g = int(table[b, p // page_size])
    return (g, p % page_size) if 0 <= g < n_pages else None


def row_positions(cu, kv_len):
    """[(sequence, position)] of the packed rows [0, cu[-1])."""
    return [(b, int(kv_len[b]) - int(cu[b + 1]) + r) for b in range(len(kv_len)) for r in range(int(cu[b]), int(cu[b + 1]))]


def gather(pages, table, b, positions):
    """Decoded entries of those positions of sequence b that hold one:
    (positions kept, float64 [n, 512])."""
    n_pages, page_size, entry = pages.shape
    at = [(p, entry_of(table, page_size, n_pages, b, p)) for p in positions]
    at = [(p, e) for p, e in at if e is not None]
    if not at:
        return np.zeros(0, dtype=np.int64), np.zeros((0, 512))
    raw = np.stack([pages[g, i] for _, (g, i) in at])
    return np.array([p for p, _ in at]), (fp4_dequant_rows if entry == 288 else fp8_window_dequant_rows)(raw)


def attend(q, pos, keys_pos, X, scale, window=0, sink=None):
    """Queries q [n, H, 512] at positions pos [n] over entries X [E, 512] at
    keys_pos -> out [n, H, 512], lse [n, H], and for error bounds
    sum_e w_e |x_e| [n, H, 512], max_e scale * sum_d |q_d x_ed| [n, H] and
    sum_e |x_e| over the entries seen [n, 1, 512]."""
    n, H, _ = q.shape
    q = np.asarray(q, dtype=np.float64)
    scale = float(np.float32(scale))
    out, mass = np.zeros((n, H, 512)), np.zeros((n, H, 512))
    lse, size, total = np.full((n, H), -np.inf), np.zeros((n, H)), np.zeros((n, 1, 512))
    for t in range(n):
        see = keys_pos <= pos[t]
        if window:
            see &= keys_pos > pos[t] - window
        x = X[see]
        s = np.full(H, -np.inf) if sink is None else np.asarray(sink, dtype=np.float64)
        logit = (q[t] @ x.T) * scale
        m = np.maximum(s, logit.max(axis=1)) if len(x) else s
        with np.errstate(invalid="ignore"):
            p = np.exp(logit - m[:, None]) if len(x) else np.zeros((H, 0))
            z = p.sum(axis=1) + np.where(s == -np.inf, 0.0, np.exp(s - m))
        with np.errstate(divide="ignore"):
            lse[t] = np.where(z > 0, m + np.log(z), -np.inf)
        if len(x):
            w = p / np.where(z > 0, z, 1.0)[:, None]
            out[t], mass[t] = w @ x, w @ np.abs(x)
            size[t] = scale * (np.abs(q[t]) @ np.abs(x).T).max(axis=1)
            total[t] = np.abs(x).sum(axis=0)
    return out, lse, mass, size, total
