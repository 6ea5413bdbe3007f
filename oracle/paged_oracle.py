"""CPU oracle of rotary positions and the paged cache -- TEST INFRASTRUCTURE ONLY.

Float64 NumPy restatements of imem_rotate, imem_append_paged, imem_attend_paged
and imem_gather_paged (include/indexmem.h), one token at a time where that is
the plainest form. The CUDA library shares no code with it. Pinned by
tests/test_oracle_paged.py.
"""
from __future__ import annotations

import math

import numpy as np


def frequencies(rot, base=10000.0, scaling="plain", factor=1.0, low=1.0, high=4.0, orig_len=8192):
    """Radians per position of each rotated pair."""
    out = []
    for i in range(rot // 2):
        theta = base ** (-2.0 * i / rot)
        if scaling == "plain":
            w = 1.0
        elif scaling == "linear":
            w = 0.0
        elif scaling == "band":
            turns = orig_len * theta / (2 * math.pi)
            w = min(1.0, max(0.0, (turns - low) / (high - low)))
        else:
            x = lambda n: rot * math.log(orig_len / (2 * math.pi * n)) / (2 * math.log(base))
            a = min(max(math.floor(x(high)), 0), rot - 1)
            b = min(max(math.ceil(x(low)), 0), rot - 1)
            w = 1.0 - min(1.0, max(0.0, (i - a) / max(b - a, 1e-3)))
        out.append(theta * (w + (1 - w) / factor))
    return np.array(out)


def rotate(x, positions, theta, layout="half", magnitude=1.0, inverse=False):
    """x [T, heads, d]: the first 2 len(theta) dimensions of every head turned."""
    x = np.array(x, dtype=np.float64)
    h = len(theta)
    a = np.asarray(positions, dtype=np.float64)[:, None, None] * theta
    cos, sin = magnitude * np.cos(a), magnitude * np.sin(a) * (-1 if inverse else 1)
    y = x.copy()
    i1, i2 = ((slice(0, h), slice(h, 2 * h)) if layout == "half"
              else (slice(0, 2 * h, 2), slice(1, 2 * h, 2)))
    y[..., i1] = x[..., i1] * cos - x[..., i2] * sin
    y[..., i2] = x[..., i2] * cos + x[..., i1] * sin
    return y


def slots(table_row, page_size, n):
    """Cache rows of positions 0..n-1 of one sequence."""
    return np.array([int(table_row[p // page_size]) * page_size + p % page_size for p in range(n)],
                    dtype=np.int64)


def attend(q, K, V, table, kv_len, tok_start, page_size, scale=None):
    """q [T, Hq, d]; K, V [n_pages, page_size, Hkv, d]. Returns out and lse, and
    what bounds of the rounding errors need: sum_j p_j |v_j| and the largest
    scale * sum_d |q_d k_d| of each row. Rows outside every sequence: NaN."""
    q = np.asarray(q, dtype=np.float64)
    T, Hq, d = q.shape
    Hkv = K.shape[2]
    G = Hq // Hkv
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out = np.full((T, Hq, d), np.nan)
    lse = np.full((T, Hq), np.nan)
    spread, size = np.zeros((T, Hq, d)), np.zeros((T, Hq))
    Kf, Vf = K.reshape(-1, Hkv, d), V.reshape(-1, Hkv, d)
    for s in range(len(kv_len)):
        t0, t1, n = int(tok_start[s]), int(tok_start[s + 1]), int(kv_len[s])
        rows = slots(table[s], page_size, n)
        k, v = np.asarray(Kf[rows], np.float64), np.asarray(Vf[rows], np.float64)
        for t in range(t0, t1):
            seen = n - (t1 - t0) + (t - t0) + 1
            for h in range(Hq):
                if seen <= 0:
                    out[t, h], lse[t, h] = 0.0, -np.inf
                    continue
                x = scale * (k[:seen, h // G] @ q[t, h])
                m = x.max()
                p = np.exp(x - m)
                lse[t, h] = m + math.log(p.sum())
                p /= p.sum()
                out[t, h] = p @ v[:seen, h // G]
                spread[t, h] = p @ np.abs(v[:seen, h // G])
                size[t, h] = scale * (np.abs(k[:seen, h // G]) @ np.abs(q[t, h])).max()
    return out, lse, spread, size
