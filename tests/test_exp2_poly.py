"""The exponential that the bf16 attention takes on the FMA units (exp2_fma in
csrc/attend_tc.cu), recomputed in fp32 from the constants in the source: its
stated error, its ends, its steps between powers of two.

A step is a fused multiply-add rounded once: emulated in fp64, whose own
rounding (2^-53) is far below."""
import os
import re

import numpy as np

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "learned_kv_cache_indexmem_b200",
                   "csrc", "attend_tc.cu")


def _exp2_fma(y):
    body = re.search(r"void exp2_fma\(.*?\n}\n", open(SRC).read(), re.S).group(0)
    magic = float(re.search(r"magic = tc::pack2\(([\d.]+)f", body).group(1))
    low = -float(re.search(r"fmaxf\(y0, -([\d.]+)f\)", body).group(1))
    first = re.search(r"fma2\(f, c2\(([\d.]+)f\), c2\(([\d.]+)f\)\)", body)
    coeffs = [float(first.group(1)), float(first.group(2))]
    coeffs += [float(x) for x in re.findall(r"p = tc::fma2\(f, p, c2\(([\d.]+)f\)\)", body)]
    assert len(coeffs) == 6 and magic == 1.5 * 2 ** 23 and low == -126
    f32 = lambda x: np.asarray(x, np.float64).astype(np.float32).astype(np.float64)
    y = np.maximum(f32(y), low)
    t = f32(y + magic)
    n = t - magic
    f = f32(y - n)
    p = np.full_like(f, float(np.float32(coeffs[0])))
    for c in coeffs[1:]:
        p = f32(f * p + float(np.float32(c)))
    bits = p.astype(np.float32).view(np.int32) + (t.astype(np.float32).view(np.int32) << 23)   # wraps, as there
    return bits.astype(np.int32).view(np.float32).astype(np.float64)


def test_relative_error():
    y = np.concatenate([np.linspace(-0.5, 0.5, 400001), np.linspace(-126, 8, 400001),
                        np.random.default_rng(0).uniform(-126, 8, 400000)])
    y = y.astype(np.float32).astype(np.float64)
    err = np.abs(_exp2_fma(y) / np.exp2(y) - 1)
    assert err.max() <= 2.4e-7


def test_ends():
    got = _exp2_fma(np.array([-126.0, -127.0, -1e30, -np.inf, 0.0, 8.0, 1.0, -1.0]))
    want = np.array([2.0 ** -126] * 4 + [1.0, 256.0, 2.0, 0.5])
    assert (np.abs(got / want - 1) <= 2.4e-7).all()
