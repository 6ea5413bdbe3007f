"""CPU pins of the paged oracle against something other than itself, and the
refusals of the paged calls (host validation, no device needed)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from learned_kv_cache_indexmem_b200 import binding as B
from oracle import paged_oracle as po


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation_is_relative_and_keeps_norms(layout):
    rng = np.random.default_rng(0)
    th = po.frequencies(32)
    q, k = rng.standard_normal((1, 1, 48)), rng.standard_normal((1, 1, 48))
    dots = []
    for shift in (0, 5, 1000):
        a = po.rotate(q, [17 + shift], th, layout)
        b = po.rotate(k, [3 + shift], th, layout)
        dots.append(float((a * b).sum()))
        assert abs(np.linalg.norm(a) - np.linalg.norm(q)) < 1e-12
        assert np.array_equal(a[..., 32:], q[..., 32:])
    assert np.allclose(dots, dots[0], atol=1e-9)
    back = po.rotate(po.rotate(q, [12345], th, layout), [12345], th, layout, inverse=True)
    assert np.allclose(back, q, atol=1e-12)


def test_rotation_against_complex_numbers():
    rng = np.random.default_rng(1)
    th = po.frequencies(16, base=500.0)
    x = rng.standard_normal((4, 2, 16))
    pos = np.array([0, 1, 77, -5])
    z = x[..., 0::2] + 1j * x[..., 1::2]
    w = z * np.exp(1j * pos[:, None, None] * th)
    y = po.rotate(x, pos, th, "interleaved")
    assert np.allclose(y[..., 0::2], w.real) and np.allclose(y[..., 1::2], w.imag)
    # the half layout is the interleaved one under a permutation of the dimensions
    perm = np.concatenate([np.arange(0, 16, 2), np.arange(1, 16, 2)])
    assert np.allclose(po.rotate(x[..., perm], pos, th, "half"), y[..., perm])


def test_inverse_rotation_is_the_gradient():
    rng = np.random.default_rng(2)
    th = po.frequencies(16)
    x, g = rng.standard_normal((3, 1, 16)), rng.standard_normal((3, 1, 16))
    pos = [4, 9, 1000]
    grad = po.rotate(g, pos, th, "half", 1.3, inverse=True)
    for i in range(16):
        e = np.zeros_like(x)
        e[..., i] = 1e-6
        num = ((po.rotate(x + e, pos, th, "half", 1.3) - po.rotate(x - e, pos, th, "half", 1.3)) * g).sum(-1) / 2e-6
        assert np.allclose(num[:, 0], grad[:, 0, i], atol=1e-6)


def test_scalings_hand_worked():
    plain = po.frequencies(128, base=500000.0)
    assert plain[0] == 1.0 and np.allclose(plain[32], 500000.0 ** -0.5)
    assert np.allclose(po.frequencies(128, 500000.0, "linear", 4.0), plain / 4)
    band = po.frequencies(128, 500000.0, "band", 8.0, 1.0, 4.0, 8192)
    turns = 8192 * plain / (2 * math.pi)
    assert np.allclose(band[turns > 4], plain[turns > 4])
    assert np.allclose(band[turns < 1], plain[turns < 1] / 8)
    assert ((band <= plain * (1 + 1e-12)) & (band >= plain / 8 * (1 - 1e-12))).all()
    ramp = po.frequencies(128, 10000.0, "ramp", 16.0, 1.0, 32.0, 4096)
    # pairs below floor(64 ln(4096/(64 pi))/ln 1e4) = 20 kept, from ceil(64 ln(4096/(2 pi))/ln 1e4) = 46 on stretched
    p = po.frequencies(128, 10000.0)
    assert np.allclose(ramp[:21], p[:21]) and np.allclose(ramp[46:], p[46:] / 16) and ramp[30] < p[30]


def test_ramp_past_the_last_pair_hand_worked():
    """The upper border is an index of dimensions, not of pairs: base 10000, 128
    dimensions, 131072 positions: from floor(64 ln(131072/(64 pi))/ln 1e4) = 45 to
    ceil(64 ln(131072/(2 pi))/ln 1e4) = 70, so that pair 63 keeps 1 - 18/25."""
    p = po.frequencies(128, 10000.0)
    ramp = po.frequencies(128, 10000.0, "ramp", 16.0, 1.0, 32.0, 131072)
    assert np.allclose(ramp[:46], p[:46], rtol=1e-14)
    w = 1 - (np.arange(46, 64) - 45) / 25
    assert np.allclose(ramp[46:], p[46:] * (w + (1 - w) / 16), rtol=1e-14)
    # 64 dimensions, 65536 positions: 20 to 33, pair 31 keeps 1 - 11/13
    p = po.frequencies(64, 10000.0)
    ramp = po.frequencies(64, 10000.0, "ramp", 4.0, 1.0, 32.0, 65536)
    w = 1 - (np.arange(21, 32) - 20) / 13
    assert np.allclose(ramp[:21], p[:21], rtol=1e-14)
    assert np.allclose(ramp[21:], p[21:] * (w + (1 - w) / 4), rtol=1e-14)


def test_attend_against_sdpa():
    rng = np.random.default_rng(3)
    Hq, Hkv, d, page = 4, 2, 8, 4
    news, lens = [3, 1, 5, 0], [10, 1, 5, 6]
    start = np.concatenate([[0], np.cumsum(news)])
    table = rng.permutation(16)[:12].reshape(4, 3)
    K, V = rng.standard_normal((2, 16, page, Hkv, d))
    q = rng.standard_normal((9, Hq, d))
    out, lse, spread, _ = po.attend(q, K, V, table, lens, start, page)
    for s in range(4):
        rows = po.slots(table[s], page, lens[s])
        k = torch.tensor(K.reshape(-1, Hkv, d)[rows]).transpose(0, 1).repeat_interleave(2, 0)
        v = torch.tensor(V.reshape(-1, Hkv, d)[rows]).transpose(0, 1).repeat_interleave(2, 0)
        qs = torch.tensor(q[start[s]:start[s + 1]]).transpose(0, 1)
        n = news[s]
        if not n:
            continue
        mask = torch.arange(lens[s])[None] <= (lens[s] - n + torch.arange(n))[:, None]
        ref = torch.nn.functional.scaled_dot_product_attention(qs, k, v, attn_mask=mask)
        assert np.allclose(out[start[s]:start[s + 1]], ref.transpose(0, 1).numpy(), atol=1e-12)
        sc = (qs @ k.transpose(1, 2) / math.sqrt(d)).masked_fill(~mask, -math.inf)
        assert np.allclose(lse[start[s]:start[s + 1]], torch.logsumexp(sc, -1).T.numpy())
    assert (spread >= np.abs(out) - 1e-12).all()


# ---------------------------------------------------------------- refusals

def _fake_context(**kw):
    """A context as far as host validation looks at it: its configuration, and
    a device that is never current, so that no call can pass it."""
    cfg = B.make_config(**{**dict(hidden=512, n_q_heads=8, n_kv_heads=2, head_dim=64, idx_dim=32,
                                  mem_r=32, lam=0.99, dtype=B.BF16), **kw})
    buf = ctypes.create_string_buffer(8192)
    ctypes.memmove(buf, ctypes.byref(cfg), ctypes.sizeof(cfg))
    ctypes.c_int.from_buffer(buf, ctypes.sizeof(cfg)).value = -1
    return buf


def _rope(**kw):
    base = dict(rot_dim=64, layout=0, scaling=0, orig_len=8192, base=1e4, factor=1.0, low=1.0,
                high=4.0, magnitude=1.0)
    base.update(kw)
    return B.Rope(**base)


def _name(fn):
    with pytest.raises(B.IndexMemError) as ei:
        fn()
    return ei.value.name


PAST = ("IMEM_ERR_CUDA", "IMEM_ERR_INVALID_ARG")   # all arguments accepted: no such device


@pytest.mark.parametrize("kw,code", [
    (dict(rot_dim=0), "IMEM_ERR_UNSUPPORTED"), (dict(rot_dim=24), "IMEM_ERR_UNSUPPORTED"),
    (dict(rot_dim=80), "IMEM_ERR_UNSUPPORTED"), (dict(layout=2), "IMEM_ERR_INVALID_ARG"),
    (dict(scaling=4), "IMEM_ERR_INVALID_ARG"), (dict(base=1.0), "IMEM_ERR_INVALID_ARG"),
    (dict(base=math.nan), "IMEM_ERR_INVALID_ARG"), (dict(base=math.inf), "IMEM_ERR_INVALID_ARG"),
    (dict(magnitude=0.0), "IMEM_ERR_INVALID_ARG"),
    (dict(scaling=1, factor=0.5), "IMEM_ERR_INVALID_ARG"),
    (dict(scaling=2, low=4.0), "IMEM_ERR_INVALID_ARG"),
    (dict(scaling=3, low=0.0), "IMEM_ERR_INVALID_ARG"),
    (dict(scaling=3, orig_len=0), "IMEM_ERR_INVALID_ARG"),
    (dict(scaling=3, high=math.inf), "IMEM_ERR_INVALID_ARG"),
])
def test_set_rope_refusals(kw, code):
    ctx = _fake_context()
    assert _name(lambda: B.set_rope(ctx, _rope(**kw))) == code
    B.set_rope(ctx, _rope())
    B.set_rope(ctx, None)


def _paged(**kw):
    base = dict(k=16, v=16, block_table=16, kv_len=16, n_pages=4, page_size=16, max_pages=2)
    base.update(kw)
    return B.make_paged(**base)


@pytest.mark.parametrize("kw,code", [
    (dict(k=0), "IMEM_ERR_INVALID_ARG"), (dict(v=8), "IMEM_ERR_ALIGN"),
    (dict(block_table=0), "IMEM_ERR_INVALID_ARG"), (dict(kv_len=4), "IMEM_ERR_ALIGN"),
    (dict(n_pages=0), "IMEM_ERR_SHAPE"), (dict(max_pages=0), "IMEM_ERR_SHAPE"),
    (dict(page_size=8), "IMEM_ERR_UNSUPPORTED"), (dict(page_size=48), "IMEM_ERR_UNSUPPORTED"),
    (dict(page_size=2048), "IMEM_ERR_UNSUPPORTED"),
    (dict(n_pages=1 << 22, page_size=1024), "IMEM_ERR_SHAPE"),
])
def test_paged_cache_refusals(kw, code):
    ctx = _fake_context()
    B.set_rope(ctx, _rope())
    pg = _paged(**kw)
    assert _name(lambda: B.append_paged(ctx, 1, 4, None, None, 16, 0, 16, 0, None, 0, None, 0, 1, pg, 0)) == code
    assert _name(lambda: B.attend_paged(ctx, 1, 4, None, 4, 32, 16, 0, pg, 0.0, 16, 0, None, 0)) == code
    assert _name(lambda: B.gather_paged(ctx, 1, 4, None, 0, pg, 16, 16, 4, 0)) == code


def test_argument_refusals():
    ctx, bare = _fake_context(), _fake_context()
    B.set_rope(ctx, _rope())

    def rotate(c=ctx, n=4, pos=16, q=16, qs=0, qo=16, k=16, ks=0, ko=16, inv=0):
        return _name(lambda: B.rotate(c, n, pos, q, qs, qo, 0, k, ks, ko, 0, inv, 0))

    assert rotate() in PAST
    assert rotate(c=bare) == "IMEM_ERR_INVALID_ARG"
    assert rotate(q=None, k=None) == "IMEM_ERR_INVALID_ARG"
    assert rotate(pos=None) == "IMEM_ERR_INVALID_ARG" and rotate(pos=8) == "IMEM_ERR_ALIGN"
    assert rotate(qo=None) == "IMEM_ERR_INVALID_ARG" and rotate(ko=2) == "IMEM_ERR_ALIGN"
    assert rotate(n=-1) == "IMEM_ERR_SHAPE" and rotate(n=1 << 25) == "IMEM_ERR_SHAPE"
    assert rotate(qs=511) == "IMEM_ERR_SHAPE" and rotate(ks=129) == "IMEM_ERR_ALIGN"
    assert rotate(inv=2) == "IMEM_ERR_INVALID_ARG"

    def append(c=ctx, b=2, n=4, start=16, pos=None, k=16, ks=0, v=16, vs=0, q=16, qo=16, rot=1):
        return _name(lambda: B.append_paged(c, b, n, start, pos, k, ks, v, vs, q, 0, qo, 0, rot, _paged(), 0))

    assert append() in PAST and append(q=None, qo=None) in PAST and append(c=bare, rot=0) in PAST
    assert append(c=bare) == "IMEM_ERR_INVALID_ARG" and append(rot=3) == "IMEM_ERR_INVALID_ARG"
    assert append(b=0) == "IMEM_ERR_SHAPE" and append(b=65536) == "IMEM_ERR_SHAPE"
    assert append(b=3, start=None) == "IMEM_ERR_SHAPE" and append(start=8) == "IMEM_ERR_ALIGN"
    assert append(pos=4) == "IMEM_ERR_ALIGN" and append(k=None) == "IMEM_ERR_INVALID_ARG"
    assert append(vs=120) == "IMEM_ERR_SHAPE" and append(qo=None) == "IMEM_ERR_INVALID_ARG"

    def attend(b=2, n=4, start=16, mx=4, ml=32, q=16, qs=0, sc=0.0, out=16, os=0, lse=None):
        return _name(lambda: B.attend_paged(ctx, b, n, start, mx, ml, q, qs, _paged(), sc, out, os, lse, 0))

    assert attend() in PAST
    assert attend(sc=-1.0) == "IMEM_ERR_INVALID_ARG" and attend(sc=math.nan) == "IMEM_ERR_INVALID_ARG"
    assert attend(sc=math.inf) == "IMEM_ERR_INVALID_ARG"
    assert attend(mx=5) == "IMEM_ERR_SHAPE" and attend(mx=-1) == "IMEM_ERR_SHAPE"
    assert attend(ml=-1) == "IMEM_ERR_SHAPE" and attend(lse=4) == "IMEM_ERR_ALIGN"
    assert attend(out=None) == "IMEM_ERR_INVALID_ARG" and attend(os=100) == "IMEM_ERR_SHAPE"

    def gather(b=2, n=4, idx=16, st=4, K=16, V=16, cap=4):
        return _name(lambda: B.gather_paged(ctx, b, n, idx, st, _paged(), K, V, cap, 0))

    assert gather() in PAST and gather(idx=None, st=0) in PAST
    assert gather(b=0) == "IMEM_ERR_SHAPE" and gather(n=-1) == "IMEM_ERR_SHAPE"
    assert gather(cap=3) == "IMEM_ERR_SHAPE" and gather(st=3) == "IMEM_ERR_SHAPE"
    assert gather(K=None) == "IMEM_ERR_INVALID_ARG" and gather(idx=4) == "IMEM_ERR_ALIGN"


def test_null_context():
    pg = _paged()
    for fn in (lambda: B.set_rope(None, _rope()),
               lambda: B.rotate(None, 4, 16, 16, 0, 16, 0, 16, 0, 16, 0, 0, 0),
               lambda: B.append_paged(None, 1, 4, 16, None, 16, 0, 16, 0, None, 0, None, 0, 1, pg, 0),
               lambda: B.attend_paged(None, 1, 4, 16, 4, 16, 16, 0, pg, 0.0, 16, 0, None, 0),
               lambda: B.gather_paged(None, 1, 4, 16, 4, pg, 16, 16, 4, 0)):
        assert _name(fn) == "IMEM_ERR_INVALID_ARG"
