"""Rotary positions and the paged cache on the GPU against the float64 oracle
(oracle/paged_oracle.py), through the layer's public methods.

Tolerances (e = torch.finfo(dtype).eps / 2, the largest relative rounding of
one value; u = 2^-24 for fp32 arithmetic):
  rotate, append  fp32 cos and sin off by at most 4u (phase to 2^-32 turns,
           sincospif to 2 ulp, one product with the magnitude), two products
           and a sum: |dy| <= 16u m |(x1, x2)| + e |y|; copies are exact.
  attend   a logit is a sum of d products in fp32 (up to 4u each on the tensor
           cores, which truncate): ds = 4 u (d + 4) max_j scale sum_d |q_d k_jd|;
           a probability is then off by 2 ds (its own exponent and the
           normaliser's) + 16u (exp2, the factors of the running maximum) and,
           for bf16, by its rounding e; the sums over n keys add 4 u (n + 4):
           |do| <= (2 ds + 16u + 4u (n + 4) + [e]) sum_j p_j |v_j| + e |o|,
           |dlse| <= ds + 4u (n + 4) + 4u |lse| + 16u.
"""
import dataclasses

import numpy as np
import pytest
import torch

from learned_kv_cache_indexmem_b200 import binding as B
from learned_kv_cache_indexmem_b200 import synth
from learned_kv_cache_indexmem_b200.layer import IndexMemLayer, PagedCache
from oracle import indexmem_oracle as om
from oracle import paged_oracle as po

from .parity import check_decode, check_memory, ill_conditioned, to_np

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def layer(dev, hq=8, hkv=2, d=64, dtype="bf16", **rope):
    shape = synth.LayerShape(hidden=512, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, idx_dim=32,
                             mem_r=32, lam=0.99, dtype=dtype)
    lay = IndexMemLayer.from_shape(shape, synth.make_weights(shape, 0, dev))
    lay.set_rope(**{**dict(rot_dim=d, base=500000.0), **rope})
    return lay


@dataclasses.dataclass
class Batch:
    q: torch.Tensor
    k: torch.Tensor
    v: torch.Tensor
    start: torch.Tensor
    cache: PagedCache
    news: list
    lens: list
    live: torch.Tensor    # cache rows below their sequence's length


def batch(dev, news, lens, hq=8, hkv=2, d=64, dtype="bf16", page=16, seed=0, pad=0, stale=float("nan"),
          fused=True):
    """New tokens as slices of one joint projection and a cache whose live rows
    are drawn and whose other rows (free pages, slots past a length) hold
    `stale`. pad: token rows behind the last sequence."""
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    T, b = sum(news) + pad, len(news)
    qkv = torch.randn(T, (hq + 2 * hkv) * d, generator=g, device=dev).to(dt)
    q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([hq * d, hkv * d, hkv * d], 1))
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    per = max(1, max(-(-max(n, 0) // page) for n in lens)) + 1
    pages = b * per + 3
    K = torch.randn(pages, page, hkv, d, generator=g, device=dev).to(dt)
    V = torch.randn(pages, page, hkv, d, generator=g, device=dev).to(dt)
    K *= 1 + 2 * (torch.rand(pages, page, 1, 1, generator=g, device=dev) < 0.05)
    table = torch.randperm(pages, generator=g, device=dev)[:b * per].view(b, per).to(torch.int32)
    live = torch.zeros(pages * page, dtype=torch.bool, device=dev)
    for s in range(b):
        live[torch.from_numpy(po.slots(table[s].tolist(), page, max(lens[s], 0))).to(dev)] = True
        table[s, -(-max(lens[s], 0) // page):] = -1    # nothing past the length is read
    K.view(-1, hkv, d)[~live] = stale
    V.view(-1, hkv, d)[~live] = stale
    ints = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)
    return Batch(q, k, v, ints(np.concatenate([[0], np.cumsum(news)])),
                 PagedCache(K, V, table, ints(lens)), news, lens, live)


def check_rotated(y, x, positions, theta, layout, m=1.0, inverse=False):
    e = torch.finfo(y.dtype).eps / 2
    y, x = to_np(y) if y.dtype != torch.float32 else y.cpu().numpy().astype(np.float64), to_np(x)
    ref = po.rotate(x, positions, theta, layout, m, inverse)
    swapped = po.rotate(np.abs(x), np.zeros(len(x)), theta, layout, m)    # m |x1|, m |x2|
    h = len(theta)
    i1, i2 = ((slice(0, h), slice(h, 2 * h)) if layout == "half"
              else (slice(0, 2 * h, 2), slice(1, 2 * h, 2)))
    tol = np.zeros_like(ref)
    tol[..., i1] = tol[..., i2] = 16 * U * np.hypot(swapped[..., i1], swapped[..., i2])
    tol[..., :2 * h] += e * np.abs(ref[..., :2 * h])
    err = np.abs(y - ref)
    assert (err <= tol).all(), "rotation off by %.3g of its tolerance" % (err / np.maximum(tol, 1e-30)).max()


def check_attend(out, lse, bt, lay_dims, scale=None, q=None, max_new=None):
    q = bt.q if q is None else q
    hq, d = q.shape[1:]
    page = bt.cache.K.shape[1]
    start = bt.start.cpu().numpy()
    ref, rl, spread, size = po.attend(to_np(q), to_np(bt.cache.K), to_np(bt.cache.V),
                                      bt.cache.block_table.cpu().numpy(), bt.lens, start, page, scale)
    e = torch.finfo(out.dtype).eps / 2
    n = max(max(bt.lens), 1)
    ds = 4 * U * (d + 4) * size
    rel = 2 * ds + 16 * U + 4 * U * (n + 4) + (e if out.dtype == torch.bfloat16 else 0.0)
    T = int(start[-1])
    o = to_np(out)[:T]
    tol = rel[:T, :, None] * spread[:T] + e * np.abs(ref[:T])
    err = np.abs(o - ref[:T])
    assert (err <= tol).all(), "output off: %.3g (tolerance %.3g there)" % (
        err.max(), tol.reshape(-1)[err.argmax()])
    if lse is not None:
        l = lse.cpu().numpy().astype(np.float64)[:T]
        seen = np.isfinite(rl[:T])
        assert np.array_equal(l[~seen], rl[:T][~seen])
        tl = (ds + 4 * U * (n + 4) + 16 * U)[:T] + 4 * U * np.abs(np.where(seen, rl[:T], 0))
        assert (np.abs(l[seen] - rl[:T][seen]) <= tl[seen]).all()


# ------------------------------------------------------------------- rotations

@pytest.mark.parametrize("dtype,d,rot,layout,scaling", [
    ("bf16", 128, 128, "half", "plain"), ("bf16", 128, 96, "interleaved", "band"),
    ("bf16", 64, 16, "half", "linear"), ("fp32", 64, 64, "half", "ramp"),
    ("fp32", 128, 32, "interleaved", "plain"), ("fp32", 64, 48, "half", "band"),
])
def test_rotate(cuda_device, dtype, d, rot, layout, scaling):
    kw = dict(base=500000.0, scaling=scaling, factor=8.0, low=1.0,
              high=32.0 if scaling == "ramp" else 4.0, orig_len=8192)
    lay = layer(cuda_device, d=d, dtype=dtype, rot_dim=rot, layout=layout, magnitude=1.25, **kw)
    th = po.frequencies(rot, **kw)
    for T in (1, 7, 300, 2500):      # one, two and eight tokens per CTA, ragged ends
        bt = batch(cuda_device, [T], [T], d=d, dtype=dtype, seed=T)
        g = np.random.default_rng(T)
        pos = g.integers(-(1 << 20), 1 << 20, T).astype(np.int32)
        pos[0] = 0 if T > 1 else 1000003
        p = torch.from_numpy(pos).to(cuda_device)
        q, k = lay.rotate(bt.q, bt.k, p)
        check_rotated(q, bt.q, pos, th, layout, 1.25)
        check_rotated(k, bt.k, pos, th, layout, 1.25)
        # only one tensor, rotated the other way, in place on its strided rows
        want = po.rotate(to_np(bt.k), pos, th, layout, 1.25, True)
        before = bt.k.clone()
        none, k2 = lay.rotate(None, bt.k, p, k_out=bt.k, inverse=True)
        assert none is None and k2.data_ptr() == bt.k.data_ptr()
        check_rotated(k2, before, pos, th, layout, 1.25, True)
        assert np.allclose(to_np(k2), want, atol=0.1)
        assert torch.equal(bt.q, batch(cuda_device, [T], [T], d=d, dtype=dtype, seed=T).q)
    lay.sync()
    lay.close()


@pytest.mark.parametrize("rot,orig_len", [(128, 131072), (64, 65536), (128, 1 << 24), (32, 100)])
def test_ramp_borders(cuda_device, rot, orig_len):
    """Ramps that end past the last pair, or before the first."""
    kw = dict(base=10000.0, scaling="ramp", factor=16.0, low=1.0, high=32.0, orig_len=orig_len)
    lay = layer(cuda_device, d=128, dtype="fp32", rot_dim=rot, layout="half", **kw)
    bt = batch(cuda_device, [300], [300], d=128, dtype="fp32")
    pos = np.random.default_rng(rot).integers(0, 1 << 20, 300).astype(np.int32)
    q, _ = lay.rotate(bt.q, None, torch.from_numpy(pos).to(cuda_device))
    check_rotated(q, bt.q, pos, po.frequencies(rot, **kw), "half")
    lay.sync()
    lay.close()


def test_far_positions_keep_their_angle(cuda_device):
    lay = layer(cuda_device, d=64, dtype="fp32", base=10000.0)
    pos = np.array([2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1, 131071], dtype=np.int32)
    x = torch.ones(4, 8, 64, device=cuda_device)
    y, _ = lay.rotate(x, None, torch.from_numpy(pos).to(cuda_device))
    ref = po.rotate(to_np(x), pos, po.frequencies(64), "half")
    # theta in fp64 is off by 2^-53 of itself: at 2^31 the angle by 2^31 * 2^-53
    tol = 16 * U * np.sqrt(2) + 2.0 ** 31 * 2.0 ** -52 * np.sqrt(2) + U * np.abs(ref)
    assert (np.abs(y.cpu().numpy() - ref) <= tol).all()
    lay.close()


# ---------------------------------------------------------------------- append

@pytest.mark.parametrize("dtype,d,hq,hkv,page,news,lens", [
    ("bf16", 128, 32, 8, 64, [1, 1, 1], [1, 64, 1000]),
    ("bf16", 64, 8, 2, 16, [5, 0, 33, 1], [5, 7, 100, 17]),
    ("fp32", 64, 4, 4, 32, [700, 1], [700, 90]),
    ("bf16", 64, 8, 1, 256, [2600], [2601]),
])
def test_append(cuda_device, dtype, d, hq, hkv, page, news, lens):
    lay = layer(cuda_device, hq, hkv, d, dtype, rot_dim=d // 2, layout="interleaved")
    th = po.frequencies(d // 2, 500000.0)
    bt = batch(cuda_device, news, lens, hq, hkv, d, dtype, page, pad=3)
    K0, V0 = bt.cache.K.clone(), bt.cache.V.clone()
    q_out = torch.full_like(bt.q, 7.0)
    got = lay.append_paged(bt.k, bt.v, bt.cache, tok_start=bt.start, q=bt.q, q_out=q_out)
    lay.sync()
    assert got.data_ptr() == q_out.data_ptr()
    T = sum(news)
    pos = np.concatenate([np.arange(l - n, l) for n, l in zip(news, lens)]).astype(np.int64)
    rows = np.concatenate([po.slots(bt.cache.block_table[s].tolist(), page, lens[s])[lens[s] - n:]
                           for s, n in enumerate(news)])
    check_rotated(got[:T], bt.q[:T], pos, th, "interleaved")
    assert (got[T:] == 7.0).all()                      # rows behind the last sequence
    Kf, Vf = bt.cache.K.view(-1, hkv, d), bt.cache.V.view(-1, hkv, d)
    rt = torch.from_numpy(rows).to(cuda_device)
    check_rotated(Kf[rt], bt.k[:T], pos, th, "interleaved")
    assert torch.equal(Vf[rt], bt.v[:T])
    other = torch.ones(Kf.shape[0], dtype=torch.bool, device=cuda_device)
    other[rt] = False
    for a, b in ((Kf, K0.view_as(Kf)), (Vf, V0.view_as(Vf))):   # everything else as it was
        assert torch.equal(a[other].nan_to_num(3.0), b[other].nan_to_num(3.0))
    # positions of the caller's own, no rotation, no queries
    own = torch.arange(T + 3, dtype=torch.int32, device=cuda_device) * 11
    lay.append_paged(bt.k, bt.v, bt.cache, tok_start=bt.start, positions=own)
    check_rotated(Kf[rt], bt.k[:T], 11 * np.arange(T), th, "interleaved")
    assert lay.append_paged(bt.k, bt.v, bt.cache, tok_start=bt.start, rotate=False) is None
    assert torch.equal(Kf[rt], bt.k[:T])
    lay.sync()
    lay.close()


def test_append_padding_in_front_and_bad_pages(cuda_device):
    lay = layer(cuda_device)
    # uniform chunks of 6, the second sequence padded in front by 4
    bt = batch(cuda_device, [6, 6], [20, 2])
    lay.append_paged(bt.k, bt.v, bt.cache)            # tok_start None
    lay.sync()
    rows = torch.from_numpy(po.slots(bt.cache.block_table[1].tolist(), 16, 2)).to(cuda_device)
    assert torch.equal(bt.cache.V.view(-1, 2, 64)[rows], bt.v[10:12])
    out, lse = lay.attend_paged(bt.q, bt.cache, return_lse=True)
    lay.sync()
    assert (out[6:10] == 0).all() and (lse[6:10] == -np.inf).all()
    check_attend(out, lse, bt, None)
    # a page outside the cache, a length beyond the table, token ranges that
    # descend: reported, nothing else written, the context usable afterwards
    for bad in ("page", "page-", "len", "start"):
        bt = batch(cuda_device, [6, 6], [20, 40])
        V0, V_table = bt.cache.V.clone(), bt.cache.block_table.clone()
        if bad == "page":
            bt.cache.block_table[1, 2] = bt.cache.K.shape[0]
        elif bad == "page-":
            bt.cache.block_table[1, 2] = -2
        elif bad == "len":
            bt.cache.kv_len[1] = 16 * bt.cache.block_table.shape[1] + 1
        else:
            bt.start[2] = 5
        for call in (lambda: lay.append_paged(bt.k, bt.v, bt.cache, tok_start=bt.start),
                     lambda: lay.attend_paged(bt.q, bt.cache, tok_start=bt.start)):
            call()
            with pytest.raises(B.IndexMemError) as ei:
                lay.sync()
            assert ei.value.name == "IMEM_ERR_RANGE"
            lay.sync()
        if bad == "start":      # the whole call's results are unspecified
            continue
        rows = torch.from_numpy(po.slots(bt.cache.block_table[0].tolist(), 16, 20)).to(cuda_device)
        assert torch.equal(bt.cache.V.view(-1, 2, 64)[rows[14:]], bt.v[:6])
        mine = torch.zeros_like(bt.live)
        mine[rows] = True
        held = torch.from_numpy(po.slots(V_table[1].tolist(), 16, 40)).to(cuda_device)
        mine[held] = True
        assert torch.equal(bt.cache.V.view(-1, 2, 64)[~mine].nan_to_num(3.0), V0.view(-1, 2, 64)[~mine].nan_to_num(3.0))
    bt = batch(cuda_device, [6, 6], [20, 40])
    out, lse = lay.attend_paged(bt.q, bt.cache, tok_start=bt.start, return_lse=True)
    lay.sync()
    check_attend(out, lse, bt, None)
    lay.close()


# ---------------------------------------------------------------------- attend

CASES = [
    # dtype, d, hq, hkv, page, new tokens, lengths
    ("bf16", 128, 32, 8, 64, [1], [1]),
    ("bf16", 128, 32, 8, 64, [1], [4096]),
    ("bf16", 128, 32, 8, 16, [1, 1, 1, 1], [17, 640, 641, 63]),
    ("bf16", 64, 8, 2, 16, [1, 1], [2049, 130]),
    ("bf16", 64, 8, 8, 128, [1, 1, 1], [300, 1, 128]),
    ("bf16", 128, 8, 1, 32, [1, 2, 1], [1500, 2, 33]),
    ("bf16", 64, 16, 2, 1024, [2, 1], [1025, 1024]),
    ("bf16", 128, 32, 8, 16, [5, 3, 4, 1], [2000, 700, 4, 129]),
    ("bf16", 128, 8, 2, 64, [64, 33], [64, 300]),
    ("bf16", 128, 8, 2, 128, [300], [1000]),
    ("bf16", 64, 8, 2, 16, [257, 1, 0, 130], [257, 400, 9, 131]),
    ("bf16", 64, 4, 4, 32, [400], [401]),
    ("bf16", 128, 8, 1, 256, [129], [700]),
    ("bf16", 64, 2, 1, 64, [128, 127], [128, 2000]),
    ("bf16", 128, 2, 2, 512, [513, 255], [520, 255]),
    ("bf16", 128, 8, 2, 16, [1, 1, 1], [9000, 12001, 30000]),     # many turns of the ring
    ("bf16", 64, 8, 2, 64, [2, 5], [20001, 9000]),
    ("bf16", 128, 16, 8, 32, [12, 11], [7000, 5001]),
    ("bf16", 64, 8, 2, 32, [70, 3], [9000, 11]),
    ("bf16", 128, 8, 1, 16, [4], [40]),                           # fewer tokens than a tile has rows
    ("bf16", 64, 2, 2, 16, [25], [25]),
    ("fp32", 64, 8, 2, 16, [1, 1], [1, 1030]),
    ("fp32", 128, 8, 2, 64, [1], [5000]),
    ("fp32", 64, 8, 2, 16, [100, 1, 0, 31], [100, 400, 5, 90]),
    ("fp32", 128, 4, 4, 32, [65], [700]),
    ("fp32", 128, 1, 1, 32, [17, 30], [5000, 31]),
    ("fp32", 64, 8, 2, 64, [8, 5, 1], [3001, 5, 64]),
    ("fp32", 64, 8, 1, 128, [3, 9], [300, 9]),
]


@pytest.mark.parametrize("dtype,d,hq,hkv,page,news,lens", CASES)
def test_attend(cuda_device, dtype, d, hq, hkv, page, news, lens):
    lay = layer(cuda_device, hq, hkv, d, dtype)
    bt = batch(cuda_device, news, lens, hq, hkv, d, dtype, page, pad=2)
    out = torch.full(bt.q.shape, 7.0, dtype=bt.q.dtype, device=cuda_device)
    lse = torch.full(bt.q.shape[:2], 7.0, device=cuda_device)
    lay.attend_paged(bt.q, bt.cache, tok_start=bt.start, max_new=max(news), max_len=max(lens), out=out, lse=lse)
    lay.sync()
    check_attend(out, lse, bt, None)
    assert (out[sum(news):] == 7.0).all() and (lse[sum(news):] == 7.0).all()
    # twice the same, and the same to rounding without the hints
    again = lay.attend_paged(bt.q, bt.cache, tok_start=bt.start, max_new=max(news), max_len=max(lens))
    assert torch.equal(again[:sum(news)], out[:sum(news)])
    o2, l2 = lay.attend_paged(bt.q, bt.cache, tok_start=bt.start, return_lse=True)
    check_attend(o2, l2, bt, None)
    # another scale, a strided output
    wide = torch.zeros(bt.q.shape[0], hq + 3, d, dtype=bt.q.dtype, device=cuda_device)
    view = wide[:, 1:1 + hq]
    lay.attend_paged(bt.q, bt.cache, tok_start=bt.start, max_new=max(news), scale=0.3, out=view)
    lay.sync()
    check_attend(view, None, bt, None, scale=0.3)
    assert (wide[:, 0] == 0).all() and (wide[:, 1 + hq:] == 0).all()
    # an output that is aligned to 16 bytes and no more
    step = 16 // bt.q.element_size()
    odd = torch.zeros(bt.q.numel() + 2 * step, dtype=bt.q.dtype, device=cuda_device)
    view = odd[step:-step].view(bt.q.shape)
    assert view.data_ptr() % 32 == 16
    lay.attend_paged(bt.q, bt.cache, tok_start=bt.start, max_new=max(news), out=view)
    lay.sync()
    check_attend(view, None, bt, None)
    assert (odd[:step] == 0).all() and (odd[-step:] == 0).all()
    lay.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attend_large_logits_and_infinite_stale_rows(cuda_device, dtype):
    """Logits far apart (a running maximum that grows by hundreds along the
    keys), stale rows of infinities, and the caller's max_new too small."""
    for news, stale in (([1, 1], np.inf), ([150, 40], -np.inf)):
        lay = layer(cuda_device, dtype=dtype)
        bt = batch(cuda_device, news, [900, 333], dtype=dtype, stale=stale)
        Kf = bt.cache.K.view(-1, 2, 64)
        for s, n in enumerate(bt.lens):
            rows = torch.from_numpy(po.slots(bt.cache.block_table[s].tolist(), 16, n)).to(cuda_device)
            grow = torch.linspace(0.1, 8, n, device=cuda_device)[:, None, None]
            Kf[rows] = (Kf[rows].float() * grow).to(Kf.dtype)
        out, lse = lay.attend_paged(bt.q, bt.cache, tok_start=bt.start, max_new=max(news), return_lse=True)
        lay.sync()
        check_attend(out, lse, bt, None)
        if max(news) > 1:
            out2 = torch.full_like(out, 7.0)
            lay.attend_paged(bt.q, bt.cache, tok_start=bt.start, max_new=39, out=out2)
            with pytest.raises(B.IndexMemError) as ei:
                lay.sync()
            assert ei.value.name == "IMEM_ERR_RANGE"
        lay.close()


@pytest.mark.parametrize("dtype,new", [("bf16", 6), ("bf16", 60), ("fp32", 3), ("fp32", 60)])
def test_attend_reports_bad_pages(cuda_device, dtype, new):
    lay = layer(cuda_device, dtype=dtype)
    for value in (-1, -2, -(1 << 31), 1 << 30, None):
        bt = batch(cuda_device, [new, new], [200, 500], dtype=dtype)
        good = lay.attend_paged(bt.q, bt.cache, tok_start=bt.start, max_new=new)
        lay.sync()
        bt.cache.block_table[1, 30] = bt.cache.K.shape[0] if value is None else value
        out = lay.attend_paged(bt.q, bt.cache, tok_start=bt.start, max_new=new)
        with pytest.raises(B.IndexMemError) as ei:
            lay.sync()
        assert ei.value.name == "IMEM_ERR_RANGE"
        assert torch.equal(out[:new], good[:new])          # the other sequence
    lay.close()


@pytest.mark.parametrize("dtype,d,new", [("bf16", 128, 2), ("bf16", 64, 70), ("bf16", 128, 200), ("fp32", 64, 1),
                                         ("fp32", 128, 33)])
def test_attend_where_nothing_or_little_is_seen(cuda_device, dtype, d, new):
    """Sequences of length 0 (all new tokens are padding in front), of one key,
    and two that share their pages; max_len as a wrong hint."""
    lay = layer(cuda_device, 8, 2, d, dtype)
    bt = batch(cuda_device, [new] * 4, [0, 1, 300, 300], 8, 2, d, dtype)
    bt.cache.block_table[3] = bt.cache.block_table[2]
    for hint in (None, 0, 7, 1 << 20):
        out, lse = lay.attend_paged(bt.q, bt.cache, tok_start=bt.start, max_new=new, max_len=hint, return_lse=True)
        lay.sync()
        assert (out[:new] == 0).all() and (lse[:new] == -np.inf).all()
        check_attend(out, lse, bt, None)
    lay.close()


def test_chunk_attention_in_a_graph_follows_its_inputs(cuda_device):
    """A captured chunk call replayed with other queries, pages and lengths."""
    lay = layer(cuda_device, 8, 2, 128)
    bt = batch(cuda_device, [90, 50], [400, 700], 8, 2, 128)
    out, lse = torch.empty_like(bt.q), torch.empty(140, 8, device=cuda_device)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    call = lambda: lay.attend_paged(bt.q, bt.cache, tok_start=bt.start, max_new=90, out=out, lse=lse)
    with torch.cuda.stream(stream):
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            call()
        other = batch(cuda_device, [40, 80], [230, 701], 8, 2, 128, seed=9)
        small = torch.arange(other.cache.K.shape[0])
        assert other.cache.K.shape[0] <= bt.cache.K.shape[0]
        bt.cache.K[:len(small)], bt.cache.V[:len(small)] = other.cache.K, other.cache.V
        bt.cache.block_table[:, :other.cache.block_table.shape[1]] = other.cache.block_table
        bt.cache.kv_len.copy_(other.cache.kv_len), bt.start.copy_(other.start)
        bt.q[:120] = other.q
        graph.replay()
    stream.synchronize()
    lay.sync()
    check_attend(out[:120], lse[:120], other, None)
    lay.close()


def test_caches_past_32_bit_offsets(cuda_device):
    """Pages whose rows lie more than 2^32 bytes and 2^31 elements into the cache."""
    hq, hkv, d, page = 8, 8, 128, 64
    n_pages = (1 << 31) // (page * hkv * d) + 40
    for dtype, new in (("bf16", 1), ("bf16", 40), ("fp32", 5)):
        lay = layer(cuda_device, hq, hkv, d, dtype)
        dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        cache = lay.new_paged(2, n_pages, page, 4, cuda_device)
        table = torch.tensor([[n_pages - 1, 3, n_pages - 7, 0], [n_pages - 20, n_pages - 21, 1, 2]])
        cache.block_table.copy_(table.to(torch.int32))
        lens = [250, 130]
        for s in range(2):
            cache.K[table[s].to(cuda_device)] = torch.randn(4, page, hkv, d, device=cuda_device).to(dt)
            cache.V[table[s].to(cuda_device)] = torch.randn(4, page, hkv, d, device=cuda_device).to(dt)
        cache.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        q, k, v = (torch.randn(2 * new, h, d, device=cuda_device).to(dt) for h in (hq, hkv, hkv))
        qr = lay.append_paged(k, v, cache, q=q)
        out, lse = lay.attend_paged(qr, cache, return_lse=True)
        K, V = lay.gather_paged(cache, n=130)
        lay.sync()
        # the same cache, its pages moved to the front
        ids = table.flatten().tolist()
        small = PagedCache(torch.stack([cache.K[i] for i in ids]), torch.stack([cache.V[i] for i in ids]),
                           torch.arange(8, dtype=torch.int32, device=cuda_device).view(2, 4), cache.kv_len)
        bt = Batch(qr, None, None, torch.tensor([0, new, 2 * new], dtype=torch.int32), small, [new, new], lens, None)
        check_attend(out, lse, bt, None)
        for s in range(2):
            rows = po.slots(small.block_table[s].tolist(), page, lens[s])
            at = torch.from_numpy(rows).to(cuda_device)
            pos = np.arange(lens[s] - new, lens[s])
            check_rotated(small.K.view(-1, hkv, d)[at[-new:]], k[s * new:(s + 1) * new], pos, po.frequencies(d, 500000.0), "half")
            assert torch.equal(small.V.view(-1, hkv, d)[at[-new:]], v[s * new:(s + 1) * new])
            assert torch.equal(K[s], small.K.view(-1, hkv, d)[at[:130]]) and torch.equal(V[s], small.V.view(-1, hkv, d)[at[:130]])
        lay.close()
        del cache


def test_attend_non_finite_values_reach_only_who_may_see_them(cuda_device):
    for dtype in ("bf16", "fp32"):
        lay = layer(cuda_device, dtype=dtype)
        bt = batch(cuda_device, [1, 300], [500, 700], dtype=dtype)
        clean = lay.attend_paged(bt.q, bt.cache, tok_start=bt.start, max_new=300)
        # position 600 of sequence 1 (its token 200): NaN key and value
        row = po.slots(bt.cache.block_table[1].tolist(), 16, 700)[600]
        bt.cache.K.view(-1, 2, 64)[row] = float("nan")
        bt.cache.V.view(-1, 2, 64)[row] = float("nan")
        out = lay.attend_paged(bt.q, bt.cache, tok_start=bt.start, max_new=300)
        lay.sync()
        assert torch.equal(out[0], clean[0])                       # another sequence
        assert out[1 + 200:].isnan().all()                         # they see it
        assert torch.equal(out[1:1 + 200 - 127], clean[1:1 + 200 - 127])
        lay.close()


# ---------------------------------------------------------------------- gather

@pytest.mark.parametrize("dtype,hkv,d,page", [("bf16", 8, 128, 64), ("bf16", 1, 64, 16), ("fp32", 2, 64, 32),
                                              ("bf16", 3, 64, 1024)])
def test_gather(cuda_device, dtype, hkv, d, page):
    lay = layer(cuda_device, hkv * 2, hkv, d, dtype)
    lens = [900, 257, 300]
    bt = batch(cuda_device, [1, 1, 1], lens, hkv * 2, hkv, d, dtype, page)
    idx = torch.stack([torch.randperm(n)[:200].sort().values for n in lens]).to(torch.int32)
    idx[0, :3] = torch.tensor([899, 0, 0])                        # any order, repeats
    rows = [po.slots(bt.cache.block_table[s].tolist(), page, n) for s, n in enumerate(lens)]
    K, V = lay.gather_paged(bt.cache, idx.to(cuda_device))
    out = torch.full((3, 205, hkv, d), 7.0, dtype=K.dtype, device=cuda_device)
    out2 = out.clone()
    lay.gather_paged(bt.cache, idx.to(cuda_device), K=out, V=out2)
    lay.sync()
    for s in range(3):
        at = torch.from_numpy(rows[s][idx[s].numpy()]).to(cuda_device)
        assert torch.equal(K[s], bt.cache.K.view(-1, hkv, d)[at])
        assert torch.equal(V[s], bt.cache.V.view(-1, hkv, d)[at])
    assert torch.equal(out[:, :200], K) and torch.equal(out2[:, :200], V)
    assert (out[:, 200:] == 7).all() and (out2[:, 200:] == 7).all()
    # the first n positions; those past a sequence's length are skipped
    out.fill_(7.0), out2.fill_(7.0)
    n = 205
    lay.gather_paged(bt.cache, n=n, K=out, V=out2)
    bt.cache.kv_len[1] = 100
    out3, out4 = torch.full_like(out, 7.0), torch.full_like(out, 7.0)
    lay.gather_paged(bt.cache, n=n, K=out3, V=out4)
    lay.sync()
    for s in range(3):
        at = torch.from_numpy(rows[s][:n]).to(cuda_device)
        assert torch.equal(out[s], bt.cache.K.view(-1, hkv, d)[at])
    assert torch.equal(out3[1, :100], out[1, :100]) and (out3[1, 100:] == 7).all() and (out4[1, 100:] == 7).all()
    # an index outside [0, kv_len): reported, its row not written
    bad = idx.clone()
    bad[2, 5], bad[0, 1] = 300, -1
    out.fill_(7.0)
    lay.gather_paged(bt.cache, bad.to(cuda_device), K=out, V=out2)
    with pytest.raises(B.IndexMemError) as ei:
        lay.sync()
    assert ei.value.name == "IMEM_ERR_RANGE"
    assert (out[2, 5] == 7).all() and (out[0, 1] == 7).all() and torch.equal(out[2, 6:200], K[2, 6:])
    lay.close()


# --------------------------------------------------------------------- together

def test_no_tokens_is_no_work(cuda_device):
    lay = layer(cuda_device)
    bt = batch(cuda_device, [0, 0], [5, 9])
    start = torch.zeros(3, dtype=torch.int32, device=cuda_device)
    q, k = lay.rotate(bt.q, bt.k, torch.empty(0, dtype=torch.int32, device=cuda_device))
    assert q.shape[0] == 0 and k.shape[0] == 0
    lay.append_paged(bt.k, bt.v, bt.cache, tok_start=start, q=bt.q)
    assert lay.attend_paged(bt.q, bt.cache, tok_start=start).shape[0] == 0
    lay.sync()
    lay.close()


def test_layer_refuses_tensors_that_do_not_fit(cuda_device):
    lay = layer(cuda_device)
    bt = batch(cuda_device, [4, 4], [20, 40])
    pos = torch.zeros(8, dtype=torch.int32, device=cuda_device)
    c = bt.cache
    for fn in (lambda: lay.rotate(bt.q.float(), None, pos),
               lambda: lay.rotate(None, None, pos),
               lambda: lay.rotate(bt.q, bt.k[:4], pos),
               lambda: lay.rotate(bt.q, None, pos.long()),
               lambda: lay.rotate(bt.q.cpu(), None, pos),
               lambda: lay.rotate(bt.q.transpose(1, 2).contiguous().transpose(1, 2), None, pos),
               lambda: lay.rotate(bt.q[:1].expand(8, -1, -1), None, pos),
               lambda: lay.attend_paged(bt.q, c, scale=0.0),
               lambda: lay.attend_paged(bt.q, c, scale=float("nan")),
               lambda: lay.attend_paged(bt.q, c, out=bt.q[:1].expand(8, -1, -1)),
               lambda: lay.append_paged(bt.k, bt.v[:, :1], c),
               lambda: lay.append_paged(bt.k, bt.v, c, tok_start=pos),
               lambda: lay.attend_paged(bt.q, c, tok_start=bt.start.cpu()),
               lambda: lay.attend_paged(bt.q, c, lse=pos),
               lambda: lay.attend_paged(bt.q, PagedCache(c.K.transpose(1, 2), c.V, c.block_table, c.kv_len)),
               lambda: lay.attend_paged(bt.q, PagedCache(c.K, c.V, c.block_table, c.kv_len[:1])),
               lambda: lay.gather_paged(c),
               lambda: lay.gather_paged(c, pos.view(2, 4).long()),
               lambda: lay.gather_paged(c, pos.view(2, 4), K=c.K, V=c.V),
               lambda: lay.set_rope(layout="other")):
        with pytest.raises(ValueError):
            fn()
    lay.set_rope(rot_dim=0)
    with pytest.raises(B.IndexMemError):
        lay.rotate(bt.q, None, pos)
    lay.sync()
    lay.close()


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("fp32", 64), ("bf16", 128)])
def test_chunks_through_the_pages_match_one_prompt(cuda_device, dtype, d):
    """A prompt in ragged chunks (append, attend), the last tokens one by one in
    a captured graph, on a stream of its own, against one prompt at once; two
    contexts at work at the same time."""
    lens, page, hq, hkv = [210, 97], 32, 8, 2
    lay, other = layer(cuda_device, hq, hkv, d, dtype), layer(cuda_device, hq, hkv, d, dtype)
    bt = batch(cuda_device, lens, lens, hq, hkv, d, dtype, page)
    fresh = lambda: PagedCache(torch.full_like(bt.cache.K, float("nan")), torch.full_like(bt.cache.V, float("nan")),
                               bt.cache.block_table, torch.zeros(2, dtype=torch.int32, device=cuda_device))
    whole, parts, busy = fresh(), fresh(), fresh()
    whole.kv_len.copy_(bt.cache.kv_len)
    q1 = lay.append_paged(bt.k, bt.v, whole, tok_start=bt.start, q=bt.q)
    o1, l1 = lay.attend_paged(q1, whole, tok_start=bt.start, max_new=210, return_lse=True)
    lay.sync()
    s0 = bt.start.tolist()
    stream, stream2 = torch.cuda.Stream(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    stream2.wait_stream(torch.cuda.current_stream())
    got, got_l = torch.zeros_like(o1), torch.zeros_like(l1)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)

    def pick(done, news):
        return torch.cat([torch.arange(s0[s] + done[s], s0[s] + done[s] + news[s]) for s in range(2)]).to(cuda_device)

    with torch.cuda.stream(stream):
        done = [0, 0]
        for news in ([130, 1], [3, 60], [64, 33]):
            at = pick(done, news)
            done = [a + n for a, n in zip(done, news)]
            parts.kv_len.copy_(ints(done))
            start = ints([0, news[0], sum(news)])
            qr = lay.append_paged(bt.k[at], bt.v[at], parts, tok_start=start, q=bt.q[at])
            o, l = lay.attend_paged(qr, parts, tok_start=start, max_new=max(news), max_len=max(done), return_lse=True)
            got[at], got_l[at] = o, l
            with torch.cuda.stream(stream2):          # another context at the same time
                busy.kv_len.copy_(ints(lens))
                other.attend_paged(other.append_paged(bt.k, bt.v, busy, tok_start=bt.start, q=bt.q), busy,
                                   tok_start=bt.start, max_new=210, out=(ob := torch.empty_like(o1)))
    assert done == [197, 94]
    # single tokens of both sequences, the step captured once and replayed
    k, v, q = (torch.empty(2, x.shape[1], d, dtype=x.dtype, device=cuda_device) for x in (bt.k, bt.v, bt.q))
    out, lse = torch.empty_like(q), torch.empty(2, hq, device=cuda_device)
    with torch.cuda.stream(stream):
        def step():
            parts.kv_len.add_(1)
            qr = lay.append_paged(k, v, parts, q=q, q_out=q)
            lay.attend_paged(qr, parts, max_len=256, out=out, lse=lse)

        keep = parts.kv_len.clone()
        k.zero_(), v.zero_(), q.zero_()
        step()                                        # set-up before the capture
        parts.kv_len.copy_(keep)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
        for i in range(3):
            at = pick(done, [1, 1])
            done = [a + 1 for a in done]
            k.copy_(bt.k[at]), v.copy_(bt.v[at]), q.copy_(bt.q[at])
            graph.replay()
            got[at], got_l[at] = out, lse
    stream.synchronize()
    stream2.synchronize()
    lay.sync()
    other.sync()
    assert torch.equal(ob, o1)
    rows = torch.cat([torch.arange(s0[s], s0[s] + done[s]) for s in range(2)]).to(cuda_device)
    live = torch.cat([torch.from_numpy(po.slots(bt.cache.block_table[s].tolist(), page, done[s])) for s in range(2)])
    flat = lambda x: x.view(-1, hkv, d)[live.to(cuda_device)]
    assert torch.equal(flat(parts.K), flat(whole.K)) and torch.equal(flat(parts.V), flat(whole.V))
    # both sides are within their tolerance of the same oracle
    Batch_ = dataclasses.replace(bt, cache=whole)
    check_attend(o1, l1, Batch_, None, q=q1)
    merged, merged_l = o1.clone(), l1.clone()
    merged[rows], merged_l[rows] = got[rows], got_l[rows]
    check_attend(merged, merged_l, Batch_, None, q=q1)
    for l_ in (lay, other):
        l_.close()


def test_readme_paged_example_runs(cuda_device):
    """The README's second example, after its first (whose layer stays open)."""
    import pathlib
    import re
    text = (pathlib.Path(__file__).resolve().parent.parent / "README.md").read_text()
    first, second = re.findall(r"```python\n(.*?)```", text, re.S)[:2]
    ns: dict = {}
    exec(compile(first.replace("layer.close()", ""), "README.md", "exec"), ns)
    exec(compile(second, "README.md", "exec"), ns)
    assert ns["o"].shape == ns["dec"]["q"][0].shape and torch.isfinite(ns["o"].float()).all()
    ns["pages"].kv_len.fill_(4000)          # shorter than the prompt: reported
    ns["layer"].evict_paged(ns["x"]["X"], ns["q_rot"], ns["pages"], ns["st"], ns["B"])
    with pytest.raises(B.IndexMemError) as ei:
        ns["layer"].sync()
    assert ei.value.name == "IMEM_ERR_RANGE"
    ns["layer"].close()


def test_paged_prompt_to_eviction_and_decode(cuda_device):
    """rotate + append + attend over pages, then the learned eviction out of the
    pages, the memory and decode steps, each stage against the oracle."""
    wl = synth.WORKLOADS["c0"]
    s = wl.shape
    L, Bg, steps, page = 320, 48, 3, 16
    w = synth.make_weights(s, 5, cuda_device)
    x = synth.make_layer_inputs(wl, w, 5, cuda_device, L=L, batch=2)
    dec = synth.make_decode_inputs(wl, w, steps, 5, cuda_device, batch=2)
    lay = IndexMemLayer.from_shape(s, w)
    lay.set_rope(layout="half")
    pages = lay.new_paged(2, 2 * L // page, page, L // page, cuda_device)
    pages.block_table.copy_(torch.randperm(2 * L // page).view(2, -1))
    flat = lambda t: t.flatten(0, 1)
    outs = []
    q = torch.empty_like(flat(x["Q"]))
    for lo, hi in ((0, 200), (200, 320)):
        pages.kv_len.fill_(hi)
        qr = lay.append_paged(flat(x["K"][:, lo:hi]), flat(x["V"][:, lo:hi]), pages, q=flat(x["Q"][:, lo:hi]))
        q.view(2, L, 8, 64)[:, lo:hi] = qr.view(2, hi - lo, 8, 64)
        outs.append(lay.attend_paged(qr, pages, max_len=L).view(2, hi - lo, 8, 64))
    out = torch.cat(outs, 1)
    st = lay.new_state(2, L, Bg, Bg + steps, cuda_device)
    lay.evict_paged(x["X"], q.view(2, L, 8, 64), pages, st, Bg, chunk=64)
    os_ = [lay.decode(dec["q"][i], dec["k_new"][i], dec["v_new"][i], st) for i in range(steps)]
    lay.sync()
    th = po.frequencies(64)
    pos = np.tile(np.arange(L), 2)
    check_rotated(q, flat(x["Q"]), pos, th, "half")
    K = torch.stack([pages.K.view(-1, 2, 64)[torch.from_numpy(po.slots(pages.block_table[b].tolist(), page, L)).to(cuda_device)]
                     for b in range(2)])
    check_rotated(flat(K), flat(x["K"]), pos, th, "half")
    bt = Batch(q, None, None, torch.tensor([0, L, 2 * L], dtype=torch.int32), pages, [L, L], [L, L], None)
    check_attend(out.flatten(0, 1), None, bt, None)
    # the decisions and states that follow are the oracle's on the GPU's inputs
    R, E = om.select_budget(to_np(st.running_max), Bg)
    assert np.array_equal(st.idx_retained.cpu().numpy(), R)
    for b in range(2):
        assert torch.equal(st.K_ret[b, :Bg], K[b, torch.from_numpy(np.asarray(R[b])).long().to(cuda_device)])
    M_ref, b_ref = om.memory_update(to_np(K), to_np(x["V"]), E, to_np(w["W_phi"]), s.lam)
    check_memory(to_np(st.M), to_np(st.bstab), M_ref, b_ref, "paged")
    KR, VR = om.compact(to_np(K), to_np(x["V"]), R, Bg + steps)
    clen = np.full(2, Bg)
    for i in range(steps):
        qi, ki, vi = (to_np(dec[n][i]) for n in ("q", "k_new", "v_new"))
        o_ref, c2, _, _, _ = om.decode_step(qi, ki, vi, KR, VR, clen, to_np(st.M), to_np(st.bstab),
                                            to_np(w["W_phi"]), to_np(w["w_gate"]))
        check_decode(to_np(os_[i]), o_ref, ill_conditioned(to_np(st.bstab), qi, to_np(w["W_phi"]), 4), "paged")
        for b in range(2):
            KR[b, clen[b]], VR[b, clen[b]] = ki[b], vi[b]
        clen = c2
    lay.close()
