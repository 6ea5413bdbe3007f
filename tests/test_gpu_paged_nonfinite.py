"""NaN and infinities among the cached keys and values, through the layer's
attend_paged, against the definition in 64 bits.

By the formulas, with IEEE arithmetic for the scores s_j of the keys that a row
sees: a score of -inf has weight 0; a NaN score makes the row's out and lse
NaN; a score of +inf makes its out NaN and its lse +inf; a row all of whose
scores are -inf is as one that sees nothing (out 0, lse -inf). Rows
that see none of them keep their values within the tolerances of
test_gpu_paged.py, which is where those are derived.
"""
import numpy as np
import pytest
import torch

from oracle import paged_oracle as po

from .parity import to_np
from .test_gpu_paged import U, batch, layer

pytestmark = pytest.mark.gpu


def definition(bt):
    """out, lse, and sum_j p_j |v_j| and the largest scale sum_d |q_d k_jd| of each
    row (over the finite entries), as po.attend, for any values."""
    q, K, V = to_np(bt.q), to_np(bt.cache.K), to_np(bt.cache.V)
    T, hq, d = q.shape
    page, hkv = K.shape[1:3]
    G, scale = hq // hkv, d ** -0.5
    table, start = bt.cache.block_table.cpu().numpy(), bt.start.cpu().numpy()
    out, lse = np.zeros((T, hq, d)), np.zeros((T, hq))
    spread, size = np.zeros((T, hq, d)), np.zeros((T, hq))
    finite = lambda x: np.where(np.isfinite(x), x, 0.0)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        for s, n in enumerate(bt.lens):
            rows, at = po.slots(table[s], page, n), slice(start[s], start[s + 1])
            k, v = K.reshape(-1, hkv, d)[rows], V.reshape(-1, hkv, d)[rows]
            new = start[s + 1] - start[s]
            seen = np.arange(n)[None] <= (n - new + np.arange(new))[:, None]       # [token, key]
            for h in range(hq):
                kk, vv, qq = k[:, h // G], v[:, h // G], q[at, h]
                x = scale * (qq[:, None] * kk).sum(2)
                x[~seen] = -np.inf
                size[at, h] = scale * np.where(seen, np.abs(qq) @ np.abs(finite(kk)).T, 0).max(1)
                nan, inf, none = np.isnan(x).any(1), (x == np.inf).any(1), (x == -np.inf).all(1)
                m = np.where(nan | inf | none, 0.0, x.max(1))
                p = np.exp(x - m[:, None])
                total = p.sum(1)
                lse[at, h] = m + np.log(total)
                p = np.where((nan | inf | none)[:, None], 0.0, p / total[:, None])
                # a value counts where its weight is not 0
                o = p @ finite(vv)
                for j, e in zip(*np.nonzero(~np.isfinite(vv))):
                    o[:, e] += np.where(p[:, j] > 0, vv[j, e], 0.0)
                o[nan | inf] = np.nan
                out[at, h], spread[at, h] = o, p @ np.abs(finite(vv))
                lse[at, h] = np.where(nan, np.nan, np.where(inf, np.inf, np.where(none, -np.inf, lse[at, h])))
    return out, lse, spread, size


def check(out, lse, bt, defined):
    ref, rl, spread, size = defined
    o, l = to_np(out), to_np(lse)
    d, n, e = o.shape[2], max(bt.lens), torch.finfo(out.dtype).eps / 2
    ds = 4 * U * (d + 4) * size
    rel = 2 * ds + 16 * U + 4 * U * (n + 4) + (e if out.dtype == torch.bfloat16 else 0.0)
    assert np.array_equal(np.isnan(o), np.isnan(ref)), "NaN in %d outputs, by definition %d" % (
        np.isnan(o).sum(), np.isnan(ref).sum())
    inf = np.isinf(ref)
    assert np.array_equal(o[inf], ref[inf]) and np.isfinite(o[~inf & ~np.isnan(ref)]).all()
    on = np.isfinite(ref)
    tol = rel[..., None] * spread + e * np.abs(ref)
    assert (np.abs(o[on] - ref[on]) <= tol[on]).all()
    on = np.isfinite(rl)
    assert np.array_equal(np.isnan(l), np.isnan(rl)) and np.array_equal(l[np.isinf(rl)], rl[np.isinf(rl)])
    tl = ds + 4 * U * (n + 4) + 16 * U + 4 * U * np.abs(rl)
    assert (np.abs(l[on] - rl[on]) <= tl[on]).all()


@pytest.mark.parametrize("kind", ["nan", "one", "inf", "all", "value"])
@pytest.mark.parametrize("dtype,d,new", [
    ("bf16", 64, 70), ("bf16", 64, 40), ("bf16", 128, 70), ("bf16", 128, 40),     # chunks: two tiles of rows, one
    ("bf16", 64, 1), ("bf16", 128, 3), ("bf16", 128, 6),                          # steps: one to three column tiles
    ("fp32", 64, 40), ("fp32", 128, 40), ("fp32", 64, 8), ("fp32", 128, 2),       # one, two, four warps to 16 rows
])
def test_non_finite_keys_and_values(cuda_device, dtype, d, new, kind):
    """Sixteen sequences, each with one such key (or value) at another of 16
    neighbouring positions, long before the new tokens, so that no place of its
    tile is masked; one KV head of two."""
    lay = layer(cuda_device, 8, 2, d, dtype)
    lens = [640 + 3 * s for s in range(16)]
    bt = batch(cuda_device, [new] * 16, lens, 8, 2, d, dtype, seed=d + new)
    Kf, Vf = bt.cache.K.view(-1, 2, d), bt.cache.V.view(-1, 2, d)
    for s in range(16):
        rows = po.slots(bt.cache.block_table[s].tolist(), 16, lens[s])
        at = int(rows[256 + s])
        if kind == "nan":
            Kf[at, 0] = float("nan")
        elif kind == "one":
            Kf[at, 0, d - 3] = float("nan")
        elif kind == "inf":          # +inf or -inf by the sign of q's first element
            Kf[at, 0, 0] = float("inf")
        elif kind == "all":
            Kf[torch.from_numpy(rows).to(cuda_device), 0, 0] = float("-inf")
        else:
            Vf[at, 0, 5], Vf[at, 0, 6], Vf[at, 0, 7] = float("inf"), float("-inf"), float("nan")
    defined = definition(bt)
    for hint in (None, 0):           # keys split over CTAs, and not
        out, lse = lay.attend_paged(bt.q, bt.cache, tok_start=bt.start, max_new=new, max_len=hint, return_lse=True)
        lay.sync()
        check(out, lse, bt, defined)
    lay.close()


@pytest.mark.parametrize("d,new", [(64, 40), (128, 8), (64, 3)])
def test_fp32_values_of_later_tokens_stay_out(cuda_device, d, new):
    """fp32: a new token's key and value that are not finite reach that token and
    those after it, and none before."""
    lay = layer(cuda_device, 8, 2, d, "fp32")
    bt = batch(cuda_device, [new, new], [300, 77], 8, 2, d, "fp32")
    for s in range(2):
        at = int(po.slots(bt.cache.block_table[s].tolist(), 16, bt.lens[s])[-1 - new // 2])
        bt.cache.K.view(-1, 2, d)[at, s] = float("inf")
        bt.cache.V.view(-1, 2, d)[at, s] = float("nan")
    out, lse = lay.attend_paged(bt.q, bt.cache, tok_start=bt.start, max_new=new, return_lse=True)
    lay.sync()
    check(out, lse, bt, definition(bt))
    lay.close()
