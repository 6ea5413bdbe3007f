"""fp32 attention over the pages, how close it is: root mean squares, which the
worst-case bounds of test_gpu_paged.py (sums over all keys and dimensions of
the largest error of each) leave far too much room for.

Tolerance. Queries, keys and values are normal, so a logit is of size 1 and its
relative errors are those of the probabilities. Of a product of two values the
split into tf32 halves drops at most 2^-21 (lo lo: 2^-22; the bits of a lo
behind its eleventh: 2^-23 on either side), with either sign. Inside the unit a
sum is cut off at 2^-23 of itself at most, 2^-24 on average, per step: 2 steps
for 16 dimensions, up to 12 for a stage of 32 keys. exp2 is off by 2^-22, its
argument and the sums of stages by 2^-24 each. In quadrature, relative to the
outputs' own size: (2^-21)^2 + (2 * 2^-24)^2 + (12 * 2^-24)^2 + (2^-22)^2 +
(2^-23)^2 < (2^-20)^2. One tf32 product in place of three, or a lo left out, is
off by some 3e-4 = 2^-11.7. The logarithm of the sum averages the same errors.
"""
import numpy as np
import pytest
import torch

from oracle import paged_oracle as po

from .parity import to_np
from .test_gpu_paged import batch, layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("length", [100, 300, 1000])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [2, 8, 20])       # four, two warps and one to 16 rows
def test_fp32_attention_is_near_fp32(cuda_device, d, new, length):
    lay = layer(cuda_device, 8, 2, d, "fp32")
    bt = batch(cuda_device, [new, new], [length, length - 37], 8, 2, d, "fp32", seed=d + length)
    g = torch.Generator(device=cuda_device).manual_seed(new)
    rows = bt.cache.K.view(-1, 2, d)
    rows[bt.live] = torch.randn(int(bt.live.sum()), 2, d, generator=g, device=cuda_device)
    for hint in (None, 0):
        out, lse = lay.attend_paged(bt.q, bt.cache, tok_start=bt.start, max_new=new, max_len=hint, return_lse=True)
        lay.sync()
        ref, rl, _, _ = po.attend(to_np(bt.q), to_np(bt.cache.K), to_np(bt.cache.V), bt.cache.block_table.cpu().numpy(),
                                  bt.lens, bt.start.cpu().numpy(), 16)
        rms = lambda x: np.sqrt(np.mean(np.square(x)))
        assert rms(to_np(out) - ref) <= 2.0 ** -20 * rms(ref), rms(to_np(out) - ref) / rms(ref)
        assert rms(to_np(lse) - rl) <= 2.0 ** -20 * rms(rl), rms(to_np(lse) - rl) / rms(rl)
    lay.close()
