"""What the paged calls report, through the layer: lengths and token ranges that
do not fit, a max_new that is too small, hints of any size."""
import pytest
import torch

from learned_kv_cache_indexmem_b200 import binding as B

from .test_gpu_paged import batch, check_attend, layer

pytestmark = pytest.mark.gpu


def reported(lay):
    """The error that sync raises (none: None); the context is clean afterwards."""
    try:
        lay.sync()
    except B.IndexMemError as e:
        lay.sync()
        return e.name
    return None


@pytest.mark.parametrize("idx", [True, False])
@pytest.mark.parametrize("bad", [-1, -(1 << 31), "room", (1 << 30) + 1, (1 << 31) - 1])
def test_gather_reports_lengths(cuda_device, idx, bad):
    """A length below 0 or above what the table can hold is reported even where
    every position asked for is inside; the other sequence's rows are copied."""
    lay = layer(cuda_device)
    bt = batch(cuda_device, [1, 1], [200, 120])
    good, _ = lay.gather_paged(bt.cache, n=50)
    assert reported(lay) is None
    bt.cache.kv_len[0] = 16 * bt.cache.block_table.shape[1] + 1 if bad == "room" else bad
    at = torch.arange(50, dtype=torch.int32, device=cuda_device).expand(2, 50).contiguous()
    K, _ = lay.gather_paged(bt.cache, at if idx else None, n=50)
    assert reported(lay) == "IMEM_ERR_RANGE"
    assert torch.equal(K[1], good[1])
    lay.close()


@pytest.mark.parametrize("start", [[0, 0, -1], [9, 9, 9], [0, 5, 3], [-1, 4, 8], [0, 4, 9], [5, 5, 0], [0, -5, 8]])
def test_append_reports_token_ranges(cuda_device, start):
    """Ranges that descend or leave [0, n_tokens], whether or not one of the
    call's tokens falls into them."""
    lay = layer(cuda_device)
    bt = batch(cuda_device, [4, 4], [20, 40])
    lay.append_paged(bt.k, bt.v, bt.cache, tok_start=bt.start)
    assert reported(lay) is None
    bad = torch.tensor(start, dtype=torch.int32, device=cuda_device)
    lay.append_paged(bt.k, bt.v, bt.cache, tok_start=bad)
    assert reported(lay) == "IMEM_ERR_RANGE"
    lay.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attend_with_max_new_zero(cuda_device, dtype):
    """max_new = 0 is right for a batch of padding alone; a sequence that has new
    tokens is reported."""
    lay = layer(cuda_device, dtype=dtype)
    bt = batch(cuda_device, [0, 0], [20, 40], dtype=dtype, pad=4)
    out, lse = torch.full_like(bt.q, 7.0), torch.full((4, 8), 7.0, device=cuda_device)
    lay.attend_paged(bt.q, bt.cache, tok_start=bt.start, max_new=0, out=out, lse=lse)
    assert reported(lay) is None
    assert (out == 7.0).all() and (lse == 7.0).all()
    bt = batch(cuda_device, [3, 1], [20, 40], dtype=dtype)
    lay.attend_paged(bt.q, bt.cache, tok_start=bt.start, max_new=0, out=out, lse=lse)
    assert reported(lay) == "IMEM_ERR_RANGE"
    assert (out == 7.0).all() and (lse == 7.0).all()
    lay.close()


@pytest.mark.parametrize("dtype,new", [("bf16", 1), ("bf16", 40), ("fp32", 1)])
def test_attend_hints_above_the_longest_length(cuda_device, dtype, new):
    """Hints past the longest length a sequence may have (2^30) split the work as
    that length does: the same sums in the same order."""
    lay = layer(cuda_device, dtype=dtype)
    bt = batch(cuda_device, [new], [3000], dtype=dtype)
    call = lambda hint: lay.attend_paged(bt.q, bt.cache, max_len=hint, return_lse=True)
    out, lse = call(1 << 30)
    for hint in ((1 << 30) + 1, (1 << 31) - 64, (1 << 31) - 1):
        o, l = call(hint)
        assert torch.equal(o, out) and torch.equal(l, lse)
    assert reported(lay) is None
    check_attend(out, lse, bt, None)
    lay.close()
