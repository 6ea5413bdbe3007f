"""The paged calls on a stream that is not torch's current one: what they make
for themselves is ordered with the call's stream, whatever the current stream
does before or after."""
import numpy as np
import pytest
import torch

from learned_kv_cache_indexmem_b200 import synth
from learned_kv_cache_indexmem_b200.layer import IndexMemLayer

pytestmark = pytest.mark.gpu
LONG = 100_000_000     # cycles of a kernel that only waits: some 50 ms


def _prompt(dev, L=320, page=16):
    """A layer, a prompt of two sequences in pages, its hidden states and queries."""
    wl = synth.WORKLOADS["c0"]
    w = synth.make_weights(wl.shape, 5, dev)
    x = synth.make_layer_inputs(wl, w, 5, dev, L=L, batch=2)
    lay = IndexMemLayer.from_shape(wl.shape, w)
    lay.set_rope()
    pages = lay.new_paged(2, 2 * L // page, page, L // page, dev)
    pages.block_table.copy_(torch.from_numpy(np.random.default_rng(0).permutation(2 * L // page)).view(2, -1))
    pages.kv_len.fill_(L)
    lay.append_paged(x["K"].flatten(0, 1), x["V"].flatten(0, 1), pages)
    lay.sync()
    return lay, pages, x


def _states(st):
    return [t.clone() for t in (st.running_max, st.idx_retained, st.idx_evicted, st.K_ret, st.V_ret, st.M, st.bstab)]


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("busy", ["current", "own"])
def test_evict_paged_on_another_stream(cuda_device, busy, handle):
    """busy = current: work queued on the current stream before the call must not
    delay what the call reads; busy = own: memory that the current stream takes
    and writes after the call must not be the call's."""
    L, Bg = 320, 48
    lay, pages, x = _prompt(cuda_device, L)
    st = lay.new_state(2, L, Bg, Bg, cuda_device)
    lay.evict_paged(x["X"], x["Q"], pages, st, Bg, chunk=64)
    lay.sync()
    want = _states(st)
    lay.close()
    lay, pages, x = _prompt(cuda_device, L)
    st = lay.new_state(2, L, Bg, Bg, cuda_device)
    side = torch.cuda.Stream()
    for _ in range(2):       # with a new workspace, then with the layer's own
        st.M.zero_(), st.bstab.zero_()
        side.wait_stream(torch.cuda.current_stream())
        if busy == "current":
            # blocks of every size the call needs, freed with writes still to come
            junk = [torch.empty(1 << k, dtype=torch.uint8, device=cuda_device) for k in range(9, 23)]
            torch.cuda._sleep(LONG)
            for t in junk:
                t.fill_(0x7f)
            del junk, t
        else:
            with torch.cuda.stream(side):
                torch.cuda._sleep(LONG)
        lay.evict_paged(x["X"], x["Q"], pages, st, Bg, chunk=64, stream=side.cuda_stream if handle else side)
        junk = [torch.full((1 << k,), 0x7f, dtype=torch.uint8, device=cuda_device) for k in range(9, 23) for _ in range(4)]
        torch.cuda.current_stream().synchronize()
        lay.sync(side)
        for got, ref in zip(_states(st), want):
            assert torch.equal(got, ref)
        del junk
    lay.close()


def test_evict_paged_on_the_default_stream_from_another(cuda_device):
    """Handle 0 is the default stream."""
    L, Bg = 320, 48
    lay, pages, x = _prompt(cuda_device, L)
    st = lay.new_state(2, L, Bg, Bg, cuda_device)
    lay.evict_paged(x["X"], x["Q"], pages, st, Bg, chunk=64)
    lay.sync()
    want = _states(st)
    st.M.zero_(), st.bstab.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        torch.cuda._sleep(LONG)
        assert lay._as_current(0).stream == torch.cuda.default_stream()
        lay.evict_paged(x["X"], x["Q"], pages, st, Bg, chunk=64, stream=0)
    lay.sync(0)
    torch.cuda.synchronize()
    for got, ref in zip(_states(st), want):
        assert torch.equal(got, ref)
    lay.close()


def test_outputs_belong_to_the_stream_of_the_call(cuda_device):
    """rotate, append, attend and gather on another stream, their outputs left to
    them: blocks that the current stream has freed, but has yet to write, are not
    taken for them; what the current stream takes afterwards is not theirs."""
    lay, pages, x = _prompt(cuda_device)
    q, k, v = (x[n].flatten(0, 1) for n in ("Q", "K", "V"))
    pos = torch.arange(q.shape[0], dtype=torch.int32, device=cuda_device)

    def calls(**kw):
        return (lay.rotate(q, k, pos, **kw) + (lay.append_paged(k, v, pages, q=q, **kw),)
                + lay.attend_paged(q, pages, return_lse=True, **kw) + lay.gather_paged(pages, n=300, **kw))

    want = [t.clone() for t in calls()]
    sizes = sorted({t.nbytes for t in want})
    for handle in (False, True):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        junk = [torch.empty(n, dtype=torch.uint8, device=cuda_device) for n in sizes for _ in range(len(want))]
        torch.cuda._sleep(LONG)
        for t in junk:
            t.fill_(0x7f)
        del junk, t
        got = calls(stream=side.cuda_stream if handle else side)
        torch.cuda.current_stream().synchronize()
        lay.sync(side)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        # dropped while the current stream still reads them: not given out again on theirs
        side.wait_stream(torch.cuda.current_stream())
        torch.cuda._sleep(LONG)
        copies = [t.clone() for t in got]
        del got, a
        over = calls(stream=side)
        for t in over:
            with torch.cuda.stream(side):
                t.fill_(1)
        torch.cuda.synchronize()
        for a, b in zip(copies, want):
            assert torch.equal(a, b)
        del over, copies
    lay.close()


def test_evict_paged_in_a_graph(cuda_device):
    """Captured after a first call, replayed after other keys went into the pages."""
    L, Bg = 320, 48
    lay, pages, x = _prompt(cuda_device, L)
    st = lay.new_state(2, L, Bg, Bg, cuda_device)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        lay.evict_paged(x["X"], x["Q"], pages, st, Bg, chunk=64)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            lay.evict_paged(x["X"], x["Q"], pages, st, Bg, chunk=64)
        lay.append_paged(x["V"].flatten(0, 1), x["K"].flatten(0, 1), pages)
        x["X"].mul_(-0.5)
        st.M.zero_(), st.bstab.zero_()
        graph.replay()
        got = _states(st)
        st.M.zero_(), st.bstab.zero_()
        lay.evict_paged(x["X"], x["Q"], pages, st, Bg, chunk=64)
    stream.synchronize()
    lay.sync()
    for a, b in zip(got, _states(st)):
        assert torch.equal(a, b)
    del graph
    lay.close()
