"""One IndexMem layer on the GPU: owns the library context and the caller-side
buffers (allocated with torch), and calls the C ABI through ``binding``.

Plumbing only -- every step of the path runs in libindexmem.so's kernels.
"""
from __future__ import annotations

import contextlib
import dataclasses
from typing import Optional

import torch

from . import binding as B_


@dataclasses.dataclass
class PrefillState:
    running_max: torch.Tensor     # [b, L] fp32
    idx_retained: torch.Tensor    # [b, B] int32
    idx_evicted: torch.Tensor     # [b, L-B] int32
    K_ret: torch.Tensor           # [b, cap, Hkv, d]
    V_ret: torch.Tensor
    cache_len: torch.Tensor       # [b] int32
    M: torch.Tensor               # [b, Hkv, r, d] fp32 (moment readout: S^T, r = d)
    bstab: torch.Tensor           # [b, Hkv, r] fp32 (moment readout: s_k)
    s_v: Optional[torch.Tensor] = None   # [b, Hkv, d] fp32, moment readout only
    n_e: Optional[torch.Tensor] = None   # [b] fp32, moment readout only


@dataclasses.dataclass
class OnlineState:
    """Decode-time online eviction: per cache slot the indexer key, the
    importance and the position; the next token's position; the position
    evicted by the last step."""
    khat_ret: torch.Tensor        # [b, cap, 64] bf16
    I_ret: torch.Tensor           # [b, cap] fp32
    pos_ret: torch.Tensor         # [b, cap] int32
    next_pos: torch.Tensor        # [b] int32
    evicted: torch.Tensor         # [b] int32


@dataclasses.dataclass
class PagedCache:
    """A paged cache of one layer: pages K, V [n_pages, page_size, Hkv, d], the
    pages of each sequence and its cached length (new tokens included; the
    caller advances it before a call with new tokens)."""
    K: torch.Tensor
    V: torch.Tensor
    block_table: torch.Tensor     # [b, max_pages] int32
    kv_len: torch.Tensor          # [b] int32


class IndexMemLayer:
    """Context for one layer. ``weights`` holds device tensors W_iq [Hq,d,dI],
    W_ik [H,dI], w_ig [H,Hq] (model dtype), W_phi [r,d], w_gate [Hq,d] (fp32).

    readout="gated" is IndexMem's memory readout; readout="moment" keeps
    MomentKV's moment statistics instead (r = d, no decay; W_phi and w_gate
    are not used): update_memory then accumulates them and decode mixes the
    retained attention with their estimate of the evicted attention."""

    def __init__(self, hidden, n_q_heads, n_kv_heads, head_dim, idx_dim, mem_r, lam, dtype,
                 weights, gate_override: Optional[float] = None, eps: float = 1e-6,
                 readout: str = "gated"):
        if readout not in ("gated", "moment"):
            raise ValueError("readout must be 'gated' or 'moment'")
        self.moment = readout == "moment"
        if self.moment:
            mem_r, lam = head_dim, 1.0
        self.dims = dict(hidden=hidden, n_q_heads=n_q_heads, n_kv_heads=n_kv_heads,
                         head_dim=head_dim, idx_dim=idx_dim, mem_r=mem_r)
        self.lam = lam
        self.torch_dtype = dtype
        self.code = B_.BF16 if dtype == torch.bfloat16 else B_.FP32
        cfg = B_.make_config(hidden, n_q_heads, n_kv_heads, head_dim, idx_dim, mem_r, lam,
                             self.code, eps=eps, gate_override=gate_override,
                             readout=B_.READOUT_MOMENT if self.moment else B_.READOUT_GATED)
        self.ctx = B_.init(cfg, weights["W_iq"], weights["W_ik"], weights["w_ig"],
                           None if self.moment else weights["W_phi"],
                           None if self.moment else weights["w_gate"])
        self._ws = None
        self._ws_key = None
        self._device = weights["W_ik"].device
        self._index = weights["W_ik"].get_device()
        self._hq, self._hkv, self._d = n_q_heads, n_kv_heads, head_dim

    @classmethod
    def from_shape(cls, shape, weights, gate_override=None, readout: str = "gated"):
        return cls(shape.hidden, shape.n_q_heads, shape.n_kv_heads, shape.head_dim,
                   shape.idx_dim, shape.mem_r, shape.lam, shape.torch_dtype, weights,
                   gate_override=gate_override, readout=readout)

    def close(self):
        if self.ctx:
            B_.destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- buffers ---------------------------------------------------------------
    def workspace(self, batch: int, L: int, B: int, device) -> torch.Tensor:
        key = (batch, L, B)
        if self._ws is None or self._ws_key != key:
            n = B_.workspace_size(self.ctx, batch, L, B)
            self._ws = torch.zeros(n, dtype=torch.uint8, device=device)   # zero-filled once
            self._ws_key = key
        return self._ws

    def workspace_evict(self, batch: int, L: int, B: int, chunk: int, device) -> torch.Tensor:
        """Workspace for pre-eviction (also serves decode)."""
        key = ("evict", batch, L, B, chunk)
        if self._ws is None or self._ws_key != key:
            n = B_.workspace_size_evict(self.ctx, batch, L, B, chunk)
            self._ws = torch.zeros(n, dtype=torch.uint8, device=device)
            self._ws_key = key
        return self._ws

    def new_state(self, batch: int, L: int, B: int, cap: int, device) -> PrefillState:
        d, Hkv, r = self.dims["head_dim"], self.dims["n_kv_heads"], self.dims["mem_r"]
        return PrefillState(
            running_max=torch.empty(batch, L, dtype=torch.float32, device=device),
            idx_retained=torch.empty(batch, B, dtype=torch.int32, device=device),
            idx_evicted=torch.empty(batch, max(L - B, 1), dtype=torch.int32, device=device),
            K_ret=torch.zeros(batch, cap, Hkv, d, dtype=self.torch_dtype, device=device),
            V_ret=torch.zeros(batch, cap, Hkv, d, dtype=self.torch_dtype, device=device),
            cache_len=torch.full((batch,), B, dtype=torch.int32, device=device),
            M=torch.zeros(batch, Hkv, r, d, dtype=torch.float32, device=device),
            bstab=torch.zeros(batch, Hkv, r, dtype=torch.float32, device=device),
            s_v=(torch.zeros(batch, Hkv, d, dtype=torch.float32, device=device)
                 if self.moment else None),
            n_e=torch.zeros(batch, dtype=torch.float32, device=device) if self.moment else None)

    # -- the path --------------------------------------------------------------
    def score_and_evict(self, X, Q, K, V, st: PrefillState, B: int, q_ranges=None,
                        stream=None):
        batch, L = X.shape[0], X.shape[1]
        ws = self.workspace(batch, L, B, X.device)
        ranges = q_ranges or [(0, L)]
        for i, (q0, q1) in enumerate(ranges):
            last = i == len(ranges) - 1
            B_.score_and_evict(self.ctx, batch, L, B, X, Q, K, V, st.running_max, q0, q1,
                               1 if last else 0, st.idx_retained,
                               st.idx_evicted if B < L else None, st.K_ret, st.V_ret,
                               st.K_ret.shape[1], ws, stream)

    def prefill_evict(self, X, Q, K, V, st: PrefillState, B: int, chunk: int,
                      mem_chunk: int = 512, stream=None, record: bool = False):
        """Chunked prefill with pre-eviction after every query range of
        ``chunk`` tokens: the cache never holds more than B tokens and the
        evicted ones enter the memory as they leave. Fills st.idx_retained
        (first min(B, L) entries), st.K_ret/V_ret, st.M, st.bstab.
        record=True returns per range the candidates' importances, the
        retained and the evicted positions (copies, for inspection)."""
        batch, L = X.shape[0], X.shape[1]
        ws = self.workspace_evict(batch, L, B, chunk, X.device)
        ev = torch.empty(batch * chunk, dtype=torch.int32, device=X.device)
        cand = (torch.empty(batch, B + chunk, dtype=torch.float32, device=X.device)
                if record else None)
        recs = []
        for q0 in range(0, L, chunk):
            q1 = min(L, q0 + chunk)
            B_.prefill_evict_chunk(self.ctx, batch, L, B, chunk, X, Q, K, V, q0, q1,
                                   st.idx_retained, ev, cand, st.M, st.bstab, mem_chunk,
                                   q1 == L, st.K_ret, st.V_ret, st.K_ret.shape[1], ws, stream)
            if record:
                B_.join(self.ctx, stream)   # the range's selection runs on a second stream
                n = min(B, q0) + (q1 - q0)
                n_ev = max(0, n - B)
                recs.append({"range": (q0, q1), "I": cand[:, :n].clone(),
                             "retained": st.idx_retained[:, :min(B, q1)].clone(),
                             "evicted": ev[:batch * n_ev].view(batch, n_ev).clone()})
        st.cache_len.fill_(min(B, L))
        return recs

    def update_memory(self, K, V, st: PrefillState, B: int, chunk: int = 512, stream=None):
        batch, L = K.shape[0], K.shape[1]
        ws = self.workspace(batch, L, B, K.device)
        idx = st.idx_evicted if B < L else None
        if self.moment:
            B_.update_moments(self.ctx, batch, L, K, V, idx, L - B, chunk, st.M, st.bstab, st.s_v,
                              st.n_e, ws, stream)
        else:
            B_.update_memory(self.ctx, batch, L, K, V, idx, L - B, chunk, st.M, st.bstab, ws,
                             stream)

    def invalidate_decode(self, batch: int, stream=None):
        """After writing a retained cache, its length or the memory state
        other than through this layer: the next decode step then loads
        nothing before its launch-dependency wait."""
        if self._ws is not None:
            B_.decode_invalidate(self.ctx, batch, self._ws, stream)

    def decode(self, q, k_new, v_new, st: PrefillState, out=None, B: Optional[int] = None,
               L: Optional[int] = None, stream=None):
        batch = q.shape[0]
        if self._ws is None:
            raise RuntimeError("decode needs the workspace of a prefill (or call workspace())")
        if out is None:
            out = torch.empty_like(q)
        if self.moment:
            B_.decode_moment(self.ctx, batch, q, k_new, v_new, st.K_ret, st.V_ret, st.cache_len,
                             st.K_ret.shape[1], st.M, st.bstab, st.s_v, st.n_e, out, self._ws,
                             stream)
        else:
            B_.decode(self.ctx, batch, q, k_new, v_new, st.K_ret, st.V_ret, st.cache_len,
                      st.K_ret.shape[1], st.M, st.bstab, out, self._ws, stream)
        return out

    def online_init(self, st: PrefillState, B: int, L: int, stream=None) -> OnlineState:
        """State for decode-time online eviction after a one-shot prefill of L
        tokens into st (same layer, same workspace); the cache has B tokens."""
        batch, cap = st.K_ret.shape[0], st.K_ret.shape[1]
        dev = st.K_ret.device
        on = OnlineState(
            khat_ret=torch.zeros(batch, cap, 64, dtype=torch.bfloat16, device=dev),
            I_ret=torch.zeros(batch, cap, dtype=torch.float32, device=dev),
            pos_ret=torch.zeros(batch, cap, dtype=torch.int32, device=dev),
            next_pos=torch.zeros(batch, dtype=torch.int32, device=dev),
            evicted=torch.zeros(batch, dtype=torch.int32, device=dev))
        B_.online_init(self.ctx, batch, L, B, st.running_max, st.idx_retained, self._ws,
                       on.khat_ret, on.I_ret, on.pos_ret, on.next_pos, cap, stream)
        return on

    def decode_online(self, x_new, q, k_new, v_new, st: PrefillState, on: OnlineState, B: int,
                      out=None, stream=None):
        """One decode step that keeps the cache at B tokens: the least
        important of the B + 1 leaves into the memory (on.evicted: its
        position)."""
        batch = q.shape[0]
        if out is None:
            out = torch.empty_like(q)
        B_.decode_online(self.ctx, batch, B, x_new, q, k_new, v_new, st.K_ret, st.V_ret,
                         on.khat_ret, on.I_ret, on.pos_ret, on.next_pos, st.cache_len,
                         st.K_ret.shape[1], st.M, st.bstab, out, on.evicted, self._ws, stream)
        return out

    def _as_current(self, stream):
        """Makes ``stream`` (a torch stream or a handle; None: the current one)
        torch's current stream, so that what is allocated and filled inside
        belongs to it."""
        if stream is None:
            return contextlib.nullcontext()
        if not isinstance(stream, torch.cuda.Stream):
            handle = int(getattr(stream, "cuda_stream", stream))
            # an ExternalStream of handle 0 would be a new stream of torch's pool
            stream = (torch.cuda.ExternalStream(handle, device=self._device) if handle
                      else torch.cuda.default_stream(self._device))
        return torch.cuda.stream(stream)

    # -- rotary positions and the paged cache -----------------------------------
    def set_rope(self, rot_dim: Optional[int] = None, base: float = 10000.0, layout: str = "half",
                 scaling: str = "plain", factor: float = 1.0, low: float = 1.0, high: float = 4.0,
                 orig_len: int = 8192, magnitude: float = 1.0):
        """The layer's rotary positions (rot_dim None: the whole head). scaling:
        "plain", "linear", "band" (turns low..high over orig_len) or "ramp"
        (YaRN's, over the pair's index); rot_dim 0 removes the rotation."""
        if layout not in B_.ROPE_LAYOUTS or scaling not in B_.ROPE_SCALINGS:
            raise ValueError("layout must be one of %s, scaling one of %s" % (
                sorted(B_.ROPE_LAYOUTS), sorted(B_.ROPE_SCALINGS)))
        rot = self.dims["head_dim"] if rot_dim is None else rot_dim
        B_.set_rope(self.ctx, B_.Rope(rot, B_.ROPE_LAYOUTS[layout], B_.ROPE_SCALINGS[scaling],
                                      orig_len, base, factor, low, high, magnitude)
                    if rot else None)

    def new_paged(self, batch: int, n_pages: int, page_size: int, max_pages: int,
                  device) -> PagedCache:
        """Empty pages and an empty table (no page assigned: entries -1)."""
        shape = (n_pages, page_size, self.dims["n_kv_heads"], self.dims["head_dim"])
        return PagedCache(
            K=torch.empty(shape, dtype=self.torch_dtype, device=device),
            V=torch.empty(shape, dtype=self.torch_dtype, device=device),
            block_table=torch.full((batch, max_pages), -1, dtype=torch.int32, device=device),
            kv_len=torch.zeros(batch, dtype=torch.int32, device=device))

    # The checks below run on every call of a decode step: few attribute reads,
    # the explanation only where one fails.
    def _tokens(self, name: str, x, n: int, heads: int) -> int:
        """Checks a token tensor [n, heads, d] (its rows may be strided);
        returns the row stride."""
        d, s = self._d, x.stride()
        if x.shape == (n, heads, d) and x.dtype is self.torch_dtype and \
                x.get_device() == self._index and s[2] == 1 and (s[1] == d or heads == 1) and \
                (n < 2 or s[0] >= heads * d):
            return s[0] if n > 1 else 0
        raise ValueError("%s must be %s [%d, %d, %d] on %s, rows apart and their heads contiguous; got %s %s"
                         " with strides %s on %s" % (name, self.torch_dtype, n, heads, d,
                                                     self._device, x.dtype, tuple(x.shape), s,
                                                     x.device))

    def _ints(self, name: str, x, shape):
        if x.dtype is not torch.int32 or x.shape != shape or x.get_device() != self._index or \
                not x.is_contiguous():
            raise ValueError("%s must be contiguous int32 %s on %s" % (name, tuple(shape),
                                                                       self._device))

    def _new(self, stream, shape, dtype):
        """A tensor for the results of a call on a given stream: memory of that stream
        (the current one's could still be written by work queued there), which
        the current one may read on."""
        caller = torch.cuda.current_stream(self._device)
        with self._as_current(stream):
            t = torch.empty(shape, dtype=dtype, device=self._device)
        t.record_stream(caller)
        return t

    def _out(self, name: str, out, like, stream, n: int, heads: int):
        """The output tensor (allocated if None) and its row stride."""
        if out is None:
            if stream is None:
                return torch.empty_like(like, memory_format=torch.contiguous_format), 0
            return self._new(stream, (n, heads, self._d), self.torch_dtype), 0
        return out, self._tokens(name, out, n, heads)

    def _paged(self, c: PagedCache):
        K, V, table = c.K, c.V, c.block_table
        sh, ts, dt, dev = K.shape, table.shape, self.torch_dtype, self._index
        if len(sh) != 4 or sh[2] != self._hkv or sh[3] != self._d or V.shape != sh or \
                K.dtype is not dt or V.dtype is not dt or K.get_device() != dev or \
                V.get_device() != dev or not K.is_contiguous() or not V.is_contiguous():
            raise ValueError("cache pages must be contiguous %s [n_pages, page_size, %d, %d] on %s"
                             % (dt, self._hkv, self._d, self._device))
        if len(ts) != 2:
            raise ValueError("block_table must be [batch, max_pages]")
        self._ints("block_table", table, ts)
        self._ints("kv_len", c.kv_len, ts[:1])
        return B_.Paged(K.data_ptr(), V.data_ptr(), table.data_ptr(), c.kv_len.data_ptr(), sh[0],
                        sh[1], ts[1]), ts[0]

    def rotate(self, q, k, positions, q_out=None, k_out=None, inverse: bool = False, stream=None):
        """Rotary positions: q [T, Hq, d] and k [T, Hkv, d] (either may be None)
        turned by positions [T]; returns (q_out, k_out). The outputs may be the
        inputs."""
        if q is None and k is None:
            raise ValueError("rotate needs q or k")
        T = (k if q is None else q).shape[0]
        self._ints("positions", positions, (T,))
        qs = qos = ks = kos = 0
        if q is None:
            q_out = None
        else:
            qs = self._tokens("q", q, T, self._hq)
            q_out, qos = self._out("q_out", q_out, q, stream, T, self._hq)
        if k is None:
            k_out = None
        else:
            ks = self._tokens("k", k, T, self._hkv)
            k_out, kos = self._out("k_out", k_out, k, stream, T, self._hkv)
        if T:
            B_.rotate(self.ctx, T, positions.data_ptr(), q if q is None else q.data_ptr(), qs,
                      q if q is None else q_out.data_ptr(), qos, k if k is None else k.data_ptr(),
                      ks, k if k is None else k_out.data_ptr(), kos, 1 if inverse else 0, stream)
        return q_out, k_out

    def append_paged(self, k, v, cache: PagedCache, tok_start=None, positions=None, q=None,
                     q_out=None, rotate: bool = True, stream=None):
        """Writes the new tokens' keys (rotated) and values [T, Hkv, d] into the
        cache; with q [T, Hq, d] returns the rotated queries. tok_start [b + 1]:
        the sequences' token ranges (None: equally many each); cache.kv_len
        already counts the new tokens."""
        pg, b = self._paged(cache)
        T = k.shape[0]
        ks, vs = self._tokens("k", k, T, self._hkv), self._tokens("v", v, T, self._hkv)
        if tok_start is not None:
            self._ints("tok_start", tok_start, (b + 1,))
        if positions is not None:
            self._ints("positions", positions, (T,))
        qs = qos = 0
        if q is None:
            q_out = None
        else:
            qs = self._tokens("q", q, T, self._hq)
            q_out, qos = self._out("q_out", q_out, q, stream, T, self._hq)
        if T:
            B_.append_paged(self.ctx, b, T, tok_start if tok_start is None else tok_start.data_ptr(),
                            positions if positions is None else positions.data_ptr(), k.data_ptr(),
                            ks, v.data_ptr(), vs, q if q is None else q.data_ptr(), qs,
                            q if q is None else q_out.data_ptr(), qos, 1 if rotate else 0, pg,
                            stream)
        return q_out

    def attend_paged(self, q, cache: PagedCache, tok_start=None, max_new: Optional[int] = None,
                     max_len: Optional[int] = None, scale: Optional[float] = None, out=None,
                     lse=None, return_lse: bool = False, stream=None):
        """Causal attention of the new tokens q [T, Hq, d] over the paged cache
        (their own rows appended before), out not overlapping q. scale: of the
        logits (default 1/sqrt(d)). max_new: most new tokens of a sequence
        (default: T, or T / b without tok_start; the kernel is chosen by it, so a
        decode step with tok_start should say 1); max_len: the longest kv_len
        expected (a hint; default: what the table can hold). Returns out, or
        (out, lse [T, Hq] fp32) with return_lse."""
        pg, b = self._paged(cache)
        T, Hq = q.shape[0], self._hq
        qs = self._tokens("q", q, T, Hq)
        out, os_ = self._out("out", out, q, stream, T, Hq)
        if tok_start is not None:
            self._ints("tok_start", tok_start, (b + 1,))
        if lse is not None:
            if lse.dtype is not torch.float32 or lse.shape != (T, Hq) or \
                    not lse.is_contiguous() or lse.get_device() != self._index:
                raise ValueError("lse must be contiguous float32 [%d, %d]" % (T, Hq))
        elif return_lse:
            lse = (torch.empty(T, Hq, dtype=torch.float32, device=q.device) if stream is None
                   else self._new(stream, (T, Hq), torch.float32))
        if scale is not None and not 1e-30 < scale < 1e30:
            raise ValueError("scale must be positive and finite")
        if max_new is None:
            max_new = T if tok_start is not None else T // max(b, 1)
        if max_len is None:
            max_len = min(pg.max_pages * pg.page_size, 2 ** 31 - 1)
        if T:
            B_.attend_paged(self.ctx, b, T, tok_start if tok_start is None else tok_start.data_ptr(),
                            max_new, max_len, q.data_ptr(), qs, pg, 0.0 if scale is None else scale,
                            out.data_ptr(), os_, lse if lse is None else lse.data_ptr(), stream)
        return (out, lse) if return_lse else out

    def gather_paged(self, cache: PagedCache, idx=None, n: Optional[int] = None, K=None, V=None,
                     stream=None):
        """Rows at positions idx [b, n] (None: positions 0..n-1) of the paged
        cache, to K, V [b, cap >= n, Hkv, d] (allocated if None). Call
        invalidate_decode after gathering into a cache that decode steps used."""
        pg, b = self._paged(cache)
        if idx is None:
            if n is None:
                raise ValueError("gather_paged needs idx or n")
        else:
            n = idx.shape[-1]
            self._ints("idx", idx, (b, n))
        tail = (self._hkv, self._d)
        if K is None and V is None:
            if stream is None:
                K, V = cache.K.new_empty((b, n) + tail), cache.K.new_empty((b, n) + tail)
            else:
                K, V = (self._new(stream, (b, n) + tail, self.torch_dtype) for _ in range(2))
        elif K is None or V is None or K.shape != V.shape or K.dim() != 4 or K.shape[0] != b or \
                K.shape[1] < n or K.shape[2:] != tail or K.dtype != self.torch_dtype or \
                V.dtype != self.torch_dtype or K.device != self._device or \
                V.device != self._device or not K.is_contiguous() or not V.is_contiguous():
            raise ValueError("K and V must be contiguous %s [%d, >= %d, %d, %d] on %s" % (
                (self.torch_dtype, b, n) + tail + (self._device,)))
        if n:
            B_.gather_paged(self.ctx, b, n, idx if idx is None else idx.data_ptr(), n, pg,
                            K.data_ptr(), V.data_ptr(), K.shape[1], stream)
        return K, V

    def evict_paged(self, X, Q, cache: PagedCache, st: PrefillState, B: int, chunk: int = 512,
                    stream=None):
        """From a paged prompt to the decode state: scores the prompt's hidden
        states X [b, L, H] and queries Q [b, L, Hq, d], keeps the B most
        important of its L cached tokens in st's retained cache and adds the
        others to the memory. Every sequence holds L tokens (a shorter one is
        reported by sync as IMEM_ERR_RANGE); the pages are free to be reused
        once the stream has passed this call."""
        b, L = X.shape[0], X.shape[1]
        caller = torch.cuda.current_stream(self._device)
        # positions, rows and a new workspace are made on the call's stream: filled
        # in its order, and their memory not given out again before it is through
        with self._as_current(stream):
            at = torch.arange(L, dtype=torch.int32, device=X.device).expand(b, L).contiguous()
            K, V = self.gather_paged(cache, at)
            self.score_and_evict(X, Q, K, V, st, B)
            self.update_memory(K, V, st, B, chunk=chunk)
            # the workspace stays with the layer, for calls on either stream
            self._ws.record_stream(torch.cuda.current_stream(self._device))
            self._ws.record_stream(caller)

    def sync(self, stream=None):
        B_.sync(self.ctx, stream)
