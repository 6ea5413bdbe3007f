// rope.cu -- rotary positions: queries and keys of n_tokens rotated, either to
// contiguous outputs (imem_rotate) or, the keys with their values, into the
// paged cache (imem_append_paged), in one launch.
//
//   pair (x1, x2) of frequency theta, position p, a = p theta:
//   y1 = m (x1 cos a - x2 sin a),  y2 = m (x2 cos a + x1 sin a)
//
// Angles. theta / (2 pi) is formed in fp64 on the host and kept as a 64-bit
// fraction of a turn; p times it, mod 2^64, is the phase with an error of at
// most |p| 2^-55 turns (2^-35 at a million tokens), where p * theta in fp32
// would be off by 2^-24 of p theta (a hundredth of a radian at 131072). Its
// top 32 bits, as a signed number of half turns, go to sincospif: one integer
// multiplication, no fp64 on the device.
//
// Bound by HBM: every element is read and written once. A CTA takes a few
// tokens: its threads put the first vectors' loads in flight, then form the
// tokens' cos and sin in shared memory (once per token and pair, shared by
// all its heads) and the cache rows, then rotate and store. A work item is 32
// bytes of a head: two 16-byte vectors, in the half layout the two that hold
// a pair's halves, so that every access is a full vector and no element is
// read twice. 64K tokens of 40 heads of 128: 203 us, 6.6 TB/s (the copy rate);
// append of 26,752 tokens, 48 heads' rows each: 105 us, 6.3 TB/s.
#include "common.cuh"
#include "internal.h"
#include "paged.cuh"

namespace imem {
namespace {

constexpr int kRotThreads = 256;
constexpr int kRotTokens = 4;    // tokens per CTA (long calls; 8: 3 % slower)

template <typename T> struct Vec { static constexpr int n = 16 / sizeof(T); };

template <typename T> __device__ __forceinline__ void unpack(const uint4& u, float* f);
template <> __device__ __forceinline__ void unpack<float>(const uint4& u, float* f) {
  f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y);
  f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
}
template <> __device__ __forceinline__ void unpack<__nv_bfloat16>(const uint4& u, float* f) {
  bf16x8_to_f32(u, f);
}
template <typename T> __device__ __forceinline__ uint4 pack(const float* f) {
  uint4 u;
  if constexpr (sizeof(T) == 4) {
    u = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                   __float_as_uint(f[3]));
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<uint32_t*>(&h);
    }
    u = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return u;
}

// One item: two vectors of a head row and what becomes of them.
struct Item {
  int src0, src1;      // element offsets within the head
  int head;            // row among the token's [q heads | k heads | v heads]
  int token;           // within the CTA
  int kind;            // 0 q, 1 k, 2 v
  bool turn;
};

// kPaged: append (k and v go to cache rows). D: head dimension. by_per:
// ceil(2^32 / items per token), which divides item numbers (below 2^16) by it.
template <typename T, int D, bool kPaged>
__global__ void __launch_bounds__(kRotThreads)
rotate_kernel(const __grid_constant__ RotateArgs a, const __grid_constant__ RopeTable rope, int Hq,
              int Hkv, int tokens, uint32_t by_per, int* __restrict__ err) {
  constexpr int V = Vec<T>::n;
  constexpr int IPH = D / (2 * V);        // items per head
  // pair f = j V + e at [e (64 / V) + j]: lanes of neighbouring items read side by side
  constexpr int VS = 64 / V;
  __shared__ float2 s_cs[kRotTokens][64];
  __shared__ long long s_row[kRotTokens];  // cache row, -1: token skipped
  __shared__ int s_pos[kRotTokens];

  const int tid = threadIdx.x;
  const int t0 = blockIdx.x * tokens;
  const int nt = min(tokens, a.n_tokens - t0);
  const int half = rope.rot_dim >> 1;
  const int nq = a.q ? Hq : 0, nk = a.k ? Hkv : 0, nv = kPaged ? Hkv : 0;
  const int per = (nq + nk + nv) * IPH;   // items per token
  const int total = per * nt;

  auto item = [&](int i) {
    Item it;
    it.token = __umulhi(i, by_per);
    const int r = i - it.token * per;
    it.head = r / IPH;
    const int j = r - it.head * IPH;
    it.kind = it.head < nq ? 0 : it.head < nq + nk ? 1 : 2;
    it.turn = false;
    it.src0 = 2 * j * V;
    it.src1 = it.src0 + V;
    if (a.rotate && it.kind < 2) {
      if (rope.interleaved) {
        it.turn = it.src0 < rope.rot_dim;
      } else if (j * V < half) {
        it.turn = true;
        it.src0 = j * V;
        it.src1 = it.src0 + half;
      }   // else: items past the pairs cover the rest of the head, as above
    }
    return it;
  };
  auto source = [&](const Item& it) -> const T* {
    const long long t = t0 + it.token;
    if (it.kind == 0) return (const T*)a.q + t * a.q_stride + it.head * D;
    if (it.kind == 1) return (const T*)a.k + t * a.k_stride + (it.head - nq) * D;
    return (const T*)a.v + t * a.v_stride + (it.head - nq - nk) * D;
  };

  // the first item's loads need nothing of what follows (two items in flight
  // per thread: 15 % slower, fewer CTAs fit)
  uint4 x0, x1;
  auto load = [&](const Item& it) {
    const T* p = source(it);
    x0 = *reinterpret_cast<const uint4*>(p + it.src0);
    x1 = *reinterpret_cast<const uint4*>(p + it.src1);
  };
  if (tid < total) load(item(tid));

  // ranges that no token falls into are looked at too, by the first CTA's warps
  // without a token
  if (kPaged && a.start && blockIdx.x == 0 && tid >= kRotTokens * 32)
    for (int i = tid - kRotTokens * 32; i < a.batch; i += kRotThreads - kRotTokens * 32) {
      const int from = a.start[i], to = a.start[i + 1];
      if (from < 0 || to < from || to > a.n_tokens) record_error(err, DEV_RANGE);
    }

  // positions and, for append, cache rows: one warp per token
  for (int k = tid >> 5; k < nt; k += kRotThreads / 32) {
    const int lane = tid & 31, t = t0 + k;
    int pos = 0;
    long long row = 0;
    if constexpr (kPaged) {
      // the sequence: how many of tok_start[1..batch] are <= t (32 at a time)
      int s = 0;
      if (a.start) {
        for (int i = lane; i < a.batch; i += 32) s += a.start[i + 1] <= t;
        s = __reduce_add_sync(0xffffffffu, s);
      } else {
        s = t / (a.n_tokens / a.batch);
      }
      row = -1;
      if (lane == 0 && s < a.batch) {
        const SeqInfo q = seq_info(s, a.batch, a.n_tokens, a.start, a.pg);
        const int i = t - q.tok0;
        if (q.bad) record_error(err, DEV_RANGE);
        if (i >= 0 && i < q.n && !q.bad) {
          pos = q.len - q.n + i;
          if (pos >= 0) {
            row = cache_row(a.pg, a.pg.table + (long long)s * a.pg.max_pages, pos);
            if (row < 0) record_error(err, DEV_RANGE);
          }
        }
      }
      if (a.positions) pos = a.positions[t];
    } else {
      pos = a.positions[t];
    }
    if (lane == 0) {
      s_pos[k] = pos;
      s_row[k] = row;
    }
  }
  __syncthreads();
  if (a.rotate) {
    for (int i = tid; i < nt * half; i += kRotThreads) {
      const int k = i / half, f = i - k * half;
      const uint64_t phase = rope.turn[f] * (uint64_t)(int64_t)s_pos[k];
      const float x = (float)(int32_t)(phase >> 32) * 0x1p-31f;   // half turns in [-1, 1)
      float sn, cs;
      sincospif(x, &sn, &cs);
      s_cs[k][f % V * VS + f / V] = make_float2(cs * rope.magnitude, (a.inverse ? -sn : sn) * rope.magnitude);
    }
    __syncthreads();
  }

  for (int i = tid; i < total; i += kRotThreads) {
    const Item it = item(i);
    if (i != tid) load(it);
    if (kPaged && s_row[it.token] < 0) continue;
    if (it.turn) {
      float f0[V], f1[V];
      unpack<T>(x0, f0);
      unpack<T>(x1, f1);
      if (rope.interleaved) {
        const float2* cs = &s_cs[it.token][it.src0 / (2 * V)];
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
          const float2 p = cs[e * VS], q = cs[(V / 2 + e) * VS];
          const float a0 = f0[2 * e], b0 = f0[2 * e + 1], a1 = f1[2 * e], b1 = f1[2 * e + 1];
          f0[2 * e] = a0 * p.x - b0 * p.y;
          f0[2 * e + 1] = b0 * p.x + a0 * p.y;
          f1[2 * e] = a1 * q.x - b1 * q.y;
          f1[2 * e + 1] = b1 * q.x + a1 * q.y;
        }
      } else {
        const float2* cs = &s_cs[it.token][it.src0 / V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float2 p = cs[e * VS];
          const float a0 = f0[e], b0 = f1[e];
          f0[e] = a0 * p.x - b0 * p.y;
          f1[e] = b0 * p.x + a0 * p.y;
        }
      }
      x0 = pack<T>(f0);
      x1 = pack<T>(f1);
    }
    const long long t = t0 + it.token;
    T* p;
    if (it.kind == 0) p = (T*)a.q_out + t * a.q_out_stride + it.head * D;
    else if (kPaged) {
      const int h = it.kind == 1 ? it.head - nq : it.head - nq - nk;
      p = (T*)(it.kind == 1 ? a.pg.k : a.pg.v) + (s_row[it.token] * Hkv + h) * D;
    } else {
      p = (T*)a.k_out + t * a.k_out_stride + (it.head - nq) * D;
    }
    *reinterpret_cast<uint4*>(p + it.src0) = x0;
    *reinterpret_cast<uint4*>(p + it.src1) = x1;
  }
}

template <typename T, int D>
cudaError_t launch_td(const Ctx& c, const RotateArgs& a, cudaStream_t st) {
  // one token per CTA until the SMs are full twice over: short calls are
  // bound by latency, long ones by HBM and by forming the angles
  const int tokens = a.n_tokens >= 2 * kRotTokens * c.num_sms ? kRotTokens
                     : a.n_tokens > 2 * c.num_sms ? 2 : 1;
  const int grid = (a.n_tokens + tokens - 1) / tokens;
  const int Hq = c.cfg.n_q_heads, Hkv = c.cfg.n_kv_heads;
  const uint32_t per = ((a.q ? Hq : 0) + (a.k ? Hkv : 0) + (a.pg.k ? Hkv : 0)) * (D * sizeof(T) / 32);
  const uint32_t by_per = 0xffffffffu / per + 1;
  if (a.pg.k)
    rotate_kernel<T, D, true><<<grid, kRotThreads, 0, st>>>(a, c.rope, Hq, Hkv, tokens, by_per, c.err);
  else
    rotate_kernel<T, D, false><<<grid, kRotThreads, 0, st>>>(a, c.rope, Hq, Hkv, tokens, by_per, c.err);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rotate(const Ctx& c, const RotateArgs& a, cudaStream_t st) {
  if (c.cfg.dtype == IMEM_BF16)
    return c.cfg.head_dim == 128 ? launch_td<__nv_bfloat16, 128>(c, a, st)
                                 : launch_td<__nv_bfloat16, 64>(c, a, st);
  return c.cfg.head_dim == 128 ? launch_td<float, 128>(c, a, st) : launch_td<float, 64>(c, a, st);
}

}  // namespace imem
