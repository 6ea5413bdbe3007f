// attend.cu -- causal attention of new tokens over the paged cache: the choice
// of the kernel, and the kernel of the fp32 model dtype.
//
//   s_ij = scale q_i . k_j,  o_i = sum_{j <= p_i} softmax(s_i)_j v_j
//
// fp32 products on the tensor cores. A value is split into hi (rounded to the
// operand format tf32, 11 significant bits) and lo = x - hi (exact, of either
// sign; its upper 11 bits are kept), and a product becomes hi hi + hi lo +
// lo hi with fp32 accumulation: what is dropped is below 2^-21 of |x y| (lo lo
// 2^-22, the bits of a lo behind its eleventh 2^-23 on either side). The
// unit cuts its sums off instead of rounding them, which over many keys
// would pull every sum towards zero, so that only short chains stay inside it
// (16 dimensions, one stage of keys) and meet by rounded additions: 1.6e-6
// off the exact outputs without that, for 1024 keys. Bound by the warp-level
// MMA: one m16n8k8 (tf32) or m16n8k16 (bf16) per 16 clocks and SM quarter, so
// three tf32 products cost as much as six bf16 ones of a three-way split with
// less arithmetic around them, and both beat the fp32 units as far as shared
// memory feeds those (1024 new tokens, 8 heads of 64: 44-47 us, 23-25 TFLOP/s; on
// the fp32 units 56 us).
//
// An infinite value has no such halves (lo = inf - inf): its products are NaN
// whatever they should be. A CTA that finds a NaN among its rows' sums and
// outputs therefore takes its keys a second time by whole products on the fp32
// units, where masked places do not enter at all: infinities then count as they
// are, and what stays NaN is NaN by the formulas.
//
// A tile's rows are the new tokens of one sequence times the G query heads of
// one KV head (row r: token r / G, head r % G), so that K and V are read once
// for the whole group. Stages of 32 keys come by cp.async, one ahead. Each of
// four warps has 16 rows (KS = 1), or, with at most 32 or 16 rows in all, two or
// four warps share 16 rows and have a part of each stage's keys (KS = 2, 4).
// The contraction's index order is free: queries and keys are taken four
// dimensions a lane (one 16-byte load for two MMA steps), values four columns
// a lane.
//
// The keys of a tile are split over a cluster of CTAs when there are too few
// tiles to fill the GPU; the states (m, l, O) meet over distributed shared
// memory, summed in a fixed order.
#include "common.cuh"
#include "internal.h"
#include "paged.cuh"
#include "tc.cuh"

#include <atomic>

namespace imem {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kThreads = 128;
constexpr float kGrow = 8.f;             // log2 growth of a maximum that is left alone

template <int D, int KS> struct F32Cfg {
  static constexpr int keys = 32;                            // per stage
  // row strides in floats: 16-byte loads of neighbouring rows (K: rows g, V:
  // rows 2 t) then fall on different banks
  static constexpr int ks = D + 16, vs = D + 4, os = D + 4;
  static constexpr int k = keys * ks, v = keys * vs;       // floats of a buffer
  static constexpr int total = 2 * (k + v) * 4;
  static constexpr int state = 16 * os + 32;                 // a warp's (m, l, O), floats
  static_assert((KS == 1 ? 4 : 4 + 4 / KS) * state * 4 <= total, "the states take the buffers' place");
  static_assert((4 * state + 2 * keys * os) * 4 <= total, "states and a stage of whole_states");
};

__device__ __forceinline__ void copy16(float* dst, const float* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(tc::smem_addr(dst)),
               "l"(src), "r"(valid ? 16 : 0) : "memory");   // 0: zero-filled
}
// x = hi + lo, hi the nearest value of 11 significant bits
__device__ __forceinline__ void split(float x, uint32_t& hi, uint32_t& lo) {
  hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;   // (cvt.rna: 48 against 44 us)
  lo = __float_as_uint(x - __uint_as_float(hi));
}
// C (16 x 8) += A (16 x 8) B (8 x 8), tf32 operands
__device__ __forceinline__ void mma8(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The states of the CTA's rows by whole products, each warp's in its place (see
// the kernel's end). Rare, so plain: a row at a time, a key a lane; out of line,
// so that the kernel's own pass keeps its registers.
template <int D, int KS>
__device__ __noinline__ void whole_states(const AttendArgs& a, float* smem, const int32_t* table,
                                          int h, int Hkv, int G, int r0, int n_rows, int tok0,
                                          int past, int n_keys, int b0, int b1) {
  using C = F32Cfg<D, KS>;
  constexpr int kKeys = C::keys, NK = kKeys / KS;   // keys of a stage, of a warp
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* so = smem + warp * C::state;               // O rows, then (m in log2 units, l)
  float* s_k = smem + 4 * C::state;
  float* s_v = s_k + kKeys * C::os;
  const int w_key = warp % KS * NK;
  const float sl2 = a.scale * kLog2e;
  __syncthreads();
  for (int i = lane; i < 16 * C::os; i += 32) so[i] = 0.f;
  so[16 * C::os + lane] = lane & 1 ? 0.f : -INFINITY;
  for (int b = b0; b < b1; ++b) {
    __syncthreads();
    for (int i = threadIdx.x; i < kKeys * (D / 4); i += kThreads) {
      const int r = i / (D / 4), c = (i % (D / 4)) * 4, key = b * kKeys + r;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
      const long long row = key < n_keys ? cache_row(a.pg, table, key) : -1;
      if (row >= 0) {
        x = *reinterpret_cast<const float4*>((const float*)a.pg.k + (row * Hkv + h) * D + c);
        y = *reinterpret_cast<const float4*>((const float*)a.pg.v + (row * Hkv + h) * D + c);
      }
      *reinterpret_cast<float4*>(s_k + r * C::os + c) = x;
      *reinterpret_cast<float4*>(s_v + r * C::os + c) = y;
    }
    __syncthreads();
    for (int r = 0; r < 16; ++r) {
      const int row = min(r0 + warp / KS * 16 + r, n_rows - 1);
      const int seen = past + row / G - (b * kKeys + w_key);   // the warp's last key that the row sees
      const float* q = (const float*)a.q + (long long)(tok0 + row / G) * a.q_stride + (h * G + row % G) * D;
      const float* k = s_k + (w_key + lane % NK) * C::os;
      float x = 0.f;
      for (int c = 0; c < D; c += 4) {
        const float4 u = *reinterpret_cast<const float4*>(q + c);
        const float4 v = *reinterpret_cast<const float4*>(k + c);
        x += u.x * v.x; x += u.y * v.y; x += u.z * v.z; x += u.w * v.w;
      }
      const bool on = lane < NK && lane <= seen;
      x = on ? x * sl2 : -INFINITY;
      const float2 ml = *reinterpret_cast<const float2*>(so + 16 * C::os + 2 * r);
      const float m = fmaxf(ml.x, warp_max(x)), base = m == -INFINITY ? 0.f : m;
      const float f = tc::ex2(ml.x - base), p = tc::ex2(x - base);
      const float l = ml.y * f + warp_sum(on ? p : 0.f);
      for (int d = lane; d < D; d += 32) so[r * C::os + d] *= f;
      for (int i = 0; i < NK && i <= seen; ++i) {
        const float pi = __shfl_sync(0xffffffffu, p, i);
        for (int d = lane; d < D; d += 32) so[r * C::os + d] += pi * s_v[(w_key + i) * C::os + d];
      }
      __syncwarp();
      if (lane == 0) *reinterpret_cast<float2*>(so + 16 * C::os + 2 * r) = make_float2(m, l);
      __syncwarp();
    }
  }
}

template <int D, int KS>
__global__ void __launch_bounds__(kThreads)
attend_f32_kernel(const __grid_constant__ AttendArgs a, int Hq, int G, int S, int tiles,
                  int* __restrict__ err) {
  using C = F32Cfg<D, KS>;
  constexpr int kKeys = C::keys;
  constexpr int NT = kKeys / 8 / KS;       // 8-key tiles of a warp per stage
  constexpr int BM = 64 / KS;              // rows of the CTA
  extern __shared__ __align__(16) float smem[];
  float* s_k = smem;
  float* s_v = smem + 2 * C::k;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int Hkv = Hq / G;
  int idx = blockIdx.x;
  const int rank = idx % S;
  idx /= S;
  const int h = idx % Hkv;
  idx /= Hkv;
  const int seq = idx % a.batch;
  const int tile = tiles - 1 - idx / a.batch;   // the longest first
  const SeqInfo sq = seq_info(seq, a.batch, a.n_tokens, a.start, a.pg);
  if (tile == 0 && rank == 0 && h == 0 && tid == 0 && (sq.bad || sq.n > a.max_new))
    record_error(err, DEV_RANGE);
  const int n_rows = min(sq.n, a.max_new) * G;
  const int r0 = tile * BM;
  if (r0 >= n_rows) return;         // the whole cluster
  const int past = sq.len - sq.n;   // position of the first new token
  const int n_tile = min(BM, n_rows - r0);
  const int n_keys = max(0, past + (r0 + n_tile - 1) / G + 1);
  const int blocks = (n_keys + kKeys - 1) / kKeys;
  const int per = (blocks + S - 1) / S;
  const int b0 = min(rank * per, blocks), b1 = min(b0 + per, blocks);
  const int32_t* table = a.pg.table + (long long)seq * a.pg.max_pages;

  // a stage's keys and values; rows that no row of the tile sees become zeros
  auto issue = [&](int b, int buf) {
    constexpr int CH = D / 4, STEP = kThreads / CH, N = kKeys / STEP;
    const int c = (tid % CH) * 4, first = b * kKeys + tid / CH;
    // all table entries first: their latencies overlap
    int page[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int key = first + i * STEP;
      page[i] = key < n_keys ? __ldg(table + (key >> a.pg.page_log)) : -1;
    }
    bool bad = false;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int key = first + i * STEP, r = tid / CH + i * STEP;
      const bool in = page[i] >= 0 && page[i] < a.pg.n_pages;
      bad |= key < n_keys && !in;
      const long long row = ((long long)(in ? page[i] : 0) << a.pg.page_log) +
                            (key & ((1 << a.pg.page_log) - 1));
      const long long at = (row * Hkv + h) * D + c;
      copy16(s_k + buf * C::k + r * C::ks + c, (const float*)a.pg.k + at, in);
      copy16(s_v + buf * C::v + r * C::vs + c, (const float*)a.pg.v + at, in);
    }
    if (bad) record_error(err, DEV_RANGE);
    asm volatile("cp.async.commit_group;\n" ::);
  };
  if (b0 < b1) issue(b0, 0);

  // this lane's rows g and g + 8 of the warp's 16, and their queries: step 2 u
  // of the contraction takes dimensions 16 u + 4 t and + 1, step 2 u + 1 the next two
  const int w_row = warp / KS * 16 + g;
  float q[2][D / 4];
  int pos[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = r0 + w_row + 8 * e, rr = min(r, n_rows - 1);
    pos[e] = past + rr / G;
    const float* p = (const float*)a.q + (long long)(sq.tok0 + rr / G) * a.q_stride + (h * G + rr % G) * D;
#pragma unroll
    for (int u = 0; u < D / 16; ++u) {
      const float4 x = *reinterpret_cast<const float4*>(p + 16 * u + 4 * t);
      q[e][4 * u] = x.x; q[e][4 * u + 1] = x.y; q[e][4 * u + 2] = x.z; q[e][4 * u + 3] = x.w;
    }
  }
  // O: tile i holds, for column 2 t + e, dimension 4 (2 t + e) + 32 (i / 4) + i % 4
  float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  const float sl2 = a.scale * kLog2e;

  for (int b = b0; b < b1; ++b) {
    const int buf = (b - b0) & 1;
    if (b + 1 < b1) {
      issue(b + 1, buf ^ 1);
      asm volatile("cp.async.wait_group 1;\n" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group 0;\n" ::: "memory");
    }
    __syncthreads();
    const int w_key = warp % KS * 8 * NT;   // the warp's keys of the stage
    const float* kb = s_k + buf * C::k + (w_key + g) * C::ks + 4 * t;
    const float* vb = s_v + buf * C::v + (w_key + 2 * t) * C::vs + 4 * g;
    float s[NT][4], lo[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
      lo[i][0] = lo[i][1] = lo[i][2] = lo[i][3] = 0.f;
    }
#pragma unroll
    for (int u = 0; u < D / 16; ++u) {
      uint32_t ah[2][4], al[2][4], bh[NT][4], bl[NT][4];
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          split(q[e][4 * u + 2 * k], ah[k][e], al[k][e]);
          split(q[e][4 * u + 2 * k + 1], ah[k][2 + e], al[k][2 + e]);
        }
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const float4 x = *reinterpret_cast<const float4*>(kb + i * 8 * C::ks + 16 * u);
        split(x.x, bh[i][0], bl[i][0]);
        split(x.y, bh[i][1], bl[i][1]);
        split(x.z, bh[i][2], bl[i][2]);
        split(x.w, bh[i][3], bl[i][3]);
      }
      // one product of every tile before the next: a dependent MMA waits for
      // its accumulator several times as long as the unit takes for it
      float part[NT][4];
#pragma unroll
      for (int i = 0; i < NT; ++i) part[i][0] = part[i][1] = part[i][2] = part[i][3] = 0.f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int i = 0; i < NT; ++i) mma8(lo[i], al[k], bh[i][2 * k], bh[i][2 * k + 1]);
#pragma unroll
        for (int i = 0; i < NT; ++i) mma8(part[i], ah[k], bh[i][2 * k], bh[i][2 * k + 1]);
#pragma unroll
        for (int i = 0; i < NT; ++i) mma8(lo[i], ah[k], bl[i][2 * k], bl[i][2 * k + 1]);
      }
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[i][e] += part[i][e];
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[i][e] += lo[i][e];
    // columns 2 t, 2 t + 1 of tile i: keys 8 i + 2 t (+ 1); rows g (0, 1), g + 8 (2, 3)
    const int key0 = b * kKeys + w_key + 2 * t;
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (key0 + 8 * i + (e & 1) > pos[e >> 1]) s[i][e] = -INFINITY;
        mx[e >> 1] = fmaxf(mx[e >> 1], s[i][e]);
      }
    float f[2];
    bool any = false;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
      mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
      const bool grown = m[e] == -INFINITY ? mx[e] > m[e] : (mx[e] - m[e]) * sl2 > kGrow;
      f[e] = grown ? tc::ex2((m[e] - mx[e]) * sl2) : 1.f;
      if (grown) m[e] = mx[e];
      any |= grown;
      const float nm = m[e] == -INFINITY ? 0.f : -m[e] * sl2;
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        s[i][2 * e] = tc::ex2(fmaf(s[i][2 * e], sl2, nm));
        s[i][2 * e + 1] = tc::ex2(fmaf(s[i][2 * e + 1], sl2, nm));
        sum += s[i][2 * e] + s[i][2 * e + 1];
      }
      l[e] = l[e] * f[e] + sum;
    }
    if (__any_sync(0xffffffffu, any)) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        o[i][0] *= f[0]; o[i][1] *= f[0]; o[i][2] *= f[1]; o[i][3] *= f[1];
      }
    }
    // step i: index t is key 8 i + 2 t, index t + 4 the key after it
    uint32_t ph[NT][4], pl[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      split(s[i][0], ph[i][0], pl[i][0]);
      split(s[i][2], ph[i][1], pl[i][1]);
      split(s[i][1], ph[i][2], pl[i][2]);
      split(s[i][3], ph[i][3], pl[i][3]);
    }
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      float part[4][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) part[k][0] = part[k][1] = part[k][2] = part[k][3] = 0.f;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const float4 x = *reinterpret_cast<const float4*>(vb + 8 * i * C::vs + 32 * c);
        const float4 y = *reinterpret_cast<const float4*>(vb + (8 * i + 1) * C::vs + 32 * c);
        const float v[2][4] = {{x.x, x.y, x.z, x.w}, {y.x, y.y, y.z, y.w}};
        uint32_t vh[2][4], vl[2][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          split(v[0][k], vh[0][k], vl[0][k]);
          split(v[1][k], vh[1][k], vl[1][k]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) mma8(part[k], pl[i], vh[0][k], vh[1][k]);
#pragma unroll
        for (int k = 0; k < 4; ++k) mma8(part[k], ph[i], vl[0][k], vl[1][k]);
#pragma unroll
        for (int k = 0; k < 4; ++k) mma8(part[k], ph[i], vh[0][k], vh[1][k]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[4 * c + k][e] += part[k][e];
    }
    __syncthreads();   // the buffer may be filled again
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
  }

  bool odd = l[0] != l[0] || l[1] != l[1];
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) odd |= o[i][e] != o[i][e];
  odd = __syncthreads_or(odd);
  if (odd) whole_states<D, KS>(a, smem, table, h, Hkv, G, r0, n_rows, sq.tok0, past, n_keys, b0, b1);

  // states: one of 16 rows for each warp, in the buffers' place
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    if (odd) break;
    float* so = smem + warp * C::state;
    const int r = g + 8 * e;
    if (t == 0) {
      so[16 * C::os + 2 * r] = m[e] == -INFINITY ? m[e] : m[e] * sl2;
      so[16 * C::os + 2 * r + 1] = l[e];
    }
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int i = 0; i < D / 8; i += 4)
        *reinterpret_cast<float4*>(so + r * C::os + 4 * (2 * t + c) + 8 * i) =
            make_float4(o[i][2 * e + c], o[i + 1][2 * e + c], o[i + 2][2 * e + c], o[i + 3][2 * e + c]);
  }
  __syncthreads();
  auto finish = [&](int r, int c, float mm, float ll, float4 x) {
    const int rr = r0 + r;
    const long long tok = sq.tok0 + rr / G;
    const int head = h * G + rr % G;
    const float inv = ll != 0.f ? 1.f / ll : 0.f;
    *reinterpret_cast<float4*>((float*)a.out + tok * a.out_stride + head * D + c) =
        make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
    if (c == 0 && a.lse) a.lse[tok * Hq + head] = lse_of(mm, ll);
  };
  // sums N states of one row, `at` giving (m, l) and four columns of the k-th
  auto meet = [&](int N, auto at, float& mm, float& ll, float4& x) {
    mm = -INFINITY;
    ll = 0.f;
    x = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < N; ++k) {
      float2 ml;
      float4 y;
      at(k, ml, y);
      const float top = fmaxf(mm, ml.x), base = top == -INFINITY ? 0.f : top;
      const float fa = tc::ex2(mm - base), fb = tc::ex2(ml.x - base);
      mm = top;
      ll = ll * fa + ml.y * fb;
      x.x = x.x * fa + y.x * fb; x.y = x.y * fa + y.y * fb;
      x.z = x.z * fa + y.z * fb; x.w = x.w * fa + y.w * fb;
    }
  };
  float* c_st = smem + 4 * C::state;   // KS > 1: the CTA's own states, 16 rows each
  for (int i = tid; i < n_tile * (D / 4); i += kThreads) {
    const int r = i / (D / 4), c = (i % (D / 4)) * 4;
    if (KS == 1 && S > 1) break;       // one state a row already
    float mm, ll;
    float4 x;
    meet(KS, [&](int k, float2& ml, float4& y) {
      const float* so = smem + ((r >> 4) * KS + k) * C::state;
      ml = *reinterpret_cast<const float2*>(so + 16 * C::os + 2 * (r & 15));
      y = *reinterpret_cast<const float4*>(so + (r & 15) * C::os + c);
    }, mm, ll, x);
    if (S == 1) {
      finish(r, c, mm, ll, x);
    } else {
      float* so = c_st + (r >> 4) * C::state;
      *reinterpret_cast<float4*>(so + (r & 15) * C::os + c) = x;
      if (c == 0) *reinterpret_cast<float2*>(so + 16 * C::os + 2 * (r & 15)) = make_float2(mm, ll);
    }
  }
  if (S == 1) return;
  tc::cluster_sync_all();
  for (int i = rank * kThreads + tid; i < n_tile * (D / 4); i += S * kThreads) {
    const int r = i / (D / 4), c = (i % (D / 4)) * 4;
    const uint32_t so = tc::smem_addr((KS == 1 ? smem : c_st) + (r >> 4) * C::state);
    float mm, ll;
    float4 x;
    meet(S, [&](int k, float2& ml, float4& y) {
      ml = tc::ld_cluster_v2(tc::mapa(so + 4u * (16 * C::os + 2 * (r & 15)), k));
      y = tc::ld_cluster_v4(tc::mapa(so + 4u * ((r & 15) * C::os + c), k));
    }, mm, ll, x);
    finish(r, c, mm, ll, x);
  }
  tc::cluster_sync_all();   // no CTA leaves while its state may still be read
}

template <int D, int KS>
cudaError_t launch_f32(const Ctx& c, const AttendArgs& a, cudaStream_t st) {
  constexpr int BM = 64 / KS, kKeys = F32Cfg<D, KS>::keys, most = 16;
  const int tiles = a.max_new ? (a.max_new * c.group + BM - 1) / BM : 1;   // 0: nothing but reports
  // CTAs that have rows, about; keys are split until four of them per SM, with
  // at least four stages each (one stage where the rows are few)
  const long long packed = ((long long)a.n_tokens * c.group + BM - 1) / BM;
  const int seqs = a.batch < a.n_tokens ? a.batch : a.n_tokens;
  const long long busy = (packed > seqs ? packed : seqs) * c.cfg.n_kv_heads;
  int S = 1;
  while (S < most && busy * S < 4 * c.num_sms && (long long)a.max_len >= 2LL * S * (KS == 1 ? 4 : 1) * kKeys) S *= 2;
  const long long grid = (long long)tiles * a.batch * c.cfg.n_kv_heads * S;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  auto k = attend_f32_kernel<D, KS>;
  constexpr int smem = F32Cfg<D, KS>::total;
  static std::atomic<uint64_t> attr_done{0};   // one bit per device
  const uint64_t bit = 1ull << (c.device & 63);
  if (!(attr_done.load() & bit)) {
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    attr_done.fetch_or(bit);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = S;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, a, c.cfg.n_q_heads, c.group, S, tiles, c.err);
}

template <int D>
cudaError_t launch_d(const Ctx& c, const AttendArgs& a, cudaStream_t st) {
  const int rows = a.max_new * c.group;
  return rows <= 16 ? launch_f32<D, 4>(c, a, st)
                    : rows <= 32 ? launch_f32<D, 2>(c, a, st) : launch_f32<D, 1>(c, a, st);
}

}  // namespace

cudaError_t launch_attend(const Ctx& c, const AttendArgs& a, cudaStream_t st) {
  if (c.cfg.dtype == IMEM_BF16)
    return attend_step_fits(c, a) ? launch_attend_step(c, a, st) : launch_attend_tc(c, a, st);
  return c.cfg.head_dim == 128 ? launch_d<128>(c, a, st) : launch_d<64>(c, a, st);
}

}  // namespace imem
