// attend_step.cu -- causal attention of a few new tokens per sequence over the
// paged cache, bf16: at most 24 query rows (new tokens x heads of the group)
// per KV head, so decode steps and short drafts.
//
// Bound by HBM: K and V are read once and 4 flops per element and row follow,
// far below the machine's balance; tiles of 128 rows on tcgen05 would be
// empty. Cache rows sit on M of the warp-level MMA, the query rows on N (8
// columns each): S = K q^T, then O^T += V^T P with V^T read by transposing
// ldmatrix and P turned from accumulator to operand by movmatrix, so nothing
// but O, m and l stays in registers between tiles.
//
// A CTA streams its share of a sequence's keys in stages of 64 through a ring
// that one producer warp fills by TMA, page by page. Two pairs of warps take
// the stages in turn, each warp 32 keys of its pair's with a softmax state of
// its own: two independent tiles per warp hide the MMAs' latency (one tile of
// 16 keys of every stage per warp: 1.3 us a stage with 20 rows), and no
// block barrier is in the loop. 96 KB of ring, two CTAs per SM, so that one's
// start and end hide behind the other's stream. The CTAs of a sequence and KV
// head form a cluster; their warps' states meet over distributed shared memory
// at the end.
//
// P is rounded to bf16 for the product with V, as in attend_tc.cu.
//
// One token of 64 sequences of up to 32768 keys (6.5 GB): 916 us, 7.1 TB/s; of
// one sequence of 4096 keys: 8 us; 5 tokens of four sequences of up to 16384
// keys in pages of 16: 48 us, 4.4 TB/s (the longest sequence's CTAs last).
#include "common.cuh"
#include "internal.h"
#include "paged.cuh"
#include "tc.cuh"

#include <atomic>
#include <mutex>

namespace imem {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kRows = 64;                // keys per stage
constexpr int kWarps = 4;                // consumers
constexpr int kThreads = kWarps * 32 + 32;
constexpr float kGrow = 8.f;             // log2 growth of a maximum that is left alone

template <int D, int NT> struct StepCfg {
  static constexpr int tile = kRows * D * 2;           // K or V of a stage
  static constexpr int half = kRows * 128;             // 64 columns of it
  static constexpr int stages = D == 128 ? 3 : 6;
  static constexpr int bars = stages * 2 * tile;
  static constexpr int o_stride = D + 4;
  static constexpr int part = NT * 8 * o_stride * 4 + NT * 8 * 8;   // one warp's state
  // three column tiles leave no registers for q: its fragments are read from
  // shared memory (rows 16 bytes apart in banks) for every 16 keys
  static constexpr bool q_smem = NT == 3;
  static constexpr int q_row = D * 2 + 16, q = bars + 128;
  static constexpr int total = q + (q_smem ? NT * 8 * q_row : 0) + 1024;
  static_assert((kWarps + 1) * part <= bars, "the states take the ring's place");
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, 2)
attend_step_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                   const __grid_constant__ AttendArgs a, int Hq, int Hkv, int G, int S,
                   int* __restrict__ err) {
  using C = StepCfg<D, NT>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sR = tc::smem_addr(smem), full = sR + C::bars, empty = full + 8 * C::stages;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int rank = blockIdx.x % S;
  const int h = (blockIdx.x / S) % Hkv, seq = blockIdx.x / S / Hkv;

  const SeqInfo sq = seq_info(seq, a.batch, a.n_tokens, a.start, a.pg);
  if (rank == 0 && h == 0 && tid == 0 && (sq.bad || sq.n > a.max_new)) record_error(err, DEV_RANGE);
  const int n_rows = min(sq.n, a.max_new) * G;   // at most 8 NT (host)
  if (n_rows == 0) return;                       // the whole cluster
  const int past = sq.len - sq.n;                // position of the first new token
  const int n_keys = max(0, past + (n_rows - 1) / G + 1);
  const int all = (n_keys + kRows - 1) / kRows;
  const int per = (all + S - 1) / S;
  const int b0 = min(rank * per, all), n = min(b0 + per, all) - b0;

  if (tid == 0) {
    for (int i = 0; i < C::stages; ++i) {
      tc::mbar_init(full + 8 * i, 1);
      tc::mbar_init(empty + 8 * i, kWarps);
    }
    tc::fence_mbar_init();
  }
  __syncthreads();

  float o[NT][D / 16][4], m[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m[nt][0] = m[nt][1] = -INFINITY;
    l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
  }

  if (warp == kWarps) {
    // -------------------------------------------------------------- producer
    const int page = 1 << a.pg.page_log;
    const int box = min(page, kRows), parts = kRows / box;
    const int32_t* table = a.pg.table + (long long)seq * a.pg.max_pages;
    // the table entries of 32 boxes at a time, one per lane: a stage's boxes
    // then cost a shuffle instead of a load's latency
    const int boxes = (n * kRows + box - 1) / box;
    int pids = -1, issued = 0;
    for (int j = 0; j < n; ++j) {
      const int first = j * parts;
      if ((first & 31) == 0) {
        const int i = first + lane, key = b0 * kRows + i * box;
        pids = i < boxes && key < n_keys ? table[key >> a.pg.page_log] : -1;
      }
      const int pid = __shfl_sync(0xffffffffu, pids, (first + (lane < parts ? lane : 0)) & 31);
      const bool load = lane < parts && pid >= 0 && pid < a.pg.n_pages;
      if (lane < parts && (b0 + j) * kRows + lane * box < n_keys && !load) record_error(err, DEV_RANGE);
      const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, load)) * box * (D * 4);
      const int st = j % C::stages;
      if (j >= C::stages && !tc::mbar_wait(empty + 8 * st, (j / C::stages - 1) & 1)) {
        record_error(err, DEV_TIMEOUT);
        break;
      }
      if (lane == 0) tc::mbar_expect_tx(full + 8 * st, bytes);
      __syncwarp();
      issued = j + 1;
      if (load) {
        const int y = (pid << a.pg.page_log) + (((b0 + j) * kRows) & (page - 1) & ~(box - 1));
        const uint32_t dst = sR + st * 2 * C::tile + lane * box * 128;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          tc::tma_load_2d(dst + c * C::half, &mk, full + 8 * st, h * D + 64 * c, y);
          tc::tma_load_2d(dst + C::tile + c * C::half, &mv, full + 8 * st, h * D + 64 * c, y);
        }
      }
    }
    // whatever happened, no copy is in flight when the ring is given up
    for (int j = max(0, issued - C::stages); j < issued; ++j)
      if (!tc::mbar_wait(full + 8 * (j % C::stages), (j / C::stages) & 1)) record_error(err, DEV_TIMEOUT);
  } else {
    // -------------------------------------------------------------- consumers
    const float sl2 = a.scale * kLog2e;
    // q as B fragments: row 8 nt + g, dims 16 s + 2 t and + 8
    constexpr int QR = C::q_smem ? 1 : NT;
    uint32_t q0[QR][D / 16], q1[QR][D / 16];
    if constexpr (C::q_smem) {
      for (int i = tid; i < NT * 8 * (D / 8); i += kWarps * 32) {
        const int r = i / (D / 8), c = i % (D / 8);
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (r < n_rows)
          x = *reinterpret_cast<const uint4*>((const __nv_bfloat16*)a.q +
                                              (long long)(sq.tok0 + r / G) * a.q_stride +
                                              (h * G + r % G) * D + c * 8);
        *reinterpret_cast<uint4*>(smem + C::q + r * C::q_row + c * 16) = x;
      }
      asm volatile("bar.sync 1, %0;\n" ::"n"(kWarps * 32) : "memory");
    }
#pragma unroll
    for (int nt = 0; nt < QR; ++nt) {
      if constexpr (C::q_smem) break;
      const int r = 8 * nt + g;
      const bool on = r < n_rows;
      const uint32_t* p = (const uint32_t*)((const __nv_bfloat16*)a.q +
                                            (long long)(sq.tok0 + (on ? r / G : 0)) * a.q_stride +
                                            (h * G + (on ? r % G : 0)) * D);
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        q0[nt][s] = on ? p[8 * s + t] : 0u;
        q1[nt][s] = on ? p[8 * s + 4 + t] : 0u;
      }
    }
    // last key that this lane's two rows of each column tile see
    int pos[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) pos[nt][e] = past + min(8 * nt + 2 * t + e, n_rows - 1) / G;

    const int w0 = (warp & 1) * 32;                        // the warp's keys of a stage
    const int kr = w0 + (lane & 15);                       // ldmatrix row of K
    const int vr = w0 + (lane & 7) + (lane >> 4) * 8;      // of V
    for (int j = 0; j < n; ++j) {
      const int st = j % C::stages;
      const uint32_t kt = sR + st * 2 * C::tile, vt = kt + C::tile;
      // every warp sees every phase of a stage's barriers: one that left out
      // the other pair's would take the phase before it for the next one
      if (!tc::mbar_wait(full + 8 * st, (j / C::stages) & 1)) {
        record_error(err, DEV_TIMEOUT);
        break;
      }
      if ((j & 1) != warp >> 1) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(empty + 8 * st);
        continue;
      }
      const int key0 = (b0 + j) * kRows + w0;
      if (key0 + 32 > n_keys) {
        // value rows that no row sees: whatever is there must not reach O
        for (int i = lane; i < 32 * (D / 8); i += 32) {
          const int r = w0 + i / (D / 8), c = i % (D / 8);
          if (key0 + i / (D / 8) >= n_keys)
            asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};\n" ::"r"(
                             vt + (c >> 3) * C::half + r * 128 + (c & 7) * 16), "r"(0u) : "memory");
        }
        __syncwarp();
      }
      // scores of two tiles of 16 keys: keys g and g + 8 of a tile, rows 2 t
      // and 2 t + 1; two chains of products each
      float s[2][NT][4], s2[2][NT][4];
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[x][nt][e] = s2[x][nt][e] = 0.f;
#pragma unroll
      for (int k = 0; k < D / 16; k += 2) {
        uint32_t af[2][2][4], qb[NT][4];
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int c = 2 * (k + u) + (lane >> 4);
            ldsm4(kt + (c >> 3) * C::half + (kr + 16 * x) * 128 + (((c & 7) ^ (kr & 7)) << 4), af[x][u]);
          }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if constexpr (C::q_smem) {   // chunks 2 k .. 2 k + 3 of rows 8 nt ..
            ldsm4(sR + C::q + (8 * nt + (lane & 7)) * C::q_row + (2 * k + (lane >> 3)) * 16, qb[nt]);
          } else {
            qb[nt][0] = q0[nt][k]; qb[nt][1] = q1[nt][k];
            qb[nt][2] = q0[nt][k + 1]; qb[nt][3] = q1[nt][k + 1];
          }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16(s[x][nt], af[x][0], qb[nt][0], qb[nt][1]);
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16(NT == 3 ? s[x][nt] : s2[x][nt], af[x][1], qb[nt][2], qb[nt][3]);
      }
      uint32_t p[2][NT][2];
      float f[NT][2];
      bool any = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float mx[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int key = key0 + 16 * x + g;
            float &a0 = s[x][nt][e], &a1 = s[x][nt][2 + e];
            if (NT != 3) { a0 += s2[x][nt][e]; a1 += s2[x][nt][2 + e]; }
            a0 = key <= pos[nt][e] ? a0 : -INFINITY;
            a1 = key + 8 <= pos[nt][e] ? a1 : -INFINITY;
          }
          mx[e] = fmaxf(fmaxf(s[0][nt][e], s[0][nt][2 + e]), fmaxf(s[1][nt][e], s[1][nt][2 + e]));
        }
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], x));
          mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], x));
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bool grown = m[nt][e] == -INFINITY ? mx[e] > m[nt][e] : (mx[e] - m[nt][e]) * sl2 > kGrow;
          f[nt][e] = grown ? tc::ex2((m[nt][e] - mx[e]) * sl2) : 1.f;
          if (grown) m[nt][e] = mx[e];
          any |= grown;
          const float nm = m[nt][e] == -INFINITY ? 0.f : -m[nt][e] * sl2;
          float sum = 0.f;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            s[x][nt][e] = tc::ex2(fmaf(s[x][nt][e], sl2, nm));
            s[x][nt][2 + e] = tc::ex2(fmaf(s[x][nt][2 + e], sl2, nm));
            sum += s[x][nt][e] + s[x][nt][2 + e];
          }
          l[nt][e] = l[nt][e] * f[nt][e] + sum;
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const __nv_bfloat162 a0 = __floats2bfloat162_rn(s[x][nt][0], s[x][nt][1]);
          const __nv_bfloat162 a1 = __floats2bfloat162_rn(s[x][nt][2], s[x][nt][3]);
          p[x][nt][0] = transpose8(*reinterpret_cast<const uint32_t*>(&a0));
          p[x][nt][1] = transpose8(*reinterpret_cast<const uint32_t*>(&a1));
        }
      }
      if (__any_sync(0xffffffffu, any)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            o[nt][i][0] *= f[nt][0]; o[nt][i][1] *= f[nt][1];
            o[nt][i][2] *= f[nt][0]; o[nt][i][3] *= f[nt][1];
          }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const int c = 2 * i + ((lane >> 3) & 1);
          uint32_t af[4];
          ldsm4_t(vt + (c >> 3) * C::half + (vr + 16 * x) * 128 + (((c & 7) ^ (vr & 7)) << 4), af);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16(o[nt][i], af, p[x][nt][0], p[x][nt][1]);
        }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(empty + 8 * st);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], x);
  }

  // the warps' states take the ring's place (every stage has been consumed)
  __syncthreads();
  float* s_st = reinterpret_cast<float*>(smem);   // per warp: O rows, then (m, l)
  const float sl2 = a.scale * kLog2e;
  if (warp < kWarps) {
    float* so = s_st + warp * (C::part / 4);
    float2* ml = reinterpret_cast<float2*>(so + NT * 8 * C::o_stride);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * nt + 2 * t + e;
        if (g == 0) ml[r] = make_float2(m[nt][e] == -INFINITY ? m[nt][e] : m[nt][e] * sl2, l[nt][e]);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          so[r * C::o_stride + 16 * i + g] = o[nt][i][e];
          so[r * C::o_stride + 16 * i + 8 + g] = o[nt][i][2 + e];
        }
      }
    }
  }
  __syncthreads();

  auto finish = [&](int r, int c, float mm, float ll, float x0, float x1, float x2, float x3) {
    const float inv = ll != 0.f ? 1.f / ll : 0.f;
    const long long tok = sq.tok0 + r / G;
    const int head = h * G + r % G;
    const __nv_bfloat162 y0 = __floats2bfloat162_rn(x0 * inv, x1 * inv);
    const __nv_bfloat162 y1 = __floats2bfloat162_rn(x2 * inv, x3 * inv);
    *reinterpret_cast<uint2*>((__nv_bfloat16*)a.out + tok * a.out_stride + head * D + c) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&y0), *reinterpret_cast<const uint32_t*>(&y1));
    if (c == 0 && a.lse) a.lse[tok * Hq + head] = lse_of(mm, ll);
  };
  // the CTA's state: its warps' meet here
  const int items = n_rows * (D / 4);
  float* c_o = s_st + kWarps * (C::part / 4);
  float2* c_ml = reinterpret_cast<float2*>(c_o + NT * 8 * C::o_stride);
  for (int i = tid; i < items; i += kThreads) {
    const int r = i / (D / 4), c = (i % (D / 4)) * 4;
    float2 ml[kWarps];
    float4 y[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float* so = s_st + w * (C::part / 4);
      ml[w] = reinterpret_cast<const float2*>(so + NT * 8 * C::o_stride)[r];
      y[w] = *reinterpret_cast<const float4*>(so + r * C::o_stride + c);
    }
    const float mm = fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x));
    const float base = mm == -INFINITY ? 0.f : mm;
    float ll = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = tc::ex2(ml[w].x - base);
      ll += f * ml[w].y;
      x.x += f * y[w].x; x.y += f * y[w].y; x.z += f * y[w].z; x.w += f * y[w].w;
    }
    if (S == 1) {
      finish(r, c, mm, ll, x.x, x.y, x.z, x.w);
    } else {
      *reinterpret_cast<float4*>(c_o + r * C::o_stride + c) = x;
      if (c == 0) c_ml[r] = make_float2(mm, ll);
    }
  }
  if (S == 1) return;
  tc::cluster_sync_all();
  // the cluster's: 16 lanes per item, one for each CTA's state, so that all the
  // remote reads of an item are in flight at once
  const uint32_t a_o = tc::smem_addr(c_o), a_ml = tc::smem_addr(c_ml);
  constexpr int kGroups = kThreads / 16;
  const int k = lane & 15;
  for (int i0 = rank * kGroups; i0 < items; i0 += S * kGroups) {
    const int i = i0 + (tid >> 4);
    const int r = min(i, items - 1) / (D / 4), c = (min(i, items - 1) % (D / 4)) * 4;
    float2 ml = make_float2(-INFINITY, 0.f);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (k < S) {
      ml = tc::ld_cluster_v2(tc::mapa(a_ml + 8u * r, k));
      x = tc::ld_cluster_v4(tc::mapa(a_o + 4u * (r * C::o_stride + c), k));
    }
    float mm = ml.x;
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, d));
    const float f = tc::ex2(ml.x - (mm == -INFINITY ? 0.f : mm));
    float v[5] = {f * ml.y, f * x.x, f * x.y, f * x.z, f * x.w};
#pragma unroll
    for (int d = 8; d > 0; d >>= 1)
#pragma unroll
      for (int e = 0; e < 5; ++e) v[e] += __shfl_xor_sync(0xffffffffu, v[e], d);
    if (k == 0 && i < items) finish(r, c, mm, v[0], v[1], v[2], v[3], v[4]);
  }
  tc::cluster_sync_all();   // no CTA leaves while its state may still be read
}

// CTAs per sequence and KV head (a cluster). Where the units fit one wave, as
// many as keep it one wave (clusters must fit the GPU's processor groups, so
// the driver is asked how many of each size are resident: 32 clusters of 9 do
// not all fit 148 SMs at two CTAs each, and a second wave doubled the time of
// four sequences of 16384 keys), two stages per CTA at least. Else several
// waves, so that ragged lengths even out, 1024 keys per CTA at least.
int step_splits(const Ctx& c, const AttendArgs& a, const int (&resident)[17]) {
  const int seqs = a.batch < a.n_tokens ? a.batch : a.n_tokens;   // sequences with new tokens, at most
  const long long units = (long long)seqs * c.cfg.n_kv_heads;
  if (units <= resident[2]) {
    const int most = (a.max_len + 2 * kRows - 1) / (2 * kRows);
    for (int S = most < 16 ? most : 16; S > 1; --S)
      if (resident[S] >= units) return S;
    return 1;
  }
  long long S = (4LL * resident[1] + units - 1) / units;
  if (S > a.max_len / 1024) S = a.max_len / 1024;
  return S < 1 ? 1 : S > 8 ? 8 : (int)S;
}

template <int D, int NT>
cudaError_t launch(const Ctx& c, const AttendArgs& a, cudaStream_t st) {
  using C = StepCfg<D, NT>;
  const int Hkv = c.cfg.n_kv_heads;
  auto k = attend_step_kernel<D, NT>;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::total;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // once per device: attributes, and how many clusters of each size are resident
  static std::atomic<const int (*)[17]> setup[64];
  static std::mutex setup_mu;
  const int dv = c.device & 63;
  const int(*resident)[17] = setup[dv].load(std::memory_order_acquire);
  if (!resident) {
    std::lock_guard<std::mutex> lock(setup_mu);
    resident = setup[dv].load(std::memory_order_relaxed);
    if (!resident) {
      cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::total);
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      static int table[64][17];
      for (int s = 1; s <= 16 && e == cudaSuccess; ++s) {
        cfg.gridDim = dim3(s, 1, 1);
        attr[0].val.clusterDim.x = s;
        e = cudaOccupancyMaxActiveClusters(&table[dv][s], k, &cfg);
      }
      if (e != cudaSuccess) return e;
      resident = &table[dv];
      setup[dv].store(resident, std::memory_order_release);
    }
  }
  const int S = step_splits(c, a, *resident);
  const long long grid = (long long)a.batch * Hkv * S;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  const int box = 1 << (a.pg.page_log < 6 ? a.pg.page_log : 6);
  CUtensorMap mk, mv;
  const uint64_t rows = (uint64_t)a.pg.n_pages << a.pg.page_log;
  if (!make_tmap_bf16(c, &mk, a.pg.k, (uint64_t)Hkv * D, rows, box) ||
      !make_tmap_bf16(c, &mv, a.pg.v, (uint64_t)Hkv * D, rows, box))
    return cudaErrorInvalidValue;
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.stream = st;
  attr[0].val.clusterDim.x = S;
  return cudaLaunchKernelEx(&cfg, k, mk, mv, a, c.cfg.n_q_heads, Hkv, c.group, S, c.err);
}

template <int D>
cudaError_t launch_d(const Ctx& c, const AttendArgs& a, cudaStream_t st) {
  const int rows = a.max_new * c.group;
  if (rows <= 8) return launch<D, 1>(c, a, st);
  if (rows <= 16) return launch<D, 2>(c, a, st);
  return launch<D, 3>(c, a, st);
}

}  // namespace

bool attend_step_fits(const Ctx& c, const AttendArgs& a) { return a.max_new * c.group <= 24; }

cudaError_t launch_attend_step(const Ctx& c, const AttendArgs& a, cudaStream_t st) {
  return c.cfg.head_dim == 128 ? launch_d<128>(c, a, st) : launch_d<64>(c, a, st);
}

}  // namespace imem
