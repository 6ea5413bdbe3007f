// attend_tc.cu -- causal attention of new tokens over the paged cache, bf16, on
// the tcgen05 tensor cores.
//
//   s_ij = scale q_i . k_j,  o_i = sum_{j <= p_i} softmax(s_i)_j v_j
//
// A CTA owns NQ tiles of 128 query rows of one sequence and KV head (row r:
// new token r / G, head r % G of the group, so K and V are read once for the
// whole group) and walks the keys in tiles of 128:
//   producer warp  TMA, page by page, into a ring of 128-row K and V tiles;
//   MMA warp       S_t = Q_t K^T into TMEM; O_t += P_t V with P_t from TMEM;
//   4 warps per tile  one row per thread: S from TMEM, running maximum, exp2,
//                  P as bf16 back into the columns of S, the row's sum.
// While one tile's softmax runs, the tensor core works on the other tile. The
// MMA warp's loop stays converged and one elected lane issues: its operands are
// then uniform (a branch on the lane cost 11 %: 474 against 426 us for 2048
// tokens at 16384 keys; a warp per query tile 562 us).
//
// MMAs of one thread run in order, so S_t of the next key tile may overwrite
// P_t once O_t += P_t V has been issued before it, and S_t being complete
// means that the product before it is: O_t may then be rescaled without a
// further wait. It is rescaled only when a row's maximum has grown by more
// than a factor of 2^8 since it was last taken: until then the sums stay below
// 2^8 times what they would be, far inside fp32 and bf16.
//
// Keys past a row's position are masked by selection, so nothing stored there
// matters; value rows past the last key that any row sees are zeroed in
// shared memory (0 * NaN would reach O).
//
// P is rounded to bf16 for the product with V, the type the tensor cores take
// beside a bf16 V, as imem_decode does: 2^-8 of each weight at most, which over
// many keys adds about as much to an output as its own rounding (error against
// the exact outputs 0.0020-0.0022 of their size, 0.0017 from that alone). The
// sum that divides is taken before the rounding. Leaving a maximum alone until
// it has grown, and sharing exp2 out between two units (below), are published
// techniques of attention kernels.
//
// Bound by the tensor cores and exp2 for long chunks (8192 new tokens at
// 131072, 32 heads of 128: 14.1-14.5 ms, 1.2 PFLOP/s; four ragged prompts of up to
// 4096: 355 us, 1.07 PFLOP/s, on the same inputs again, 410-419 us, 0.92, on
// others each time; 2048 tokens at 16384 keys, heads of 64: 359 us, 0.72), by HBM
// for a few tokens.
//
// With too few tiles to fill the GPU the keys of a tile are split over a
// cluster; the states (m, l, O) meet over distributed shared memory and are
// summed in rank order.
#include "common.cuh"
#include "internal.h"
#include "paged.cuh"
#include "tc.cuh"

#include <atomic>
#include <mutex>
#include <type_traits>

namespace imem {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kKeys = 128;       // keys per tile
constexpr float kGrow = 8.f;     // log2 growth of a maximum that is left alone

// 2^y for two values y >= -126 (below, and for NaN: 2^-126) on the FMA units: y = n + f with
// n the nearest integer (added and taken off 1.5 * 2^23), 2^f on [-1/2, 1/2]
// by the polynomial of degree 5 with the smallest largest relative error
// (fitted by the exchange algorithm; 2.4e-7 in fp32, ex2.approx has 1.2e-7), n
// added to the exponent. The special-function unit gives 16 results per clock
// and SM, the tensor cores wait for 16384 per tile: sharing them out between
// the two units shortens the softmax.
__device__ __forceinline__ void exp2_fma(uint64_t y, float& e0, float& e1) {
  const uint64_t magic = tc::pack2(12582912.f, 12582912.f);
  const uint64_t nmagic = tc::pack2(-12582912.f, -12582912.f);
  float y0, y1;
  tc::unpack2(y, y0, y1);
  y = tc::pack2(fmaxf(y0, -126.f), fmaxf(y1, -126.f));
  const uint64_t t = tc::add2(y, magic);
  const uint64_t f = tc::fma2(tc::add2(t, nmagic), tc::pack2(-1.f, -1.f), y);
  auto c2 = [](float c) { return tc::pack2(c, c); };
  uint64_t p = tc::fma2(f, c2(0.0013276472454890609f), c2(0.009675540961325169f));
  p = tc::fma2(f, p, c2(0.05550713092088699f));
  p = tc::fma2(f, p, c2(0.24022120237350464f));
  p = tc::fma2(f, p, c2(0.6931469440460205f));
  p = tc::fma2(f, p, c2(1.0000001192092896f));
  float p0, p1, t0, t1;
  tc::unpack2(p, p0, p1);
  tc::unpack2(t, t0, t1);
  e0 = __uint_as_float(__float_as_uint(p0) + (__float_as_uint(t0) << 23));
  e1 = __uint_as_float(__float_as_uint(p1) + (__float_as_uint(t1) << 23));
}
// Of 8 neighbouring pairs, those taken by exp2_fma: with heads of 128 one (none
// or three: 2 % slower), with heads of 64, where the products take half the
// time, two (none: 7 % slower, one or three: 4 %).
template <int D> constexpr int kFmaOf8 = D == 64 ? 2 : 1;

template <int D, int NQ> struct TcCfg {
  static constexpr int threads = NQ * 128 + 128;
  static constexpr int tile = kKeys * D * 2;                   // bytes of 128 rows
  static constexpr int half = kKeys * 128;                     // of 64 columns of them
  static constexpr int stages = D == 128 ? (NQ == 2 ? 5 : 6) : 8;
  static constexpr int ring = NQ * tile;                       // behind Q
  static constexpr int bars = ring + stages * tile;
  static constexpr int total = bars + 256 + 1024;
  static constexpr int o_stride = D + 4;                       // floats, merge buffer
  static constexpr uint32_t tmem_cols = NQ * (128 + D) <= 256 ? 256 : 512;
  static_assert(NQ * 128 * o_stride * 4 + NQ * 128 * 8 <= bars, "merge buffer fits");
  static_assert(total <= 232448, "shared memory of a CTA");
};

// Registers: two query tiles launch with 384 threads x 168; the softmax warps
// hold a row of S (128 values) and take 216, paid for by the other four warps
// (256 x 216 + 128 x 72 = 384 x 168; nobody changes its share again, so the
// softmax warps' request is met as soon as the others have given theirs up).
// One tile's 256 threads need no split.
constexpr int kRegsLaunch = 168, kRegsSoftmax = 216, kRegsOther = 72;
static_assert(256 * kRegsSoftmax + 128 * kRegsOther <= 384 * kRegsLaunch, "register pool");

template <int D, int NQ>
__global__ void __launch_bounds__(NQ * 128 + 128, 1)
attend_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                 const __grid_constant__ CUtensorMap mv, const __grid_constant__ AttendArgs a,
                 int Hq, int Hkv, int G, int S, int tiles, int* __restrict__ err) {
  using C = TcCfg<D, NQ>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sQ = tc::smem_addr(smem), sR = sQ + C::ring, bar = sQ + C::bars;
  const uint32_t q_full = bar, r_full = bar + 8, r_empty = r_full + 8 * C::stages,
                 s_full = r_empty + 8 * C::stages, p_full = s_full + 8 * NQ, o_full = p_full + 16 * NQ;
  __shared__ uint32_t s_tmem;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // linear grid, the longest tiles first, heads fastest (neighbours share
  // nothing but run alike; the tiles of one head meet in L2)
  int idx = blockIdx.x;
  const int rank = idx % S;
  idx /= S;
  const int h = idx % Hkv;
  idx /= Hkv;
  const int seq = idx % a.batch;
  const int tile = tiles - 1 - idx / a.batch;

  if (tid == 0) {
    for (int i = 0; i < C::stages; ++i) {
      tc::mbar_init(r_full + 8 * i, 1);
      tc::mbar_init(r_empty + 8 * i, 1);
    }
    for (int t = 0; t < NQ; ++t) {
      tc::mbar_init(s_full + 8 * t, 1);
      tc::mbar_init(p_full + 16 * t, 4);
      tc::mbar_init(p_full + 16 * t + 8, 4);
      tc::mbar_init(o_full + 8 * t, 1);
    }
    tc::fence_mbar_init();
  }

  const SeqInfo sq = seq_info(seq, a.batch, a.n_tokens, a.start, a.pg);
  if (tile == 0 && rank == 0 && h == 0 && tid == 0 && (sq.bad || sq.n > a.max_new))
    record_error(err, DEV_RANGE);
  const int n_rows = min(sq.n, a.max_new) * G;
  const int r0 = tile * (NQ * 128);
  if (r0 >= n_rows) return;                  // the whole cluster
  const int past = sq.len - sq.n;            // position of the first new token
  // keys that the rows of the CTA see, and their tiles of this rank
  auto keys_of = [&](int row_end) { return max(0, past + (row_end - 1) / G + 1); };
  const int n_keys = keys_of(min(n_rows, r0 + NQ * 128));
  const int all = (n_keys + kKeys - 1) / kKeys;
  const int per = (all + S - 1) / S;
  const int b0 = min(rank * per, all), n = min(b0 + per, all) - b0;
  int cnt[NQ];   // of each query tile
#pragma unroll
  for (int t = 0; t < NQ; ++t) {
    const int lo = r0 + t * 128;
    const int k = lo < n_rows ? keys_of(min(n_rows, lo + 128)) : 0;
    cnt[t] = min(max((k + kKeys - 1) / kKeys - b0, 0), n);
  }

  // the producer's first table entries and the queries' copy, behind the set-up
  const int box = min(1 << a.pg.page_log, kKeys);
  int first = -1;
  if (warp == NQ * 4 + 1 && n > 0 && lane < kKeys / box && b0 * kKeys + lane * box < n_keys)
    first = a.pg.table[(long long)seq * a.pg.max_pages + ((b0 * kKeys + lane * box) >> a.pg.page_log)];
  if (warp == NQ * 4 + 1 && lane == 0) {
    tc::mbar_init(q_full, 1);
    tc::fence_mbar_init();
    if (n > 0) {
      tc::mbar_expect_tx(q_full, NQ * C::tile);
      for (int t = 0; t < NQ; ++t)
        for (int c = 0; c < D / 64; ++c)
          tc::tma_load_3d(sQ + t * C::tile + c * C::half, &mq, q_full, 64 * c, h * G,
                          sq.tok0 + (r0 + t * 128) / G);
    }
  }
  if (warp == NQ * 4) {
    tc::tmem_alloc(tc::smem_addr(&s_tmem), C::tmem_cols);
    tc::tmem_relinquish();
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = s_tmem;

  float m = -INFINITY, l = 0.f;   // softmax threads: this row's state (m: raw scores)
  const int row = r0 + tid;       // softmax threads: warps 0 .. 4 NQ - 1
  const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
  const int my = warp >> 2;       // their query tile

  if (warp >= NQ * 4) {
    if constexpr (NQ == 2) tc::regs_release<kRegsOther>();
    if (warp == NQ * 4 + 1 && n > 0) {
      // ------------------------------------------------------------ producer
      const int page = 1 << a.pg.page_log;
      const int parts = kKeys / box;   // boxes per tile
      const int32_t* table = a.pg.table + (long long)seq * a.pg.max_pages;
      auto needs = [&](int j) {   // this lane has a box of key tile j
        return j < n && lane < parts && (b0 + j) * kKeys + lane * box < n_keys;
      };
      auto page_of = [&](int j) {
        return needs(j) ? table[((b0 + j) * kKeys + lane * box) >> a.pg.page_log] : -1;
      };
      int next = first, issued = 0;
      bool ok = true;
      for (int j = 0; j < n && ok; ++j) {
        const int pid = next;
        next = page_of(j + 1);
        const bool load = pid >= 0 && pid < a.pg.n_pages;
        if (needs(j) && !load) record_error(err, DEV_RANGE);
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, load)) * box * (D * 2);
        const int y = (pid << a.pg.page_log) + (((b0 + j) * kKeys) & (page - 1) & ~(box - 1));
        for (int v = 0; v < 2; ++v) {
          const int i = 2 * j + v, st = i % C::stages;
          if (i >= C::stages && !tc::mbar_wait(r_empty + 8 * st, (i / C::stages - 1) & 1)) {
            record_error(err, DEV_TIMEOUT);
            ok = false;
            break;
          }
          if (lane == 0) tc::mbar_expect_tx(r_full + 8 * st, bytes);
          __syncwarp();
          issued = i + 1;
          if (load) {
            const uint32_t dst = sR + st * C::tile + lane * box * 128;
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
              tc::tma_load_2d(dst + c * C::half, v ? &mv : &mk, r_full + 8 * st, h * D + 64 * c, y);
          }
        }
      }
      // whatever happened, no copy is in flight when the CTA ends
      if (!tc::mbar_wait(q_full, 0)) record_error(err, DEV_TIMEOUT);
      for (int i = max(0, issued - C::stages); i < issued; ++i)
        if (!tc::mbar_wait(r_full + 8 * (i % C::stages), (i / C::stages) & 1)) record_error(err, DEV_TIMEOUT);
    } else if (warp == NQ * 4 && n > 0) {
      // ------------------------------------------------------------ MMA issuer
      constexpr uint32_t IQK = tc::idesc(tc::kFmtBF16, 128, kKeys, false, false);
      constexpr uint32_t IPV = tc::idesc(tc::kFmtBF16, 128, D, false, true);
      auto wait = [&](uint32_t b, int phase) {
        const bool ok = tc::mbar_wait(b, phase & 1);
        if (!ok) record_error(err, DEV_TIMEOUT);
        return ok;
      };
      auto full = [&](int i) { return wait(r_full + 8 * (i % C::stages), i / C::stages); };
      auto release = [&](int i) {
        if (tc::elect_one()) tc::mma_commit(r_empty + 8 * (i % C::stages));
      };
      auto qk = [&](int t, int j) {   // S_t = Q_t K_j^T
        if (tc::elect_one()) {
          // descriptors step by 32 bytes along K within a 64-column half
          uint64_t dq = tc::sdesc_sw128(sQ + t * C::tile, 16, 1024);
          uint64_t dk = tc::sdesc_sw128(sR + ((2 * j) % C::stages) * C::tile, 16, 1024);
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
#pragma unroll
            for (int s = 0; s < 4; ++s)
              tc::mma_f16(tmem + t * 128, dq + 2 * s, dk + 2 * s, IQK, (c | s) > 0);
            dq += C::half >> 4;
            dk += C::half >> 4;
          }
          tc::mma_commit(s_full + 8 * t);
        }
      };
      bool ok = wait(q_full, 0) && full(0);
      if (ok) {
#pragma unroll
        for (int t = 0; t < NQ; ++t)
          if (cnt[t] > 0) qk(t, 0);
        release(0);
      }
      for (int j = 0; j < n && ok; ++j) {
        if (!full(2 * j + 1)) break;
        const uint32_t v = sR + ((2 * j + 1) % C::stages) * C::tile;
        const int live = n_keys - (b0 + j) * kKeys;   // rows of this tile that any row sees
        if (live < kKeys) {
          for (int i = lane; i < (kKeys - live) * (D / 8); i += 32) {
            const int r = live + i / (D / 8), c = i % (D / 8);
            asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};\n" ::"r"(
                             v + (c >> 3) * C::half + r * 128 + (c & 7) * 16), "r"(0u) : "memory");
          }
          tc::fence_proxy_async();
          __syncwarp();
        }
        const bool have_k = j + 1 < n;
        if (have_k && !full(2 * j + 2)) break;
#pragma unroll
        for (int t = 0; t < NQ; ++t) {
          if (j >= cnt[t] || !ok) continue;
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {   // 64 keys each
            const uint64_t dv = tc::sdesc_sw128(v + hf * 8192, C::half, 1024);
            if (!ok || !wait(p_full + 16 * t + 8 * hf, j)) { ok = false; continue; }
            tc::fence_after();
            if (tc::elect_one()) {
#pragma unroll
              for (int s = 0; s < 4; ++s)   // 16 keys: 2 KB of V, 8 columns of P
                tc::mma_f16_ta(tmem + NQ * 128 + t * D, tmem + t * 128 + 32 * hf + s * 8,
                               dv + 128 * s, IPV, (j | hf | s) > 0);
            }
          }
          if (!ok) continue;
          if (j + 1 < cnt[t]) {
            qk(t, j + 1);
          } else if (tc::elect_one()) {
            tc::mma_commit(o_full + 8 * t);
          }
        }
        if (!ok) break;
        release(2 * j + 1);
        if (have_k) release(2 * j + 2);
      }
    }
    // the CTA's end, in step with the softmax warps'
    tc::fence_before();
    __syncthreads();
    if (S > 1) tc::cluster_sync_all();
    tc::fence_after();
    if (warp == NQ * 4) tc::tmem_dealloc(tmem, C::tmem_cols);
    if (S > 1) tc::cluster_sync_all();
    return;
  }

  if constexpr (NQ == 2) tc::regs_take<kRegsSoftmax>();
  const uint32_t tO = tmem + lane_base + NQ * 128 + my * D;
  const float sl2 = a.scale * kLog2e;
  if (n > 0) {
    // ------------------------------------------------------------ softmax
    const uint32_t tS = tmem + lane_base + my * 128;
    const uint64_t scale2 = tc::pack2(sl2, sl2);
    const int pos = past + row / G;            // rows past n_rows: whatever comes, not written
    const int warp_pos = past + (row - lane) / G;
    uint64_t sum = 0;                          // two partial sums
    bool ok = true;
    for (int j = 0; j < cnt[my] && ok; ++j) {
      if (!tc::mbar_wait(s_full + 8 * my, j & 1)) {
        record_error(err, DEV_TIMEOUT);
        ok = false;
        break;
      }
      tc::fence_after();
      uint32_t s[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tc::tmem_ld32_async(tS + 32 * c, s[c]);
      tc::tmem_wait_ld_dep<true>(s[0]);
#pragma unroll
      for (int c = 1; c < 4; ++c) tc::tmem_wait_ld_dep<false>(s[c]);
      const int key0 = (b0 + j) * kKeys;
      const bool edge = key0 + kKeys - 1 > warp_pos;
      if (edge) {
        const int lim = pos - key0;            // columns up to it are seen
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int x = 0; x < 32; ++x)
            if (32 * c + x > lim) s[c][x] = 0xff800000u;
      }
      float mx[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        mx[c] = tc::max_nan(__uint_as_float(s[c][0]), __uint_as_float(s[c][1]));
#pragma unroll
        for (int x = 2; x < 32; x += 2)
          mx[c] = tc::max3_nan(mx[c], __uint_as_float(s[c][x]), __uint_as_float(s[c][x + 1]));
      }
      const float mj = tc::max_nan(tc::max_nan(mx[0], mx[1]), tc::max_nan(mx[2], mx[3]));
      // a NaN score makes mj NaN and counts as grown: the sum and O are NaN from
      // there on, by the factor f and by the special-function unit's columns
      const bool grown = m == -INFINITY ? !(mj <= m) : !((mj - m) * sl2 <= kGrow);
      float f = 1.f;
      if (grown) {
        f = tc::ex2((m - mj) * sl2);
        m = mj;
      }
      if (j > 0 && __any_sync(0xffffffffu, grown)) {
        float lo, hi;
        tc::unpack2(sum, lo, hi);
        sum = tc::pack2(lo * f, hi * f);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tc::tmem_ld32_async(tO + 32 * c, o);
          tc::tmem_wait_ld_dep<true>(o);
#pragma unroll
          for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
          tc::tmem_st32(tO + 32 * c, o);
        }
      }
      const float nm = m == -INFINITY ? 0.f : -m * sl2;
      const uint64_t nm2 = tc::pack2(nm, nm);
      // two halves of 64 keys, each handed to the tensor core as it is done
      auto half = [&](int hf, auto masked) {
        uint32_t p[32];
#pragma unroll
        for (int x = 0; x < 64; x += 2) {
          const uint32_t(&v)[32] = s[2 * hf + (x >> 5)];
          const uint64_t y = tc::fma2(
              tc::pack2(__uint_as_float(v[x & 31]), __uint_as_float(v[(x & 31) + 1])), scale2, nm2);
          float e0, e1;
          // masked scores are -inf: exactly 0 from the special-function unit
          if (!decltype(masked)::value && ((x >> 1) * kFmaOf8<D>) % 8 < kFmaOf8<D>) {
            exp2_fma(y, e0, e1);
          } else {
            tc::unpack2(y, e0, e1);
            e0 = tc::ex2(e0);
            e1 = tc::ex2(e1);
          }
          sum = tc::add2(sum, tc::pack2(e0, e1));
          const __nv_bfloat162 b = __floats2bfloat162_rn(e0, e1);
          p[x >> 1] = *reinterpret_cast<const uint32_t*>(&b);
        }
        tc::tmem_st32(tS + 32 * hf, p);
        tc::tmem_wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(p_full + 8 * (2 * my + hf));
      };
      if (edge) {
        half(0, std::true_type());
        half(1, std::true_type());
      } else {
        half(0, std::false_type());
        half(1, std::false_type());
      }
    }
    float lo, hi;
    tc::unpack2(sum, lo, hi);
    l = lo + hi;
    // what exp2_fma made of scores beside +inf, or of -inf alone, is no sum
    if (m == INFINITY) l = NAN;
    if (m == -INFINITY && l == l) l = 0.f;
    if (cnt[my] > 0 && ok && !tc::mbar_wait(o_full + 8 * my, 0)) record_error(err, DEV_TIMEOUT);
    tc::fence_after();
  }

  // ---------------------------------------------------------------- outputs
  auto out_at = [&](int r) {
    return (__nv_bfloat16*)a.out + (long long)(sq.tok0 + r / G) * a.out_stride + (h * G + r % G) * D;
  };
  auto put_lse = [&](int r, float m2, float ll) {   // m2: maximum of the log2 scores
    if (a.lse)
      a.lse[(long long)(sq.tok0 + r / G) * Hq + h * G + r % G] = lse_of(m2, ll);
  };
  const bool mine = n > 0 && cnt[my] > 0;
  if (S == 1) {
    const float inv = l != 0.f ? 1.f / l : 0.f;
    // whole 32-byte sectors where the rows allow it
    const bool wide = (((uintptr_t)a.out | (uintptr_t)(a.out_stride * 2)) & 31) == 0;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      uint32_t o[32];
      if (mine) {
        tc::tmem_ld32_async(tO + 32 * c, o);
        tc::tmem_wait_ld_dep<true>(o);
      } else {
#pragma unroll
        for (int x = 0; x < 32; ++x) o[x] = 0u;
      }
      if (row < n_rows) {
        __nv_bfloat16* p = out_at(row) + 32 * c;
#pragma unroll
        for (int x = 0; x < 32; x += 16) {
          uint32_t y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(o[x + 2 * e]) * inv,
                                                           __uint_as_float(o[x + 2 * e + 1]) * inv);
            y[e] = *reinterpret_cast<const uint32_t*>(&b);
          }
          if (wide) {
            asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(p + x), "r"(y[0]),
                         "r"(y[1]), "r"(y[2]), "r"(y[3]), "r"(y[4]), "r"(y[5]), "r"(y[6]), "r"(y[7])
                         : "memory");
          } else {
            *reinterpret_cast<uint4*>(p + x) = make_uint4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<uint4*>(p + x + 8) = make_uint4(y[4], y[5], y[6], y[7]);
          }
        }
      }
    }
    if (row < n_rows) put_lse(row, m * sl2, l);
    tc::fence_before();
    __syncthreads();
    return;
  }
  // states into shared memory (every copy and MMA of the CTA is complete: the
  // MMA warp waited for the copies, the softmax warps for the last MMA)
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  float* s_o = reinterpret_cast<float*>(smem);
  float2* s_ml = reinterpret_cast<float2*>(smem + NQ * 128 * C::o_stride * 4);
  s_ml[tid] = make_float2(m == -INFINITY ? m : m * sl2, l);
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    uint32_t o[32];
    if (mine) {
      tc::tmem_ld32_async(tO + 32 * c, o);
      tc::tmem_wait_ld_dep<true>(o);
    } else {
#pragma unroll
      for (int x = 0; x < 32; ++x) o[x] = 0u;
    }
#pragma unroll
    for (int x = 0; x < 32; x += 4)
      *reinterpret_cast<uint4*>(s_o + tid * C::o_stride + 32 * c + x) =
          make_uint4(o[x], o[x + 1], o[x + 2], o[x + 3]);
  }
  tc::fence_before();
  tc::cluster_sync_all();
  const uint32_t a_o = tc::smem_addr(s_o), a_ml = tc::smem_addr(s_ml);
  const int live_rows = min(NQ * 128, n_rows - r0);
  for (int i = rank * (NQ * 128) + tid; i < live_rows * (D / 8); i += S * (NQ * 128)) {
    const int r = i / (D / 8), c = (i % (D / 8)) * 8;
    float mm = -INFINITY, ll = 0.f, f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = 0.f;
    for (int k = 0; k < S; ++k) mm = fmaxf(mm, tc::ld_cluster_v2(tc::mapa(a_ml + 8u * r, k)).x);
    const float base = mm == -INFINITY ? 0.f : mm;
    for (int k = 0; k < S; ++k) {
      const float2 st = tc::ld_cluster_v2(tc::mapa(a_ml + 8u * r, k));
      const float4 x = tc::ld_cluster_v4(tc::mapa(a_o + 4u * (r * C::o_stride + c), k));
      const float4 y = tc::ld_cluster_v4(tc::mapa(a_o + 4u * (r * C::o_stride + c + 4), k));
      const float w = tc::ex2(st.x - base);
      ll += w * st.y;
      f[0] += w * x.x; f[1] += w * x.y; f[2] += w * x.z; f[3] += w * x.w;
      f[4] += w * y.x; f[5] += w * y.y; f[6] += w * y.z; f[7] += w * y.w;
    }
    const float inv = ll != 0.f ? 1.f / ll : 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= inv;
    store8(out_at(r0 + r) + c, f);
    if (c == 0) put_lse(r0 + r, mm, ll);
  }
  tc::cluster_sync_all();   // no CTA leaves while its state may still be read
}

// How many CTAs share a tile's keys, and what that is expected to take (us).
struct Plan {
  int S;
  double us;
};

// Keys are split while the clusters stay one wave (16 clusters of 8 do not all
// fit the GPU's processor groups: 47 against 26 us for eight sequences of 30
// tokens at 7518 keys) and a CTA keeps two key tiles. A CTA takes about 7 us to
// start and end, and per key tile 1.8 us with two query tiles, 1.3 with one.
template <int D, int NQ>
cudaError_t plan(const Ctx& c, const AttendArgs& a, Plan* p) {
  using C = TcCfg<D, NQ>;
  // once per device: attributes, and how many clusters of 1, 2, 4, 8 are resident
  static std::atomic<const int (*)[4]> setup[64];
  static std::mutex setup_mu;
  const int dv = c.device & 63;
  const int(*resident)[4] = setup[dv].load(std::memory_order_acquire);
  if (!resident) {
    std::lock_guard<std::mutex> lock(setup_mu);
    resident = setup[dv].load(std::memory_order_relaxed);
    if (!resident) {
      auto k = attend_tc_kernel<D, NQ>;
      cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::total);
      static int table[64][4];
      cudaLaunchConfig_t cfg = {};
      cfg.blockDim = dim3(C::threads, 1, 1);
      cfg.dynamicSmemBytes = C::total;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      for (int s = 0; s < 4 && e == cudaSuccess; ++s) {
        cfg.gridDim = dim3(1 << s, 1, 1);
        attr[0].val.clusterDim.x = 1 << s;
        e = cudaOccupancyMaxActiveClusters(&table[dv][s], k, &cfg);
      }
      if (e != cudaSuccess) return e;
      resident = &table[dv];
      setup[dv].store(resident, std::memory_order_release);
    }
  }
  // tiles that have rows: about packed tokens over full tiles, one for each
  // sequence with tokens at least
  const long long packed = ((long long)a.n_tokens * c.group + NQ * 128 - 1) / (NQ * 128);
  const int seqs = a.batch < a.n_tokens ? a.batch : a.n_tokens;
  const long long busy = (packed > seqs ? packed : seqs) * c.cfg.n_kv_heads;
  int s = 0;
  while (s < 3 && busy <= (*resident)[s + 1] && (long long)a.max_len >= (4LL << s) * kKeys) ++s;
  const int fit = (*resident)[s] > 0 ? (*resident)[s] : 1;
  const double waves = (double)((busy + fit - 1) / fit);
  const double key_tiles = (a.max_len / kKeys + 1.0) / (1 << s);
  p->S = 1 << s;
  p->us = waves * (7.0 + key_tiles * (NQ == 2 ? 1.8 : 1.3));
  return cudaSuccess;
}

template <int D, int NQ>
cudaError_t launch(const Ctx& c, const AttendArgs& a, int S, cudaStream_t st) {
  using C = TcCfg<D, NQ>;
  const int G = c.group, Hkv = c.cfg.n_kv_heads;
  const int tiles = (a.max_new * G + NQ * 128 - 1) / (NQ * 128);
  const long long grid = (long long)tiles * a.batch * Hkv * S;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  const int box = 1 << (a.pg.page_log < 7 ? a.pg.page_log : 7);
  CUtensorMap mq, mk, mv;
  const uint64_t rows = (uint64_t)a.pg.n_pages << a.pg.page_log;
  if (!make_tmap_tokens(c, &mq, a.q, D, c.cfg.n_q_heads, a.n_tokens, a.q_stride, G, 128 / G) ||
      !make_tmap_bf16(c, &mk, a.pg.k, (uint64_t)Hkv * D, rows, box) ||
      !make_tmap_bf16(c, &mv, a.pg.v, (uint64_t)Hkv * D, rows, box))
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(C::threads, 1, 1);
  cfg.dynamicSmemBytes = C::total;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = S;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attend_tc_kernel<D, NQ>, mq, mk, mv, a, c.cfg.n_q_heads, Hkv, G, S,
                            tiles, c.err);
}

// One or two query tiles per CTA, whichever is expected to be faster: two pass
// over the keys at 0.9 us per tile and query tile, one fills the SMs with half
// the rows (two sequences of 543 tokens at 1302 keys 15.4 against 20.2 us, 512
// tokens at 131072 keys 1435 against 880).
template <int D>
cudaError_t launch_d(const Ctx& c, const AttendArgs& a, cudaStream_t st) {
  Plan one, two;
  cudaError_t e = plan<D, 1>(c, a, &one);
  if (e == cudaSuccess) e = plan<D, 2>(c, a, &two);
  if (e != cudaSuccess) return e;
  return a.max_new * c.group <= 128 || one.us < two.us ? launch<D, 1>(c, a, one.S, st)
                                                       : launch<D, 2>(c, a, two.S, st);
}

}  // namespace

cudaError_t launch_attend_tc(const Ctx& c, const AttendArgs& a, cudaStream_t st) {
  return c.cfg.head_dim == 128 ? launch_d<128>(c, a, st) : launch_d<64>(c, a, st);
}

}  // namespace imem
