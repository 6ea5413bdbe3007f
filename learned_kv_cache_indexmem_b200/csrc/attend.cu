// attend.cu -- causal attention of new tokens over the paged cache in fp32
// arithmetic: every case of the fp32 model dtype.
//
//   s_ij = scale q_i . k_j,  o_i = sum_{j <= p_i} softmax(s_i)_j v_j
//
// One pass over the keys with the running maximum and sum of the softmax
// (m, l, O rescaled when m grows). A tile's rows are the new tokens of one
// sequence times the G query heads of one KV head (row r: token r / G, head
// r % G), so that K and V are read once for the whole group. The keys of a
// tile are split over a cluster of CTAs when there are too few tiles to fill
// the GPU; their states (m, l, O) meet over distributed shared memory, summed
// in rank order.
#include "common.cuh"
#include "internal.h"
#include "paged.cuh"
#include "tc.cuh"

#include <atomic>
#include <type_traits>

namespace imem {
namespace {

constexpr int kSimtThreads = 256;
constexpr int kSimtKeys = 64;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int D, int BM> struct SimtSmem {
  static constexpr int QS = D + 4, PS = kSimtKeys + 4;
  static constexpr size_t q = 0;
  static constexpr size_t k = q + sizeof(float) * BM * QS;
  static constexpr size_t v = k + sizeof(float) * kSimtKeys * QS;
  static constexpr size_t p = v + sizeof(float) * kSimtKeys * QS;
  static constexpr size_t total = p + sizeof(float) * BM * PS;
};

// BM rows (16 * RM) per tile; thread (ty, tx) of 16 x 16 owns rows ty * RM ..
// and keys tx + 16 j of the scores, dims 4 tx + 64 c of the output.
template <typename T, int D, int BM>
__global__ void __launch_bounds__(kSimtThreads)
attend_simt_kernel(const __grid_constant__ AttendArgs a, int Hq, int G, int S, int tiles,
                   int* __restrict__ err) {
  constexpr int RM = BM / 16, DC = D / 64;
  constexpr int QS = SimtSmem<D, BM>::QS, PS = SimtSmem<D, BM>::PS;
  extern __shared__ float smem[];
  float* s_q = smem;
  float* s_k = smem + SimtSmem<D, BM>::k / 4;
  float* s_v = smem + SimtSmem<D, BM>::v / 4;
  float* s_p = smem + SimtSmem<D, BM>::p / 4;

  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int rank = blockIdx.x % S;
  const int tile = tiles - 1 - blockIdx.x / S;   // the longest first
  const int h = blockIdx.y, seq = blockIdx.z;
  const SeqInfo sq = seq_info(seq, a.batch, a.n_tokens, a.start, a.pg);
  if (tile == 0 && rank == 0 && h == 0 && tid == 0 && (sq.bad || sq.n > a.max_new))
    record_error(err, DEV_RANGE);
  const int n_rows = min(sq.n, a.max_new) * G;
  const int r0 = tile * BM;
  if (r0 >= n_rows) return;   // the whole cluster
  const int past = sq.len - sq.n;   // position of the first new token
  const int n_tile = min(BM, n_rows - r0);
  // keys the tile sees: up to its last row's position
  const int n_keys = max(0, past + (r0 + n_tile - 1) / G + 1);
  const int blocks = (n_keys + kSimtKeys - 1) / kSimtKeys;
  const int per = (blocks + S - 1) / S;
  const int b0 = min(rank * per, blocks), b1 = min(b0 + per, blocks);

  // queries, as they are (the scale goes on the scores)
  for (int i = tid; i < BM * (D / 4); i += kSimtThreads) {
    const int r = i / (D / 4), c = (i % (D / 4)) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < n_tile) {
      const int rr = r0 + r;
      const T* p = (const T*)a.q + (long long)(sq.tok0 + rr / G) * a.q_stride + (h * G + rr % G) * D + c;
      if constexpr (std::is_same<T, float>::value) {
        x = *reinterpret_cast<const float4*>(p);
      } else {
        x = make_float4(Elem<T>::to_f(p[0]), Elem<T>::to_f(p[1]), Elem<T>::to_f(p[2]), Elem<T>::to_f(p[3]));
      }
    }
    *reinterpret_cast<float4*>(s_q + r * QS + c) = x;
  }

  float o[RM][DC][4], m[RM], l[RM];
#pragma unroll
  for (int i = 0; i < RM; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < DC; ++c) o[i][c][0] = o[i][c][1] = o[i][c][2] = o[i][c][3] = 0.f;
  }
  const float sl2 = a.scale * kLog2e;
  const int32_t* table = a.pg.table + (long long)seq * a.pg.max_pages;
  const int Hkv = Hq / G;

  for (int b = b0; b < b1; ++b) {
    const int key0 = b * kSimtKeys;
    __syncthreads();
    for (int i = tid; i < kSimtKeys * (D / 4); i += kSimtThreads) {
      const int r = i / (D / 4), c = (i % (D / 4)) * 4;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
      if (key0 + r < n_keys) {
        const long long row = cache_row(a.pg, table, key0 + r);
        if (row >= 0) {
          const T* kp = (const T*)a.pg.k + (row * Hkv + h) * D + c;
          const T* vp = (const T*)a.pg.v + (row * Hkv + h) * D + c;
          if constexpr (std::is_same<T, float>::value) {
            x = *reinterpret_cast<const float4*>(kp);
            y = *reinterpret_cast<const float4*>(vp);
          } else {
            x = make_float4(Elem<T>::to_f(kp[0]), Elem<T>::to_f(kp[1]), Elem<T>::to_f(kp[2]), Elem<T>::to_f(kp[3]));
            y = make_float4(Elem<T>::to_f(vp[0]), Elem<T>::to_f(vp[1]), Elem<T>::to_f(vp[2]), Elem<T>::to_f(vp[3]));
          }
        } else if (c == 0) {
          record_error(err, DEV_RANGE);
        }
      }
      *reinterpret_cast<float4*>(s_k + r * QS + c) = x;
      *reinterpret_cast<float4*>(s_v + r * QS + c) = y;
    }
    __syncthreads();
    float s[RM][4];
#pragma unroll
    for (int i = 0; i < RM; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
      float4 q[RM], k[4];
#pragma unroll
      for (int i = 0; i < RM; ++i) q[i] = *reinterpret_cast<const float4*>(s_q + (ty * RM + i) * QS + c);
#pragma unroll
      for (int j = 0; j < 4; ++j) k[j] = *reinterpret_cast<const float4*>(s_k + (tx + 16 * j) * QS + c);
#pragma unroll
      for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          s[i][j] += q[i].x * k[j].x + q[i].y * k[j].y + q[i].z * k[j].z + q[i].w * k[j].w;
    }
#pragma unroll
    for (int i = 0; i < RM; ++i) {
      const int rr = r0 + ty * RM + i;
      const int pos = rr < n_rows ? past + rr / G : -1;
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = key0 + tx + 16 * j <= pos ? s[i][j] * sl2 : -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
#pragma unroll
      for (int d = 8; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
      const float mn = fmaxf(m[i], mx);
      const float base = mn == -INFINITY ? 0.f : mn;   // a row with no key yet
      const float f = exp2f(m[i] - base);
      m[i] = mn;
      l[i] *= f;
#pragma unroll
      for (int c = 0; c < DC; ++c) { o[i][c][0] *= f; o[i][c][1] *= f; o[i][c][2] *= f; o[i][c][3] *= f; }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = exp2f(s[i][j] - base);
        l[i] += p;
        s_p[(ty * RM + i) * PS + tx + 16 * j] = p;
      }
    }
    __syncwarp();   // a row's scores stay within one half warp
#pragma unroll 2
    for (int kk = 0; kk < kSimtKeys; kk += 4) {
      float4 p[RM];
#pragma unroll
      for (int i = 0; i < RM; ++i) p[i] = *reinterpret_cast<const float4*>(s_p + (ty * RM + i) * PS + kk);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
#pragma unroll
        for (int c = 0; c < DC; ++c) {
          const float4 v = *reinterpret_cast<const float4*>(s_v + (kk + u) * QS + 4 * tx + 64 * c);
#pragma unroll
          for (int i = 0; i < RM; ++i) {
            const float pu = u == 0 ? p[i].x : u == 1 ? p[i].y : u == 2 ? p[i].z : p[i].w;
            o[i][c][0] += pu * v.x; o[i][c][1] += pu * v.y; o[i][c][2] += pu * v.z; o[i][c][3] += pu * v.w;
          }
        }
      }
    }
  }

#pragma unroll
  for (int i = 0; i < RM; ++i)
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);

  auto write = [&](int r, int c, float x0, float x1, float x2, float x3) {
    const int rr = r0 + r;
    T* p = (T*)a.out + (long long)(sq.tok0 + rr / G) * a.out_stride + (h * G + rr % G) * D + c;
    if constexpr (std::is_same<T, float>::value) {
      *reinterpret_cast<float4*>(p) = make_float4(x0, x1, x2, x3);
    } else {
      p[0] = Elem<T>::from_f(x0); p[1] = Elem<T>::from_f(x1);
      p[2] = Elem<T>::from_f(x2); p[3] = Elem<T>::from_f(x3);
    }
  };
  auto write_lse = [&](int r, float mm, float ll) {
    const int rr = r0 + r;
    if (a.lse)
      a.lse[(long long)(sq.tok0 + rr / G) * Hq + h * G + rr % G] =
          ll != 0.f ? (mm + log2f(ll)) * kLn2 : -INFINITY;   // NaN stays NaN
  };

  if (S == 1) {
#pragma unroll
    for (int i = 0; i < RM; ++i) {
      const int r = ty * RM + i;
      if (r >= n_tile) continue;
      const float inv = l[i] != 0.f ? 1.f / l[i] : 0.f;
#pragma unroll
      for (int c = 0; c < DC; ++c)
        write(r, 4 * tx + 64 * c, o[i][c][0] * inv, o[i][c][1] * inv, o[i][c][2] * inv, o[i][c][3] * inv);
      if (tx == 0) write_lse(r, m[i], l[i]);
    }
    return;
  }
  // states into this CTA's shared memory (over Q and K), then every CTA of the
  // cluster merges its share of the output
  __syncthreads();
  float2* s_ml = reinterpret_cast<float2*>(s_p);
  float* s_o = s_q;   // [BM][D]
#pragma unroll
  for (int i = 0; i < RM; ++i) {
    const int r = ty * RM + i;
    if (tx == 0) s_ml[r] = make_float2(m[i], l[i]);
#pragma unroll
    for (int c = 0; c < DC; ++c)
      *reinterpret_cast<float4*>(s_o + r * D + 4 * tx + 64 * c) = make_float4(o[i][c][0], o[i][c][1], o[i][c][2], o[i][c][3]);
  }
  tc::cluster_sync_all();
  const uint32_t a_ml = tc::smem_addr(s_ml), a_o = tc::smem_addr(s_o);
  for (int i = rank * kSimtThreads + tid; i < n_tile * (D / 4); i += S * kSimtThreads) {
    const int r = i / (D / 4), c = (i % (D / 4)) * 4;
    float mm = -INFINITY, ll = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < S; ++k) {
      const float2 st = tc::ld_cluster_v2(tc::mapa(a_ml + 8u * r, k));
      mm = fmaxf(mm, st.x);
    }
    const float base = mm == -INFINITY ? 0.f : mm;
    for (int k = 0; k < S; ++k) {
      const float2 st = tc::ld_cluster_v2(tc::mapa(a_ml + 8u * r, k));
      const float4 y = tc::ld_cluster_v4(tc::mapa(a_o + 4u * (r * D + c), k));
      const float w = exp2f(st.x - base);
      ll += w * st.y;
      x.x += w * y.x; x.y += w * y.y; x.z += w * y.z; x.w += w * y.w;
    }
    const float inv = ll != 0.f ? 1.f / ll : 0.f;
    write(r, c, x.x * inv, x.y * inv, x.z * inv, x.w * inv);
    if (c == 0) write_lse(r, mm, ll);
  }
  tc::cluster_sync_all();   // no CTA leaves while its state may still be read
}

template <typename T, int D, int BM>
cudaError_t launch_simt(const Ctx& c, const AttendArgs& a, cudaStream_t st) {
  const int rows = a.max_new * c.group;
  const int tiles = (rows + BM - 1) / BM;
  const long long items = (long long)tiles * c.cfg.n_kv_heads * a.batch;
  // split the keys until two CTAs per SM, at least four key blocks each
  int S = 1;
  while (S < 8 && items * S < 2 * c.num_sms && (long long)a.max_len >= 2LL * S * 4 * kSimtKeys) S *= 2;
  auto k = attend_simt_kernel<T, D, BM>;
  constexpr size_t smem = SimtSmem<D, BM>::total;
  static std::atomic<uint64_t> attr_done{0};   // one bit per device
  const uint64_t bit = 1ull << (c.device & 63);
  if (!(attr_done.load() & bit)) {
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    attr_done.fetch_or(bit);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * S), c.cfg.n_kv_heads, a.batch);
  cfg.blockDim = dim3(kSimtThreads, 1, 1);
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

template <typename T, int D>
cudaError_t launch_td(const Ctx& c, const AttendArgs& a, cudaStream_t st) {
  return a.max_new * c.group <= 16 ? launch_simt<T, D, 16>(c, a, st) : launch_simt<T, D, 64>(c, a, st);
}

}  // namespace

cudaError_t launch_attend(const Ctx& c, const AttendArgs& a, cudaStream_t st) {
  if (c.cfg.dtype == IMEM_BF16)
    return attend_step_fits(c, a) ? launch_attend_step(c, a, st) : launch_attend_tc(c, a, st);
  return c.cfg.head_dim == 128 ? launch_td<float, 128>(c, a, st) : launch_td<float, 64>(c, a, st);
}

}  // namespace imem
