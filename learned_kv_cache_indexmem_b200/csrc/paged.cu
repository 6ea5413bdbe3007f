// paged.cu -- rows of the paged cache at given positions, copied to contiguous
// arrays: the retained tokens into the decode cache, the evicted ones for the
// memory update.
//
// Bound by HBM: K and V rows (Hkv * d elements each) are read and written
// once. A group of lanes copies one token's K and V row; each lane has up to
// eight 16-byte loads in flight, and the group's index and table lookups are
// the only dependent reads before them. 117,965 rows of 2 + 2 KB: 149 us,
// 6.5 TB/s (the copy rate); 4 x 1024 rows: 5 us.
#include "common.cuh"
#include "internal.h"
#include "paged.cuh"

#include <type_traits>

namespace imem {
namespace {

constexpr int kGatherThreads = 256;

// LPR lanes per row, vecs 16-byte vectors per row.
template <int LPR>
__global__ void __launch_bounds__(kGatherThreads)
gather_paged_kernel(const __grid_constant__ PagedView pg, int batch, int n,
                    const int32_t* __restrict__ idx, int idx_stride, int vecs,
                    uint4* __restrict__ K, uint4* __restrict__ V, int cap, int* __restrict__ err) {
  const int lane = threadIdx.x % LPR;
  const long long r = (long long)blockIdx.x * (kGatherThreads / LPR) + threadIdx.x / LPR;
  if (r >= (long long)batch * n) return;
  const int s = (int)(r / n), i = (int)(r - (long long)s * n);
  const int pos = idx ? idx[(long long)s * idx_stride + i] : i;
  const int len = pg.len[s];
  const long long room = min((long long)pg.max_pages << pg.page_log, 1LL << 30);
  const bool bad = len < 0 || len > room;   // as seq_info
  if (bad && i == 0 && lane == 0) record_error(err, DEV_RANGE);
  if (pos < 0 || pos >= len || pos >= room) {
    if (lane == 0 && idx) record_error(err, DEV_RANGE);
    return;
  }
  const long long row = cache_row(pg, pg.table + (long long)s * pg.max_pages, pos);
  if (row < 0) {
    if (lane == 0) record_error(err, DEV_RANGE);
    return;
  }
  const uint4* ks = (const uint4*)pg.k + row * vecs;
  const uint4* vs = (const uint4*)pg.v + row * vecs;
  uint4* kd = K + ((long long)s * cap + i) * vecs;
  uint4* vd = V + ((long long)s * cap + i) * vecs;
  for (int b = lane; b < vecs; b += 4 * LPR) {
    uint4 x[4], y[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (b + u * LPR < vecs) { x[u] = __ldcs(ks + b + u * LPR); y[u] = __ldcs(vs + b + u * LPR); }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (b + u * LPR < vecs) { kd[b + u * LPR] = x[u]; vd[b + u * LPR] = y[u]; }
  }
}

}  // namespace

cudaError_t launch_gather_paged(const Ctx& c, int batch, int n, const int32_t* idx, int idx_stride,
                                const PagedView& pg, void* K, void* V, int cap, cudaStream_t st) {
  const int esize = c.cfg.dtype == IMEM_BF16 ? 2 : 4;
  const int vecs = c.cfg.n_kv_heads * c.cfg.head_dim * esize / 16;   // >= 8
  const long long rows = (long long)batch * n;
  auto run = [&](auto lpr) {
    constexpr int LPR = decltype(lpr)::value;
    const long long grid = (rows + kGatherThreads / LPR - 1) / (kGatherThreads / LPR);
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    gather_paged_kernel<LPR><<<(unsigned)grid, kGatherThreads, 0, st>>>(
        pg, batch, n, idx, idx_stride, vecs, (uint4*)K, (uint4*)V, cap, c.err);
    return cudaGetLastError();
  };
  // as many lanes as a row has vectors, a warp at most
  if (vecs < 16) return run(std::integral_constant<int, 8>());
  if (vecs < 32) return run(std::integral_constant<int, 16>());
  return run(std::integral_constant<int, 32>());
}

}  // namespace imem
