// Eviction of cached tokens by their accumulated mass (contract:
// include/dsa_l4.h): rank, select, compact.
//
//   rank     the mass as a ranking score: +inf for the first `sinks` and last
//            `recent` tokens, a NaN as -inf, any other infinity as the largest
//            finite value (so that a protected token is never outranked)
//   select   the exact top-k of the step (ties to the lower position,
//            positions ascending)
//   compact  a warp copies a few kept tokens' rows of every pool
#include <float.h>
#include <math.h>

#include <algorithm>

#include "latent4.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 256;

struct EvictParams {
  dsa_pool_t pools[DSA_EVICT_MAX_POOLS];
  int n_pools;
  const int32_t *seq_lens;
  const int32_t *src_table;
  const int32_t *dst_table;
  int src_max_pages, src_pages, dst_max_pages, dst_pages;
  int max_len, budget, sinks, recent;
  const float *mass;
  int64_t mass_ld;
  float *mass_dst;
  int64_t mass_dst_ld;
  int32_t *new_lens;
  int32_t *lens;  // scratch [num_seqs]: lengths clamped to max_len
  const int32_t *kept;
  int64_t kept_ld;
  float *rank;
  int64_t rank_ld;
  DevStatus *status;
};

__global__ void __launch_bounds__(kThreads) rank_kernel(const EvictParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.y;
  const int n = max(0, min(p.seq_lens[b], p.max_len));
  if (blockIdx.x == 0 && threadIdx.x == 0) p.lens[b] = n;
  for (int s = blockIdx.x * kThreads + threadIdx.x; s < n; s += gridDim.x * kThreads) {
    const float m = p.mass[b * p.mass_ld + s];
    float v = (m != m) ? -INFINITY : fminf(m, FLT_MAX);
    if (s < p.sinks || s >= n - p.recent) v = INFINITY;
    p.rank[b * p.rank_ld + s] = v;
  }
}

// kRows kept tokens per warp: a lane each resolves them, then the warp copies
// their rows pool by pool, flattened over (row, unit), kFlight units per lane in
// flight: four rows of 336 bytes are 84 units, of 256 bytes 64.  Four rows where
// they fill the device, two where they do not (latency).  4 x 131,072 tokens to
// 16,384, 592 bytes each, the whole call: 36.6 us; eight rows and four or six
// units in flight 38.9 and 39.5, two rows 41.0.
constexpr int kFlight = 3;
template <int kRows, typename T>
__device__ __forceinline__ void copy_rows(const dsa_pool_t &q, int src, int dst, int lane) {
  const int n = q.row_bytes / static_cast<int>(sizeof(T));  // units per row
  // t / n = t * inv >> 26, exactly: t < 2^13, and inv n exceeds 2^26 by less than n <= 2^10
  const uint32_t inv = ((1u << 26) + n - 1) / n;
  const T *s = static_cast<const T *>(q.src);
  T *d = static_cast<T *>(q.dst);
  for (int t0 = 0; t0 < kRows * n; t0 += 32 * kFlight) {
    T v[kFlight];
    int64_t at[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const int t = t0 + 32 * u + lane;
      const int r = min(static_cast<int>((static_cast<uint64_t>(t) * inv) >> 26), kRows - 1);
      const int c = t - r * n;
      const int from = __shfl_sync(0xffffffffu, src, r), to = __shfl_sync(0xffffffffu, dst, r);
      at[u] = t < kRows * n && from >= 0 ? static_cast<int64_t>(to) * n + c : -1;
      if (at[u] >= 0) v[u] = s[static_cast<int64_t>(from) * n + c];
    }
#pragma unroll
    for (int u = 0; u < kFlight; ++u)
      if (at[u] >= 0) d[at[u]] = v[u];
  }
}

template <int kRows>
__global__ void __launch_bounds__(kThreads) compact_kernel(const EvictParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.y, lane = lane_id();
  const int n = min(p.lens[b], p.budget);
  // not in rank_kernel: new_lens may be seq_lens, which all its CTAs read
  if (blockIdx.x == 0 && threadIdx.x == 0) p.new_lens[b] = n;
  const int step = gridDim.x * (kThreads / 32) * kRows;
  for (int i0 = (blockIdx.x * (kThreads / 32) + warp_id()) * kRows; i0 < n; i0 += step) {
    const int i = i0 + lane;
    int src = -1, dst = -1;
    if (lane < kRows && i < n) {
      // a selection that timed out (and was reported) may have left anything here
      const int pos = min(max(p.kept[b * p.kept_ld + i], 0), p.lens[b] - 1);
      const int sp = p.src_table[static_cast<int64_t>(b) * p.src_max_pages + pos / kPageSize];
      const int dp = p.dst_table[static_cast<int64_t>(b) * p.dst_max_pages + i / kPageSize];
      if (p.mass_dst) p.mass_dst[b * p.mass_dst_ld + i] = p.mass[b * p.mass_ld + pos];
      if (sp < 0 || sp >= p.src_pages || dp < 0 || dp >= p.dst_pages) {
        report(p.status, kErrBadPage, (kKernEvict << 24) | (i & 0xFFFF));
      } else {
        src = sp * kPageSize + pos % kPageSize;
        dst = dp * kPageSize + i % kPageSize;
      }
    }
    for (int k = 0; k < p.n_pools; ++k) {
      if (p.pools[k].row_bytes % 16 == 0) copy_rows<kRows, uint4>(p.pools[k], src, dst, lane);
      else copy_rows<kRows, uint32_t>(p.pools[k], src, dst, lane);
    }
  }
}

}  // namespace

dsa_status_t launch_evict(const EvictLaunch &a, cudaStream_t stream) {
  EvictParams p;
  for (int i = 0; i < DSA_EVICT_MAX_POOLS; ++i) p.pools[i] = a.pools[i];
  p.n_pools = a.n_pools;
  p.seq_lens = a.cache.seq_lens;
  p.src_table = a.cache.block_table;
  p.dst_table = a.evict.dst_block_table;
  p.src_max_pages = a.cache.max_pages;
  p.src_pages = a.cache.num_pages;
  p.dst_max_pages = a.evict.dst_max_pages;
  p.dst_pages = a.evict.dst_num_pages;
  p.max_len = a.cache.max_seq_len;
  p.budget = a.evict.budget;
  p.sinks = a.evict.sinks;
  p.recent = a.evict.recent;
  p.mass = a.mass;
  p.mass_ld = a.mass_ld;
  p.mass_dst = a.mass_dst;
  p.mass_dst_ld = a.mass_dst_ld;
  p.new_lens = a.new_lens;
  p.lens = a.lens;
  p.kept = a.kept;
  p.kept_ld = a.kept_ld;
  p.rank = a.rank;
  p.rank_ld = a.rank_ld;
  p.status = a.status;
  const unsigned B = static_cast<unsigned>(a.cache.num_seqs);
  const unsigned tiles = static_cast<unsigned>(std::min<int64_t>(256, (a.rank_ld + kThreads - 1) / kThreads));
  if (launch_pdl(rank_kernel, dim3(tiles, B), dim3(kThreads), 0, stream, 1, p) != cudaSuccess)
    return DSA_ERR_CUDA;
  TopkLaunch t;
  t.scores = a.rank;
  t.ld = a.rank_ld;
  t.n_q = a.cache.num_seqs;
  t.valid_len = a.lens;
  t.causal_base = 0;
  t.k = static_cast<int>(a.kept_ld);
  t.idx = a.kept;
  t.max_len = static_cast<int>(a.rank_ld);
  t.status = a.status;
  const dsa_status_t st = launch_topk(t, stream);
  if (st != DSA_OK) return st;
  const int64_t most = std::min<int64_t>(a.evict.budget, a.cache.max_seq_len);
  const bool many = most * B >= static_cast<int64_t>(device_sm_count()) * 128;
  const int64_t per_cta = static_cast<int64_t>(kThreads / 32) * (many ? 4 : 2);
  const unsigned rows = static_cast<unsigned>(
      std::max<int64_t>(1, std::min<int64_t>(2048, (most + per_cta - 1) / per_cta)));
  return launch_pdl(many ? compact_kernel<4> : compact_kernel<2>, dim3(rows, B), dim3(kThreads), 0, stream, 1, p) == cudaSuccess
             ? DSA_OK
             : DSA_ERR_CUDA;
}

}  // namespace dsa
