// Launchers of the 4-bit latent cache, attention-mass and eviction kernels
// (internal to libdsa; the contract is in include/dsa_l4.h).
#pragma once

#include "../../include/dsa_l4.h"
#include "dsa_internal.h"

namespace dsa {

// kernel ids of the status block's event codes, after those of dsa_common.cuh
enum : unsigned int { kKernRead4 = 7u, kKernMla4 = 8u, kKernMass = 9u, kKernEvict = 10u };

// bytes of a stored row of W columns: codes, block scales, exponent, rounded up
__host__ __device__ constexpr int l4_row_bytes(int W) { return (W / 2 + W / 16 + 1 + 15) / 16 * 16; }

// the paged view and the row rules that every kernel here shares
struct PagedRows {
  const int32_t *seq_lens;
  const int32_t *block_table;
  int max_pages, num_pages;
  int causal, q_pos0;
};

struct Append4Launch {
  const uint16_t *k_new;
  const uint16_t *lat_new;
  uint16_t *k_pages;
  uint8_t *lat_pages;
  PagedRows rows;
  int n_q, D_I, W;
  DevStatus *status;
};
dsa_status_t launch_append4(const Append4Launch &a, cudaStream_t stream);

struct Read4Launch {
  const uint8_t *lat_pages;
  PagedRows rows;
  const int32_t *idx;
  uint16_t *out;
  int n_q, k, W;
  DevStatus *status;
};
dsa_status_t launch_read4(const Read4Launch &a, cudaStream_t stream);

struct Mla4Launch {
  const uint16_t *q;
  const uint8_t *latent;
  PagedRows rows;
  const int32_t *idx;
  float *out;
  float *lse;
  int n_q, H, R, P, topk;
  float scale;
  void *scratch;
  size_t scratch_bytes;
  DevStatus *status;
  // 1: q is complete before the kernel preceding this one in the stream started
  // (the whole step), so its tile is written before that kernel has ended
  int early_q = 0;
};
size_t mla4_scratch_bytes(int n_q, int topk, int R);
dsa_status_t launch_mla4(const Mla4Launch &a, cudaStream_t stream);

enum LatentFormat { kLatBf16 = 0, kLatE4m3 = 1, kLatL4 = 2 };
struct MassLaunch {
  LatentFormat format;
  const uint16_t *q;
  const void *latent;
  const float *lat_scale;  // kLatE4m3: one fp32 scale per pool row
  PagedRows rows;
  const int32_t *idx;
  const float *lse;
  const float *mass_in;
  float *mass_out;
  int64_t mass_ld;
  int max_len;  // a sequence's length counts up to this one (<= mass_ld)
  int n_q, num_seqs, H, R, P, topk;
  float scale, decay;
  void *scratch;  // causal chunks: 64-bit sums [q_pos0 + n_q]
  DevStatus *status;
};
size_t mass_scratch_bytes(const dsa_dims_t &d);
dsa_status_t launch_mass(const MassLaunch &a, cudaStream_t stream);

struct EvictLaunch {
  dsa_pool_t pools[DSA_EVICT_MAX_POOLS];
  int n_pools;
  dsa_cache_t cache;
  dsa_evict_t evict;
  const float *mass;
  int64_t mass_ld;
  float *mass_dst;
  int64_t mass_dst_ld;
  int32_t *new_lens;
  int32_t *kept;     // [num_seqs, kept_ld]: kept_ld positions per sequence
  int64_t kept_ld;
  int32_t *lens;     // scratch [num_seqs]: lengths clamped to max_seq_len
  float *rank;       // scratch [num_seqs, rank_ld]
  int64_t rank_ld;
  DevStatus *status;
};
dsa_status_t launch_evict(const EvictLaunch &a, cudaStream_t stream);

}  // namespace dsa
