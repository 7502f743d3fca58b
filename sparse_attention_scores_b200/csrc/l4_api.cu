// The entry points of include/dsa_l4.h: argument checks on the host, workspace
// layout and launch sequences.
#include <math.h>

#include <algorithm>

#include "l4_internal.h"

namespace dsa {
namespace {

constexpr size_t kStatusBytes = sizeof(DevStatus);
constexpr int kMaxRowBytes = 4096;

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
cudaStream_t as_stream(dsa_stream_t s) {
  return s ? reinterpret_cast<cudaStream_t>(s) : cudaStreamPerThread;
}
DevStatus *status_of(void *ws) { return static_cast<DevStatus *>(ws); }

dsa_status_t check_ws(const void *ws, size_t ws_bytes, size_t need) {
  return (ws == nullptr || !aligned(ws, 256) || ws_bytes < need) ? DSA_ERR_WORKSPACE : DSA_OK;
}

#define DSA_TRY(expr)                        \
  do {                                       \
    const dsa_status_t st__ = (expr);        \
    if (st__ != DSA_OK) return st__;         \
  } while (0)

dsa_status_t check_row(int R, int P) {
  return (R < 64 || R > 512 || R % 64 != 0 || P < 0 || P % 16 != 0 || R + P > 576)
             ? DSA_ERR_UNSUPPORTED
             : DSA_OK;
}

// tokens the longest query row sees, and the step's row stride of scores
int64_t max_keys(const dsa_dims_t &d, const dsa_cache_t &c) {
  return d.causal ? static_cast<int64_t>(d.q_pos0) + d.n_q : static_cast<int64_t>(c.max_seq_len);
}
int64_t scores_ld(const dsa_dims_t &d, const dsa_cache_t &c) {
  return std::max<int64_t>(4, (max_keys(d, c) + 3) & ~static_cast<int64_t>(3));
}

// check_cache, and positions that fit 32 bits up to the block table's last slot
dsa_status_t check_cache_l4(const dsa_cache_t *c, const dsa_dims_t &d) {
  DSA_TRY(check_cache(c, d));
  return c->max_pages > INT32_MAX / kPageSize ? DSA_ERR_UNSUPPORTED : DSA_OK;
}

PagedRows paged(const dsa_cache_t &c, const dsa_dims_t &d) {
  return PagedRows{c.seq_lens, c.block_table, c.max_pages, c.num_pages, d.causal, d.q_pos0};
}

int64_t evict_rank_ld(const dsa_cache_t &c) {
  return std::max<int64_t>(4, (static_cast<int64_t>(c.max_seq_len) + 3) & ~static_cast<int64_t>(3));
}
dsa_status_t check_evict_cache(const dsa_cache_t *c) {
  dsa_dims_t d = {};
  if (c != nullptr) d.n_q = c->num_seqs;
  DSA_TRY(check_cache_l4(c, d));
  return c->num_seqs > 65535 ? DSA_ERR_UNSUPPORTED : DSA_OK;  // grid.y
}

size_t ws_bytes_for(dsa_l4_op_t op, const dsa_dims_t &d, const dsa_cache_t &c) {
  switch (op) {
    case DSA_L4_OP_STATUS:
      return kStatusBytes;
    case DSA_L4_OP_SPARSE_MLA:
      return kStatusBytes + align256(mla4_scratch_bytes(d.n_q, d.topk, d.R));
    case DSA_L4_OP_ATTENTION_FORWARD:
      return kStatusBytes + align256(static_cast<size_t>(d.n_q) * scores_ld(d, c) * 4) +
             align256(static_cast<size_t>(d.n_q) * d.topk * 4) +
             align256(mla4_scratch_bytes(d.n_q, d.topk, d.R));
    case DSA_L4_OP_ATTENTION_MASS:
      return kStatusBytes + align256(mass_scratch_bytes(d));
    case DSA_L4_OP_CACHE_EVICT:  // lengths, ranks, kept positions
      return kStatusBytes + align256(static_cast<size_t>(c.num_seqs) * 4) +
             2 * align256(static_cast<size_t>(c.num_seqs) * evict_rank_ld(c) * 4);
  }
  return 0;
}

dsa_status_t run_mla4(const uint16_t *q, const uint8_t *latent, const dsa_cache_t &c,
                      const int32_t *idx, const dsa_dims_t &d, float *out, float *lse,
                      void *scratch, size_t scratch_bytes, DevStatus *st, cudaStream_t s,
                      int early_q = 0) {
  Mla4Launch a;
  a.q = q;
  a.latent = latent;
  a.rows = paged(c, d);
  a.idx = idx;
  a.out = out;
  a.lse = lse;
  a.n_q = d.n_q;
  a.H = d.H;
  a.R = d.R;
  a.P = d.P;
  a.topk = d.topk;
  a.scale = d.scale;
  a.scratch = scratch;
  a.scratch_bytes = scratch_bytes;
  a.status = st;
  a.early_q = early_q;
  return launch_mla4(a, s);
}

dsa_status_t mla4_entry(const uint16_t *q, const uint8_t *latent, const dsa_cache_t *cache,
                        const int32_t *idx, const dsa_dims_t *dims, float *out, float *lse,
                        void *ws, size_t ws_bytes, dsa_stream_t stream, int want_causal) {
  DSA_TRY(check_dims_common(dims));
  if (dims->causal != want_causal) return DSA_ERR_INVALID_ARG;
  DSA_TRY(check_mla_dims(*dims));
  DSA_TRY(check_cache_l4(cache, *dims));
  if (q == nullptr || latent == nullptr || idx == nullptr || out == nullptr || lse == nullptr)
    return DSA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(latent, 16) || !aligned(idx, 4) || !aligned(out, 4) ||
      !aligned(lse, 4))
    return DSA_ERR_INVALID_ARG;
  DSA_TRY(check_ws(ws, ws_bytes, ws_bytes_for(DSA_L4_OP_SPARSE_MLA, *dims, *cache)));
  if (dims->n_q == 0) return DSA_OK;
  return run_mla4(q, latent, *cache, idx, *dims, out, lse, static_cast<uint8_t *>(ws) + kStatusBytes,
                  ws_bytes - kStatusBytes, status_of(ws), as_stream(stream));
}

dsa_status_t mass_entry(LatentFormat format, const uint16_t *q, const void *latent,
                        const float *lat_scale, const dsa_cache_t *cache, const int32_t *idx,
                        const float *lse, const dsa_dims_t *dims, float decay, const float *mass_in,
                        float *mass_out, int64_t mass_ld, void *ws, size_t ws_bytes,
                        dsa_stream_t stream) {
  DSA_TRY(check_dims_common(dims));
  DSA_TRY(check_mla_dims(*dims));
  DSA_TRY(check_cache_l4(cache, *dims));
  if (q == nullptr || latent == nullptr || idx == nullptr || lse == nullptr || mass_out == nullptr ||
      (format == kLatE4m3 && lat_scale == nullptr))
    return DSA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(latent, 16) || !aligned(idx, 4) || !aligned(lse, 4) ||
      !aligned(mass_out, 4) || (mass_in && !aligned(mass_in, 4)) ||
      (lat_scale && !aligned(lat_scale, 4)))
    return DSA_ERR_INVALID_ARG;
  if (!isfinite(decay) || decay < 0.f) return DSA_ERR_INVALID_ARG;
  if (mass_ld < 1 || mass_ld < max_keys(*dims, *cache) || mass_ld > INT32_MAX)
    return DSA_ERR_INVALID_ARG;
  DSA_TRY(check_ws(ws, ws_bytes, ws_bytes_for(DSA_L4_OP_ATTENTION_MASS, *dims, *cache)));
  if (dims->n_q == 0) return DSA_OK;
  MassLaunch a;
  a.format = format;
  a.q = q;
  a.latent = latent;
  a.lat_scale = lat_scale;
  a.rows = paged(*cache, *dims);
  a.idx = idx;
  a.lse = lse;
  a.mass_in = mass_in;
  a.mass_out = mass_out;
  a.mass_ld = mass_ld;
  a.max_len = static_cast<int>(max_keys(*dims, *cache));
  a.n_q = dims->n_q;
  a.num_seqs = cache->num_seqs;
  a.H = dims->H;
  a.R = dims->R;
  a.P = dims->P;
  a.topk = dims->topk;
  a.scale = dims->scale;
  a.decay = decay;
  a.scratch = static_cast<uint8_t *>(ws) + kStatusBytes;
  a.status = status_of(ws);
  return launch_mass(a, as_stream(stream));
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" {

size_t dsa_l4_row_bytes(int32_t R, int32_t P) {
  return check_row(R, P) == DSA_OK ? static_cast<size_t>(l4_row_bytes(R + P)) : 0;
}

size_t dsa_l4_workspace_bytes(dsa_l4_op_t op, const dsa_dims_t *dims, const dsa_cache_t *cache) {
  if (op == DSA_L4_OP_CACHE_EVICT)
    return check_evict_cache(cache) == DSA_OK ? ws_bytes_for(op, dsa_dims_t{}, *cache) : 0;
  if (check_dims_common(dims) != DSA_OK) return 0;
  if (op == DSA_L4_OP_STATUS) return kStatusBytes;
  if (check_mla_dims(*dims) != DSA_OK) return 0;
  if (op == DSA_L4_OP_ATTENTION_FORWARD && check_cache_l4(cache, *dims) != DSA_OK) return 0;
  return ws_bytes_for(op, *dims, cache ? *cache : dsa_cache_t{});
}

dsa_status_t dsa_cache_append_l4(const uint16_t *k_idx_new, const uint16_t *latent_new,
                                 uint16_t *k_idx_pages, uint8_t *latent4_pages,
                                 const dsa_cache_t *cache, const dsa_dims_t *dims, void *ws,
                                 size_t ws_bytes, dsa_stream_t stream) {
  DSA_TRY(check_dims_common(dims));
  const dsa_dims_t &d = *dims;
  if (d.D_I != 32 && d.D_I != 64 && d.D_I != 128) return DSA_ERR_UNSUPPORTED;
  DSA_TRY(check_row(d.R, d.P));
  DSA_TRY(check_cache_l4(cache, d));
  if (k_idx_new == nullptr || latent_new == nullptr || k_idx_pages == nullptr ||
      latent4_pages == nullptr)
    return DSA_ERR_INVALID_ARG;
  if (!aligned(k_idx_new, 16) || !aligned(latent_new, 16) || !aligned(k_idx_pages, 16) ||
      !aligned(latent4_pages, 16))
    return DSA_ERR_INVALID_ARG;
  DSA_TRY(check_ws(ws, ws_bytes, kStatusBytes));
  if (d.n_q == 0) return DSA_OK;
  Append4Launch a;
  a.k_new = k_idx_new;
  a.lat_new = latent_new;
  a.k_pages = k_idx_pages;
  a.lat_pages = latent4_pages;
  a.rows = paged(*cache, d);
  a.n_q = d.n_q;
  a.D_I = d.D_I;
  a.W = d.R + d.P;
  a.status = status_of(ws);
  return launch_append4(a, as_stream(stream));
}

dsa_status_t dsa_cache_read_l4(const uint8_t *latent4_pages, const dsa_cache_t *cache,
                               const int32_t *idx, const dsa_dims_t *dims, uint16_t *rows,
                               void *ws, size_t ws_bytes, dsa_stream_t stream) {
  DSA_TRY(check_dims_common(dims));
  const dsa_dims_t &d = *dims;
  DSA_TRY(check_row(d.R, d.P));
  if (d.topk < 1) return DSA_ERR_INVALID_ARG;
  DSA_TRY(check_cache_l4(cache, d));
  if (latent4_pages == nullptr || idx == nullptr || rows == nullptr) return DSA_ERR_INVALID_ARG;
  if (!aligned(latent4_pages, 16) || !aligned(idx, 4) || !aligned(rows, 16))
    return DSA_ERR_INVALID_ARG;
  DSA_TRY(check_ws(ws, ws_bytes, kStatusBytes));
  if (d.n_q == 0) return DSA_OK;
  Read4Launch a;
  a.lat_pages = latent4_pages;
  a.rows = paged(*cache, d);
  a.idx = idx;
  a.out = rows;
  a.n_q = d.n_q;
  a.k = d.topk;
  a.W = d.R + d.P;
  a.status = status_of(ws);
  return launch_read4(a, as_stream(stream));
}

dsa_status_t dsa_sparse_mla_decode_l4(const uint16_t *q, const uint8_t *latent4_pages,
                                      const dsa_cache_t *cache, const int32_t *idx,
                                      const dsa_dims_t *dims, float *out, float *lse, void *ws,
                                      size_t ws_bytes, dsa_stream_t stream) {
  return mla4_entry(q, latent4_pages, cache, idx, dims, out, lse, ws, ws_bytes, stream, 0);
}

dsa_status_t dsa_sparse_mla_prefill_l4(const uint16_t *q, const uint8_t *latent4_pages,
                                       const dsa_cache_t *cache, const int32_t *idx,
                                       const dsa_dims_t *dims, float *out, float *lse, void *ws,
                                       size_t ws_bytes, dsa_stream_t stream) {
  return mla4_entry(q, latent4_pages, cache, idx, dims, out, lse, ws, ws_bytes, stream, 1);
}

dsa_status_t dsa_attention_forward_l4(const uint16_t *q_idx, const float *w,
                                      const uint16_t *k_idx_pages, const uint16_t *q,
                                      const uint8_t *latent4_pages, const dsa_cache_t *cache,
                                      const dsa_dims_t *dims, int32_t *idx_out, float *out,
                                      float *lse, void *ws, size_t ws_bytes, dsa_stream_t stream) {
  DSA_TRY(check_dims_common(dims));
  DSA_TRY(check_mla_dims(*dims));
  DSA_TRY(check_cache_l4(cache, *dims));
  if (q == nullptr || latent4_pages == nullptr || out == nullptr || lse == nullptr)
    return DSA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(latent4_pages, 16) || !aligned(out, 4) || !aligned(lse, 4) ||
      (idx_out && !aligned(idx_out, 4)))
    return DSA_ERR_INVALID_ARG;
  const dsa_dims_t &d = *dims;
  const dsa_cache_t &c = *cache;
  DSA_TRY(check_ws(ws, ws_bytes, ws_bytes_for(DSA_L4_OP_ATTENTION_FORWARD, d, c)));
  const int64_t ld = scores_ld(d, c);
  uint8_t *at = static_cast<uint8_t *>(ws) + kStatusBytes;
  float *scores = reinterpret_cast<float *>(at);
  at += align256(static_cast<size_t>(d.n_q) * ld * 4);
  int32_t *idx = idx_out ? idx_out : reinterpret_cast<int32_t *>(at);
  at += align256(static_cast<size_t>(d.n_q) * d.topk * 4);
  // the first two steps through their own entry points, which check the rest
  // (indexer dims, q_idx, w, keys) before anything is launched; an empty batch
  // (n_q = 0) is checked by the indexer too, and has no rows to rank
  DSA_TRY(dsa_indexer_scores(q_idx, w, k_idx_pages, cache, dims, scores, ld, ws, ws_bytes, stream));
  if (d.n_q == 0) return DSA_OK;
  DSA_TRY(dsa_topk(scores, ld, d.n_q, d.causal ? nullptr : c.seq_lens, d.q_pos0, d.topk, idx, ws,
                   ws_bytes, stream));
  return run_mla4(q, latent4_pages, c, idx, d, out, lse, at,
                  ws_bytes - static_cast<size_t>(at - static_cast<uint8_t *>(ws)), status_of(ws),
                  as_stream(stream), /*early_q=*/1);
}

dsa_status_t dsa_attention_mass(const uint16_t *q, const uint16_t *latent_pages,
                                const dsa_cache_t *cache, const int32_t *idx, const float *lse,
                                const dsa_dims_t *dims, float decay, const float *mass_in,
                                float *mass_out, int64_t mass_ld, void *ws, size_t ws_bytes,
                                dsa_stream_t stream) {
  return mass_entry(kLatBf16, q, latent_pages, nullptr, cache, idx, lse, dims, decay, mass_in,
                    mass_out, mass_ld, ws, ws_bytes, stream);
}

dsa_status_t dsa_attention_mass_l8(const uint16_t *q, const uint8_t *latent8_pages,
                                   const float *latent_scale, const dsa_cache_t *cache,
                                   const int32_t *idx, const float *lse, const dsa_dims_t *dims,
                                   float decay, const float *mass_in, float *mass_out,
                                   int64_t mass_ld, void *ws, size_t ws_bytes,
                                   dsa_stream_t stream) {
  return mass_entry(kLatE4m3, q, latent8_pages, latent_scale, cache, idx, lse, dims, decay, mass_in,
                    mass_out, mass_ld, ws, ws_bytes, stream);
}

dsa_status_t dsa_attention_mass_l4(const uint16_t *q, const uint8_t *latent4_pages,
                                   const dsa_cache_t *cache, const int32_t *idx, const float *lse,
                                   const dsa_dims_t *dims, float decay, const float *mass_in,
                                   float *mass_out, int64_t mass_ld, void *ws, size_t ws_bytes,
                                   dsa_stream_t stream) {
  return mass_entry(kLatL4, q, latent4_pages, nullptr, cache, idx, lse, dims, decay, mass_in,
                    mass_out, mass_ld, ws, ws_bytes, stream);
}

dsa_status_t dsa_cache_evict(const dsa_pool_t *pools, int32_t n_pools, const dsa_cache_t *cache,
                             const dsa_evict_t *evict, const float *mass, int64_t mass_ld,
                             float *mass_dst, int64_t mass_dst_ld, int32_t *new_lens,
                             int32_t *kept, void *ws, size_t ws_bytes, dsa_stream_t stream) {
  DSA_TRY(check_evict_cache(cache));
  if (evict == nullptr || mass == nullptr || new_lens == nullptr) return DSA_ERR_INVALID_ARG;
  if (n_pools < 0 || n_pools > DSA_EVICT_MAX_POOLS || (n_pools > 0 && pools == nullptr))
    return DSA_ERR_INVALID_ARG;
  const dsa_evict_t &e = *evict;
  if (e.budget < 1 || e.sinks < 0 || e.recent < 0 ||
      static_cast<int64_t>(e.sinks) + e.recent > e.budget)
    return DSA_ERR_INVALID_ARG;
  const int64_t most = std::min<int64_t>(e.budget, cache->max_seq_len);
  if (e.dst_block_table == nullptr || !aligned(e.dst_block_table, 4) || e.dst_max_pages < 1 ||
      e.dst_num_pages < 1 || static_cast<int64_t>(e.dst_max_pages) * kPageSize < most)
    return DSA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(e.dst_num_pages) * kPageSize > INT32_MAX) return DSA_ERR_UNSUPPORTED;
  if (!aligned(mass, 4) || !aligned(new_lens, 4) || (mass_dst && !aligned(mass_dst, 4)) ||
      (kept && !aligned(kept, 4)))
    return DSA_ERR_INVALID_ARG;
  if (mass_dst == mass) return DSA_ERR_INVALID_ARG;  // moved by warps in any order
  if (mass_ld < cache->max_seq_len || (mass_dst && mass_dst_ld < most)) return DSA_ERR_INVALID_ARG;
  EvictLaunch a = {};
  for (int i = 0; i < n_pools; ++i) {
    const dsa_pool_t &q = pools[i];
    if (q.src == nullptr || q.dst == nullptr || q.row_bytes < 4 || q.row_bytes % 4 != 0)
      return DSA_ERR_INVALID_ARG;
    if (q.row_bytes > kMaxRowBytes) return DSA_ERR_UNSUPPORTED;
    const uintptr_t al = q.row_bytes % 16 == 0 ? 16 : 4;
    if (!aligned(q.src, al) || !aligned(q.dst, al)) return DSA_ERR_INVALID_ARG;
    a.pools[i] = q;
  }
  DSA_TRY(check_ws(ws, ws_bytes, ws_bytes_for(DSA_L4_OP_CACHE_EVICT, dsa_dims_t{}, *cache)));
  a.n_pools = n_pools;
  a.cache = *cache;
  a.evict = e;
  a.mass = mass;
  a.mass_ld = mass_ld;
  a.mass_dst = mass_dst;
  a.mass_dst_ld = mass_dst_ld;
  a.new_lens = new_lens;
  a.rank_ld = evict_rank_ld(*cache);
  uint8_t *at = static_cast<uint8_t *>(ws) + kStatusBytes;
  a.lens = reinterpret_cast<int32_t *>(at);
  at += align256(static_cast<size_t>(cache->num_seqs) * 4);
  a.rank = reinterpret_cast<float *>(at);
  at += align256(static_cast<size_t>(cache->num_seqs) * a.rank_ld * 4);
  // without `kept` the positions stay in the workspace, as many as can be kept
  a.kept = kept ? kept : reinterpret_cast<int32_t *>(at);
  a.kept_ld = kept ? e.budget : std::max<int64_t>(1, most);
  a.status = status_of(ws);
  return launch_evict(a, as_stream(stream));
}

}  // extern "C"
