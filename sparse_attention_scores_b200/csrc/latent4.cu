// 4-bit latent cache: quantising append and exact read-back (the row format is
// in include/dsa_l4.h).
//
// Append, for a new row x of W columns:
//   e    = least exponent with max|x| <= 2688 * 2^e
//   s[b] = E4M3(max|x_b| / (6 * 2^e))     per block b of 16 columns
//   v    = e2m1(x / (s[b] * 2^e))
// Both divisions are IEEE fp32 ones.  x has 8 significant bits and every
// rounding boundary of E4M3 and e2m1 at most 5, so a quotient that is not a
// boundary differs from it by far more than an fp32 rounding: the stored codes
// are those of the exact quotients.
//
// One warp per row, one block of 16 columns per lane (36 blocks at W = 576, so
// up to two per lane): 32 bytes in, 8 + 1 bytes out per block.  Both kernels
// move each byte once; they are bound by the copy bandwidth at many rows and
// by launch latency at few.
#include <cuda_bf16.h>

#include "latent4.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 128;
constexpr int kRowsPerCta = kThreads / 32;
constexpr int kMaxBlocks = 2;  // blocks per lane: W <= 576 -> 36 blocks over 32 lanes

struct Append4Params {
  const uint4 *k_new;
  const uint4 *lat_new;
  uint4 *k_pages;
  uint8_t *lat_pages;
  PagedRows rows;
  int n_q, kw, W;  // kw: 16-byte pieces of one key row
  DevStatus *status;
};

__device__ __forceinline__ float2 bf16x2_to_f32(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}

__global__ void __launch_bounds__(kThreads) append4_kernel(const Append4Params p) {
  // the new rows, the block table and seq_lens may come from earlier work
  griddep_wait();
  griddep_launch_dependents();
  const int r = blockIdx.x * kRowsPerCta + warp_id(), lane = lane_id();
  if (r >= p.n_q) return;
  const int seq = p.rows.causal ? 0 : r;
  const int pos = p.rows.causal ? p.rows.q_pos0 + r : p.rows.seq_lens[r] - 1;
  if (pos < 0 || pos >= p.rows.max_pages * kPageSize) {
    if (lane == 0) report(p.status, kErrBadIndex, (kKernAppend << 24) | (r & 0xFFFF));
    return;
  }
  const int page =
      p.rows.block_table[static_cast<int64_t>(seq) * p.rows.max_pages + pos / kPageSize];
  if (page < 0 || page >= p.rows.num_pages) {
    if (lane == 0) report(p.status, kErrBadPage, (kKernAppend << 24) | (r & 0xFFFF));
    return;
  }
  const int64_t slot = static_cast<int64_t>(page) * kPageSize + pos % kPageSize;
  const uint4 *ks = p.k_new + static_cast<int64_t>(r) * p.kw;
  for (int i = lane; i < p.kw; i += 32) p.k_pages[slot * p.kw + i] = ks[i];

  const int nb = p.W / kL4Block;
  const uint4 *src = p.lat_new + static_cast<int64_t>(r) * (p.W / 8);
  uint32_t x[kMaxBlocks][8];  // bf16 pairs
  float bmax[kMaxBlocks];
#pragma unroll
  for (int i = 0; i < kMaxBlocks; ++i) {
    const int b = lane + 32 * i;
    bmax[i] = 0.f;
    if (b < nb) {
      const uint4 lo = src[2 * b], hi = src[2 * b + 1];
      x[i][0] = lo.x; x[i][1] = lo.y; x[i][2] = lo.z; x[i][3] = lo.w;
      x[i][4] = hi.x; x[i][5] = hi.y; x[i][6] = hi.z; x[i][7] = hi.w;
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const float2 v = bf16x2_to_f32(x[i][t]);
        bmax[i] = fmaxf(bmax[i], fmaxf(fabsf(v.x), fabsf(v.y)));
      }
    }
  }
  float amax = fmaxf(bmax[0], bmax[1]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const int e = l4_row_exponent(amax);
  const float inv = pow2i(-e);  // exact: |e| <= 60
  uint8_t *dst = p.lat_pages + slot * l4_row_bytes(p.W);
#pragma unroll
  for (int i = 0; i < kMaxBlocks; ++i) {
    const int b = lane + 32 * i;
    if (b >= nb) break;
    const uint32_t code = f32_to_e4m3(bmax[i] * inv / 6.f);
    const float s = __low2float(e4m3_to_half2(code));
    uint32_t out[2] = {0u, 0u};
    if (s > 0.f) {
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const float2 v = bf16x2_to_f32(x[i][t]);
        out[t >> 2] |= f32x2_to_e2m1(v.x * inv / s, v.y * inv / s) << (8 * (t & 3));
      }
    }
    *reinterpret_cast<uint2 *>(dst + 8 * b) = make_uint2(out[0], out[1]);
    dst[p.W / 2 + b] = static_cast<uint8_t>(code);
  }
  const int used = p.W / 2 + nb;
  for (int i = used + lane; i < l4_row_bytes(p.W); i += 32)
    dst[i] = (i == used) ? static_cast<uint8_t>(e + 127) : static_cast<uint8_t>(0);
}

struct Read4Params {
  const uint8_t *lat_pages;
  PagedRows rows;
  const int32_t *idx;
  uint4 *out;
  int64_t total;  // n_q * k
  int k, W;
  DevStatus *status;
};

__global__ void __launch_bounds__(kThreads) read4_kernel(const Read4Params p) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t g = static_cast<int64_t>(blockIdx.x) * kRowsPerCta + warp_id();
  const int lane = lane_id();
  if (g >= p.total) return;
  const int r = static_cast<int>(g / p.k), j = static_cast<int>(g % p.k);
  const int limit = l4_limit(p.rows, l4_row_len(p.rows, r));
  int row = -1;
  if (lane == 0) row = l4_pool_row(p.rows, r, p.idx[g], limit, p.status, kKernRead4, j);
  row = __shfl_sync(0xffffffffu, row, 0);
  uint4 *dst = p.out + g * (p.W / 8);
  if (row < 0) {
    for (int i = lane; i < p.W / 8; i += 32) dst[i] = make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  const int nb = p.W / kL4Block;
  const uint8_t *src = p.lat_pages + static_cast<int64_t>(row) * l4_row_bytes(p.W);
  const float t = pow2i(l4_exponent(src[p.W / 2 + nb]));
  for (int b = lane; b < nb; b += 32) {
    const uint2 c = *reinterpret_cast<const uint2 *>(src + 8 * b);
    const __half2 s = e4m3_to_half2(src[p.W / 2 + b]);
    uint32_t o[8], h[4];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      e2m1x8_to_f16x2(half ? c.y : c.x, h);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = __half22float2(__hmul2(as_half2(h[i]), s));  // exact: 6 bits
        const __nv_bfloat162 w = __floats2bfloat162_rn(v.x * t, v.y * t);
        o[4 * half + i] = *reinterpret_cast<const uint32_t *>(&w);
      }
    }
    dst[2 * b] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[2 * b + 1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

}  // namespace

dsa_status_t launch_append4(const Append4Launch &a, cudaStream_t stream) {
  Append4Params p;
  p.k_new = reinterpret_cast<const uint4 *>(a.k_new);
  p.lat_new = reinterpret_cast<const uint4 *>(a.lat_new);
  p.k_pages = reinterpret_cast<uint4 *>(a.k_pages);
  p.lat_pages = a.lat_pages;
  p.rows = a.rows;
  p.n_q = a.n_q;
  p.kw = a.D_I * 2 / 16;
  p.W = a.W;
  p.status = a.status;
  const unsigned grid = static_cast<unsigned>((a.n_q + kRowsPerCta - 1) / kRowsPerCta);
  return launch_pdl(append4_kernel, dim3(grid), dim3(kThreads), 0, stream, 1, p) == cudaSuccess
             ? DSA_OK
             : DSA_ERR_CUDA;
}

dsa_status_t launch_read4(const Read4Launch &a, cudaStream_t stream) {
  Read4Params p;
  p.lat_pages = a.lat_pages;
  p.rows = a.rows;
  p.idx = a.idx;
  p.out = reinterpret_cast<uint4 *>(a.out);
  p.total = static_cast<int64_t>(a.n_q) * a.k;
  p.k = a.k;
  p.W = a.W;
  p.status = a.status;
  const int64_t grid = (p.total + kRowsPerCta - 1) / kRowsPerCta;
  if (grid > INT32_MAX) return DSA_ERR_UNSUPPORTED;
  return launch_pdl(read4_kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, stream, 1,
                    p) == cudaSuccess
             ? DSA_OK
             : DSA_ERR_CUDA;
}

}  // namespace dsa
