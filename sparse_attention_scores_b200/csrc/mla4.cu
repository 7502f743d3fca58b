// Sparse MLA over a 4-bit latent cache (row format and contract:
// include/dsa_l4.h).
//
//   z[h, j]   = scale * q[h, :] . L[idx_j, :],   L = 2^e * s * v
//   out[h, :] = sum_j softmax_j(z[h, :]) * L[idx_j, 0:R],   lse[h] = log sum_j exp z[h, j]
//
// One CTA of eight warps per (query row, eight heads), one warp per head:
// chunks of kKeys selected rows are decoded into shared memory as fp16 (s * v,
// exact), the warp forms its logits by dot products over its lanes, and keeps
// a running maximum and sum; lane l accumulates the output columns l, l + 32,
// ... in fp32 registers.  Everything is fp32 on CUDA cores.
#include <math.h>

#include <algorithm>

#include "latent4.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 256;
constexpr int kHeadsPerCta = kThreads / 32;
constexpr int kKeys = 32;
constexpr int kMaxPairs = 9;  // column pairs per lane: 576 / 64

struct Mla4Params {
  const uint16_t *q;
  const uint8_t *latent;
  PagedRows rows;
  const int32_t *idx;
  float *out;
  float *lse;
  int H, R, W, topk;
  float scale;
  DevStatus *status;
};

__global__ void __launch_bounds__(kThreads) mla4_simple_kernel(const Mla4Params p) {
  __shared__ __half2 tile[kKeys][288];
  __shared__ float two_e[kKeys];
  __shared__ int rowi[kKeys];
  griddep_wait();
  griddep_launch_dependents();
  const int r = blockIdx.x, warp = warp_id(), lane = lane_id(), tid = threadIdx.x;
  const int h = blockIdx.y * kHeadsPerCta + warp;
  const int W = p.W, pairs = W / 2, nb = W / kL4Block;
  const int len = l4_row_len(p.rows, r), limit = l4_limit(p.rows, len);
  const int nsel = max(0, min(p.topk, len));
  float2 q[kMaxPairs], acc[kMaxPairs];
#pragma unroll
  for (int i = 0; i < kMaxPairs; ++i) {
    const int c = lane + 32 * i;
    q[i] = acc[i] = make_float2(0.f, 0.f);
    if (c < pairs && h < p.H) {
      const uint32_t v = reinterpret_cast<const uint32_t *>(
          p.q + (static_cast<int64_t>(r) * p.H + h) * W)[c];
      q[i] = make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
    }
  }
  float m = -INFINITY, l = 0.f;
  for (int j0 = 0; j0 < nsel; j0 += kKeys) {
    __syncthreads();
    if (tid < kKeys) {
      const int j = j0 + tid;
      const int pos = j < nsel ? p.idx[static_cast<int64_t>(r) * p.topk + j] : -1;
      const int row = l4_pool_row(p.rows, r, pos, limit, blockIdx.y == 0 ? p.status : nullptr,
                                  kKernMla4, j);
      rowi[tid] = row;
      two_e[tid] = row < 0 ? 0.f
                           : pow2i(l4_exponent(p.latent[static_cast<int64_t>(row) * l4_row_bytes(W) +
                                                        W / 2 + nb]));
    }
    __syncthreads();
    for (int u = tid; u < kKeys * nb; u += kThreads) {
      const int k = u / nb, b = u % nb;
      uint32_t hv[4];
      if (rowi[k] < 0) continue;
      const uint8_t *src = p.latent + static_cast<int64_t>(rowi[k]) * l4_row_bytes(W);
      const uint2 c = *reinterpret_cast<const uint2 *>(src + 8 * b);
      const __half2 s = e4m3_to_half2(src[W / 2 + b]);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        e2m1x8_to_f16x2(half ? c.y : c.x, hv);
#pragma unroll
        for (int i = 0; i < 4; ++i) tile[k][8 * b + 4 * half + i] = __hmul2(as_half2(hv[i]), s);
      }
    }
    __syncthreads();
    for (int k = 0; k < kKeys; ++k) {
      if (rowi[k] < 0) continue;  // the same for every thread
      float2 v[kMaxPairs];
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < kMaxPairs; ++i) {
        const int c = lane + 32 * i;
        v[i] = c < pairs ? __half22float2(tile[k][c]) : make_float2(0.f, 0.f);
        dot += q[i].x * v[i].x + q[i].y * v[i].y;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      const float z = dot * two_e[k] * p.scale;
      const float mn = fmaxf(m, z), a = expf(m - mn), w = expf(z - mn);
      m = mn;
      l = l * a + w;
      const float wt = w * two_e[k];
#pragma unroll
      for (int i = 0; i < kMaxPairs; ++i) {
        acc[i].x = acc[i].x * a + wt * v[i].x;
        acc[i].y = acc[i].y * a + wt * v[i].y;
      }
    }
  }
  if (h >= p.H) return;
  const float inv = l > 0.f ? 1.f / l : 0.f;
  float *out = p.out + (static_cast<int64_t>(r) * p.H + h) * p.R;
#pragma unroll
  for (int i = 0; i < kMaxPairs; ++i) {
    const int c = 2 * (lane + 32 * i);
    if (c < p.R) {
      out[c] = acc[i].x * inv;
      out[c + 1] = acc[i].y * inv;
    }
  }
  if (lane == 0) p.lse[static_cast<int64_t>(r) * p.H + h] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t mla4_scratch_bytes(int, int, int) { return 0; }

dsa_status_t launch_mla4(const Mla4Launch &a, cudaStream_t stream) {
  Mla4Params p;
  p.q = a.q;
  p.latent = a.latent;
  p.rows = a.rows;
  p.idx = a.idx;
  p.out = a.out;
  p.lse = a.lse;
  p.H = a.H;
  p.R = a.R;
  p.W = a.R + a.P;
  p.topk = a.topk;
  p.scale = a.scale;
  p.status = a.status;
  const dim3 grid(static_cast<unsigned>(a.n_q),
                  static_cast<unsigned>((a.H + kHeadsPerCta - 1) / kHeadsPerCta));
  return launch_pdl(mla4_simple_kernel, grid, dim3(kThreads), 0, stream, 1, p) == cudaSuccess
             ? DSA_OK
             : DSA_ERR_CUDA;
}

}  // namespace dsa
