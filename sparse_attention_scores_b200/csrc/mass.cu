// Accumulated attention weight per cached token (contract: include/dsa_l4.h):
//
//   mass_out[b, s] = decay * mass_in[b, s] + sum_{r, h, j: idx[r,j] = s} exp(z[r,h,j] - lse[r,h])
//
// Two kernels.  decay_kernel writes decay * mass_in over the live positions
// (and clears the 64-bit sums of a causal chunk).  mass_kernel recomputes the
// logits of every kept row - one CTA of eight warps per query row, one warp
// per kept token, the lanes over the columns - and adds the head sum.  A
// decode row adds in fp32 (its positions are its own); the rows of a causal
// chunk add to one sequence, in 64-bit fixed point so that the order does not
// matter, and fold_kernel turns the sums into fp32.
#include <cuda_bf16.h>
#include <math.h>

#include "latent4.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 9;
constexpr double kFixedOne = 1099511627776.0;  // 2^40: a weight of 64 heads x 2^17 rows stays below 2^63

struct MassParams {
  const uint16_t *q;
  const uint8_t *latent;
  const float *lat_scale;
  PagedRows rows;
  const int32_t *idx;
  const float *lse;
  const float *mass_in;
  float *mass_out;
  unsigned long long *fixed;
  int64_t mass_ld;
  int n_q, num_seqs, H, R, W, topk;
  float scale, decay;
  DevStatus *status;
};

// tokens of sequence b whose mass is kept, at most the row stride
__device__ __forceinline__ int mass_len(const MassParams &p, int b) {
  const int len = p.rows.causal ? p.rows.q_pos0 + p.n_q : p.rows.seq_lens[b];
  return static_cast<int>(min(static_cast<int64_t>(max(0, len)), p.mass_ld));
}

__global__ void __launch_bounds__(kThreads) decay_kernel(const MassParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.y, n = mass_len(p, b);
  for (int s = blockIdx.x * kThreads + threadIdx.x; s < n; s += gridDim.x * kThreads) {
    const int64_t at = b * p.mass_ld + s;
    p.mass_out[at] = p.mass_in ? p.decay * p.mass_in[at] : 0.f;
    if (p.fixed) p.fixed[s] = 0ull;
  }
}

template <int F>
__device__ __forceinline__ float2 latent_pair(const uint8_t *row, int W, int c) {
  if constexpr (F == kLatBf16) {
    const uint32_t v = reinterpret_cast<const uint32_t *>(row)[c];
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
  } else if constexpr (F == kLatE4m3) {
    return make_float2(__low2float(e4m3_to_half2(row[2 * c])), __low2float(e4m3_to_half2(row[2 * c + 1])));
  } else {
    uint32_t h[4];
    e2m1x8_to_f16x2(reinterpret_cast<const uint32_t *>(row)[c / 4], h);
    const uint32_t pair = (c & 2) ? ((c & 1) ? h[3] : h[2]) : ((c & 1) ? h[1] : h[0]);
    return __half22float2(__hmul2(as_half2(pair), e4m3_to_half2(row[W / 2 + c / 8])));
  }
}

template <int F>
__global__ void __launch_bounds__(kThreads) mass_simple_kernel(const MassParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int r = blockIdx.x, warp = warp_id(), lane = lane_id();
  const int W = p.W, pairs = W / 2;
  const int bytes = F == kLatBf16 ? 2 * W : (F == kLatE4m3 ? W : l4_row_bytes(W));
  const int len = l4_row_len(p.rows, r), limit = l4_limit(p.rows, len);
  const int nsel = max(0, min(p.topk, len));
  for (int j = blockIdx.y * (kThreads / 32) + warp; j < nsel; j += gridDim.y * (kThreads / 32)) {
    const int pos = p.idx[static_cast<int64_t>(r) * p.topk + j];
    int row = -1;
    if (lane == 0) row = l4_pool_row(p.rows, r, pos, limit, p.status, kKernMass, j);
    row = __shfl_sync(0xffffffffu, row, 0);
    if (row < 0 || pos >= p.mass_ld) continue;
    const uint8_t *src = p.latent + static_cast<int64_t>(row) * bytes;
    const float t = F == kLatL4 ? pow2i(l4_exponent(src[W / 2 + W / kL4Block]))
                                : (F == kLatE4m3 ? p.lat_scale[row] : 1.f);
    float2 v[kMaxPairs];
#pragma unroll
    for (int i = 0; i < kMaxPairs; ++i) {
      const int c = lane + 32 * i;
      v[i] = c < pairs ? latent_pair<F>(src, W, c) : make_float2(0.f, 0.f);
    }
    float w = 0.f;
    for (int h = 0; h < p.H; ++h) {
      const uint32_t *q = reinterpret_cast<const uint32_t *>(p.q + (static_cast<int64_t>(r) * p.H + h) * W);
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < kMaxPairs; ++i) {
        const int c = lane + 32 * i;
        if (c < pairs)
          dot += __uint_as_float(q[c] << 16) * v[i].x + __uint_as_float(q[c] & 0xFFFF0000u) * v[i].y;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      const float lse = p.lse[static_cast<int64_t>(r) * p.H + h];
      if (lse > -INFINITY) w += expf(dot * t * p.scale - lse);
    }
    if (lane == 0) {
      if (p.rows.causal)
        atomicAdd(&p.fixed[pos], static_cast<unsigned long long>(__double2ll_rn(static_cast<double>(w) * kFixedOne)));
      else
        atomicAdd(&p.mass_out[static_cast<int64_t>(r) * p.mass_ld + pos], w);
    }
  }
}

__global__ void __launch_bounds__(kThreads) fold_kernel(const MassParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int n = mass_len(p, 0);
  for (int s = blockIdx.x * kThreads + threadIdx.x; s < n; s += gridDim.x * kThreads)
    p.mass_out[s] = static_cast<float>(static_cast<double>(p.mass_out[s]) +
                                       static_cast<double>(p.fixed[s]) * (1.0 / kFixedOne));
}

}  // namespace

size_t mass_scratch_bytes(const dsa_dims_t &d) {
  return d.causal ? static_cast<size_t>(static_cast<int64_t>(d.q_pos0) + d.n_q) * 8 : 0;
}

dsa_status_t launch_mass(const MassLaunch &a, cudaStream_t stream) {
  MassParams p;
  p.q = a.q;
  p.latent = static_cast<const uint8_t *>(a.latent);
  p.lat_scale = a.lat_scale;
  p.rows = a.rows;
  p.idx = a.idx;
  p.lse = a.lse;
  p.mass_in = a.mass_in;
  p.mass_out = a.mass_out;
  p.fixed = a.rows.causal ? static_cast<unsigned long long *>(a.scratch) : nullptr;
  p.mass_ld = a.mass_ld;
  p.n_q = a.n_q;
  p.num_seqs = a.num_seqs;
  p.H = a.H;
  p.R = a.R;
  p.W = a.R + a.P;
  p.topk = a.topk;
  p.scale = a.scale;
  p.decay = a.decay;
  p.status = a.status;
  const unsigned seqs = a.rows.causal ? 1u : static_cast<unsigned>(a.num_seqs);
  if (launch_pdl(decay_kernel, dim3(32, seqs), dim3(kThreads), 0, stream, 1, p) != cudaSuccess)
    return DSA_ERR_CUDA;
  const dim3 grid(static_cast<unsigned>(a.n_q), 8);
  const cudaError_t e =
      a.format == kLatBf16   ? launch_pdl(mass_simple_kernel<kLatBf16>, grid, dim3(kThreads), 0, stream, 1, p)
      : a.format == kLatE4m3 ? launch_pdl(mass_simple_kernel<kLatE4m3>, grid, dim3(kThreads), 0, stream, 1, p)
                             : launch_pdl(mass_simple_kernel<kLatL4>, grid, dim3(kThreads), 0, stream, 1, p);
  if (e != cudaSuccess) return DSA_ERR_CUDA;
  if (a.rows.causal &&
      launch_pdl(fold_kernel, dim3(32), dim3(kThreads), 0, stream, 1, p) != cudaSuccess)
    return DSA_ERR_CUDA;
  return DSA_OK;
}

}  // namespace dsa
