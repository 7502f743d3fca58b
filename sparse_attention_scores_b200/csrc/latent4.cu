// 4-bit latent cache: quantising append and exact read-back (the row format is
// in include/dsa_l4.h).
//
// Append, for a new row x of W columns:
//   e    = least exponent with max|x| <= 2688 * 2^e
//   s[b] = E4M3(max|x_b| / (6 * 2^e))     per block b of 16 columns
//   v    = e2m1(x / (s[b] * 2^e))
// x has 8 significant bits, s 4 and every boundary between two e2m1 codes 3, so
// a boundary times s fits 8 bits too: a quotient that is not a boundary differs
// from it by 2^-8 or more, relative.  So the quotient is taken as x times an
// approximate reciprocal (2^-21) and rounded to fp16 (2^-12), which puts a
// quotient that is a boundary back onto it and moves none across: the codes are
// those of the exact quotients, without an exact division.  The same holds for
// the scale, whose boundaries have 5 bits, 7 times 6.
//
// A warp takes one row, a lane a 16-byte piece of 8 columns (72 pieces at
// W = 576, three rounds), two lanes a block.  Both kernels move each byte once;
// they are bound by the copy bandwidth at many rows and by launch latency at
// few.
#include <cuda_bf16.h>

#include "latent4.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 128;
constexpr int kRowsPerCta = kThreads / 32;
constexpr int kRounds = 3;  // 16-byte pieces per lane: W <= 576 -> 72 over 32 lanes

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
  const int pieces = p.W / 8;
  const uint4 *src = p.lat_new + static_cast<int64_t>(r) * pieces;
  const uint4 *ks = p.k_new + static_cast<int64_t>(r) * p.kw;
  // the row itself does not depend on where it goes
  uint4 x[kRounds];
#pragma unroll
  for (int i = 0; i < kRounds; ++i)
    x[i] = lane + 32 * i < pieces ? src[lane + 32 * i] : make_uint4(0u, 0u, 0u, 0u);
  const uint4 key = lane < p.kw ? ks[lane] : make_uint4(0u, 0u, 0u, 0u);  // D_I <= 128: one piece per lane
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
  if (lane < p.kw) p.k_pages[slot * p.kw + lane] = key;

  float bmax[kRounds], amax = 0.f;
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    float m = 0.f;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const float2 v = bf16x2_to_f32(w[t]);
      m = fmaxf(m, fmaxf(fabsf(v.x), fabsf(v.y)));
    }
    bmax[i] = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));  // the block's other half
    amax = fmaxf(amax, bmax[i]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const int e = l4_row_exponent(amax);
  const float inv = pow2i(-e);  // exact: |e| <= 60
  const int rb = l4_row_bytes(p.W), nb = p.W / kL4Block;
  uint8_t *dst = p.lat_pages + slot * rb;
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const int c = lane + 32 * i;
    const uint32_t code = f16_to_e4m3(__float2half_rn(fminf(bmax[i] * inv * (1.f / 6.f), 448.f)));
    const float s = __low2float(e4m3_to_half2(code));
    const float rs = s > 0.f ? __fdividef(inv, s) : 0.f;  // a block whose scale is 0 is stored as zeros
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    uint32_t out = 0u;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const float2 v = bf16x2_to_f32(w[t]);
      const float2 q = __half22float2(__floats2half2_rn(v.x * rs, v.y * rs));
      out |= f32x2_to_e2m1(q.x, q.y) << (8 * t);
    }
    if (c < pieces) {
      *reinterpret_cast<uint32_t *>(dst + 4 * c) = out;
      if (!(c & 1)) dst[p.W / 2 + (c >> 1)] = static_cast<uint8_t>(code);
    }
  }
  const int used = p.W / 2 + nb;
  for (int i = used + lane; i < rb; i += 32)
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

// kRows rows per warp: lanes resolve them together, and the bytes of all of
// them are in flight at once.  Four where the rows fill the device (65,536 rows
// of 576: 20.0 us against 22.3 with one; 16,384: 5.9 against 6.0), one where
// they do not (64 rows: 1.9 us).
template <int kRows>
__global__ void __launch_bounds__(kThreads) read4_kernel(const Read4Params p) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t g0 = (static_cast<int64_t>(blockIdx.x) * kRowsPerCta + warp_id()) * kRows;
  const int lane = lane_id();
  if (g0 >= p.total) return;
  const int nb = p.W / kL4Block, rb = l4_row_bytes(p.W), pieces = p.W / 8;
  int row = -1;
  if (lane < kRows && g0 + lane < p.total) {
    const int64_t g = g0 + lane;
    const int r = static_cast<int>(g / p.k), j = static_cast<int>(g - static_cast<int64_t>(r) * p.k);
    row = l4_pool_row(p.rows, r, p.idx[g], l4_limit(p.rows, l4_row_len(p.rows, r)), p.status,
                      kKernRead4, j);
  }
  // a lane's pieces of 8 columns: their codes, block scale and exponent
  uint32_t code[kRows][kRounds], sc[kRows][kRounds], eb[kRows];
  int rows[kRows];
#pragma unroll
  for (int x = 0; x < kRows; ++x) {
    rows[x] = __shfl_sync(0xffffffffu, row, x);
    const uint8_t *src = p.lat_pages + static_cast<int64_t>(max(rows[x], 0)) * rb;
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
      const int c = min(lane + 32 * i, pieces - 1);
      code[x][i] = *reinterpret_cast<const uint32_t *>(src + 4 * c);
      sc[x][i] = src[p.W / 2 + (c >> 1)];
    }
    eb[x] = src[p.W / 2 + nb];
  }
#pragma unroll
  for (int x = 0; x < kRows; ++x) {
    if (g0 + x >= p.total) break;
    uint4 *dst = p.out + (g0 + x) * pieces;
    const float t = pow2i(l4_exponent(eb[x]));
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
      const int c = lane + 32 * i;
      if (c >= pieces) break;
      const __half2 s = e4m3_to_half2(sc[x][i]);
      uint32_t h[4], o[4];
      e2m1x8_to_f16x2(code[x][i], h);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 v = __half22float2(__hmul2(as_half2(h[q]), s));  // exact: 6 bits
        const __nv_bfloat162 w = __floats2bfloat162_rn(v.x * t, v.y * t);
        o[q] = rows[x] < 0 ? 0u : *reinterpret_cast<const uint32_t *>(&w);
      }
      dst[c] = make_uint4(o[0], o[1], o[2], o[3]);
    }
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
  const int per_warp = p.total >= static_cast<int64_t>(device_sm_count()) * 64 ? 4 : 1;
  const int64_t grid = (p.total + kRowsPerCta * per_warp - 1) / (kRowsPerCta * per_warp);
  if (grid > INT32_MAX) return DSA_ERR_UNSUPPORTED;
  return launch_pdl(per_warp == 4 ? read4_kernel<4> : read4_kernel<1>,
                    dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, stream, 1, p) == cudaSuccess
             ? DSA_OK
             : DSA_ERR_CUDA;
}

}  // namespace dsa
