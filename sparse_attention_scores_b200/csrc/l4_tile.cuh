// Pieces that the tensor-core kernels over gathered latent rows share: the
// roles of a 512-thread CTA, bounded waits, fp16 / bf16 MMA issue from a
// converged warp, and the 64-head query tile.
#pragma once

#include <math.h>

#include "latent4.cuh"
#include "warp_wait.cuh"

namespace dsa {

constexpr int kThreads = 512;
constexpr int kSoftWarps = 4;            // warps 0-3: they read S
constexpr int kWideWarps = 9;            // warps 4-11 and 14: they fill the tile
constexpr int kMmaWarp = 12, kRowWarp = 13, kLastWideWarp = 14;
constexpr int kWorkers = 32 * (kSoftWarps + kWideWarps);
// Registers: 128 a thread at launch (512 threads); the warps that read S take
// what the others give up, 128 x 168 + 384 x 112 = 64,512 of the 65,536
constexpr int kSoftRegs = 168, kOtherRegs = 112;
constexpr int kHeads = 64;               // head columns of every tile
constexpr int kKeys = 64;                // keys per slot
constexpr int kAtom = kKeys * 128;       // bytes of a 64-column atom of 64 rows (tile or query)
constexpr int kMaxQ = (kHeads * 72 + kWorkers - 1) / kWorkers;  // 16-byte query pieces per worker at W = 576

// barrier over `n` threads that also returns whether any of them passed true
__device__ __forceinline__ bool bar_or(int id, int n, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(v)), "r"(id), "r"(n)
      : "memory");
  return r != 0u;
}
__device__ __forceinline__ void bar_sync(int id, int n) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}
// whether the phase with the given parity has completed, without waiting:
// mbarrier.try_wait may suspend the thread for a while, which would keep the
// MMA warp from the other product it could issue
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0u;
}
template <int kRegs>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
// kind::f16 instruction descriptor: fp32 D, fp16 operands (bf16: both bf16)
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, int a_mn_major, int bf16 = 0) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (static_cast<uint32_t>(a_mn_major) << 15) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// D (+)= A . B^T, fp16 operands, issued by one lane of a converged warp
__device__ __forceinline__ void mma_f16_elect(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                              uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// one lane's commit: arrives once every MMA that lane issued has completed
// (the same lane is elected each time)
__device__ __forceinline__ void commit_elect(uint64_t *bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_u32(bar))
      : "memory");
}
// 16 lanes x 64 columns: thread t gets columns 8 i + 2 (t % 4) + {0, 1} of lane
// t / 4 in r[4 i], r[4 i + 1] and of lane t / 4 + 8 in r[4 i + 2], r[4 i + 3]
__device__ __forceinline__ void tmem_ld_16x256b_x8(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void sts_v4(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}
__device__ __forceinline__ void sts_u32(uint32_t a, uint32_t x) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(x) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// loads of 16 and 8 bits into a 32-bit register as they are: a conversion after
// the load would be waited for at once, and these are issued a slot ahead
__device__ __forceinline__ uint32_t ldg_u16(const void *a) {
  uint32_t v;
  asm volatile("ld.global.u16 %0, [%1];" : "=r"(v) : "l"(a));
  return v;
}
__device__ __forceinline__ uint32_t ldg_u8(const void *a) {
  uint32_t v;
  asm volatile("ld.global.u8 %0, [%1];" : "=r"(v) : "l"(a));
  return v;
}
__device__ __forceinline__ void prefetch_l2(const void *a) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(a));
}
// w[t] = w[(t + n) % 4]
__device__ __forceinline__ void rotate4(uint32_t (&w)[4], int n) {
  const uint32_t a = w[0], b = w[1], c = w[2], d = w[3];
  const bool one = n & 1, two = n & 2;
  const uint32_t x0 = one ? b : a, x1 = one ? c : b, x2 = one ? d : c, x3 = one ? a : d;
  w[0] = two ? x2 : x0;
  w[1] = two ? x3 : x1;
  w[2] = two ? x0 : x2;
  w[3] = two ? x1 : x3;
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// ceil(2^20 / (W / 8)): t / (W / 8) = t * this >> 20 for t < 64 * 72
__host__ inline uint32_t query_pieces_inverse(int W) { return ((1u << 20) + W / 8 - 1) / (W / 8); }

// The 64-head query tile of one row (heads >= H zero), 128B-swizzled, K-major,
// by the worker threads (wtid in [0, kWorkers)), each holding up to twelve
// 16-byte pieces: load() issues the loads, store() writes the tile.  One pass over
// the row: the pieces stay in registers while its largest magnitude is found.
struct QueryPieces {
  uint4 v[kMaxQ];

  __device__ __forceinline__ void load(const uint16_t *q, int H, int W, int wtid) {
    const uint4 *src = reinterpret_cast<const uint4 *>(q);
    const int n = H * (W / 8);
#pragma unroll
    for (int i = 0; i < kMaxQ; ++i) {
      const int t = wtid + kWorkers * i;
      v[i] = t < n ? src[t] : make_uint4(0u, 0u, 0u, 0u);
    }
  }

  // the exponent of the power of two that puts the row's largest magnitude in
  // [2^14, 2^15) (all workers call it: they meet at a barrier)
  __device__ __forceinline__ int scale_exponent(int wtid, float *qmax) const {
    float mx = 0.f;
#pragma unroll
    for (int i = 0; i < kMaxQ; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int t = 0; t < 4; ++t)
        mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(w[t] << 16)),
                             fabsf(__uint_as_float(w[t] & 0xFFFF0000u))));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (lane_id() == 0) qmax[wtid >> 5] = mx;
    bar_sync(2, kWorkers);
#pragma unroll
    for (int i = 0; i < kSoftWarps + kWideWarps; ++i) mx = fmaxf(mx, qmax[i]);
    const int ex = static_cast<int>(__float_as_uint(mx) >> 23) - 127;
    return mx == 0.f ? 0 : min(126, 14 - ex);  // ex <= 127: at least -113
  }

  // kScaled: as fp16, times 2^k; else as it is (bf16).  Each worker warp
  // arrives on qready once.
  template <bool kScaled>
  __device__ __forceinline__ void store(uint32_t qs, int W, uint32_t cpr_inv, int wtid, int k,
                                        uint64_t *qready) const {
    const int cpr = W / 8;  // 16-byte pieces per head
    const float f = pow2i(k);
#pragma unroll
    for (int i = 0; i < kMaxQ; ++i) {
      const int t = wtid + kWorkers * i;
      if (t < kHeads * cpr) {
        const int h = static_cast<int>((static_cast<uint32_t>(t) * cpr_inv) >> 20);  // t / cpr
        const int c = t - h * cpr;
        uint32_t o[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        if constexpr (kScaled) {
#pragma unroll
          for (int x = 0; x < 4; ++x)
            o[x] = pack_f16(__uint_as_float(o[x] << 16) * f, __uint_as_float(o[x] & 0xFFFF0000u) * f);
        }
        sts_v4(qs + (c >> 3) * kAtom + h * 128 + (((c & 7) ^ (h & 7)) << 4), o[0], o[1], o[2], o[3]);
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane_id() == 0) mbar_arrive(qready);
  }
};

}  // namespace dsa
