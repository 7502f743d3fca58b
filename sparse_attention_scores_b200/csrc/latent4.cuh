// Device-side pieces of the 4-bit latent row format (include/dsa_l4.h): the
// paged lookup, decoding of codes and scales, and the rounding into them.
#pragma once

#include <cuda_fp16.h>

#include "l4_internal.h"

namespace dsa {

constexpr int kL4Block = 16;      // columns per block scale
constexpr int kL4MaxExp = 60;     // |e| of a row's power of two

// position -> pool row of query row r (its sequence: r, or 0 in a causal
// chunk); -1 for an unused slot, and for a position outside [0, limit) or a
// page outside the pool, which are reported
__device__ __forceinline__ int l4_pool_row(const PagedRows &p, int r, int pos, int limit,
                                           DevStatus *status, unsigned kernel, int slot) {
  if (pos < 0) return -1;
  if (pos >= limit) {
    report(status, kErrBadIndex, (kernel << 24) | (slot & 0xFFFF));
    return -1;
  }
  const int seq = p.causal ? 0 : r;
  const int page = p.block_table[static_cast<int64_t>(seq) * p.max_pages + pos / kPageSize];
  if (page < 0 || page >= p.num_pages) {
    report(status, kErrBadPage, (kernel << 24) | (slot & 0xFFFF));
    return -1;
  }
  return page * kPageSize + pos % kPageSize;
}
// tokens query row r sees, and the positions its block table can hold
__device__ __forceinline__ int l4_row_len(const PagedRows &p, int r) {
  return p.causal ? p.q_pos0 + r + 1 : p.seq_lens[r];
}
__device__ __forceinline__ int l4_limit(const PagedRows &p, int len) {
  return min(len, p.max_pages * kPageSize);
}

// four code bytes (8 columns) as four fp16 pairs, exactly.  w is a loaded
// 32-bit word: with a single zero-extended byte in it the compiler (12.9)
// drops that byte's conversion and the pair reads as zero.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
// an E4M3 byte as fp16 in both halves of a pair, exactly
__device__ __forceinline__ __half2 e4m3_to_half2(uint32_t byte) {
  uint32_t h;
  const uint16_t two = static_cast<uint16_t>((byte & 0xFFu) * 0x0101u);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
  return *reinterpret_cast<const __half2 *>(&h);
}
// two E4M3 bytes as an fp16 pair (low byte first), exactly
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  return h;
}
__device__ __forceinline__ __half2 as_half2(uint32_t v) { return *reinterpret_cast<const __half2 *>(&v); }

// the row's power of two from its exponent byte (clamped to the format's range)
__device__ __forceinline__ int l4_exponent(uint32_t byte) {
  return max(-kL4MaxExp, min(kL4MaxExp, static_cast<int>(byte) - 127));
}
// 2^e for |e| <= 126
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// least e with amax <= 2688 * 2^e, clamped; 0 for amax = 0.  2688 = 6 * 448, the
// largest |s v|, is 1.3125 * 2^11: mantissa bits 0x280000
__device__ __forceinline__ int l4_row_exponent(float amax) {
  if (amax == 0.f) return 0;
  const uint32_t u = __float_as_uint(amax);
  const int ex = static_cast<int>(u >> 23) - 127;  // bf16 subnormals clamp below
  const int e = ex - 11 + ((u & 0x7FFFFFu) > 0x280000u ? 1 : 0);
  return max(-kL4MaxExp, min(kL4MaxExp, e));
}
// E4M3 code of x >= 0, round to nearest even, saturating
__device__ __forceinline__ uint32_t f16_to_e4m3(__half x) {
  uint16_t r;
  const uint32_t two = __half_as_ushort(x);
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(two));
  return r & 0xFFu;
}
// two e2m1 codes, a in the low nibble, round to nearest even, saturating
__device__ __forceinline__ uint32_t f32x2_to_e2m1(float a, float b) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n\tcvt.u32.u8 %0, t;\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b));
  return r;
}

}  // namespace dsa
