// Sparse MLA over a 4-bit latent cache (row format and contract:
// include/dsa_l4.h).
//
//   z[h, j]   = scale * q[h, :] . L[idx_j, :],   L = 2^e * s * v
//   out[h, :] = sum_j softmax_j(z[h, :]) * L[idx_j, 0:R],   lse[h] = log sum_j exp z[h, j]
//
// Every s * v has at most 6 significant bits and lies in [2^-10, 2688]: an
// fp16 value.  So the selected rows are widened to fp16 tiles in shared memory
// (exactly) and both products run on tcgen05 in kind::f16 with fp16 operands:
//   S = Q . L^T   M = 64 heads, N = 64 keys, K = R + P      (Q: fp16, below)
//   O^T += L^T . P^T   M = 128 latent columns per block, N = 64 heads, K = 64 keys
// The row's 2^e stays out of the tiles.  In base-2 units, with z2 = z log2(e):
//   w[h, j] = 2^(z2 + e_j - m_h),  m_h a running maximum of z2 + e_j,
//   out = sum w s v / l,   lse = (m + log2 l) ln 2,   l = sum 2^(z2 - m)
// so weights stay in (0, 1] whatever the tokens' sizes, and enter the second
// product as two fp16 terms, hi + lo (22 bits), scaled by 2^6: an element of out
// loses what is below 2^-31 of the row's largest product w s v.  q enters as fp16
// after one power of two per query row that puts its largest magnitude in
// [2^14, 2^15).
//   l is summed as w 2^-e_j while every token has |e| <= 24 (rows whose largest
// magnitude is between 8e-5 and 4.5e10): a w that fp32 flushes, below 2^-126, is
// then below 2^-78 of l.  With larger |e| it need not be: 2^-120 lies between e =
// -60 and e = 60.  From the first such slot on, l is summed from z2 itself against
// a running maximum of z2 and brought back to m's units at the end; the merge of
// the splits does likewise.
//
// One CTA per SM takes a contiguous run of 64-key slots of one query row:
//   warps 0-3       softmax of each slot (warp w: heads 16 w ..), the rare
//                   rescale of O
//   warps 4-11, 14  widening: decode a slot from registers, into which the next
//                   slot's bytes are loaded as soon as they are free
//   warp 13         turns the selected positions into pool rows, ahead of them
//   warp 12         issues the MMAs: S of a slot as soon as it is widened, its
//                   PV product as soon as its weights are written
// (the first two kinds write the query tile before that).
// Two slots of the tile ring; S is double-buffered in tensor memory, so S of
// one slot runs under the softmax of the other, and widening under both
// products.
//
// What bounds it: a slot's chain of widening, S, softmax and PV with two slots in
// flight, 8,700 cycles for two at W = 576 (148 rows of top-2,048: 89 us), of which
// the MMAs' issue is busy for 5,900.  Operands, tiles and weights are 400 KB of
// shared-memory traffic per slot, 6,200 cycles for two at 128 bytes a cycle.
//
// A row split over several CTAs leaves (m, l, O) partials in global scratch
// (they stay in L2) and a merge kernel combines them.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "l4_tile.cuh"

namespace dsa {
namespace {

constexpr int kOutWarps = 12;          // warps that read O out, three per tensor memory quadrant
constexpr int kTasks = 4;              // widening tasks per warp and slot: 36 over 9 warps
constexpr int kWeightLog2 = 6;         // weights enter the tensor cores scaled by 2^6
constexpr float kRescaleLog2 = 8.f;    // the running maximum moves when exceeded by 2^8
constexpr float kLn2 = 0.69314718055994531f;
constexpr int kMisc = 2048;
constexpr int kFarExp = 24;            // rows that hold a token with a larger |e| have l summed from z2
constexpr int kMaxSplits = 148;
constexpr int kMaxAtoms = 9;           // 64-column atoms of a row of 576

struct Mla4Params {
  const uint16_t *q;
  const uint8_t *latent;
  PagedRows rows;
  const int32_t *idx;
  float *out;
  float *lse;
  float *part_o;   // [n_q, nsplit, H, R]      (nsplit > 1)
  float *part_ml;  // [n_q, nsplit, 2, H]
  int n_q, H, R, W, topk, nsplit;
  int ncb;  // CTAs that share a split's output columns
  uint32_t cpr_inv;  // query_pieces_inverse(W)
  float scale_log2;
  uint64_t wait_ns;
  int early_q;  // q is complete before the kernel before this one started
  int debug_stall;
  DevStatus *status;
};

// Shared memory: slot 0's nT 64-column atoms (all that PV reads, 2 nmb, and all
// but one of what S reads, nQ), then three atoms
// [hi 0 | lo | hi 1], then those of slot 1, the query tile, barriers.  A slot's
// atom nT, where it has one (columns that only S reads), lies in its hi
// atom, which P hi overwrites once S is done with it.  With hi and lo side by
// side, either slot's weights are one operand of 128 columns (hi | lo, or
// lo | hi): a wide block of O^T takes both terms in one instruction, at 64
// cycles against 2 x 48 (measured), and keeps their sums apart until the end.
struct Layout {
  int nQ, nmb, nT;    // query atoms, 128-column blocks of the latent rows, tile atoms
  uint32_t off_p, off_tile1, off_q, off_misc, bytes;
};
__host__ __device__ inline Layout layout_of(int R, int W) {
  Layout l;
  l.nQ = (W + 63) / 64;
  l.nmb = (R + 127) / 128;
  l.nT = 2 * l.nmb > l.nQ - 1 ? 2 * l.nmb : l.nQ - 1;
  l.off_p = static_cast<uint32_t>(l.nT) * kAtom;
  l.off_tile1 = l.off_p + 3u * kAtom;
  l.off_q = l.off_tile1 + static_cast<uint32_t>(l.nT) * kAtom;
  l.off_misc = l.off_q + static_cast<uint32_t>(l.nQ) * kAtom;
  l.bytes = l.off_misc + kMisc;
  return l;
}
// Tensor memory: S of slot s at columns 64 s, then the CTA's n blocks of O^T,
// `wide` of which keep the sums of the two terms side by side.  In the others
// each small lo product truncates the large sum once more: 1,024 keys a CTA leave
// up to 2.1e-6 of the largest element in columns 0-255 and 4.1e-6 in 256-511, 512
// keys 1.5e-6 and 2.3e-6.  Four wide blocks would need 640 of 512 columns; one
// buffer of S would make room for them, and end the overlap of S and softmax.
constexpr int kWideCols = 128;  // columns of a wide block, against 64
struct Blocks {
  int n, wide;
  __device__ __forceinline__ explicit Blocks(int blocks) : n(blocks) {
    const int spare = (512 - 2 * kKeys) / kHeads - blocks;
    wide = blocks < spare ? blocks : spare;
  }
  __device__ __forceinline__ int col(int mb) const {
    return 2 * kKeys + (mb < wide ? mb * kWideCols : wide * kWideCols + (mb - wide) * kHeads);
  }
};

// What the MMA warp issues is unrolled: an instruction's operands have to be in
// uniform registers, and to compute them in loops took longer than some of the
// instructions run (148 rows of top-2,048 at W = 576: 98.3 us with loops over
// atoms and blocks, 89.0 unrolled; one row 13.3 against 12.9).
//
// kAtoms atoms of S, four K steps each
template <int kAtoms>
__device__ __forceinline__ void issue_s(uint32_t d, uint64_t d_q, uint64_t d_l, uint32_t idesc, uint32_t more) {
#pragma unroll
  for (int k = 0; k < 4 * kAtoms; ++k) {
    const uint32_t at = ((k >> 2) * kAtom + (k & 3) * 32) >> 4;
    mma_f16_elect(d, d_q + at, d_l + at, idesc, k ? 1u : more);
  }
}
// PV of one slot over kN blocks.  d_v: the CTA's first block in the tile; d_both:
// [hi | lo] or [lo | hi].
template <int kN, int kWide>
__device__ __forceinline__ void issue_pv(uint32_t o, uint64_t d_v, uint64_t d_both, uint64_t d_hi,
                                         uint64_t d_lo, uint32_t more, uint64_t *lofree) {
  constexpr uint32_t idesc_wide = idesc_f16_f32(128, kWideCols, 1), idesc_narrow = idesc_f16_f32(128, kHeads, 1);
#pragma unroll
  for (int mb = 0; mb < kWide; ++mb)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      mma_f16_elect(o + mb * kWideCols, d_v + ((2 * mb * kAtom + k * 2048) >> 4), d_both + (k * 32 >> 4),
                    idesc_wide, k ? 1u : more);
#pragma unroll
  for (int t = 0; t < 2; ++t) {
#pragma unroll
    for (int mb = kWide; mb < kN; ++mb)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        mma_f16_elect(o + kWide * kWideCols + (mb - kWide) * kHeads, d_v + ((2 * mb * kAtom + k * 2048) >> 4),
                      (t ? d_hi : d_lo) + (k * 32 >> 4), idesc_narrow, k | t ? 1u : more);
    if (t == 0) commit_elect(lofree);
  }
}

// z2 of two keys, k = their (2^e, e), under the thread's two heads: 8 columns of
// S; -inf where a key is unused
__device__ __forceinline__ void load_z(uint32_t taddr, const float4 &k, float zscale, float (&z)[4]) {
  uint32_t v[4];
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(taddr));
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float scale = i & 1 ? k.z : k.x;  // 0: unused
    z[i] = scale == 0.f ? -INFINITY : __uint_as_float(v[i]) * (scale * zscale);
  }
}
// moves a running maximum that a slot exceeds by 2^8; what its sums are multiplied by
__device__ __forceinline__ float raise(float &m, float x) {
  if (!(x > m + kRescaleLog2 || m == -INFINITY)) return 1.f;
  const float a = x == m ? 1.f : ex2(m - x);
  m = x;
  return a;
}

__global__ void __launch_bounds__(kThreads, 1) mla4_kernel(const Mla4Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const int W = p.W, R = p.R;
  const Layout lay = layout_of(R, W);
  const uint32_t tile = smem_u32(smem), qs = tile + lay.off_q;
  const uint32_t hi_base = tile + lay.off_p, lo_buf = hi_base + kAtom;  // hi of slot s: + 2 s atoms
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + lay.off_misc);
  uint64_t *full = bars;        // [2] slot widened, its keys' powers of two written (widening warps, row warp)
  uint64_t *empty = bars + 2;   // [2] PV of the slot completed (MMA commit)
  uint64_t *sfull = bars + 4;   // [2] S of the slot in tensor memory (MMA commit)
  uint64_t *pready = bars + 6;  // the current slot's weights written (one arrive per softmax warp)
  uint64_t *lofree = bars + 7;  // P lo of the current slot read (MMA commit)
  uint64_t *qready = bars + 8;  // query tile written (one arrive per warp that wrote some)
  uint64_t *bar_drain = bars + 9;
  uint64_t *bar_stall = bars + 10;
  uint64_t *rowfull = bars + 11;  // [2] the slot's pool rows known (row warp)
  uint64_t *rowfree = bars + 13;  // [2] and read (one arrive per widening warp)
  // [0] tensor memory base, [1] failed
  volatile uint32_t *misc = reinterpret_cast<volatile uint32_t *>(bars + 16);
  volatile uint32_t *failed = misc + 1;
  float *qmax = reinterpret_cast<float *>(bars + 18);   // [13], padded to 16
  float *alpha = qmax + 16;                             // [64]
  float2 *keys = reinterpret_cast<float2 *>(alpha + kHeads);    // [2][64] (2^e, e); (0, -inf): unused
  int *rowi = reinterpret_cast<int *>(keys + 2 * kKeys);        // [2][64] pool row, -1: none
  // [2] a key of this slot, or of one in its place before, has |e| > kFarExp
  volatile uint32_t *far = reinterpret_cast<uint32_t *>(rowi + 2 * kKeys);
  float *mfin = reinterpret_cast<float *>(keys);                // [64], [64]: after the loop
  float *lfin = mfin + kHeads;

  const int tid = threadIdx.x, warp = warp_id(), lane = lane_id();
  const int split = blockIdx.x;  // blockIdx.z: the output columns
  // causal rows grow with their number: the longest ones start first
  const int row = p.rows.causal ? p.n_q - 1 - static_cast<int>(blockIdx.y) : static_cast<int>(blockIdx.y);

  // tensor memory: S of slot s at columns 64 s, O^T from column 128
  const Blocks ob(lay.nmb / p.ncb);  // this CTA's blocks of O^T, from mb0
  const int mb0 = static_cast<int>(blockIdx.z) * ob.n;
  const int o_cols = ob.col(ob.n) - 2 * kKeys;
  uint32_t tmem_cols = 32;
  while (tmem_cols < static_cast<uint32_t>(2 * kKeys + o_cols)) tmem_cols <<= 1;
  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&full[s], kWideWarps + 1);
      mbar_init(&empty[s], 1);
      mbar_init(&sfull[s], 1);
      mbar_init(&rowfull[s], 1);
      mbar_init(&rowfree[s], kWideWarps);
    }
    mbar_init(pready, kSoftWarps);
    mbar_init(lofree, 1);
    mbar_init(qready, kSoftWarps + kWideWarps);
    mbar_init(bar_drain, 1);
    mbar_init(bar_stall, 1);
    *failed = 0u;
    far[0] = far[1] = 0u;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(const_cast<uint32_t *>(&misc[0]), tmem_cols);
    tmem_relinquish();
  }
  const bool worker = warp < kMmaWarp || warp == kLastWideWarp;
  const int wtid = warp == kLastWideWarp ? kWorkers - 32 + lane : tid;
  const uint16_t *qrow = p.q + static_cast<int64_t>(row) * p.H * W;
  float zscale = 0.f;  // logit units: log2(e) * scale / the query's power of two
  // in the whole step q predates the kernel before this one: its tile is
  // written under that kernel's tail
  if (p.early_q) {
    __syncthreads();
    if (worker) {
      QueryPieces q;
      q.load(qrow, p.H, W, wtid);
      const int k = q.scale_exponent(wtid, qmax);
      zscale = pow2i(-k) * p.scale_log2;
      q.store<true>(qs, W, p.cpr_inv, wtid, k, qready);
    }
  }
  griddep_wait();
  griddep_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  if (p.debug_stall) {
    if (tid == 0 && !mbar_wait(bar_stall, 0u, p.wait_ns)) *failed = 1u;
    __syncthreads();
  }

  // this CTA's slots: a row keeps at most min(topk, len) tokens, in its first
  // places, and its slots are shared out evenly over the splits
  const int len = l4_row_len(p.rows, row);
  const int limit = l4_limit(p.rows, len);
  const int nsel = max(0, min(p.topk, len));
  const int nh_row = (nsel + kKeys - 1) / kKeys;
  const int per = (nh_row + p.nsplit - 1) / p.nsplit;
  const int h_begin = min(nh_row, split * per);
  const int nh = min(nh_row, h_begin + per) - h_begin;

  // Widening: the bytes of a slot's 64 rows come in 36 tasks of 32 16-byte
  // code units, four per warp.  Task t < 32: units 0-15 of rows 2 t and 2 t + 1,
  // sixteen lanes side by side per row (with four lanes per row the loads took
  // twice the cache lines each, and the load path, which the tile's stores
  // share, was the limit); task 32 + t: units 16 and 17 of rows 16 t .. 16 t + 15.
  const int g = warp == kLastWideWarp ? kWideWarps - 1 : warp - kSoftWarps, nb = W / kL4Block, units = (nb + 1) / 2, rb = l4_row_bytes(W);
  auto task_row = [&](int i) {
    const int t = g + kWideWarps * i;
    return t < 32 ? 2 * t + (lane >> 4) : 16 * (t - 32) + (lane >> 1);
  };
  auto task_unit = [&](int i) { return g + kWideWarps * i < 32 ? (lane & 15) : 16 + (lane & 1); };
  uint4 code[kTasks];
  uint32_t sc[kTasks];    // the unit's two block scales
  uint32_t have = 0u;               // bit i: task i's row exists
  // The next slot's bytes, into registers.  Every lane loads, from the pool's
  // first row and the row's first unit where it has none of its own (a branch
  // around the loads cost more than they do); the scales are dropped later.
  auto load_rows = [&](int j) -> bool {
    const int s = j & 1;
    if (!wait_or_fail(&rowfull[s], (j >> 1) & 1, p.wait_ns, failed)) return false;
    int r[kTasks];
#pragma unroll
    for (int i = 0; i < kTasks; ++i) r[i] = rowi[s * kKeys + task_row(i)];
    have = 0u;
#pragma unroll
    for (int i = 0; i < kTasks; ++i) {
      const int u = task_unit(i) < units ? task_unit(i) : 0;
      have |= (r[i] >= 0 ? 1u : 0u) << i;
      const uint8_t *src = p.latent + static_cast<int64_t>(max(r[i], 0)) * rb;
      code[i] = *reinterpret_cast<const uint4 *>(src + 16 * u);
      sc[i] = ldg_u16(src + W / 2 + 2 * u);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&rowfree[s]);
    return true;
  };

  bool loaded = false;
  if (worker && !p.early_q && nh > 0) {
    QueryPieces q;
    q.load(qrow, p.H, W, wtid);
    const int k = q.scale_exponent(wtid, qmax);
    zscale = pow2i(-k) * p.scale_log2;
    q.store<true>(qs, W, p.cpr_inv, wtid, k, qready);
    if (warp >= kSoftWarps) loaded = load_rows(0);
  } else if (worker && warp >= kSoftWarps && nh > 0) {
    loaded = load_rows(0);
  }
  if (warp < kSoftWarps) regs_inc<kSoftRegs>();
  else regs_dec<kOtherRegs>();

  if (warp < kSoftWarps) {
    // --------------------------------------------------------------- softmax
    const int r0 = lane >> 2, c2 = 2 * (lane & 3);
    const int h0 = 16 * warp + r0, h1 = h0 + 8;  // this thread's two heads
    const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t prow0 = h0 * 128, prow1 = h1 * 128, pcol = c2 * 2;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    bool alive = true;
    // O times what the sums of the slots before slot j > 0 are multiplied by
    auto rescale = [&](int j, float a0, float a1) {
      // O holds every earlier slot once PV(j - 1) has completed
      if ((lane & 3) == 0) {
        alpha[h0] = a0;
        alpha[h1] = a1;
      }
      alive = wait_or_fail(&empty[(j - 1) & 1], ((j - 1) >> 1) & 1, p.wait_ns, failed);
      bar_sync(1, 32 * kSoftWarps);
      tc_fence_after();
      if (alive)
        for (int u = 0; u < o_cols / 32; ++u) {
          const uint32_t ta = tmem + lane_off + 2 * kKeys + 32 * u;
          uint32_t o[32];
          tmem_ld_32x32b_x32(ta, o);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i)
            o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha[32 * (u & 1) + i]);
          tmem_st_32x32b_x32(ta, o);
        }
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      bar_sync(1, 32 * kSoftWarps);  // alpha may be rewritten
    };
    int j = 0;
    bool from_z = false;
    for (; j < nh; ++j) {
      const int s = j & 1;
      const uint32_t par = (j >> 1) & 1;
      alive = alive && wait_or_fail(&sfull[s], par, p.wait_ns, failed) &&
              wait_or_fail(&full[s], par, p.wait_ns, failed);
      tc_fence_after();
      from_z = far[s];  // the same for all four warps
      // z2 + e of this thread's 16 keys of two heads
      uint32_t v[32];
      tmem_ld_16x256b_x8(tmem + lane_off + kKeys * s, v);
      tmem_ld_wait();
      float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 k = *reinterpret_cast<const float4 *>(&keys[s * kKeys + 8 * i + c2]);
        const float ka = k.x * zscale, kb = k.z * zscale;
        const float a0 = fmaf(__uint_as_float(v[4 * i]), ka, k.y);
        const float b0 = fmaf(__uint_as_float(v[4 * i + 1]), kb, k.w);
        const float a1 = fmaf(__uint_as_float(v[4 * i + 2]), ka, k.y);
        const float b1 = fmaf(__uint_as_float(v[4 * i + 3]), kb, k.w);
        x0 = fmaxf(x0, fmaxf(a0, b0));
        x1 = fmaxf(x1, fmaxf(a1, b1));
        v[4 * i] = __float_as_uint(a0);
        v[4 * i + 1] = __float_as_uint(b0);
        v[4 * i + 2] = __float_as_uint(a1);
        v[4 * i + 3] = __float_as_uint(b1);
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, o));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, o));
      }
      float a0 = 1.f, a1 = 1.f;
      if (x0 > m0 + kRescaleLog2 || m0 == -INFINITY) {
        a0 = x0 == m0 ? 1.f : ex2(m0 - x0);
        m0 = x0;
      }
      if (x1 > m1 + kRescaleLog2 || m1 == -INFINITY) {
        a1 = x1 == m1 ? 1.f : ex2(m1 - x1);
        m1 = x1;
      }
      const bool need = from_z || (j > 0 && ((a0 != 1.f && h0 < p.H) || (a1 != 1.f && h1 < p.H)));
      if (bar_or(1, 32 * kSoftWarps, need || !alive)) {
        if (bar_or(1, 32 * kSoftWarps, !alive)) {
          from_z = false;  // in every warp: none goes on below
          break;
        }
        if (j > 0) rescale(j, a0, a1);
        if (from_z) {
          l0 *= a0;
          l1 *= a1;
          break;
        }
      }
      // weights, 2^6 of them, and their share of l
      const float f0 = (m0 == -INFINITY ? 0.f : m0) - kWeightLog2;
      const float f1 = (m1 == -INFINITY ? 0.f : m1) - kWeightLog2;
      float s0 = 0.f, s1 = 0.f;
      uint32_t lw0[8], lw1[8];
      const uint32_t hb = hi_base + 2 * s * kAtom;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float wa0 = ex2(__uint_as_float(v[4 * i]) - f0), wb0 = ex2(__uint_as_float(v[4 * i + 1]) - f0);
        const float wa1 = ex2(__uint_as_float(v[4 * i + 2]) - f1), wb1 = ex2(__uint_as_float(v[4 * i + 3]) - f1);
        const float4 k = *reinterpret_cast<const float4 *>(&keys[s * kKeys + 8 * i + c2]);
        const float ia = __uint_as_float((254u << 23) - __float_as_uint(k.x));  // 2^-e
        const float ib = __uint_as_float((254u << 23) - __float_as_uint(k.z));
        s0 = fmaf(wb0, ib, fmaf(wa0, ia, s0));
        s1 = fmaf(wb1, ib, fmaf(wa1, ia, s1));
        const uint32_t hi0 = pack_f16(wa0, wb0), hi1 = pack_f16(wa1, wb1);
        const float2 g0 = __half22float2(as_half2(hi0)), g1 = __half22float2(as_half2(hi1));
        lw0[i] = pack_f16(wa0 - g0.x, wb0 - g0.y);
        lw1[i] = pack_f16(wa1 - g1.x, wb1 - g1.y);
        const uint32_t ch = static_cast<uint32_t>((i ^ r0) << 4) + pcol;  // h0 % 8 = h1 % 8 = r0
        sts_u32(hb + prow0 + ch, hi0);
        sts_u32(hb + prow1 + ch, hi1);
      }
      l0 = fmaf(l0, a0, s0);
      l1 = fmaf(l1, a1, s1);
      if (j > 0) alive = wait_or_fail(lofree, (j - 1) & 1, p.wait_ns, failed) && alive;
      if (alive) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t ch = static_cast<uint32_t>((i ^ r0) << 4) + pcol;
          sts_u32(lo_buf + prow0 + ch, lw0[i]);
          sts_u32(lo_buf + prow1 + ch, lw1[i]);
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && alive) mbar_arrive(pready);
    }
    // The same from the first slot with a far key on, l apart from the weights (a
    // second exponential per key).  A rolled loop of its own, from S in tensor
    // memory: inside the loop above, or unrolled beside it, it took registers from
    // every row (2,300 causal rows 883 and 845 us, 823 so, 813 without it; 819 since
    // the waits vote).  With far keys in every row: 997.
    if (j < nh && from_z) {
      float n0 = m0, n1 = m1;  // what l is relative to
      for (; j < nh; ++j) {
        const int s = j & 1;
        const uint32_t par = (j >> 1) & 1;
        alive = alive && wait_or_fail(&sfull[s], par, p.wait_ns, failed) &&
                wait_or_fail(&full[s], par, p.wait_ns, failed);
        tc_fence_after();
        const uint32_t ta = tmem + lane_off + kKeys * s;
        const float2 *key = keys + s * kKeys + c2;
        float x0 = -INFINITY, x1 = -INFINITY, y0 = -INFINITY, y1 = -INFINITY;
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
          const float4 k = *reinterpret_cast<const float4 *>(key + 8 * i);
          float z[4];
          load_z(ta + 8 * i, k, zscale, z);
          x0 = fmaxf(x0, fmaxf(z[0] + k.y, z[1] + k.w));
          x1 = fmaxf(x1, fmaxf(z[2] + k.y, z[3] + k.w));
          y0 = fmaxf(y0, fmaxf(z[0], z[1]));
          y1 = fmaxf(y1, fmaxf(z[2], z[3]));
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, o));
          x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, o));
          y0 = fmaxf(y0, __shfl_xor_sync(0xffffffffu, y0, o));
          y1 = fmaxf(y1, __shfl_xor_sync(0xffffffffu, y1, o));
        }
        const float a0 = raise(m0, x0), a1 = raise(m1, x1);
        l0 *= raise(n0, y0);
        l1 *= raise(n1, y1);
        const bool need = j > 0 && ((a0 != 1.f && h0 < p.H) || (a1 != 1.f && h1 < p.H));
        if (bar_or(1, 32 * kSoftWarps, need || !alive)) {
          if (bar_or(1, 32 * kSoftWarps, !alive)) break;
          rescale(j, a0, a1);
        }
        if (j > 0) alive = wait_or_fail(lofree, (j - 1) & 1, p.wait_ns, failed) && alive;
        const float f0 = (m0 == -INFINITY ? 0.f : m0) - kWeightLog2;
        const float f1 = (m1 == -INFINITY ? 0.f : m1) - kWeightLog2;
        const float g0 = (n0 == -INFINITY ? 0.f : n0) - kWeightLog2;
        const float g1 = (n1 == -INFINITY ? 0.f : n1) - kWeightLog2;
        const uint32_t hb = hi_base + 2 * s * kAtom;
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
          const float4 k = *reinterpret_cast<const float4 *>(key + 8 * i);
          float z[4];
          load_z(ta + 8 * i, k, zscale, z);
          l0 += ex2(z[0] - g0) + ex2(z[1] - g0);
          l1 += ex2(z[2] - g1) + ex2(z[3] - g1);
          const float wa0 = ex2(z[0] + k.y - f0), wb0 = ex2(z[1] + k.w - f0);
          const float wa1 = ex2(z[2] + k.y - f1), wb1 = ex2(z[3] + k.w - f1);
          const uint32_t hi0 = pack_f16(wa0, wb0), hi1 = pack_f16(wa1, wb1);
          const float2 t0 = __half22float2(as_half2(hi0)), t1 = __half22float2(as_half2(hi1));
          const uint32_t ch = static_cast<uint32_t>((i ^ r0) << 4) + pcol;
          if (alive) {
            sts_u32(hb + prow0 + ch, hi0);
            sts_u32(hb + prow1 + ch, hi1);
            sts_u32(lo_buf + prow0 + ch, pack_f16(wa0 - t0.x, wb0 - t0.y));
            sts_u32(lo_buf + prow1 + ch, pack_f16(wa1 - t1.x, wb1 - t1.y));
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && alive) mbar_arrive(pready);
      }
      // into m's units: |e| <= 60 keeps n - m within 100, and l inside fp32
      l0 = l0 != 0.f ? l0 * ex2(n0 - m0) : 0.f;
      l1 = l1 != 0.f ? l1 * ex2(n1 - m1) : 0.f;
    }
    // the last PV has to complete before O and the lo buffer are used
    if (nh > 0) wait_or_fail(&empty[(nh - 1) & 1], ((nh - 1) >> 1) & 1, p.wait_ns, failed);
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, o);
      l1 += __shfl_xor_sync(0xffffffffu, l1, o);
    }
    bar_sync(1, 32 * kSoftWarps);
    if ((lane & 3) == 0) {
      const bool good = nh > 0 && !*failed;
      mfin[h0] = good ? m0 - kWeightLog2 : -INFINITY;
      mfin[h1] = good ? m1 - kWeightLog2 : -INFINITY;
      lfin[h0] = good ? l0 : 0.f;
      lfin[h1] = good ? l1 : 0.f;
    }
  } else if (worker) {
    // -------------------------------------------------------------- widening
    for (int j = 0; j < nh && loaded; ++j) {
      const int s = j & 1;
      if (j >= 2 && !wait_or_fail(&empty[s], ((j >> 1) - 1) & 1, p.wait_ns, failed)) break;
#pragma unroll
      for (int i = 0; i < kTasks; ++i) {
        const int u = task_unit(i), r = task_row(i), a = u >> 1;
        const bool live = (have >> i) & 1u;
        const uint32_t dst = r * 128 + (a < lay.nT ? tile + a * kAtom + s * lay.off_tile1
                                                        : hi_base + 2 * s * kAtom);
        // the four words in an order turned by the unit, so that eight
        // neighbouring lanes store to eight different 16-byte columns
        const int rot = a & 3;
        const uint32_t x = (4 * (u & 1)) ^ (r & 7);
        uint32_t w[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
        rotate4(w, rot);
        const uint32_t both = e4m3x2_to_f16x2(live ? sc[i] : 0u);  // no row: zeros
        const __half2 s_lo = as_half2(__byte_perm(both, 0u, 0x1010)), s_hi = as_half2(__byte_perm(both, 0u, 0x3232));
        // at W = 16 (mod 32) the last unit's second block is no column
        const int words = u >= units ? 0 : (2 * u + 1 < nb ? 4 : 2);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int tw = (t + rot) & 3;  // the word, 8 columns
          uint32_t h[4];
          e2m1x8_to_f16x2(w[t], h);
          const __half2 sv = tw < 2 ? s_lo : s_hi;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const __half2 y = __hmul2(as_half2(h[q]), sv);
            h[q] = *reinterpret_cast<const uint32_t *>(&y);
          }
          if (tw < words) sts_v4(dst + ((x ^ tw) << 4), h[0], h[1], h[2], h[3]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[s]);
      if (j + 1 < nh) loaded = load_rows(j + 1);
    }
  } else if (warp == kRowWarp) {
    // -------------------------------------------------------------- pool rows
    // Places 2 lane and 2 lane + 1 of each slot: position, page, pool row; the
    // next slot's positions are loaded before this one's pages are waited for.
    // Positions outside the context and bad pages are dropped and reported.
    const int32_t *idx = p.idx + static_cast<int64_t>(row) * p.topk;
    auto position = [&](int j, int x) -> int {
      const int place = (h_begin + j) * kKeys + 2 * lane + x;
      return j < nh && place < nsel ? idx[place] : -1;
    };
    bool live[2] = {false, false};
    uint32_t eb[2] = {0u, 0u};
    // the keys' powers of two, a slot behind the rows, so that no slot's rows
    // wait for them, and whether one is far
    auto publish = [&](int j) -> bool {
      const int s = j & 1;
      float2 k[2];
      bool wide = false;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int e = l4_exponent(eb[x]);
        wide |= live[x] && eb[x] - (127u - kFarExp) > 2u * kFarExp;
        k[x] = live[x] ? make_float2(pow2i(e), static_cast<float>(e)) : make_float2(0.f, -INFINITY);
      }
      if (j >= 2 && !wait_or_fail(&empty[s], ((j >> 1) - 1) & 1, p.wait_ns, failed)) return false;
      *reinterpret_cast<float4 *>(&keys[s * kKeys + 2 * lane]) = make_float4(k[0].x, k[0].y, k[1].x, k[1].y);
      if (wide) far[s] = 1u;
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[s]);
      return true;
    };
    int pos[2] = {position(0, 0), position(0, 1)};
    for (int j = 0; j < nh; ++j) {
      const int s = j & 1;
      const int next[2] = {position(j + 1, 0), position(j + 1, 1)};
      int r[2];
#pragma unroll
      for (int x = 0; x < 2; ++x)
        r[x] = l4_pool_row(p.rows, row, pos[x], limit, p.status, kKernMla4,
                           (h_begin + j) * kKeys + 2 * lane + x);
      if (j > 0 && !publish(j - 1)) break;
      if (j >= 2 && !wait_or_fail(&rowfree[s], ((j >> 1) - 1) & 1, p.wait_ns, failed)) break;
      // into L2 ahead of the widening warps' loads: a row is 336 bytes at
      // W = 576, four lines at most
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (r[x] >= 0) {
          const uint8_t *src = p.latent + static_cast<int64_t>(r[x]) * rb;
          for (int b = 0; b < rb; b += 128) prefetch_l2(src + b);
          prefetch_l2(src + rb - 1);
        }
      *reinterpret_cast<int2 *>(&rowi[s * kKeys + 2 * lane]) = make_int2(r[0], r[1]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&rowfull[s]);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        live[x] = r[x] >= 0;
        eb[x] = ldg_u8(p.latent + static_cast<int64_t>(max(r[x], 0)) * rb + W / 2 + nb);
      }
      pos[0] = next[0];
      pos[1] = next[1];
    }
    if (nh > 0 && !warp_failed(failed)) publish(nh - 1);
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------- MMA issue
    // The whole warp runs this and branches on votes, so that the descriptors
    // are computed once per warp, in uniform registers; each instruction goes
    // out from one lane.  (From a single-thread branch an instruction took 110
    // cycles to issue, against the 45 to 64 it runs.)
    const uint32_t idesc_s = idesc_f16_f32(kHeads, kKeys, 0);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0), tile_u = __shfl_sync(0xffffffffu, tile, 0);
    const uint32_t p_u = tile_u + lay.off_p;
    const int full_atoms = W / 64, tail = W / 16 - 4 * full_atoms;  // of the query; K steps after them
    const uint64_t d_q = smem_desc(tile_u + lay.off_q, 16, 1024, kLayoutSW128);
    bool ok = nh == 0 || wait_or_fail(qready, 0u, p.wait_ns, failed);
    int ns = 0, npv = 0;
    uint64_t t0 = 0;
    uint32_t spins = 0;
    while (ok && npv < nh) {
      bool progressed = false;
      if (ns < nh && ns <= npv + 1 &&
          __all_sync(0xffffffffu, mbar_test(&full[ns & 1], (ns >> 1) & 1))) {
        fence_proxy_async_smem();
        tc_fence_after();
        const int s = ns & 1;
        const uint32_t d = tm + kKeys * s;
        const uint64_t d_l = smem_desc(tile_u + s * lay.off_tile1, 16, 1024, kLayoutSW128);
        const uint64_t d_p = smem_desc(p_u + 2 * s * kAtom, 16, 1024, kLayoutSW128);
        if (full_atoms == kMaxAtoms) {  // the ninth lies in the hi atom
          issue_s<kMaxAtoms - 1>(d, d_q, d_l, idesc_s, 0u);
          issue_s<1>(d, d_q + ((kMaxAtoms - 1) * kAtom >> 4), d_p, idesc_s, 1u);
        } else {
          uint64_t q = d_q;
          for (int a = 0; a < full_atoms; ++a, q += kAtom >> 4)
            issue_s<1>(d, q, a < lay.nT ? d_l + (a * kAtom >> 4) : d_p, idesc_s, a ? 1u : 0u);
          const uint64_t l = full_atoms < lay.nT ? d_l + (full_atoms * kAtom >> 4) : d_p;
          for (int k = 0; k < tail; ++k)
            mma_f16_elect(d, q + (k * 32 >> 4), l + (k * 32 >> 4), idesc_s, full_atoms | k ? 1u : 0u);
        }
        commit_elect(&sfull[s]);
        ++ns;
        progressed = true;
      }
      if (npv < ns && __all_sync(0xffffffffu, mbar_test(pready, npv & 1))) {
        tc_fence_after();
        const int s = npv & 1;
        const uint32_t more = npv > 0 ? 1u : 0u;
        const uint64_t d_v = smem_desc(tile_u + s * lay.off_tile1 + 2 * mb0 * kAtom, kAtom, 1024, kLayoutSW128);
        const uint64_t d_both = smem_desc(p_u + s * kAtom, 16, 1024, kLayoutSW128);
        const uint64_t d_hi = smem_desc(p_u + 2 * s * kAtom, 16, 1024, kLayoutSW128);
        const uint64_t d_lo = smem_desc(p_u + kAtom, 16, 1024, kLayoutSW128);
        const uint32_t o = tm + 2 * kKeys;
        if (ob.n == 4) issue_pv<4, 2>(o, d_v, d_both, d_hi, d_lo, more, lofree);
        else if (ob.n == 3) issue_pv<3, 3>(o, d_v, d_both, d_hi, d_lo, more, lofree);
        else if (ob.n == 2) issue_pv<2, 2>(o, d_v, d_both, d_hi, d_lo, more, lofree);
        else issue_pv<1, 1>(o, d_v, d_both, d_hi, d_lo, more, lofree);
        commit_elect(&empty[s]);
        ++npv;
        progressed = true;
      }
      if (progressed) {
        spins = 0;
      } else if (++spins % 64 == 0) {
        const uint64_t now = global_timer_ns();
        if (spins == 64) t0 = now;
        if (__any_sync(0xffffffffu, *failed != 0u || now - t0 > p.wait_ns)) {
          *failed = 1u;
          ok = false;
        }
      }
    }
    if (warp_failed(failed)) {
      commit_elect(bar_drain);  // fires once every MMA issued above has completed
      mbar_wait(bar_drain, 0u, kDrainLimitNs);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const bool bad = *failed != 0u;
  if (bad && tid == 0) report(p.status, kErrTimeout, (kKernMla4 << 24) | 1u);
  const bool have_o = !bad && nh > 0;
  if (bad && tid < kHeads) {  // whatever the softmax warps left
    mfin[tid] = -INFINITY;
    lfin[tid] = 0.f;
  }
  if (bad) __syncthreads();
  // Output, or the split's partial result: units of 32 latent columns (the
  // warp's lane quadrant) x 32 heads, 128 bytes per head and store.  (Staging
  // the block in shared memory for one bulk copy took longer.)
  float *dst = p.nsplit == 1 ? p.out + static_cast<int64_t>(row) * p.H * R
                             : p.part_o + (static_cast<int64_t>(row) * p.nsplit + split) * p.H * R;
  if (p.nsplit == 1) {  // what O is multiplied by: 1 / l, 0 for an empty row; a NaN stays one
    if (tid < kHeads) {
      const float l = lfin[tid];
      alpha[tid] = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
    }
    __syncthreads();
  }
  if (warp < kOutWarps && (have_o || p.nsplit == 1)) {
    const int q4 = warp & 3;
    for (int u = warp >> 2; u < 2 * ob.n; u += kOutWarps / 4) {
      const int mb = u >> 1, hb = 32 * (u & 1);
      if (hb >= p.H) continue;
      uint32_t v[32];
      if (have_o) {
        const uint32_t ta = tmem + (static_cast<uint32_t>(q4 * 32) << 16) + ob.col(mb) + hb;
        tmem_ld_32x32b_x32(ta, v);
        if (mb < ob.wide) {
          uint32_t w[32];
          tmem_ld_32x32b_x32(ta + kHeads, w);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i)
            v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(w[i]));
        } else {
          tmem_ld_wait();
        }
      }
      const int c = (mb0 + mb) * 128 + q4 * 32 + lane, left = p.H - hb;
      if (c < R) {
        float *at = dst + static_cast<int64_t>(hb) * R + c;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          float o = have_o ? __uint_as_float(v[i]) : 0.f;
          if (p.nsplit == 1) o *= alpha[hb + i];
          if (i < left) *at = o;
          at += R;
        }
      }
    }
  }
  if (tid < p.H && mb0 == 0) {
    if (p.nsplit == 1) {
      const float l = lfin[tid];
      p.lse[static_cast<int64_t>(row) * p.H + tid] =
          l > 0.f ? (mfin[tid] + log2f(l)) * kLn2 : (l == l ? -INFINITY : l);
    } else {
      float *ml = p.part_ml + (static_cast<int64_t>(row) * p.nsplit + split) * 2 * p.H;
      ml[tid] = mfin[tid];
      ml[p.H + tid] = lfin[tid];
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) {
    __syncwarp();
    tmem_dealloc(tmem, tmem_cols);
  }
}

// Combine the split partials of one (row, head):
//   out = sum_s 2^(m_s - M) O_s / (2^D L),  lse = (M + D + log2 L) ln 2,
//   L = sum_s 2^(m_s - M - D) l_s
// D is 0 while no m_s is below M - 60 (l_s is between 2^-54 and 2^97), else an
// integer near log2 of the largest 2^(m_s - M) l_s: what a split with a small m
// holds of l may be most of it (l counts tokens by their weight, m by their weight
// times their size), however far 2^(m_s - M) lies below fp32.
// One CTA per (row, head): kGroups groups of 128 threads take every kGroups-th
// split, a thread four columns.  The loads of O (kMergeBatch splits per group
// at once) are in flight while one warp forms the splits' weights, so the
// kernel waits on memory once for up to kGroups * kMergeBatch splits; few
// splits come with many rows and take one group, so that more CTAs fit an SM.
// A split without keys has l = 0 and wrote no O: what its place holds is read
// and dropped.
constexpr int kMergeBatch = 8;
template <int kGroups>
__global__ void __launch_bounds__(128 * kGroups) mla4_merge_kernel(const Mla4Params p) {
  __shared__ float wt[kMaxSplits];
  __shared__ float tot[3];
  __shared__ float4 part[kGroups][128];
  griddep_wait();
  griddep_launch_dependents();
  const int row = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, lane = lane_id();
  const int grp = tid >> 7, c = 4 * (tid & 127);
  const int64_t stride = static_cast<int64_t>(p.H) * p.R;
  const float *po = p.part_o + static_cast<int64_t>(row) * p.nsplit * stride + static_cast<int64_t>(h) * p.R;
  float4 v[kMergeBatch];
  auto load = [&](int s0) {
#pragma unroll
    for (int i = 0; i < kMergeBatch; ++i) {
      const int s = s0 + kGroups * i;
      v[i] = s < p.nsplit && c < p.R ? *reinterpret_cast<const float4 *>(po + s * stride + c)
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  load(grp);
  const float *ml = p.part_ml + static_cast<int64_t>(row) * p.nsplit * 2 * p.H;
  if (tid < 32) {
    float M = -INFINITY, D = 0.f, L = 0.f;
    // rolled for many splits: unrolled it takes 82 registers, which leaves one CTA of
    // 512 threads an SM (the step at 4 x 131,072: 69.7 us, 68.1 rolled); few splits
    // run the loop once (32 rows: 38.5 us rolled, 38.2 unrolled)
    constexpr int kUnroll = kGroups == 4 ? 1 : 4;
#pragma unroll kUnroll
    for (int s = lane; s < p.nsplit; s += 32) M = fmaxf(M, ml[s * 2 * p.H + h]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    bool far = false;
    for (int s = lane; s < p.nsplit; s += 32) {
      const float m = ml[s * 2 * p.H + h], l = ml[s * 2 * p.H + p.H + h];
      const float w = m == -INFINITY ? 0.f : exp2f(m - M);
      far |= m != -INFINITY && m - M < -60.f;
      wt[s] = w;
      L += w == 0.f ? 0.f : w * l;
    }
    if (__any_sync(0xffffffffu, far)) {
      D = -126.f;
      L = 0.f;
#pragma unroll 1
      for (int s = lane; s < p.nsplit; s += 32) {
        const float m = ml[s * 2 * p.H + h], l = ml[s * 2 * p.H + p.H + h];  // l > 0 where m is finite
        const int k = static_cast<int>(__float_as_uint(l) >> 23) - 127;
        if (m != -INFINITY) D = fmaxf(D, ceilf(m - M) + static_cast<float>(k));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) D = fmaxf(D, __shfl_xor_sync(0xffffffffu, D, o));
      D = fminf(D, 126.f);
#pragma unroll 1
      for (int s = lane; s < p.nsplit; s += 32) {
        const float m = ml[s * 2 * p.H + h], l = ml[s * 2 * p.H + p.H + h];
        L += m == -INFINITY ? 0.f : exp2f(m - M - D) * l;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    if (lane == 0) {
      tot[0] = M;
      tot[1] = L;
      tot[2] = D;
    }
  }
  __syncthreads();
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = grp; s0 < p.nsplit; s0 += kGroups * kMergeBatch) {
    if (s0 != grp) load(s0);
#pragma unroll
    for (int i = 0; i < kMergeBatch; ++i) {
      const int s = s0 + kGroups * i;
      const float w = s < p.nsplit ? wt[s] : 0.f;
      if (w != 0.f) {
        acc.x = fmaf(w, v[i].x, acc.x);
        acc.y = fmaf(w, v[i].y, acc.y);
        acc.z = fmaf(w, v[i].z, acc.z);
        acc.w = fmaf(w, v[i].w, acc.w);
      }
    }
  }
  if constexpr (kGroups > 1) {
    part[grp][tid & 127] = acc;
    __syncthreads();
    if (grp == 0) {
#pragma unroll
      for (int g = 1; g < kGroups; ++g) {
        const float4 b = part[g][tid];
        acc.x += b.x;
        acc.y += b.y;
        acc.z += b.z;
        acc.w += b.w;
      }
    }
  }
  const float L = tot[1], D = tot[2];
  const float il = L > 0.f ? pow2i(-static_cast<int>(D)) / L : (L == L ? 0.f : L);
  if (grp == 0 && c < p.R) {
    float *out = p.out + (static_cast<int64_t>(row) * p.H + h) * p.R + c;  // 4-byte aligned only
    out[0] = acc.x * il;
    out[1] = acc.y * il;
    out[2] = acc.z * il;
    out[3] = acc.w * il;
  }
  if (tid == 0)
    p.lse[static_cast<int64_t>(row) * p.H + h] =
        L > 0.f ? (tot[0] + (D + log2f(L))) * kLn2 : (L == L ? -INFINITY : L);
}

// Splits of a row: while rows leave SMs idle, as many CTAs per row as fit one
// wave, one slot each at least.
int plan_splits(int n_q, int topk) {
  const int nh = (topk + kKeys - 1) / kKeys;
  const int want = std::min(kMaxSplits, device_sm_count()) / std::max(1, n_q);
  const int ns = std::max(1, std::min(want, nh));
  const int per = (nh + ns - 1) / ns;
  return (nh + per - 1) / per;
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
// O^T partials, at H = 64: the size does not depend on the call's head count
size_t part_o_bytes(int n_q, int ns, int R) {
  return align256(static_cast<size_t>(n_q) * ns * kHeads * R * 4);
}

}  // namespace

size_t mla4_scratch_bytes(int n_q, int topk, int R) {
  const int ns = plan_splits(n_q, topk);
  if (ns == 1) return 0;
  return part_o_bytes(n_q, ns, R) + align256(static_cast<size_t>(n_q) * ns * 2 * kHeads * 4);
}

dsa_status_t launch_mla4(const Mla4Launch &a, cudaStream_t stream) {
  const int W = a.R + a.P;
  const size_t smem = 1024 + layout_of(a.R, W).bytes;
  if (smem > device_max_smem_optin()) return DSA_ERR_UNSUPPORTED;
  if (func_attr_once(reinterpret_cast<const void *>(mla4_kernel),
                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                     static_cast<int>(device_max_smem_optin())) != cudaSuccess)
    return DSA_ERR_CUDA;
  Mla4Params p;
  p.q = a.q;
  p.latent = a.latent;
  p.rows = a.rows;
  p.idx = a.idx;
  p.out = a.out;
  p.lse = a.lse;
  p.n_q = a.n_q;
  p.H = a.H;
  p.R = a.R;
  p.W = W;
  p.topk = a.topk;
  p.nsplit = plan_splits(a.n_q, a.topk);
  p.cpr_inv = query_pieces_inverse(W);
  p.part_o = nullptr;
  p.part_ml = nullptr;
  if (p.nsplit > 1) {
    if (a.scratch == nullptr || a.scratch_bytes < mla4_scratch_bytes(a.n_q, a.topk, a.R))
      return DSA_ERR_WORKSPACE;
    p.part_o = static_cast<float *>(a.scratch);
    p.part_ml = reinterpret_cast<float *>(static_cast<uint8_t *>(a.scratch) +
                                          part_o_bytes(a.n_q, p.nsplit, a.R));
  }
  p.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
  p.wait_ns = wait_limit_ns();
  p.early_q = a.early_q;
  p.debug_stall = debug_stall() == static_cast<int>(kKernMla4) ? 1 : 0;
  p.status = a.status;
  // While CTAs still leave SMs idle, a split's output columns go to 2 or 4 of
  // them: each forms the logits anew, but multiplies and stores its share only
  // (one row of top-2,048: 15.1 us with one CTA a split, 13.0 with four).
  const int nmb = (a.R + 127) / 128;
  p.ncb = 1;
  for (int c = 2; c <= 4; c *= 2)
    if (nmb % c == 0 && static_cast<int64_t>(a.n_q) * p.nsplit * c <= device_sm_count()) p.ncb = c;
  if (launch_pdl(mla4_kernel,
                 dim3(static_cast<unsigned>(p.nsplit), static_cast<unsigned>(a.n_q),
                      static_cast<unsigned>(p.ncb)),
                 dim3(kThreads), smem, stream, 1u, p) != cudaSuccess)
    return DSA_ERR_CUDA;
  if (p.nsplit == 1) return DSA_OK;
  const int groups = p.nsplit > 2 * kMergeBatch ? 4 : (p.nsplit > kMergeBatch ? 2 : 1);
  void (*merge)(const Mla4Params) = groups == 4   ? mla4_merge_kernel<4>
                                    : groups == 2 ? mla4_merge_kernel<2>
                                                  : mla4_merge_kernel<1>;
  return launch_pdl(merge, dim3(static_cast<unsigned>(a.n_q), static_cast<unsigned>(a.H)),
                    dim3(128u * groups), 0, stream, 1u, p) == cudaSuccess
             ? DSA_OK
             : DSA_ERR_CUDA;
}

}  // namespace dsa
