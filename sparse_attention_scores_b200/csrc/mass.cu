// Accumulated attention weight per cached token (contract: include/dsa_l4.h):
//
//   mass_out[b, s] = decay * mass_in[b, s] + sum_{r, h, j: idx[r,j] = s} exp(z[r,h,j] - lse[r,h])
//
// decay_kernel writes decay * mass_in over the live positions (and clears the
// 64-bit sums of a causal chunk).  mass_kernel recomputes the logits on tcgen05
//   S = L . Q^T   M = 64 kept keys, N = 64 heads, K = R + P
// over the same pipeline as the attention over a 4-bit cache, without its
// second product: a row warp turns positions into pool rows, nine warps fill
// one of two 64-key slots (4-bit and E4M3 rows widened to fp16, exactly; bf16
// rows as they are), one issues the MMAs, four read S with a key per lane
// quad, so the sum over heads stays inside a thread but for two shuffles.  A
// decode row adds in fp32 (its positions are its own); the rows of a causal
// chunk add to one sequence, in 64-bit fixed point so that the order does not
// matter, and fold_kernel turns the sums into fp32.
#include <algorithm>

#include "l4_tile.cuh"

namespace dsa {
namespace {

constexpr int kSweep = 256;  // threads of the sweeps over positions
// A chunk's sums are whole numbers of steps of 2^-f: the finest for which n_q rows
// of weights below kMostWeight stay below 2^63 (f = 40 at 65,535 rows, the most a
// chunk has, 47 at 512, 56 at one; a weight below half a step adds nothing)
constexpr float kMostWeight = 128.f;
inline int fixed_bits(int n_q) {
  int c = 0;  // n_q <= 2^c
  while ((static_cast<int64_t>(1) << c) < n_q) ++c;
  return 63 - 7 - c;
}

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
  int max_len;
  int n_q, H, W, topk, nsplit;
  uint32_t cpr_inv, units_inv;  // inverses of 16-byte pieces per query head and per stored row, at 2^20
  float scale_log2, decay;
  double fixed_one;  // 2^fixed_bits
  uint64_t wait_ns;
  int debug_stall;
  DevStatus *status;
};

// tokens of sequence b, at most max_len
__device__ __forceinline__ int mass_len(const MassParams &p, int b) {
  const int len = p.rows.causal ? p.rows.q_pos0 + p.n_q : p.rows.seq_lens[b];
  return max(0, min(len, p.max_len));
}

__global__ void __launch_bounds__(kSweep) decay_kernel(const MassParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.y, n = mass_len(p, b);
#pragma unroll 4
  for (int s = blockIdx.x * kSweep + threadIdx.x; s < n; s += gridDim.x * kSweep) {
    const int64_t at = b * p.mass_ld + s;
    p.mass_out[at] = p.mass_in ? p.decay * p.mass_in[at] : 0.f;
    if (p.fixed) p.fixed[s] = 0ull;
  }
}

// One row's weight of one kept position.  With the step's lse it is at most the
// number of heads; a NaN, and the weights of some other lse, do not go through
// the fixed point but straight to the result, where a NaN stays one.
__device__ __forceinline__ void add_weight(const MassParams &p, int row, int pos, float w) {
  if (pos < 0 || pos >= p.max_len) return;
  if (p.rows.causal && w < kMostWeight)
    atomicAdd(&p.fixed[pos], static_cast<unsigned long long>(
                                 __double2ll_rn(static_cast<double>(w) * p.fixed_one)));
  else
    atomicAdd(&p.mass_out[p.rows.causal ? pos : row * p.mass_ld + pos], w);
}


// Shared memory: two slots of the tile (64 keys x W), the query tile, barriers.
// Tensor memory: kParts partial sums of S per slot, which the reader adds.  The
// tensor cores truncate each accumulation towards zero, and the errors of a
// chain add up in the logit: 512 causal rows of 2,048 keys are off by 1.4e-6
// with one chain of 36, 6.5e-7 with two of 18 (3% slower), 3.4e-7 with four (6%);
// fp32 additions give 6e-8.  Two were chosen: what is left is below what the
// attention's own sums lose.
constexpr int kMisc = 2048;
constexpr int kParts = 2;
struct Layout {
  int nQ;
  uint32_t slot, off_q, off_misc, bytes;
};
__host__ __device__ inline Layout layout_of(int W) {
  Layout l;
  l.nQ = (W + 63) / 64;
  l.slot = static_cast<uint32_t>(l.nQ) * kAtom;
  l.off_q = 2u * l.slot;
  l.off_misc = l.off_q + l.slot;
  l.bytes = l.off_misc + kMisc;
  return l;
}
// 16-byte units of a stored row's columns, and the tasks of 32 units a filling
// warp takes per slot at W = 576
template <int F>
__host__ __device__ constexpr int units_of(int W) {
  return F == kLatBf16 ? W / 8 : (F == kLatE4m3 ? W / 16 : (W / kL4Block + 1) / 2);
}
template <int F>
constexpr int kTasksOf = (2 * units_of<F>(576) + kWideWarps - 1) / kWideWarps;
// Warps that fill a slot.  bf16 rows are copied, which takes no registers: four
// warps fill the even slots and four the odd ones, so that a slot is announced
// when its own copies have landed (with one group for both, one slot's copies
// were issued between another's arrival and its announcement: 349 us against
// 266 for 512 causal rows of 2,048 keys; 231 since S's issue is unrolled).  What is left is the copies' own rate,
// about 17 bytes a cycle and SM.
template <int F>
constexpr int kFillers = F == kLatBf16 ? 4 : kWideWarps;

// The four K steps of atom a.  Unrolled over the atoms of a row of 576: an
// instruction's operands have to be in uniform registers, and to compute them in
// a loop took longer than it runs.
constexpr int kMaxAtoms = 9;
__device__ __forceinline__ void issue_atom(uint32_t d, int a, uint64_t d_l, uint64_t d_q, uint32_t idesc) {
#pragma unroll
  for (int k = 0; k < 4; ++k)
    mma_f16_elect(d + (a & (kParts - 1)) * kHeads, d_l + ((a * kAtom + k * 32) >> 4),
                  d_q + ((a * kAtom + k * 32) >> 4), idesc, a >= kParts || k != 0 ? 1u : 0u);
}

template <int F>
__global__ void __launch_bounds__(kThreads, 1) mass_kernel(const MassParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const int W = p.W;
  const Layout lay = layout_of(W);
  const uint32_t tile = smem_u32(smem), qs = tile + lay.off_q;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + lay.off_misc);
  uint64_t *full = bars;         // [2] slot filled, its key factors written (filling warps, row warp)
  uint64_t *sread = bars + 2;    // [2] S and key factors read (one arrive per summing warp)
  uint64_t *sfull = bars + 4;    // [2] S in tensor memory, the slot's tile free (MMA commit)
  uint64_t *rowfull = bars + 6;  // [2] the slot's pool rows known (row warp)
  uint64_t *rowfree = bars + 8;  // [2] and read (one arrive per filling warp)
  uint64_t *qready = bars + 10;
  uint64_t *bar_drain = bars + 11;
  uint64_t *bar_stall = bars + 12;
  // [0] tensor memory base, [1] failed
  volatile uint32_t *misc = reinterpret_cast<volatile uint32_t *>(bars + 14);
  volatile uint32_t *failed = misc + 1;
  float *qmax = reinterpret_cast<float *>(bars + 16);      // [13], padded to 16
  float *factor = qmax + 16;                                // [2][64] a key's scale
  int *rowi = reinterpret_cast<int *>(factor + 2 * kKeys);  // [2][64] pool row, -1: none
  uint2 *used = reinterpret_cast<uint2 *>(rowi + 2 * kKeys);  // [2] the slot's used keys: even ones, odd ones

  const int tid = threadIdx.x, warp = warp_id(), lane = lane_id();
  const int split = blockIdx.x;
  const int row = p.rows.causal ? p.n_q - 1 - static_cast<int>(blockIdx.y) : static_cast<int>(blockIdx.y);
  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&full[s], kFillers<F> + 1);
      mbar_init(&sread[s], kSoftWarps);
      mbar_init(&sfull[s], 1);
      mbar_init(&rowfull[s], 1);
      mbar_init(&rowfree[s], kFillers<F>);
    }
    mbar_init(qready, kSoftWarps + kWideWarps);
    mbar_init(bar_drain, 1);
    mbar_init(bar_stall, 1);
    *failed = 0u;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(const_cast<uint32_t *>(&misc[0]), 2 * kParts * kHeads);
    tmem_relinquish();
  }
  // What this kernel reads is older than decay_kernel, which had waited for it
  // before it let this one start; only the sums have to wait for decay_kernel
  // itself (before their first add).
  griddep_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  if (p.debug_stall) {
    if (tid == 0 && !mbar_wait(bar_stall, 0u, p.wait_ns)) *failed = 1u;
    __syncthreads();
  }
  const int len = min(l4_row_len(p.rows, row), p.max_len), limit = l4_limit(p.rows, len);
  const int nsel = max(0, min(p.topk, len));
  const int nh_row = (nsel + kKeys - 1) / kKeys;
  const int per = (nh_row + p.nsplit - 1) / p.nsplit;
  const int h_begin = min(nh_row, split * per);
  const int nh = min(nh_row, h_begin + per) - h_begin;
  const int32_t *idx = p.idx + static_cast<int64_t>(row) * p.topk;

  const bool worker = warp < kMmaWarp || warp == kLastWideWarp;
  float zscale = 0.f;
  if (worker && nh > 0) {
    const int wtid = warp == kLastWideWarp ? kWorkers - 32 + lane : tid;
    QueryPieces q;
    q.load(p.q + static_cast<int64_t>(row) * p.H * W, p.H, W, wtid);
    const int k = F != kLatBf16 ? q.scale_exponent(wtid, qmax) : 0;
    zscale = pow2i(-k) * p.scale_log2;
    q.store<F != kLatBf16>(qs, W, p.cpr_inv, wtid, k, qready);
  }
  if (warp < kSoftWarps) regs_inc<kSoftRegs>();
  else regs_dec<kOtherRegs>();

  if (warp < kSoftWarps) {
    // --------------------------------------------------------------- head sums
    // lane t reads keys 16 warp + t / 4 (+ 8), heads 8 i + 2 (t % 4) + {0, 1}
    const int k0 = 16 * warp + (lane >> 2), c2 = 2 * (lane & 3);
    const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
    float ls[16];  // log2 units; +inf where the head adds nothing
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int h = 8 * (i >> 1) + c2 + (i & 1);
      const float l = h < p.H ? p.lse[static_cast<int64_t>(row) * p.H + h] : -INFINITY;
      ls[i] = l == -INFINITY ? INFINITY : l * 1.44269504088896341f;
    }
    auto place = [&](int j, int x) -> int {
      const int at = (h_begin + j) * kKeys + k0 + 8 * x;
      return j < nh && at < nsel ? idx[at] : -1;
    };
    int pos[2] = {place(0, 0), place(0, 1)};
    griddep_wait();
    for (int j = 0; j < nh; ++j) {
      const int s = j & 1;
      const uint32_t par = (j >> 1) & 1;
      if (!wait_or_fail(&sfull[s], par, p.wait_ns, failed) ||
          !wait_or_fail(&full[s], par, p.wait_ns, failed))
        break;
      const int next[2] = {place(j + 1, 0), place(j + 1, 1)};
      tc_fence_after();
      uint32_t v[32];
      tmem_ld_16x256b_x8(tmem + lane_off + s * kParts * kHeads, v);
      const float *f = factor + s * kKeys + k0;
      const float f0 = f[0], f1 = f[8];
      const uint32_t mine = (k0 & 1 ? used[s].y : used[s].x) >> (k0 >> 1);  // bits 0 and 4: k0 and k0 + 8
      tmem_ld_wait();
      for (int x = 1; x < min(kParts, lay.nQ); ++x) {
        uint32_t u[32];
        tmem_ld_16x256b_x8(tmem + lane_off + (s * kParts + x) * kHeads, u);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i)
          v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(u[i]));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sread[s]);
      const float t0 = f0 * zscale, t1 = f1 * zscale;
      float w0 = 0.f, w1 = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        w0 += ex2(fmaf(__uint_as_float(v[4 * i]), t0, -ls[2 * i])) +
              ex2(fmaf(__uint_as_float(v[4 * i + 1]), t0, -ls[2 * i + 1]));
        w1 += ex2(fmaf(__uint_as_float(v[4 * i + 2]), t1, -ls[2 * i])) +
              ex2(fmaf(__uint_as_float(v[4 * i + 3]), t1, -ls[2 * i + 1]));
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        w0 += __shfl_xor_sync(0xffffffffu, w0, o);
        w1 += __shfl_xor_sync(0xffffffffu, w1, o);
      }
      if ((lane & 3) == 0) {
        if (mine & 1u) add_weight(p, row, pos[0], w0);
        if (mine & 16u) add_weight(p, row, pos[1], w1);
      }
      pos[0] = next[0];
      pos[1] = next[1];
    }
  } else if (worker) {
    // ----------------------------------------------------------------- filling
    // A slot's 64 x units 16-byte units, 32 neighbours per task: coalesced, and
    // eight neighbouring lanes store to eight different 16-byte columns
    const int g = warp == kLastWideWarp ? kWideWarps - 1 : warp - kSoftWarps;
    const int units = units_of<F>(W), nb = W / kL4Block;
    const int bytes = F == kLatBf16 ? 2 * W : (F == kLatE4m3 ? W : l4_row_bytes(W));
    if constexpr (F == kLatBf16) {
      for (int j = g >> 2; j < nh && g < 2 * kFillers<F>; j += 2) {
        const int s = j & 1;
        if (!wait_or_fail(&rowfull[s], (j >> 1) & 1, p.wait_ns, failed)) break;
        if (j >= 2 && !wait_or_fail(&sfull[s], ((j >> 1) - 1) & 1, p.wait_ns, failed)) break;
#pragma unroll 6
        for (int t = (g & 3) * 32 + lane; t < kKeys * units; t += 32 * kFillers<F>) {
          const int r = static_cast<int>((static_cast<uint32_t>(t) * p.units_inv) >> 20);
          const int u = t - r * units, at = rowi[s * kKeys + r];
          const uint8_t *src = p.latent + static_cast<int64_t>(max(at, 0)) * bytes + 16 * u;
          cp_async_16(tile + s * lay.slot + (u >> 3) * kAtom + r * 128 + (((u & 7) ^ (r & 7)) << 4), src,
                      at >= 0 ? 16u : 0u);
        }
        cp_async_commit();
        __syncwarp();
        if (lane == 0) mbar_arrive(&rowfree[s]);
        cp_async_wait_all();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[s]);
      }
      cp_async_wait_all();
    } else {
      constexpr int kT = kTasksOf<F>;
      int r_of[kT], u_of[kT];  // row -1: no unit
#pragma unroll
      for (int i = 0; i < kT; ++i) {
        const uint32_t t = static_cast<uint32_t>((g + kWideWarps * i) * 32 + lane);
        const int r = static_cast<int>((t * p.units_inv) >> 20);
        r_of[i] = r < kKeys ? r : -1;
        u_of[i] = static_cast<int>(t) - r * units;
      }
      uint4 data[kT];
      uint32_t sc[kT];  // 4-bit rows: the unit's two block scales
      uint32_t have = 0u;
      auto load_rows = [&](int j) -> bool {
        const int s = j & 1;
        if (!wait_or_fail(&rowfull[s], (j >> 1) & 1, p.wait_ns, failed)) return false;
        have = 0u;
#pragma unroll
        for (int i = 0; i < kT; ++i) {
          const int at = r_of[i] >= 0 ? rowi[s * kKeys + r_of[i]] : -1;
          have |= (at >= 0 ? 1u : 0u) << i;
          const int u = r_of[i] >= 0 ? u_of[i] : 0;
          const uint8_t *src = p.latent + static_cast<int64_t>(max(at, 0)) * bytes;
          data[i] = *reinterpret_cast<const uint4 *>(src + 16 * u);
          if constexpr (F == kLatL4) sc[i] = ldg_u16(src + W / 2 + 2 * u);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&rowfree[s]);
        return true;
      };
      bool loaded = nh > 0 && load_rows(0);
      for (int j = 0; j < nh && loaded; ++j) {
        const int s = j & 1;
        if (j >= 2 && !wait_or_fail(&sfull[s], ((j >> 1) - 1) & 1, p.wait_ns, failed)) break;
#pragma unroll
        for (int i = 0; i < kT; ++i) {
          if (r_of[i] < 0) continue;
          const int r = r_of[i], u = u_of[i];
          const bool live = (have >> i) & 1u;
          const uint32_t base = tile + s * lay.slot + r * 128;
          uint32_t w[4] = {data[i].x, data[i].y, data[i].z, data[i].w};
          if constexpr (F == kLatL4) {
            const uint32_t dst = base + (u >> 1) * kAtom;
            const int rot = (u >> 1) & 3;
            const uint32_t x = (4 * (u & 1)) ^ (r & 7);
            rotate4(w, rot);
            const uint32_t both = e4m3x2_to_f16x2(live ? sc[i] : 0u);
            const __half2 s_lo = as_half2(__byte_perm(both, 0u, 0x1010)), s_hi = as_half2(__byte_perm(both, 0u, 0x3232));
            const int words = 2 * u + 1 < nb ? 4 : 2;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const int tw = (t + rot) & 3;
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
          } else {
            // 16 E4M3 values: two 16-byte columns of fp16, in an order turned
            // by the unit
            const uint32_t dst = base + (u >> 2) * kAtom;
            const int turn = (u >> 2) & 1;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const int half = t ^ turn;
              const uint32_t a = half ? w[2] : w[0], b = half ? w[3] : w[1];
              const uint32_t keep = live ? 0xFFFFFFFFu : 0u;
              sts_v4(dst + ((((2 * u + half) & 7) ^ (r & 7)) << 4), e4m3x2_to_f16x2(a & keep & 0xFFFFu),
                     e4m3x2_to_f16x2((a & keep) >> 16), e4m3x2_to_f16x2(b & keep & 0xFFFFu),
                     e4m3x2_to_f16x2((b & keep) >> 16));
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[s]);
        if (j + 1 < nh) loaded = load_rows(j + 1);
      }
    }
  } else if (warp == kRowWarp) {
    // --------------------------------------------------------------- pool rows
    // Places 2 lane and 2 lane + 1 of each slot: position, page, pool row, the
    // key's factor.  The factors are published a slot later, after the next
    // slot's rows, so that no rows wait for them (read
    // by the filling warps beside the units: 75.3 us against 68.8 for 148 rows of
    // 2,048 4-bit keys, 90.2 against 82.8 for E4M3).
    bool live[2] = {false, false};
    uint32_t f[2] = {0u, 0u};  // E4M3: the scale; 4-bit: the exponent byte
    auto publish = [&](int j) -> bool {
      // after slot j - 2 was read: its factors are free, and `full` cannot pass
      // through this slot's phase while a summing warp has yet to see that one's
      if (j >= 2 && !wait_or_fail(&sread[j & 1], ((j >> 1) - 1) & 1, p.wait_ns, failed)) return false;
      float v[2];
#pragma unroll
      for (int x = 0; x < 2; ++x)
        v[x] = !live[x] ? 0.f
                        : (F == kLatBf16 ? 1.f : (F == kLatE4m3 ? __uint_as_float(f[x]) : pow2i(l4_exponent(f[x]))));
      *reinterpret_cast<float2 *>(&factor[(j & 1) * kKeys + 2 * lane]) = make_float2(v[0], v[1]);
      const uint32_t even = __ballot_sync(0xffffffffu, live[0]), odd = __ballot_sync(0xffffffffu, live[1]);
      if (lane == 0) used[j & 1] = make_uint2(even, odd);
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[j & 1]);
      return true;
    };
    auto position = [&](int j, int x) -> int {
      const int at = (h_begin + j) * kKeys + 2 * lane + x;
      return j < nh && at < nsel ? idx[at] : -1;
    };
    int pos[2] = {position(0, 0), position(0, 1)};
    for (int j = 0; j < nh; ++j) {
      const int s = j & 1;
      const int next[2] = {position(j + 1, 0), position(j + 1, 1)};
      int r[2];
#pragma unroll
      for (int x = 0; x < 2; ++x)
        r[x] = l4_pool_row(p.rows, row, pos[x], limit, p.status, kKernMass,
                           (h_begin + j) * kKeys + 2 * lane + x);
      if (j >= 2 && !wait_or_fail(&rowfree[s], ((j >> 1) - 1) & 1, p.wait_ns, failed)) break;
      *reinterpret_cast<int2 *>(&rowi[s * kKeys + 2 * lane]) = make_int2(r[0], r[1]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&rowfull[s]);
      if (j > 0 && !publish(j - 1)) break;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        live[x] = r[x] >= 0;
        const int64_t at = max(r[x], 0);
        if constexpr (F == kLatE4m3) f[x] = __float_as_uint(p.lat_scale[at]);
        if constexpr (F == kLatL4) f[x] = ldg_u8(p.latent + at * l4_row_bytes(W) + W / 2 + W / kL4Block);
      }
      pos[0] = next[0];
      pos[1] = next[1];
    }
    if (nh > 0 && !warp_failed(failed)) publish(nh - 1);
  } else if (warp == kMmaWarp) {
    // --------------------------------------------------------------- MMA issue
    // S = L . Q^T, M = 64 keys, N = 64 heads, K = W; the converged warp computes
    // the descriptors in uniform registers
    const uint32_t idesc = idesc_f16_f32(kKeys, kHeads, 0, F == kLatBf16 ? 1 : 0);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0), tile_u = __shfl_sync(0xffffffffu, tile, 0);
    const uint64_t d_q = smem_desc(tile_u + lay.off_q, 16, 1024, kLayoutSW128);
    const int full_atoms = W / 64, tail = W / 16 - 4 * full_atoms;
    bool ok = nh == 0 || wait_or_fail(qready, 0u, p.wait_ns, failed);
    for (int j = 0; j < nh && ok; ++j) {
      const int s = j & 1;
      if (!wait_or_fail(&full[s], (j >> 1) & 1, p.wait_ns, failed)) break;
      if (j >= 2 && !wait_or_fail(&sread[s], ((j >> 1) - 1) & 1, p.wait_ns, failed)) break;
      fence_proxy_async_smem();
      tc_fence_after();
      const uint32_t d = tm + s * kParts * kHeads;
      const uint64_t d_l = smem_desc(tile_u + s * lay.slot, 16, 1024, kLayoutSW128);
      // 64-column atom a adds to partial sum a % kParts
      if (full_atoms == kMaxAtoms) {
#pragma unroll
        for (int a = 0; a < kMaxAtoms; ++a) issue_atom(d, a, d_l, d_q, idesc);
      } else {
        for (int a = 0; a < full_atoms; ++a) issue_atom(d, a, d_l, d_q, idesc);
      }
      for (int k = 0; k < tail; ++k)
        mma_f16_elect(d + (full_atoms & (kParts - 1)) * kHeads,
                      d_l + ((full_atoms * kAtom + k * 32) >> 4),
                      d_q + ((full_atoms * kAtom + k * 32) >> 4), idesc,
                      full_atoms >= kParts || k != 0 ? 1u : 0u);
      commit_elect(&sfull[s]);
    }
    if (warp_failed(failed)) {
      commit_elect(bar_drain);
      mbar_wait(bar_drain, 0u, kDrainLimitNs);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (*failed && tid == 0) report(p.status, kErrTimeout, (kKernMass << 24) | 1u);
  if (warp == kMmaWarp) {
    __syncwarp();
    tmem_dealloc(tmem, 2 * kParts * kHeads);
  }
}

__global__ void __launch_bounds__(kSweep) fold_kernel(const MassParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int n = mass_len(p, 0);
  for (int s = blockIdx.x * kSweep + threadIdx.x; s < n; s += gridDim.x * kSweep)
    p.mass_out[s] = static_cast<float>(static_cast<double>(p.mass_out[s]) +
                                       static_cast<double>(p.fixed[s]) * (1.0 / p.fixed_one));
}

template <int F>
dsa_status_t launch_sums(MassParams p, cudaStream_t stream) {
  const size_t smem = 1024 + layout_of(p.W).bytes;
  if (smem > device_max_smem_optin()) return DSA_ERR_UNSUPPORTED;
  if (func_attr_once(reinterpret_cast<const void *>(mass_kernel<F>),
                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                     static_cast<int>(device_max_smem_optin())) != cudaSuccess)
    return DSA_ERR_CUDA;
  const int units = units_of<F>(p.W);
  p.units_inv = ((1u << 20) + units - 1) / units;
  return launch_pdl(mass_kernel<F>, dim3(static_cast<unsigned>(p.nsplit), static_cast<unsigned>(p.n_q)),
                    dim3(kThreads), smem, stream, 1u, p) == cudaSuccess
             ? DSA_OK
             : DSA_ERR_CUDA;
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
  p.max_len = a.max_len;
  p.n_q = a.n_q;
  p.H = a.H;
  p.W = a.R + a.P;
  p.topk = a.topk;
  p.cpr_inv = query_pieces_inverse(p.W);
  p.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
  p.decay = a.decay;
  p.fixed_one = ldexp(1.0, fixed_bits(a.n_q));
  p.wait_ns = wait_limit_ns();
  p.debug_stall = debug_stall() == static_cast<int>(kKernMass) ? 1 : 0;
  p.status = a.status;
  // a row's 64-key slots over as many CTAs as fit one wave
  const int slots = (a.topk + kKeys - 1) / kKeys;
  p.nsplit = std::max(1, std::min(slots, device_sm_count() / std::max(1, a.n_q)));
  const unsigned seqs = a.rows.causal ? 1u : static_cast<unsigned>(a.num_seqs);
  const unsigned sweep = static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(128, (a.mass_ld + 4 * kSweep - 1) / (4 * kSweep))));
  if (launch_pdl(decay_kernel, dim3(sweep, seqs), dim3(kSweep), 0, stream, 1, p) != cudaSuccess)
    return DSA_ERR_CUDA;
  const dsa_status_t st = a.format == kLatBf16   ? launch_sums<kLatBf16>(p, stream)
                          : a.format == kLatE4m3 ? launch_sums<kLatE4m3>(p, stream)
                                                 : launch_sums<kLatL4>(p, stream);
  if (st != DSA_OK) return st;
  if (a.rows.causal &&
      launch_pdl(fold_kernel, dim3(sweep), dim3(kSweep), 0, stream, 1, p) != cudaSuccess)
    return DSA_ERR_CUDA;
  return DSA_OK;
}

}  // namespace dsa
