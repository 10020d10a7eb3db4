// mxnorm_wgrad.cu -- weight gradient of MXNormLinear from the 8-bit
// checkpoint, on the tensor cores:
//     dW[n, k] = bf16(sum_t dout[t, n] h[t, k]),  h[t, k] = RN_bf16(rho~[t] x^[t, k]),
// x^ the MXFP8 codes times their block scales and rho~ the forward's inverse
// RMS; products exact, sums in fp32.
//
// The sum runs over rows, along which both operands are strided: both are
// MN-major for the MMA (tcgen05 kind::f16, bf16).  Tiles of 256 features n x W
// columns k (W a multiple of 64 up to 256) by a pair of CTAs (cta_group::2,
// M = 256, N = W), persistent pairs, 64 rows t a stage.  dout comes by TMA in
// the MMA's layout (boxes of 64 columns x 64 rows, 128-byte swizzle), the
// codes as they are, and h is made from them in shared memory, so the
// checkpoint is never expanded in device memory.  Per CTA:
//   warp 0         TMA of this CTA's 128 dout columns (on the leader's
//                  "ab_full");
//   warp 1         leader: MMA issuer, once "ab_full" shows both CTAs' dout
//                  and h; frees the slot in both CTAs ("ab_empty"), and
//                  commits to "acc_full" after a tile's last stage;
//   warp 2         TMA of this CTA's codes ("c_full");
//   warps 3-6      scales, every fourth stage each: 2^e of the blocks and rho~
//                  of the rows to shared memory ("p_full"), loaded before the
//                  slot is free so that the loads' latency is hidden;
//   warps 7-10     epilogue: two accumulators in TMEM, so a tile's stores run
//                  under the next tile's MMAs;
//   warps 11-26    h, two groups with a stage in turn: a block of 32 codes a
//                  thread to products with RN(rho~ 2^e), rounded to bf16 and
//                  stored swizzled; then "ab_full" at the leader.
// Two accumulators (512 features) share a stage's h where there are features
// enough: made once for twice the MMAs, h stops bounding the loop (by the
// bandwidth of shared memory: dout in, h in, both out to the MMA).  16384 x
// 4096 x 4096, replayed from a graph: 303 to 307 us, 1800 TFLOP/s, 96 % of the
// measured bf16 rate of a library product (1872 TFLOP/s in a short burst) and
// 93 % of that product at this size (285 us, on h expanded beforehand); single
// calls 335 to 340 us; one accumulator 447 us.
// Narrow tiles of one are bound by the MMA chain (some 115 clocks each).
// Where tiles are few, the rows are split over S pairs a tile: fp32 partial
// sums go to the caller's workspace [S][N][K] and a second kernel adds them in
// order (the same bits every time).  Rows past T load as zeros and get p = 0.
// Waits are bounded (2 s); on expiry bit 0 of the error word is set and the
// waiter arrives on no barrier any more, so that no phase completes that the
// copies or the MMAs have not earned: the other roles' waits run out in turn,
// each lets its own copies and MMAs end, and TMEM is freed.
#include <algorithm>

#include "launch_fp4.h"
#include "mx_row.cuh"
#include "quant_device.cuh"
#include "tc_device.cuh"

namespace mxnorm {

__device__ unsigned int g_wgrad_error_word = 0u;

namespace {

using namespace tc;

constexpr int kFeat = 256;                    // features per pair and accumulator
constexpr int kMaxW = 256;                    // columns per pair
constexpr int kBT = 64;                       // rows per stage
constexpr int kBlkBytes = kBT * 128;          // 64 columns x 64 rows of bf16
constexpr int kStageA = 2 * kBlkBytes;        // this CTA's 128 dout columns of one accumulator

// A stage's shared memory for MT accumulators; NARROW: W <= 128.  Ring depths
// of the MMA's operands (dout and h) and of what h is made of (codes and
// scales): the bytes in flight over the latency of L2 bound a stage from
// below (five slots of 16 KB of dout: 500 clocks whatever W is), so narrow
// tiles, whose slots are smaller, get deeper rings.
template <int MT, bool NARROW>
struct Cfg {
  static constexpr int kMaxG = NARROW ? 2 : 4;                     // blocks of a row
  static constexpr int kStageB = (NARROW ? 1 : 2) * kBlkBytes;     // this CTA's W / 2 columns of h
  static constexpr int kCodeCols = NARROW ? 64 : 128;              // columns of a codes box (W / 2 or more)
  static constexpr int kStageC = kBT * kCodeCols;
  static constexpr int kStageP = kBT * (kMaxG + 1) * 4;            // 2^e of the rows' blocks, then the rows' rho~
  static constexpr int kRingB = NARROW ? (MT == 1 ? 7 : 4) : (MT == 1 ? 5 : 3);
  static constexpr int kRingC = NARROW ? 8 : 6;
  static constexpr size_t kSmem =
      1024 + (size_t)kRingB * (MT * kStageA + kStageB) + (size_t)kRingC * (kStageC + kStageP) + 512;
  static_assert(kSmem <= 232448, "shared memory of a CTA");
};
constexpr int kScaleWarps = 4;
constexpr int kHWarps = 8;                     // warps that make a stage's h
constexpr int kHGroups = 2;                    // groups of them, a stage in turn each
constexpr int kFirstScale = 3, kFirstEpi = kFirstScale + kScaleWarps, kFirstH = kFirstEpi + 4;
constexpr int kThreads = 32 * (kFirstH + kHGroups * kHWarps);
static_assert(kBT * Cfg<1, false>::kMaxG == 32 * kHWarps, "one block of 32 columns a thread of an h group");
// Warps that take turns run ahead of the others: a parity wait must not pass
// on an older phase of its slot.  An h group's turn comes within the ring's
// depth.  A scale warp that waits for stage i - kRingC to be consumed wrote
// stage i - kScaleWarps before, so stage i - kScaleWarps - kRingC is consumed;
// the same group then consumed stage i - 2 kRingC, the slot's phase before.
template <class C>
constexpr bool turns_fit = kHGroups <= C::kRingB && kScaleWarps <= C::kRingC &&
                           (C::kRingC - kScaleWarps) % kHGroups == 0 && C::kRingC % kHGroups == 0;
static_assert(turns_fit<Cfg<1, false>> && turns_fit<Cfg<2, false>> && turns_fit<Cfg<1, true>> &&
                  turns_fit<Cfg<2, true>>,
              "turns stay within the rings");

// A wait without a result: the probe first, and the bounded wait only where no
// earlier one ran out.
__device__ __forceinline__ void wait_or_walk(uint32_t bar, uint32_t parity, unsigned long long limit_ns, bool& dead) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  if (!ok && !dead) dead = !tc::wait_bounded(bar, parity, &g_wgrad_error_word, limit_ns);
}

// MN-major operand with 128-byte swizzle: 64 columns x 8 rows an atom (1024
// bytes), the next 64 columns kBlkBytes on, the next 8 rows 1024 bytes on.
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)(kBlkBytes >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// kind::f16: fp32 accumulators, bf16 x bf16, both MN-major, M = 256, N = W.
__device__ __forceinline__ uint32_t idesc_bf16(int W) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) | ((uint32_t)(W >> 3) << 17) |
         ((uint32_t)(kFeat >> 4) << 24);
}

__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void commit_pair(uint32_t bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(mask)
      : "memory");
}

__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ void sts16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// Four E4M3 codes to four products with p (both halves), as packed bf16.
__device__ __forceinline__ void h4(uint32_t w, unsigned long long p, uint32_t& o0, uint32_t& o1) {
  float a, b, c, d;
  e4m3x2_to_f32(w & 0xFFFFu, a, b);
  e4m3x2_to_f32(w >> 16, c, d);
  f2_unpack(f2_mul(f2_pack(a, b), p), a, b);
  f2_unpack(f2_mul(f2_pack(c, d), p), c, d);
  o0 = pack_bf16(a, b);
  o1 = pack_bf16(c, d);
}

// Geometry of a launch: tile width, row split.
struct Plan {
  int MT;  // accumulators, 256 features each, that share the h of a stage
  int W;
  int split;
};

struct Item {  // one pair's work: a tile and a range of stages
  int n0, k0, st0, st1, part;
};

__device__ __forceinline__ Item item_of(int64_t i, int64_t num_n, int num_k, int F, int W, int split, int stages) {
  Item r;
  r.part = (int)(i % split);
  int64_t mt;
  int nt;
  tile_coords(i / split, num_n, num_k, mt, nt);
  r.n0 = (int)mt * F;
  r.k0 = nt * W;
  r.st0 = (int)((int64_t)stages * r.part / split);
  r.st1 = (int)((int64_t)stages * (r.part + 1) / split);
  return r;
}

// V8: rows of dw (or of the partial sums, where the rows are split) take
// 32-byte stores.
// MT: accumulators per pair; NARROW: W <= 128.
template <int MT, bool NARROW, bool V8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    wgrad_kernel(const __grid_constant__ CUtensorMap tm_d, const __grid_constant__ CUtensorMap tm_c,
                 const uint8_t* __restrict__ scales, int tiled, const float* __restrict__ inv_rms,
                 uint16_t* __restrict__ dw, float* __restrict__ ws, int64_t T, int K, int N, Plan plan,
                 WaitDrill drill) {
  using C = Cfg<MT, NARROW>;
  constexpr int F = MT * kFeat, kRingB = C::kRingB, kRingC = C::kRingC, kMaxG = C::kMaxG;
  constexpr int kStageB = C::kStageB, kStageC = C::kStageC, kStageP = C::kStageP;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + kRingB * MT * kStageA;
  uint8_t* sC = sB + kRingB * kStageB;
  float* sP = reinterpret_cast<float*>(sC + kRingC * kStageC);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sP + kRingC * (kStageP / 4));
  // ab_full (leader: both CTAs' dout and h), ab_empty (each CTA: MMAs done); c_full, p_full (this CTA's codes, scales),
  // c_empty (h made of both); acc_full[2], acc_empty[2] (leader), drain; then the TMEM base word.
  const uint32_t ab_full0 = saddr(bars), ab_empty0 = ab_full0 + 8 * kRingB;
  const uint32_t c_full0 = ab_empty0 + 8 * kRingB, p_full0 = c_full0 + 8 * kRingC, c_empty0 = p_full0 + 8 * kRingC;
  const uint32_t acc_full0 = c_empty0 + 8 * kRingC, acc_empty0 = acc_full0 + 16, drain = acc_empty0 + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kRingB + 3 * kRingC + 5);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t rank;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int64_t pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int W = plan.W, HW = W / 2, split = plan.split;
  const int64_t num_n = (N + F - 1) / F;
  const int num_k = (K + W - 1) / W;
  const int stages = (int)((T + kBT - 1) / kBT);
  const int64_t items = num_n * num_k * split;
  auto wait_warp = [&drill](uint32_t bar, uint32_t parity) {
    return tc::wait_warp(bar, parity, &g_wgrad_error_word, drill.limit_ns);
  };
  auto wait_pair = [&drill](uint32_t bar, uint32_t parity) {  // for arrivals of both CTAs
    return tc::wait_warp<true>(bar, parity, &g_wgrad_error_word, drill.limit_ns);
  };

  if (threadIdx.x == 0) {
    auto init = [](uint32_t bar, uint32_t n, int count) {
      for (int j = 0; j < count; ++j)
        asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar + 8 * j), "r"(n));
    };
    init(ab_full0, 1 + 2 * kHWarps, kRingB);
    init(ab_empty0, 1, kRingB);
    init(c_full0, 1, kRingC);
    init(p_full0, 1, kRingC);
    init(c_empty0, kHWarps, kRingC);
    for (int b = 0; b < 2; ++b) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(acc_full0 + 8 * b));
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 8;" ::"r"(acc_empty0 + 8 * b));
    }
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(drain));
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(tmem_slot)),
                 "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncwarp();
  cluster_sync();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = *tmem_slot;
  pdl_launch_dependents();  // not before this kernel holds its TMEM: a dependent could take it first and wait
  pdl_wait();

  if (warp == 0) {
    Ring<kRingB> q;
    bool ok = true;
    int64_t left = drill.load == 0 ? drill.stage : -1;  // stages before the withheld one
    for (int64_t i = pair; i < items && ok; i += npairs) {
      const Item m = item_of(i, num_n, num_k, F, W, split, stages);
      const int nx = m.n0 + 128 * (int)rank;
      for (int st = m.st0; st < m.st1; ++st, q.next()) {
        if (!q.first && !(ok = wait_warp(ab_empty0 + 8 * q.s, q.phase ^ 1u))) break;
        if (left-- != 0 && elect_one()) {
          if (rank == 0)
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(ab_full0 + 8 * q.s),
                         "r"(2 * MT * kStageA)
                         : "memory");
          const uint32_t fb = map_to_rank(ab_full0 + 8 * q.s, 0), dst = saddr(sA + q.s * MT * kStageA);
#pragma unroll
          for (int a = 0; a < MT; ++a) {
            tma_2d_pair(dst + a * kStageA, &tm_d, nx + a * kFeat, st * kBT, fb);
            tma_2d_pair(dst + a * kStageA + kBlkBytes, &tm_d, nx + a * kFeat + 64, st * kBT, fb);
          }
        }
        __syncwarp();
      }
    }
    // Neither CTA may exit before the commits that arrive here have, nor the pair before its copies have landed: the
    // last commit of each slot shows both.  Once a wait has run out, the pair's copies alone; the last one was then
    // issued a whole limit ago.
    uint32_t ph;
    for (int j = 0; j < kRingB && ok; ++j)
      if (q.last(j, ph)) ok = wait_warp(ab_empty0 + 8 * j, ph);
    if (!ok && rank == 0)
      for (int j = 0; j < kRingB; ++j)
        if (q.last(j, ph) && !wait_warp(ab_full0 + 8 * j, ph)) break;
  } else if (warp == 1) {
    if (rank == 0) {
      // One wait, 4 MT MMAs and one commit a stage, the descriptors by addition: this warp's own time can bound the
      // loop (a second commit a stage cost 26 %).
      Ring<kRingB> q;
      const uint64_t a0 = desc_mn(saddr(sA)), b0 = desc_mn(saddr(sB));
      const uint32_t idesc = idesc_bf16(W);
      int64_t tcount = 0;
      bool ok = true;
      for (int64_t i = pair; i < items && ok; i += npairs, ++tcount) {
        const Item m = item_of(i, num_n, num_k, F, W, split, stages);
        // one accumulator: the two halves of TMEM in turn; two: both, once the tile before is read
        const int b = MT == 1 ? (int)(tcount & 1) : 0;
        const int64_t use = MT == 1 ? tcount / 2 : tcount;
        if (use > 0 && !(ok = wait_pair(acc_empty0 + 8 * b, (uint32_t)(use - 1) & 1u))) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t acc = tmem + 256 * b;
        uint32_t accum = 0;
        for (int st = m.st0; st < m.st1; ++st, q.next()) {
          const uint64_t da = a0 + (uint64_t)((q.s * MT * kStageA) >> 4), db = b0 + (uint64_t)((q.s * kStageB) >> 4);
          if (!(ok = wait_pair(ab_full0 + 8 * q.s, q.phase))) break;
          acquire_shared_cluster();  // the peer's h
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          if (elect_one()) {
#pragma unroll
            for (int j = 0; j < kBT / 16; ++j) {
#pragma unroll
              for (int a = 0; a < MT; ++a)
                asm volatile(
                    "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                    "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(acc + 256 * a),
                    "l"(da + (uint64_t)(128 * j + (a * kStageA >> 4))), "l"(db + (uint64_t)(128 * j)), "r"(idesc),
                    "r"(j > 0 ? 1u : accum));
            }
            commit_pair(ab_empty0 + 8 * q.s, 3);
          }
          __syncwarp();
          accum = 1;
        }
        if (!ok) break;
        if (elect_one()) commit_pair(acc_full0 + 8 * b, 3);
        __syncwarp();
      }
      if (elect_one()) commit_pair(drain, 1);
      __syncwarp();
      (void)wait_warp(drain, 0);
    }
  } else if (warp == 2) {
    Ring<kRingC> q;
    bool ok = true;
    int64_t left = drill.load == 1 ? drill.stage : -1;
    for (int64_t i = pair; i < items && ok; i += npairs) {
      const Item m = item_of(i, num_n, num_k, F, W, split, stages);
      const int kx = m.k0 + HW * (int)rank;
      for (int st = m.st0; st < m.st1; ++st, q.next()) {
        if (!q.first && !(ok = wait_warp(c_empty0 + 8 * q.s, q.phase ^ 1u))) break;
        if (left-- != 0 && elect_one()) {
          asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(c_full0 + 8 * q.s), "r"(kStageC)
                       : "memory");
          tma_2d(saddr(sC + q.s * kStageC), &tm_c, kx, st * kBT, c_full0 + 8 * q.s);
        }
        __syncwarp();
      }
    }
    uint32_t ph;
    for (int j = 0; j < kRingC; ++j)
      if (q.last(j, ph) && !wait_warp(c_full0 + 8 * j, ph)) break;
  } else if (warp < kFirstEpi) {
    // 2^e of the G blocks of this CTA's columns, and rho~ of the rows.  Neighbouring lanes take neighbouring blocks of
    // a row, so that a load instruction touches 32 / G rows' sectors and not 32.
    const int KB = K / kBlock, G = W / 64;
    const uint32_t inv_g = (65536u + G - 1) / G;  // idx / G = idx inv_g >> 16 for idx < 64 G
    Ring<kRingC> q;
    int turn = 0;
    bool ok = true;
    for (int64_t i = pair; i < items && ok; i += npairs) {
      const Item m = item_of(i, num_n, num_k, F, W, split, stages);
      const int kb0 = (m.k0 + HW * (int)rank) / kBlock;
      // this lane's scale bytes: the row in the stage and the offset from the stage's first byte, the same in every
      // stage of the item (a stage is half a row tile of atoms)
      int at[2 * kMaxG], row[2 * kMaxG];
#pragma unroll
      for (int j = 0; j < 2 * kMaxG; ++j) {
        const int idx = lane + 32 * j;
        const int r = (int)((uint32_t)idx * inv_g >> 16), kb = kb0 + idx - r * G;
        row[j] = j < 2 * G && kb < KB ? r : kBT;  // kBT: no such block
        at[j] = tiled ? (r & 31) * 16 + (r >> 5) * 4 + (kb >> 2) * 512 + (kb & 3) : r * KB + kb;
      }
      for (int st = m.st0; st < m.st1; ++st, q.next(), turn = (turn + 1) % kScaleWarps) {
        if (turn != warp - kFirstScale) continue;
        const uint8_t* base = tiled ? scales + (int64_t)(st >> 1) * (KB >> 2) * 512 + (st & 1) * 8
                                    : scales + (int64_t)st * kBT * KB;
        const int rows = (int)min((int64_t)kBT, T - (int64_t)st * kBT);
        uint32_t e[2 * kMaxG];
#pragma unroll
        for (int j = 0; j < 2 * kMaxG; ++j) {
          e[j] = 127u;
          if (row[j] < rows) e[j] = __ldg(base + at[j]);
        }
        float r0 = 0.0f, r1 = 0.0f;  // rows past T: h = 0
        if (lane < rows) r0 = inv_rms != nullptr ? __ldg(inv_rms + (int64_t)st * kBT + lane) : 1.0f;
        if (lane + 32 < rows) r1 = inv_rms != nullptr ? __ldg(inv_rms + (int64_t)st * kBT + lane + 32) : 1.0f;
        if (!q.first && !(ok = wait_warp(c_empty0 + 8 * q.s, q.phase ^ 1u))) break;
        float* dst = sP + q.s * (kStageP / 4);
#pragma unroll
        for (int j = 0; j < 2 * kMaxG; ++j)
          if (j < 2 * G) dst[lane + 32 * j] = e8m0_value(e[j]);
        dst[kBT * kMaxG + lane] = row_factor(r0);  // here, where the loads need to have ended anyway
        dst[kBT * kMaxG + lane + 32] = row_factor(r1);
        __syncwarp();
        if (lane == 0)
          asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(p_full0 + 8 * q.s) : "memory");
      }
    }
  } else if (warp < kFirstH) {
    const int quad = warp & 3;
    int64_t tcount = 0;
    for (int64_t i = pair; i < items; i += npairs, ++tcount) {
      const Item m = item_of(i, num_n, num_k, F, W, split, stages);
      const int b = MT == 1 ? (int)(tcount & 1) : 0;
      if (!wait_warp(acc_full0 + 8 * b, (uint32_t)(MT == 1 ? tcount / 2 : tcount) & 1u)) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const int cols = min(W, K - m.k0);  // a multiple of 32
      for (int ac = 0; ac < MT * cols; ac += 32) {
        const int a = MT > 1 && ac >= cols ? 1 : 0, c = ac - a * cols;  // accumulator, column
        const uint32_t taddr = tmem + 256 * (a + b) + ((uint32_t)(32 * quad) << 16);
        const int n = m.n0 + a * kFeat + 128 * (int)rank + 32 * quad + lane;
        __syncwarp();
        uint32_t v[32];
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
            "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
            : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
              "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
              "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
              "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
            : "r"(taddr + (uint32_t)c));
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
        if (n >= N) {  // a row past the last feature
        } else if (split > 1) {
          float* dst = ws + ((int64_t)m.part * N + n) * K + m.k0 + c;
#pragma unroll
          for (int q = 0; q < 32; q += 8) store32<V8>(dst + q, v + q);
        } else {
          uint16_t* dst = dw + (int64_t)n * K + m.k0 + c;
#pragma unroll
          for (int q = 0; q < 32; q += 16) {
            uint32_t o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
              o[e] = pack_bf16(__uint_as_float(v[q + 2 * e]), __uint_as_float(v[q + 2 * e + 1]));
            store32<V8>(dst + q, o);
          }
        }
      }
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) arrive_remote(map_to_rank(acc_empty0 + 8 * b, 0));
    }
  } else {
    // h: a thread owns one block of 32 columns of one row of the stage, the same place in every stage.  Eight
    // neighbouring lanes take eight rows of one block: their 16-byte loads and stores, both swizzled by the row, fall on
    // all banks.
    const int tid = (threadIdx.x - 32 * kFirstH) % (32 * kHWarps);
    const int group = (warp - kFirstH) / kHWarps;
    const int G = W / 64;
    const int u = tid >> 3, blk = u % G, row = u / G * 8 + (tid & 7);
    const bool mine = row < kBT;
    uint32_t from[2], to[4];  // the block's chunks of 16 bytes: of codes, of h
#pragma unroll
    for (int q = 0; q < 2; ++q)  // 128-byte rows and swizzle, or 64-byte ones
      from[q] = NARROW ? (uint32_t)(row * 64) + (((uint32_t)(2 * blk + q) ^ ((row >> 1) & 3)) << 4)
                       : (uint32_t)(row * 128) + (((uint32_t)(2 * blk + q) ^ (row & 7)) << 4);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      to[q] = (uint32_t)((blk >> 1) * kBlkBytes + row * 128) + (((uint32_t)(4 * (blk & 1) + q) ^ (row & 7)) << 4);
    Ring<kRingB> rb;
    Ring<kRingC> rc;
    int turn = 0;
    // A lane whose wait ran out waits no more but walks on, so that every lane takes part in every warp barrier (a vote
    // a wait, to stop the warp as one, cost 10 % at 2043 x 768 x 768).  Lane 0 arrives for the warp, and once its own
    // wait has run out it arrives no more: what the lanes then read and write is of no consequence.
    bool dead = false;
    for (int64_t i = pair; i < items; i += npairs) {
      const Item m = item_of(i, num_n, num_k, F, W, split, stages);
      for (int st = m.st0; st < m.st1; ++st, rb.next(), rc.next(), turn = (turn + 1) % kHGroups) {
        if (turn != group) continue;
        wait_or_walk(c_full0 + 8 * rc.s, rc.phase, drill.limit_ns, dead);
        wait_or_walk(p_full0 + 8 * rc.s, rc.phase, drill.limit_ns, dead);
        uint4 a, b;
        float pf = 0.0f;
        if (mine) {
          const uint32_t src = saddr(sC + rc.s * kStageC);
          a = lds16(src + from[0]);
          b = lds16(src + from[1]);
          const float* ps = sP + rc.s * (kStageP / 4);
          pf = __fmul_rn(ps[kBT * kMaxG + row], ps[row * G + blk]);
        }
        __syncwarp();
        if (lane == 0 && !dead)
          asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(c_empty0 + 8 * rc.s) : "memory");
        if (!rb.first) wait_or_walk(ab_empty0 + 8 * rb.s, rb.phase ^ 1u, drill.limit_ns, dead);
        if (mine) {
          const uint32_t dst = saddr(sB + rb.s * kStageB);
          const unsigned long long p = f2_pack(pf, pf);
          uint32_t o[8];
          h4(a.x, p, o[0], o[1]);
          h4(a.y, p, o[2], o[3]);
          h4(a.z, p, o[4], o[5]);
          h4(a.w, p, o[6], o[7]);
          sts16(dst + to[0], o[0], o[1], o[2], o[3]);
          sts16(dst + to[1], o[4], o[5], o[6], o[7]);
          h4(b.x, p, o[0], o[1]);
          h4(b.y, p, o[2], o[3]);
          h4(b.z, p, o[4], o[5]);
          h4(b.w, p, o[6], o[7]);
          sts16(dst + to[2], o[0], o[1], o[2], o[3]);
          sts16(dst + to[3], o[4], o[5], o[6], o[7]);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0 && !dead) arrive_remote_release(map_to_rank(ab_full0 + 8 * rb.s, 0));
      }
    }
  }

  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncwarp();
  cluster_sync();
  if (warp == 1) {
    __syncwarp();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
  }
}

// dw = bf16(sum over the split's partial sums, in order): 4 elements a thread,
// the loads of 8 partial sums in flight.
__global__ void __launch_bounds__(256)
    wgrad_join_kernel(const float* __restrict__ ws, int split, int64_t n, uint16_t* __restrict__ dw) {
  pdl_enter();
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < n; i += (int64_t)gridDim.x * 256 * 4) {
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int p0 = 0; p0 < split; p0 += 8) {
      float4 c[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        c[j] = p0 + j < split ? __ldcs(reinterpret_cast<const float4*>(ws + (int64_t)(p0 + j) * n + i))
                              : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        a.x = __fadd_rn(a.x, c[j].x);
        a.y = __fadd_rn(a.y, c[j].y);
        a.z = __fadd_rn(a.z, c[j].z);
        a.w = __fadd_rn(a.w, c[j].w);
      }
    }
    stg8(dw + i, pack_bf16(a.x, a.y), pack_bf16(a.z, a.w));
  }
}

bool encode_2d(CUtensorMap* map, CUtensorMapDataType type, int size, const void* base, int64_t cols, int64_t rows,
               uint32_t box_cols, CUtensorMapSwizzle swizzle) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)(cols * size)};
  cuuint32_t box[2] = {box_cols, (cuuint32_t)kBT};
  cuuint32_t estr[2] = {1, 1};
  return enc(map, type, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MT, bool NARROW>
cudaError_t raise_smem() {
  for (const void* k : {reinterpret_cast<const void*>(wgrad_kernel<MT, NARROW, true>),
                        reinterpret_cast<const void*>(wgrad_kernel<MT, NARROW, false>)}) {
    cudaError_t err = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg<MT, NARROW>::kSmem);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

template <int MT, bool NARROW>
cudaError_t launch_plan(const WgradArgs& a, const Plan& p, int grid, const CUtensorMap& tm_d, const CUtensorMap& tm_c,
                        cudaStream_t s) {
  const uintptr_t dst = reinterpret_cast<uintptr_t>(p.split > 1 ? a.workspace : a.dw);
  auto kern = (dst & 31) == 0 ? wgrad_kernel<MT, NARROW, true> : wgrad_kernel<MT, NARROW, false>;
  return launch_pdl(kern, dim3((unsigned)grid), dim3(kThreads), Cfg<MT, NARROW>::kSmem, s, tm_d, tm_c, a.scales,
                    a.scale_tiled, a.inv_rms, static_cast<uint16_t*>(a.dw), static_cast<float*>(a.workspace), a.T,
                    (int)a.K, (int)a.N, p, a.drill);
}

// CTA pairs that the current device runs at the same time, cached per device.
cudaError_t resident_pairs(int* out) {
  static std::mutex mu;
  static int cache[64] = {0};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  std::lock_guard<std::mutex> lock(mu);
  if (dev >= 0 && dev < 64 && cache[dev] > 0) {
    *out = cache[dev];
    return cudaSuccess;
  }
  if ((err = raise_smem<1, false>()) != cudaSuccess || (err = raise_smem<2, false>()) != cudaSuccess ||
      (err = raise_smem<1, true>()) != cudaSuccess || (err = raise_smem<2, true>()) != cudaSuccess)
    return err;
  int sms = 0;
  if ((err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return err;
  // one CTA an SM in every form
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(sms - sms % 2));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<1, false>::kSmem;
  int clusters = 0;
  if ((err = cudaOccupancyMaxActiveClusters(&clusters, reinterpret_cast<const void*>(wgrad_kernel<1, false, true>),
                                            &cfg)) != cudaSuccess)
    return err;
  if (clusters < 1) return cudaErrorInvalidConfiguration;
  if (dev >= 0 && dev < 64) cache[dev] = clusters;
  *out = clusters;
  return cudaSuccess;
}

constexpr int kPlanPairs = 76;   // pairs of a GB300; the plan must not depend on the device's state
constexpr int kMaxSplit = 64;

// Clocks of a stage, measured at 512 x 512 over 32768 rows: narrow tiles are
// bound by the least time of a chain of MMAs into one accumulator (some 115
// clocks each, 460 a stage) and the making of h beside it.
double stage_clocks(int MT, int W) {
  if (MT == 1) return W == 64 ? 575 : W == 128 ? 590 : W == 192 ? 760 : 846;
  return W == 64 ? 680 : W == 128 ? 690 : W == 192 ? 1000 : 1150;
}

// Accumulators, width and split by estimated clocks, fitted to a sweep of
// plans over sizes from 64 x 4096 x 4096 to 30001 x 416 x 264: the stages, an
// item's start, fill and store (two accumulators store nothing under the next
// tile's MMAs), a join with its parts and its traffic, which past half the L2
// is HBM's (65536 x 4096 x 4096: 1270 us whole, 1310 in four parts of rows).
// 3000 of the join's constant are measured; 6000 stand for its launch and
// workspace, which an eager caller waits for where the kernel is short (2043 x
// 768 x 768: 14.6 us whole and 11.7 in four parts on the device, but 14 and 18
// a call of the host's time; 4096 x 1024 x 1024: 27 whole, 17 in four).  So a
// caller that replays a graph is off the best plan by up to 25 % there, 14 % at
// 2048 x 2048 x 512 and 12 % at 30001 x 416 x 264; at the other 14 sizes swept
// by 10 % at most, at 11 of them by 1 %.
Plan search(int64_t T, int64_t K, int64_t N) {
  const int64_t stages = (T + kBT - 1) / kBT;
  Plan best{1, kMaxW, 1};
  double best_cost = 1e30;
  for (int MT = 1; MT <= 2; ++MT) {
    if (MT == 2 && N <= kFeat) break;
    const int64_t num_n = (N + MT * kFeat - 1) / (MT * kFeat);
    for (int W = kMaxW; W >= 64; W -= 64) {
      if (W > 64 && W - 64 >= K) continue;
      const int64_t tiles = num_n * ((K + W - 1) / W);
      for (int S = 1; S <= kMaxSplit && S <= stages; ++S) {
        const int64_t waves = (tiles * S + kPlanPairs - 1) / kPlanPairs;
        const double item =
            (double)((stages + S - 1) / S) * stage_clocks(MT, W) + (MT == 1 ? 2000 : W <= 128 ? 2500 : 4000);
        const double bytes = 4.0 * S * N * K;
        const double join =
            S > 1 ? 9000 + 100 * S + 300 * std::max(0, S - 8) + (bytes > 64e6 ? 1.3e-3 : 0.52e-3) * bytes : 0;
        const double cost = 7000 + waves * item + join;
        if (cost < best_cost * 0.999) {
          best_cost = cost;
          best = Plan{MT, W, S};
        }
      }
    }
  }
  return best;
}

// The plan of a size, a function of the size alone.  A call asks three times
// and a training loop comes back with the same few sizes, so a thread keeps
// the last ones instead of searching again.
Plan choose(int64_t T, int64_t K, int64_t N) {
  struct Entry {
    int64_t T = -1, K = 0, N = 0;
    Plan plan;
  };
  static thread_local Entry cache[16];
  Entry& e = cache[(T + 5 * (K / kBlock) + 3 * (N / 8)) & 15];
  if (e.T != T || e.K != K || e.N != N) {
    e.T = T;
    e.K = K;
    e.N = N;
    e.plan = search(T, K, N);
  }
  return e.plan;
}

}  // namespace

int64_t wgrad_workspace_bytes(int64_t T, int64_t K, int64_t N) {
  const Plan p = choose(T, K, N);
  return p.split > 1 ? (int64_t)p.split * N * K * 4 : 0;
}

cudaError_t launch_mxnorm_wgrad(const WgradArgs& a, cudaStream_t s) {
  int pairs = 0;
  cudaError_t err = resident_pairs(&pairs);
  if (err != cudaSuccess) return err;
  const Plan p = choose(a.T, a.K, a.N);
  const bool narrow = p.W <= 128;
  CUtensorMap tm_d, tm_c;
  if (!encode_2d(&tm_d, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.dout, a.N, a.T, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_2d(&tm_c, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.codes, a.K, a.T, narrow ? 64 : 128,
                 narrow ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  const int64_t items = ((a.N + p.MT * kFeat - 1) / (p.MT * kFeat)) * ((a.K + p.W - 1) / p.W) * p.split;
  const int grid = (int)(2 * std::min<int64_t>(items, pairs));
  if (p.MT == 1)
    err = narrow ? launch_plan<1, true>(a, p, grid, tm_d, tm_c, s) : launch_plan<1, false>(a, p, grid, tm_d, tm_c, s);
  else
    err = narrow ? launch_plan<2, true>(a, p, grid, tm_d, tm_c, s) : launch_plan<2, false>(a, p, grid, tm_d, tm_c, s);
  if (err != cudaSuccess || p.split == 1) return err;
  const int64_t n = a.N * a.K;
  const int join = persistent_grid(reinterpret_cast<const void*>(wgrad_join_kernel), 256, (n / 4 + 255) / 256);
  return launch_pdl(wgrad_join_kernel, dim3((unsigned)join), dim3(256), 0, s, static_cast<const float*>(a.workspace),
                    p.split, n, static_cast<uint16_t*>(a.dw));
}

cudaError_t read_wgrad_error_word(uint32_t* out, bool clear) {
  unsigned int v = 0;
  cudaError_t err = cudaMemcpyFromSymbol(&v, g_wgrad_error_word, sizeof v);
  if (err != cudaSuccess) return err;
  *out = v;
  if (clear) {
    const unsigned int zero = 0;
    err = cudaMemcpyToSymbol(g_wgrad_error_word, &zero, sizeof zero);
  }
  return err;
}

}  // namespace mxnorm
