// fp4_linear.cu -- MXNormLinear's product on FP4 codes, many rows:
//     out[t, n] = bf16(alpha[t] sum_k x^[t, k] w^[n, k]),
// alpha[t] = RN(inv_rms[t] RN(g_x g_w)), x^ and w^ the E2M1 codes times their
// block scales (MXFP4: E8M0 per 32 elements; NVFP4: UE4M3 per 16, with the
// fp32 tensor scales g_x and g_w taken out of the sum).  The block scales are
// applied by the tensor cores (tcgen05 kind::mxf4 / kind::mxf4nvf4), which
// accumulate exact products in fp32; alpha commutes with the sum over k and
// is applied once per output in the epilogue.
//
// Tiling as the MXFP8 kernel (mxnorm_linear.cu): 256 x 256 output tiles by a
// pair of CTAs (cta_group::2, M = 256, N = 256), persistent pairs, K staged
// 128 bytes (256 elements) at a time through a ring, one instruction per 64
// elements.  A stage holds this CTA's 128 x rows, its half of the tile's 256
// w rows, and the scale atoms of those 256 elements (2 atoms of 512 bytes a
// 128-row tile for MXFP4, 4 for NVFP4; own x tile, both w tiles).  Roles:
//   warp 0         TMA producer (both CTAs), completing on the leader's
//                  "full" barrier;
//   warp 1         leader: MMA issuer, a stage at a time once "sf_full" shows
//                  its scales in TMEM; commits to both CTAs' "empty", and to
//                  "acc_full" after a tile's last stage;
//   warp 2         leader: scale copier (tcgen05.cp of both CTAs' atoms), so
//                  that the copies overlap the MMAs in flight;
//   warps 3-10     epilogue, two per TMEM lane quadrant with 128 columns
//                  each: all columns read and TMEM handed back before the
//                  scaling, rounding and stores.
// TMEM (512 columns): accumulators 0-255, ring stage s's scales at
// 256 + s kSfCols: A atoms j at 4 j, then B atoms j of both w tiles at
// 4 kAtoms + 8 j (the two tiles' words side by side, as N = 256 reads them).
// Rows and scale atoms past T, N or K load as zeros (TMA): zero codes times
// zero scales add nothing.  Every mbarrier wait is bounded (2 s); on expiry
// bit 0 of the error word is set and the pair winds down after its own copies
// and MMAs.
// 65536 x 4096 x 4096, replayed from a graph: NVFP4 332 to 350 us, 6300 to
// 6600 TFLOP/s, MXFP4 324 to 338; single calls 366 to 380 us.  A library's
// NVFP4 product takes 300 us on the same chip, so what follows is where the
// time goes and no floor.  A stage writes 38 KB (NVFP4) and its MMAs and scale
// copies read 38 KB, some 600 clocks of shared memory's 128 bytes a clock
// beside 512 of tensor time; 656 are measured.  Some 1000 more a tile pass
// while the accumulators are handed over: a second set (256 more columns) has
// no room in TMEM beside any scales, half a set would have with two or three
// scale slots instead of the ring's five.  Neither that nor instructions of
// K = 96 is built, so neither is timed.  Of 332 us, leaving out the output's
// stores gave 286 and leaving out the scale copies 300.  Swapping pieces
// between lanes so that a store fills whole lines was slower (4096 x 4096 x
// 4096: 30.7 us against 29.5).
#include <algorithm>

#include "fp4_tc.cuh"

namespace mxnorm {

__device__ unsigned int g_fp4_linear_error_word = 0u;

namespace {

using namespace fp4;

constexpr int BM = 128, BN = 256, BK = kStepBytes;
constexpr int kStageA = BM * BK;
constexpr int kStageB = (BN / 2) * BK;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (3 + kEpiWarps);
constexpr uint32_t kTmemCols = 512;
constexpr int kStages = 5;

template <bool NV>
struct Cfg {
  static constexpr int kAtoms = fp4::kAtoms<NV>;
  static constexpr int kSfBytes = 3 * kAtoms * 512;         // own x tile, both w tiles
  static constexpr int kSfCols = 12 * kAtoms;               // TMEM columns of a stage's scales
  static constexpr int kStageBytes = kStageA + kStageB + kSfBytes;
  static_assert(256 + kStages * kSfCols <= (int)kTmemCols, "accumulators and scales fit TMEM");
};

// Unaligned rows: a warp's 32 rows x 64 columns pass through shared memory
// (33 words a row) so that a store instruction writes along one row.
constexpr int kStageOutWords = 32 * 33;

template <bool NV>
constexpr size_t smem_bytes() {
  return 1024 + (size_t)kStages * Cfg<NV>::kStageBytes + (size_t)kEpiWarps * kStageOutWords * 4 + 256;
}
static_assert(smem_bytes<true>() <= 232448, "shared memory of a CTA");

template <bool NV>
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         uint32_t accum) {
  if constexpr (NV)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accum));
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accum));
}

// 3-D tiled TMA load of scale atoms (128 bytes x 4 rows an atom x row tile).
__device__ __forceinline__ void tma_3d_pair(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, "
      "{%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void commit_pair(uint32_t bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(mask)
      : "memory");
}

// A lane's row of `cols` (<= 128) outputs in 16-column pieces; rows start
// 32-byte (V8) or 16-byte aligned and N is a multiple of 16 or 8.
template <bool V8>
__device__ __forceinline__ void store_row(uint16_t* dst, const uint32_t (&o)[64], int cols) {
#pragma unroll
  for (int q = 0; q < 64; q += 8) {
    if (V8 ? 2 * q < cols : 2 * q + 8 < cols) store32<V8>(dst + 2 * q, o + q);
    else if (!V8 && 2 * q < cols) stg16(dst + 2 * q, o[q], o[q + 1], o[q + 2], o[q + 3]);
  }
}

// The warp's 32 rows x 128 columns for rows of any alignment, 64 columns at a
// time through shared memory; `rows` and `cols` are how many are stored.
__device__ __forceinline__ void store_block_any(uint16_t* out, int64_t row0, int rows, int64_t N, int c0, int cols,
                                                const uint32_t (&o)[64], uint32_t* buf, int lane) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int i = 0; i < 32; ++i) buf[lane * 33 + i] = o[32 * h + i];
    __syncwarp();
    const int left = cols - 64 * h;
    for (int r = 0; r < rows; ++r) {
      uint16_t* dst = out + (row0 + r) * N + c0 + 64 * h;
      const uint16_t* src = reinterpret_cast<const uint16_t*>(buf + r * 33);
      if (lane < left) dst[lane] = src[lane];
      if (lane + 32 < left) dst[lane + 32] = src[lane + 32];
    }
    __syncwarp();
  }
}

// One pair's work: a tile of 256 rows x 256 features, or a half of one (128
// features).  The tiles past the last whole wave are halved where that gives
// each pair at most one half: a half takes about two thirds of a tile's time
// (4096 x 4096 x 4096, 256 tiles on 76 pairs: 28.8 us, 27.3 halved; 2200 x
// 4096 x 1024, 36 tiles: 10.2 and 9.5).
struct Work {
  int64_t mt;  // 256-row tile
  int n0;      // first feature
  bool full;
};
__device__ __forceinline__ Work work_of(int64_t i, int64_t whole, int64_t num_m, int num_n) {
  Work w;
  int nt;
  w.full = i < whole;
  tile_coords(w.full ? i : whole + (i - whole) / 2, num_m, num_n, w.mt, nt);
  w.n0 = nt * BN + (w.full ? 0 : (int)((i - whole) & 1) * (BN / 2));
  return w;
}

// STORE: 2 rows 32-byte aligned, 1 rows 16-byte aligned, 0 any alignment.
// whole: tiles that are not halved.
template <bool NV, int STORE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    fp4_linear_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                      const __grid_constant__ CUtensorMap tm_wh, const __grid_constant__ CUtensorMap tm_sfx,
                      const __grid_constant__ CUtensorMap tm_sfw,
                      const float* __restrict__ inv_rms, const float* __restrict__ xg, const float* __restrict__ wg,
                      uint16_t* __restrict__ out, int64_t T, int K, int N, int64_t whole, WaitDrill drill) {
  using C = Cfg<NV>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + kStages * kStageA;
  uint8_t* sSF = sB + kStages * kStageB;
  uint32_t* sOut = reinterpret_cast<uint32_t*>(sSF + kStages * C::kSfBytes);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sOut + kEpiWarps * kStageOutWords);
  // bars: full, empty, sf_full [kStages] each, then acc_full, acc_empty, drain, drain_sf; the TMEM base word.
  const uint32_t full0 = saddr(bars), empty0 = saddr(bars + kStages), sf_full0 = saddr(bars + 2 * kStages);
  const uint32_t acc_full = saddr(bars + 3 * kStages), acc_empty = saddr(bars + 3 * kStages + 1);
  const uint32_t drain = saddr(bars + 3 * kStages + 2), drain_sf = saddr(bars + 3 * kStages + 3);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 3 * kStages + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t rank;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int64_t pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int num_n = (N + BN - 1) / BN, num_kt = (K + 2 * BK - 1) / (2 * BK);
  const int last_mmas = (K - (num_kt - 1) * 2 * BK + 63) / 64;  // MMAs of the last stage
  const int64_t num_m = (T + 2 * BM - 1) / (2 * BM);
  const int64_t items = whole + 2 * (num_m * num_n - whole);
  auto wait_warp = [&drill](uint32_t bar, uint32_t parity) {
    return tc::wait_warp(bar, parity, &g_fp4_linear_error_word, drill.limit_ns);
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(full0 + 8 * s));
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(empty0 + 8 * s));
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(sf_full0 + 8 * s));
    }
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(acc_full));
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(acc_empty), "r"(2 * kEpiWarps));
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(drain));
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(drain_sf));
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(tmem_slot)),
                 "r"(kTmemCols));
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
    Ring<kStages> q;
    bool ok = true;
    int64_t left = drill.stage;  // stages before the withheld one
    for (int64_t i = pair; i < items && ok; i += npairs) {
      const Work m = work_of(i, whole, num_m, num_n);
      const int xtile = (int)(2 * m.mt) + (int)rank;  // 128-row tile of x
      const int wtile = m.n0 / 128;                   // and of w
      const int bytes = m.full ? C::kStageBytes : C::kStageBytes - kStageB / 2 - C::kAtoms * 512;
      for (int kt = 0; kt < num_kt; ++kt, q.next()) {
        if (!q.first && !(ok = wait_warp(empty0 + 8 * q.s, q.phase ^ 1u))) break;
        if (left-- != 0 && elect_one()) {
          const uint32_t fb = map_to_rank(full0 + 8 * q.s, 0);
          if (rank == 0)
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(full0 + 8 * q.s),
                         "r"(2 * bytes)
                         : "memory");
          tma_2d_pair(saddr(sA + q.s * kStageA), &tm_x, kt * BK, xtile * BM, fb);
          if (m.full) tma_2d_pair(saddr(sB + q.s * kStageB), &tm_w, kt * BK, m.n0 + (int)rank * (BN / 2), fb);
          else tma_2d_pair(saddr(sB + q.s * kStageB), &tm_wh, kt * BK, m.n0 + (int)rank * (BN / 4), fb);
          const uint32_t sf = saddr(sSF + q.s * C::kSfBytes);
          const int y = 4 * C::kAtoms * kt;
          tma_3d_pair(sf, &tm_sfx, 0, y, xtile, fb);
          tma_3d_pair(sf + C::kAtoms * 512, &tm_sfw, 0, y, wtile, fb);
          if (m.full) tma_3d_pair(sf + 2 * C::kAtoms * 512, &tm_sfw, 0, y, wtile + 1, fb);
        }
        __syncwarp();
      }
    }
    // Neither CTA may exit before the commits that arrive here have, nor the pair before its copies have landed: the
    // last commit of each slot shows both.  Once a wait has run out, the pair's copies alone; the last one was then
    // issued a whole limit ago.
    uint32_t ph;
    for (int j = 0; j < kStages && ok; ++j)
      if (q.last(j, ph)) ok = wait_warp(empty0 + 8 * j, ph);
    if (!ok && rank == 0)
      for (int j = 0; j < kStages; ++j)
        if (q.last(j, ph) && !wait_warp(full0 + 8 * j, ph)) break;
  } else if (warp == 1) {
    if (rank == 0) {
      Ring<kStages> q;
      const uint64_t a0 = desc_sw128(saddr(sA)), b0 = desc_sw128(saddr(sB));
      int64_t tcount = 0;
      bool ok = true;
      for (int64_t i = pair; i < items && ok; i += npairs, ++tcount) {
        const int n = i < whole ? BN : BN / 2;
        if (tcount > 0 &&
            !(ok = tc::wait_warp<true>(acc_empty, (uint32_t)((tcount - 1) & 1), &g_fp4_linear_error_word,
                                       drill.limit_ns)))
          break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        for (int kt = 0; kt < num_kt; ++kt, q.next()) {
          if (!(ok = wait_warp(sf_full0 + 8 * q.s, q.phase))) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint32_t tsf = tmem + 256 + C::kSfCols * q.s;
          const uint64_t da = a0 + (uint64_t)((q.s * kStageA) >> 4), db = b0 + (uint64_t)((q.s * kStageB) >> 4);
          const int mmas = kt == num_kt - 1 ? last_mmas : 4;
          if (elect_one()) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (j < mmas)
                mma_pair<NV>(tmem, da + (uint64_t)(2 * j), db + (uint64_t)(2 * j),
                             idesc_fp4<NV>(2 * BM, n, sf_byte<NV>(j)), tsf + 4 * sf_atom<NV>(j),
                             tsf + 4 * C::kAtoms + 8 * sf_atom<NV>(j), (kt | j) ? 1u : 0u);
            commit_pair(empty0 + 8 * q.s, 3);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (elect_one()) commit_pair(acc_full, 3);
        __syncwarp();
      }
      if (elect_one()) commit_pair(drain, 1);  // all MMAs complete before TMEM is freed
      __syncwarp();
      (void)wait_warp(drain, 0);
    }
  } else if (warp == 2) {
    if (rank == 0) {
      // Slot s of TMEM is free once full[s] shows the stage's next use: the
      // producer refilled it only after the MMAs that read the slot.
      Ring<kStages> q;
      const uint64_t s0 = desc_atom(saddr(sSF));
      const int64_t my_items = pair < items ? (items - 1 - pair) / npairs + 1 : 0;
      const int64_t my_whole = pair < whole ? (whole - 1 - pair) / npairs + 1 : 0;  // the whole tiles come first
      const int64_t total = my_items * num_kt;
      for (int64_t it = 0; it < total; ++it, q.next()) {
        const bool full = it < my_whole * num_kt;
        if (!wait_warp(full0 + 8 * q.s, q.phase)) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t tsf = tmem + 256 + C::kSfCols * q.s;
        const uint64_t sf = s0 + (uint64_t)((q.s * C::kSfBytes) >> 4);
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < C::kAtoms; ++j) {
            asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tsf + 4 * j),
                         "l"(sf + (uint64_t)(32 * j)));
            asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tsf + 4 * C::kAtoms + 8 * j),
                         "l"(sf + (uint64_t)(32 * (C::kAtoms + j))));
            if (full)
              asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tsf + 4 * C::kAtoms + 8 * j + 4),
                           "l"(sf + (uint64_t)(32 * (2 * C::kAtoms + j))));
          }
          commit_pair(sf_full0 + 8 * q.s, 1);
        }
        __syncwarp();
      }
      if (elect_one()) commit_pair(drain_sf, 1);
      __syncwarp();
      (void)wait_warp(drain_sf, 0);
    }
  } else {
    const int quad = warp & 3;
    const int half = (warp - 3) / 4;
    const uint32_t acc_empty_leader = map_to_rank(acc_empty, 0);
    const float g = NV ? __fmul_rn(*xg, *wg) : 1.0f;
    int64_t tcount = 0;
    for (int64_t i = pair; i < items; i += npairs, ++tcount) {
      const Work m = work_of(i, whole, num_m, num_n);
      if (!wait_warp(acc_full, (uint32_t)(tcount & 1))) break;
      if (!m.full && half) {  // no columns for this warp
        if (lane == 0) arrive_remote(acc_empty_leader);
        continue;
      }
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t taddr = tmem + ((uint32_t)(32 * quad) << 16) + (uint32_t)(128 * half);
      uint32_t v[128];
      tmem_load64(taddr, *reinterpret_cast<uint32_t(*)[64]>(v));
      tmem_load64(taddr + 64, *reinterpret_cast<uint32_t(*)[64]>(v + 64));
      asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) arrive_remote(acc_empty_leader);
      const int64_t row0 = (2 * m.mt + rank) * BM + 32 * quad;
      const int64_t row = row0 + lane;
      const int c0 = m.n0 + 128 * half;
      const int cols = min(128, N - c0);
      float r = g;
      if (inv_rms != nullptr) r = row < T ? __fmul_rn(row_factor(inv_rms[row]), g) : 0.0f;
      uint32_t o[64];
      scale_pack64(*reinterpret_cast<uint32_t(*)[64]>(v), r, o);
      scale_pack64(*reinterpret_cast<uint32_t(*)[64]>(v + 64), r, o + 32);
      if constexpr (STORE == 0) {
        const int rows = (int)min((int64_t)32, T - row0);
        if (cols > 0 && rows > 0)
          store_block_any(out, row0, rows, N, c0, cols, o, sOut + (warp - 3) * kStageOutWords, lane);
      } else {
        if (row < T) store_row<STORE == 2>(out + row * (int64_t)N + c0, o, cols);
      }
    }
  }

  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncwarp();
  cluster_sync();
  if (warp == 1) {
    __syncwarp();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
  }
}

// CTA pairs that the current device runs at the same time, cached per device.
cudaError_t resident_pairs(const void* kern, size_t smem, int variant, int* out) {
  static std::mutex mu;
  static int cache[6][64] = {{0}};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  std::lock_guard<std::mutex> lock(mu);
  if (dev >= 0 && dev < 64 && cache[variant][dev] > 0) {
    *out = cache[variant][dev];
    return cudaSuccess;
  }
  if ((err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess)
    return err;
  int sms = 0;
  if ((err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(sms - sms % 2));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  int clusters = 0;
  if ((err = cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg)) != cudaSuccess) return err;
  if (clusters < 1) return cudaErrorInvalidConfiguration;
  if (dev >= 0 && dev < 64) cache[variant][dev] = clusters;
  *out = clusters;
  return cudaSuccess;
}

template <bool NV, int STORE>
cudaError_t launch_store(const Fp4LinearArgs& a, const CUtensorMap (&tm)[5], cudaStream_t s) {
  auto kern = fp4_linear_kernel<NV, STORE>;
  int co_resident = 0;
  cudaError_t err =
      resident_pairs(reinterpret_cast<const void*>(kern), smem_bytes<NV>(), 3 * (NV ? 1 : 0) + STORE, &co_resident);
  if (err != cudaSuccess) return err;
  const int64_t tiles = ((a.T + 2 * BM - 1) / (2 * BM)) * ((a.N + BN - 1) / BN);
  const int64_t rest = tiles % co_resident;
  const int64_t whole = 2 * rest <= co_resident ? tiles - rest : tiles;
  const int grid = (int)(2 * std::min<int64_t>(whole + 2 * (tiles - whole), co_resident));
  return launch_pdl(kern, dim3((unsigned)grid), dim3(kThreads), smem_bytes<NV>(), s, tm[0], tm[1], tm[2], tm[3], tm[4],
                    a.inv_rms, a.xg, a.wg, static_cast<uint16_t*>(a.out), a.T, (int)a.K, (int)a.N, whole, a.drill);
}

template <bool NV>
cudaError_t launch_many(const Fp4LinearArgs& a, cudaStream_t s) {
  CUtensorMap tm[5];
  if (!encode_codes(&tm[0], a.x_codes, a.T, a.K, BM) || !encode_codes(&tm[1], a.w_codes, a.N, a.K, BN / 2) ||
      !encode_codes(&tm[2], a.w_codes, a.N, a.K, BN / 4) || !encode_scales(&tm[3], a.x_scales, a.T, a.K, NV) ||
      !encode_scales(&tm[4], a.w_scales, a.N, a.K, NV))
    return cudaErrorInvalidValue;
  if (a.N % 16 == 0 && (reinterpret_cast<uintptr_t>(a.out) & 31) == 0) return launch_store<NV, 2>(a, tm, s);
  if (a.N % 8 == 0) return launch_store<NV, 1>(a, tm, s);
  return launch_store<NV, 0>(a, tm, s);
}

}  // namespace

cudaError_t launch_fp4_linear_many(const Fp4LinearArgs& a, cudaStream_t s) {
  return a.nvfp4 ? launch_many<true>(a, s) : launch_many<false>(a, s);
}

cudaError_t read_fp4_linear_error_word(uint32_t* out, bool clear) {
  unsigned int v = 0;
  cudaError_t err = cudaMemcpyFromSymbol(&v, g_fp4_linear_error_word, sizeof v);
  if (err != cudaSuccess) return err;
  *out = v;
  if (clear) {
    const unsigned int zero = 0;
    err = cudaMemcpyToSymbol(g_fp4_linear_error_word, &zero, sizeof zero);
  }
  return err;
}

}  // namespace mxnorm
