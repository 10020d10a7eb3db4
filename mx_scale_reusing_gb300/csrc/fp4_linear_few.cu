// fp4_linear_few.cu -- MXNormLinear's product on FP4 codes for few rows, from
// a single token: the same sum as fp4_linear.cu,
//     out[t, n] = bf16(alpha[t] sum_k x^[t, k] w^[n, k]).
//
// With few rows the weight's bytes bound it.  The operands change sides: the
// weight is the MMA's M side (128 features a CTA), the rows are its N side (R
// = rows of the tile rounded up to 16, at most 128), so the tensor cores do no
// work for rows that are not there and every weight byte is read once.  K runs
// 128 bytes (256 elements) a stage through a TMA ring; where there are few
// feature tiles, the CTAs of a cluster split K and join their fp32 partial
// sums through distributed shared memory, in rank order (the same bits every
// time), each finishing its share of the rows.
//
// 1 x 4096 x 28672 (66 MB of weight, cold) takes 12.2 us back to back, 5.4
// TB/s; 1 x 4096 x 4096 4.9 us, of which the launch, the first bytes' latency
// and the join are most (10.4 us by CTA pairs).
//
// One CTA: warp 0 loads, warp 1 copies scales to TMEM and issues the MMAs (in
// order, one elected lane), warps 2-5 store.  In the epilogue a
// lane is a feature, so a store instruction writes 32 neighbouring outputs of
// one row whatever the alignment of the rows.  Waits are bounded as in
// fp4_linear.cu.
#include <algorithm>
#include <atomic>

#include "fp4_tc.cuh"

namespace mxnorm {

__device__ unsigned int g_fp4_few_error_word = 0u;

namespace {

using namespace fp4;

constexpr int kFeat = 128;       // features per CTA
constexpr int kMaxRows = 128;    // rows per CTA
constexpr int kMaxStages = 8;
constexpr int kThreads = 32 * 6;
constexpr int kSms = 152;
constexpr size_t kSmemOne = 227 * 1024;  // one CTA per SM
constexpr size_t kSmemTwo = 113 * 1024;  // two

__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void prefetch_2d(const CUtensorMap* map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

template <bool NV>
__device__ __forceinline__ void mma_one(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        uint32_t accum) {
  if constexpr (NV)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accum));
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accum));
}

__device__ __forceinline__ void tmem_load16(uint32_t taddr, float (&v)[16]) {
  uint32_t* w = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7]), "=r"(w[8]),
        "=r"(w[9]), "=r"(w[10]), "=r"(w[11]), "=r"(w[12]), "=r"(w[13]), "=r"(w[14]), "=r"(w[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ float4 ld_peer(uint32_t cluster_addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr)
               : "memory");
  return v;
}

__device__ __forceinline__ uint16_t bf16_bits(float v) {
  const __nv_bfloat16 b = __float2bfloat16_rn(v);
  return *reinterpret_cast<const uint16_t*>(&b);
}

// This rank's share of the rows joined over the cluster's S partial sums, in
// rank order: a warp takes a row's 128 features at a time, 4 a lane, and has
// the S loads of U rows in flight.
template <int S>
__device__ __forceinline__ void join_rows(uint32_t part, const float* alpha, int r0, int r1, int n0, int N, int lane,
                                          int warp, uint16_t* out) {
  constexpr int U = 16 / S;
  const int n = n0 + 4 * lane;
  for (int r = r0 + warp * U; r < r1; r += 4 * U) {
    float4 v[U][S];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int p = 0; p < S; ++p)
        v[u][p] = ld_peer(map_to_rank(part + 4 * (min(r + u, r1 - 1) * kFeat + 4 * lane), p));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float4 t = v[u][0];
#pragma unroll
      for (int p = 1; p < S; ++p) {
        t.x = __fadd_rn(t.x, v[u][p].x);
        t.y = __fadd_rn(t.y, v[u][p].y);
        t.z = __fadd_rn(t.z, v[u][p].z);
        t.w = __fadd_rn(t.w, v[u][p].w);
      }
      if (r + u < r1) {
        const float a = alpha[r + u];
        uint16_t* dst = out + (int64_t)(r + u) * N + n;
        const float o0 = __fmul_rn(t.x, a), o1 = __fmul_rn(t.y, a), o2 = __fmul_rn(t.z, a), o3 = __fmul_rn(t.w, a);
        if (n + 3 < N && (reinterpret_cast<uintptr_t>(dst) & 7) == 0) {
          stg8(dst, pack_bf16(o0, o1), pack_bf16(o2, o3));
        } else {
          if (n < N) dst[0] = bf16_bits(o0);
          if (n + 1 < N) dst[1] = bf16_bits(o1);
          if (n + 2 < N) dst[2] = bf16_bits(o2);
          if (n + 3 < N) dst[3] = bf16_bits(o3);
        }
      }
    }
  }
}

// Geometry of a launch, the same on host and device.
struct Few {
  int R;          // rows per CTA: the MMA's N, a multiple of 16
  int stages;     // ring depth
  int tmem_cols;  // power of two
  int split;      // CTAs of a cluster along K
};

template <bool NV>
__host__ __device__ constexpr int stage_bytes(int R) {
  return kFeat * kStepBytes + R * kStepBytes + 2 * kAtoms<NV> * 512;
}
// The partial sums of a split K, R x 128 floats, lie over the ring: they end
// below the barriers since 4 R <= stages (128 + R) for R <= 128 and two stages,
// which the smallest ring has.
constexpr int extra_bytes(int R) { return 1024 + 8 * (2 * kMaxStages + 2) + 4 * R; }
static_assert(((int)kSmemTwo - extra_bytes(kMaxRows)) / stage_bytes<true>(kMaxRows) >= 2 &&
                  4 * kMaxRows <= 2 * (kFeat + kMaxRows),
              "partial sums fit the ring");
template <bool NV>
constexpr int kSfCols = 8 * kAtoms<NV>;  // TMEM columns of a stage's scales, w then x
__host__ __device__ inline int acc_cols(int R) { return R <= 32 ? 32 : (R + 31) & ~31; }

template <bool NV>
__global__ void __launch_bounds__(kThreads)
    fp4_linear_few_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                          const __grid_constant__ CUtensorMap tm_sfx, const __grid_constant__ CUtensorMap tm_sfw,
                          const float* __restrict__ inv_rms, const float* __restrict__ xg,
                          const float* __restrict__ wg, uint16_t* __restrict__ out, int64_t T, int K, int N, Few f,
                          int l2_prefetch, WaitDrill drill) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int R = f.R, stages = f.stages;
  uint8_t* sA = smem;                                        // [stages][128 x 128]
  uint8_t* sB = sA + stages * kFeat * kStepBytes;            // [stages][R x 128]
  uint8_t* sSF = sB + stages * R * kStepBytes;               // [stages][w, x][kAtoms x 512]
  constexpr int sf_bytes = 2 * kAtoms<NV> * 512;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sSF + stages * sf_bytes);
  // bars: full[kMaxStages], empty[kMaxStages], acc_full; the TMEM base word; alpha[R]
  const uint32_t full0 = saddr(bars), empty0 = saddr(bars + kMaxStages), acc_full = saddr(bars + 2 * kMaxStages);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kMaxStages + 1);
  float* alpha = reinterpret_cast<float*>(bars + 2 * kMaxStages + 2);
  float* part = reinterpret_cast<float*>(smem);  // [R][128] partial sums, over the ring once it is done

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = f.split > 1 ? (int)(blockIdx.x % f.split) : 0;  // clusters lie along x
  const int n0 = (int)(blockIdx.x / f.split) * kFeat;
  const int64_t t0 = (int64_t)blockIdx.y * R;
  const int rows = (int)min((int64_t)R, T - t0);
  const int num_kt = (K + kStepElems - 1) / kStepElems;
  auto wait_warp = [&drill](uint32_t bar, uint32_t parity) {
    return tc::wait_warp(bar, parity, &g_fp4_few_error_word, drill.limit_ns);
  };
  const int kt0 = (int)((int64_t)num_kt * rank / f.split), kt1 = (int)((int64_t)num_kt * (rank + 1) / f.split);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(full0 + 8 * s));
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(empty0 + 8 * s));
    }
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(acc_full));
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(tmem_slot)),
                 "r"((uint32_t)f.tmem_cols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = *tmem_slot;
  pdl_launch_dependents();  // not before this kernel holds its TMEM: a dependent could take it first and wait
  const uint32_t sf_base = tmem + acc_cols(R);
  // The weight's first stages may come into L2 while the previous kernel on
  // the stream ends (a hint: mx_device.cuh, prefetch_l2).
  if (l2_prefetch && warp == 0 && lane == 0)
    for (int kt = kt0; kt < min(kt1, kt0 + stages); ++kt) prefetch_2d(&tm_w, kt * kStepBytes, n0);
  pdl_wait();

  bool done = true;  // the accumulators are complete (epilogue warps)
  if (warp == 0) {
    const uint32_t tx = (uint32_t)(kFeat * kStepBytes + R * kStepBytes + sf_bytes);
    int s = 0, filled = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int kt = kt0; kt < kt1; ++kt) {
      if (filled >= stages && !(ok = wait_warp(empty0 + 8 * s, phase ^ 1u))) break;
      if (kt - kt0 != drill.stage && elect_one()) {
        const uint32_t fb = full0 + 8 * s;
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(fb), "r"(tx) : "memory");
        tma_2d(saddr(sA + s * kFeat * kStepBytes), &tm_w, kt * kStepBytes, n0, fb);
        tma_2d(saddr(sB + s * R * kStepBytes), &tm_x, kt * kStepBytes, (int)t0, fb);
        const uint32_t sf = saddr(sSF + s * sf_bytes);
        const int y = 4 * kAtoms<NV> * kt;
        tma_3d(sf, &tm_sfw, 0, y, n0 / 128, fb);
        tma_3d(sf + kAtoms<NV> * 512, &tm_sfx, 0, y, (int)(t0 / 128), fb);
      }
      __syncwarp();
      ++filled;
      if (++s == stages) {
        s = 0;
        phase ^= 1u;
      }
    }
    // every copy issued has landed and every commit has arrived before the CTA may exit: the last commit of each slot
    // shows both; once a wait has run out, the copies alone (the last one was then issued a whole limit ago)
    for (int j = 0; j < min(stages, filled) && ok; ++j) ok = wait_warp(empty0 + 8 * j, j < s ? phase : phase ^ 1u);
    if (!ok)
      for (int j = 0; j < min(stages, filled); ++j)
        if (!wait_warp(full0 + 8 * j, j < s ? phase : phase ^ 1u)) break;
  } else if (warp == 1) {
    const int last_mmas = (K - (num_kt - 1) * kStepElems + 63) / 64;
    const uint64_t a0 = desc_sw128(saddr(sA)), b0 = desc_sw128(saddr(sB)), f0 = desc_atom(saddr(sSF));
    int s = 0;
    uint32_t phase = 0;
    for (int kt = kt0; kt < kt1; ++kt) {
      if (!wait_warp(full0 + 8 * s, phase)) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint64_t sf = f0 + (uint64_t)((s * sf_bytes) >> 4);
      const uint32_t sfa = sf_base + kSfCols<NV> * s, sfb = sfa + 4 * kAtoms<NV>;
      const uint64_t da = a0 + (uint64_t)((s * kFeat * kStepBytes) >> 4), db = b0 + (uint64_t)((s * R * kStepBytes) >> 4);
      const int mmas = kt == num_kt - 1 ? last_mmas : 4;
      if (elect_one()) {
#pragma unroll
        for (int j = 0; j < kAtoms<NV>; ++j) {
          asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(sfa + 4 * j), "l"(sf + (uint64_t)(32 * j)));
          asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(sfb + 4 * j),
                       "l"(sf + (uint64_t)(32 * (kAtoms<NV> + j))));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < mmas)
            mma_one<NV>(tmem, da + (uint64_t)(2 * i), db + (uint64_t)(2 * i), idesc_fp4<NV>(kFeat, R, sf_byte<NV>(i)),
                        sfa + 4 * sf_atom<NV>(i), sfb + 4 * sf_atom<NV>(i), (kt > kt0 || i > 0) ? 1u : 0u);
        commit(empty0 + 8 * s);
      }
      __syncwarp();
      if (++s == stages) {
        s = 0;
        phase ^= 1u;
      }
    }
    if (elect_one()) commit(acc_full);  // and all MMAs and copies are complete before TMEM is freed
    __syncwarp();
    (void)wait_warp(acc_full, 0);
  } else {
    const float g = NV ? __fmul_rn(*xg, *wg) : 1.0f;
    for (int r = threadIdx.x - 64; r < rows; r += kThreads - 64)
      alpha[r] = inv_rms ? __fmul_rn(row_factor(inv_rms[t0 + r]), g) : g;
    asm volatile("bar.sync 1, %0;" ::"n"(kThreads - 64) : "memory");  // the epilogue warps' alphas
    done = wait_warp(acc_full, 0);
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const int quad = warp & 3;
    const uint32_t taddr = tmem + ((uint32_t)(32 * quad) << 16);
    const int feat = 32 * quad + lane;
    const int n = n0 + feat;
    for (int r0 = 0; done && r0 < rows; r0 += 16) {
      float v[16];
      tmem_load16(taddr + r0, v);
      if (f.split > 1) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (r0 + i < rows) part[(r0 + i) * kFeat + feat] = v[i];
      } else if (n < N) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (r0 + i < rows) {
            out[(t0 + r0 + i) * (int64_t)N + n] = bf16_bits(__fmul_rn(v[i], alpha[r0 + i]));
          }
        }
      }
    }
  }

  __syncwarp();
  if (f.split > 1) {
    cluster_sync();  // every rank's partial sums are in its shared memory
    if (warp >= 2) {
      const int per = (rows + f.split - 1) / f.split;
      const int ra = rank * per, rb = min(rows, ra + per);
      uint16_t* o = out + t0 * (int64_t)N;
      const uint32_t pa = saddr(part);
      if (f.split == 2) join_rows<2>(pa, alpha, ra, rb, n0, N, lane, warp - 2, o);
      else if (f.split == 4) join_rows<4>(pa, alpha, ra, rb, n0, N, lane, warp - 2, o);
      else join_rows<8>(pa, alpha, ra, rb, n0, N, lane, warp - 2, o);
    }
    __syncwarp();
    cluster_sync();  // no rank leaves while another reads its sums
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == 1) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"((uint32_t)f.tmem_cols));
  }
}

// CTAs of clusters of `split` that run at once with one CTA an SM.
constexpr int clusters_fit(int split) { return split == 8 ? 120 : split == 4 ? 144 : kSms; }

int64_t few_tiles(int64_t T, int64_t N) { return ((N + kFeat - 1) / kFeat) * ((T + kMaxRows - 1) / kMaxRows); }

template <bool NV>
Few choose(int64_t T, int64_t K, int64_t N, size_t* smem) {
  Few f;
  // one row tile of a multiple of 16 rows, or tiles of 128 (whole scale atoms)
  f.R = T <= kMaxRows ? (int)((T + 15) / 16 * 16) : kMaxRows;
  const int num_kt = (int)((K + kStepElems - 1) / kStepElems);
  const int64_t tiles = few_tiles(T, N);
  // K is split while the CTAs of all tiles still run at once, which fewer do
  // the larger their clusters (clusters_fit).  Up to 32 rows, whose CTAs
  // mostly wait for memory, it goes on to two CTAs an SM.  us: 1 x 4096 x 4096
  // (32 tiles) split 8 4.8, 4 5.1, 2 5.5; 65 x 4096 x 2048 (16 tiles) split 8,
  // in two waves, 10.9, 4 5.9, 2 6.7; 65 x 4096 x 6144 (48 tiles) 4 8.0, 2 7.6.
  // A cluster of eight needs two stages a CTA (1 x 2048 x 1536: 3.5 against
  // 3.1 for four), and short rows of many tiles stay whole (1 x 1024 x 4096:
  // 3.4 against 3.7).
  f.split = 1;
  for (int s = 2; s <= 8 && s <= num_kt; s *= 2) {
    if ((s == 8 && num_kt < 16) || (num_kt < 8 && tiles > 20)) break;
    if (f.R <= 32 ? tiles * s >= 2 * kSms : tiles * s > (s == 2 ? 256 : clusters_fit(s))) break;
    f.split = s;
  }
  const int extra = extra_bytes(f.R);
  const int per = stage_bytes<NV>(f.R);
  // More CTAs than SMs share an SM two by two, with shallower rings, rather
  // than run in two waves (128 x 4096 x 28672: 20.7 us against 26.5).
  const bool two = tiles * f.split > clusters_fit(f.split);
  f.stages = std::min(kMaxStages, (int)(((two ? kSmemTwo : kSmemOne) - extra) / per));
  const int tmem = two ? 256 : 512;
  f.stages = std::min(f.stages, (tmem - acc_cols(f.R)) / kSfCols<NV>);
  f.tmem_cols = 32;
  while (f.tmem_cols < acc_cols(f.R) + f.stages * kSfCols<NV>) f.tmem_cols *= 2;
  *smem = (size_t)(f.stages * per + extra);
  return f;
}

template <bool NV>
cudaError_t launch_few(const Fp4LinearArgs& a, cudaStream_t s) {
  size_t smem = 0;
  const Few f = choose<NV>(a.T, a.K, a.N, &smem);
  CUtensorMap tm[4];
  if (!encode_codes(&tm[0], a.x_codes, a.T, a.K, f.R) || !encode_codes(&tm[1], a.w_codes, a.N, a.K, kFeat) ||
      !encode_scales(&tm[2], a.x_scales, a.T, a.K, NV) || !encode_scales(&tm[3], a.w_scales, a.N, a.K, NV))
    return cudaErrorInvalidValue;
  auto kern = fp4_linear_few_kernel<NV>;
  static std::atomic<bool> ready[64];  // the shared-memory limit is raised once per device
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64 || !ready[dev].load(std::memory_order_acquire)) {
    if ((err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemOne)) != cudaSuccess)
      return err;
    if (dev >= 0 && dev < 64) ready[dev].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((a.N + kFeat - 1) / kFeat) * f.split), (unsigned)((a.T + f.R - 1) / f.R));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)f.split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, tm[0], tm[1], tm[2], tm[3], a.inv_rms, a.xg, a.wg,
                            static_cast<uint16_t*>(a.out), a.T, (int)a.K, (int)a.N, f,
                            is_device_memory(a.w_codes) ? 1 : 0, a.drill);
}

}  // namespace

// Up to 64 rows the weight's bytes bound the product and this kernel reads
// them once whatever N is.  Above, the pairs walk all of K where this kernel
// splits it: it wins while K is long for its tiles' number and rows (us, this
// kernel / CTA pairs: 200 x 4096 x 2048 7.4 / 8.3, 200 x 8192 x 4096 11.0 /
// 13.2, 512 x 14336 x 3200 19.1 / 20.3, 65 x 4096 x 6144 7.6 / 8.7; but 200 x
// 2048 x 2048 6.7 / 6.1, 200 x 4096 x 6144 11.1 / 9.1, 512 x 1024 x 1024 6.8 /
// 4.7, 512 x 14336 x 4096 21.9 / 20.8).
cudaError_t launch_fp4_linear(const Fp4LinearArgs& a, cudaStream_t s) {
  const int64_t num_kt = (a.K + kStepElems - 1) / kStepElems;
  const int64_t rows = a.T <= kMaxRows ? (a.T + 15) / 16 * 16 : (a.T + kMaxRows - 1) / kMaxRows * kMaxRows;
  if (a.T <= 64 || (num_kt > 8 && (a.N + kFeat - 1) / kFeat * rows <= 2 * kMaxRows * num_kt))
    return a.nvfp4 ? launch_few<true>(a, s) : launch_few<false>(a, s);
  return launch_fp4_linear_many(a, s);
}

cudaError_t read_fp4_few_error_word(uint32_t* out, bool clear) {
  unsigned int v = 0;
  cudaError_t err = cudaMemcpyFromSymbol(&v, g_fp4_few_error_word, sizeof v);
  if (err != cudaSuccess) return err;
  *out = v;
  if (clear) {
    const unsigned int zero = 0;
    err = cudaMemcpyToSymbol(g_fp4_few_error_word, &zero, sizeof zero);
  }
  return err;
}

}  // namespace mxnorm
