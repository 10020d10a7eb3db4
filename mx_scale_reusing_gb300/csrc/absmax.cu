// absmax.cu -- the largest magnitude of a tensor or of a gain-folded weight,
// and the NVFP4 tensor scale derived from it (RN(a / 2688), a the largest
// finite magnitude; 1 where that quotient is 0, for gain-folded values below
// 2688 2^-150 too).
//
// Non-negative floats order like their bits, so a maximum is an integer
// maximum of the magnitudes' bits (NaN above Inf above every finite value;
// the scale skips both).  Bound by HBM at 2 bytes an element, a thread with 64
// to 128 bytes of loads in flight: 35.1 us at 28672 x 4096, the copy peak; with
// gains, a product and a test an element more, 40.6.  Up to kSmallElems
// elements one cluster of 8 CTAs does it all, joining through distributed
// shared memory: one launch (3.2 us at 768 x 768) where the wide form zeroes
// the result first, takes an atomic a CTA and converts the scale after.
#include <numeric>

#include "launch_fp4.h"
#include "mx_row.cuh"

namespace mxnorm {
namespace {

constexpr int kThreads = 256;        // of a CTA of the wide form
constexpr int kSmallThreads = 1024;  // of the cluster's
constexpr int kCluster = 8;
constexpr int64_t kSmallElems = 1 << 20;

struct FlatSrc {  // n values from x
  const uint16_t* x;
  int64_t n;
};
struct GainSrc {  // the rows of w[n, k] g_k
  const uint16_t* w;
  int64_t N;
  int K;
  const float* gamma;  // or null (ones)
  float c;
  int L;  // lanes that walk a row side by side: gcd(K / 16, 32)
};

template <bool FINITE>
__device__ __forceinline__ uint32_t mag(float v) {
  const uint32_t b = __float_as_uint(v) & 0x7FFFFFFFu;
  return !FINITE || b < 0x7F800000u ? b : 0u;
}

// Thread `tid` of `nthreads`.
template <bool FINITE>
__device__ __forceinline__ uint32_t scan(const FlatSrc& s, int64_t tid, int64_t nthreads) {
  uint32_t m = 0u;
  const bool vec = (reinterpret_cast<uintptr_t>(s.x) & 15) == 0;
  const int64_t nv = vec ? s.n / 8 : 0;
  for (int64_t i = tid; i < nv; i += 4 * nthreads) {
    uint4 t[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      t[u] = make_uint4(0u, 0u, 0u, 0u);
      if (i + u * nthreads < nv) t[u] = ldg_stream16(s.x + 8 * (i + u * nthreads));
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t w[4] = {t[u].x, t[u].y, t[u].z, t[u].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) m = max(m, max(mag<FINITE>(bf16lo(w[q])), mag<FINITE>(bf16hi(w[q]))));
    }
  }
  for (int64_t i = 8 * nv + tid; i < s.n; i += nthreads) m = max(m, mag<FINITE>(bf16lo(s.x[i])));
  return m;
}

template <bool FINITE>
__device__ __forceinline__ uint32_t scan(const GainSrc& s, int64_t tid, int64_t nthreads) {
  constexpr int VEC = 16, ROWS = 4;
  const int strips = s.K / (VEC * s.L);
  const int lane = (int)(tid & 31), rows_per_warp = 32 / s.L;
  const int64_t warp = tid >> 5, warps = nthreads >> 5;
  const int64_t row_groups = (s.N + rows_per_warp - 1) / rows_per_warp;
  uint32_t m = 0u;
  // warps share out the strips, then the rows of a strip
  for (int64_t strip = warp % strips; strip < strips; strip += warps) {
    const int64_t first = warp / strips, step = max((int64_t)1, warps / strips);
    const int col = (int)(strip * s.L + lane % s.L) * VEC;
    float g[VEC];
#pragma unroll
    for (int q = 0; q < VEC / 4; ++q) {
      float4 t = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
      if (s.gamma != nullptr) t = __ldg(reinterpret_cast<const float4*>(s.gamma + col) + q);
      g[4 * q] = __fmul_rn(s.c, t.x);
      g[4 * q + 1] = __fmul_rn(s.c, t.y);
      g[4 * q + 2] = __fmul_rn(s.c, t.z);
      g[4 * q + 3] = __fmul_rn(s.c, t.w);
    }
    if (first >= step) continue;  // warps left over when the strips do not divide them
    for (int64_t rg = first; rg < row_groups; rg += ROWS * step) {
      uint32_t buf[ROWS][VEC / 2];
#pragma unroll
      for (int u = 0; u < ROWS; ++u) {
        const int64_t r = (rg + u * step) * rows_per_warp + lane / s.L;
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) buf[u][i] = 0u;
        if (r < s.N) load_lane<VEC, false>(s.w + r * (int64_t)s.K + col, buf[u]);
      }
#pragma unroll
      for (int u = 0; u < ROWS; ++u)
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i)
          m = max(m, max(mag<FINITE>(__fmul_rn(bf16lo(buf[u][i]), g[2 * i])),
                         mag<FINITE>(__fmul_rn(bf16hi(buf[u][i]), g[2 * i + 1]))));
    }
  }
  return m;
}

// The CTA's maximum, in thread 0.
template <int THREADS>
__device__ __forceinline__ uint32_t cta_max(uint32_t m, uint32_t* red) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int i = 1; i < THREADS / 32; ++i) m = max(m, red[i]);
  return m;
}

__device__ __forceinline__ float scale_of(uint32_t bits) {
  const float g = __fdiv_rn(__uint_as_float(bits), 2688.0f);
  return g > 0.0f ? g : 1.0f;
}

// Starts as an ordinary launch, after everything before it on the stream; the
// scan below may start while it runs (the input is complete by then) and waits
// for it only before its first atomic.
__global__ void zero_word_kernel(unsigned int* out) {
  pdl_launch_dependents();
  *out = 0u;
}

template <class Src, bool FINITE>
__global__ void __launch_bounds__(kThreads) absmax_wide_kernel(Src s, unsigned int* out) {
  __shared__ uint32_t red[kThreads / 32];
  pdl_launch_dependents();
  const uint32_t m = cta_max<kThreads>(
      scan<FINITE>(s, (int64_t)blockIdx.x * kThreads + threadIdx.x, (int64_t)gridDim.x * kThreads), red);
  if (threadIdx.x == 0) {
    pdl_wait();  // *out is zeroed
    atomicMax(out, m);
  }
}

template <class Src, bool FINITE, bool TO_SCALE>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kSmallThreads)
    absmax_small_kernel(Src s, float* out) {
  __shared__ uint32_t red[kSmallThreads / 32];
  __shared__ uint32_t all[kCluster];
  // CTA 0 has to have started before another one stores to its shared memory: every CTA says so here, the wait comes
  // after the scan, where it costs nothing.
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  pdl_enter();
  uint32_t m = cta_max<kSmallThreads>(
      scan<FINITE>(s, (int64_t)blockIdx.x * kSmallThreads + threadIdx.x, kCluster * kSmallThreads), red);
  asm volatile("barrier.cluster.wait;" ::: "memory");
  if (threadIdx.x == 0) {
    uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(&all[blockIdx.x])), there;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(there) : "r"(dst));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(there), "r"(m) : "memory");
  }
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    for (int i = 0; i < kCluster; ++i) m = max(m, all[i]);
    *out = TO_SCALE ? scale_of(m) : __uint_as_float(m);
  }
}

__global__ void scale_from_amax_kernel(float* g) {
  pdl_enter();
  *g = scale_of(*reinterpret_cast<const unsigned int*>(g));
}

// TO_SCALE: the tensor scale of the finite values, else the maximum itself.
template <class Src, bool TO_SCALE>
cudaError_t launch(const Src& src, int64_t elems, float* out, cudaStream_t s) {
  if (elems <= kSmallElems)
    return launch_pdl(absmax_small_kernel<Src, TO_SCALE, TO_SCALE>, dim3(kCluster), dim3(kSmallThreads), 0, s, src, out);
  zero_word_kernel<<<1, 1, 0, s>>>(reinterpret_cast<unsigned int*>(out));
  cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  auto kern = absmax_wide_kernel<Src, TO_SCALE>;
  const int grid =
      persistent_grid(reinterpret_cast<const void*>(kern), kThreads, (elems + 32 * kThreads - 1) / (32 * kThreads));
  err = launch_pdl(kern, dim3((unsigned)grid), dim3(kThreads), 0, s, src, reinterpret_cast<unsigned int*>(out));
  if (err != cudaSuccess || !TO_SCALE) return err;
  return launch_pdl(scale_from_amax_kernel, dim3(1), dim3(1), 0, s, out);
}

GainSrc gain_src(const void* w, int64_t N, int64_t K, const float* gamma, float c) {
  return GainSrc{static_cast<const uint16_t*>(w), N, (int)K, gamma, c, std::gcd((int)(K / 16), 32)};
}

}  // namespace

cudaError_t launch_absmax_bf16(const void* x, int64_t n, float* amax, cudaStream_t s) {
  return launch<FlatSrc, false>(FlatSrc{static_cast<const uint16_t*>(x), n}, n, amax, s);
}

cudaError_t launch_nvfp4_tensor_scale(const void* x, int64_t n, float* g, cudaStream_t s) {
  return launch<FlatSrc, true>(FlatSrc{static_cast<const uint16_t*>(x), n}, n, g, s);
}

cudaError_t launch_absmax_gain(const void* w, int64_t N, int64_t K, const float* gamma, float c, float* amax,
                               cudaStream_t s) {
  if (gamma == nullptr && c == 1.0f) return launch_absmax_bf16(w, N * K, amax, s);
  return launch<GainSrc, false>(gain_src(w, N, K, gamma, c), N * K, amax, s);
}

cudaError_t launch_nvfp4_tensor_scale_gain(const void* w, int64_t N, int64_t K, const float* gamma, float c, float* g,
                                           cudaStream_t s) {
  if (gamma == nullptr && c == 1.0f) return launch_nvfp4_tensor_scale(w, N * K, g, s);
  return launch<GainSrc, true>(gain_src(w, N, K, gamma, c), N * K, g, s);
}

}  // namespace mxnorm
