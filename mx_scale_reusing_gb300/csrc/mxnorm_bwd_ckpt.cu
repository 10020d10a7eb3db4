// mxnorm_bwd_ckpt.cu -- straight-through backward of MXNorm from the 8-bit
// checkpoint: the E4M3 codes and E8M0 scales that the forward wrote stand in
// for the bf16 input, so training keeps 1.03 bytes an element instead of 2.
//
// "MXNorm: Reusing MXFP block scales for efficient tensor normalisation",
// Resumen tecnico, 2. Metodologia, "Gradientes" (RMSNorm's gradient through a
// straight-through estimator), with x^_j = code_j 2^e and rho~ the forward's
// inverse RMS, in the grouping of mxnorm_bwd.cu:
//     xh_j = rho~ x^_j,  m = (1/H) sum_j dy_j xh_j,  dx_j = rho~ (dy_j - xh_j m).
// A code has 4 significant bits and rho~ 2^e is exact (within the fp32
// range), so xh_j = RN(code_j RN(rho~ 2^e)) rounds once.
//
// Bound by HBM: 5.03 bytes an element (codes, scales, dy in; dx out):
// 204 us at 65536 x 4096, 99 % of the copy peak.  A warp or a CTA per row
// (cta_per_row); a lane takes 16 elements (16 bytes of codes, 32 of dy) of
// each chunk of 512 a warp.  Rows of up to 8 (warp) or 4 (CTA) chunks stay in
// registers between the sum and the output (13 words a chunk), so nothing is
// read twice; rows beyond 16384 elements are read again from L2.
#include "launch_fp4.h"
#include "mx_row.cuh"
#include "quant_device.cuh"

namespace mxnorm {
namespace {

constexpr int kWarps = 8;
constexpr int kChunk = 512;
constexpr int64_t kPrefetchElems = 1 << 20;

// A warp keeps rows of up to 4096 elements in registers; longer rows take a
// CTA each, and so do rows too few to fill the GPU with a warp each (us, a CTA
// / a warp per row: 64 x 768 1.3 / 1.8, 1000 x 2048 3.9 / 5.3, 2500 x 4096
// 11.0 / 14.1; 1000 x 1024 3.5 / 3.5, 2500 x 2048 7.8 / 6.3, 8192 x 4096
// 30.8 / 29.6; two passes by a warp took 16.9 at 1000 x 8192, a CTA 8.6).
// Rows of up to 128 and 256 elements share a warp four and two at a time.
inline bool cta_per_row(int64_t T, int64_t H) {
  return H > 8 * kChunk || (H >= 768 && T <= 1024) || (H > 2048 && T <= 4096);
}

__device__ __forceinline__ unsigned long long f2_fma(unsigned long long a, unsigned long long b,
                                                     unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// A lane's share of one chunk: 16 codes, 16 bf16 gradients, the block scale byte.
struct Share {
  uint32_t c[4];
  uint32_t d[8];
  uint32_t sb;
};

template <bool LOAD32>
__device__ __forceinline__ void load_share(const uint8_t* cr, const uint16_t* gr, const uint8_t* sr, int e0, int tiled,
                                           Share& s) {
  const uint4 t = ldg_stream16(cr + e0);
  s.c[0] = t.x;
  s.c[1] = t.y;
  s.c[2] = t.z;
  s.c[3] = t.w;
  load_lane<16, LOAD32>(gr + e0, s.d);
  const int kb = e0 / kBlock;
  s.sb = sr[(kb >> 2) * (tiled ? 512 : 4) + (kb & 3)];
}

// xh of elements 2i, 2i + 1 of a share; p = RN(rho~ 2^e) in both halves.
__device__ __forceinline__ unsigned long long xh_pair(const Share& s, int i, unsigned long long p) {
  float lo, hi;
  e4m3x2_to_f32(s.c[i / 2] >> (16 * (i % 2)), lo, hi);
  return f2_mul(f2_pack(lo, hi), p);
}

__device__ __forceinline__ unsigned long long share_scale(const Share& s, float r) {
  const float p = __fmul_rn(r, e8m0_value(s.sb));
  return f2_pack(p, p);
}

// Sum over the share of dy xh, each product rounded to fp32, pairwise.
__device__ __forceinline__ float share_dot(const Share& s, float r) {
  const unsigned long long p = share_scale(s, r);
  unsigned long long t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = f2_mul(xh_pair(s, i, p), f2_pack(bf16lo(s.d[i]), bf16hi(s.d[i])));
#pragma unroll
  for (int w = 4; w >= 1; w >>= 1)
#pragma unroll
    for (int i = 0; i < w; ++i) t[i] = f2_add(t[i], t[i + w]);
  float lo, hi;
  f2_unpack(t[0], lo, hi);
  return __fadd_rn(lo, hi);
}

__device__ __forceinline__ void store_share(uint16_t* dst, const Share& s, float r, float m) {
  const unsigned long long p = share_scale(s, r), nm = f2_pack(-m, -m), r2 = f2_pack(r, r);
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float lo, hi;
    f2_unpack(f2_mul(r2, f2_fma(xh_pair(s, i, p), nm, f2_pack(bf16lo(s.d[i]), bf16hi(s.d[i])))), lo, hi);
    o[i] = pack_bf16(lo, hi);
  }
  stg16(dst, o[0], o[1], o[2], o[3]);
  stg16(dst + 8, o[4], o[5], o[6], o[7]);
}

// Sum over the LANES threads of a row, in each of them: a tree of shuffles,
// and for a CTA a tree over the warps' sums in shared memory.  `red`
// alternates between rows, so that one barrier a row is enough.
template <int LANES>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int off = (LANES < 32 ? LANES : 32) / 2; off > 0; off >>= 1)
    v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, off));
  if constexpr (LANES > 32) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float t[kWarps];
#pragma unroll
    for (int i = 0; i < kWarps; ++i) t[i] = red[i];
#pragma unroll
    for (int w = kWarps / 2; w >= 1; w >>= 1)
#pragma unroll
      for (int i = 0; i < w; ++i) t[i] = __fadd_rn(t[i], t[i + w]);
    v = t[0];
  }
  return v;
}

// A row whose r is +Inf (row_factor) gets zeros.  A branch of its own: taking r
// as 0 from the start held the next row's loads back (65536 x 4096: 214 us, 204
// so).
template <int LANES>
__device__ __noinline__ void zero_row(uint16_t* dr, int t, int Hr) {
  for (int e0 = t * 16; e0 < Hr; e0 += LANES * 16) {
    stg16(dr + e0, 0u, 0u, 0u, 0u);
    stg16(dr + e0 + 8, 0u, 0u, 0u, 0u);
  }
}

// LANES: threads that share a row (8 or 16: several rows a warp; 32; or a
// whole CTA).  NCHUNK > 0: rows of at most NCHUNK chunks of LANES x 16
// elements, held in registers; NCHUNK == 0: any H, two passes over the row.
template <int LANES, int NCHUNK, bool LOAD32, int MINB>
__global__ void __launch_bounds__(kWarps * 32, MINB)
    mxnorm_bwd_ckpt_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int tiled,
                           const uint16_t* __restrict__ dy, const float* __restrict__ inv_rms, int64_t T, int H,
                           uint16_t* __restrict__ dx, int l2_prefetch) {
  constexpr int kStep = LANES * 16;
  constexpr int kRows = kWarps * 32 / LANES;       // rows of a CTA at a time
  constexpr int kGroup = LANES < 32 ? 32 / LANES : 1;  // rows of a warp at a time
  __shared__ float red[2][kWarps];
  const int t = threadIdx.x % LANES;  // thread of the row
  const int sub = LANES < 32 ? (threadIdx.x & 31) / LANES : 0;
  // the warp's (or CTA's) first row: the loop and the sums are uniform in a warp, rows past T only sit out
  const int64_t w0 = (int64_t)blockIdx.x * kRows + threadIdx.x / (LANES * kGroup) * kGroup;
  pdl_launch_dependents();
  if (l2_prefetch && w0 + sub < T) {  // the first row
    if (t == 0) prefetch_l2(dy + (w0 + sub) * (int64_t)H, (uint32_t)min(2 * H, 65536));
    if (t == 1) prefetch_l2(codes + (w0 + sub) * (int64_t)H, (uint32_t)min(H, 65536));
  }
  pdl_wait();
  const int KB = H / kBlock;
  int turn = 0;
  for (int64_t row0 = w0; row0 < T; row0 += (int64_t)gridDim.x * kRows, turn ^= 1) {
    const int64_t row = row0 + sub;
    const int Hr = row < T ? H : 0;  // elements of this thread's row that exist
    const uint8_t* cr = codes + row * (int64_t)H;
    const uint16_t* gr = dy + row * (int64_t)H;
    const uint8_t* sr = scale_row(const_cast<uint8_t*>(scales), row, KB, tiled);
    uint16_t* dr = dx + row * (int64_t)H;
    const float r = row < T ? inv_rms[row] : 0.0f;
    float dot = 0.0f;
    if constexpr (NCHUNK > 0) {
      Share s[NCHUNK];
#pragma unroll
      for (int c = 0; c < NCHUNK; ++c) {
        const int e0 = c * kStep + t * 16;
        if (e0 < Hr) load_share<LOAD32>(cr, gr, sr, e0, tiled, s[c]);
      }
#pragma unroll
      for (int c = 0; c < NCHUNK; ++c)
        if (c * kStep + t * 16 < Hr) dot = __fadd_rn(dot, share_dot(s[c], r));
      const float m = __fdiv_rn(row_sum<LANES>(dot, red[turn]), (float)H);
      if (empty_row(r)) {
        zero_row<LANES>(dr, t, Hr);
        continue;
      }
#pragma unroll
      for (int c = 0; c < NCHUNK; ++c) {
        const int e0 = c * kStep + t * 16;
        if (e0 < Hr) store_share(dr + e0, s[c], r, m);
      }
    } else {
      constexpr int B = 4;
      Share s[B];
      for (int c0 = 0; c0 * kStep < H; c0 += B) {
#pragma unroll
        for (int b = 0; b < B; ++b) {
          const int e0 = (c0 + b) * kStep + t * 16;
          if (e0 < Hr) load_share<LOAD32>(cr, gr, sr, e0, tiled, s[b]);
        }
#pragma unroll
        for (int b = 0; b < B; ++b)
          if ((c0 + b) * kStep + t * 16 < Hr) dot = __fadd_rn(dot, share_dot(s[b], r));
      }
      const float m = __fdiv_rn(row_sum<LANES>(dot, red[turn]), (float)H);
      if (empty_row(r)) {
        zero_row<LANES>(dr, t, Hr);
        continue;
      }
      for (int c0 = 0; c0 * kStep < H; c0 += B) {
#pragma unroll
        for (int b = 0; b < B; ++b) {
          const int e0 = (c0 + b) * kStep + t * 16;
          if (e0 < Hr) load_share<LOAD32>(cr, gr, sr, e0, tiled, s[b]);
        }
#pragma unroll
        for (int b = 0; b < B; ++b) {
          const int e0 = (c0 + b) * kStep + t * 16;
          if (e0 < Hr) store_share(dr + e0, s[b], r, m);
        }
      }
    }
  }
}

template <int LANES, int NCHUNK, bool LOAD32, int MINB>
cudaError_t launch_one(const BwdCkptArgs& a, cudaStream_t s) {
  auto kern = mxnorm_bwd_ckpt_kernel<LANES, NCHUNK, LOAD32, MINB>;
  constexpr int kRows = kWarps * 32 / LANES;
  const int grid = persistent_grid(reinterpret_cast<const void*>(kern), kWarps * 32, (a.T + kRows - 1) / kRows);
  // the first rows' prefetch pays where rows stream from HBM; for a few rows the pointers' lookup costs more
  const bool stream = a.T * a.H >= kPrefetchElems;
  return launch_pdl(kern, dim3((unsigned)grid), dim3(kWarps * 32), 0, s, static_cast<const uint8_t*>(a.codes),
                    a.scales, a.scale_tiled, static_cast<const uint16_t*>(a.dy), a.inv_rms, a.T, (int)a.H,
                    static_cast<uint16_t*>(a.dx), stream && is_device_memory(a.codes) && is_device_memory(a.dy) ? 1 : 0);
}

template <bool LOAD32>
cudaError_t launch_by_h(const BwdCkptArgs& a, cudaStream_t s) {
  if (cta_per_row(a.T, a.H)) {
    const int64_t chunks = (a.H + kWarps * kChunk - 1) / (kWarps * kChunk);
    if (chunks == 1) return launch_one<kWarps * 32, 1, LOAD32, 4>(a, s);
    if (chunks == 2) return launch_one<kWarps * 32, 2, LOAD32, 4>(a, s);
    if (chunks <= 4) return launch_one<kWarps * 32, 4, LOAD32, 3>(a, s);
    return launch_one<kWarps * 32, 0, LOAD32, 2>(a, s);
  }
  switch ((a.H + kChunk - 1) / kChunk) {
    case 1:
      if (a.H <= 128) return launch_one<8, 1, LOAD32, 4>(a, s);
      if (a.H <= 256) return launch_one<16, 1, LOAD32, 4>(a, s);
      return launch_one<32, 1, LOAD32, 4>(a, s);
    case 2: return launch_one<32, 2, LOAD32, 4>(a, s);
    case 3:
    case 4: return launch_one<32, 4, LOAD32, 3>(a, s);
    default: return launch_one<32, 8, LOAD32, 1>(a, s);
  }
}

}  // namespace

cudaError_t launch_mxnorm_bwd_ckpt(const BwdCkptArgs& a, cudaStream_t s) {
  // rows are 64-byte multiples: 32-byte loads when dy starts on one
  return (reinterpret_cast<uintptr_t>(a.dy) & 31) == 0 ? launch_by_h<true>(a, s) : launch_by_h<false>(a, s);
}

}  // namespace mxnorm
