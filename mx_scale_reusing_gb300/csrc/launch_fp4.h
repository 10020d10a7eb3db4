// launch_fp4.h -- internal launcher interface of the FP4 products and 8-bit
// checkpoints, as launch.h for the MX passes.  Not installed; not part of the
// ABI.
#pragma once

#include "launch.h"

namespace mxnorm {

// FP4 cast of a weight (or of any bf16 rows): mx_cast_fp4.cu
struct Fp4CastArgs {
  const void* w;        // bf16 [N, K]
  int64_t N;
  int64_t K;
  int fmt;              // kFmtE2M1, kFmtE2M1H16, kFmtE2M1H32 or kFmtNvfp4
  const float* gamma;   // f32 [K] or null (ones)
  float c;
  const float* g_dev;   // NVFP4: device word holding the tensor scale
  void* codes;          // u8 [N, K/2]
  uint8_t* scales;      // E8M0 [N, K/32] or UE4M3 [N, K/16], row-major or MMA atoms
  int scale_tiled;
};

struct DequantArgs {
  const void* codes;
  const uint8_t* scales;
  int64_t T;
  int64_t H;
  int fmt;              // any mxnorm_fmt
  int scale_tiled;
  const float* g_dev;   // NVFP4: device word holding the tensor scale
  void* out;            // bf16 [T, H]
};

// Failure-detection drill of a kernel with a load pipeline: the waits' limit,
// and one load that is never issued, so that the waits behind it run out.
struct WaitDrill {
  unsigned long long limit_ns = 2000000000ull;
  int64_t stage = -1;  // of each CTA's (or pair's) stages, from 0; -1: none is withheld
  int load = 0;        // which of the stage's loads
};

struct Fp4LinearArgs {
  const void* x_codes;       // E2M1 [T, K/2]
  const uint8_t* x_scales;   // MMA atoms
  const float* inv_rms;      // f32 [T] or null (ones)
  const void* w_codes;       // E2M1 [N, K/2]
  const uint8_t* w_scales;   // MMA atoms
  int64_t T;
  int64_t K;
  int64_t N;
  int nvfp4;                 // 1: UE4M3 scales per 16, else E8M0 per 32
  const float* xg;           // NVFP4 tensor scales (device words)
  const float* wg;
  void* out;                 // bf16 [T, N]
  WaitDrill drill = {};      // all loads of the stage
};

struct BwdCkptArgs {
  const void* codes;         // E4M3 [T, H]
  const uint8_t* scales;     // E8M0
  int scale_tiled;
  const void* dy;            // bf16 [T, H]
  const float* inv_rms;      // f32 [T]
  int64_t T;
  int64_t H;
  void* dx;                  // bf16 [T, H]
};

struct WgradArgs {
  const void* codes;         // E4M3 [T, K]
  const uint8_t* scales;     // E8M0
  int scale_tiled;
  const float* inv_rms;      // f32 [T] or null (ones)
  const void* dout;          // bf16 [T, N]
  int64_t T;
  int64_t K;
  int64_t N;
  void* dw;                  // bf16 [N, K]
  void* workspace;           // wgrad_workspace_bytes(T, K, N) bytes
  WaitDrill drill = {};      // load 0: dout's tile, 1: the codes'
};

// launch_nvfp4 with the scales in the MMA atom layout where scale_tiled != 0.
cudaError_t launch_nvfp4_layout(const Nvfp4Args& a, int scale_tiled, cudaStream_t s);
cudaError_t launch_mx_cast_fp4(const Fp4CastArgs& a, cudaStream_t s);
// The NVFP4 tensor scale of the gain-folded weight (gamma null: ones).
cudaError_t launch_nvfp4_tensor_scale_gain(const void* w, int64_t N, int64_t K, const float* gamma, float c, float* g,
                                           cudaStream_t s);
// Largest magnitude of the gain-folded weight (NaN above Inf above finite).
cudaError_t launch_absmax_gain(const void* w, int64_t N, int64_t K, const float* gamma, float c, float* amax,
                               cudaStream_t s);
cudaError_t read_fp4_cast_error_word(uint32_t* out, bool clear);
cudaError_t launch_mx_dequant(const DequantArgs& a, cudaStream_t s);
cudaError_t launch_fp4_linear(const Fp4LinearArgs& a, cudaStream_t s);
cudaError_t launch_fp4_linear_many(const Fp4LinearArgs& a, cudaStream_t s);
cudaError_t read_fp4_linear_error_word(uint32_t* out, bool clear);
cudaError_t read_fp4_few_error_word(uint32_t* out, bool clear);
cudaError_t launch_mxnorm_bwd_ckpt(const BwdCkptArgs& a, cudaStream_t s);
cudaError_t launch_mxnorm_wgrad(const WgradArgs& a, cudaStream_t s);
int64_t wgrad_workspace_bytes(int64_t T, int64_t K, int64_t N);
cudaError_t read_wgrad_error_word(uint32_t* out, bool clear);

}  // namespace mxnorm
