// quant_device.cuh -- what the FP4 product and checkpoint kernels share beyond
// the MX passes' building blocks: quantised codes and scales back to fp32.
#pragma once

#include "mx_device.cuh"

namespace mxnorm {

// NVFP4 (16-element blocks, UE4M3 scales, tensor scale) where a call takes it
// beside the MX formats; not a format of the MX passes.
constexpr int kFmtNvfp4 = 6;

// Two E4M3 codes (low 16 bits of w) -> two fp32 values, exactly.
__device__ __forceinline__ void e4m3x2_to_f32(uint32_t w, float& lo, float& hi) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)w));
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
}
// Two E2M1 codes (low byte of w, the first in the low nibble) -> two fp32 values.
__device__ __forceinline__ void e2m1x2_to_f32(uint32_t w, float& lo, float& hi) {
  uint32_t h;
  asm("{\n\t.reg .b8 q;\n\tcvt.u8.u32 q, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, q;\n\t}" : "=r"(h) : "r"(w));
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
}
// Two fp32 -> packed bf16x2, round to nearest even.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// A row's inverse RMS as a factor.  The NVFP4 pass gives +Inf for a row whose
// block scales are all 0 (padding, or values lost beside the tensor's largest):
// the forward multiplied zeros there, so the row counts as 0 and not as the NaN
// of 0 times Inf, which a single padded row would carry into all of dW.
__device__ __forceinline__ bool empty_row(float inv_rms) { return inv_rms == __uint_as_float(0x7F800000u); }
__device__ __forceinline__ float row_factor(float inv_rms) { return empty_row(inv_rms) ? 0.0f : inv_rms; }
// Value of an E8M0 scale byte: 2^(b - 127) (b = 0: the subnormal 2^-127; 0xFF: NaN).
__device__ __forceinline__ float e8m0_value(uint32_t b) {
  return b == 0u ? 0x1p-127f : __uint_as_float(b == 0xFFu ? 0x7FC00000u : b << 23);
}

}  // namespace mxnorm
