// Layout of a 4-bit cache row, shared by its writer, its reader, the page
// summaries and the attention kernel, and the conversions of its codes.
#pragma once
#include <cuda_fp16.h>
#include <stdint.h>

namespace mla {

constexpr int kF4Row = 416;        // bytes per token: 256 of codes, 16 fp16 scales, 64 bf16 k_rope
constexpr int kF4ScaleOff = 256;
constexpr int kF4RopeOff = 288;
constexpr float kF4MaxScale = 10912.f;   // the largest fp16 s with 6 s <= 65504

namespace ptx {

// Two floats -> two E2M1 codes (lo in the low nibble), rounded to nearest even and saturated at +-6.
__device__ __forceinline__ uint32_t cvt_e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\t.reg .b16 u;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\t"
      "cvt.u16.u8 u, t;\n\tcvt.u32.u16 %0, u;\n\t}"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r;
}

// Two E2M1 codes (the low byte) -> an fp16 pair, exact.
__device__ __forceinline__ uint32_t cvt_f16x2_e2m1x2(uint32_t codes) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\t.reg .b16 u;\n\t"
      "cvt.u16.u32 u, %1;\n\tcvt.u8.u16 t, u;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, t;\n\t}"
      : "=r"(r)
      : "r"(codes));
  return r;
}

// Eight E2M1 codes (low nibble first) times a group's scale pair s2 = (s, s)
// -> four fp16 pairs: widened exactly, multiplied, rounded once.  The conversion
// takes two codes at the rate of any other integer instruction (64 lanes a
// clock per SM, measured; the E4M3 one runs at half of that), so a byte-permute table
// look-up (19 instructions for 8 codes against these 8) was slower.
__device__ __forceinline__ void dequant_e2m1x8_f16(uint32_t codes, uint32_t s2, uint32_t (&o)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t.reg .b32 x0, x1, x2, x3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 x0, b0;\n\tcvt.rn.f16x2.e2m1x2 x1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 x2, b2;\n\tcvt.rn.f16x2.e2m1x2 x3, b3;\n\t"
      "mul.rn.f16x2 %0, x0, %5;\n\tmul.rn.f16x2 %1, x1, %5;\n\t"
      "mul.rn.f16x2 %2, x2, %5;\n\tmul.rn.f16x2 %3, x3, %5;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(codes), "r"(s2));
}

}  // namespace ptx
}  // namespace mla
