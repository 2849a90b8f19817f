// fa_kv8.cuh — device helpers of the 8-bit cache format: e4m3 codes with one fp32
// scale for a block of tokens of a key head.  A code has four significant bits and
// lies between 2^-9 and 448, so fp16 holds it exactly.
#pragma once

#include "fa_kv4.cuh"

namespace fa {

// The two e4m3 numbers in the high 16 bits of w as two fp16 values (exact).
__device__ __forceinline__ uint32_t e4m3x2_f16x2_hi(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}\n"
      : "=r"(r) : "r"(w));
  return r;
}

// Two fp32 as e4m3 numbers in the low 16 bits (lo in the low byte): round to
// nearest, ties to even, 448 at most.
__device__ __forceinline__ uint32_t f32x2_e4m3x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %1, %2;\n\tcvt.u32.u16 %0, h;\n\t}\n"
      : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two fp16 as e4m3 numbers in the low 16 bits, likewise; a NaN stays one.
__device__ __forceinline__ uint32_t f16x2_e4m3x2(uint32_t x) {
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.rn.satfinite.e4m3x2.f16x2 h, %1;\n\tcvt.u32.u16 %0, h;\n\t}\n"
      : "=r"(r) : "r"(x));
  return r;
}

// Exponents of the scales that are stored.
constexpr int kScaleExp = 40;

// What the softmax needs of a block's scales: weights carry the value's scale,
//   2^(s + log2 vs - m) = e^(score) vs 2^-m,
// so that O = sum w code / sum (w / vs) takes one exponential a score and no
// weight is above the largest, whatever the scales of other blocks are.
struct BlockScale {
  float k, v_log, v_inv;
  // A scale that is not positive counts as zero for keys; values' count as the
  // nearest in 2^-40 .. 2^40 (so that sums of w and of w / vs lose nothing to fp32's
  // range: a weight below 2^-126 of the largest is 2^-46 of the sum at most).
  __device__ __forceinline__ void set(float ks, float vs) {
    k = fmaxf(ks, 0.f);
    vs = fminf(fmaxf(vs, pow2(-kScaleExp)), pow2(kScaleExp));
    // by the exponent and a number in 1 .. 2, whose logarithm is good to 2^-22; a
    // power of two, as fa_kv8_append stores them, has an exact one
    const uint32_t bits = __float_as_uint(vs);
    float part;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(part) : "f"(__uint_as_float((bits & 0x7FFFFFu) | 0x3F800000u)));
    v_log = static_cast<float>(static_cast<int>(bits >> 23) - 127) + part;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(v_inv) : "f"(vs));
  }
};

}  // namespace fa
