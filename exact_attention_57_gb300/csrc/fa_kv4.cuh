// fa_kv4.cuh — device helpers of the 4-bit cache format: e2m1 codes (two a
// byte, the even element in the low half) with one e4m3 scale for 16
// elements.  A value code * scale has at most six significant bits and lies
// between 2^-10 and 2688, so fp16, bf16 and fp32 all hold it exactly.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

namespace fa {

// 32 bytes at a time.
struct alignas(32) B32 {
  uint32_t w[8];
};
__device__ __forceinline__ B32 load32(const void *p) {
  B32 x;
  asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(x.w[0]), "=r"(x.w[1]), "=r"(x.w[2]), "=r"(x.w[3]), "=r"(x.w[4]), "=r"(x.w[5]),
                 "=r"(x.w[6]), "=r"(x.w[7])
               : "l"(p));
  return x;
}
__device__ __forceinline__ void store32(void *p, const B32 &x) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x.w[0]),
               "r"(x.w[1]), "r"(x.w[2]), "r"(x.w[3]), "r"(x.w[4]), "r"(x.w[5]), "r"(x.w[6]), "r"(x.w[7])
               : "memory");
}

// Byte `I` of w (two e2m1 codes) as two fp16 values, the low half first.
template <int I>
__device__ __forceinline__ uint32_t e2m1x2_f16x2(uint32_t w) {
  uint32_t r;
  if constexpr (I == 0)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t}\n" : "=r"(r) : "r"(w));
  else if constexpr (I == 1)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b;\n\t}\n" : "=r"(r) : "r"(w));
  else if constexpr (I == 2)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, c;\n\t}\n" : "=r"(r) : "r"(w));
  else
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, d;\n\t}\n" : "=r"(r) : "r"(w));
  return r;
}

// The two e4m3 numbers in the low 16 bits of w as two fp16 values (exact).
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}\n"
      : "=r"(r) : "r"(w));
  return r;
}

// x as e4m3: round to nearest even, 448 at most.
__device__ __forceinline__ uint32_t f32_e4m3(float x) {
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %1, %2;\n\tcvt.u32.u16 %0, h;\n\t}\n"
      : "=r"(r) : "f"(0.f), "f"(x));
  return r & 0xFFu;
}

// Two fp32 as e2m1 codes in one byte (lo in the low half): round to nearest,
// ties to the even code, 6 at most.
__device__ __forceinline__ uint32_t f32x2_e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\tcvt.u32.u8 %0, b;\n\t}\n"
      : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Product of two fp16 pairs.
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}

// 2^e for e in [-126, 127].
__device__ __forceinline__ float pow2(int e) { return __int_as_float((127 + e) << 23); }

__device__ __forceinline__ float2 f16x2_f32(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

}  // namespace fa
