// fa_kv4_cache.cu — rows of keys and values written into the paged 4-bit
// cache, and read back.
//
// A group is 16 consecutive elements of a row: its scale is
// s = e4m3(max|x| / 6), its codes e2m1(x / s), both rounded to nearest with
// ties to the even number (the stored value is code * s * 2^exp; x is scaled
// by 2^-exp first, exactly).  A group whose scale rounds to zero stores zeros.
//
// Borders decide codes, so x / s has to fall on the right side of them.
// fp32 input divides: the correctly rounded quotient lies on a border only if
// the exact one does (a neighbour x of s * border differs from it by at least
// 1 / 1.875 units in the quotient's last place, and max|x| / 6 likewise).
// 16-bit input has at most 11 significant bits and s * border at most 7, so a
// quotient off a border is off by 2^-11 of it at least: it is enough to
// multiply by 1 / s (error below 2^-22) and round the product to 14 bits,
// which puts quotients on a border back there and moves no other across.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa.h"
#include "fa_kv4.cuh"
#include "fa_serve.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;

// Byte-row index of (slot, head) in the cache; slot in [0, num_blocks * bs).
__device__ __forceinline__ long long cache_row(const Kv4Store &c, long long slot, int h) {
  const long long block = slot >> c.bs_log2, off = slot & ((1 << c.bs_log2) - 1);
  return ((block * c.Hk + h) << c.bs_log2) + off;
}

template <typename T>
__device__ __forceinline__ void load16(const T *src, float (&x)[16]) {
  constexpr int W = 16 / sizeof(T);
#pragma unroll
  for (int i = 0; i < 16 / W; ++i) {
    const uint4 v = reinterpret_cast<const uint4 *>(src)[i];
    const T *e = reinterpret_cast<const T *>(&v);
#pragma unroll
    for (int j = 0; j < W; ++j) x[i * W + j] = static_cast<float>(e[j]);
  }
}

// One thread: one group of one row of K (blockIdx.y = 0) or V (1).
template <typename T>
__global__ void __launch_bounds__(kThreads)
    fa_kv4_append_kernel(const T *k, const T *v, long long k_stride, long long v_stride,
                         const long long *slots, int T_, const Kv4Store c) {
  griddep_wait();
  griddep_launch_dependents();
  const bool is_v = blockIdx.y != 0;
  const int groups = c.d / 16, per_row = c.Hk * groups;
  const long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  const long long row = i / per_row;
  if (row >= T_) return;
  const long long slot = slots[row];
  if (slot < 0 || slot >= (static_cast<long long>(c.num_blocks) << c.bs_log2)) return;
  const int hg = static_cast<int>(i - row * per_row), h = hg / groups, g = hg - h * groups;
  float x[16];
  load16((is_v ? v + row * v_stride : k + row * k_stride) + hg * 16, x);
  const float unit = pow2(-(is_v ? c.v_exp : c.k_exp));
  float amax = 0.f;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    x[j] *= unit;
    amax = fmaxf(amax, fabsf(x[j]));
  }
  const uint32_t sb = f32_e4m3(__fdiv_rn(amax, 6.f));
  const float s = f16x2_f32(e4m3x2_f16x2(sb)).x;
  uint32_t codes[2] = {0, 0};
  if (s > 0.f) {
    if constexpr (sizeof(T) == 2) {
      const float r = __fdiv_rn(1.f, s);
#pragma unroll
      for (int j = 0; j < 16; ++j)  // to 14 significant bits; a NaN becomes 8, stored as +6
        x[j] = __uint_as_float((__float_as_uint(fminf(x[j] * r, 8.f)) + 0x200u) & ~0x3FFu);
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] = __fdiv_rn(x[j], s);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      codes[j / 4] |= f32x2_e2m1x2(x[2 * j], x[2 * j + 1]) << (8 * (j & 3));
  }
  const long long at = cache_row(c, slot, h);
  reinterpret_cast<uint2 *>(is_v ? c.v_codes : c.k_codes)[at * groups + g] =
      make_uint2(codes[0], codes[1]);
  (is_v ? c.v_scales : c.k_scales)[at * groups + g] = static_cast<uint8_t>(sb);
}

// One thread: 16 elements of one row of K or V; a slot outside the cache
// reads zeros.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    fa_kv4_gather_kernel(const long long *slots, int R, const Kv4Store c, T *k_out, T *v_out) {
  griddep_wait();
  griddep_launch_dependents();
  const bool is_v = blockIdx.y != 0;
  const int groups = c.d / 16, per_row = c.Hk * groups;
  const long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  const long long row = i / per_row;
  if (row >= R) return;
  const long long slot = slots[row];
  const int hg = static_cast<int>(i - row * per_row), h = hg / groups, g = hg - h * groups;
  uint2 codes = make_uint2(0, 0);
  float s = 0.f;
  if (slot >= 0 && slot < (static_cast<long long>(c.num_blocks) << c.bs_log2)) {
    const long long at = cache_row(c, slot, h);
    codes = reinterpret_cast<const uint2 *>(is_v ? c.v_codes : c.k_codes)[at * groups + g];
    s = f16x2_f32(e4m3x2_f16x2((is_v ? c.v_scales : c.k_scales)[at * groups + g])).x *
        pow2(is_v ? c.v_exp : c.k_exp);
  }
  T *out = (is_v ? v_out : k_out) + i * 16;
  constexpr int W = 16 / sizeof(T);
  const uint32_t pairs[8] = {e2m1x2_f16x2<0>(codes.x), e2m1x2_f16x2<1>(codes.x),
                             e2m1x2_f16x2<2>(codes.x), e2m1x2_f16x2<3>(codes.x),
                             e2m1x2_f16x2<0>(codes.y), e2m1x2_f16x2<1>(codes.y),
                             e2m1x2_f16x2<2>(codes.y), e2m1x2_f16x2<3>(codes.y)};
#pragma unroll
  for (int n = 0; n < 16 / W; ++n) {
    alignas(16) T e[W];
#pragma unroll
    for (int j = 0; j < W / 2; ++j) {
      const float2 f = f16x2_f32(pairs[n * W / 2 + j]);
      e[2 * j] = static_cast<T>(f.x * s);
      e[2 * j + 1] = static_cast<T>(f.y * s);
    }
    reinterpret_cast<uint4 *>(out)[n] = *reinterpret_cast<const uint4 *>(e);
  }
}

template <typename... A>
cudaError_t launch(void (*kern)(A...), long long threads, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  const long long gx = (threads + kThreads - 1) / kThreads;
  if (gx > 2147483647LL) return cudaErrorInvalidConfiguration;
  cfg.gridDim = dim3(static_cast<unsigned>(gx), 2);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <typename T>
cudaError_t append(const void *k, const void *v, long long ks, long long vs,
                   const long long *slots, int T_, const Kv4Store &c, cudaStream_t s) {
  return launch<const T *, const T *, long long, long long, const long long *, int,
                const Kv4Store>(fa_kv4_append_kernel<T>,
                                static_cast<long long>(T_) * c.Hk * (c.d / 16), s,
                                static_cast<const T *>(k), static_cast<const T *>(v), ks, vs,
                                slots, T_, c);
}

template <typename T>
cudaError_t gather(const long long *slots, int R, const Kv4Store &c, void *k, void *v,
                   cudaStream_t s) {
  return launch<const long long *, int, const Kv4Store, T *, T *>(
      fa_kv4_gather_kernel<T>, static_cast<long long>(R) * c.Hk * (c.d / 16), s, slots, R, c,
      static_cast<T *>(k), static_cast<T *>(v));
}

}  // namespace

cudaError_t launch_kv4_append(const void *k, const void *v, long long k_stride, long long v_stride,
                              const long long *slots, int T, const Kv4Store &c, int dtype,
                              cudaStream_t s) {
  if (dtype == FA_DTYPE_BF16)
    return append<__nv_bfloat16>(k, v, k_stride, v_stride, slots, T, c, s);
  if (dtype == FA_DTYPE_F16) return append<__half>(k, v, k_stride, v_stride, slots, T, c, s);
  return append<float>(k, v, k_stride, v_stride, slots, T, c, s);
}

cudaError_t launch_kv4_gather(const long long *slots, int R, const Kv4Store &c, void *k_out,
                              void *v_out, int dtype, cudaStream_t s) {
  if (dtype == FA_DTYPE_BF16) return gather<__nv_bfloat16>(slots, R, c, k_out, v_out, s);
  if (dtype == FA_DTYPE_F16) return gather<__half>(slots, R, c, k_out, v_out, s);
  return gather<float>(slots, R, c, k_out, v_out, s);
}

}  // namespace fa
