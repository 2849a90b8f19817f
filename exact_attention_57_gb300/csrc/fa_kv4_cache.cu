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
// quotient off a border (0.25 .. 5) is off by 2^-11 of it, 2^-13, at least: it
// is enough to multiply by 1 / s (error below 2^-22 of it, 2^-19) and round to
// a multiple of 2^-16, by an addition of 1.5 * 2^7 and its subtraction, which
// puts quotients on a border back there and moves no other across.
//
// Both kernels are bound by memory and near the rate at which instructions are
// issued, so a thread takes the same 16 elements of K and of V (one slot, one
// index computation, 32 bytes a load).  16383 fp16 rows of 8 x 128 elements
// written and 24575 read back (215 MB) take 37.6 us as two launches, 5.7 TB/s or
// 85% of the measured copy rate (52 us with one group a thread and 64-bit
// divisions; 45 with 16-byte accesses, which rows off 32 bytes get); fp32 rows 63 us
// of 57 at the copy rate.  The writing alone takes 16 us from 16-bit rows (5.2 to
// 5.5 TB/s) and 26 from fp32 ones (5.9 TB/s: their divisions hide behind twice the
// bytes).  64 rows written and read back take 3.4 us in a captured graph, two
// launches, and 6 as two calls.
#include <type_traits>

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

// Where a thread's 16 elements are: row, and head * (d / 16) + group.
struct At {
  long long row;
  int hg;
};
__device__ __forceinline__ At place(const Kv4Store &c) {
  const int per_row = c.Hk * (c.d / 16);
  const long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >> 32 == 0) {  // the common case: a 32-bit division
    const unsigned u = static_cast<unsigned>(i), row = u / per_row;
    return At{row, static_cast<int>(u - row * per_row)};
  }
  const long long row = i / per_row;
  return At{row, static_cast<int>(i - row * per_row)};
}

// Index of a slot's 16 elements in the cache, in units of 16.
__device__ __forceinline__ long long cache_at(const Kv4Store &c, long long slot, int hg) {
  const int groups = c.d / 16, h = hg / groups;
  return cache_row(c, slot, h) * groups + (hg - h * groups);
}

template <typename T>
struct Group {  // 16 elements
  uint4 w[sizeof(T)];
};
template <typename T>
__device__ __forceinline__ Group<T> load_group(const T *p, bool wide) {
  Group<T> x;
  if (wide) {
#pragma unroll
    for (int n = 0; n < static_cast<int>(sizeof(T)) / 2; ++n)
      reinterpret_cast<B32 *>(&x)[n] = load32(reinterpret_cast<const uint8_t *>(p) + 32 * n);
  } else {
#pragma unroll
    for (int n = 0; n < static_cast<int>(sizeof(T)); ++n)
      x.w[n] = __ldg(reinterpret_cast<const uint4 *>(p) + n);
  }
  return x;
}

// Codes and scale of a group.
template <typename T>
__device__ __forceinline__ void quantise(const Group<T> &x, float unit, uint2 *codes, uint8_t *scale) {
  float amax;
  if constexpr (sizeof(T) == 2) {
    using P = std::conditional_t<std::is_same_v<T, __half>, __half2, __nv_bfloat162>;
    const P *p = reinterpret_cast<const P *>(&x);
    P top = __habs2(p[0]);
#pragma unroll
    for (int j = 1; j < 8; ++j) top = __hmax2(top, __habs2(p[j]));
    // a NaN does not count, and where there is nothing else the maximum is zero
    amax = fmaxf(fmaxf(static_cast<float>(top.x), static_cast<float>(top.y)), 0.f) * unit;
  } else {
    const float *p = reinterpret_cast<const float *>(&x);
    amax = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) amax = fmaxf(amax, fabsf(p[j]));
    amax *= unit;
  }
  const uint32_t sb = f32_e4m3(__fdiv_rn(amax, 6.f));
  const float s = f16x2_f32(e4m3x2_f16x2(sb)).x;
  uint32_t c[2] = {0, 0};
  if (s > 0.f) {
    float y[16];
    if constexpr (sizeof(T) == 2) {
      const T *p = reinterpret_cast<const T *>(&x);
      const float r = __fdiv_rn(1.f, s) * unit, C = 192.f;
#pragma unroll
      for (int j = 0; j < 16; ++j)  // to a multiple of 2^-16
        y[j] = __fadd_rn(__fmaf_rn(static_cast<float>(p[j]), r, C), -C);
    } else {
      const float *p = reinterpret_cast<const float *>(&x);
#pragma unroll
      for (int j = 0; j < 16; ++j) y[j] = __fdiv_rn(p[j] * unit, s);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j / 4] |= f32x2_e2m1x2(y[2 * j], y[2 * j + 1]) << (8 * (j & 3));
  }
  *codes = make_uint2(c[0], c[1]);
  *scale = static_cast<uint8_t>(sb);
}

// One thread: one group of one row of K and of V.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    fa_kv4_append_kernel(const T *k, const T *v, long long k_stride, long long v_stride,
                         const long long *slots, int T_, const Kv4Store c, bool wide) {
  griddep_wait();
  griddep_launch_dependents();
  const At at = place(c);
  if (at.row >= T_) return;
  const Group<T> kx = load_group(k + at.row * k_stride + at.hg * 16, wide);
  const Group<T> vx = load_group(v + at.row * v_stride + at.hg * 16, wide);
  const long long slot = __ldg(slots + at.row);
  if (slot < 0 || slot >= (static_cast<long long>(c.num_blocks) << c.bs_log2)) return;
  const long long to = cache_at(c, slot, at.hg);
  quantise(kx, pow2(-c.k_exp), reinterpret_cast<uint2 *>(c.k_codes) + to, c.k_scales + to);
  quantise(vx, pow2(-c.v_exp), reinterpret_cast<uint2 *>(c.v_codes) + to, c.v_scales + to);
}

// 16 elements from their codes and scale.
template <typename T>
__device__ __forceinline__ void expand(uint2 codes, uint32_t scale, int exp, T *out, bool wide) {
  const uint32_t pairs[8] = {e2m1x2_f16x2<0>(codes.x), e2m1x2_f16x2<1>(codes.x),
                             e2m1x2_f16x2<2>(codes.x), e2m1x2_f16x2<3>(codes.x),
                             e2m1x2_f16x2<0>(codes.y), e2m1x2_f16x2<1>(codes.y),
                             e2m1x2_f16x2<2>(codes.y), e2m1x2_f16x2<3>(codes.y)};
  const uint32_t s16 = __byte_perm(e4m3x2_f16x2(scale), 0, 0x1010);
  alignas(32) T e[16];
  if (std::is_same_v<T, __half> && exp == 0) {  // the product is exact in fp16
#pragma unroll
    for (int j = 0; j < 8; ++j) reinterpret_cast<uint32_t *>(e)[j] = hmul2(pairs[j], s16);
  } else {
    const float s = f16x2_f32(s16).x * pow2(exp);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 f = f16x2_f32(pairs[j]);
      e[2 * j] = static_cast<T>(f.x * s);
      e[2 * j + 1] = static_cast<T>(f.y * s);
    }
  }
#pragma unroll
  for (int n = 0; n < static_cast<int>(sizeof(T)) / 2; ++n) {
    if (wide) {
      store32(reinterpret_cast<uint8_t *>(out) + 32 * n, reinterpret_cast<const B32 *>(e)[n]);
    } else {
      reinterpret_cast<uint4 *>(out)[2 * n] = reinterpret_cast<const uint4 *>(e)[2 * n];
      reinterpret_cast<uint4 *>(out)[2 * n + 1] = reinterpret_cast<const uint4 *>(e)[2 * n + 1];
    }
  }
}

// One thread: 16 elements of one row of K and of V; a slot outside the cache
// reads zeros.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    fa_kv4_gather_kernel(const long long *slots, int R, const Kv4Store c, T *k_out, T *v_out,
                         bool wide) {
  griddep_wait();
  griddep_launch_dependents();
  const At at = place(c);
  if (at.row >= R) return;
  const long long slot = __ldg(slots + at.row);
  uint2 kc = make_uint2(0, 0), vc = make_uint2(0, 0);
  uint32_t ks = 0, vs = 0;
  if (slot >= 0 && slot < (static_cast<long long>(c.num_blocks) << c.bs_log2)) {
    const long long from = cache_at(c, slot, at.hg);
    kc = __ldg(reinterpret_cast<const uint2 *>(c.k_codes) + from);
    vc = __ldg(reinterpret_cast<const uint2 *>(c.v_codes) + from);
    ks = __ldg(c.k_scales + from);
    vs = __ldg(c.v_scales + from);
  }
  const long long to = (at.row * c.Hk * (c.d / 16) + at.hg) * 16;
  expand(kc, ks, c.k_exp, k_out + to, wide);
  expand(vc, vs, c.v_exp, v_out + to, wide);
}

template <typename... A>
cudaError_t launch(void (*kern)(A...), long long threads, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  const long long gx = (threads + kThreads - 1) / kThreads;
  if (gx > 2147483647LL) return cudaErrorInvalidConfiguration;
  cfg.gridDim = dim3(static_cast<unsigned>(gx));
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
  const long long es = sizeof(T);
  const bool wide = (reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) % 32 == 0 &&
                    ks * es % 32 == 0 && vs * es % 32 == 0;
  return launch<const T *, const T *, long long, long long, const long long *, int, const Kv4Store,
                bool>(fa_kv4_append_kernel<T>, static_cast<long long>(T_) * c.Hk * (c.d / 16), s,
                      static_cast<const T *>(k), static_cast<const T *>(v), ks, vs, slots, T_, c,
                      wide);
}

template <typename T>
cudaError_t gather(const long long *slots, int R, const Kv4Store &c, void *k, void *v,
                   cudaStream_t s) {
  const bool wide = (reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) % 32 == 0;
  return launch<const long long *, int, const Kv4Store, T *, T *, bool>(
      fa_kv4_gather_kernel<T>, static_cast<long long>(R) * c.Hk * (c.d / 16), s, slots, R, c,
      static_cast<T *>(k), static_cast<T *>(v), wide);
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
