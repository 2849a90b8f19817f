// fa_kv8_cache.cu — rows of keys and values written into the paged 8-bit cache,
// and read back.
//
// A block of tokens of one key head has one scale, for keys and for values.  With
// a = max|x| over the finite elements that a call writes into it and e the least
// integer in -40 .. 40 with a <= 448 * 2^e,
//   scale' = 2^e            if the call writes the block's first token,
//            max(scale, 2^e) otherwise,
// codes are e4m3(x / scale'), rounded to nearest, ties to even; and where the scale
// has grown, the tokens ahead of the first one written keep their values:
// code' = e4m3(code * scale / scale').  e4m3 is a floating-point format, so a power
// of two for a scale costs no accuracy, both quotients are exact, and growing
// re-rounds nothing but what becomes subnormal (below scale' * 2^-6).
//
// The rows of one block follow one another in a call (as fa_kv_plan deals them): a
// run.  A team of bs / 16 warps takes a run for one key head and for K or V, a warp the
// rows of 16 of the block's tokens, all loaded at once and kept in registers between
// the maximum, which the team shares through shared memory, and the codes: each row is
// read once, and with 4 KB in flight a warp.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "fa.h"
#include "fa_kv8.cuh"
#include "fa_serve.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;

// Eight elements.
template <typename T>
struct Eight {
  uint4 w[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Eight<T> load_eight(const T *p) {
  Eight<T> x;
#pragma unroll
  for (int n = 0; n < static_cast<int>(sizeof(T)) / 2; ++n)
    x.w[n] = __ldg(reinterpret_cast<const uint4 *>(p) + n);
  return x;
}

// The larger of `top` and the elements' sizes; NaNs do not count, infinities only
// where asked.
template <bool kFinite, typename T>
__device__ __forceinline__ float size_of(const Eight<T> &x, float top) {
  if constexpr (!kFinite && sizeof(T) == 2) {
    using P = std::conditional_t<std::is_same_v<T, __half>, __half2, __nv_bfloat162>;
    const P *p = reinterpret_cast<const P *>(&x);
    const P m = __hmax2(__hmax2(__habs2(p[0]), __habs2(p[1])), __hmax2(__habs2(p[2]), __habs2(p[3])));
    return fmaxf(top, fmaxf(static_cast<float>(m.x), static_cast<float>(m.y)));
  }
  const T *e = reinterpret_cast<const T *>(&x);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float a = fabsf(static_cast<float>(e[j]));
    top = fmaxf(top, kFinite && a == INFINITY ? 0.f : a);
  }
  return top;
}

// Eight codes.  `by`: 1 / scale where that is a power of two, else the scale.
template <typename T>
__device__ __forceinline__ uint2 codes_of(const Eight<T> &x, float by, bool exact) {
  const T *e = reinterpret_cast<const T *>(&x);
  uint32_t c[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float y[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const float f = static_cast<float>(e[2 * j + n]);
      y[n] = fminf(exact ? f * by : __fdiv_rn(f, by), 448.f);  // (a NaN becomes 448)
    }
    c[j] = f32x2_e4m3x2(y[0], y[1]);
  }
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// Eight codes times `by`, as codes.
__device__ __forceinline__ uint2 rescaled(uint2 c, float by) {
  uint32_t r[2] = {c.x, c.y};
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const float2 lo = f16x2_f32(e4m3x2_f16x2(r[n])), hi = f16x2_f32(e4m3x2_f16x2_hi(r[n]));
    r[n] = f32x2_e4m3x2(fminf(lo.x * by, 448.f), fminf(lo.y * by, 448.f)) |
           f32x2_e4m3x2(fminf(hi.x * by, 448.f), fminf(hi.y * by, 448.f)) << 16;
  }
  return make_uint2(r[0], r[1]);
}

// The scale for elements of up to `a`: 2^e, e the least in -40 .. 40 with
// a <= 448 * 2^e = 1.75 * 2^(8 + e).
__device__ __forceinline__ float scale_for(float a) {
  const uint32_t bits = __float_as_uint(a);
  const int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u);
  return pow2(min(max(e, -kScaleExp), kScaleExp));
}

// Rows that a CTA looks through for runs that begin there, at most.
constexpr int kWindow = 64;

// The runs that begin among rows [window, window + the CTA's share), for one key head of
// K or V.  Rows that are skipped do not end a run.  kSteps: rows of a warp by what it
// loads at a time, 32 / (d / 8), at least ceil(16 / that).
template <typename T, int kSteps>
__global__ void __launch_bounds__(kThreads)
    fa_kv8_append_kernel(const T *k, const T *v, long long k_stride, long long v_stride,
                         const long long *slots, int T_, int window, const KvStore c) {
  constexpr int kWarps = kThreads / 32;
  __shared__ int s_row[kWarps][16];            // a warp's rows by the token in the block
  __shared__ float s_top[2][kWarps];           // runs in turn
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int heads = 2 * c.Hk, hv = static_cast<int>(blockIdx.x % heads), h = hv / 2;
  const bool is_v = hv & 1;
  const T *x = is_v ? v : k;
  const long long stride = is_v ? v_stride : k_stride;
  uint8_t *codes = is_v ? c.v_codes : c.k_codes;
  float *scales = reinterpret_cast<float *>(is_v ? c.v_scales : c.k_scales);
  const long long all = static_cast<long long>(c.num_blocks) << c.bs_log2;
  const int off_mask = (1 << c.bs_log2) - 1;
  const int team_log2 = c.bs_log2 - 4, team = warp >> team_log2, teams = kWarps >> team_log2;
  const int mate = warp - (team << team_log2);  // which 16 tokens of the block
  auto slot_at = [&](long long t) -> long long {
    const long long s = t >= 0 && t < T_ ? __ldg(slots + t) : -1;
    return s < all ? s : -1;
  };
  // a warp takes `per` rows at a time, d / 8 lanes each
  const int lanes = c.d / 8, per = 32 / lanes, sub = lane / lanes, col = (lane - sub * lanes) * 8;
  const T *src = x + static_cast<long long>(h) * c.d + col;
  int runs = 0;  // begun in the window so far
  int turn = 0;
  const long long w0 = static_cast<long long>(blockIdx.x / heads) * window;
  long long before = -1;  // the block of the last row that counts ahead of the rows at hand
  for (int part = 0; part < window; part += 32) {
    const long long t0 = w0 + part;
    if (t0 >= T_) break;
    const long long mine = lane < window - part ? slot_at(t0 + lane) : -1;
    const unsigned there = __ballot_sync(~0u, mine >= 0);
    if (there == 0) continue;
    for (long long t = t0; before < 0 && t > 0; t -= 32) {
      const long long s = slot_at(t - 32 + lane);
      const unsigned some = __ballot_sync(~0u, s >= 0);
      if (some) before = __shfl_sync(~0u, s, 31 - __clz(some)) >> c.bs_log2;
    }
    const unsigned lower = there & ((1u << lane) - 1u);
    const long long prev = __shfl_sync(~0u, mine, lower ? 31 - __clz(lower) : 0) >> c.bs_log2;
    const bool leads = mine >= 0 && (mine >> c.bs_log2) != (lower ? prev : before);
    unsigned leaders = __ballot_sync(~0u, leads);
    before = __shfl_sync(~0u, mine, 31 - __clz(there)) >> c.bs_log2;
    while (leaders) {
      const int first = __ffs(leaders) - 1;
      leaders &= leaders - 1;
      const long long block = __shfl_sync(~0u, mine, first) >> c.bs_log2;
      if (runs++ % teams != team) continue;  // (the whole team)
      // the run's rows among this warp's tokens, and its first token
      if (lane < 16) s_row[warp][lane] = -1;
      __syncwarp();
      int low = off_mask;
      for (long long base = t0 + first; base < T_; base += 32) {
        const long long s = slot_at(base + lane);
        const unsigned stop = __ballot_sync(~0u, s >= 0 && (s >> c.bs_log2) != block);
        const unsigned in = stop ? (stop & (0u - stop)) - 1u : ~0u;
        if (s >= 0 && (in >> lane & 1)) {
          const int off = static_cast<int>(s) & off_mask;
          low = min(low, off);
          if (off >> 4 == mate) s_row[warp][off & 15] = static_cast<int>(base + lane);
        }
        if (stop) break;
      }
      __syncwarp();
      Eight<T> e[kSteps];
      int row[kSteps];
#pragma unroll
      for (int n = 0; n < kSteps; ++n) {
        const int y = n * per + sub;
        row[n] = sub < per && y < 16 ? s_row[warp][y] : -1;
        if (row[n] >= 0) e[n] = load_eight(src + row[n] * stride);
      }
      float *where = scales + block * c.Hk + h;
      float old = *where;
      float top = 0.f;
#pragma unroll
      for (int n = 0; n < kSteps; ++n)
        if (row[n] >= 0) top = size_of<false>(e[n], top);
      for (int o = 16; o; o /= 2) {
        top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
        low = min(low, __shfl_xor_sync(~0u, low, o));
      }
      float finite = top;
      if (top == INFINITY) {
        finite = 0.f;
#pragma unroll
        for (int n = 0; n < kSteps; ++n)
          if (row[n] >= 0) finite = size_of<true>(e[n], finite);
        for (int o = 16; o; o /= 2) finite = fmaxf(finite, __shfl_xor_sync(~0u, finite, o));
      }
      if (team_log2 > 0) {
        if (lane == 0) s_top[turn][warp] = finite;
        named_bar_sync(1 + team, 32 << team_log2);
        for (int n = 0; n < 1 << team_log2; ++n)
          finite = fmaxf(finite, s_top[turn][(team << team_log2) + n]);
        turn ^= 1;
      }
      const float fit = scale_for(finite);
      float scale = fit;
      uint8_t *to = codes + ((((block * c.Hk + h) << c.bs_log2) + 16 * mate) * c.d) + col;
      if (low > 0) {
        old = old > 0.f && old < INFINITY ? old : 0.f;
        scale = fmaxf(old, fit);
        if (scale != old) {
          const float by = __fdiv_rn(old, scale);
          for (int y = sub; y < min(low - 16 * mate, 16); y += per) {
            uint2 *p = reinterpret_cast<uint2 *>(to + y * c.d);
            if (sub < per) *p = rescaled(*p, by);
          }
        }
      }
      const bool exact = (__float_as_uint(scale) & 0x7FFFFFu) == 0;  // (and not subnormal)
      const float by = exact ? __frcp_rn(scale) : scale;
#pragma unroll
      for (int n = 0; n < kSteps; ++n)
        if (row[n] >= 0)
          *reinterpret_cast<uint2 *>(to + (n * per + sub) * c.d) = codes_of(e[n], by, exact);
      // every warp of the team has read the old scale: one alone here, or the barrier
      __syncwarp();
      if (mate == 0 && lane == 0) *where = scale;
    }
  }
}

// 16 elements from their codes and scale.
template <typename T>
__device__ __forceinline__ void expand(uint4 codes, float scale, T *out, bool wide) {
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
  alignas(32) T e[16];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 lo = f16x2_f32(e4m3x2_f16x2(w[j])), hi = f16x2_f32(e4m3x2_f16x2_hi(w[j]));
    e[4 * j] = static_cast<T>(lo.x * scale);
    e[4 * j + 1] = static_cast<T>(lo.y * scale);
    e[4 * j + 2] = static_cast<T>(hi.x * scale);
    e[4 * j + 3] = static_cast<T>(hi.y * scale);
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
    fa_kv8_gather_kernel(const long long *slots, int R, const KvStore c, T *k_out, T *v_out,
                         bool wide) {
  griddep_wait();
  griddep_launch_dependents();
  const int groups = c.d / 16, per_row = c.Hk * groups;
  const long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  long long row;
  int hg;
  if (i >> 32 == 0) {  // the common case: a 32-bit division
    const unsigned u = static_cast<unsigned>(i);
    row = u / per_row, hg = static_cast<int>(u - static_cast<unsigned>(row) * per_row);
  } else {
    row = i / per_row, hg = static_cast<int>(i - row * per_row);
  }
  if (row >= R) return;
  const int h = hg / groups, g = hg - h * groups;
  const long long slot = __ldg(slots + row);
  uint4 kc = make_uint4(0, 0, 0, 0), vc = kc;
  float ks = 0.f, vs = 0.f;
  if (slot >= 0 && slot < (static_cast<long long>(c.num_blocks) << c.bs_log2)) {
    const long long block = (slot >> c.bs_log2) * c.Hk + h;
    const long long at = ((block << c.bs_log2) + (slot & ((1 << c.bs_log2) - 1))) * c.d + g * 16;
    kc = __ldg(reinterpret_cast<const uint4 *>(c.k_codes + at));
    vc = __ldg(reinterpret_cast<const uint4 *>(c.v_codes + at));
    ks = __ldg(reinterpret_cast<const float *>(c.k_scales) + block);
    vs = __ldg(reinterpret_cast<const float *>(c.v_scales) + block);
  }
  const long long to = (row * per_row + hg) * 16;
  expand(kc, ks, k_out + to, wide);
  expand(vc, vs, v_out + to, wide);
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

template <typename T, int kSteps>
cudaError_t append_steps(const void *k, const void *v, long long ks, long long vs,
                         const long long *slots, int T_, const KvStore &c, cudaStream_t s) {
  // Windows of as many rows as a CTA has teams where the rows are few (each may begin a
  // run), of up to 64 where they are many.
  const long long heads = 2LL * c.Hk;
  int window = kThreads / 32 >> (c.bs_log2 - 4);
  while (window < kWindow && (T_ + window - 1LL) / window * heads > 2048) window *= 2;
  const long long ctas = (T_ + window - 1LL) / window * heads;
  return launch<const T *, const T *, long long, long long, const long long *, int, int,
                const KvStore>(fa_kv8_append_kernel<T, kSteps>, ctas * kThreads, s,
                               static_cast<const T *>(k), static_cast<const T *>(v), ks, vs, slots,
                               T_, window, c);
}

template <typename T>
cudaError_t append(const void *k, const void *v, long long ks, long long vs,
                   const long long *slots, int T_, const KvStore &c, cudaStream_t s) {
  const int per = 32 / (c.d / 8), steps = (16 + per - 1) / per;
  if (steps <= 4) return append_steps<T, 4>(k, v, ks, vs, slots, T_, c, s);
  if (steps <= 8) return append_steps<T, 8>(k, v, ks, vs, slots, T_, c, s);
  return append_steps<T, 16>(k, v, ks, vs, slots, T_, c, s);
}

template <typename T>
cudaError_t gather(const long long *slots, int R, const KvStore &c, void *k, void *v,
                   cudaStream_t s) {
  const bool wide = (reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) % 32 == 0;
  return launch<const long long *, int, const KvStore, T *, T *, bool>(
      fa_kv8_gather_kernel<T>, static_cast<long long>(R) * c.Hk * (c.d / 16), s, slots, R, c,
      static_cast<T *>(k), static_cast<T *>(v), wide);
}

}  // namespace

cudaError_t launch_kv8_append(const void *k, const void *v, long long k_stride, long long v_stride,
                              const long long *slots, int T, const KvStore &c, int dtype,
                              cudaStream_t s) {
  if (dtype == FA_DTYPE_BF16)
    return append<__nv_bfloat16>(k, v, k_stride, v_stride, slots, T, c, s);
  if (dtype == FA_DTYPE_F16) return append<__half>(k, v, k_stride, v_stride, slots, T, c, s);
  return append<float>(k, v, k_stride, v_stride, slots, T, c, s);
}

cudaError_t launch_kv8_gather(const long long *slots, int R, const KvStore &c, void *k_out,
                              void *v_out, int dtype, cudaStream_t s) {
  if (dtype == FA_DTYPE_BF16) return gather<__nv_bfloat16>(slots, R, c, k_out, v_out, s);
  if (dtype == FA_DTYPE_F16) return gather<__half>(slots, R, c, k_out, v_out, s);
  return gather<float>(slots, R, c, k_out, v_out, s);
}

}  // namespace fa
