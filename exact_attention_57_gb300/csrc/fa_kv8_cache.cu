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
// run.  A CTA finds the runs that begin in a window of rows and takes them for a share
// of the pairs (K or V, key head), so that finding them is paid once for several:
//   few runs (prompts): a team of bs / 16 warps takes a run, pair after pair, a warp the
//     rows of 16 of the block's tokens, all loaded at once and kept in registers between
//     the maximum, which the team shares through shared memory, and the codes;
//   many (new tokens of many requests): a warp takes a run, lanes and registers spread
//     over the pairs.
// Rows that are skipped, as those that fill a padded batch, are looked at by the whole
// CTA, once: 64 new tokens in a batch of 4096 rows take 7.8 us (187 when each warp walked
// to the end of its run, 32 rows a step, for each of its pairs), in one of 8192 20 (135).
//
// 30299 rows of 4 prompts (8 heads of 128, fp16) take 44 us, 4.2 TB/s or 62% of the copy
// rate (fp32 62; its variant of four steps spills 64 bytes a thread): a CTA finds its runs,
// loads, meets its team, converts and stores in turn, and the three of an SM cover for one
// another only in part.  A warp a run and pair, with divisions in line, took 105; slots read
// anew for every 32 rows of the window 48; the next pair's loads into registers as they fall
// free 49 (registers spill; with two CTAs 51).  Reading 30299 rows back takes 30 us, 6.3 TB/s
// (93%); one row of each of 64 requests 3.7 us and reading them back 1.8, a launch each.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
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

// The largest size among elements; infinity if there is one or, of 16 bits, a NaN among
// them (of 32 bits, NaNs do not count).
template <typename T>
struct Largest {
  using P = std::conditional_t<std::is_same_v<T, __half>, __half2, __nv_bfloat162>;
  std::conditional_t<sizeof(T) == 4, float, P> top;

  __device__ __forceinline__ Largest() {
    if constexpr (sizeof(T) == 4) top = 0.f;
    else top = pair(0.f);
  }
  static __device__ __forceinline__ P pair(float x) {
    if constexpr (std::is_same_v<T, __half>) return __float2half2_rn(x);
    else return __float2bfloat162_rn(x);
  }
  __device__ __forceinline__ void add(const Eight<T> &x) {
    if constexpr (sizeof(T) == 4) {
      const float *e = reinterpret_cast<const float *>(&x);
#pragma unroll
      for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(e[j]));
    } else {
      const P *p = reinterpret_cast<const P *>(&x);
#pragma unroll
      for (int j = 0; j < 4; ++j) top = __hmax2_nan(top, __habs2(p[j]));
    }
  }
  __device__ __forceinline__ float get() const {
    if constexpr (sizeof(T) == 4) {
      return top;
    } else {
      const float a = static_cast<float>(top.x), b = static_cast<float>(top.y);
      return a <= FLT_MAX && b <= FLT_MAX ? fmaxf(a, b) : INFINITY;
    }
  }
};
// The larger of `top` and the elements' finite sizes.
template <typename T>
__device__ __forceinline__ float finite_size(const Eight<T> &x, float top) {
  const T *e = reinterpret_cast<const T *>(&x);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float a = fabsf(static_cast<float>(e[j]));
    top = fmaxf(top, a == INFINITY ? 0.f : a);
  }
  return top;
}

__device__ __forceinline__ bool power_of_two(float scale) {  // (and not subnormal: 2^-40 at least)
  return (__float_as_uint(scale) & 0x7FFFFFu) == 0;
}

// Whether codes_by does for elements whose largest size is not infinity (`plain`).  The
// caches that fa_kv8_append fills have no other scales than powers of two; fp16 elements
// are scaled in fp16, so 1 / scale has to be one of its normal numbers.
template <typename T>
__device__ __forceinline__ bool quick(float scale, bool plain) {
  return plain && power_of_two(scale) &&
         (!std::is_same_v<T, __half> || (scale >= 0x1p-15f && scale <= 0x1p14f));
}

// Eight codes, by 1 / scale, a power of two: an exact product (of fp16 elements, unless
// it is below 2^-14, where every code is zero).  An fp32 NaN becomes 448.
template <typename T>
__device__ __forceinline__ uint2 codes_by(const Eight<T> &x, float inv) {
  uint32_t c[4];
  if constexpr (std::is_same_v<T, __half>) {
    const __half2 by = __float2half2_rn(inv);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __half2 y = __hmul2(reinterpret_cast<const __half2 *>(&x)[j], by);
      c[j] = f16x2_e4m3x2(reinterpret_cast<const uint32_t &>(y));
    }
  } else if constexpr (std::is_same_v<T, __nv_bfloat16>) {
    const __nv_bfloat162 by = __float2bfloat162_rn(inv);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 y = __bfloat1622float2(__hmul2(reinterpret_cast<const __nv_bfloat162 *>(&x)[j], by));
      c[j] = f32x2_e4m3x2(y.x, y.y);
    }
  } else {
    const float *e = reinterpret_cast<const float *>(&x);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c[j] = f32x2_e4m3x2(fminf(e[2 * j] * inv, 448.f), fminf(e[2 * j + 1] * inv, 448.f));
  }
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}
// For any scale and elements, a NaN becoming 448 (not inlined: eight correctly rounded
// divisions; in line, they made the kernel's every element pay for their branches).
template <typename T>
__device__ __noinline__ uint2 codes_over(Eight<T> x, float scale) {
  const T *e = reinterpret_cast<const T *>(&x);
  uint32_t c[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    c[j] = f32x2_e4m3x2(fminf(__fdiv_rn(static_cast<float>(e[2 * j]), scale), 448.f),
                        fminf(__fdiv_rn(static_cast<float>(e[2 * j + 1]), scale), 448.f));
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// Eight codes times `by`, as codes; with a scale that does not count, `by` is 0, and a
// NaN among them (of memory that nobody has written, say) is none of its values.
__device__ __forceinline__ uint2 rescaled(uint2 c, float by) {
  if (by == 0.f) return make_uint2(0, 0);
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

constexpr int kWarps = kThreads / 32;

template <typename T>
struct Append {
  const T *k, *v;
  long long k_stride, v_stride;
  const long long *slots;
  int T_;
  int window;   // rows of a CTA's window
  int groups;   // CTAs that share a window's pairs
  int per_cta;  // pairs of each
  KvStore c;

  // Pair n: key head n of K, then of V.
  __device__ __forceinline__ const T *rows(int n) const {
    return n < c.Hk ? k + static_cast<long long>(n) * c.d : v + static_cast<long long>(n - c.Hk) * c.d;
  }
  __device__ __forceinline__ long long stride(int n) const { return n < c.Hk ? k_stride : v_stride; }
  // Index of the pair's scale for a block.
  __device__ __forceinline__ long long at(int n, long long block) const {
    return block * c.Hk + (n < c.Hk ? n : n - c.Hk);
  }
  __device__ __forceinline__ float *scales(int n) const {
    return reinterpret_cast<float *>(n < c.Hk ? c.k_scales : c.v_scales);
  }
  __device__ __forceinline__ uint8_t *codes(int n) const { return n < c.Hk ? c.k_codes : c.v_codes; }
  // The slot of row t, -1 for rows that are skipped.
  __device__ __forceinline__ long long slot(long long t) const {
    const long long s = t >= 0 && t < T_ ? __ldg(slots + t) : -1;
    return s < limit() ? s : -1;
  }
  __device__ __forceinline__ long long limit() const {
    return static_cast<long long>(c.num_blocks) << c.bs_log2;
  }
};

constexpr int kMostTokens = 128;  // of a block

// The rows that a CTA looks at, numbered from its window's first: kThreads of them, which
// follow one another, and where the window's last run goes on behind those, the rest of
// its rows, kThreads + t being that of token t of the block.  All in shared memory, so that
// a run is walked at no cost for the rows that are skipped on its way.
struct Slots {
  const long long *near;  // [kThreads]
  const int *far;         // [kMostTokens]: a row, or -1
  long long w0;           // the window's first row
  int end;                // behind the last that counts

  // The slot of row i, which may be one of the last run's, in `block`.
  __device__ __forceinline__ long long at(int i, long long block, int bs_log2) const {
    if (i < kThreads) return near[i];
    return far[i - kThreads] >= 0 ? (block << bs_log2) + (i - kThreads) : -1;
  }
  __device__ __forceinline__ long long row(int i) const {
    return i < kThreads ? w0 + i : far[i - kThreads];
  }
};

// Rows that a thread looks at side by side, outside the window.
constexpr int kAtOnce = 16;

// The slots of rows from + step * (thread, thread + kThreads, ...), as far as there are rows
// (else -1): all loads ahead of what is made of them (one after the other they took 4.4 us
// for a CTA's 4096 rows).
__device__ __forceinline__ void look(const long long *slots, int T, long long limit, long long from,
                                     int step, long long (&s)[kAtOnce]) {
#pragma unroll
  for (int i = 0; i < kAtOnce; ++i) {
    const long long t = from + step * static_cast<int>(i * kThreads + threadIdx.x);
    s[i] = __ldg(slots + min(max(t, 0LL), T - 1LL));
  }
#pragma unroll
  for (int i = 0; i < kAtOnce; ++i) {
    const long long t = from + step * static_cast<int>(i * kThreads + threadIdx.x);
    s[i] = t >= 0 && t < T && s[i] < limit ? s[i] : -1;
  }
}

// The least of `x` over the CTA.
__device__ __forceinline__ unsigned least_of(unsigned x, unsigned *least) {
  x = __reduce_min_sync(~0u, x);
  if ((threadIdx.x & 31) == 0) least[threadIdx.x / 32] = x;
  __syncthreads();
  for (int w = 0; w < kWarps; ++w) x = min(x, least[w]);
  return x;
}

// Notes the rows of `block` from row `from` on, up to the first of another block, in far
// (of -1 before), by the whole CTA; whether there are any.
__device__ __noinline__ bool find_far(const long long *slots, int T, long long limit, int bs_log2,
                                      long long from, long long block, int *far, unsigned *least) {
  constexpr unsigned kChunk = kAtOnce * kThreads;
  const int off_mask = (1 << bs_log2) - 1;
  bool found = false;
  for (; from < T; from += kChunk) {
    long long s[kAtOnce];
    look(slots, T, limit, from, 1, s);
    unsigned other = kChunk;  // the first row of another block
    bool some = false;
#pragma unroll
    for (int i = kAtOnce - 1; i >= 0; --i) {
      some |= s[i] >= 0;
      if (s[i] >= 0 && s[i] >> bs_log2 != block) other = i * kThreads + threadIdx.x;
    }
    if (!__syncthreads_or(some)) continue;
    other = least_of(other, least);
    bool mine = false;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const unsigned n = i * kThreads + threadIdx.x;
      if (s[i] >= 0 && s[i] >> bs_log2 == block && n < other) {
        far[static_cast<int>(s[i]) & off_mask] = static_cast<int>(from + n);
        mine = true;
      }
    }
    found |= __syncthreads_or(mine) != 0;
    if (other < kChunk) break;
  }
  return found;
}

// The slot of the last row that counts ahead of row `to`, or -1, by the whole CTA.  (Read
// once, as all slots are: warps that saw different ones would wait for one another in vain.)
__device__ __noinline__ long long find_back(const long long *slots, int T, long long limit,
                                            long long to, unsigned *least, long long *found) {
  constexpr unsigned kChunk = kAtOnce * kThreads;
  for (; to > 0; to -= kChunk) {
    long long s[kAtOnce];
    look(slots, T, limit, to - 1, -1, s);
    unsigned back = kChunk;
#pragma unroll
    for (int i = kAtOnce - 1; i >= 0; --i)
      if (s[i] >= 0) back = i * kThreads + threadIdx.x;
    if (!__syncthreads_or(back < kChunk)) continue;
    back = least_of(back, least);
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
      if (back == i * kThreads + threadIdx.x) *found = s[i];
    __syncthreads();
    return *found;
  }
  return -1;
}

// The scale of a block that held `old`; *by: what its codes are multiplied with.
__device__ __forceinline__ float grown(float old, float fit, float *by) {
  old = old > 0.f && old < INFINITY ? old : 0.f;
  const float scale = fmaxf(old, fit);
  *by = __fdiv_rn(old, scale);
  return scale;
}

// A run: the rows of one block that follow one another.  Of rows base .. base + 31 the
// lanes hold the slots, and `in` has those of the run; `more`: it may go on behind them.
struct Run {
  int base;
  long long slot, block;
  unsigned in;
  bool more;

  // The part of it among rows `from` .. `from` + 31 of `slots`.
  __device__ __forceinline__ Run(const Slots &slots, int bs_log2, int from, long long slot, int first,
                                 long long block)
      : base(from), slot(slot), block(block) {
    const bool ahead = (threadIdx.x & 31) < first;
    const unsigned stop = __ballot_sync(~0u, !ahead && slot >= 0 && (slot >> bs_log2) != block);
    in = __ballot_sync(~0u, !ahead && slot >= 0) & (stop ? (stop & (0u - stop)) - 1u : ~0u);
    more = stop == 0 && from + 32 < slots.end;
  }
  __device__ __forceinline__ Run next(const Slots &slots, int bs_log2) const {
    return Run(slots, bs_log2, base + 32, slots.at(base + 32 + (threadIdx.x & 31), block, bs_log2), 0,
               block);
  }
};

// f(row, token of the block) for each row of a run, by the whole warp.
template <typename F>
__device__ __forceinline__ void for_rows(const Slots &slots, int bs_log2, Run run, F f) {
  const int off_mask = (1 << bs_log2) - 1;
  for (;;) {
    for (unsigned in = run.in; in; in &= in - 1) {
      const int j = __ffs(in) - 1;
      f(slots.row(run.base + j), static_cast<int>(__shfl_sync(~0u, run.slot, j)) & off_mask);
    }
    if (!run.more) break;
    run = run.next(slots, bs_log2);
  }
}

// A run by one warp, pairs [n0, n1): `lanes` (a power of two) lanes a row, as many pairs
// side by side as there are lanes for.
template <typename T>
__device__ __forceinline__ void append_across(const Append<T> &p, const Slots &slots, const Run &run,
                                              int n0, int n1) {
  const int lane = threadIdx.x & 31, per_row = p.c.d / 8;
  const int lanes = 1 << (32 - __clz(per_row - 1)), per = 32 / lanes;  // (per_row 2 .. 32)
  const int sub = lane / lanes, x = lane - sub * lanes, col = x * 8;
  for (int n = n0 + sub; n - sub < n1; n += per) {
    const bool on = n < n1 && x < per_row;
    const T *src = p.rows(on ? n : n0) + (on ? col : 0);
    const long long stride = p.stride(on ? n : n0), at = p.at(on ? n : n0, run.block);
    const float old = p.scales(on ? n : n0)[at];
    Eight<T> e;
    Largest<T> largest;
    int low = 1 << p.c.bs_log2, rows = 0;
    for_rows(slots, p.c.bs_log2, run, [&](long long row, int off) {
      low = min(low, off);
      ++rows;
      e = load_eight(src + row * stride);
      if (on) largest.add(e);
    });
    float top = largest.get();
    for (int o = 1; o < lanes; o *= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    const bool plain = top < INFINITY;
    if (__any_sync(~0u, !plain)) {  // infinities, which do not count
      top = 0.f;
      for_rows(slots, p.c.bs_log2, run, [&](long long row, int) {
        if (on) top = finite_size(load_eight(src + row * stride), top);
      });
      for (int o = 1; o < lanes; o *= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    }
    float scale = scale_for(top), by = 1.f;
    if (low > 0) scale = grown(old, scale, &by);
    uint8_t *to = p.codes(on ? n : n0) + (at << p.c.bs_log2) * p.c.d + col;
    if (on && by != 1.f) {
      for (int off = 0; off < low; ++off) {
        uint2 *c = reinterpret_cast<uint2 *>(to + off * p.c.d);
        *c = rescaled(*c, by);
      }
    }
    const float inv = __frcp_rn(scale);
    for_rows(slots, p.c.bs_log2, run, [&](long long row, int off) {
      if (rows > 1) e = load_eight(src + row * stride);
      if (on)
        *reinterpret_cast<uint2 *>(to + off * p.c.d) =
            quick<T>(scale, plain) ? codes_by(e, inv) : codes_over(e, scale);
    });
    __syncwarp();  // (all lanes have read the old scales)
    if (on && x == 0) p.scales(n)[at] = scale;
  }
}

// A run by a team of bs / 16 warps, pair after pair; a warp takes the block's tokens 16
// mate and on.  kSteps: rounds of loads for 16 rows.  map: 16 rows a warp; top_of: a
// number a warp, twice, in turn.
template <typename T, int kSteps>
__device__ __forceinline__ void append_along(const Append<T> &p, const Slots &slots, const Run &whole,
                                             int n0, int n1, int *map, float (*top_of)[kWarps],
                                             int *turn) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int team_log2 = p.c.bs_log2 - 4, team = warp >> team_log2;
  const int mate = warp - (team << team_log2), off_mask = (1 << p.c.bs_log2) - 1;
  const int lanes = p.c.d / 8, per = 32 / lanes, sub = lane / lanes, col = (lane - sub * lanes) * 8;
  // the run's rows among this warp's tokens, and its first token
  __syncwarp();
  if (lane < 16) map[lane] = -1;
  __syncwarp();
  int low = off_mask;
  for (Run run = whole;; run = run.next(slots, p.c.bs_log2)) {
    if (run.in >> lane & 1) {
      const int off = static_cast<int>(run.slot) & off_mask;
      low = min(low, off);
      if (off >> 4 == mate) map[off & 15] = static_cast<int>(slots.row(run.base + lane));
    }
    if (!run.more) break;
  }
  for (int o = 16; o; o /= 2) low = min(low, __shfl_xor_sync(~0u, low, o));
  __syncwarp();
  // the row of round i for this lane, or -1
  auto row_of = [&](int i) { return sub < per && i * per + sub < 16 ? map[i * per + sub] : -1; };
  for (int n = n0; n < n1; ++n) {
    const T *src = p.rows(n) + col;
    const long long stride = p.stride(n), at = p.at(n, whole.block);
    Eight<T> e[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int row = row_of(i);
      if (row >= 0)
        e[i] = load_eight(src + row * stride);
      else
#pragma unroll
        for (uint4 &w : e[i].w) w = make_uint4(0, 0, 0, 0);
    }
    const float old = p.scales(n)[at];
    Largest<T> largest;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) largest.add(e[i]);
    float top = largest.get();
    for (int o = 16; o; o /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    const bool plain = top < INFINITY;
    if (!plain) {
      top = 0.f;
#pragma unroll 1
      for (int i = 0; i < kSteps; ++i)
        if (row_of(i) >= 0) top = finite_size(load_eight(src + row_of(i) * stride), top);
      for (int o = 16; o; o /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    }
    if (team_log2 > 0) {
      if (lane == 0) top_of[*turn][warp] = top;
      named_bar_sync(1 + team, 32 << team_log2);
      for (int w = 0; w < 1 << team_log2; ++w) top = fmaxf(top, top_of[*turn][(team << team_log2) + w]);
      *turn ^= 1;
    }
    float scale = scale_for(top), by = 1.f;
    uint8_t *to = p.codes(n) + ((at << p.c.bs_log2) + 16 * mate) * p.c.d + col;
    if (low > 0) scale = grown(old, scale, &by);
    if (by != 1.f) {
      for (int y = sub; y < min(low - 16 * mate, 16); y += per) {
        uint2 *c = reinterpret_cast<uint2 *>(to + y * p.c.d);
        if (sub < per) *c = rescaled(*c, by);
      }
    }
    if (quick<T>(scale, plain)) {
      const float inv = __frcp_rn(scale);
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
        if (row_of(i) >= 0) *reinterpret_cast<uint2 *>(to + (i * per + sub) * p.c.d) = codes_by(e[i], inv);
    } else {
#pragma unroll 1
      for (int i = 0; i < kSteps; ++i)
        if (row_of(i) >= 0)
          *reinterpret_cast<uint2 *>(to + (i * per + sub) * p.c.d) =
              codes_over(load_eight(src + row_of(i) * stride), scale);
    }
    // the whole team has read the old scale: a warp alone here, others ahead of the barrier
    __syncwarp();
    if (mate == 0 && lane == 0) p.scales(n)[at] = scale;
  }
}

template <typename T, int kSteps>
__global__ void __launch_bounds__(kThreads, kSteps * sizeof(T) <= 16 ? 3 : kSteps * sizeof(T) <= 32 ? 2 : 1)
    fa_kv8_append_kernel(const __grid_constant__ Append<T> p) {
  __shared__ int s_map[kWarps][16];
  __shared__ float s_top[2][kWarps];
  __shared__ long long s_slots[kThreads], s_ahead[32];
  __shared__ unsigned s_there[kWarps], s_least[kWarps];  // rows of s_slots that count
  __shared__ int s_far[kMostTokens];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int bs_log2 = p.c.bs_log2, team_log2 = bs_log2 - 4;
  const int team = warp >> team_log2, teams = kWarps >> team_log2;
  const int group = static_cast<int>(blockIdx.x % p.groups);
  const long long w0 = static_cast<long long>(blockIdx.x / p.groups) * p.window;
  const int n0 = group * p.per_cta, n1 = min(n0 + p.per_cta, 2 * p.c.Hk);
  const long long near = p.slot(w0 + threadIdx.x);
  // (with the loads of the window's own: mostly it is the row ahead that tells)
  const long long ahead = p.slot(w0 - 32 + lane);
  s_slots[threadIdx.x] = near;
  const unsigned counts = __ballot_sync(~0u, near >= 0);
  if (lane == 0) s_there[warp] = counts;
  if (warp == 0) s_ahead[lane] = ahead;
  __syncthreads();
  // the last row that counts in the window, and among the rows at hand
  const unsigned at_hand = lane < kWarps ? s_there[lane] : 0u;
  const int left = p.window - 32 * lane;
  const unsigned inside = left >= 32 ? at_hand : left > 0 ? at_hand & ((1u << left) - 1u) : 0u;
  auto last_of = [](unsigned rows) {  // of 32 rows a lane
    const int at = 31 - __clz(__ballot_sync(~0u, rows != 0));
    return 32 * at + 31 - __clz(__shfl_sync(~0u, rows, at & 31));
  };
  if (!__any_sync(~0u, inside != 0)) return;
  const int last = last_of(inside), last_near = last_of(at_hand);
  // the block of the last row that counts ahead of the window's
  long long before = -1;
  if (w0 > 0) {
    const unsigned some = __ballot_sync(~0u, s_ahead[lane] >= 0);
    before = (some ? s_ahead[31 - __clz(some)]
                   : find_back(p.slots, p.T_, p.limit(), w0 - 32, s_least, s_ahead)) >> bs_log2;
  }
  // The window's last run may go on behind the rows at hand, if no other block's follow:
  // skipped rows may lie between its rows.
  const long long block = s_slots[last] >> bs_log2;
  Slots slots = {s_slots, s_far, w0, last_near + 1};
  if (s_slots[last_near] >> bs_log2 == block && w0 + kThreads < p.T_) {
    if (threadIdx.x < kMostTokens) s_far[threadIdx.x] = -1;
    __syncthreads();
    if (find_far(p.slots, p.T_, p.limit(), bs_log2, w0 + kThreads, block, s_far, s_least))
      slots.end = kThreads + (1 << bs_log2);
  }
  int runs = 0, turn = 0;
  for (int part = 0; part < p.window; part += 32) {
    const long long mine = s_slots[part + lane];  // (also behind the window)
    const unsigned own = p.window - part < 32 ? (1u << (p.window - part)) - 1u : ~0u;
    const unsigned there = __ballot_sync(~0u, mine >= 0) & own;
    if (there == 0) continue;
    const unsigned lower = there & ((1u << lane) - 1u);
    const long long prev = __shfl_sync(~0u, mine, lower ? 31 - __clz(lower) : 0) >> bs_log2;
    const bool leads = (there >> lane & 1) && (mine >> bs_log2) != (lower ? prev : before);
    unsigned leaders = __ballot_sync(~0u, leads);
    before = __shfl_sync(~0u, mine, 31 - __clz(there)) >> bs_log2;
    // runs of up to four rows, on average: a warp each
    const bool many = __popc(leaders) * 4 >= __popc(there);
    while (leaders) {
      const int first = __ffs(leaders) - 1;
      leaders &= leaders - 1;
      if (runs++ % (many ? kWarps : teams) != (many ? warp : team)) continue;
      const Run run(slots, bs_log2, part, mine, first, __shfl_sync(~0u, mine, first) >> bs_log2);
      if (many)
        append_across(p, slots, run, n0, n1);
      else
        append_along<T, kSteps>(p, slots, run, n0, n1, s_map[warp], s_top, &turn);
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

template <typename T>
cudaError_t append(const void *k, const void *v, long long ks, long long vs,
                   const long long *slots, int T_, const KvStore &c, cudaStream_t s) {
  Append<T> p = {static_cast<const T *>(k), static_cast<const T *>(v), ks, vs, slots, T_, 0, 0, 0, c};
  // Windows of a row a warp where the rows are few, since each may begin a run, else of
  // 16 rows a warp, as teams take them; about a thousand CTAs, but no fewer pairs each
  // than a warp's lanes hold of one row.  (In us when the prompts above took 49, windows of
  // 8 / 16 / 32 / 64 / 128 rows: 8192 rows of one prompt 47 / 29 / 20 / 25 / 21, those
  // prompts 262 / 58 / 54 / 57 / 49; one row of each of 4500 requests 26 / 30 / 38 / 45 / 53,
  // of 2504 17 / 24 / 24 / 27 / -: batches above 4096 requests pay for the prompts.  Now 512
  // / 640 / 1024 / 1800 CTAs: 44 / 44 / 45 / 47, the same in blocks of 16 tokens 49 / 49 / 45
  // / -, 2048 rows of one prompt 19 / 16 / 13 / -.)
  p.window = T_ <= 4096 ? kWarps : 16 * kWarps;
  const long long windows = (T_ + p.window - 1LL) / p.window;
  const int per = 32 / (c.d / 8), pairs = 2 * c.Hk, most = (pairs + per - 1) / per;
  const long long want = (1024 + windows - 1) / windows;
  p.groups = static_cast<int>(want < most ? want : most);
  p.per_cta = (pairs + p.groups - 1) / p.groups;
  p.groups = (pairs + p.per_cta - 1) / p.per_cta;
  const long long threads = windows * p.groups * kThreads;
  const int steps = (16 + per - 1) / per;
  if (steps <= 4) return launch<const Append<T>>(fa_kv8_append_kernel<T, 4>, threads, s, p);
  if (steps <= 8) return launch<const Append<T>>(fa_kv8_append_kernel<T, 8>, threads, s, p);
  return launch<const Append<T>>(fa_kv8_append_kernel<T, 16>, threads, s, p);
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
