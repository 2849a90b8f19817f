// fa_kv4_split.cuh — how the attention kernels over the 4-bit cache deal their
// work: all tiles of all sequences lie in one line of units (a unit is a step
// along the keys), every CTA takes an equal share of the line, and tiles that
// shares cut are joined by a second kernel from parts in the workspace.
#pragma once

#include "fa_kv4.cuh"
#include "fa_serve.h"
#include "ptx.cuh"

namespace fa {

// One sequence as this kernel sees it.
struct Seq {
  int r0, nq, nk;
};

__device__ __forceinline__ Seq load_seq(const Kv4Attn &p, int b) {
  Seq s = {b, 1, 0};
  if (p.cu_q) {
    s.r0 = min(max(p.cu_q[b], 0), p.total_q);
    s.nq = min(max(min(max(p.cu_q[b + 1], 0), p.total_q) - s.r0, 0), p.max_q);
  }
  s.nk = min(max(p.lens[b], 0), p.max_k);  // (max_k keeps to the table's width)
  return s;
}

// Weights are 2^(s - m) with m = (the maximum so far) - kHeadroom, and m follows
// the maximum once that has grown by more than kGrow: 2^(kHeadroom + kGrow) at
// most, which fp16 holds, while a weight down to 2^-21 of the largest is still a
// normal fp16 number.  Of the largest weight itself, 2^-32 is the most that
// fp16's subnormals take from one; without the headroom it were 2^-25, which
// showed in rows whose value comes from a weight of e^-13 alone.
constexpr float kHeadroom = 7.f, kGrow = 8.f;
static_assert(kHeadroom + kGrow < 16.f, "weights up to 2^15 are finite in fp16");

// A row's results from its m, the sum l of its weights and a sum of weighted
// values (inv = v_mul / l).  l is zero for a row without keys, and for no other
// row whose scores are numbers: its largest weight is 2^kHeadroom.  A NaN among
// the scores of a row is in l, whatever m, and so in its results, as in those of
// fa_fwd; a NaN weight of a part stays one in the sums that join the parts, since
// 0 * NaN is NaN.
__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.f ? -INFINITY : (m + kHeadroom) * 0.6931471805599453f + logf(l * 0.0078125f);
}
__device__ __forceinline__ float value_of(float sum, float l, float inv) {
  return l == 0.f ? 0.f : sum * inv;
}
static_assert(kHeadroom == 7.f, "lse_of divides by 2^kHeadroom");

// What a CTA says to the joining kernel, at the workspace's start, about the
// tile (sequence, key head, query tile) whose first part, but not last, is its
// own: the tile's first query row, key head and rows (0: there is no such
// tile), and the CTA with its last part.
struct Share {
  int row0, h, rows, last;
};
static_assert(sizeof(Share) == 16, "one 16-byte load");

// The CTA whose share of `total` units, dealt to `den` CTAs, holds unit u.
__device__ __forceinline__ int cta_of(long long u, long long total, int den) {
  // the last n with floor(total * n / den) <= u
  return static_cast<int>(((u + 1) * den - 1) / total);
}

// Part `which` (0: of a tile begun before the CTA, 1: of one it begins) of
// CTA n: rows of D sums, then (m, sum of weights) a row.
template <int D, int R>
__device__ __forceinline__ float *part_of(float *ws, int n, int which) {
  return ws + kKv4MaxCtas * (sizeof(Share) / sizeof(float)) +
         static_cast<long long>(2 * n + which) * R * (D + 2);
}

// Where a unit lies in the line of all units.
struct Place {
  long long total;   // units in all
  long long before;  // units before sequence b
  int b;
};

// The place of unit floor(total * num / den), `units(b)` being those of
// sequence b, all key heads (all kWarps * 32 threads get it); den becomes the
// smaller of itself and the units in all.  `sums` holds a prefix sum a thread.
template <int kWarps, typename F>
__device__ Place find_unit(const Kv4Attn &p, F units, int num, int *den, long long *target,
                           long long *sums, long long (*warp_sums)[kWarps]) {
  constexpr int kThreads = kWarps * 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Place at = {0, 0, 0};
  if (p.B <= 32) {
    // one a lane: every warp finds it by itself (0.4 us less than by way of shared
    // memory, of 16.8 for 16 sequences of up to 3001 keys)
    const long long n = lane < p.B ? units(lane) : 0;
    long long incl = n;
    for (int o = 1; o < 32; o *= 2) {
      const long long x = __shfl_up_sync(~0u, incl, o);
      if (lane >= o) incl += x;
    }
    at.total = __shfl_sync(~0u, incl, 31);
    *den = static_cast<int>(min(static_cast<long long>(*den), at.total));
    if (num >= *den) return at;  // more CTAs than units
    *target = at.total * num / *den;
    at.b = 31 - __clz(__ballot_sync(~0u, incl - n <= *target));
    at.before = __shfl_sync(~0u, incl - n, at.b);
    return at;
  }
  // total first, where one round of requests does not show it
  if (p.B > kThreads) {
    long long n = 0;
    for (int b = tid; b < p.B; b += kThreads) n += units(b);
    for (int o = 16; o; o /= 2) n += __shfl_xor_sync(~0u, n, o);
    if (lane == 0) warp_sums[1][warp] = n;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) at.total += warp_sums[1][w];
  }
  for (int base = 0;; base += kThreads) {
    const int b = base + tid;
    const long long n = b < p.B ? units(b) : 0;
    long long incl = n;
    for (int o = 1; o < 32; o *= 2) {
      const long long x = __shfl_up_sync(~0u, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) warp_sums[0][warp] = incl;
    __syncthreads();
    long long pre = at.before, all = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) pre += warp_sums[0][w];
      all += warp_sums[0][w];
    }
    sums[tid] = pre + incl - n;
    __syncthreads();
    if (p.B <= kThreads) at.total = all;
    if (base == 0) {
      *den = static_cast<int>(min(static_cast<long long>(*den), at.total));
      if (num >= *den) return at;  // more CTAs than units
      *target = at.total * num / *den;
    }
    if (*target < at.before + all || base + kThreads >= p.B) {
      int lo = 0, hi = kThreads;  // the last i with sums[i] <= target
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (sums[mid] <= *target) lo = mid;
        else hi = mid;
      }
      at.b = base + lo;
      at.before = sums[lo];
      return at;
    }
    at.before += all;
    __syncthreads();
  }
}

// Joins the parts of the tiles that more than one CTA shared: CTA n takes what
// CTA n of the grid above began and others went on with (n's part 1, then the
// parts 0 of n + 1, n + 2, ... up to the one that ends it), four rows of it.
// Row r of a tile is head r % group of its token r / group.  The eight warps
// share the parts, each with a maximum of its own, so that a tile split over
// the whole grid costs a few rounds of loads: about 4 us, a launch and two
// dependent loads (the counts of finished parts that would let the last CTA join
// them would have to be zero before the call, and the workspace is the caller's).
constexpr int kJoinRows = 4, kJoinThreads = 256;

template <typename T, int D, int R>
__global__ void __launch_bounds__(kJoinThreads) fa_kv4_join_kernel(const Kv4Attn p, float *ws) {
  constexpr int kWarps = kJoinThreads / 32;
  constexpr int W = D / 32;  // columns a lane
  __shared__ float s_sum[kWarps][kJoinRows][D];
  __shared__ float s_m[kWarps][kJoinRows], s_l[kWarps][kJoinRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, first = blockIdx.x;
  const int row0 = blockIdx.y * kJoinRows;
  griddep_wait();
  griddep_launch_dependents();
  const Share mine = reinterpret_cast<const Share *>(ws)[first];
  if (row0 >= mine.rows) return;
  // two parts at a time, all their loads ahead of the sums (rows behind the
  // tile's last repeat it: nothing of them is written)
  float mm[kJoinRows], ll[kJoinRows], sum[kJoinRows][W] = {};
#pragma unroll
  for (int y = 0; y < kJoinRows; ++y) mm[y] = -INFINITY, ll[y] = 0.f;
  constexpr int AT = 2;
  for (int n = first + warp; n <= mine.last; n += AT * kWarps) {
    float2 ml[AT][kJoinRows];
    float v[AT][kJoinRows][W];
#pragma unroll
    for (int x = 0; x < AT; ++x) {
      const int from = min(n + x * kWarps, mine.last);
      const float *src = part_of<D, R>(ws, from, from == first);
#pragma unroll
      for (int y = 0; y < kJoinRows; ++y) {
        const int row = min(row0 + y, mine.rows - 1);
        ml[x][y] = reinterpret_cast<const float2 *>(src + R * D)[row];
        if constexpr (W == 4)
          *reinterpret_cast<float4 *>(v[x][y]) =
              *reinterpret_cast<const float4 *>(src + row * D + lane * 4);
        else
          *reinterpret_cast<float2 *>(v[x][y]) =
              *reinterpret_cast<const float2 *>(src + row * D + lane * 2);
      }
    }
#pragma unroll
    for (int x = 0; x < AT; ++x) {
      if (n + x * kWarps > mine.last) break;
#pragma unroll
      for (int y = 0; y < kJoinRows; ++y) {
        // A part without weights adds nothing.  Leaving it out keeps both parts'
        // loads ahead of the sums (89 registers instead of 66), which a join of few
        // rows wants, whose latency counts (one sequence of 131071 keys 35.5 us
        // instead of 36.2); the many CTAs of a join of 128 rows want the registers
        // (428 us for two chunks of 2048 queries, 437 with it).
        if (R < kKv4ManyRows && ml[x][y].y == 0.f) continue;
        const float to = fmaxf(mm[y], ml[x][y].x), off = to == -INFINITY ? 0.f : to;
        const float f = ex2_approx(mm[y] - off), g = ex2_approx(ml[x][y].x - off);
        mm[y] = to;
        ll[y] = f * ll[y] + g * ml[x][y].y;
#pragma unroll
        for (int z = 0; z < W; ++z) sum[y][z] = f * sum[y][z] + g * v[x][y][z];
      }
    }
  }
#pragma unroll
  for (int y = 0; y < kJoinRows; ++y) {
#pragma unroll
    for (int x = 0; x < W; ++x) s_sum[warp][y][lane * W + x] = sum[y][x];
    if (lane == 0) s_m[warp][y] = mm[y], s_l[warp][y] = ll[y];
  }
  __syncthreads();
  if (warp >= kJoinRows || row0 + warp >= mine.rows) return;
  float m = -INFINITY, l = 0.f, total[W] = {};
#pragma unroll
  for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s_m[w][warp]);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const float f = m == -INFINITY ? 0.f : ex2_approx(s_m[w][warp] - m);
    l += f * s_l[w][warp];
#pragma unroll
    for (int x = 0; x < W; ++x) total[x] += f * s_sum[w][warp][lane * W + x];
  }
  const int row = row0 + warp, y = row / p.group, j = row - y * p.group, i = mine.row0 + y;
  const int head = mine.h * p.group + j;
  T *out = static_cast<T *>(p.o) + (static_cast<long long>(i) * p.Hq + head) * D + lane * W;
  const float inv = p.v_mul / l;
  alignas(8) T e[W];
#pragma unroll
  for (int x = 0; x < W; ++x) e[x] = static_cast<T>(value_of(total[x], l, inv));
  if constexpr (W == 4)
    *reinterpret_cast<uint2 *>(out) = *reinterpret_cast<const uint2 *>(e);
  else
    *reinterpret_cast<uint32_t *>(out) = *reinterpret_cast<const uint32_t *>(e);
  if (lane == 0)
    p.lse[static_cast<long long>(head) * p.total_q + i] = lse_of(m, l);
}

}  // namespace fa
