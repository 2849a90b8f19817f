// fa_kv4_attn.cu — attention of a few queries a sequence over the paged 4-bit
// cache (decoding and drafted tokens): the cache is read once, and every
// query row of a sequence that shares a key head rides along.
//
// Query token i of sequence b (n_q queries, n_k cached tokens, its own among
// them) sees key j iff j < n_k and, when causal, j <= n_k - n_q + i; query
// head h reads key head h / group.  Row i * group + (h mod group) of key head
// h / group is one column of the tile: with Q^T as the B operand,
//   S^T = K Q^T   (m = 16 tokens, n = 8 rows, k = head dim)
//   O^T += V^T P^T  (m = 16 columns of V, n = 8 rows, k = 16 tokens)
// the streamed operand is always the wide A of mma.m16n8k16, so eight rows
// cost no more than one and O^T takes D / 4 registers for eight rows.  (The
// rows are too few for tcgen05, whose tiles have 128: a decode step is bound
// by reading the cache, which keeps the tensor pipe below a third of the time.)
//
// K and V go from global memory to registers and from there to the tensor
// core, with no shared memory: the order of k in S^T and of the columns of
// V^T is free, so lane (r, c) = (lane / 4, lane % 4) takes D / 4 consecutive
// elements of tokens r, r + 8 of K (one 16-byte load each at D = 128) and
// D / 8 consecutive columns of tokens 2c, 2c + 1, 2c + 8, 2c + 9 of V.  Codes
// become fp16 pairs by cvt (V: the nibbles of two tokens are merged into
// bytes first, since a register holds two tokens of one column), times the
// scale, exactly: a value has six significant bits.  Q is brought to fp16 by
// a power of two a row, P is rounded to fp16 (relative 2^-11, one rounding of
// the order of the output's own; kHeadroom keeps it from its subnormals),
// everything is summed in fp32.
//
// Work is dealt in units of 128 tokens (16 for each of 8 warps) of one
// sequence and key head, in one line over all of them, equal shares to the
// CTAs of one resident wave: ragged lengths and few long sequences balance
// alike.  A sequence and key head begins with kLead units that stand for what
// it costs beside its keys (its queries, the pipeline's start, the warps'
// meeting).  A CTA's first and last sequence may be shared with its neighbours;
// such parts go to the workspace (two a CTA, whatever the lengths), and a
// second kernel joins them.  Where one wave of CTAs holds a cluster of 1, 2, 4 or
// 8 for every sequence and key head, and their caches are short, a cluster takes
// the keys of one instead and joins its parts through shared memory.
//
// Measured at 8 key heads of 128 elements, four query heads each: 64 sequences of
// up to 8192 keys (327 MB of cache) 70 us, 4.7 TB/s or 69% of the measured copy
// rate, the loads alone without a product 65; one of 131071 (151 MB) 35 us; one of
// 1023 4.3 us in a captured graph, the latencies of one launch (5.1 to 5.6 a call).
// What bounds it is the time that loads of 64-byte rows take at two tiles in flight
// a warp, and about 330 instructions a tile of 16 tokens.  Not faster: codes through
// shared memory by bulk copies (75 to 87 us), tiles of 32 tokens (91), a third tile
// in registers (77 to 80 at 128 elements, spilling; no change at 64), prefetches
// into L2 two tiles ahead (83).
#include <atomic>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa.h"
#include "fa_internal.h"
#include "fa_kv4_split.cuh"

namespace fa {
namespace {

// Warps of a CTA, resident CTAs, and the units that stand for a sequence's cost
// beside its keys, by rows (8 NT) and head dim.  Measured, in us, at 64 sequences
// of up to 8192 keys and 8 key heads, D = 128 unless said:
//   8 rows   two CTAs of 8 warps 70, three (with Q in shared memory) 93; D = 64:
//            50, three CTAs 50; lead 0/1/2/3/5/8: 92/84/79/78/79/81
//   16 rows  the registers of two CTAs would spill; lead 3/4/6/8: 121/117/110/111;
//            D = 64: one CTA 89, two 63, lead 4/6/8: 63/64/65
//   32 rows  (all 255 registers and some spilling: 260 bytes stored, 364 loaded)
//            lead 3/4/6/8: 266/258/259/263, two CTAs of 4 warps 246, but 18 instead
//            of 15 for one sequence of 4096; D = 64: 8 warps 109, twice 4 101
template <int NT, int D>
struct Shape {
  static constexpr int kWarps = NT == 4 && D == 64 ? 4 : 8;
  static constexpr int kCtas = NT == 1 || D == 64 ? 2 : 1;
  static constexpr int kLead = NT == 1 ? 3 : NT == 2 && D == 64 ? 4 : 6;
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transposes an 8 x 8 matrix of 16-bit numbers held as mma fragments.
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int W>
__device__ __forceinline__ void load_words(uint32_t (&x)[W], const uint8_t *p) {
  if constexpr (W == 4)
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "l"(p));
  else if constexpr (W == 2)
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
                 : "=r"(x[0]), "=r"(x[1]) : "l"(p));
  else
    asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(x[0]) : "l"(p));
}

// Units of one key head of a sequence, kLead of them ahead of its keys; a
// sequence without keys still has one more (its rows get their zeros), one
// with more than `rows` rows none (the kernel for many queries takes it).
template <int kUnit, int kLead>
__device__ __forceinline__ int units_of(const Seq &s, int group, int rows) {
  if (s.nq == 0 || static_cast<long long>(s.nq) * group > rows) return 0;
  return kLead + max(1, (s.nk + kUnit - 1) / kUnit);
}

// Units a CTA of a cluster may have at most.  Measured in us, one query a sequence,
// 8 key heads of 128, as a cluster and along the line: 1 x 1023 keys 5.0 and 8.0,
// 1 x 8192 (8 units of 128 a CTA) 9.7 and 11.1, 1 x 16384 14.9 and 13.0; 8 x 4096
// (clusters of 4) 12.3 and 14.0; 16 x 2048 (of 2) 12.0 and 13.0, 16 x 4096 19.0 and
// 16.7; 32 x 1023 (of 1) 11.0 and 13.8.  More clusters than one wave holds lose:
// 64 x 1023 24 to 70 us in clusters of 2 to 8, 20 along the line.
constexpr int kClusterUnits = 8;

// Of the whole CTA; its aligned instructions want every warp together, which the
// loops before it leave row by row.
__device__ __forceinline__ void cluster_barrier() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
               "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Shared memory address `addr` as CTA `rank` of the cluster has it.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, int rank) {
  uint32_t y;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(y) : "r"(addr), "r"(rank));
  return y;
}
__device__ __forceinline__ float4 cluster_load4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float2 cluster_load2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
               : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

// 16 tokens of one page as lane (r, c) holds them.
template <int D>
struct Tile {
  uint32_t k[2][D / 32], v[4][D / 64];
  uint32_t ks[2], vs[4];
};

template <typename T>
__device__ __forceinline__ float2 pair_f32(uint32_t x) {
  if constexpr (sizeof(T) == 2) {
    const T *e = reinterpret_cast<const T *>(&x);
    return make_float2(static_cast<float>(e[0]), static_cast<float>(e[1]));
  }
}

template <int NT, int D>
constexpr int smem_bytes() {
  return (Shape<NT, D>::kWarps * (D + 4 + 2) + D + 4) * NT * 8 * 4;
}

// CL > 0: the CTAs of a cluster, as many, share one sequence and key head and join
// their parts through shared memory; 0: every CTA takes its share of the line of
// all units, and the join is another kernel's.
template <typename T, int D, int NT, int CL>
__global__ void __launch_bounds__(Shape<NT, D>::kWarps * 32, Shape<NT, D>::kCtas)
    fa_kv4_attn_kernel(const Kv4Attn p, float *ws) {
  constexpr int R = NT * 8;              // rows of the tile
  constexpr int kWarps = Shape<NT, D>::kWarps, kThreads = kWarps * 32, kUnit = kWarps * 16;
  constexpr int kLead = Shape<NT, D>::kLead;
  constexpr int KS = D / 16;             // k steps of S^T, m tiles of O^T
  constexpr int LD = D + 4;
  extern __shared__ float smem[];
  __shared__ long long s_sums[kThreads], s_warp[2][kWarps];
  float *s_o = smem;                     // [warp][R][LD]
  float *s_m = smem + kWarps * R * LD;   // [warp][R]
  float *s_l = s_m + kWarps * R;
  float *s_part = s_l + kWarps * R;      // [R][LD], CL: this CTA's part
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = lane >> 2, c = lane & 3;
  griddep_wait();
  griddep_launch_dependents();
  // four columns of a finished row
  auto put = [&](int i, int head, int col, float4 sum, float m, float l) {
    const long long out = static_cast<long long>(i) * p.Hq + head;
    const float inv = p.v_mul / l;
    alignas(8) T e[4] = {
        static_cast<T>(value_of(sum.x, l, inv)), static_cast<T>(value_of(sum.y, l, inv)),
        static_cast<T>(value_of(sum.z, l, inv)), static_cast<T>(value_of(sum.w, l, inv))};
    *reinterpret_cast<uint2 *>(static_cast<T *>(p.o) + out * D + col) =
        *reinterpret_cast<const uint2 *>(e);
    if (col == 0) p.lse[static_cast<long long>(head) * p.total_q + i] = lse_of(m, l);
  };
  const int bs = 1 << p.c.bs_log2;
  int den = gridDim.x, b, h, unit = 0, n_units;
  long long u = 0, u1 = 0;
  Place at = {0, 0, 0};
  Seq sq;
  Share share = {0, 0, 0, 0};
  if constexpr (CL > 0) {
    const int item = blockIdx.x / CL;
    b = item / p.c.Hk;
    h = item - b * p.c.Hk;
    sq = load_seq(p, b);
    n_units = units_of<kUnit, kLead>(sq, p.group, R);
    if (n_units == 0) return;  // the whole cluster
  } else {
    at = find_unit<kWarps>(
        p,
        [&](int b) {
          return static_cast<long long>(units_of<kUnit, kLead>(load_seq(p, b), p.group, R)) * p.c.Hk;
        },
        blockIdx.x, &den, &u, s_sums, s_warp);
    if (static_cast<int>(blockIdx.x) >= den) {
      if (tid == 0) reinterpret_cast<Share *>(ws)[blockIdx.x] = share;
      return;
    }
    u1 = at.total * (blockIdx.x + 1) / den;
    b = at.b;
    sq = load_seq(p, b);
    n_units = units_of<kUnit, kLead>(sq, p.group, R);
    const long long into = u - at.before;
    h = static_cast<int>(into / n_units);
    unit = static_cast<int>(into - static_cast<long long>(h) * n_units);
  }
  do {
    int t_lo, t_hi, last = 0;  // units [t_lo, t_hi) of the n_units - kLead with keys
    if constexpr (CL > 0) {
      const int rank = blockIdx.x % CL;
      t_lo = static_cast<int>(static_cast<long long>(n_units - kLead) * rank / CL);
      t_hi = static_cast<int>(static_cast<long long>(n_units - kLead) * (rank + 1) / CL);
    } else {
      while (n_units == 0) {  // another sequence of this kernel follows, since u < total
        sq = load_seq(p, ++b);
        n_units = units_of<kUnit, kLead>(sq, p.group, R);
        h = 0;
      }
      const int unit_hi = static_cast<int>(min(static_cast<long long>(n_units), unit + (u1 - u)));
      t_lo = max(unit - kLead, 0), t_hi = max(unit_hi - kLead, 0);
      // the CTA with the last of them
      last = cta_of(u - unit + n_units - 1, at.total, den);
      u += unit_hi - unit;
      unit = 0;
      if (t_lo == t_hi) break;  // only the lead fell to this CTA: its share is done
    }
    const int rows = sq.nq * p.group;

    // Q fragments: lane (r, c) holds D / 4 elements of row nt * 8 + r
    uint32_t qf[NT][D / 8];
    float qs[NT][2];
    int lim[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = nt * 8 + r;
      const int i = row / p.group, j = row - i * p.group;
      float x[D / 4], amax = 0.f;
      if (row < rows) {
        const uint4 *src = reinterpret_cast<const uint4 *>(
            static_cast<const T *>(p.q) +
            (static_cast<long long>(sq.r0 + i) * p.Hq + h * p.group + j) * D + c * (D / 4));
#pragma unroll
        for (int n = 0; n < D / 32; ++n) {
          const uint4 w = src[n];
          const uint32_t e[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const float2 f = pair_f32<T>(e[y]);
            x[n * 8 + 2 * y] = f.x;
            x[n * 8 + 2 * y + 1] = f.y;
            amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        }
      } else {
#pragma unroll
        for (int n = 0; n < D / 4; ++n) x[n] = 0.f;
      }
      amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 2));
      // 2^e brings the row's largest element to 1 .. 2 (an exact scaling)
      const int e = min(max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -126), 126);
      const float mul = pow2(-e), back = p.scale_log2 * pow2(e);
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
        qf[nt][n] = pack_f16x2(x[2 * n] * mul, x[2 * n + 1] * mul);
      // this lane's columns of S^T and O^T are rows 2c, 2c + 1
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        qs[nt][y] = __shfl_sync(~0u, back, (2 * c + y) * 4);
        const int qi = (nt * 8 + 2 * c + y) / p.group;
        lim[nt][y] = p.causal && qi < sq.nq ? sq.nk - sq.nq + qi + 1 : sq.nk;
      }
    }
    // keys below this are seen by every row
    const int all_see = p.causal ? sq.nk - sq.nq + 1 : sq.nk;

    float o[NT][KS][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int y = 0; y < 2; ++y) m[nt][y] = -INFINITY, l[nt][y] = 0.f;
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int y = 0; y < 4; ++y) o[nt][s][y] = 0.f;
    }

    // tokens [t_lo, t_hi) units, every kWarps-th tile of 16
    const int end = min(t_hi * kUnit, sq.nk);
    const int *ids = p.table + static_cast<long long>(b) * p.width;
    const uint8_t *kc = p.c.k_codes + r * (D / 2) + c * (D / 8);
    const uint8_t *ks = p.c.k_scales + r * (D / 16) + (D == 128 ? 2 * c : c);
    const uint8_t *vc = p.c.v_codes + 2 * c * (D / 2) + r * (D / 16);
    const uint8_t *vs = p.c.v_scales + 2 * c * (D / 16) + (D == 128 ? r : r / 2);
    auto page = [&](int t) { return t < end ? ids[t >> p.c.bs_log2] : -1; };
    auto load = [&](Tile<D> &x, int t, int id) {
      if (static_cast<unsigned>(id) >= static_cast<unsigned>(p.c.num_blocks)) return;
      const long long row =
          ((static_cast<long long>(id) * p.c.Hk + h) << p.c.bs_log2) + (t & (bs - 1));
      const uint8_t *a = kc + row * (D / 2), *w = vc + row * (D / 2);
      load_words(x.k[0], a);
      load_words(x.k[1], a + 8 * (D / 2));
      load_words(x.v[0], w);
      load_words(x.v[1], w + D / 2);
      load_words(x.v[2], w + 8 * (D / 2));
      load_words(x.v[3], w + 9 * (D / 2));
      const uint8_t *f = ks + row * (D / 16), *y = vs + row * (D / 16);
      if constexpr (D == 128) {
        x.ks[0] = __ldg(reinterpret_cast<const uint16_t *>(f));
        x.ks[1] = __ldg(reinterpret_cast<const uint16_t *>(f + 8 * (D / 16)));
      } else {
        x.ks[0] = __ldg(f);
        x.ks[1] = __ldg(f + 8 * (D / 16));
      }
      x.vs[0] = __ldg(y);
      x.vs[1] = __ldg(y + D / 16);
      x.vs[2] = __ldg(y + 8 * (D / 16));
      x.vs[3] = __ldg(y + 9 * (D / 16));
    };
    auto compute = [&](const Tile<D> &x, int t, int id) {
      if (static_cast<unsigned>(id) >= static_cast<unsigned>(p.c.num_blocks)) return;
      float s[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int y = 0; y < 4; ++y) s[nt][y] = 0.f;
      // scales of tokens r and r + 8, as pairs of one number
      const uint32_t f0 = e4m3x2_f16x2(x.ks[0]), f1 = e4m3x2_f16x2(x.ks[1]);
      const uint32_t a_lo = __byte_perm(f0, 0, 0x1010), a_hi = __byte_perm(f0, 0, 0x3232);
      const uint32_t b_lo = __byte_perm(f1, 0, 0x1010), b_hi = __byte_perm(f1, 0, 0x3232);
#pragma unroll
      for (int st = 0; st < KS; ++st) {
        const bool hi = D == 128 && st >= KS / 2;
        const uint32_t w0 = x.k[0][st / 2], w1 = x.k[1][st / 2];
        const uint32_t fa = hi ? a_hi : a_lo, fb = hi ? b_hi : b_lo;
        uint32_t a[4];
        if (st & 1) {
          a[0] = e2m1x2_f16x2<2>(w0), a[1] = e2m1x2_f16x2<2>(w1);
          a[2] = e2m1x2_f16x2<3>(w0), a[3] = e2m1x2_f16x2<3>(w1);
        } else {
          a[0] = e2m1x2_f16x2<0>(w0), a[1] = e2m1x2_f16x2<0>(w1);
          a[2] = e2m1x2_f16x2<1>(w0), a[3] = e2m1x2_f16x2<1>(w1);
        }
        a[0] = hmul2(a[0], fa), a[1] = hmul2(a[1], fb);
        a[2] = hmul2(a[2], fa), a[3] = hmul2(a[3], fb);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma_f16(s[nt], a[0], a[1], a[2], a[3], qf[nt][2 * st], qf[nt][2 * st + 1]);
      }
      uint32_t pf[NT][2];
      bool grow = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int y = 0; y < 4; ++y) s[nt][y] *= qs[nt][y & 1];
        if (t + 16 > all_see) {
#pragma unroll
          for (int y = 0; y < 4; ++y)
            if (t + r + (y >> 1) * 8 >= lim[nt][y & 1]) s[nt][y] = -INFINITY;
        }
        grow |= fmaxf(s[nt][0], s[nt][2]) > m[nt][0] + (kHeadroom + kGrow);
        grow |= fmaxf(s[nt][1], s[nt][3]) > m[nt][1] + (kHeadroom + kGrow);
      }
      if (__any_sync(~0u, grow)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float f[2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            float v = fmaxf(s[nt][y], s[nt][y + 2]);
            v = fmaxf(v, __shfl_xor_sync(~0u, v, 4));
            v = fmaxf(v, __shfl_xor_sync(~0u, v, 8));
            v = fmaxf(v, __shfl_xor_sync(~0u, v, 16));
            v = fmaxf(v - kHeadroom, m[nt][y]);
            f[y] = v == -INFINITY ? 1.f : ex2_approx(m[nt][y] - v);
            m[nt][y] = v;
            l[nt][y] *= f[y];
          }
#pragma unroll
          for (int st = 0; st < KS; ++st)
#pragma unroll
            for (int y = 0; y < 4; ++y) o[nt][st][y] *= f[y & 1];
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float e[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const float off = m[nt][y & 1] == -INFINITY ? 0.f : m[nt][y & 1];
          e[y] = ex2_approx(s[nt][y] - off);
        }
        l[nt][0] += e[0] + e[2];
        l[nt][1] += e[1] + e[3];
        pf[nt][0] = movmatrix(pack_f16x2(e[0], e[1]));
        pf[nt][1] = movmatrix(pack_f16x2(e[2], e[3]));
      }
      // scales of tokens (2c, 2c + 1) and (2c + 8, 2c + 9); a token behind the
      // sequence has P = 0, and its scale, which may be anything, becomes 0
      uint32_t v0 = x.vs[0] | x.vs[1] << 8, v1 = x.vs[2] | x.vs[3] << 8;
      if (t + 16 > sq.nk) {
        const int left = sq.nk - t - 2 * c;
        v0 &= left > 1 ? 0xFFFFu : left == 1 ? 0xFFu : 0u;
        v1 &= left > 9 ? 0xFFFFu : left == 9 ? 0xFFu : 0u;
      }
      const uint32_t g0 = e4m3x2_f16x2(v0), g1 = e4m3x2_f16x2(v1);
#pragma unroll
      for (int w = 0; w < D / 64; ++w) {
        // byte n: column 2n (even) or 2n + 1 (odd) of the word's 8, of both tokens
        constexpr uint32_t M = 0x0F0F0F0Fu;
        const uint32_t ev0 = (x.v[0][w] & M) | ((x.v[1][w] << 4) & ~M);
        const uint32_t od0 = ((x.v[0][w] >> 4) & M) | (x.v[1][w] & ~M);
        const uint32_t ev1 = (x.v[2][w] & M) | ((x.v[3][w] << 4) & ~M);
        const uint32_t od1 = ((x.v[2][w] >> 4) & M) | (x.v[3][w] & ~M);
        auto step = [&](auto n) {
          constexpr int N = decltype(n)::value;
          const uint32_t a0 = hmul2(e2m1x2_f16x2<N>(ev0), g0), a1 = hmul2(e2m1x2_f16x2<N>(od0), g0);
          const uint32_t a2 = hmul2(e2m1x2_f16x2<N>(ev1), g1), a3 = hmul2(e2m1x2_f16x2<N>(od1), g1);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma_f16(o[nt][w * 4 + N], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
        };
        step(std::integral_constant<int, 0>{});
        step(std::integral_constant<int, 1>{});
        step(std::integral_constant<int, 2>{});
        step(std::integral_constant<int, 3>{});
      }
    };

    {
      int t = (t_lo * kWarps + warp) * 16;
      Tile<D> x0, x1;
      int id0 = page(t), id1 = page(t + kUnit);
      load(x0, t, id0);
      while (t < end) {
        load(x1, t + kUnit, id1);
        const int id2 = page(t + 2 * kUnit);
        compute(x0, t, id0);
        t += kUnit;
        if (t >= end) break;
        load(x0, t + kUnit, id2);
        const int id3 = page(t + 2 * kUnit);
        compute(x1, t, id1);
        t += kUnit;
        id0 = id2;
        id1 = id3;
      }
    }

    // the warps' parts meet in shared memory
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float v = l[nt][y];
        v += __shfl_xor_sync(~0u, v, 4);
        v += __shfl_xor_sync(~0u, v, 8);
        v += __shfl_xor_sync(~0u, v, 16);
        const int row = nt * 8 + 2 * c + y;
        float *dst = s_o + (warp * R + row) * LD + r * (D / 8);
#pragma unroll
        for (int st = 0; st < KS; st += 2)
          *reinterpret_cast<float4 *>(dst + 2 * st) =
              make_float4(o[nt][st][y], o[nt][st][y + 2], o[nt][st + 1][y], o[nt][st + 1][y + 2]);
        if (r == 0) {
          s_m[warp * R + row] = m[nt][y];
          s_l[warp * R + row] = v;
        }
      }
    __syncthreads();
    const bool begins = t_lo == 0, ends = t_hi == n_units - kLead, whole = begins && ends;
    if (begins && !ends) share = Share{sq.r0, h, rows, last};
    for (int x = tid; x < R * (D / 4); x += kThreads) {
      const int row = x / (D / 4), col = (x - row * (D / 4)) * 4;
      if (row >= rows) break;
      float mm = -INFINITY, ll = 0.f, f[kWarps];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_m[w * R + row]);
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        f[w] = mm == -INFINITY ? 0.f : ex2_approx(s_m[w * R + row] - mm);
        ll += f[w] * s_l[w * R + row];
        const float4 v = *reinterpret_cast<const float4 *>(s_o + (w * R + row) * LD + col);
        sum.x += f[w] * v.x, sum.y += f[w] * v.y, sum.z += f[w] * v.z, sum.w += f[w] * v.w;
      }
      if constexpr (CL > 0) {
        *reinterpret_cast<float4 *>(s_part + row * LD + col) = sum;
        if (col == 0) *reinterpret_cast<float2 *>(s_part + row * LD + D) = make_float2(mm, ll);
      } else if (whole) {
        const int i = row / p.group, j = row - i * p.group;
        put(sq.r0 + i, h * p.group + j, col, sum, mm, ll);
      } else {
        float *dst = part_of<D, R>(ws, blockIdx.x, begins);
        *reinterpret_cast<float4 *>(dst + row * D + col) = sum;
        if (col == 0) {
          dst[R * D + 2 * row] = mm;
          dst[R * D + 2 * row + 1] = ll;
        }
      }
    }
    if constexpr (CL == 0) {
      __syncthreads();
      if (++h == p.c.Hk) n_units = 0;
    }
  } while (CL == 0 && u < u1);
  if constexpr (CL > 0) {
    cluster_barrier();
    for (int x = tid; x < R / CL * (D / 4); x += kThreads) {  // row by row to the CTAs
      const int row = blockIdx.x % CL + CL * (x / (D / 4)), col = x % (D / 4) * 4;
      if (row >= sq.nq * p.group) break;
      const uint32_t src = smem_u32(s_part + row * LD);
      float2 ml[CL];
      float4 v[CL], sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int n = 0; n < CL; ++n) {
        const uint32_t from = cluster_addr(src, n);
        ml[n] = cluster_load2(from + D * 4);
        v[n] = cluster_load4(from + col * 4);
      }
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int n = 0; n < CL; ++n) m = fmaxf(m, ml[n].x);
#pragma unroll
      for (int n = 0; n < CL; ++n) {
        const float f = m == -INFINITY ? 0.f : ex2_approx(ml[n].x - m);
        l += f * ml[n].y;
        sum.x += f * v[n].x, sum.y += f * v[n].y, sum.z += f * v[n].z, sum.w += f * v[n].w;
      }
      const int i = row / p.group, j = row - i * p.group;
      put(sq.r0 + i, h * p.group + j, col, sum, m, l);
    }
    cluster_barrier();  // the others may still read this CTA's part
  } else {
    if (tid == 0) reinterpret_cast<Share *>(ws)[blockIdx.x] = share;
  }
}

template <typename T, int D, int NT, int CL>
cudaError_t launch_kernel(const Kv4Attn &p, float *ws, int ctas, cudaStream_t s) {
  static std::atomic<unsigned long long> attr_done{0};
  constexpr int smem = smem_bytes<NT, D>();
  cudaError_t e = smem_attr_once(fa_kv4_attn_kernel<T, D, NT, CL>, smem, &attr_done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(Shape<NT, D>::kWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CL;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CL > 1 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, fa_kv4_attn_kernel<T, D, NT, CL>, p, ws);
  if (e != cudaSuccess || CL > 0 || ctas == 1) return e;
  const long long rows = static_cast<long long>(p.max_q) * p.group;
  cfg.blockDim = dim3(kJoinThreads);
  cfg.gridDim = dim3(static_cast<unsigned>(ctas - 1),
                     static_cast<unsigned>((min(rows, NT * 8LL) + kJoinRows - 1) / kJoinRows));
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, fa_kv4_join_kernel<T, D, NT * 8>, p, ws);
}

template <typename T, int D, int NT>
cudaError_t launch(const Kv4Attn &p, const Kv4Grid &g, float *ws, cudaStream_t s) {
  if constexpr (NT <= 2) {
    if (g.cluster == 8) return launch_kernel<T, D, NT, 8>(p, ws, g.ctas, s);
    if (g.cluster == 4) return launch_kernel<T, D, NT, 4>(p, ws, g.ctas, s);
    if (g.cluster == 2) return launch_kernel<T, D, NT, 2>(p, ws, g.ctas, s);
    if (g.cluster == 1) return launch_kernel<T, D, NT, 1>(p, ws, g.ctas, s);
  }
  return launch_kernel<T, D, NT, 0>(p, ws, g.ctas, s);
}

// The grid for `heads` sequences and key heads with up to max_k keys.
template <int NT, int D>
void shape_grid(long long heads, int max_k, int num_sms, Kv4Grid *g) {
  constexpr int kUnit = Shape<NT, D>::kWarps * 16;
  const long long wave = static_cast<long long>(num_sms) * Shape<NT, D>::kCtas;
  const long long units = max_k < kUnit ? 1 : (static_cast<long long>(max_k) + kUnit - 1) / kUnit;
  if (NT <= 2) {
    // the largest cluster of which one wave holds one for every sequence and key
    // head, if that leaves a CTA at most kClusterUnits units: one launch
    for (int cl = 8; cl > 0; cl /= 2)
      if (heads * cl <= wave && units <= cl * kClusterUnits) {
        g->cluster = cl;
        g->ctas = static_cast<int>(heads * cl);
        return;
      }
  }
  // one resident wave, no more CTAs than there can be units
  const long long ctas = wave < heads * units ? wave : heads * units;
  g->ctas = static_cast<int>(ctas < kKv4MaxCtas ? ctas : kKv4MaxCtas);
}

template <typename T, int D>
cudaError_t launch_rows(const Kv4Attn &p, const Kv4Grid &g, float *ws, cudaStream_t s) {
  if (g.rows == 8) return launch<T, D, 1>(p, g, ws, s);
  if (g.rows == 16) return launch<T, D, 2>(p, g, ws, s);
  return launch<T, D, 4>(p, g, ws, s);
}

}  // namespace

int kv4_tile_rows(int group, int max_q, int d, long long keys) {
  auto fit = [](long long n) { return n <= 8 ? 8 : n <= 16 ? 16 : n <= 32 ? 32 : 0; };
  int rows = fit(static_cast<long long>(group) * max_q);
  if (rows == 0) rows = fit(group);
  // 32 rows of 128 elements fill the registers; where there is work for every
  // tile of the other kernel, that is faster (8 heads, 32 rows: 1 x 131071 keys 99
  // us here, 93 there; 64 x 8192 259 and 212; 16 x 4096 45 and 52; 1 x 1023 14 and 18)
  return rows == 32 && d == 128 && keys >= 1000000 ? 0 : rows;
}

size_t kv4_workspace(int rows, int d) {
  const int ctas = rows == kKv4ManyRows ? kKv4ManyCtas : kKv4MaxCtas;
  return kKv4MaxCtas * sizeof(Share) +
         static_cast<size_t>(2 * ctas) * rows * (d + 2) * sizeof(float);
}

Kv4Grid kv4_grid(int B, int Hk, int group, int d, int max_q, int max_k, int num_sms) {
  const long long heads = static_cast<long long>(B) * Hk;
  if (num_sms < 1) num_sms = 1;
  Kv4Grid g = {kv4_tile_rows(group, max_q, d, heads * max_k), 0, 0, 0};
  if (g.rows == 8)
    d == 64 ? shape_grid<1, 64>(heads, max_k, num_sms, &g)
            : shape_grid<1, 128>(heads, max_k, num_sms, &g);
  else if (g.rows == 16)
    d == 64 ? shape_grid<2, 64>(heads, max_k, num_sms, &g)
            : shape_grid<2, 128>(heads, max_k, num_sms, &g);
  else if (g.rows == 32)
    d == 64 ? shape_grid<4, 64>(heads, max_k, num_sms, &g)
            : shape_grid<4, 128>(heads, max_k, num_sms, &g);
  if (static_cast<long long>(max_q) * group > g.rows) {
    // one CTA on each SM, no more than there can be units (steps of 128 keys)
    const int tokens = kKv4ManyRows / group;
    const long long tiles = (static_cast<long long>(max_q) + tokens - 1) / tokens;
    const double most = static_cast<double>(heads) * tiles *
                        (max_k < 128 ? 1.0 : (max_k + 127.0) / 128.0);
    g.many = num_sms < kKv4ManyCtas ? num_sms : kKv4ManyCtas;
    if (g.many > most) g.many = static_cast<int>(most);
  }
  return g;
}

cudaError_t launch_kv4_attn(const Kv4Attn &p, const Kv4Grid &g, int dtype, float *ws,
                            cudaStream_t s) {
  if (dtype == FA_DTYPE_BF16)
    return p.c.d == 64 ? launch_rows<__nv_bfloat16, 64>(p, g, ws, s)
                       : launch_rows<__nv_bfloat16, 128>(p, g, ws, s);
  return p.c.d == 64 ? launch_rows<__half, 64>(p, g, ws, s)
                     : launch_rows<__half, 128>(p, g, ws, s);
}

}  // namespace fa
