// fa_rope.cu — rotary positions with several axes on queries and keys, and
// the inverse rotation (the gradient: a rotation's transpose).
//
// Pair i of a row's first d_rot elements, (x1, x2), turns by the angle
// t = pos[axis_i] * f_i:  y1 = x1 cos t - x2 sin t,  y2 = x2 cos t + x1 sin t
// (sin t negated for the inverse).  The elements behind d_rot are copied.
//
// The angle is kept in turns as a 64-bit fixed-point fraction: the table holds
// f_i / 2 pi scaled by 2^64, and pos * table[i] modulo 2^64 is the fraction of
// a turn, exact in integers, so a position of 2^31 loses nothing (an fp32
// product would be off by whole radians, and fp64 runs at a small fraction of
// the fp32 rate on this chip).  Its upper 32 bits, as a number in
// [-1, 1) half turns, go to sincospif.
//
// Memory bounds it: 18432 tokens of 32 bf16 heads of 128 elements (302 MB in and
// out) take 50 us, 6.0 TB/s or 89% of the measured copy rate; 64 tokens take 2.5 us
// in a captured graph, a launch, and 5.3 to 6 as a call, the host's.  Rows whose
// half of d_rot is no multiple of 4 go an element at a time: 18432 tokens of 32 heads
// of 72 elements with 36 turned take 104 us in bf16 where all 72 take 34, in fp32 106
// and 53.  A thread issues one head's loads ahead of its stores; four heads' together
// (111 registers, so half the warps) took 75 us, one head ahead 53 to 64, streaming
// cache hints changed nothing.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa.h"
#include "fa_serve.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ float to_f32(T x) {
  return static_cast<float>(x);
}
template <typename T>
__device__ __forceinline__ T from_f32(float x) {
  return static_cast<T>(x);  // round to nearest even
}

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T x[V];
};

// One thread: V pairs of one row (or, behind the rotated part, V elements to
// copy), for `hpt` heads of q and k, so that its sines and cosines serve them
// all.  INTER: pair i is elements (2i, 2i + 1), else (i, i + d_rot / 2).  TAIL:
// there are elements to copy; a warp's threads then load together before they
// part (apart, a partial rotation of fp32 rows took 58 us instead of 45), which
// full rotations do without (50 us instead of 57).  Eight pairs and a tail spill
// at six CTAs an SM (34 us, 31 at five).
template <typename T, int V, bool INTER, bool TAIL>
__global__ void __launch_bounds__(kThreads, V == 8 && TAIL ? 5 : 6)
    fa_rope_kernel(const RopeParams p, int nvec, int hpt) {
  griddep_wait();
  griddep_launch_dependents();
  const int rows_cta = kThreads / nvec;
  const int slot = threadIdx.x / nvec, vec = threadIdx.x - slot * nvec;
  const long long row = static_cast<long long>(blockIdx.x) * rows_cta + slot;
  if (slot >= rows_cta || row >= p.rows) return;
  const int half = p.d_rot / 2, nrot = half / V;
  const long long b = row / p.N, n = row - b * p.N;
  const int h0 = blockIdx.y * hpt, h1 = min(h0 + hpt, p.q.heads + p.k.heads);
  const bool rot = !TAIL || vec < nrot;
  const int e0 = !rot ? p.d_rot + (vec - nrot) * V : INTER ? vec * 2 * V : vec * V;
  const int e1 = INTER ? e0 + V : e0 + half;
  Vec<T, V> x, y;
  auto load = [&](int h) {
    const RopeTensor &t = h < p.q.heads ? p.q : p.k;
    const T *in = static_cast<const T *>(t.in) + b * t.ib +
                  (h < p.q.heads ? h : h - p.q.heads) * t.ih + n * t.in_row;
    x = *reinterpret_cast<const Vec<T, V> *>(in + e0);
    if (rot) y = *reinterpret_cast<const Vec<T, V> *>(in + e1);
  };
  float c[V], s[V];
  if (rot) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const unsigned long long w = p.table[vec * V + j];
      // a table entry's two low bits name the axis; out of range reads the last
      const int a = min(static_cast<int>(w & 3), p.axes - 1);
      const long long pos = p.positions[a * p.rows + row];
      const unsigned long long turn = static_cast<unsigned long long>(pos) * (w & ~3ull);
      const int frac = static_cast<int>(static_cast<unsigned>((turn + (1ull << 31)) >> 32));
      sincospif(static_cast<float>(frac) * 4.656612873077393e-10f /* 2^-31 */, &s[j], &c[j]);
      if (p.inverse) s[j] = -s[j];
    }
  }
  for (int h = h0; h < h1; ++h) {
    load(h);
    const RopeTensor &t = h < p.q.heads ? p.q : p.k;
    T *out = static_cast<T *>(t.out) + b * t.ob + (h < p.q.heads ? h : h - p.q.heads) * t.oh +
             n * t.out_row;
    if (rot) {
      Vec<T, V> u, w;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        // pair j: with INTER the pairs lie side by side in the 2V elements
        const float a = INTER ? to_f32(2 * j < V ? x.x[(2 * j) % V] : y.x[(2 * j) % V])
                              : to_f32(x.x[j]);
        const float q = INTER ? to_f32(2 * j + 1 < V ? x.x[(2 * j + 1) % V] : y.x[(2 * j + 1) % V])
                              : to_f32(y.x[j]);
        const T r1 = from_f32<T>(a * c[j] - q * s[j]), r2 = from_f32<T>(q * c[j] + a * s[j]);
        if constexpr (INTER) {
          (2 * j < V ? u : w).x[(2 * j) % V] = r1;
          (2 * j + 1 < V ? u : w).x[(2 * j + 1) % V] = r2;
        } else {
          u.x[j] = r1;
          w.x[j] = r2;
        }
      }
      *reinterpret_cast<Vec<T, V> *>(out + e0) = u;
      *reinterpret_cast<Vec<T, V> *>(out + e1) = w;
    } else {
      *reinterpret_cast<Vec<T, V> *>(out + e0) = x;
    }
  }
}

bool aligned(const RopeTensor &t, long long bytes, long long es) {
  if (t.heads == 0) return true;
  const uintptr_t any = reinterpret_cast<uintptr_t>(t.in) | reinterpret_cast<uintptr_t>(t.out);
  const long long strides = t.ib | t.ih | t.in_row | t.ob | t.oh | t.out_row;
  return any % bytes == 0 && (strides * es) % bytes == 0;
}

template <typename T, int V>
cudaError_t launch_vec(const RopeParams &p, int num_sms, cudaStream_t s) {
  const int nvec = p.d_rot / 2 / V + (p.d - p.d_rot) / V;
  const int rows_cta = kThreads / nvec;
  const long long gx = (p.rows + rows_cta - 1) / rows_cta;
  if (gx > 2147483647LL) return cudaErrorInvalidConfiguration;
  const int heads = p.q.heads + p.k.heads;
  // Heads per thread: as many as leave about eight CTAs an SM, up to eight (18432
  // tokens of 32 heads: 2 ran in 64.9 us, 4 in 53.3, 8 in 52.3, 16 in 54.5; their
  // sines and cosines cost less than what a short last wave does), in even shares.
  int hpt = static_cast<int>(gx * heads / (8LL * (num_sms > 0 ? num_sms : 1)));
  hpt = hpt < 1 ? 1 : (hpt > 8 ? 8 : hpt);
  const int shares = (heads + hpt - 1) / hpt;
  hpt = (heads + shares - 1) / shares;
  while ((heads + hpt - 1) / hpt > 65535) ++hpt;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(gx), static_cast<unsigned>((heads + hpt - 1) / hpt));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (p.d_rot < p.d)
    return p.interleaved ? cudaLaunchKernelEx(&cfg, fa_rope_kernel<T, V, true, true>, p, nvec, hpt)
                         : cudaLaunchKernelEx(&cfg, fa_rope_kernel<T, V, false, true>, p, nvec, hpt);
  return p.interleaved ? cudaLaunchKernelEx(&cfg, fa_rope_kernel<T, V, true, false>, p, nvec, hpt)
                       : cudaLaunchKernelEx(&cfg, fa_rope_kernel<T, V, false, false>, p, nvec, hpt);
}

template <typename T>
cudaError_t launch_type(const RopeParams &p, int num_sms, cudaStream_t s) {
  constexpr int es = sizeof(T), W = 16 / es;
  auto fits = [&](int v) {
    return p.d_rot / 2 % v == 0 && (p.d - p.d_rot) % v == 0 && aligned(p.q, v * es, es) &&
           aligned(p.k, v * es, es);
  };
  // 16-byte accesses where strides and addresses allow them, 8-byte ones where
  // only those (18432 bf16 tokens: 50 us, 56 with 8 bytes, 131 an element at a
  // time; 6001 fp32 tokens of 40 heads: 42 and 61 us)
  if (fits(W)) return launch_vec<T, W>(p, num_sms, s);
  if (es == 2 && fits(4)) return launch_vec<T, 4>(p, num_sms, s);
  return launch_vec<T, 1>(p, num_sms, s);
}

}  // namespace

cudaError_t launch_rope(const RopeParams &p, int dtype, int num_sms, cudaStream_t s) {
  if (dtype == FA_DTYPE_BF16) return launch_type<__nv_bfloat16>(p, num_sms, s);
  if (dtype == FA_DTYPE_F16) return launch_type<__half>(p, num_sms, s);
  return launch_type<float>(p, num_sms, s);
}

}  // namespace fa
