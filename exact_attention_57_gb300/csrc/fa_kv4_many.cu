// fa_kv4_many.cu — attention of sequences with many queries over the paged
// 4-bit cache (those that fa_kv4_attn.cu leaves out).
//
// Query token i of sequence b (n_q queries, n_k cached tokens, its own among
// them) sees key j iff j < n_k and, when causal, j <= n_k - n_q + i; query
// head h reads key head h / group.  One warp per query row: each lane scores
// one of 32 keys from its dequantised row, the warp keeps the running maximum
// and sum, then every lane adds p_j * v_j for its d / 32 columns.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa.h"
#include "fa_kv4.cuh"
#include "fa_serve.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;

template <typename T, int D>
__global__ void __launch_bounds__(32 * kWarps)
    fa_kv4_many_kernel(const Kv4Attn p, int tile_rows) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ float sq[kWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.z, h = blockIdx.y;
  int r0 = b, nq = 1;
  if (p.cu_q) {
    r0 = min(max(p.cu_q[b], 0), p.total_q);
    nq = min(min(max(p.cu_q[b + 1], 0), p.total_q) - r0, p.max_q);
  }
  const int i = blockIdx.x * kWarps + warp;
  if (i >= nq || static_cast<long long>(nq) * p.group <= tile_rows) return;
  const int bs = 1 << p.c.bs_log2;
  const int nk = static_cast<int>(min(static_cast<long long>(min(max(p.lens[b], 0), p.max_k)),
                                      static_cast<long long>(p.width) << p.c.bs_log2));
  const int last = p.causal ? min(nk, nk - nq + i + 1) : nk;  // keys [0, last)
  const long long row = static_cast<long long>(r0 + i) * p.Hq + h;
  const T *q = static_cast<const T *>(p.q) + row * D;
  for (int x = lane; x < D; x += 32) sq[warp][x] = static_cast<float>(q[x]) * p.scale_log2;
  __syncwarp();
  const int hk = h / p.group;
  float m = -INFINITY, l = 0.f, acc[D / 32] = {};
  for (int j0 = 0; j0 < last; j0 += 32) {
    const int j = j0 + lane;
    const int id = j < last ? p.table[static_cast<long long>(b) * p.width + (j >> p.c.bs_log2)] : -1;
    const bool ok = static_cast<unsigned>(id) < static_cast<unsigned>(p.c.num_blocks);
    const long long at =
        ok ? ((static_cast<long long>(id) * p.c.Hk + hk) << p.c.bs_log2) + (j & (bs - 1)) : 0;
    float sc = -INFINITY;
    if (ok) {
      sc = 0.f;
      for (int g = 0; g < D / 16; ++g) {
        const uint2 w = reinterpret_cast<const uint2 *>(p.c.k_codes)[at * (D / 16) + g];
        const float s = f16x2_f32(e4m3x2_f16x2(p.c.k_scales[at * (D / 16) + g])).x;
        const uint32_t pr[8] = {e2m1x2_f16x2<0>(w.x), e2m1x2_f16x2<1>(w.x), e2m1x2_f16x2<2>(w.x),
                                e2m1x2_f16x2<3>(w.x), e2m1x2_f16x2<0>(w.y), e2m1x2_f16x2<1>(w.y),
                                e2m1x2_f16x2<2>(w.y), e2m1x2_f16x2<3>(w.y)};
        float dot = 0.f;
        for (int n = 0; n < 8; ++n) {
          const float2 f = f16x2_f32(pr[n]);
          dot += f.x * sq[warp][g * 16 + 2 * n] + f.y * sq[warp][g * 16 + 2 * n + 1];
        }
        sc += dot * s;
      }
    }
    float mt = sc;
    for (int o = 16; o; o /= 2) mt = fmaxf(mt, __shfl_xor_sync(~0u, mt, o));
    if (mt == -INFINITY) continue;
    const float mn = fmaxf(m, mt), f = exp2f(m - mn), pj = exp2f(sc - mn);
    m = mn;
    l = l * f + pj;
    for (float &a : acc) a *= f;
    for (int t = 0; t < 32; ++t) {
      const float w = __shfl_sync(~0u, pj, t);
      const long long vt = __shfl_sync(~0u, at, t);
      if (w == 0.f) continue;
#pragma unroll
      for (int n = 0; n < D / 32; ++n) {
        const int x = lane + 32 * n;
        const uint32_t byte = p.c.v_codes[vt * (D / 2) + x / 2];
        const float2 f2 = f16x2_f32(e2m1x2_f16x2<0>(byte));
        const float s = f16x2_f32(e4m3x2_f16x2(p.c.v_scales[vt * (D / 16) + x / 16])).x;
        acc[n] += w * s * ((x & 1) ? f2.y : f2.x);
      }
    }
  }
  for (int o = 16; o; o /= 2) l += __shfl_xor_sync(~0u, l, o);
  T *out = static_cast<T *>(p.o) + row * D;
  const float inv = l > 0.f ? p.v_mul / l : 0.f;
  for (int n = 0; n < D / 32; ++n) out[lane + 32 * n] = static_cast<T>(acc[n] * inv);
  if (lane == 0)
    p.lse[static_cast<long long>(h) * p.total_q + r0 + i] =
        l > 0.f ? m * 0.6931471805599453f + logf(l) : -INFINITY;
}

template <typename T, int D>
cudaError_t launch(const Kv4Attn &p, int tile_rows, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.max_q + kWarps - 1) / kWarps, p.Hq, p.B);
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fa_kv4_many_kernel<T, D>, p, tile_rows);
}

}  // namespace

cudaError_t launch_kv4_many(const Kv4Attn &p, int tile_rows, int dtype, cudaStream_t s) {
  if (dtype == FA_DTYPE_BF16)
    return p.c.d == 64 ? launch<__nv_bfloat16, 64>(p, tile_rows, s)
                       : launch<__nv_bfloat16, 128>(p, tile_rows, s);
  return p.c.d == 64 ? launch<__half, 64>(p, tile_rows, s) : launch<__half, 128>(p, tile_rows, s);
}

}  // namespace fa
