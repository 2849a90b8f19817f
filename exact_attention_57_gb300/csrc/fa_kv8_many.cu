// fa_kv8_many.cu — attention of sequences with many queries over the paged 8-bit
// cache: the kernel of fa_kv_many.cuh for codes of e4m3 with one scale for a block
// of tokens of a key head.  Rows become fp16 by one conversion for two elements; the
// scales go to the softmax, three numbers for 16 keys (BlockScale).
#include "fa_kv8.cuh"
#include "fa_kv_many.cuh"

namespace fa {
namespace {

template <int D_>
struct Many8 {
  static constexpr int D = D_;
  static constexpr bool kBlockScales = true;

  struct Row {
    uint4 c[D / 16];
    float ks, vs;

    __device__ __forceinline__ void load(const uint8_t *codes, const uint8_t *, long long row) {
      const uint4 *src = reinterpret_cast<const uint4 *>(codes + row * D);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) c[i] = __ldg(src + i);
    }
    __device__ __forceinline__ void load_scales(const KvStore &p, long long row) {
      ks = vs = 1.f;  // of a page that is missing: its scores are masked
      if (row < 0) return;
      ks = __ldg(reinterpret_cast<const float *>(p.k_scales) + (row >> p.bs_log2));
      vs = __ldg(reinterpret_cast<const float *>(p.v_scales) + (row >> p.bs_log2));
    }
    __device__ __forceinline__ void store_scales(float *to) const {
      BlockScale s;
      s.set(ks, vs);
      to[0] = s.k;
      to[8] = s.v_log;
      to[16] = s.v_inv;
    }
    // 8 codes make a unit.
    template <typename At>
    __device__ __forceinline__ void expand(bool valid, At at) const {
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const uint32_t w[4] = {valid ? c[i].x : 0u, valid ? c[i].y : 0u, valid ? c[i].z : 0u,
                               valid ? c[i].w : 0u};
#pragma unroll
        for (int y = 0; y < 2; ++y)
          *at(2 * i + y) = make_uint4(e4m3x2_f16x2(w[2 * y]), e4m3x2_f16x2_hi(w[2 * y]),
                                      e4m3x2_f16x2(w[2 * y + 1]), e4m3x2_f16x2_hi(w[2 * y + 1]));
      }
    }
  };
};

}  // namespace

cudaError_t launch_kv8_many(const KvAttn &p, const KvGrid &g, int dtype, float *ws,
                            unsigned *status, unsigned long long wait_limit_ns, int skip_load,
                            cudaStream_t s) {
  const ManyCtl ctl = {status, wait_limit_ns, skip_load, g.rows, R / p.group};
  if (dtype == FA_DTYPE_BF16)
    return p.c.d == 64 ? launch_many<__nv_bfloat16, Many8<64>>(p, ctl, ws, g.many, s)
                       : launch_many<__nv_bfloat16, Many8<128>>(p, ctl, ws, g.many, s);
  return p.c.d == 64 ? launch_many<__half, Many8<64>>(p, ctl, ws, g.many, s)
                     : launch_many<__half, Many8<128>>(p, ctl, ws, g.many, s);
}

}  // namespace fa
