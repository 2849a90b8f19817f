// fa_kv4_many.cu — attention of sequences with many queries over the paged 4-bit
// cache: the kernel of fa_kv_many.cuh for codes of e2m1 with an e4m3 scale for 16
// elements.
//
// The products of a 128 x 128 step need about 1000 cycles of the tensor pipe
// and the softmax 850 of its warps; expanding the step's K and V costs 512
// conversions, 512 multiplications and 128 16-byte stores a warp, which the
// eight warps of their own hide beside them.
//
// Two prompts' chunks of 2048 queries (32 query heads on 8 key heads of 128,
// causal) take 428 us, 1100 TFLOP/s or 56% of the measured bf16 rate; 1024 queries
// on 65536 keys 866 us, 1260 TFLOP/s.  Without expanding the codes the first took
// 400 (of 451 then): what bounds it is the softmax warps and the tensor pipe (46%
// busy) waiting for each other, and every query tile of a sequence and key head
// expands the same codes.  Against 451: a tile of 256 rows as two halves that take
// turns took 641 us (64 registers fewer a softmax thread), masks applied in registers
// 475, queries brought by the expanding warps 612, K and V expanded by the same four
// warps (with those queries) 695.
#include "fa_kv_many.cuh"

namespace fa {
namespace {

template <int D_>
struct Many4 {
  static constexpr int D = D_;
  static constexpr bool kBlockScales = false, kStreams = false;

  struct Row {
    uint4 c[D / 32];
    uint2 f;

    __device__ __forceinline__ void load(const uint8_t *codes, const uint8_t *scales, long long row) {
      const uint4 *src = reinterpret_cast<const uint4 *>(codes + row * (D / 2));
#pragma unroll
      for (int i = 0; i < D / 32; ++i) c[i] = __ldg(src + i);
      if constexpr (D == 128)
        f = __ldg(reinterpret_cast<const uint2 *>(scales + row * (D / 16)));
      else
        f.x = __ldg(reinterpret_cast<const uint32_t *>(scales + row * (D / 16)));
    }
    // 32 code bits make a unit, two units share a scale.
    template <typename At>
    __device__ __forceinline__ void expand(bool valid, At at) const {
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t pair = (i < 2 ? f.x : f.y) >> ((i & 1) * 16);
        const uint32_t two = valid ? e4m3x2_f16x2(pair) : 0u;  // 0 * code = 0
        const uint32_t sc[2] = {__byte_perm(two, 0, 0x1010), __byte_perm(two, 0, 0x3232)};
        const uint32_t wd[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const uint32_t g = sc[y / 2];
          uint4 v;
          v.x = hmul2(e2m1x2_f16x2<0>(wd[y]), g);
          v.y = hmul2(e2m1x2_f16x2<1>(wd[y]), g);
          v.z = hmul2(e2m1x2_f16x2<2>(wd[y]), g);
          v.w = hmul2(e2m1x2_f16x2<3>(wd[y]), g);
          *at(4 * i + y) = v;
        }
      }
    }
  };
};

}  // namespace

cudaError_t launch_kv4_many(const KvAttn &p, const KvGrid &g, int dtype, float *ws,
                            unsigned *status, unsigned long long wait_limit_ns, int skip_load,
                            cudaStream_t s) {
  const ManyCtl ctl = {status, wait_limit_ns, skip_load, g.rows, R / p.group};
  if (dtype == FA_DTYPE_BF16)
    return p.c.d == 64 ? launch_many<__nv_bfloat16, Many4<64>>(p, ctl, ws, g.many, s)
                       : launch_many<__nv_bfloat16, Many4<128>>(p, ctl, ws, g.many, s);
  return p.c.d == 64 ? launch_many<__half, Many4<64>>(p, ctl, ws, g.many, s)
                     : launch_many<__half, Many4<128>>(p, ctl, ws, g.many, s);
}

}  // namespace fa
