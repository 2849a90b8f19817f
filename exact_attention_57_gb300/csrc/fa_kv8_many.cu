// fa_kv8_many.cu — attention of sequences with many queries over the paged 8-bit
// cache: the kernel of fa_kv_many.cuh for codes of e4m3 with one scale for a block
// of tokens of a key head.  Rows become fp16 by one conversion for two elements; the
// scales go to the softmax, three numbers for 16 keys (BlockScale).
//
// The products of a 128 x 128 step need about 1000 of the 2660 cycles that it takes, the
// unit for exponentials is in use for 550 of them (20.5% of 995,000 over 374 steps a CTA),
// expanding K and V takes 16 loads and 32 stores of 16 bytes and 128 conversions a lane of
// two warps a scheduler; a load of a step's codes is issued a step ahead, into the register
// that its predecessor left.
//
// Two prompts' chunks of 2048 queries (32 query heads on 8 key heads of 128, causal, up
// to 8192 keys) take 540 us, 875 TFLOP/s; 1024 queries on 65536 keys 1130 us, 965
// TFLOP/s; the first at d = 64 439 us.  Of the 540 this kernel is 508, joining its parts 20,
// the launch for sequences of few rows, of which there are none, the most of the rest.
// Softmax and expanding bound it together: of 541
// with queries of zeros, 509 were left without any loads, 528 without exponentials, and
// of 448 at d = 64 386 without scales; issue slots are 53% busy, the tensor pipe 38%, and
// 36 bytes a thread are spilled at either head dim (72 loaded).  Against 546 then:
// scales applied by the expanding warps took 630 us, two steps of codes in registers 1650
// (they spill), codes of K as e4m3 operands with Q as a sum of two or three e4m3 numbers
// and codes of V by way of shared memory 670 (0.1 us less a step and 24 us more a tile).
#include "fa_kv8.cuh"
#include "fa_kv_many.cuh"

namespace fa {
namespace {

// 16 bytes that this SM reads once (without a place in L1: 535 instead of 541 us for the
// two chunks above, with queries of zeros).
__device__ __forceinline__ uint4 load_once(const uint8_t *p) {
  uint4 x;
  asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
      : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
      : "l"(p));
  return x;
}

template <int D_>
struct Many8 {
  static constexpr int D = D_;
  static constexpr bool kBlockScales = true, kStreams = true;

  // Lane l takes 16 codes of every kRows-th token, from the one l / kLanes on, so that
  // a load of the warp covers whole rows.
  static constexpr int kLanes = D / 16, kRows = 32 / kLanes, kAt = kLanes;
  struct Row {
    uint4 c[kAt];
    float ks, vs;

    // The codes of one step: tokens 0 .. 15 and 16 .. 31 lie in one block each.
    struct From {
      const uint8_t *half[2];
      unsigned good;  // tokens that there are
      __device__ __forceinline__ From(const uint8_t *codes, long long row)
          : good(__ballot_sync(~0u, row >= 0) >> ((threadIdx.x & 31) / kLanes)) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int n = 0; n < 2; ++n)
          half[n] = codes + (__shfl_sync(~0u, row, 16 * n) + lane / kLanes) * D + lane % kLanes * 16;
      }
      __device__ __forceinline__ uint4 piece(int i) const {
        constexpr int kHalf = kAt / 2;
        return good >> (i * kRows) & 1
                   ? load_once(half[i / kHalf] + i % kHalf * kRows * D)
                   : make_uint4(0, 0, 0, 0);
      }
    };
    __device__ __forceinline__ void begin(const uint8_t *codes, long long row) {
      const From from(codes, row);
#pragma unroll
      for (int i = 0; i < kAt; ++i) c[i] = from.piece(i);
    }
    // 8 codes make a unit.  The lanes of a row's second half store their units in the
    // other order, so that eight lanes at a time meet every bank once.
    __device__ __forceinline__ void stream(const uint8_t *codes, long long next, uint8_t *tile,
                                           int chunk) {
      const From from(codes, next);
      const int lane = threadIdx.x & 31, u = 2 * (lane % kLanes);
      const bool swap = u >= 8;
      uint8_t *to = tile + (lane / kLanes) * 128 + (u >> 3) * chunk;
#pragma unroll
      for (int i = 0; i < kAt; ++i) {
        const uint32_t w[4] = {swap ? c[i].z : c[i].x, swap ? c[i].w : c[i].y,
                               swap ? c[i].x : c[i].z, swap ? c[i].y : c[i].w};
        c[i] = from.piece(i);
        const int low = (i * kRows + lane / kLanes) & 7;
#pragma unroll
        for (int n = 0; n < 2; ++n)
          *reinterpret_cast<uint4 *>(to + i * kRows * 128 + ((((u + (n != swap)) & 7) ^ low) << 4)) =
              make_uint4(e4m3x2_f16x2(w[2 * n]), e4m3x2_f16x2_hi(w[2 * n]),
                         e4m3x2_f16x2(w[2 * n + 1]), e4m3x2_f16x2_hi(w[2 * n + 1]));
      }
    }
    __device__ __forceinline__ void load_scales(const KvStore &p, long long row) {
      ks = vs = 1.f;  // of a page that is missing: its scores are masked
      if (row < 0) return;
      ks = __ldg(reinterpret_cast<const float *>(p.k_scales) + (row >> p.bs_log2));
      vs = __ldg(reinterpret_cast<const float *>(p.v_scales) + (row >> p.bs_log2));
    }
    __device__ __forceinline__ BlockScale scales() const {
      BlockScale s;
      s.set(ks, vs);
      return s;
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
