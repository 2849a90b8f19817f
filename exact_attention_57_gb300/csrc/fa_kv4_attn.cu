// fa_kv4_attn.cu — attention of a few queries a sequence over the paged 4-bit
// cache: the kernel of fa_kv_attn.cuh for codes of e2m1 with an e4m3 scale for 16
// elements.
//
// Codes become fp16 pairs by cvt (V: the nibbles of two tokens are merged into
// bytes first, since a register holds two tokens of one column), times the
// scale, exactly: a value has six significant bits.
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
#include "fa_kv_attn.cuh"

namespace fa {
namespace {

template <int D_>
struct Cache4 {
  static constexpr int D = D_, KS = D / 16;

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
  template <int NT, int>
  struct Shape {
    static constexpr int kWarps = NT == 4 && D == 64 ? 4 : 8;
    static constexpr int kCtas = NT == 1 || D == 64 ? 2 : 1;
    static constexpr int kLead = NT == 1 ? 3 : NT == 2 && D == 64 ? 4 : 6;
    static constexpr int kMost = kClusterUnits;
  };

  struct Tile {
    uint32_t k[2][D / 32], v[4][D / 64];
    uint32_t ks[2], vs[4];
  };

  struct Lane {
    const uint8_t *kc, *ks, *vc, *vs;
    int h;
    __device__ __forceinline__ Lane(const KvStore &p, int h, int r, int c)
        : kc(p.k_codes + r * (D / 2) + c * (D / 8)),
          ks(p.k_scales + r * (D / 16) + (D == 128 ? 2 * c : c)),
          vc(p.v_codes + 2 * c * (D / 2) + r * (D / 16)),
          vs(p.v_scales + 2 * c * (D / 16) + (D == 128 ? r : r / 2)), h(h) {}
    // Tokens off .. off + 15 of block id.
    __device__ __forceinline__ void load(Tile &x, const KvStore &p, int id, int off) const {
      const long long row = ((static_cast<long long>(id) * p.Hk + h) << p.bs_log2) + off;
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
    }
  };

  struct Scale {
    __device__ __forceinline__ float score(float s, float q) const { return s * q; }
    __device__ __forceinline__ float add(float l, float w) const { return l + w; }
  };
  static __device__ __forceinline__ Scale scale_of(const Tile &) { return {}; }

  template <int NT>
  static __device__ __forceinline__ void scores(const Tile &x, const uint32_t (&qf)[NT][D / 8],
                                                float (&s)[NT][4]) {
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
  }

  // `left`: tokens of the sequence from the tile's first on.
  template <int NT>
  static __device__ __forceinline__ void values(const Tile &x, int left, int c,
                                                const uint32_t (&pf)[NT][2], float (&o)[NT][KS][4]) {
    // scales of tokens (2c, 2c + 1) and (2c + 8, 2c + 9); a token behind the
    // sequence has P = 0, and its scale, which may be anything, becomes 0
    uint32_t v0 = x.vs[0] | x.vs[1] << 8, v1 = x.vs[2] | x.vs[3] << 8;
    if (left < 16) {
      left -= 2 * c;
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
  }
};

}  // namespace

int kv4_tile_rows(int group, int max_q, int d, long long keys) {
  const int rows = fit_rows(group, max_q);
  // 32 rows of 128 elements fill the registers; where there is work for every
  // tile of the other kernel, that is faster (8 heads, 32 rows: 1 x 131071 keys 99
  // us here, 93 there; 64 x 8192 259 and 212; 16 x 4096 45 and 52; 1 x 1023 14 and 18)
  return rows == 32 && d == 128 && keys >= 1000000 ? 0 : rows;
}

size_t kv_workspace(int rows, int d) {
  const int ctas = rows == kKvManyRows ? kKvManyCtas : kKvMaxCtas;
  return kKvMaxCtas * sizeof(Share) +
         static_cast<size_t>(2 * ctas) * rows * (d + 2) * sizeof(float);
}

KvGrid kv4_grid(int B, int Hk, int group, int d, int max_q, int max_k, int num_sms) {
  const long long heads = static_cast<long long>(B) * Hk;
  if (num_sms < 1) num_sms = 1;
  KvGrid g = {kv4_tile_rows(group, max_q, d, heads * max_k), 0, 0, 0};
  if (d == 64)
    rows_grid<Cache4<64>>(heads, max_k, num_sms, &g);
  else
    rows_grid<Cache4<128>>(heads, max_k, num_sms, &g);
  many_grid(heads, group, max_q, max_k, num_sms, &g);
  return g;
}

cudaError_t launch_kv4_attn(const KvAttn &p, const KvGrid &g, int dtype, float *ws,
                            cudaStream_t s) {
  if (dtype == FA_DTYPE_BF16)
    return p.c.d == 64 ? launch_rows<__nv_bfloat16, Cache4<64>>(p, g, ws, s)
                       : launch_rows<__nv_bfloat16, Cache4<128>>(p, g, ws, s);
  return p.c.d == 64 ? launch_rows<__half, Cache4<64>>(p, g, ws, s)
                     : launch_rows<__half, Cache4<128>>(p, g, ws, s);
}

}  // namespace fa
