// fa_kv8_attn.cu — attention of a few queries a sequence over the paged 8-bit
// cache: the kernel of fa_kv_attn.cuh for codes of e4m3 with one scale for a block
// of tokens of a key head.
//
// Codes become fp16 pairs by cvt, exactly (V: the bytes of two tokens are paired
// first, since a register holds two tokens of one column); the block's scales enter
// the softmax instead (BlockScale), one multiplication and addition a score.
//
// 64 sequences of up to 8192 keys (32 query heads on 8 key heads of 128) take 97 us: 6.0
// TB/s, 89% of the copy rate, so reading the cache bounds it.  One sequence of 1023 keys
// takes 4.3 in a captured graph, a launch and its dependent loads; 16 sequences of up to
// 3001 keys and 4 queries (16 heads of 64) 17.3 of 8.5 that their bytes need: 256 short
// pieces, most of them cut and joined by the second kernel.
#include "fa_kv8.cuh"
#include "fa_kv_attn.cuh"

namespace fa {
namespace {

template <int D_>
struct Cache8 {
  static constexpr int D = D_, KS = D / 16;

  // Warps of a CTA, resident CTAs, and the units that stand for a sequence's cost
  // beside its keys, by rows (8 NT) and head dim; clusters of more than one CTA take 8
  // warps (one sequence of 1023 keys 4.3 us, 4.7 with six).  Measured along the line, in
  // us, at 64 sequences of up to 8192 keys and 8 key heads, D = 128 unless said:
  //   8 rows   CTAs x warps: 1 x 8 113, 1 x 12 100, 1 x 16 106, 2 x 5 102, 2 x 6 97,
  //            2 x 7 106 and 2 x 8 103 (registers spill); lead 2/3/4: 99/97/97;
  //            D = 64: 2 x 8 57, 2 x 10 53, 2 x 12 54 (registers spill)
  //   16 rows  (4 key heads) 1 x 8 67, 1 x 10 91 (registers spill)
  //   32 rows  D = 64 alone, 1 x 8
  // Units of a CTA of a cluster: for CTAs that take a sequence and key head alone (CL = 1)
  // 16 instead of 8, cluster and line in us: 37 x 1023 keys, 8 key heads of 128 11.7 and
  // 14.4, 37 x 1536 16.6 and 17.9, of 64 37 x 2048 13.3 and 15.8, 20 x 1500 9.3 and 10.5 (20
  // x 2500, half a wave, 14.2 and 12.4); 16 rows 18 x 2048 15.5 and 18.6; with 24, 32 x
  // 2048 21.8 and 21.0.  With 16 for wider clusters: 1 x 16384 14.1 and 12.5, 4 x 8192
  // 16.2 and 15.5.
  template <int NT, int CL>
  struct Shape {
    static constexpr bool kLine = NT == 1 && CL < 2;
    static constexpr int kWarps = !kLine ? 8 : D == 128 ? 6 : 10;
    static constexpr int kCtas = kLine || (D == 64 && NT <= 2) ? 2 : 1;
    static constexpr int kLead = NT == 1 ? 3 : NT == 2 && D == 64 ? 4 : 6;
    static constexpr int kMost = CL == 1 ? 16 : kClusterUnits;
  };

  struct Tile {
    uint32_t k[2][D / 16], v[4][D / 32];
    float ks, vs;
  };

  struct Lane {
    const uint8_t *kc, *vc;
    int h;
    __device__ __forceinline__ Lane(const KvStore &p, int h, int r, int c)
        : kc(p.k_codes + r * D + c * (D / 4)), vc(p.v_codes + 2 * c * D + r * (D / 8)), h(h) {}
    // Tokens off .. off + 15 of block id.
    __device__ __forceinline__ void load(Tile &x, const KvStore &p, int id, int off) const {
      const long long block = static_cast<long long>(id) * p.Hk + h;
      const long long row = (block << p.bs_log2) + off;
      const uint8_t *a = kc + row * D, *w = vc + row * D;
      load_words(x.k[0], a);
      load_words(x.k[1], a + 8 * D);
      load_words(x.v[0], w);
      load_words(x.v[1], w + D);
      load_words(x.v[2], w + 8 * D);
      load_words(x.v[3], w + 9 * D);
      x.ks = __ldg(reinterpret_cast<const float *>(p.k_scales) + block);
      x.vs = __ldg(reinterpret_cast<const float *>(p.v_scales) + block);
    }
  };

  struct Scale : BlockScale {
    __device__ __forceinline__ float score(float s, float q) const { return fmaf(s, q * k, v_log); }
    __device__ __forceinline__ float add(float l, float w) const { return fmaf(w, v_inv, l); }
  };
  static __device__ __forceinline__ Scale scale_of(const Tile &x) {
    Scale s;
    s.set(x.ks, x.vs);
    return s;
  }

  template <int NT>
  static __device__ __forceinline__ void scores(const Tile &x, const uint32_t (&qf)[NT][D / 8],
                                                float (&s)[NT][4]) {
#pragma unroll
    for (int st = 0; st < KS; ++st) {
      const uint32_t w0 = x.k[0][st], w1 = x.k[1][st];
      const uint32_t a0 = e4m3x2_f16x2(w0), a1 = e4m3x2_f16x2(w1);
      const uint32_t a2 = e4m3x2_f16x2_hi(w0), a3 = e4m3x2_f16x2_hi(w1);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        mma_f16(s[nt], a0, a1, a2, a3, qf[nt][2 * st], qf[nt][2 * st + 1]);
    }
  }

  // `left`: tokens of the sequence from the tile's first on.
  template <int NT>
  static __device__ __forceinline__ void values(const Tile &x, int left, int c,
                                                const uint32_t (&pf)[NT][2], float (&o)[NT][KS][4]) {
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
      uint32_t v[4] = {x.v[0][w], x.v[1][w], x.v[2][w], x.v[3][w]};
      if (left < 16) {  // a token behind the sequence has P = 0, and codes that may be anything
#pragma unroll
        for (int n = 0; n < 4; ++n)
          if (2 * c + (n & 1) + 4 * (n & 2) >= left) v[n] = 0;
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {  // columns 4w + 2n and one on, of tokens (0, 1) and (2, 3)
        const uint32_t e = __byte_perm(v[0], v[1], n ? 0x7362 : 0x5140);
        const uint32_t f = __byte_perm(v[2], v[3], n ? 0x7362 : 0x5140);
        const uint32_t a0 = e4m3x2_f16x2(e), a1 = e4m3x2_f16x2_hi(e);
        const uint32_t a2 = e4m3x2_f16x2(f), a3 = e4m3x2_f16x2_hi(f);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma_f16(o[nt][2 * w + n], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
      }
    }
  }
};

}  // namespace

int kv8_tile_rows(int group, int max_q, int d) {
  const int rows = fit_rows(group, max_q);
  // (two tiles of codes beside 32 rows' sums would not fit the registers)
  return rows == 32 && d == 128 ? 0 : rows;
}

KvGrid kv8_grid(int B, int Hk, int group, int d, int max_q, int max_k, int num_sms) {
  const long long heads = static_cast<long long>(B) * Hk;
  if (num_sms < 1) num_sms = 1;
  KvGrid g = {kv8_tile_rows(group, max_q, d), 0, 0, 0};
  if (d == 64)
    rows_grid<Cache8<64>>(heads, max_k, num_sms, &g);
  else
    rows_grid<Cache8<128>>(heads, max_k, num_sms, &g);
  many_grid(heads, group, max_q, max_k, num_sms, &g);
  return g;
}

template <typename T>
cudaError_t launch_type(const KvAttn &p, const KvGrid &g, float *ws, cudaStream_t s) {
  if (p.c.d == 64) return launch_rows<T, Cache8<64>>(p, g, ws, s);
  return g.rows == 8 ? launch<T, Cache8<128>, 1>(p, g, ws, s)
                     : launch<T, Cache8<128>, 2>(p, g, ws, s);
}

cudaError_t launch_kv8_attn(const KvAttn &p, const KvGrid &g, int dtype, float *ws,
                            cudaStream_t s) {
  return dtype == FA_DTYPE_BF16 ? launch_type<__nv_bfloat16>(p, g, ws, s)
                                : launch_type<__half>(p, g, ws, s);
}

}  // namespace fa
