// fa_kv8_many.cu — attention of sequences with many queries over the paged 8-bit
// cache: the kernel of fa_kv_many.cuh for codes of e4m3 with one scale for a block
// of tokens of a key head.
#include <type_traits>

#include "fa_kv_many.cuh"

namespace fa {
namespace {

template <int D_>
struct Many8 {
  static constexpr int D = D_;
  static constexpr bool kDirectKeys = true;
  // Significant bits of T, four to a number.
  template <typename T>
  static constexpr int kTerms = std::is_same_v<T, __half> ? 3 : 2;
  struct Keys {
    CUtensorMap k, v;  // [block][all heads' tokens][D], k's swizzled
  };
};

template <typename T, int D>
cudaError_t launch_type(const KvAttn &p, const ManyCtl &ctl, float *ws, int ctas, cudaStream_t s) {
  typename Many8<D>::Keys keys;
  const long long rows = static_cast<long long>(p.c.Hk) << p.c.bs_log2;
  if (api_encode_bytes(&keys.k, p.c.k_codes, D, rows, p.c.num_blocks, 1 << p.c.bs_log2, true) != 0 ||
      api_encode_bytes(&keys.v, p.c.v_codes, D, rows, p.c.num_blocks, 1 << p.c.bs_log2, false) != 0)
    return cudaErrorUnknown;
  return launch_many<T, Many8<D>>(p, ctl, ws, keys, ctas, s);
}

}  // namespace

cudaError_t launch_kv8_many(const KvAttn &p, const KvGrid &g, int dtype, float *ws,
                            unsigned *status, unsigned long long wait_limit_ns, int skip_load,
                            cudaStream_t s) {
  const ManyCtl ctl = {status, wait_limit_ns, skip_load, g.rows, R / p.group};
  if (dtype == FA_DTYPE_BF16)
    return p.c.d == 64 ? launch_type<__nv_bfloat16, 64>(p, ctl, ws, g.many, s)
                       : launch_type<__nv_bfloat16, 128>(p, ctl, ws, g.many, s);
  return p.c.d == 64 ? launch_type<__half, 64>(p, ctl, ws, g.many, s)
                     : launch_type<__half, 128>(p, ctl, ws, g.many, s);
}

}  // namespace fa
