// fa_serve_api.cu — host side of the serving operators declared in
// include/fa.h: argument checks, device checks and dispatch.  Nothing here
// computes; the kernels are in fa_plan.cu, fa_rope.cu, fa_pages.cu, fa_kv4_cache.cu,
// fa_kv8_cache.cu, and fa_kv_attn.cuh and fa_kv_many.cuh for either cache.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <utility>

#include "fa.h"
#include "fa_serve.h"

namespace {

using u64 = unsigned long long;

bool off_by(const void *p, unsigned n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

struct Span {
  const void *p;
  size_t n;
};

bool meet(const Span &a, const Span &b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && a.n && b.n && x < y + b.n && y < x + a.n;
}

// Whether some span of `out` overlaps another one of `out` or one of `in`.
template <int O, int I>
bool any_meet(const Span (&out)[O], const Span (&in)[I]) {
  for (int a = 0; a < O; ++a) {
    for (int b = a + 1; b < O; ++b)
      if (meet(out[a], out[b])) return true;
    for (const Span &x : in)
      if (meet(out[a], x)) return true;
  }
  return false;
}

bool known_dtype(int dtype) {
  return dtype == FA_DTYPE_BF16 || dtype == FA_DTYPE_F16 || dtype == FA_DTYPE_F32 ||
         dtype == FA_DTYPE_F32_SIMT;
}

size_t type_size(int dtype) { return dtype == FA_DTYPE_BF16 || dtype == FA_DTYPE_F16 ? 2 : 4; }

// log2 of an allowed block size, or -1.
int block_log2(int bs) { return bs == 16 ? 4 : bs == 32 ? 5 : bs == 64 ? 6 : bs == 128 ? 7 : -1; }

// The checks every entry point over the 4-bit cache shares.
int cache_store(void *k_codes, void *k_scales, void *v_codes, void *v_scales, int num_blocks,
                int Hk, int block_size, int d, int k_exp, int v_exp, fa::KvStore *c) {
  if (!k_codes || !k_scales || !v_codes || !v_scales) return FA_ERR_INVALID_ARG;
  if (off_by(k_codes, 16) || off_by(k_scales, 16) || off_by(v_codes, 16) || off_by(v_scales, 16))
    return FA_ERR_INVALID_ARG;
  if (num_blocks < 1 || Hk < 1 || Hk > 65535 || d < 1) return FA_ERR_INVALID_ARG;
  if (block_log2(block_size) < 0) return FA_ERR_INVALID_ARG;
  if (k_exp < -64 || k_exp > 64 || v_exp < -64 || v_exp > 64) return FA_ERR_INVALID_ARG;
  if (d % 16 != 0 || d > 256) return FA_ERR_UNSUPPORTED;
  c->k_codes = static_cast<uint8_t *>(k_codes);
  c->k_scales = static_cast<uint8_t *>(k_scales);
  c->v_codes = static_cast<uint8_t *>(v_codes);
  c->v_scales = static_cast<uint8_t *>(v_scales);
  c->num_blocks = num_blocks;
  c->Hk = Hk;
  c->bs_log2 = block_log2(block_size);
  c->d = d;
  c->k_exp = k_exp;
  c->v_exp = v_exp;
  return FA_OK;
}

// The same over the 8-bit cache.
int cache8_store(void *k_codes, float *k_scales, void *v_codes, float *v_scales, int num_blocks,
                 int Hk, int block_size, int d, fa::KvStore *c) {
  if (!k_codes || !k_scales || !v_codes || !v_scales) return FA_ERR_INVALID_ARG;
  if (off_by(k_codes, 32) || off_by(k_scales, 4) || off_by(v_codes, 32) || off_by(v_scales, 4))
    return FA_ERR_INVALID_ARG;
  if (num_blocks < 1 || Hk < 1 || Hk > 65535 || d < 1) return FA_ERR_INVALID_ARG;
  if (block_log2(block_size) < 0) return FA_ERR_INVALID_ARG;
  if (d % 16 != 0 || d > 256) return FA_ERR_UNSUPPORTED;
  *c = fa::KvStore{static_cast<uint8_t *>(k_codes), reinterpret_cast<uint8_t *>(k_scales),
                   static_cast<uint8_t *>(v_codes), reinterpret_cast<uint8_t *>(v_scales),
                   num_blocks, Hk, block_log2(block_size), d, 0, 0};
  return FA_OK;
}

size_t cache_rows(const fa::KvStore &c) {
  return (static_cast<size_t>(c.num_blocks) * c.Hk) << c.bs_log2;
}

// Bytes of a cache's codes and of its scales.
struct CacheBytes {
  size_t codes, scales;
};
CacheBytes cache_bytes(const fa::KvStore &c, bool eight) {
  const size_t rows = cache_rows(c);
  return eight ? CacheBytes{rows * c.d, static_cast<size_t>(c.num_blocks) * c.Hk * 4}
               : CacheBytes{rows * c.d / 2, rows * c.d / 16};
}

struct Dim {
  long long stride;
  int count;
};

// Rows of `row` bytes at every combination of three strides (bytes, not negative).
struct Rows {
  const void *p;
  long long row;
  Dim dims[3];
  // From the first byte to behind the last.  (Below 2^63: see kMaxExtent.)
  long long extent() const {
    long long n = row;
    for (const Dim &x : dims) n += x.stride * (x.count - 1);
    return n;
  }
};
// Each dimension's reach, in bytes: the sum of three and their products below
// stay far from 64 bits, and no address space is larger.
constexpr long long kMaxExtent = 1LL << 56;

// Whether a byte may be in both: their spans meet, and no pitch keeps them apart.
// A pitch is one of their strides; the strides that are multiples of it only move
// rows by whole pitches, so the two lie apart where the columns modulo the pitch
// that the others cover do (q and k as slices of one projection's rows).  Rows
// that interleave in another way count as meeting.
bool may_meet(const Rows &a, const Rows &b) {
  if (!a.p || !b.p) return false;
  if (!meet(Span{a.p, static_cast<size_t>(a.extent())}, Span{b.p, static_cast<size_t>(b.extent())}))
    return false;
  for (const Rows *from : {&a, &b})
    for (const Dim &x : from->dims) {
      const long long pitch = x.stride;
      if (x.count == 1 || pitch == 0) continue;
      auto columns = [&](const Rows &r) {
        long long n = r.row;
        for (const Dim &y : r.dims)
          if (y.stride % pitch != 0) n += y.stride * (y.count - 1);
        return n;
      };
      const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
      const long long down = static_cast<long long>((pa < pb ? pb - pa : pa - pb) % pitch);
      const long long ahead = pa < pb || down == 0 ? down : pitch - down;  // of a to b
      if (ahead >= columns(a) && ahead + columns(b) <= pitch) return false;
    }
  return true;
}

// Whether the rows of d elements at every combination of three strides lie
// apart: taken by ascending stride, each stride covers what lies below it.
bool disjoint_rows(long long d, Dim a, Dim b, Dim c) {
  if (a.stride > b.stride) std::swap(a, b);
  if (b.stride > c.stride) std::swap(b, c);
  if (a.stride > b.stride) std::swap(a, b);
  long long extent = d;
  for (const Dim &x : {a, b, c}) {
    if (x.count == 1) continue;
    if (x.stride < extent) return false;
    extent += x.stride * (x.count - 1);
  }
  return true;
}

// The checks of a list of arrays, host pointers to read from and to write to.  Each
// array keeps to itself, but for the arrays read, which may be those written.
int pages_args(const void *const *from, void *const *to, const u64 *bytes, int num, int from_blocks,
               int to_blocks) {
  if (num == 0) return FA_OK;
  if (num < 0 || !from || !to || !bytes) return FA_ERR_INVALID_ARG;
  if (num > fa::kMaxArrays) return FA_ERR_UNSUPPORTED;
  for (int i = 0; i < num; ++i)
    if (!from[i] || !to[i] || bytes[i] < 1 || bytes[i] > 2147483647ull) return FA_ERR_INVALID_ARG;
  struct Piece {
    uintptr_t begin, end;
    bool written;
  } x[2 * fa::kMaxArrays];
  int n = 0;
  for (int i = 0; i < num; ++i) {
    const uintptr_t t = reinterpret_cast<uintptr_t>(to[i]), f = reinterpret_cast<uintptr_t>(from[i]);
    x[n++] = {t, t + bytes[i] * to_blocks, true};
    if (f != t)
      x[n++] = {f, f + bytes[i] * from_blocks, false};
    else if (from_blocks > to_blocks)  // what is read behind the pages written
      x[n++] = {t + bytes[i] * to_blocks, f + bytes[i] * from_blocks, false};
  }
  std::sort(x, x + n, [](const Piece &a, const Piece &b) { return a.begin < b.begin; });
  uintptr_t any = 0, out = 0;  // where the arrays so far end, and the written ones
  for (int i = 0; i < n; ++i) {
    if (x[i].begin < (x[i].written ? any : out)) return FA_ERR_INVALID_ARG;
    any = std::max(any, x[i].end);
    if (x[i].written) out = std::max(out, x[i].end);
  }
  return FA_OK;
}

bool meets_pages(const Span &x, const void *const *arrays, const u64 *bytes, int num, int blocks) {
  for (int i = 0; i < num; ++i)
    if (meet(x, Span{arrays[i], bytes[i] * blocks})) return true;
  return false;
}

// The head dims and groups that attention over either cache is built for.
bool kv_attends(int d, int group) {
  return (d == 64 || d == 128) && group <= fa::kKvManyRows;
}

// The bound on a sequence's keys that the kernels get: the caller's, what the
// table holds, and what they count in 32 bits.
int kv_max_keys(int max_seqlen_k, int max_blocks, int bs_log2) {
  long long n = static_cast<long long>(max_blocks) << bs_log2;
  if (n > max_seqlen_k) n = max_seqlen_k;
  return n > fa::kKvMaxKeys ? fa::kKvMaxKeys : static_cast<int>(n);
}

int done(cudaError_t e) { return e == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

fa::KvGrid attention_grid(bool eight, int B, int Hk, int group, int d, int max_q, int max_k,
                          int num_sms) {
  return eight ? fa::kv8_grid(B, Hk, group, d, max_q, max_k, num_sms)
               : fa::kv4_grid(B, Hk, group, d, max_q, max_k, num_sms);
}

int attention_schedule(bool eight, int B, int Hq, int Hk, int max_seqlen_q, int max_seqlen_k,
                       int max_blocks, int block_size, int d, int num_sms, int *max_keys,
                       int *tile_rows, int *cluster, int *ctas, int *many_ctas) {
  if (!max_keys || !tile_rows || !cluster || !ctas || !many_ctas) return FA_ERR_INVALID_ARG;
  const int lg = block_log2(block_size);
  if (B < 1 || B > 65535 || Hq < 1 || Hq > 65535 || Hk < 1 || Hq % Hk != 0 || max_seqlen_q < 1 ||
      max_seqlen_k < 0 || max_blocks < 1 || lg < 0 || d < 1 || num_sms < 1 ||
      num_sms > 65535)
    return FA_ERR_INVALID_ARG;
  if ((static_cast<long long>(max_blocks) << lg) > 2147483647LL) return FA_ERR_INVALID_ARG;
  if (!kv_attends(d, Hq / Hk)) return FA_ERR_UNSUPPORTED;
  *max_keys = kv_max_keys(max_seqlen_k, max_blocks, lg);
  const fa::KvGrid g = attention_grid(eight, B, Hk, Hq / Hk, d, max_seqlen_q, *max_keys, num_sms);
  *tile_rows = g.rows;
  *cluster = g.cluster;
  *ctas = g.ctas;
  *many_ctas = g.many;
  return FA_OK;
}

u64 attention_workspace(bool eight, int B, int Hq, int Hk, int max_seqlen_q, int d) {
  if (B < 1 || Hq < 1 || Hk < 1 || Hq % Hk != 0 || max_seqlen_q < 1) return 0;
  if (!kv_attends(d, Hq / Hk)) return 0;
  const int group = Hq / Hk, tile = eight ? fa::kv8_tile_rows(group, max_seqlen_q, d)
                                          : fa::kv4_tile_rows(group, max_seqlen_q, d, 0);
  const size_t few = tile ? fa::kv_workspace(tile, d) : 0;
  // (with many keys the other kernel may take what 32 rows hold)
  const size_t many = static_cast<long long>(max_seqlen_q) * group > tile || tile == 32
                          ? fa::kv_workspace(fa::kKvManyRows, d)
                          : 0;
  return few > many ? few : many;
}

// Attention over a cache whose arrays have passed their checks; k_exp and v_exp are
// in c.
int attention(bool eight, const void *q, void *o, float *lse, const fa::KvStore &c,
              const int *block_table, const int *seq_lens_k, const int *cu_seqlens_q, int B, int Hq,
              int total_q, int max_seqlen_q, int max_seqlen_k, int max_blocks, float scale,
              int causal, int dtype, void *workspace, u64 workspace_bytes, void *stream) {
  if (Hq % c.Hk != 0) return FA_ERR_INVALID_ARG;
  if ((static_cast<long long>(max_blocks) << c.bs_log2) > 2147483647LL) return FA_ERR_INVALID_ARG;
  const float scale_log2 =
      static_cast<float>(std::ldexp(static_cast<double>(scale) * 1.4426950408889634, c.k_exp));
  if (!std::isfinite(scale_log2)) return FA_ERR_INVALID_ARG;
  if (off_by(q, 16) || off_by(o, 16) || off_by(lse, 4) || off_by(block_table, 4) ||
      off_by(seq_lens_k, 4) || off_by(cu_seqlens_q, 4))
    return FA_ERR_INVALID_ARG;
  const size_t es = type_size(dtype);
  const CacheBytes n = cache_bytes(c, eight);
  const size_t qn = static_cast<size_t>(total_q) * Hq * c.d * es;
  const size_t need = attention_workspace(eight, B, Hq, c.Hk, max_seqlen_q, c.d);
  const Span out[] = {{o, qn}, {lse, static_cast<size_t>(total_q) * Hq * 4}, {workspace, need}};
  const Span in[] = {{q, qn}, {c.k_codes, n.codes}, {c.k_scales, n.scales},
                     {c.v_codes, n.codes}, {c.v_scales, n.scales},
                     {block_table, static_cast<size_t>(B) * max_blocks * 4},
                     {seq_lens_k, static_cast<size_t>(B) * 4},
                     {cu_seqlens_q, static_cast<size_t>(B + 1) * 4}};
  if (any_meet(out, in)) return FA_ERR_INVALID_ARG;
  if (dtype != FA_DTYPE_BF16 && dtype != FA_DTYPE_F16) return FA_ERR_UNSUPPORTED;
  if (!kv_attends(c.d, Hq / c.Hk)) return FA_ERR_UNSUPPORTED;
  if (need > 0 && (!workspace || off_by(workspace, 256) || workspace_bytes < need))
    return FA_ERR_INVALID_ARG;
  unsigned *status = nullptr;
  const int rc = fa::api_device_status(&status);
  if (rc != FA_OK) return rc;
  fa::KvAttn p;
  p.q = q;
  p.o = o;
  p.lse = lse;
  p.c = c;
  p.table = block_table;
  p.lens = seq_lens_k;
  p.cu_q = cu_seqlens_q;
  p.B = B;
  p.Hq = Hq;
  p.group = Hq / c.Hk;
  p.total_q = total_q;
  p.max_q = max_seqlen_q;
  p.max_k = kv_max_keys(max_seqlen_k, max_blocks, c.bs_log2);
  p.width = max_blocks;
  p.scale_log2 = scale_log2;
  p.v_mul = static_cast<float>(std::ldexp(1.0, c.v_exp));
  p.causal = causal;
  const fa::KvGrid g =
      attention_grid(eight, B, c.Hk, p.group, c.d, max_seqlen_q, p.max_k, fa::api_sm_count());
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  float *ws = static_cast<float *>(workspace);
  cudaError_t e = cudaSuccess;
  if (g.rows > 0)
    e = eight ? fa::launch_kv8_attn(p, g, dtype, ws, s) : fa::launch_kv4_attn(p, g, dtype, ws, s);
  if (e == cudaSuccess && g.many > 0)
    e = (eight ? fa::launch_kv8_many : fa::launch_kv4_many)(
        p, g, dtype, ws, status, fa::api_wait_limit(), fa::api_skip_load(), s);
  return done(e);
}

// The checks of fa_fwd_kv4 and fa_fwd_kv8 ahead of the cache's.
int attention_args(const void *q, const void *o, const float *lse, const int *block_table,
                   const int *seq_lens_k, const int *cu_seqlens_q, int B, int Hq, int total_q,
                   int max_seqlen_q, int max_seqlen_k, int max_blocks, float scale, int causal,
                   int dtype) {
  if (!q || !o || !lse || !block_table || !seq_lens_k) return FA_ERR_INVALID_ARG;
  if (B < 1 || B > 65535 || Hq < 1 || Hq > 65535 || total_q < 1 || max_blocks < 1)
    return FA_ERR_INVALID_ARG;
  if (max_seqlen_q < 1 || max_seqlen_q > total_q || max_seqlen_k < 0) return FA_ERR_INVALID_ARG;
  if (!cu_seqlens_q && (max_seqlen_q != 1 || total_q != B)) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || (causal != 0 && causal != 1)) return FA_ERR_INVALID_ARG;
  if (!known_dtype(dtype)) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

}  // namespace

extern "C" int fa_kv_plan(const int *cached_lens, const int *new_lens, const int *free_blocks,
                          const int *free_head, int *block_table, long long *slots,
                          int *positions, int *cu_seqlens, int *seq_lens, int *counts, int B,
                          int max_blocks, int block_size, int num_free, int capacity,
                          void *stream) {
  if (!cached_lens || !new_lens || !block_table || !slots || !positions || !cu_seqlens ||
      !seq_lens || !counts)
    return FA_ERR_INVALID_ARG;
  if (B < 1 || B > 65535 || max_blocks < 1 || num_free < 0 || capacity < 1)
    return FA_ERR_INVALID_ARG;
  if (num_free > 0 && !free_blocks) return FA_ERR_INVALID_ARG;
  const int lg = block_log2(block_size);
  if (lg < 0 || (static_cast<long long>(max_blocks) << lg) > 2147483647LL)
    return FA_ERR_INVALID_ARG;
  for (const void *p : {static_cast<const void *>(cached_lens), static_cast<const void *>(new_lens),
                        static_cast<const void *>(free_blocks),
                        static_cast<const void *>(free_head),
                        static_cast<const void *>(block_table),
                        static_cast<const void *>(positions),
                        static_cast<const void *>(cu_seqlens), static_cast<const void *>(seq_lens),
                        static_cast<const void *>(counts)})
    if (off_by(p, 4)) return FA_ERR_INVALID_ARG;
  if (off_by(slots, 8)) return FA_ERR_INVALID_ARG;
  const size_t n = B;
  const Span out[] = {{block_table, n * max_blocks * 4}, {slots, static_cast<size_t>(capacity) * 8},
                      {positions, static_cast<size_t>(capacity) * 4}, {cu_seqlens, (n + 1) * 4},
                      {seq_lens, n * 4}, {counts, 8}};
  const Span in[] = {{cached_lens, n * 4}, {new_lens, n * 4},
                     {free_blocks, static_cast<size_t>(num_free) * 4}, {free_head, 4}};
  if (any_meet(out, in)) return FA_ERR_INVALID_ARG;
  int rc;
  if ((rc = fa::api_device_check()) != FA_OK) return rc;
  const fa::PlanParams p = {cached_lens, new_lens, free_blocks, free_head, block_table, slots,
                            positions, cu_seqlens, seq_lens, counts, B, max_blocks, lg, num_free,
                            capacity};
  return done(fa::launch_plan(p, static_cast<cudaStream_t>(stream)));
}

extern "C" int fa_rope_table(const double *inv_freq, const int *axis, int n,
                             unsigned long long *table) {
  if (!inv_freq || !table || n < 1) return FA_ERR_INVALID_ARG;
  // 1 / (2 pi) as a sum of two doubles
  constexpr double hi = 0.15915494309189535, lo = -9.839338337591243e-18;
  for (int i = 0; i < n; ++i) {
    const double f = inv_freq[i];
    const int a = axis ? axis[i] : 0;
    if (!(std::fabs(f) <= 1.0e6) || a < 0 || a > 3) return FA_ERR_INVALID_ARG;
  }
  for (int i = 0; i < n; ++i) {
    // |f| / (2 pi) = t + e with |e| below t's last place; turns modulo one,
    // scaled by 2^64 in two 32-bit steps so that no bit of t is lost (t minus
    // its floor is exact for t >= 0)
    const double f = std::fabs(inv_freq[i]), t = f * hi;
    const double e = std::fma(f, hi, -t) + f * lo;
    const double frac = std::ldexp(t - std::floor(t), 32), top = std::floor(frac);
    u64 w = static_cast<u64>(top) << 32;
    w += static_cast<u64>(std::ldexp(frac - top, 32));
    w += static_cast<u64>(static_cast<long long>(std::llrint(std::ldexp(e, 64))));
    if (inv_freq[i] < 0) w = 0 - w;
    table[i] = (w & ~3ull) | static_cast<u64>(axis ? axis[i] : 0);
  }
  return FA_OK;
}

extern "C" int fa_rope(const void *q, void *q_out, const long long *q_strides, int Hq,
                       const void *k, void *k_out, const long long *k_strides, int Hk,
                       const int *positions, int num_axes, const unsigned long long *table, int B,
                       int N, int d, int d_rot, int interleaved, int inverse, int dtype,
                       void *stream) {
  if (!q || !q_out || !positions || !table) return FA_ERR_INVALID_ARG;
  if (Hq < 1 || Hk < 0 || Hq > 65535 || Hk > 65535 || B < 1 || N < 1 || d < 1)
    return FA_ERR_INVALID_ARG;
  if (Hk > 0 && (!k || !k_out)) return FA_ERR_INVALID_ARG;
  if (num_axes < 1 || num_axes > 4) return FA_ERR_INVALID_ARG;
  if (d_rot < 2 || d_rot % 2 != 0 || d_rot > d) return FA_ERR_INVALID_ARG;
  if ((interleaved != 0 && interleaved != 1) || (inverse != 0 && inverse != 1))
    return FA_ERR_INVALID_ARG;
  if (!known_dtype(dtype)) return FA_ERR_INVALID_ARG;
  const unsigned es = static_cast<unsigned>(type_size(dtype));
  if (off_by(q, es) || off_by(q_out, es) || off_by(k, es) || off_by(k_out, es) ||
      off_by(positions, 4) || off_by(table, 8))
    return FA_ERR_INVALID_ARG;
  if (d > 256) return FA_ERR_UNSUPPORTED;
  auto tensor = [&](const void *in, void *out, const long long *st, int heads) {
    fa::RopeTensor t = {in, out, 0, 0, 0, 0, 0, 0, heads};
    if (st) {
      t.ib = st[0], t.ih = st[1], t.in_row = st[2];
      t.ob = st[3], t.oh = st[4], t.out_row = st[5];
    } else {
      t.ib = t.ob = static_cast<long long>(heads) * N * d;
      t.ih = t.oh = static_cast<long long>(N) * d;
      t.in_row = t.out_row = d;
    }
    return t;
  };
  fa::RopeParams p = {tensor(q, q_out, q_strides, Hq), tensor(k, k_out, k_strides, Hk), positions,
                      table, static_cast<long long>(B) * N, N, d, d_rot, num_axes, interleaved,
                      inverse};
  // Outputs overlap nothing but, in place, their own input at its own strides.
  auto rows = [&](const void *base, long long sb, long long sh, long long sn, int heads) {
    auto dim = [&](long long s, int n) { return Dim{n == 1 ? 0 : s * es, n}; };
    return Rows{base, static_cast<long long>(d) * es, {dim(sb, B), dim(sh, heads), dim(sn, N)}};
  };
  auto in_reach = [&](long long stride, int count) {
    return stride >= 0 && (count == 1 || stride <= kMaxExtent / es / (count - 1));
  };
  Rows in[2] = {}, out[2] = {};
  for (int i = 0; i < 2; ++i) {
    const fa::RopeTensor &t = i == 0 ? p.q : p.k;
    if (t.heads == 0) continue;
    if (!in_reach(t.ib, B) || !in_reach(t.ih, t.heads) || !in_reach(t.in_row, N) ||
        !in_reach(t.ob, B) || !in_reach(t.oh, t.heads) || !in_reach(t.out_row, N))
      return FA_ERR_INVALID_ARG;
    if (!disjoint_rows(d, {t.ob, B}, {t.oh, t.heads}, {t.out_row, N})) return FA_ERR_INVALID_ARG;
    in[i] = rows(t.in, t.ib, t.ih, t.in_row, t.heads);
    out[i] = rows(t.out, t.ob, t.oh, t.out_row, t.heads);
    const bool same = t.in == t.out;
    if (same ? (B > 1 && t.ib != t.ob) || (t.heads > 1 && t.ih != t.oh) ||
                   (N > 1 && t.in_row != t.out_row)
             : may_meet(out[i], in[i]))
      return FA_ERR_INVALID_ARG;
    const Span to[] = {{out[i].p, static_cast<size_t>(out[i].extent())}};
    const Span from[] = {{positions, static_cast<size_t>(num_axes) * p.rows * 4},
                         {table, static_cast<size_t>(d_rot / 2) * 8}};
    if (any_meet(to, from)) return FA_ERR_INVALID_ARG;
  }
  if (may_meet(out[0], out[1]) || may_meet(out[0], in[1]) || may_meet(out[1], in[0]))
    return FA_ERR_INVALID_ARG;
  int rc;
  if ((rc = fa::api_device_check()) != FA_OK) return rc;
  return done(fa::launch_rope(p, dtype, fa::api_sm_count(), static_cast<cudaStream_t>(stream)));
}

extern "C" int fa_kv4_append(const void *k, const void *v, long long k_stride, long long v_stride,
                             const long long *slots, int T, void *k_codes, void *k_scales,
                             void *v_codes, void *v_scales, int num_blocks, int Hk,
                             int block_size, int d, int k_exp, int v_exp, int dtype,
                             void *stream) {
  if (!k || !v || !slots || T < 1) return FA_ERR_INVALID_ARG;
  if (!known_dtype(dtype)) return FA_ERR_INVALID_ARG;
  fa::KvStore c;
  int rc = cache_store(k_codes, k_scales, v_codes, v_scales, num_blocks, Hk, block_size, d, k_exp,
                       v_exp, &c);
  if (rc != FA_OK) return rc;
  const size_t es = type_size(dtype), row = static_cast<size_t>(Hk) * d;
  if (off_by(k, 16) || off_by(v, 16) || off_by(slots, 8)) return FA_ERR_INVALID_ARG;
  if (k_stride < static_cast<long long>(row) || v_stride < static_cast<long long>(row) ||
      k_stride * es % 16 != 0 || v_stride * es % 16 != 0)
    return FA_ERR_INVALID_ARG;
  const size_t rows = cache_rows(c);
  const Span out[] = {{k_codes, rows * d / 2}, {k_scales, rows * d / 16}, {v_codes, rows * d / 2},
                      {v_scales, rows * d / 16}};
  const Span in[] = {{k, ((T - 1) * static_cast<size_t>(k_stride) + row) * es},
                     {v, ((T - 1) * static_cast<size_t>(v_stride) + row) * es},
                     {slots, static_cast<size_t>(T) * 8}};
  if (any_meet(out, in)) return FA_ERR_INVALID_ARG;
  if ((rc = fa::api_device_check()) != FA_OK) return rc;
  return done(fa::launch_kv4_append(k, v, k_stride, v_stride, slots, T, c, dtype,
                                    static_cast<cudaStream_t>(stream)));
}

extern "C" int fa_kv4_gather(const long long *slots, int R, const void *k_codes,
                             const void *k_scales, const void *v_codes, const void *v_scales,
                             void *k_out, void *v_out, int num_blocks, int Hk, int block_size,
                             int d, int k_exp, int v_exp, int dtype, void *stream) {
  if (!slots || !k_out || !v_out || R < 1) return FA_ERR_INVALID_ARG;
  if (!known_dtype(dtype)) return FA_ERR_INVALID_ARG;
  fa::KvStore c;
  int rc = cache_store(const_cast<void *>(k_codes), const_cast<void *>(k_scales),
                       const_cast<void *>(v_codes), const_cast<void *>(v_scales), num_blocks, Hk,
                       block_size, d, k_exp, v_exp, &c);
  if (rc != FA_OK) return rc;
  if (off_by(k_out, 16) || off_by(v_out, 16) || off_by(slots, 8)) return FA_ERR_INVALID_ARG;
  const size_t rows = cache_rows(c), n = static_cast<size_t>(R) * Hk * d * type_size(dtype);
  const Span out[] = {{k_out, n}, {v_out, n}};
  const Span in[] = {{k_codes, rows * d / 2}, {k_scales, rows * d / 16}, {v_codes, rows * d / 2},
                     {v_scales, rows * d / 16}, {slots, static_cast<size_t>(R) * 8}};
  if (any_meet(out, in)) return FA_ERR_INVALID_ARG;
  if ((rc = fa::api_device_check()) != FA_OK) return rc;
  return done(fa::launch_kv4_gather(slots, R, c, k_out, v_out, dtype,
                                    static_cast<cudaStream_t>(stream)));
}

extern "C" int fa_fwd_kv4_schedule(int B, int Hq, int Hk, int max_seqlen_q, int max_seqlen_k,
                                   int max_blocks, int block_size, int d, int num_sms,
                                   int *max_keys, int *tile_rows, int *cluster, int *ctas,
                                   int *many_ctas) {
  return attention_schedule(false, B, Hq, Hk, max_seqlen_q, max_seqlen_k, max_blocks, block_size, d,
                            num_sms, max_keys, tile_rows, cluster, ctas, many_ctas);
}

extern "C" int fa_fwd_kv8_schedule(int B, int Hq, int Hk, int max_seqlen_q, int max_seqlen_k,
                                   int max_blocks, int block_size, int d, int num_sms,
                                   int *max_keys, int *tile_rows, int *cluster, int *ctas,
                                   int *many_ctas) {
  return attention_schedule(true, B, Hq, Hk, max_seqlen_q, max_seqlen_k, max_blocks, block_size, d,
                            num_sms, max_keys, tile_rows, cluster, ctas, many_ctas);
}

extern "C" unsigned long long fa_fwd_kv4_workspace(int B, int Hq, int Hk, int max_seqlen_q, int d) {
  return attention_workspace(false, B, Hq, Hk, max_seqlen_q, d);
}

extern "C" unsigned long long fa_fwd_kv8_workspace(int B, int Hq, int Hk, int max_seqlen_q, int d) {
  return attention_workspace(true, B, Hq, Hk, max_seqlen_q, d);
}

extern "C" int fa_fwd_kv4(const void *q, void *o, float *lse, const void *k_codes,
                          const void *k_scales, const void *v_codes, const void *v_scales,
                          const int *block_table, const int *seq_lens_k, const int *cu_seqlens_q,
                          int B, int Hq, int Hk, int total_q, int max_seqlen_q, int max_seqlen_k,
                          int num_blocks, int block_size, int max_blocks, int d, float scale,
                          int causal, int k_exp, int v_exp, int dtype, void *workspace,
                          unsigned long long workspace_bytes, void *stream) {
  int rc = attention_args(q, o, lse, block_table, seq_lens_k, cu_seqlens_q, B, Hq, total_q,
                          max_seqlen_q, max_seqlen_k, max_blocks, scale, causal, dtype);
  if (rc != FA_OK) return rc;
  fa::KvStore c;
  rc = cache_store(const_cast<void *>(k_codes), const_cast<void *>(k_scales),
                   const_cast<void *>(v_codes), const_cast<void *>(v_scales), num_blocks, Hk,
                   block_size, d, k_exp, v_exp, &c);
  if (rc != FA_OK) return rc;
  return attention(false, q, o, lse, c, block_table, seq_lens_k, cu_seqlens_q, B, Hq, total_q,
                   max_seqlen_q, max_seqlen_k, max_blocks, scale, causal, dtype, workspace,
                   workspace_bytes, stream);
}

extern "C" int fa_fwd_kv8(const void *q, void *o, float *lse, const void *k_codes,
                          const float *k_scales, const void *v_codes, const float *v_scales,
                          const int *block_table, const int *seq_lens_k, const int *cu_seqlens_q,
                          int B, int Hq, int Hk, int total_q, int max_seqlen_q, int max_seqlen_k,
                          int num_blocks, int block_size, int max_blocks, int d, float scale,
                          int causal, int dtype, void *workspace,
                          unsigned long long workspace_bytes, void *stream) {
  int rc = attention_args(q, o, lse, block_table, seq_lens_k, cu_seqlens_q, B, Hq, total_q,
                          max_seqlen_q, max_seqlen_k, max_blocks, scale, causal, dtype);
  if (rc != FA_OK) return rc;
  fa::KvStore c;
  rc = cache8_store(const_cast<void *>(k_codes), const_cast<float *>(k_scales),
                    const_cast<void *>(v_codes), const_cast<float *>(v_scales), num_blocks, Hk,
                    block_size, d, &c);
  if (rc != FA_OK) return rc;
  return attention(true, q, o, lse, c, block_table, seq_lens_k, cu_seqlens_q, B, Hq, total_q,
                   max_seqlen_q, max_seqlen_k, max_blocks, scale, causal, dtype, workspace,
                   workspace_bytes, stream);
}

extern "C" int fa_kv8_append(const void *k, const void *v, long long k_stride, long long v_stride,
                             const long long *slots, int T, void *k_codes, float *k_scales,
                             void *v_codes, float *v_scales, int num_blocks, int Hk,
                             int block_size, int d, int dtype, void *stream) {
  if (!k || !v || !slots || T < 1) return FA_ERR_INVALID_ARG;
  if (!known_dtype(dtype)) return FA_ERR_INVALID_ARG;
  fa::KvStore c;
  int rc = cache8_store(k_codes, k_scales, v_codes, v_scales, num_blocks, Hk, block_size, d, &c);
  if (rc != FA_OK) return rc;
  const size_t es = type_size(dtype), row = static_cast<size_t>(Hk) * d;
  if (off_by(k, 16) || off_by(v, 16) || off_by(slots, 8)) return FA_ERR_INVALID_ARG;
  if (k_stride < static_cast<long long>(row) || v_stride < static_cast<long long>(row) ||
      k_stride * es % 16 != 0 || v_stride * es % 16 != 0)
    return FA_ERR_INVALID_ARG;
  const CacheBytes n = cache_bytes(c, true);
  const Span out[] = {{k_codes, n.codes}, {k_scales, n.scales}, {v_codes, n.codes},
                      {v_scales, n.scales}};
  const Span in[] = {{k, ((T - 1) * static_cast<size_t>(k_stride) + row) * es},
                     {v, ((T - 1) * static_cast<size_t>(v_stride) + row) * es},
                     {slots, static_cast<size_t>(T) * 8}};
  if (any_meet(out, in)) return FA_ERR_INVALID_ARG;
  if ((rc = fa::api_device_check()) != FA_OK) return rc;
  return done(fa::launch_kv8_append(k, v, k_stride, v_stride, slots, T, c, dtype,
                                    static_cast<cudaStream_t>(stream)));
}

extern "C" int fa_kv8_gather(const long long *slots, int R, const void *k_codes,
                             const float *k_scales, const void *v_codes, const float *v_scales,
                             void *k_out, void *v_out, int num_blocks, int Hk, int block_size,
                             int d, int dtype, void *stream) {
  if (!slots || !k_out || !v_out || R < 1) return FA_ERR_INVALID_ARG;
  if (!known_dtype(dtype)) return FA_ERR_INVALID_ARG;
  fa::KvStore c;
  int rc = cache8_store(const_cast<void *>(k_codes), const_cast<float *>(k_scales),
                        const_cast<void *>(v_codes), const_cast<float *>(v_scales), num_blocks, Hk,
                        block_size, d, &c);
  if (rc != FA_OK) return rc;
  if (off_by(k_out, 16) || off_by(v_out, 16) || off_by(slots, 8)) return FA_ERR_INVALID_ARG;
  const CacheBytes b = cache_bytes(c, true);
  const size_t n = static_cast<size_t>(R) * Hk * d * type_size(dtype);
  const Span out[] = {{k_out, n}, {v_out, n}};
  const Span in[] = {{k_codes, b.codes}, {k_scales, b.scales}, {v_codes, b.codes},
                     {v_scales, b.scales}, {slots, static_cast<size_t>(R) * 8}};
  if (any_meet(out, in)) return FA_ERR_INVALID_ARG;
  if ((rc = fa::api_device_check()) != FA_OK) return rc;
  return done(fa::launch_kv8_gather(slots, R, c, k_out, v_out, dtype,
                                    static_cast<cudaStream_t>(stream)));
}

extern "C" int fa_kv_copy(const int *src, const int *dst, int n, const void *const *from,
                          void *const *to, const unsigned long long *page_bytes, int num_arrays,
                          int from_blocks, int to_blocks, void *stream) {
  if (!src || !dst || off_by(src, 4) || off_by(dst, 4) || n < 1) return FA_ERR_INVALID_ARG;
  if (from_blocks < 1 || to_blocks < 1 || num_arrays < 1) return FA_ERR_INVALID_ARG;
  int rc = pages_args(from, to, page_bytes, num_arrays, from_blocks, to_blocks);
  if (rc != FA_OK) return rc;
  const Span ids[] = {{src, static_cast<size_t>(n) * 4}, {dst, static_cast<size_t>(n) * 4}};
  for (const Span &x : ids)
    if (meets_pages(x, to, page_bytes, num_arrays, to_blocks)) return FA_ERR_INVALID_ARG;
  if ((rc = fa::api_device_check()) != FA_OK) return rc;
  return done(fa::launch_kv_copy({from, to, page_bytes, num_arrays}, src, dst, n, from_blocks,
                                 to_blocks, fa::api_sm_count(), static_cast<cudaStream_t>(stream)));
}

extern "C" int fa_kv_fork(const int *block_table, const int *seq_lens, const int *parents,
                          const int *free_blocks, const int *free_head, int *table_out,
                          int *lens_out, int *counts, int B, int n, int max_blocks, int block_size,
                          int num_free, int num_blocks, int parents_end, void *const *arrays,
                          const unsigned long long *page_bytes, int num_arrays, void *stream) {
  if (!block_table || !seq_lens || !parents || !table_out || !lens_out || !counts)
    return FA_ERR_INVALID_ARG;
  if (B < 1 || B > 65535 || n < 1 || n > 65535 || max_blocks < 1 || num_free < 0 || num_blocks < 1 ||
      num_arrays < 0)
    return FA_ERR_INVALID_ARG;
  if (num_free > 0 && !free_blocks) return FA_ERR_INVALID_ARG;
  if (parents_end != 0 && parents_end != 1) return FA_ERR_INVALID_ARG;
  const int lg = block_log2(block_size);
  if (lg < 0 || (static_cast<long long>(max_blocks) << lg) > 2147483647LL)
    return FA_ERR_INVALID_ARG;
  const size_t w = static_cast<size_t>(max_blocks) * 4;
  const Span out[] = {{table_out, n * w}, {lens_out, static_cast<size_t>(n) * 4}, {counts, 8}};
  const Span in[] = {{block_table, B * w}, {seq_lens, static_cast<size_t>(B) * 4},
                     {parents, static_cast<size_t>(n) * 4},
                     {free_blocks, static_cast<size_t>(num_free) * 4}, {free_head, 4}};
  for (const Span &x : out)
    if (off_by(x.p, 4)) return FA_ERR_INVALID_ARG;
  for (const Span &x : in)
    if (off_by(x.p, 4)) return FA_ERR_INVALID_ARG;
  if (any_meet(out, in)) return FA_ERR_INVALID_ARG;
  int rc = pages_args(arrays, arrays, page_bytes, num_arrays, num_blocks, num_blocks);
  if (rc != FA_OK) return rc;
  for (const Span &x : out)
    if (meets_pages(x, arrays, page_bytes, num_arrays, num_blocks)) return FA_ERR_INVALID_ARG;
  for (const Span &x : in)
    if (meets_pages(x, arrays, page_bytes, num_arrays, num_blocks)) return FA_ERR_INVALID_ARG;
  if ((rc = fa::api_device_check()) != FA_OK) return rc;
  const fa::ForkParams p = {block_table, seq_lens, parents, free_blocks, free_head, table_out,
                            lens_out, counts, B, n, max_blocks, lg, num_free, num_blocks,
                            parents_end};
  return done(fa::launch_kv_fork({const_cast<const void *const *>(arrays), arrays, page_bytes,
                                  num_arrays}, p, fa::api_sm_count(),
                                 static_cast<cudaStream_t>(stream)));
}

extern "C" int fa_kv_free(const int *block_table, int *seq_lens, const unsigned char *ended,
                          int *free_blocks, int *free_head, int B, int max_blocks, int block_size,
                          int num_blocks, void *stream) {
  if (!block_table || !seq_lens || !free_blocks || !free_head) return FA_ERR_INVALID_ARG;
  if (B < 1 || B > 65535 || max_blocks < 1 || num_blocks < 1) return FA_ERR_INVALID_ARG;
  const int lg = block_log2(block_size);
  if (lg < 0 || (static_cast<long long>(max_blocks) << lg) > 2147483647LL)
    return FA_ERR_INVALID_ARG;
  const size_t n = B;
  const Span out[] = {{seq_lens, n * 4}, {free_blocks, static_cast<size_t>(num_blocks) * 4},
                      {free_head, 4}};
  const Span in[] = {{block_table, n * max_blocks * 4}, {ended, n}};
  for (const void *p : {static_cast<const void *>(block_table), static_cast<const void *>(seq_lens),
                        static_cast<const void *>(free_blocks), static_cast<const void *>(free_head)})
    if (off_by(p, 4)) return FA_ERR_INVALID_ARG;
  if (any_meet(out, in)) return FA_ERR_INVALID_ARG;
  if (num_blocks > fa::kMaxSweep) return FA_ERR_UNSUPPORTED;
  const int rc = fa::api_device_check();
  if (rc != FA_OK) return rc;
  return done(fa::launch_kv_free({block_table, seq_lens, ended, free_blocks, free_head, B, max_blocks,
                                  lg, num_blocks}, static_cast<cudaStream_t>(stream)));
}

extern "C" unsigned long long fa_kv_compact_workspace(int num_blocks) {
  if (num_blocks < 1 || num_blocks > fa::kMaxSweep) return 0;
  return 8ull * (num_blocks / 2) + 8;
}

extern "C" int fa_kv_compact(const int *block_table, const int *seq_lens, int *table_out,
                             int *new_ids, int *counts, int B, int max_blocks, int block_size,
                             int num_blocks, void *const *arrays,
                             const unsigned long long *page_bytes, int num_arrays, void *workspace,
                             unsigned long long workspace_bytes, void *stream) {
  if (!block_table || !seq_lens || !table_out || !new_ids || !counts) return FA_ERR_INVALID_ARG;
  if (B < 1 || B > 65535 || max_blocks < 1 || num_blocks < 1 || num_arrays < 0)
    return FA_ERR_INVALID_ARG;
  const int lg = block_log2(block_size);
  if (lg < 0 || (static_cast<long long>(max_blocks) << lg) > 2147483647LL)
    return FA_ERR_INVALID_ARG;
  if (num_blocks > fa::kMaxSweep) return FA_ERR_UNSUPPORTED;
  const size_t n = B, table = n * max_blocks * 4, need = fa_kv_compact_workspace(num_blocks);
  if (!workspace || off_by(workspace, 4) || workspace_bytes < need) return FA_ERR_INVALID_ARG;
  const Span out[] = {{table_out, table}, {new_ids, static_cast<size_t>(num_blocks) * 4}, {counts, 8},
                      {workspace, need}};
  // (the table may be renumbered in place)
  const Span in[] = {{table_out == block_table ? nullptr : block_table, table}, {seq_lens, n * 4}};
  for (const void *p : {static_cast<const void *>(block_table), static_cast<const void *>(seq_lens),
                        static_cast<const void *>(table_out), static_cast<const void *>(new_ids),
                        static_cast<const void *>(counts)})
    if (off_by(p, 4)) return FA_ERR_INVALID_ARG;
  if (any_meet(out, in)) return FA_ERR_INVALID_ARG;
  int rc = pages_args(arrays, arrays, page_bytes, num_arrays, num_blocks, num_blocks);
  if (rc != FA_OK) return rc;
  for (const Span &x : out)
    if (meets_pages(x, arrays, page_bytes, num_arrays, num_blocks)) return FA_ERR_INVALID_ARG;
  for (const Span &x : {Span{block_table, table}, Span{seq_lens, n * 4}})
    if (meets_pages(x, arrays, page_bytes, num_arrays, num_blocks)) return FA_ERR_INVALID_ARG;
  if ((rc = fa::api_device_check()) != FA_OK) return rc;
  return done(fa::launch_kv_compact({const_cast<const void *const *>(arrays), arrays, page_bytes,
                                     num_arrays},
                                    {block_table, seq_lens, table_out, new_ids, counts,
                                     static_cast<int *>(workspace), B, max_blocks, lg, num_blocks},
                                    fa::api_sm_count(), static_cast<cudaStream_t>(stream)));
}
