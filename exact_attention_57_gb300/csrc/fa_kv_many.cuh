// fa_kv_many.cuh — attention of sequences with many queries over a paged cache of
// codes (chunks of prompts; the sequences that fa_kv_attn.cuh's tiles do not hold),
// on tcgen05, for any format F of the cache.
//
// A tile is 128 rows of one sequence and key head: row r is head r % group of
// query token t * tokens + r / group, tokens = 128 / group, so the heads that
// share a key head share its expanded keys and values.  Work is dealt as in
// fa_kv_split.cuh, a unit being 128 keys of one tile: one CTA on each SM,
// equal shares, whatever the lengths, the mask and the number of tiles.
//
// Warps 0-3    softmax, correction and epilogue, one row a thread.
// Warps 4-7    expand the codes of K, warps 8-11 those of V: thread r loads
//              token r of the 128 (a page lookup, the codes, the format's scales,
//              one step ahead), turns them into fp16 (exactly)
//              and writes them as a 128-byte-swizzled row.
//              Tokens behind the sequence or on a missing page become zeros
//              and are reported in a bit mask.
// Warp 12, 13  issue S = Q K^T (three score buffers) and O += P V (P in tensor
//              memory), kind::f16, fp32 accumulators; warp 12 owns the tensor
//              memory.
// Warp 14, 15  bring the next tile's Q into shared memory (two buffers), as
//              fp16 times a power of two a row.
//
// A format F has D, kBlockScales (the scales of 16 keys are one number each, which
// the softmax applies), and Row, a thread's share of the codes of its warp's 32
// tokens.  Without kStreams: load() of the thread's own token, expand() to fp16 by
// 16-byte units.  With kStreams: begin() loads the first step's, stream() turns one
// step's into fp16 and each register, once free, over to the next step's codes.  With
// kBlockScales, load_scales() and scales() by the threads of tokens 16 n.
//
// Every wait is bounded; on expiry the CTA raises its abort flag, records the
// role in the status word, drains its products, frees tensor memory and ends.
#include <atomic>
#include <cfloat>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa.h"
#include "fa_internal.h"
#include "fa_kv_split.cuh"
#include "fa_wait.cuh"

namespace fa {
namespace {

constexpr int kThreads = 512, kWarps = 16;
constexpr int R = kKvManyRows;

struct ManyCtl {
  unsigned *status;
  unsigned long long wait_limit_ns;
  int skip_load, tile_rows, tokens;  // tokens of a tile
};

constexpr int WALK_BYTES = 80;

template <class F>
struct ManyCfg {
  static constexpr int D = F::D;
  static constexpr int NCH = D / 64;               // 128-byte chunks of a row
  static constexpr int CHUNK = 128 * 128;
  static constexpr int TILE = NCH * CHUNK;
  static constexpr int NS = 3;                     // score buffers
  static constexpr int KST = D == 128 ? 3 : 4;     // K stages
  static constexpr int VST = D == 128 ? 2 : 4;     // V stages
  static constexpr int ST = KST > VST ? KST : VST;
  // Steps whose key masks (and scales) are kept: K of step n is expanded once S of
  // step n - KST is complete, which was issued when the softmax had done with step
  // n - KST - NS.
  static constexpr int MASKS = KST + NS;
  static constexpr uint32_t COL_O = NS * 128;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + 2 * TILE;
  static constexpr int OFF_V = OFF_K + KST * TILE;
  static constexpr int OFF_MASK = OFF_V + VST * TILE;
  // An exponent a row of the tiles in flight: Q of tile g is written when the
  // last S of tile g - 2 is complete, and with tiles of one step the softmax
  // may then still be at tile g - 4 (three score buffers).
  static constexpr int QES = 5;
  // Of 16 keys each, eight to a step: K's scale twice (for pairs of columns), log2 of V's,
  // its inverse.
  static constexpr int SCALES = F::kBlockScales ? 8 * 16 : 0;
  static constexpr int OFF_SCALE = OFF_MASK + MASKS * 16;
  static constexpr int OFF_QE = OFF_SCALE + MASKS * SCALES;
  static constexpr int OFF_BAR = OFF_QE + QES * 128;
  // qfull[2], qempty[2], ofree, fin[2], kfull, kempty, vfull, vempty [ST],
  // sfull, pfull, odone [NS]
  static constexpr int NBAR = 7 + 4 * ST + 3 * NS;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;  // tmem base, abort flag, CTAs, -, units
  static constexpr int OFF_SUMS = OFF_K;           // before the first tile arrives
  static constexpr int OFF_WALK = OFF_MISC + 24;     // a walk for each warp
  static constexpr int USED = OFF_WALK + kWarps * WALK_BYTES;
  static constexpr int MAX_SMEM = 227 * 1024;
  // room to align the base to 1024 bytes, as far as there is any (dynamic shared
  // memory starts aligned when there is no static one; the kernel checks)
  static constexpr int SMEM = USED + 1024 <= MAX_SMEM ? USED + 1024 : MAX_SMEM;
  static_assert(USED <= MAX_SMEM, "shared memory budget");
};
constexpr uint32_t kRegSoftmax = 216, kRegExpand = 104, kRegIssue = 88;
static_assert(128 * (kRegSoftmax + 2 * kRegExpand + kRegIssue) <= kThreads * 128,
              "the register split must fit in what the block is launched with");

// Sum over i in [0, n) of floor((a i + b) / m), for n, a, b >= 0, m > 0, by the
// well-known reduction that goes like Euclid's algorithm on (m, a): whole quotients
// are taken out, and the lattice points below the rest are counted along the other
// axis.
__device__ __noinline__ long long floor_sum(long long n, long long m, long long a, long long b) {
  long long s = 0;
  for (;;) {
    s += (n - 1) * n / 2 * (a / m) + n * (b / m);
    a %= m;
    b %= m;
    const long long top = a * n + b;
    if (top < m) return s;
    n = top / m;
    b = top % m;
    const long long t = m;
    m = a;
    a = t;
  }
}

__device__ __forceinline__ int ceil128(int x) { return (x + 127) >> 7; }

// Tiles of one key head of a sequence (0: the other kernel's, or no queries).
__device__ __forceinline__ int tiles_of(const KvAttn &p, const ManyCtl &c, const Seq &s) {
  if (static_cast<long long>(s.nq) * p.group <= c.tile_rows) return 0;
  return static_cast<int>((static_cast<long long>(s.nq) + c.tokens - 1) / c.tokens);
}

// Units of tile t of n.  A tile that sees no key has one, for its zeros.
__device__ __forceinline__ int tile_units(const KvAttn &p, const ManyCtl &c, const Seq &s, int t,
                                          int n) {
  const long long seen = !p.causal || t == n - 1
                             ? s.nk
                             : static_cast<long long>(s.nk) - s.nq + (t + 1LL) * c.tokens;
  return seen <= 0 ? 1 : ceil128(static_cast<int>(seen));
}

// Units of the first t of n tiles, in closed form (tile x sees nk - nq +
// (x + 1) tokens keys when causal, the last one all).
__device__ __noinline__ long long units_before(const KvAttn &p, const ManyCtl &c, const Seq &s, int t, int n) {
  if (t == 0) return 0;
  const long long full = s.nk > 0 ? ceil128(s.nk) : 1;
  if (!p.causal) return t * full;
  const int m = min(t, n - 1);  // without the last tile
  const long long v0 = static_cast<long long>(s.nk) - s.nq;
  const long long none = v0 < 0 ? min(static_cast<long long>(m), -v0 / c.tokens) : 0;
  long long sum = none + (t == n ? full : 0);
  if (m > none)
    sum += floor_sum(m - none, 128, c.tokens, v0 + (none + 1) * c.tokens + 127);
  return sum;
}

// A CTA's share as a list of parts of tiles.  Every warp walks it by itself, in
// a record of its own in shared memory, which leaves the registers to the
// inner loops.
struct Part {
  int b, h, qt, lo, hi, units;  // steps [lo, hi) of `units`
  Seq s;
};
struct Walk {
  long long left;         // units of the share not yet walked
  int b, h, qt, unit, n;  // n tiles of sequence b
  Seq s;
  Part part;
  int more;
};
static_assert(sizeof(Walk) == WALK_BYTES, "the layout of shared memory counts on it");

// The next part of the warp's walk, for all its lanes (they converge here).
__device__ __forceinline__ bool next_part(const KvAttn &p, const ManyCtl &c, Walk *k, Part &x) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) {
    k->more = k->left > 0;
    if (k->more) {
      while (k->qt >= k->n) {
        if (k->n > 0 && k->h + 1 < p.c.Hk) {
          ++k->h;
        } else {  // another sequence of this kernel follows: units are left
          k->s = load_seq(p, ++k->b);
          k->n = tiles_of(p, c, k->s);
          k->h = 0;
        }
        k->qt = 0;
      }
      const int units = tile_units(p, c, k->s, k->qt, k->n);
      const int hi = static_cast<int>(min(static_cast<long long>(units), k->unit + k->left));
      k->part = Part{k->b, k->h, k->qt, k->unit, hi, units, k->s};
      k->left -= hi - k->unit;
      k->unit = 0;
      ++k->qt;
    }
  }
  __syncwarp();
  x = k->part;
  return k->more != 0;
}

template <typename T, class F>
__global__ void __launch_bounds__(kThreads, 1)
    fa_kv_many_kernel(const __grid_constant__ KvAttn p, const __grid_constant__ ManyCtl ctl,
                       float *ws) {
  constexpr int D = F::D;
  using C = ManyCfg<F>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t sQ = sbase + C::OFF_Q, sK = sbase + C::OFF_K, sV = sbase + C::OFF_V;
  const uint32_t bQfull = sbase + C::OFF_BAR, bQempty = bQfull + 16, bOfree = bQempty + 16;
  const uint32_t bFin = bOfree + 8;                // + 8 * issuer
  const uint32_t bKfull = bFin + 16, bKempty = bKfull + 8 * C::ST;
  const uint32_t bVfull = bKempty + 8 * C::ST, bVempty = bVfull + 8 * C::ST;
  const uint32_t bSfull = bVempty + 8 * C::ST, bPfull = bSfull + 8 * C::NS;
  const uint32_t bOdone = bPfull + 8 * C::NS;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 4);
  int *s_den = reinterpret_cast<int *>(smem + C::OFF_MISC + 8);
  long long *s_total = reinterpret_cast<long long *>(smem + C::OFF_MISC + 16);
  long long *s_sums = reinterpret_cast<long long *>(smem + C::OFF_SUMS);
  auto s_warp = reinterpret_cast<long long (*)[kWarps]>(s_sums + kThreads);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (smem + C::USED > smem_raw + C::SMEM) {  // see ManyCfg::SMEM
    griddep_wait();
    if (threadIdx.x == 0) {
      atomicOr(ctl.status, kStatusSmemLayout);
      reinterpret_cast<Share *>(ws)[blockIdx.x] = Share{0, 0, 0, 0};
    }
    return;
  }

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(bQfull + 8 * s, 64);
      mbar_init(bQempty + 8 * s, 1);
    }
    mbar_init(bOfree, 128);
    mbar_init(bFin, 1);
    mbar_init(bFin + 8, 1);
#pragma unroll
    for (int s = 0; s < C::ST; ++s) {
      mbar_init(bKfull + 8 * s, 128);
      mbar_init(bKempty + 8 * s, 1);
      mbar_init(bVfull + 8 * s, 128);
      mbar_init(bVempty + 8 * s, 1);
    }
#pragma unroll
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(bSfull + 8 * s, 1);
      mbar_init(bPfull + 8 * s, 128);
      mbar_init(bOdone + 8 * s, 1);
    }
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  griddep_wait();
  griddep_launch_dependents();
  // this CTA's share of the line of units
  int den = gridDim.x;
  long long u0 = 0;
  const Place at = find_unit<kWarps>(
      p,
      [&](int b) {
        const Seq s = load_seq(p, b);
        const int n = tiles_of(p, ctl, s);
        return units_before(p, ctl, s, n, n) * p.c.Hk;
      },
      blockIdx.x, &den, &u0, s_sums, s_warp);
  if (threadIdx.x == 0) reinterpret_cast<Share *>(ws)[blockIdx.x] = Share{0, 0, 0, 0};
  if (static_cast<int>(blockIdx.x) >= den) return;
  Walk *walk = reinterpret_cast<Walk *>(smem + C::OFF_WALK) + warp;
  if (lane == 0) {
    Walk k = {};
    k.left = at.total * (blockIdx.x + 1) / den - u0;
    k.b = at.b;
    k.s = load_seq(p, at.b);
    k.n = tiles_of(p, ctl, k.s);
    const long long per_head = units_before(p, ctl, k.s, k.n, k.n);
    const long long into = u0 - at.before;
    k.h = static_cast<int>(into / per_head);
    const long long rest = into - k.h * per_head;
    int lo = 0, hi = k.n;  // the last tile that begins at or before `rest`
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (units_before(p, ctl, k.s, mid, k.n) <= rest) lo = mid;
      else hi = mid;
    }
    k.qt = lo;
    k.unit = static_cast<int>(rest - units_before(p, ctl, k.s, lo, k.n));
    *walk = k;
    if (warp == 0) *s_den = den, *s_total = at.total;
  }
  __syncwarp();  // tcgen05's aligned instructions want the warp together
  if (warp == 12) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  WaitCtl w{abort_flag, ctl.status, ctl.wait_limit_ns, 0u};

  if (warp >= 12) {
    setmaxnreg_dec<kRegIssue>();
    w.role = kStatusMma;
    if (warp == 12) {
      // ---------------------------------------------- S = Q K^T
      constexpr uint32_t kIdesc = make_idesc(0u, 128, 128, 0u, 0u);
      bool ok = true;
      int b = 0, bph = 0, s = 0, sph = 0, issued = 0;
      Part x;
      for (int g = 0; ok && next_part(p, ctl, walk, x); ++g) {
        if (lane == 0) {
          ok = bounded_wait(bQfull + 8 * (g & 1), (g >> 1) & 1, w);
          for (int j = x.lo; ok && j < x.hi; ++j, ++issued) {
            // score buffer b last held P of three steps ago
            if (issued >= C::NS && !(ok = bounded_wait(bOdone + 8 * b, bph ^ 1, w))) break;
            if (!(ok = bounded_wait(bKfull + 8 * s, sph, w))) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = (kk >> 2) * C::CHUNK + (kk & 3) * 32;
              umma_ss<false>(tmem + b * 128, sdesc_sw128(sQ + (g & 1) * C::TILE + off, 16, 1024),
                             sdesc_sw128(sK + s * C::TILE + off, 16, 1024), kIdesc,
                             kk > 0 ? 1u : 0u);
            }
            tc_commit(bKempty + 8 * s);
            tc_commit(bSfull + 8 * b);
            if (++b == C::NS) b = 0, bph ^= 1;
            if (++s == C::KST) s = 0, sph ^= 1;
          }
          if (ok) tc_commit(bQempty + 8 * (g & 1));
        }
        ok = __shfl_sync(~0u, ok, 0);
      }
      if (lane == 0) {
        tc_commit(bFin);
        bounded_wait(bFin, 0, w, false);
      }
    } else if (warp == 13) {
      // ---------------------------------------------- O += P V
      constexpr uint32_t kIdesc = make_idesc(0u, 128, D, 0u, 1u);
      bool ok = true;
      int b = 0, bph = 0, s = 0, sph = 0;
      Part x;
      for (int g = 0; ok && next_part(p, ctl, walk, x); ++g) {
        if (lane == 0) {
          // O of the previous tile has been read
          ok = g == 0 || bounded_wait(bOfree, (g - 1) & 1, w);
          for (int j = x.lo; ok && j < x.hi; ++j) {
            if (!(ok = bounded_wait(bPfull + 8 * b, bph, w))) break;
            if (!(ok = bounded_wait(bVfull + 8 * s, sph, w))) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              umma_ts<false>(tmem + C::COL_O, tmem + b * 128 + kk * 8,
                             sdesc_sw128(sV + s * C::TILE + kk * 16 * 128, C::CHUNK, 1024), kIdesc,
                             (j > x.lo || kk > 0) ? 1u : 0u);
            tc_commit(bVempty + 8 * s);
            tc_commit(bOdone + 8 * b);
            if (++b == C::NS) b = 0, bph ^= 1;
            if (++s == C::VST) s = 0, sph ^= 1;
          }
        }
        ok = __shfl_sync(~0u, ok, 0);
      }
      if (lane == 0) {
        tc_commit(bFin + 8);
        bounded_wait(bFin + 8, 0, w, false);
      }
    } else {
      // ---------------------------------------------- Q rows
      w.role = kStatusProducer;
      // the sign of the scale goes into Q, a zero scale makes Q zero
      const float sign = p.scale_log2 == 0.f ? 0.f : p.scale_log2 < 0.f ? -1.f : 1.f;
      Part x;
      for (int g = 0; next_part(p, ctl, walk, x); ++g) {
        if (!__all_sync(~0u, g < 2 || bounded_wait(bQempty + 8 * (g & 1), ((g >> 1) - 1) & 1, w)))
          break;
        uint8_t *tile = smem + C::OFF_Q + (g & 1) * C::TILE;
#pragma unroll 1
        for (int n = 0; n < 2; ++n) {
          const int r = (threadIdx.x & 63) + 64 * n;
          const int ti = r / p.group, tj = r - ti * p.group, i = x.qt * ctl.tokens + ti;
          const bool in = ti < ctl.tokens && i < x.s.nq;
          float amax = 0.f;
          const uint4 *src = reinterpret_cast<const uint4 *>(
              static_cast<const T *>(p.q) +
              (in ? (static_cast<long long>(x.s.r0 + i) * p.Hq + x.h * p.group + tj) * D : 0));
#pragma unroll 4
          for (int u = 0; u < D / 8; ++u) {
            const uint4 q = in ? __ldg(src + u) : make_uint4(0, 0, 0, 0);
            const T *f = reinterpret_cast<const T *>(&q);
#pragma unroll
            for (int y = 0; y < 8; ++y) amax = fmaxf(amax, fabsf(static_cast<float>(f[y])));
          }
          // 2^e brings the row's largest element to 1 .. 2 (an exact scaling)
          const int e = min(max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -126), 126);
          const float mul = pow2(-e) * sign;
#pragma unroll 4
          for (int u = 0; u < D / 8; ++u) {
            const uint4 q = in ? __ldg(src + u) : make_uint4(0, 0, 0, 0);
            const T *f = reinterpret_cast<const T *>(&q);
            uint4 v;
            v.x = pack_f16x2(static_cast<float>(f[0]) * mul, static_cast<float>(f[1]) * mul);
            v.y = pack_f16x2(static_cast<float>(f[2]) * mul, static_cast<float>(f[3]) * mul);
            v.z = pack_f16x2(static_cast<float>(f[4]) * mul, static_cast<float>(f[5]) * mul);
            v.w = pack_f16x2(static_cast<float>(f[6]) * mul, static_cast<float>(f[7]) * mul);
            *reinterpret_cast<uint4 *>(tile + (u >> 3) * C::CHUNK + r * 128 +
                                       (((u & 7) ^ (r & 7)) << 4)) = v;
          }
          reinterpret_cast<int8_t *>(smem + C::OFF_QE)[g % C::QES * 128 + r] = static_cast<int8_t>(e);
        }
        fence_proxy_async_smem();
        mbar_arrive(bQfull + 8 * (g & 1));
      }
    }
    __syncwarp();
  } else if (warp >= 4) {
    setmaxnreg_dec<kRegExpand>();
    // ------------------------------------------------ codes -> fp16 rows
    w.role = kStatusProducer;
    const bool is_v = warp >= 8;
    const int r = threadIdx.x & 127;  // token of the tile
    const uint8_t *codes = is_v ? p.c.v_codes : p.c.k_codes;
    const uint8_t *scales = is_v ? p.c.v_scales : p.c.k_scales;
    uint8_t *tiles = smem + (is_v ? C::OFF_V : C::OFF_K);
    const uint32_t full = is_v ? bVfull : bKfull, empty = is_v ? bVempty : bKempty;
    bool past = false;
    struct Row : F::Row {
      bool valid, past;  // past: behind the sequence
    };
    auto load = [&](Row &x, long long row) {
      x.valid = row >= 0;
      x.past = past;
      if constexpr (!F::kStreams)
        if (row >= 0) x.load(codes, scales, row);
      if constexpr (F::kBlockScales)
        if (!is_v && (r & 15) == 0) x.load_scales(p.c, row);
    };
    // The cursor runs over the steps of all parts, two ahead of the one that
    // is written: its page is on its way while the step before it is loaded.
    Part x;
    bool have = next_part(p, ctl, walk, x);
    int j = have ? x.lo : 0, id = -1, off = 0, head = 0;
    const int bs = 1 << p.c.bs_log2;
    auto lookup = [&]() {  // the cursor's page, then one step on; whether there was a step
      const bool was = have;
      const int t = j * 128 + r;
      past = t >= x.s.nk;
      id = have && !past
               ? __ldg(p.table + static_cast<long long>(x.b) * p.width + (t >> p.c.bs_log2))
               : -1;
      off = t & (bs - 1);
      head = x.h;
      if (have && ++j >= x.hi) {
        have = next_part(p, ctl, walk, x);
        j = x.lo;
      }
      return was;
    };
    auto row_of = [&]() -> long long {
      if (static_cast<unsigned>(id) >= static_cast<unsigned>(p.c.num_blocks)) return -1;
      return ((static_cast<long long>(id) * p.c.Hk + head) << p.c.bs_log2) + off;
    };
    const int stages = is_v ? C::VST : C::KST;
    Row row;
    bool now = lookup();
    load(row, row_of());
    if constexpr (F::kStreams) row.begin(codes, row_of());
    bool next = lookup();
    for (int step = 0, st = 0, ph = 0; now; ++step) {
      if (is_v && ctl.skip_load && step == 0) {  // test hook: the P V issuer's wait runs out
        if (r == 0) atomicOr(ctl.status, kStatusInjected);
        break;
      }
      if (!__all_sync(~0u, step < stages || bounded_wait(empty + 8 * st, ph ^ 1, w))) break;
      if (!is_v) {
        const unsigned bits = __ballot_sync(~0u, row.valid || row.past);
        if (lane == 0)
          reinterpret_cast<unsigned *>(smem + C::OFF_MASK)[(step % C::MASKS) * 4 + warp - 4] = bits;
        if constexpr (F::kBlockScales)
          if ((r & 15) == 0) {
            const auto x = row.scales();
            reinterpret_cast<float4 *>(smem + C::OFF_SCALE + step % C::MASKS * C::SCALES)[r / 16] =
                make_float4(x.k, x.k, x.v_log, x.v_inv);
          }
      }
      // unit u of a chunk of row y is at u ^ (y & 7)
      uint8_t *tile = tiles + st * C::TILE;
      if constexpr (F::kStreams)
        row.stream(codes, next ? row_of() : -1, tile + (r & ~31) * 128, C::CHUNK);
      else
        row.expand(row.valid, [&](int unit) {
          return reinterpret_cast<uint4 *>(tile + (unit >> 3) * C::CHUNK + r * 128 +
                                           (((unit & 7) ^ (r & 7)) << 4));
        });
      fence_proxy_async_smem();
      mbar_arrive(full + 8 * st);
      if (++st == stages) st = 0, ph ^= 1;
      if (next) load(row, row_of());
      now = next;
      next = next && lookup();
    }
  } else {
    setmaxnreg_inc<kRegSoftmax>();
    // ------------------------------------------------ softmax + epilogue
    w.role = kStatusSoftmax;
    const int r = threadIdx.x;
    const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t o_tm = tmem + lane_off + C::COL_O;
    const int ti = r / p.group, tj = r - ti * p.group;  // token of the tile, head of the group
    const float mag = p.scale_log2 == 0.f ? 1.f : fabsf(p.scale_log2);
    bool ok = true;
    Part x;
    bool have = next_part(p, ctl, walk, x);
    int buf = 0, bph = 0, pbuf = C::NS - 1, pbph = 1, step = 0;
    for (int g = 0; have; ++g) {
      const int i = x.qt * ctl.tokens + ti;
      const bool in = ti < ctl.tokens && i < x.s.nq;
      // keys [0, lim) are this row's
      const int lim = p.causal && in ? x.s.nk - x.s.nq + i + 1 : x.s.nk;
      float sl2 = 0.f, m_used = -INFINITY, l = 0.f;
      for (int j = x.lo; j < x.hi; ++j, ++step) {
        ok = __all_sync(~0u, bounded_wait(bSfull + 8 * buf, bph, w));
        if (!ok) break;
        tc_fence_after();
        const uint32_t s_tm = tmem + lane_off + buf * 128;
        if (j == x.lo)  // written before the Q row that this S read
          sl2 = fmaxf(
              mag * pow2(reinterpret_cast<const int8_t *>(smem + C::OFF_QE)[g % C::QES * 128 + r]), FLT_MIN);
        const uint4 bits = reinterpret_cast<const uint4 *>(smem + C::OFF_MASK)[step % C::MASKS];
        uint32_t sr[4][32];
        const int cut = lim - j * 128;  // columns [0, cut) are seen
        if (__any_sync(~0u, cut < 128 || (bits.x & bits.y & bits.z & bits.w) != ~0u)) {
          // scores that do not count become -inf in tensor memory
#pragma unroll 1
          for (int n = 0; n < 4; ++n) {
            const uint32_t word = n == 0 ? bits.x : n == 1 ? bits.y : n == 2 ? bits.z : bits.w;
            const int c = cut - 32 * n;
            const uint32_t see = word & (c >= 32 ? ~0u : c <= 0 ? 0u : (1u << c) - 1u);
            if (__all_sync(~0u, see == ~0u)) continue;
            tmem_ld32(s_tm + 32 * n, sr[0]);
            tmem_ld_wait();
            reg_fence32(sr[0]);
#pragma unroll
            for (int y = 0; y < 32; ++y)
              if (!(see >> y & 1)) sr[0][y] = 0xff800000u;
            tmem_st32(s_tm + 32 * n, sr[0]);
          }
          tmem_st_wait();
        }
        tmem_ld32(s_tm + 0, sr[0]);
        tmem_ld32(s_tm + 32, sr[1]);
        tmem_ld32(s_tm + 64, sr[2]);
        tmem_ld32(s_tm + 96, sr[3]);
        tmem_ld_wait();
        reg_fence32(sr[0]);
        reg_fence32(sr[1]);
        reg_fence32(sr[2]);
        reg_fence32(sr[3]);
        auto S = [&](int c) -> float { return __uint_as_float(sr[c >> 5][c & 31]); };
        // The offset moves only when a row's maximum grows by more than kGrow.
        // P is formed with the offset at hand; a row sum of at most 2^15 proves
        // that no term is above it.  A tile's first step, and rows that have
        // seen nothing yet, take the maximum first.
        constexpr float kSumLimit = 32768.f;
        bool with_max = __any_sync(~0u, m_used == -INFINITY), formed = false;
        float tsum = 0.f;  // (of the weights without their values' scales)
        // of columns 16 n and on: the scores' factor, twice (positive, for the -inf of a masked
        // one), log2 of V's scale, its inverse
        auto scale_at = [&](int n) {
          return reinterpret_cast<const ulonglong2 *>(smem + C::OFF_SCALE +
                                                      step % C::MASKS * C::SCALES)[n];
        };
        auto factor = [&](uint64_t k) {
          return ffma2(k, pk2(sl2, sl2), pk2(FLT_MIN, FLT_MIN));
        };
        for (;;) {
          if (with_max) {
            float part[8];
#pragma unroll
            for (int n = 0; n < 8; ++n) part[n] = -INFINITY;
#pragma unroll
            for (int c = 0; c < 128; c += 2) {
              const int n = F::kBlockScales ? c / 16 : (c >> 1) & 7;
              part[n] = max3f(part[n], S(c), S(c + 1));
            }
            if constexpr (F::kBlockScales) {
#pragma unroll
              for (int n = 0; n < 8; ++n) {
                const ulonglong2 x = scale_at(n);
                float by, log, unused;
                upk2(factor(x.x), by, unused);
                upk2(x.y, log, unused);
                part[n] = fmaf(part[n], by, log);
              }
            }
            const float mx = max3f(max3f(part[0], part[1], part[2]),
                                   max3f(part[3], part[4], part[5]), fmaxf(part[6], part[7]));
            const float m_new =
                fmaxf(m_used, F::kBlockScales ? mx - kHeadroom : fmaf(mx, sl2, -kHeadroom));
            if (j == x.lo) {
              m_used = m_new;
            } else {
              const bool need = m_new - m_used > kGrow;  // false for -inf - -inf
              const bool move = __any_sync(~0u, need);
              if (formed && !move) break;  // P and its sum stand
              if (move) {
                // O is rescaled once the last product into it has completed
                ok = __all_sync(~0u, bounded_wait(bOdone + 8 * pbuf, pbph, w));
                if (!ok) break;
                tc_fence_after();
                const float alpha = need ? ex2_approx(m_used - m_new) : 1.f;
                const uint64_t a2 = pk2(alpha, alpha);
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                  uint32_t o[32];
                  tmem_ld32(o_tm + c, o);
                  tmem_ld_wait();
                  reg_fence32(o);
#pragma unroll
                  for (int n = 0; n < 32; n += 2) {
                    float lo, hi;
                    upk2(fmul2(pk2(__uint_as_float(o[n]), __uint_as_float(o[n + 1])), a2), lo, hi);
                    o[n] = __float_as_uint(lo);
                    o[n + 1] = __float_as_uint(hi);
                  }
                  tmem_st32(o_tm + c, o);
                }
                tmem_st_wait();
                if (need) {
                  l *= alpha;
                  m_used = m_new;
                }
                __syncwarp();  // ahead of P's stores
              }
            }
          }
          const float off = m_used == -INFINITY ? 0.f : -m_used;
          uint64_t sl2_2 = pk2(sl2, sl2), nm_2 = pk2(off, off);
          uint64_t acc[2] = {0ull, 0ull};
          // with scales: those of the next columns, loaded ahead; the weights' factor in the
          // sum, and the least such factor, which bounds the weights by the sum
          ulonglong2 ahead = {};
          uint64_t inv_2 = 0ull;
          float least = F::kBlockScales ? INFINITY : 1.f;
          if constexpr (F::kBlockScales) ahead = scale_at(0);
#pragma unroll
          for (int blk = 0; blk < 2; ++blk) {
            uint32_t pk[32];
#pragma unroll
            for (int n = 0; n < 32; ++n) {
              const int c0 = 2 * (blk * 32 + n);
              if (F::kBlockScales && n % 8 == 0) {
                float log, inv;
                upk2(ahead.y, log, inv);
                sl2_2 = factor(ahead.x);
                nm_2 = pk2(log + off, log + off);
                inv_2 = pk2(inv, inv);
                least = fminf(least, inv);
                if (c0 < 112) ahead = scale_at(c0 / 16 + 1);
              }
              float x0, x1;
              upk2(ffma2(pk2(S(c0), S(c0 + 1)), sl2_2, nm_2), x0, x1);
              const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
              acc[n & 1] = F::kBlockScales ? ffma2(pk2(p0, p1), inv_2, acc[n & 1])
                                           : fadd2(acc[n & 1], pk2(p0, p1));
              pk[n] = pack_f16x2(p0, p1);
            }
            tmem_st32(s_tm + blk * 32, pk);
          }
          float a0, a1, b0, b1;
          upk2(acc[0], a0, a1);
          upk2(acc[1], b0, b1);
          tsum = (a0 + a1) + (b0 + b1);
          if (with_max || __all_sync(~0u, tsum <= kSumLimit * least)) break;
          with_max = formed = true;
          tmem_st_wait();  // the second pass rewrites the same columns
        }
        if (!ok) break;
        l += tsum;
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bPfull + 8 * buf);
        pbuf = buf;
        pbph = bph;
        if (++buf == C::NS) buf = 0, bph ^= 1;
      }
      if (ok) ok = __all_sync(~0u, bounded_wait(bOdone + 8 * pbuf, pbph, w));
      if (ok) {
        tc_fence_after();
        const bool begins = x.lo == 0, ends = x.hi == x.units;
        if (r == 0 && begins && !ends) {
          // the CTA with the tile's last step: `units` from its first on
          const long long end = *s_total * (blockIdx.x + 1) / *s_den - walk->left - x.hi + x.units;
          reinterpret_cast<Share *>(ws)[blockIdx.x] =
              Share{x.s.r0 + x.qt * ctl.tokens, x.h,
                    min(x.s.nq - x.qt * ctl.tokens, ctl.tokens) * p.group,
                    cta_of(end - 1, *s_total, *s_den)};
        }
        const bool whole = begins && ends;
        // 32 bytes a store, as rows lie far apart: 16 took 454 us instead of then 451 for
        // the two chunks above, 525 instead of 516 for 8 prompts of 2048
        const bool wide = reinterpret_cast<uintptr_t>(p.o) % 32 == 0;
        const float inv = p.v_mul / l;
        const int head = x.h * p.group + tj;
        T *out = static_cast<T *>(p.o) +
                 (in ? (static_cast<long long>(x.s.r0 + i) * p.Hq + head) * D : 0);
        float *part = part_of<D, R>(ws, blockIdx.x, begins);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          alignas(32) uint32_t o[32];
          __syncwarp();  // rows without a query left the loop's last turn early
          tmem_ld32(o_tm + c, o);
          tmem_ld_wait();
          reg_fence32(o);
          if (!in) continue;
          if (whole) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              alignas(32) T e[16];
#pragma unroll
              for (int y = 0; y < 16; ++y)
                e[y] = static_cast<T>(value_of(__uint_as_float(o[16 * u + y]), l, inv));
              if (wide) {
                store32(out + c + 16 * u, *reinterpret_cast<const B32 *>(e));
              } else {
                reinterpret_cast<uint4 *>(out + c)[2 * u] = reinterpret_cast<const uint4 *>(e)[0];
                reinterpret_cast<uint4 *>(out + c)[2 * u + 1] = reinterpret_cast<const uint4 *>(e)[1];
              }
            }
          } else {
#pragma unroll
            for (int u = 0; u < 4; ++u)
              store32(part + r * D + c + 8 * u, *reinterpret_cast<const B32 *>(o + 8 * u));
          }
        }
        if (in && whole)
          p.lse[static_cast<long long>(head) * p.total_q + x.s.r0 + i] = lse_of(m_used, l);
        if (in && !whole)
          reinterpret_cast<float2 *>(part + R * D)[r] = make_float2(m_used, l);
        tc_fence_before();
        mbar_arrive(bOfree);
      }
      // the four warps take one decision to go on or stop
      if (named_bar_or(1, 128, !ok || *abort_flag != 0)) break;
      have = next_part(p, ctl, walk, x);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <typename T, class F>
cudaError_t launch_many(const KvAttn &p, const ManyCtl &ctl, float *ws, int ctas, cudaStream_t s) {
  static std::atomic<unsigned long long> attr_done{0};
  constexpr int smem = ManyCfg<F>::SMEM;
  cudaError_t e = smem_attr_once(fa_kv_many_kernel<T, F>, smem, &attr_done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, fa_kv_many_kernel<T, F>, p, ctl, ws);
  if (e != cudaSuccess || ctas == 1) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(ctas - 1), R / kJoinRows);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, fa_kv_join_kernel<T, F::D, R>, p, ws);
}

}  // namespace
}  // namespace fa
