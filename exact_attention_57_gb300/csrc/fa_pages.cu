// fa_pages.cu — pages of a paged cache: copied, forked with their requests,
// collected and compacted.
//
// Which blocks are held stands in the block tables alone: nothing counts
// references.  A call that wants to know marks the blocks of all rows in a bit map
// (a set, so blocks that rows share and rows that are listed twice make no
// difference) and sweeps it, so every output is a function of the inputs and in
// ascending order.  The bit map lies in the shared memory of one cluster of up to
// eight CTAs (2^23 blocks at most), whose CTAs each own a range of blocks and set
// bits in one another's memory: one launch, no workspace to clear, no grid-wide
// wait.
//
// Pages are copied by items of 16 KB dealt to the CTAs of one wave, 64 bytes in flight
// a thread.  In captured graphs, pages of 8 heads of 128 and 64 tokens: 938 of a 4-bit
// cache take 23.0 us, 6.0 TB/s or 89% of the copy rate; forking 64 requests into 256 (256
// pages of an 8-bit cache, of 64) 12.6, of 6.2 that the bytes need, and listing what is free
// then (256 rows of 128 entries) 7.8, one cluster's chain of dependent steps: marks,
// counts, lists.  Compacting 32 requests of up to 8192 tokens takes 49.6 us, 42.7 by its
// bytes, about 6 of it the plan ahead of the copies.  Nine small pages: 1.6 us.
#include <atomic>
#include <cstdint>

#include "fa_internal.h"
#include "fa_serve.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int kPiece = 16384;  // bytes of a page that a CTA copies at a time

// The arrays of a cache as a kernel gets them.
template <int kMax>
struct PageArgs {
  const void *from[kMax];
  void *to[kMax];
  unsigned long long bytes[kMax];  // of a page
  int first[kMax + 1];             // pieces of a page before this array's
  int num;
};
template <int kMax>
PageArgs<kMax> page_args(const Pages &p) {
  PageArgs<kMax> a;
  a.num = p.num;
  a.first[0] = 0;
  for (int i = 0; i < p.num; ++i) {
    a.from[i] = p.from[i];
    a.to[i] = p.to[i];
    a.bytes[i] = p.bytes[i];
    a.first[i + 1] = a.first[i] + static_cast<int>((p.bytes[i] + kPiece - 1) / kPiece);
  }
  return a;
}

// `n` bytes by the whole CTA, by the widest accesses that the addresses allow.
__device__ __forceinline__ void copy_bytes(const uint8_t *src, uint8_t *dst, int n) {
  const int tid = threadIdx.x;
  const uintptr_t low = reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst) |
                        static_cast<uintptr_t>(n);
  if (low % 16 == 0) {
    constexpr int kAt = kPiece / 16 / kThreads;
    uint4 x[kAt];
    const uint4 *s = reinterpret_cast<const uint4 *>(src);
    uint4 *d = reinterpret_cast<uint4 *>(dst);
    n /= 16;
#pragma unroll
    for (int i = 0; i < kAt; ++i)
      if (tid + i * kThreads < n) x[i] = s[tid + i * kThreads];
#pragma unroll
    for (int i = 0; i < kAt; ++i)
      if (tid + i * kThreads < n) d[tid + i * kThreads] = x[i];
  } else if (low % 4 == 0) {
    for (int i = tid; i < n / 4; i += kThreads)
      reinterpret_cast<uint32_t *>(dst)[i] = reinterpret_cast<const uint32_t *>(src)[i];
  } else {
    for (int i = tid; i < n; i += kThreads) dst[i] = src[i];
  }
}

// Piece `piece` of page `from` to page `to`, by the whole CTA.
template <int kMax>
__device__ __forceinline__ void copy_piece(const PageArgs<kMax> &a, int from, int to, int piece) {
  int lo = 0, hi = a.num;  // the last array that begins at or before it
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.first[mid] <= piece) lo = mid;
    else hi = mid;
  }
  const unsigned long long at = static_cast<unsigned long long>(piece - a.first[lo]) * kPiece;
  const unsigned long long left = a.bytes[lo] - at;
  const unsigned long long page = a.bytes[lo];
  copy_bytes(static_cast<const uint8_t *>(a.from[lo]) + from * page + at,
             static_cast<uint8_t *>(a.to[lo]) + to * page + at,
             left < kPiece ? static_cast<int>(left) : kPiece);
}

__device__ __forceinline__ bool in_range(int id, int blocks) {
  return static_cast<unsigned>(id) < static_cast<unsigned>(blocks);
}

// Blocks that a row of `width` entries needs for `len` tokens.
__device__ __forceinline__ int blocks_of(int len, int width, int bs_log2) {
  const long long n = (static_cast<long long>(max(len, 0)) + (1 << bs_log2) - 1) >> bs_log2;
  return static_cast<int>(min(n, static_cast<long long>(width)));
}

// ------------------------------------------------------------------ copy
// Pages src[i] -> dst[i]; with a count, as many as that says.
template <int kMax>
__global__ void __launch_bounds__(kThreads)
    fa_kv_copy_kernel(const __grid_constant__ PageArgs<kMax> a, const int *src, const int *dst, int n,
                      int from_blocks, int to_blocks) {
  griddep_wait();
  griddep_launch_dependents();
  const int pieces = a.first[a.num];
  const long long items = static_cast<long long>(n) * pieces;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int i = static_cast<int>(it / pieces), piece = static_cast<int>(it - static_cast<long long>(i) * pieces);
    const int from = __ldg(src + i), to = __ldg(dst + i);
    if (in_range(from, from_blocks) && in_range(to, to_blocks)) copy_piece(a, from, to, piece);
  }
}

// ------------------------------------------------------------------ fork
// Every CTA plans all children, 256 at a time (a scan over who needs a block),
// instead of waiting for another kernel to do it, and takes its share of the
// round's items: per child one for its row of the table and the pieces of its page.
template <int kMax>
__global__ void __launch_bounds__(kThreads)
    fa_kv_fork_kernel(const __grid_constant__ PageArgs<kMax> a, const ForkParams p) {
  constexpr int kWarps = kThreads / 32;
  __shared__ int s_parent[kThreads], s_len[kThreads], s_src[kThreads], s_last[kThreads];
  __shared__ int s_sum[kWarps];
  __shared__ unsigned s_seen[65536 / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_wait();
  griddep_launch_dependents();
  const long long head = p.free_head ? max(0, __ldg(p.free_head)) : 0;
  const int mask = (1 << p.bs_log2) - 1;
  const long long reach = static_cast<long long>(p.width) << p.bs_log2;
  const int pieces = a.num ? a.first[a.num] : 0, per = pieces + 1;
  if (p.parents_end)
    for (int i = tid; i < 65536 / 32; i += kThreads) s_seen[i] = 0;
  long long used = 0;  // blocks taken by the rounds so far
  for (int base = 0; base < p.n; base += kThreads) {
    __syncthreads();  // the round before has been read
    const int i = base + tid;
    int parent = i < p.n ? __ldg(p.parents + i) : -1;
    if (!in_range(parent, p.B)) parent = -1;
    const int len = parent >= 0
                        ? static_cast<int>(min(static_cast<long long>(max(__ldg(p.lens + parent), 0)), reach))
                        : 0;
    const bool part = (len & mask) != 0;
    const int src = part ? __ldg(p.table + static_cast<long long>(parent) * p.width + (len >> p.bs_log2)) : -1;
    bool takes = false;
    if (p.parents_end) {  // a parent's first child takes its last block over
      for (int w = 0; w < kWarps; ++w) {
        if (w == warp) {
          const unsigned same = __match_any_sync(~0u, parent);
          const bool lowest = __ffs(same) - 1 == lane;
          takes = lowest && parent >= 0 && !(s_seen[parent / 32] >> (parent & 31) & 1);
          __syncwarp();
          if (takes) atomicOr(&s_seen[parent / 32], 1u << (parent & 31));
        }
        __syncthreads();
      }
    }
    const bool need = part && !takes && in_range(src, p.num_blocks);
    const unsigned who = __ballot_sync(~0u, need);
    if (lane == 0) s_sum[warp] = __popc(who);
    __syncthreads();
    int before = __popc(who & ((1u << lane) - 1u)), all = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += s_sum[w];
      all += s_sum[w];
    }
    int fresh = -1;
    if (need) {
      const long long at = head + used + before;
      if (at < p.num_free) fresh = __ldg(p.free_blocks + at);
      if (!in_range(fresh, p.num_blocks)) fresh = -1;
    }
    s_parent[tid] = parent;
    s_len[tid] = len;
    s_src[tid] = fresh >= 0 ? src : -1;  // to copy
    s_last[tid] = need ? fresh : takes && part ? src : -1;
    used += all;
    __syncthreads();
    const int here = min(kThreads, p.n - base);
    for (long long it = blockIdx.x; it < static_cast<long long>(here) * per; it += gridDim.x) {
      const int y = static_cast<int>(it / per), piece = static_cast<int>(it - static_cast<long long>(y) * per) - 1;
      if (piece >= 0) {
        if (s_src[y] >= 0) copy_piece(a, s_src[y], s_last[y], piece);
        continue;
      }
      const int full = s_len[y] >> p.bs_log2;
      const bool more = (s_len[y] & mask) != 0;
      const int *row = p.table + static_cast<long long>(max(s_parent[y], 0)) * p.width;
      int *out = p.table_out + static_cast<long long>(base + y) * p.width;
      for (int j = tid; j < p.width; j += kThreads)
        out[j] = j < full ? __ldg(row + j) : j == full && more ? s_last[y] : -1;
      if (tid == 0) p.lens_out[base + y] = s_len[y];
    }
  }
  if (blockIdx.x == 0 && tid == 0) {
    p.counts[0] = static_cast<int>(used);
    p.counts[1] = static_cast<int>(min(head + used, static_cast<long long>(max(p.num_free, 0))));
  }
}

// ------------------------------------------------------------------ mark and sweep
constexpr int kSweepThreads = 1024, kSweepWarps = kSweepThreads / 32;

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
               "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, int rank) {
  uint32_t y;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(y) : "r"(addr), "r"(rank));
  return y;
}
__device__ __forceinline__ void cluster_or(uint32_t addr, unsigned x) {
  asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(addr), "r"(x) : "memory");
}
__device__ __forceinline__ int cluster_load(uint32_t addr) {
  int x;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x) : "r"(addr) : "memory");
  return x;
}

// What the CTAs of a cluster tell one another.
struct SweepShared {
  int held;                 // blocks held in this CTA's range
  int warp_held[kSweepWarps];
  int free_below;           // unheld ids below the number held, in this CTA's range
};

// Marks the blocks that the rows hold.  words: of this CTA's range, zero before.
template <int CL>
__device__ void mark(const int *table, const int *lens, const unsigned char *ended, int B, int width,
                     int bs_log2, int num_blocks, unsigned *words, int per_cta) {
  const int rank = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kSeg = 256;  // entries of a warp's item
  const int segs = (width + kSeg - 1) / kSeg;
  const uint32_t mine = smem_u32(words);
  const long long items = static_cast<long long>(B) * segs;
  for (long long it = static_cast<long long>(warp) * CL + rank; it < items; it += CL * kSweepWarps) {
    const int b = static_cast<int>(it / segs), s = static_cast<int>(it - static_cast<long long>(b) * segs);
    if (ended && __ldg(ended + b)) continue;
    const int need = blocks_of(__ldg(lens + b), width, bs_log2);
    const int *row = table + static_cast<long long>(b) * width;
    int id[kSeg / 32];
#pragma unroll
    for (int n = 0; n < kSeg / 32; ++n) {
      const int j = s * kSeg + n * 32 + lane;
      id[n] = j < need ? __ldg(row + j) : -1;
    }
#pragma unroll
    for (int n = 0; n < kSeg / 32; ++n) {
      if (!in_range(id[n], num_blocks)) continue;
      const int w = id[n] / 32;
      if constexpr (CL == 1) {
        atomicOr(words + w, 1u << (id[n] & 31));
      } else {
        const int owner = w / per_cta;
        cluster_or(cluster_addr(mine + (w - owner * per_cta) * 4, owner), 1u << (id[n] & 31));
      }
    }
  }
}

template <int CL>
__device__ __forceinline__ void all_meet() {
  if constexpr (CL == 1) {
    __syncthreads();
  } else {
    __syncwarp();
    cluster_barrier();
  }
}

// The words of a warp: [lo, hi) of its CTA's per_cta.
struct Words {
  int lo, hi;
};
__device__ __forceinline__ Words words_of(int per_cta) {
  const int warp = threadIdx.x >> 5, chunk = (per_cta + kSweepWarps - 1) / kSweepWarps;
  return {min(warp * chunk, per_cta), min((warp + 1) * chunk, per_cta)};
}

// Counts the blocks held: of this warp's words into s->warp_held, of the CTA into
// s->held; *before: held in the ranges of the CTAs and warps before this warp's,
// *total: in all.
template <int CL>
__device__ void count_held(const unsigned *words, int per_cta, SweepShared *s, int *before, int *total) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Words mine = words_of(per_cta);
  int n = 0;
  for (int w = mine.lo + lane; w < mine.hi; w += 32) n += __popc(words[w]);
  for (int o = 16; o; o /= 2) n += __shfl_xor_sync(~0u, n, o);
  if (lane == 0) s->warp_held[warp] = n;
  __syncthreads();
  int all = s->warp_held[lane], pre = lane < warp ? all : 0;
  for (int o = 16; o; o /= 2) {
    all += __shfl_xor_sync(~0u, all, o);
    pre += __shfl_xor_sync(~0u, pre, o);
  }
  if constexpr (CL == 1) {
    *before = pre;
    *total = all;
  } else {
    if (tid == 0) s->held = all;
    all_meet<CL>();
    const uint32_t at = smem_u32(&s->held);
    *total = 0;
    for (int c = 0; c < CL; ++c) {
      const int x = cluster_load(cluster_addr(at, c));
      if (c < static_cast<int>(blockIdx.x)) pre += x;
      *total += x;
    }
    *before = pre;
  }
}

// The list of all blocks that no row holds, ascending, at the end of free_blocks.
template <int CL>
__global__ void __launch_bounds__(kSweepThreads, 1) fa_kv_free_kernel(const FreeParams p, int per_cta) {
  extern __shared__ unsigned words[];
  __shared__ SweepShared s;
  const int tid = threadIdx.x, lane = tid & 31, rank = blockIdx.x;
  for (int w = tid; w < per_cta; w += kSweepThreads) words[w] = 0;
  griddep_wait();
  griddep_launch_dependents();
  all_meet<CL>();
  mark<CL>(p.table, p.lens, p.ended, p.B, p.width, p.bs_log2, p.num_blocks, words, per_cta);
  all_meet<CL>();
  int before, held;
  count_held<CL>(words, per_cta, &s, &before, &held);
  const Words mine = words_of(per_cta);
  for (int w = mine.lo; w < mine.hi; ++w) {
    const unsigned bits = words[w];
    const int id = (rank * per_cta + w) * 32 + lane;
    const int below = before + __popc(bits & ((1u << lane) - 1u));  // held ids below this one
    if (id < p.num_blocks && !(bits >> lane & 1)) p.free_blocks[held + id - below] = id;
    before += __popc(bits);
  }
  for (int i = rank * kSweepThreads + tid; i < held; i += CL * kSweepThreads) p.free_blocks[i] = -1;
  if (rank == 0 && tid == 0) *p.free_head = held;
  if (p.ended)
    for (int b = rank * kSweepThreads + tid; b < p.B; b += CL * kSweepThreads)
      if (p.ended[b]) p.lens[b] = 0;
  if constexpr (CL > 1) all_meet<CL>();  // the others may still read this CTA's count
}

// Which page goes where: the k-th held id from `held` on to the k-th unheld one
// below it.  moves: sources, then, half the blocks further, destinations.
template <int CL>
__global__ void __launch_bounds__(kSweepThreads, 1) fa_kv_compact_kernel(const CompactParams p, int per_cta) {
  extern __shared__ unsigned words[];
  __shared__ SweepShared s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = blockIdx.x;
  for (int w = tid; w < per_cta; w += kSweepThreads) words[w] = 0;
  griddep_wait();
  griddep_launch_dependents();
  all_meet<CL>();
  mark<CL>(p.table, p.lens, nullptr, p.B, p.width, p.bs_log2, p.num_blocks, words, per_cta);
  all_meet<CL>();
  int before, held;
  count_held<CL>(words, per_cta, &s, &before, &held);
  const Words mine = words_of(per_cta);
  int *src = p.moves, *dst = p.moves + p.num_blocks / 2;
  // unheld ids below `held` of this warp, this CTA, all: as many as pages move
  int n = 0;
  for (int w = mine.lo + lane; w < mine.hi; w += 32) {
    const int id = (rank * per_cta + w) * 32;
    const int inside = min(max(held - id, 0), 32);
    n += __popc(~words[w] & (inside == 32 ? ~0u : (1u << inside) - 1u));
  }
  for (int o = 16; o; o /= 2) n += __shfl_xor_sync(~0u, n, o);
  __syncthreads();  // warp_held has been read
  if (lane == 0) s.warp_held[warp] = n;
  __syncthreads();
  int moved = s.warp_held[lane];
  for (int o = 16; o; o /= 2) moved += __shfl_xor_sync(~0u, moved, o);
  if constexpr (CL > 1) {
    if (tid == 0) s.free_below = moved;
    all_meet<CL>();
    moved = 0;
    for (int c = 0; c < CL; ++c) moved += cluster_load(cluster_addr(smem_u32(&s.free_below), c));
  }
  int run = before;
  for (int w = mine.lo; w < mine.hi; ++w) {
    const unsigned bits = words[w];
    const int id = (rank * per_cta + w) * 32 + lane;
    const int below = run + __popc(bits & ((1u << lane) - 1u));  // held ids below this one
    run += __popc(bits);
    if (id >= p.num_blocks) continue;
    if (!(bits >> lane & 1)) {
      p.new_ids[id] = -1;
      if (id < held) dst[id - below] = id;
    } else if (id < held) {
      p.new_ids[id] = id;
    } else {
      src[below - (held - moved)] = id;
    }
  }
  all_meet<CL>();
  for (int k = rank * kSweepThreads + tid; k < moved; k += CL * kSweepThreads) p.new_ids[src[k]] = dst[k];
  if (rank == 0 && tid == 0) {
    p.counts[0] = held;
    p.counts[1] = moved;
  }
  if constexpr (CL > 1) all_meet<CL>();
}

// The pages' way, and the tables under the new ids.
template <int kMax>
__global__ void __launch_bounds__(kThreads)
    fa_kv_move_kernel(const __grid_constant__ PageArgs<kMax> a, const CompactParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int pieces = a.num ? a.first[a.num] : 0;
  const int *src = p.moves, *dst = p.moves + p.num_blocks / 2;
  const long long items = static_cast<long long>(p.counts[1]) * pieces + p.B;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    if (it >= p.B) {
      const long long x = it - p.B;
      const int i = static_cast<int>(x / pieces);
      copy_piece(a, src[i], dst[i], static_cast<int>(x - static_cast<long long>(i) * pieces));
      continue;
    }
    const int b = static_cast<int>(it), need = blocks_of(p.lens[b], p.width, p.bs_log2);
    const int *row = p.table + static_cast<long long>(b) * p.width;
    int *out = p.table_out + static_cast<long long>(b) * p.width;
    for (int j = threadIdx.x; j < p.width; j += kThreads) {
      const int id = j < need ? row[j] : -1;
      out[j] = in_range(id, p.num_blocks) ? p.new_ids[id] : -1;
    }
  }
}

template <typename... K, typename... A>
cudaError_t launch(void (*kern)(K...), int ctas, int threads, int smem, int cluster, cudaStream_t s,
                   const A &...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// CTAs for so many items: up to four on each SM.
int ctas_for(long long items, int num_sms) {
  const long long most = 4LL * (num_sms < 1 ? 1 : num_sms);
  return static_cast<int>(items < 1 ? 1 : items < most ? items : most);
}

int pieces_of(const Pages &p) {
  int n = 0;
  for (int i = 0; i < p.num; ++i) n += static_cast<int>((p.bytes[i] + kPiece - 1) / kPiece);
  return n;
}

// Up to so many arrays go to a kernel as a short list (of parameters that every launch
// carries), more as one of kMaxArrays.
constexpr int kFewArrays = 8;

// A cluster of eight where the marking or the sweeping is long.  Entries of the table, blocks,
// and the us of fa_kv_free and of fa_kv_compact (tables alone) with one CTA and with eight,
// in captured graphs:
//      512     600   2.4  4.7    4.2  8.0        512   32768   4.8  7.7    4.7  8.3
//     4096    8192   3.4  6.4    4.7  8.6        512   65536   7.3 11.1    4.9  8.6
//     8192    8192   4.1  7.1    5.1  8.9        512  131072  12.3 16.4    5.7  9.8
//    16384   16384   5.1  8.9    5.9  9.9      32768   65536  13.5 23.4    8.4 13.3
//    32768   16384   9.6 12.9    7.8 11.4      32768  262144  27.7 52.0    9.7 16.6
// Two and four CTAs are behind one of the others in nearly all of these (at 16384 entries
// 7.6 12.5 and 6.6 10.8, at 65536 blocks 6.3 10.4 and 5.2 9.0).
int sweep_cluster(int B, int width, int num_blocks) {
  return static_cast<long long>(B) * width > 8192 || num_blocks > 32768 ? 8 : 1;
}
int words_per_cta(int num_blocks, int cluster) {
  const int words = (num_blocks + 31) / 32;
  return (words + cluster - 1) / cluster;
}

// What a kernel may ask for is a property of the kernel, not of a launch, and other
// threads launch it for caches of other sizes: the most that any of them needs.
constexpr int kSweepSmem = kMaxSweep / 32 / 8 * 4;

}  // namespace

cudaError_t launch_kv_copy(const Pages &pages, const int *src, const int *dst, int n, int from_blocks,
                           int to_blocks, int num_sms, cudaStream_t s) {
  const int ctas = ctas_for(static_cast<long long>(n) * pieces_of(pages), num_sms);
  if (pages.num <= kFewArrays)
    return launch(fa_kv_copy_kernel<kFewArrays>, ctas, kThreads, 0, 1, s, page_args<kFewArrays>(pages),
                  src, dst, n, from_blocks, to_blocks);
  return launch(fa_kv_copy_kernel<kMaxArrays>, ctas, kThreads, 0, 1, s, page_args<kMaxArrays>(pages),
                src, dst, n, from_blocks, to_blocks);
}

cudaError_t launch_kv_fork(const Pages &pages, const ForkParams &p, int num_sms, cudaStream_t s) {
  const int here = p.n < kThreads ? p.n : kThreads;
  const int ctas = ctas_for(static_cast<long long>(here) * (pieces_of(pages) + 1), num_sms);
  if (pages.num <= kFewArrays)
    return launch(fa_kv_fork_kernel<kFewArrays>, ctas, kThreads, 0, 1, s, page_args<kFewArrays>(pages), p);
  return launch(fa_kv_fork_kernel<kMaxArrays>, ctas, kThreads, 0, 1, s, page_args<kMaxArrays>(pages), p);
}

cudaError_t launch_kv_free(const FreeParams &p, cudaStream_t s) {
  const int cl = sweep_cluster(p.B, p.width, p.num_blocks);
  const int per_cta = words_per_cta(p.num_blocks, cl), smem = per_cta * 4;
  if (cl == 1) return launch(fa_kv_free_kernel<1>, 1, kSweepThreads, smem, 1, s, p, per_cta);
  static std::atomic<unsigned long long> attr_done{0};
  const cudaError_t e = smem_attr_once(fa_kv_free_kernel<8>, kSweepSmem, &attr_done);
  return e != cudaSuccess ? e : launch(fa_kv_free_kernel<8>, 8, kSweepThreads, smem, 8, s, p, per_cta);
}

cudaError_t launch_kv_compact(const Pages &pages, const CompactParams &p, int num_sms, cudaStream_t s) {
  const int cl = sweep_cluster(p.B, p.width, p.num_blocks);
  const int per_cta = words_per_cta(p.num_blocks, cl), smem = per_cta * 4;
  cudaError_t e = cudaSuccess;
  if (cl == 1) {
    e = launch(fa_kv_compact_kernel<1>, 1, kSweepThreads, smem, 1, s, p, per_cta);
  } else {
    static std::atomic<unsigned long long> attr_done{0};
    e = smem_attr_once(fa_kv_compact_kernel<8>, kSweepSmem, &attr_done);
    if (e == cudaSuccess) e = launch(fa_kv_compact_kernel<8>, 8, kSweepThreads, smem, 8, s, p, per_cta);
  }
  if (e != cudaSuccess) return e;
  const int ctas = ctas_for(static_cast<long long>(p.num_blocks / 2) * pieces_of(pages) + p.B, num_sms);
  if (pages.num <= kFewArrays)
    return launch(fa_kv_move_kernel<kFewArrays>, ctas, kThreads, 0, 1, s, page_args<kFewArrays>(pages), p);
  return launch(fa_kv_move_kernel<kMaxArrays>, ctas, kThreads, 0, 1, s, page_args<kMaxArrays>(pages), p);
}

}  // namespace fa
