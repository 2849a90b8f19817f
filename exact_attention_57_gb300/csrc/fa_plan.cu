// fa_plan.cu — block tables and slot maps of a paged cache from request
// lengths, in one launch.
//
// With have_b = ceil(cached_b / bs), tot_b = ceil((cached_b + new_b) / bs):
// request b takes tot_b - have_b blocks of the free list behind those of the
// requests before it, table[b][have_b + j] = free[head + off_b + j], and its
// i-th new token sits at position p = cached_b + i in slot
// table[b][p / bs] * bs + p % bs.  off_b and the token offsets cu_b are prefix
// sums over the requests.
//
// Every CTA makes the prefix sums itself, 256 or 1024 requests at a time in shared
// memory, instead of waiting for a scan kernel: at the few hundred requests of
// a server that is one round of two loads a thread and a scan, less than a
// second launch.  CTA c owns kTokens token slots (it finds each one's request
// by bisection in the prefix sums at hand), and the requests of every
// gridDim-th round (their lengths and offsets).  A token whose block is new reads
// the free list, not the table, so no CTA waits for another's table entries, and
// the first token of a new block writes its entry; those of blocks whose tokens
// lie behind the capacity are CTA 0's.
//
// Latency bounds it: in a captured graph 256 requests of one token take 2.3 us, a
// launch (a call 3.2, the host's), and 37 prompts with 148000 tokens (1.8 MB
// written) 3.9 us (a call 4.1 to 4.7), which are the requests' loads, the scan, the
// bisection and the table's loads one after the other.
#include "fa_serve.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 1024;  // token slots of one CTA

// Exclusive prefix sums of a and b over the CTA; *sum_a and *sum_b get the totals.
__device__ __forceinline__ void scan2(long long &a, long long &b, long long *sum_a,
                                      long long *sum_b, long long (*warp_sums)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long a0 = a, b0 = b;
  for (int o = 1; o < 32; o *= 2) {
    const long long x = __shfl_up_sync(~0u, a, o), y = __shfl_up_sync(~0u, b, o);
    if (lane >= o) {
      a += x;
      b += y;
    }
  }
  if (lane == 31) {
    warp_sums[warp][0] = a;
    warp_sums[warp][1] = b;
  }
  __syncthreads();
  long long ba = 0, bb = 0, ta = 0, tb = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) {
      ba += warp_sums[w][0];
      bb += warp_sums[w][1];
    }
    ta += warp_sums[w][0];
    tb += warp_sums[w][1];
  }
  a += ba - a0;
  b += bb - b0;
  *sum_a = ta;
  *sum_b = tb;
}

// Largest i in 0 .. kRound - 1 with v[i] <= x (v ascending, v[0] <= x).
template <int kRound>
__device__ __forceinline__ int bisect(const long long *v, long long x) {
  int i = 0;
  for (int step = kRound / 2; step > 0; step /= 2)
    if (v[i + step] <= x) i += step;
  return i;
}

// kPer: requests of a thread in a round.
template <int kPer>
__global__ void __launch_bounds__(kThreads) fa_plan_kernel(const PlanParams p) {
  constexpr int kRound = kThreads * kPer;
  __shared__ long long s_tok[kRound], s_blk[kRound];
  __shared__ int s_cached[kRound], s_have[kRound];
  __shared__ long long s_warp[kThreads / 32][2];
  const int tid = threadIdx.x, cta = blockIdx.x, ctas = gridDim.x;
  griddep_wait();
  griddep_launch_dependents();
  const long long head = p.free_head ? max(0, *p.free_head) : 0;
  const long long reach = static_cast<long long>(p.width) << p.bs_log2;  // tokens of a table row
  const int mask = (1 << p.bs_log2) - 1;
  const long long t0 = static_cast<long long>(cta) * kTokens;
  const long long t1 = min(t0 + kTokens, static_cast<long long>(p.capacity));
  const int rounds = (p.B + kRound - 1) / kRound;
  // The block with index `at` in the order of allocation.
  auto fresh_block = [&](long long at) {
    at += head;
    return at < p.num_free ? p.free_blocks[at] : -1;
  };

  long long tok = 0, blk = 0;  // tokens and new blocks of the rounds so far
  for (int r = 0; r < rounds; ++r) {
    // CTA 0 goes through all rounds (it writes the totals); the others stop
    // behind their tokens and their last round of requests
    const int next_own = r + ((cta - r) % ctas + ctas) % ctas;
    if (cta != 0 && tok >= t1 && next_own >= rounds) break;
    const int b0 = r * kRound + tid * kPer;
    long long fresh[kPer], len[kPer], need[kPer], a = 0, n = 0, sum_tok, sum_blk;
#pragma unroll
    for (int y = 0; y < kPer; ++y) {
      const bool there = b0 + y < p.B;
      const long long cached = there ? max(0, p.cached[b0 + y]) : 0;
      fresh[y] = there ? max(0, p.fresh[b0 + y]) : 0;
      len[y] = min(cached + fresh[y], reach);
      const int have = static_cast<int>((min(cached, reach) + mask) >> p.bs_log2);
      need[y] = ((len[y] + mask) >> p.bs_log2) - have;
      s_cached[tid * kPer + y] = static_cast<int>(cached);
      s_have[tid * kPer + y] = have;
      a += fresh[y];
      n += need[y];
    }
    scan2(a, n, &sum_tok, &sum_blk, s_warp);
    a += tok;
    n += blk;
#pragma unroll
    for (int y = 0; y < kPer; ++y) {
      s_tok[tid * kPer + y] = a;
      s_blk[tid * kPer + y] = n;
      if (r % ctas == cta && b0 + y < p.B) {
        p.cu[b0 + y] = static_cast<int>(min(a, static_cast<long long>(p.capacity)));
        p.lens[b0 + y] = static_cast<int>(len[y]);
      }
      a += fresh[y];
      n += need[y];
    }
    __syncthreads();
    if (cta == 0 && tok + sum_tok > p.capacity) {
      for (long long j = blk + tid; j < blk + sum_blk; j += kThreads) {
        const int i = bisect<kRound>(s_blk, j);
        const long long at = s_have[i] + (j - s_blk[i]);
        if (s_tok[i] + (at << p.bs_log2) - s_cached[i] >= p.capacity)
          p.table[(static_cast<long long>(r) * kRound + i) * p.width + at] = fresh_block(j);
      }
    }
    for (long long t = max(t0, tok) + tid; t < min(t1, tok + sum_tok); t += kThreads) {
      const int i = bisect<kRound>(s_tok, t);
      const long long pos = s_cached[i] + (t - s_tok[i]);
      long long slot = -1;
      if (pos < reach) {
        const int j = static_cast<int>(pos >> p.bs_log2);
        int *entry = p.table + (static_cast<long long>(r) * kRound + i) * p.width + j;
        const int block = j < s_have[i] ? *entry : fresh_block(s_blk[i] + j - s_have[i]);
        if (j >= s_have[i] && (pos & mask) == 0) *entry = block;
        if (block >= 0) slot = (static_cast<long long>(block) << p.bs_log2) + (pos & mask);
      }
      p.slots[t] = slot;
      p.positions[t] = static_cast<int>(min(pos, 2147483647ll));
    }
    tok += sum_tok;
    blk += sum_blk;
    __syncthreads();
  }
  for (long long t = max(t0, tok) + tid; t < t1; t += kThreads) {  // behind the last token
    p.slots[t] = -1;
    p.positions[t] = 0;
  }
  if (cta == 0 && tid == 0) {
    p.cu[p.B] = static_cast<int>(min(tok, static_cast<long long>(p.capacity)));
    p.counts[0] = static_cast<int>(min(blk, 2147483647ll));
    p.counts[1] = static_cast<int>(min(tok, 2147483647ll));
  }
}

}  // namespace

cudaError_t launch_plan(const PlanParams &p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.capacity + kTokens - 1LL) / kTokens));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // One request a thread where a round then holds them all, four otherwise.  In a
  // captured graph, one and four: 37 requests of 4000 tokens 3.9 and 4.5 us, 256 of
  // one 2.1 and 2.6; 257 of one 3.4 and 3.0, 1000 6.0 and 4.4, 2000 of 500 22 and 16,
  // 30000 of 2 93 and 41.
  return p.B <= kThreads ? cudaLaunchKernelEx(&cfg, fa_plan_kernel<1>, p)
                         : cudaLaunchKernelEx(&cfg, fa_plan_kernel<4>, p);
}

}  // namespace fa
