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
// Every CTA makes the prefix sums itself, 256 requests at a time in shared
// memory, instead of waiting for a scan kernel: at the few hundred requests of
// a server that is one round of two loads a thread and a scan, less than a
// second launch.  CTA c owns kTokens token slots (it finds each one's request
// by bisection in the 256 prefix sums at hand), and the requests of every
// gridDim-th round (their lengths and offsets).  A token whose block is new reads
// the free list, not the table, so no CTA waits for another's table entries, and
// the first token of a new block writes its entry; those of blocks whose tokens
// lie behind the capacity are CTA 0's.
//
// Latency bounds it: 256 requests of one token 2.5 us, a launch; 37 prompts with
// 148000 tokens (1.8 MB written) 6.0 us, which are the requests' loads, the scan,
// the bisection and the table's loads one after the other.
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

// Largest i in 0 .. 255 with v[i] <= x (v ascending, v[0] <= x).
__device__ __forceinline__ int bisect(const long long *v, long long x) {
  int i = 0;
  for (int step = kThreads / 2; step > 0; step /= 2)
    if (v[i + step] <= x) i += step;
  return i;
}

__global__ void __launch_bounds__(kThreads) fa_plan_kernel(const PlanParams p) {
  __shared__ long long s_tok[kThreads], s_blk[kThreads];
  __shared__ int s_cached[kThreads], s_have[kThreads];
  __shared__ long long s_warp[kThreads / 32][2];
  const int tid = threadIdx.x, cta = blockIdx.x, ctas = gridDim.x;
  griddep_wait();
  griddep_launch_dependents();
  const long long head = p.free_head ? max(0, *p.free_head) : 0;
  const long long reach = static_cast<long long>(p.width) << p.bs_log2;  // tokens of a table row
  const int mask = (1 << p.bs_log2) - 1;
  const long long t0 = static_cast<long long>(cta) * kTokens;
  const long long t1 = min(t0 + kTokens, static_cast<long long>(p.capacity));
  const int rounds = (p.B + kThreads - 1) / kThreads;
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
    const int b = r * kThreads + tid;
    long long cached = 0, fresh = 0;
    if (b < p.B) {
      cached = max(0, p.cached[b]);
      fresh = max(0, p.fresh[b]);
    }
    const long long len = min(cached + fresh, reach);
    const int have = static_cast<int>((min(cached, reach) + mask) >> p.bs_log2);
    const long long need = ((len + mask) >> p.bs_log2) - have;
    long long a = fresh, n = need, sum_tok, sum_blk;
    scan2(a, n, &sum_tok, &sum_blk, s_warp);
    s_tok[tid] = tok + a;
    s_blk[tid] = blk + n;
    s_cached[tid] = static_cast<int>(cached);
    s_have[tid] = have;
    __syncthreads();
    if (r % ctas == cta) {
      if (b < p.B) {
        p.cu[b] = static_cast<int>(min(s_tok[tid], static_cast<long long>(p.capacity)));
        p.lens[b] = static_cast<int>(len);
      }
    }
    if (cta == 0 && tok + sum_tok > p.capacity) {
      for (long long j = blk + tid; j < blk + sum_blk; j += kThreads) {
        const int i = bisect(s_blk, j);
        const long long at = s_have[i] + (j - s_blk[i]);
        if (s_tok[i] + (at << p.bs_log2) - s_cached[i] >= p.capacity)
          p.table[(static_cast<long long>(r) * kThreads + i) * p.width + at] = fresh_block(j);
      }
    }
    for (long long t = max(t0, tok) + tid; t < min(t1, tok + sum_tok); t += kThreads) {
      const int i = bisect(s_tok, t);
      const long long pos = s_cached[i] + (t - s_tok[i]);
      long long slot = -1;
      if (pos < reach) {
        const int j = static_cast<int>(pos >> p.bs_log2);
        int *entry = p.table + (static_cast<long long>(r) * kThreads + i) * p.width + j;
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
  return cudaLaunchKernelEx(&cfg, fa_plan_kernel, p);
}

}  // namespace fa
