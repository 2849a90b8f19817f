// fa_serve.h — declarations of the serving operators' kernels (block tables,
// rotary positions, the 4-bit cache and attention over it), shared by their
// host API (fa_serve_api.cu) and their translation units.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace fa {

// Host helpers of fa_api.cu.  The current device must be sm_103: FA_OK,
// FA_ERR_UNSUPPORTED or FA_ERR_CUDA.  api_device_check touches no device
// memory; api_device_status also hands out the per-device status word (made
// on the first call on a device).
int api_device_check();
int api_device_status(unsigned **status);
int api_sm_count();
unsigned long long api_wait_limit();
int api_skip_load();  // the test hook of fa_set_test_hooks

// ------------------------------------------------------------ block tables
struct PlanParams {
  const int *cached, *fresh;      // [B] tokens held, tokens to come
  const int *free_blocks;         // [num_free]
  const int *free_head;           // entries of free_blocks already used, or null
  int *table;                     // [B][width]
  long long *slots;               // [capacity]
  int *positions;                 // [capacity]
  int *cu;                        // [B + 1]
  int *lens;                      // [B]
  int *counts;                    // {blocks needed, tokens}
  int B, width, bs_log2, num_free, capacity;
};
cudaError_t launch_plan(const PlanParams &p, cudaStream_t s);

// ------------------------------------------------------------ rotary
struct RopeTensor {
  const void *in;
  void *out;
  long long ib, ih, in_row, ob, oh, out_row;  // strides in elements
  int heads;
};
struct RopeParams {
  RopeTensor q, k;                // k.heads = 0: none
  const int *positions;           // [axes][rows]
  const unsigned long long *table;  // [d_rot / 2]
  long long rows;                 // B * N
  int N, d, d_rot, axes, interleaved, inverse;
};
// dtype: FA_DTYPE_BF16, FA_DTYPE_F16 or FA_DTYPE_F32.
cudaError_t launch_rope(const RopeParams &p, int dtype, int num_sms, cudaStream_t s);

// ------------------------------------------------------------ caches
// Row (block, head, offset) of the 4-bit cache: d/2 bytes of codes and d/16 bytes
// of scales, rows in that order.
struct KvStore {
  uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
  int num_blocks, Hk, bs_log2, d;
  int k_exp, v_exp;
};
cudaError_t launch_kv4_append(const void *k, const void *v, long long k_stride, long long v_stride,
                              const long long *slots, int T, const KvStore &c, int dtype,
                              cudaStream_t s);
cudaError_t launch_kv4_gather(const long long *slots, int R, const KvStore &c, void *k_out,
                              void *v_out, int dtype, cudaStream_t s);

// The 8-bit cache: d bytes of codes a row, an fp32 scale for (block, head) in
// k_scales and v_scales; k_exp and v_exp are 0.
cudaError_t launch_kv8_append(const void *k, const void *v, long long k_stride, long long v_stride,
                              const long long *slots, int T, const KvStore &c, int dtype,
                              cudaStream_t s);
cudaError_t launch_kv8_gather(const long long *slots, int R, const KvStore &c, void *k_out,
                              void *v_out, int dtype, cudaStream_t s);

// ------------------------------------------------------------ pages
// The arrays of a cache, pages of bytes[i] bytes: read from, written to.
constexpr int kMaxArrays = 256;
constexpr int kMaxSweep = 1 << 23;  // blocks that launch_kv_free and launch_kv_compact take
struct Pages {
  const void *const *from;
  void *const *to;
  const unsigned long long *bytes;
  int num;
};
cudaError_t launch_kv_copy(const Pages &pages, const int *src, const int *dst, int n, int from_blocks,
                           int to_blocks, int num_sms, cudaStream_t s);
struct ForkParams {
  const int *table, *lens;        // [B][width], [B]
  const int *parents;             // [n]
  const int *free_blocks;         // [num_free]
  const int *free_head;           // entries of free_blocks already used, or null
  int *table_out, *lens_out;      // [n][width], [n]
  int *counts;                    // {blocks needed, entries of free_blocks used}
  int B, n, width, bs_log2, num_free, num_blocks, parents_end;
};
cudaError_t launch_kv_fork(const Pages &pages, const ForkParams &p, int num_sms, cudaStream_t s);
struct FreeParams {
  const int *table;               // [B][width]
  int *lens;                      // [B]
  const unsigned char *ended;     // [B] or null
  int *free_blocks, *free_head;   // [num_blocks], {blocks held}
  int B, width, bs_log2, num_blocks;
};
cudaError_t launch_kv_free(const FreeParams &p, cudaStream_t s);
struct CompactParams {
  const int *table, *lens;        // [B][width], [B]
  int *table_out, *new_ids;       // [B][width], [num_blocks]
  int *counts;                    // {blocks held, pages moved}
  int *moves;                     // [2][num_blocks / 2]
  int B, width, bs_log2, num_blocks;
};
cudaError_t launch_kv_compact(const Pages &pages, const CompactParams &p, int num_sms, cudaStream_t s);

// ------------------------------------------------------------ attention
struct KvAttn {
  const void *q;                  // [total_q][Hq][d]
  void *o;
  float *lse;                     // [Hq][total_q]
  KvStore c;
  const int *table;               // [B][width]
  const int *lens;                // [B]
  const int *cu_q;                // [B + 1] or null (one query a sequence)
  int B, Hq, group;               // group = Hq / Hk
  int total_q, max_q;
  int max_k;                      // at most width blocks, and kKvMaxKeys
  int width;
  float scale_log2;               // scale * 2^k_exp * log2(e)
  float v_mul;                    // 2^v_exp
  int causal;
};
// Sequences with at most `rows` rows (queries x group) go through
// launch_kv4_attn's (kv8) tile of that many rows, longer ones through
// launch_kv4_many (kv8).  kv4_tile_rows: 8, 16 or 32, the smallest that holds the
// longest sequence, else the smallest that holds one query; 0: none, either
// because none does or because the other kernel is faster at so many keys (the
// longest sequence's, times sequences and key heads).
constexpr int kKvMaxCtas = 304;   // two on each of 152 SMs
constexpr int kKvManyCtas = 152;  // launch_kv4_many: one on each
constexpr int kKvManyRows = 128;  // and tiles of that many rows, so group <= 128
// Keys of a sequence at most: the kernels count in 32 bits and look up to three
// steps of 128 keys past the last one, and round up to whole steps.
constexpr int kKvMaxKeys = 2147483647 - 4095;
int kv4_tile_rows(int group, int max_q, int d, long long keys);
int kv8_tile_rows(int group, int max_q, int d);
// What a call launches: `rows` of launch_kv4_attn's tile (0: not launched), the
// CTAs of its clusters (0: none, the line of units) and in all; and the CTAs of
// launch_kv4_many (0: not launched).  max_k as in KvAttn.
struct KvGrid {
  int rows, cluster, ctas, many;
};
KvGrid kv4_grid(int B, int Hk, int group, int d, int max_q, int max_k, int num_sms);
KvGrid kv8_grid(int B, int Hk, int group, int d, int max_q, int max_k, int num_sms);
size_t kv_workspace(int rows, int d);  // of either kernel, by its rows
cudaError_t launch_kv4_attn(const KvAttn &p, const KvGrid &g, int dtype, float *ws,
                            cudaStream_t s);
// status: the device's status word; wait_limit_ns bounds its barrier waits;
// skip_load: the test hook that leaves out a tile's values.
cudaError_t launch_kv8_attn(const KvAttn &p, const KvGrid &g, int dtype, float *ws,
                            cudaStream_t s);
cudaError_t launch_kv4_many(const KvAttn &p, const KvGrid &g, int dtype, float *ws,
                            unsigned *status, unsigned long long wait_limit_ns, int skip_load,
                            cudaStream_t s);
cudaError_t launch_kv8_many(const KvAttn &p, const KvGrid &g, int dtype, float *ws,
                            unsigned *status, unsigned long long wait_limit_ns, int skip_load,
                            cudaStream_t s);

}  // namespace fa
