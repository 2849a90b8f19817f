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

// ------------------------------------------------------------ 4-bit cache
// Row (block, head, offset) of the cache: d/2 bytes of codes and d/16 bytes
// of scales, rows in that order.
struct Kv4Store {
  uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
  int num_blocks, Hk, bs_log2, d;
  int k_exp, v_exp;
};
cudaError_t launch_kv4_append(const void *k, const void *v, long long k_stride, long long v_stride,
                              const long long *slots, int T, const Kv4Store &c, int dtype,
                              cudaStream_t s);
cudaError_t launch_kv4_gather(const long long *slots, int R, const Kv4Store &c, void *k_out,
                              void *v_out, int dtype, cudaStream_t s);

// ------------------------------------------------------------ attention
struct Kv4Attn {
  const void *q;                  // [total_q][Hq][d]
  void *o;
  float *lse;                     // [Hq][total_q]
  Kv4Store c;
  const int *table;               // [B][width]
  const int *lens;                // [B]
  const int *cu_q;                // [B + 1] or null (one query a sequence)
  int B, Hq, group;               // group = Hq / Hk
  int total_q, max_q;
  int max_k;                      // at most width blocks, and kKv4MaxKeys
  int width;
  float scale_log2;               // scale * 2^k_exp * log2(e)
  float v_mul;                    // 2^v_exp
  int causal;
};
// Sequences with at most `rows` rows (queries x group) go through
// launch_kv4_attn's tile of that many rows, longer ones through
// launch_kv4_many.  kv4_tile_rows: 8, 16 or 32, the smallest that holds the
// longest sequence, else the smallest that holds one query; 0: none, either
// because none does or because the other kernel is faster at so many keys (the
// longest sequence's, times sequences and key heads).
constexpr int kKv4MaxCtas = 304;   // two on each of 152 SMs
constexpr int kKv4ManyCtas = 152;  // launch_kv4_many: one on each
constexpr int kKv4ManyRows = 128;  // and tiles of that many rows, so group <= 128
// Keys of a sequence at most: the kernels count in 32 bits and look up to three
// steps of 128 keys past the last one, and round up to whole steps.
constexpr int kKv4MaxKeys = 2147483647 - 4095;
int kv4_tile_rows(int group, int max_q, int d, long long keys);
// What a call launches: `rows` of launch_kv4_attn's tile (0: not launched), the
// CTAs of its clusters (0: none, the line of units) and in all; and the CTAs of
// launch_kv4_many (0: not launched).  max_k as in Kv4Attn.
struct Kv4Grid {
  int rows, cluster, ctas, many;
};
Kv4Grid kv4_grid(int B, int Hk, int group, int d, int max_q, int max_k, int num_sms);
size_t kv4_workspace(int rows, int d);  // of either kernel, by its rows
cudaError_t launch_kv4_attn(const Kv4Attn &p, const Kv4Grid &g, int dtype, float *ws,
                            cudaStream_t s);
// status: the device's status word; wait_limit_ns bounds its barrier waits;
// skip_load: the test hook that leaves out a tile's values.
cudaError_t launch_kv4_many(const Kv4Attn &p, const Kv4Grid &g, int dtype, float *ws,
                            unsigned *status, unsigned long long wait_limit_ns, int skip_load,
                            cudaStream_t s);

}  // namespace fa
