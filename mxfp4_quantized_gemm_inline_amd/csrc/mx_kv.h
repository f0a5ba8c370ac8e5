// mx_kv.h - the paged MXFP4 key/value cache: layout, and the launchers behind the mx_kv_* calls.
// Sizes are validated by the caller (mx_kv_api.cpp) before any launcher runs.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx.h"

namespace mx {

// One (page, head) block of P tokens of D elements: K codes, V codes, K scales, V scales (the
// layout is written out in mx.h). Offsets are in bytes from the block's start.
struct KvLayout {
  int P, D;
  __host__ __device__ int64_t block_bytes() const { return (int64_t)P * D * 17 / 16; }
  __host__ __device__ int v_codes() const { return P * D / 2; }
  __host__ __device__ int k_scales() const { return P * D; }
  __host__ __device__ int v_scales() const { return P * D + P * (D / 32); }
  // byte of K element pair (d, d + 1), d even, of the page's token t
  __host__ __device__ int k_code(int t, int d) const {
    return (((t >> 4) * (D / 32) + (d >> 5)) * 16 + (t & 15)) * 16 + ((d & 31) >> 1);
  }
  __host__ __device__ int v_code(int t, int d) const {
    return v_codes() + (t >> 4) * (D * 8) + ((((t & 15) >> 2) * 16 + ((d & 31) >> 1)) * (D / 32) + (d >> 5)) * 4 +
           (t & 3);
  }
  __host__ __device__ int k_scale(int t, int d) const {
    return k_scales() + ((t >> 4) * (D / 32) + (d >> 5)) * 16 + (t & 15);
  }
  __host__ __device__ int v_scale(int t, int d) const { return v_scales() + t * (D / 32) + (d >> 5); }
};

struct KvTablesArgs {
  const int32_t *old_lens, *new_lens;
  int32_t *block_table, *free_pages;
  const int32_t* free_count;
  int32_t *free_count_out, *cu_q;
  int64_t* slots;
  int32_t *positions, *status;
  int B, max_blocks, capacity, T_max, log2_page;
};
size_t kv_tables_workspace_bytes(int64_t B, int64_t T_max);
hipError_t launch_kv_tables(const KvTablesArgs& a, void* workspace, hipStream_t st);

hipError_t launch_kv_write(const void* k, int64_t k_stride, const void* v, int64_t v_stride, const int64_t* slots,
                           int64_t T, void* cache, int64_t num_pages, int64_t P, int64_t heads, int64_t D,
                           hipStream_t st);
hipError_t launch_kv_read(const void* cache, int64_t num_pages, int64_t P, int64_t heads, int64_t D,
                          const int64_t* slots, int64_t T, void* k, void* v, hipStream_t st);

struct KvAppendArgs {
  const uint16_t *q, *k, *v;
  const int32_t* positions;
  const int64_t* slots;
  uint8_t* cache;
  const float *q_weight, *k_weight, *inv_freq;
  uint16_t* q_out;
  int64_t q_stride, k_stride, v_stride, q_out_stride, num_slots;
  int T, Hq, H, D, log2_page, rot, pairs;
  float eps, rope_scale;
};
hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t st);

struct VerifyArgs {
  const float *p, *q;  // target's and draft's probabilities (q may be null)
  int64_t p_stride, q_stride;
  const int32_t *tokens, *cu_q, *kv_lens;
  const float *accept, *sample;
  int32_t *out, *accepted, *new_lens;
  int T, B, V;
};
size_t verify_workspace_bytes(int64_t B, int64_t V);
hipError_t launch_verify(const VerifyArgs& a, void* workspace, hipStream_t st);

struct KvAttnArgs {
  const uint16_t* q;
  const uint8_t* cache;
  const int32_t *block_table, *cu_q, *kv_lens;
  uint16_t* out;
  int64_t q_stride, out_stride, num_pages, block_bytes;  // block_bytes: of one (page, head)
  int T, B, max_blocks, log2_page, Hq, H, G, D, causal, window;
  float scale;
};
// Sizes that choose the launch.
struct KvAttnSizes {
  int64_t B, T, Hq, H, D, max_q, max_kv, window;
};
size_t kv_attn_workspace_bytes(const KvAttnSizes& z);
hipError_t launch_kv_attn(const KvAttnArgs& a, const KvAttnSizes& z, void* workspace, size_t workspace_bytes,
                          hipStream_t st);
void kv_attn_plan(const KvAttnSizes& z, size_t workspace_bytes, char* buf, size_t len);

}  // namespace mx
