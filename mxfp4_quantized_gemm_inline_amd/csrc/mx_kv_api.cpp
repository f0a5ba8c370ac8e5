// mx_kv_api.cpp - the C ABI of the paged MXFP4 key/value cache: argument validation (pure host
// code, before any HIP call), the gfx950 check and dispatch to the launchers.
#include "mx.h"
#include "mx_internal.h"
#include "mx_kv.h"

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 30;   // row counts stay in 32 bits, also rounded up
constexpr int64_t kMaxBatch = int64_t(1) << 20;
constexpr int64_t kMaxStride = int64_t(1) << 32;  // elements: rows times stride stay in 63 bits
constexpr int64_t kMaxPages = int64_t(1) << 31;
constexpr int64_t kMaxHeads = 1024;
constexpr int64_t kMaxTiles = int64_t(1) << 22;   // requests times heads: a launch holds under 2^32 threads
constexpr float kMaxScale = 0x1p127f;             // times log2 e it is finite in FP32
constexpr int64_t kMaxTokens = int64_t(1) << 30;  // of one request: positions stay in 32 bits, also past a tile's end

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool page_ok(int64_t P) { return P >= 16 && P <= 1024 && (P & (P - 1)) == 0; }
bool head_ok(int64_t D) { return D == 64 || D == 128 || D == 256; }
bool table_ok(int64_t max_blocks, int64_t P) { return max_blocks >= 1 && max_blocks <= kMaxTokens / P; }
bool stride_ok(int64_t s, int64_t least) { return s >= least && s < kMaxStride && s % 8 == 0; }
int log2_of(int64_t P) { return __builtin_ctzll((unsigned long long)P); }
mx_status from_hip(hipError_t e) { return e == hipSuccess ? MX_OK : MX_ERR_HIP; }

bool attn_sizes_ok(const mx::KvAttnSizes& z) {
  return z.B >= 0 && z.B <= kMaxBatch && z.T >= 0 && z.T <= kMaxRows && z.H >= 1 && z.H <= kMaxHeads && z.Hq >= 1 &&
         z.Hq <= kMaxHeads && z.Hq % z.H == 0 && z.T <= kMaxRows / z.Hq &&
         z.B * z.H <= kMaxTiles && head_ok(z.D) && z.max_q >= 1 &&
         z.max_kv >= 1 && z.window >= 0;
}

}  // namespace

extern "C" {

size_t mx_kv_cache_bytes(int64_t num_pages, int64_t page_size, int64_t heads, int64_t D) {
  if (num_pages < 1 || num_pages >= kMaxPages || !page_ok(page_size) || heads < 1 || heads > kMaxHeads || !head_ok(D))
    return 0;
  return (size_t)num_pages * (size_t)heads * (size_t)(page_size * D / 16 * 17);
}

size_t mx_kv_tables_workspace_bytes(int64_t B, int64_t T_max) {
  if (B < 0 || B > kMaxBatch || T_max < 0 || T_max > kMaxRows) return 0;
  return mx::kv_tables_workspace_bytes(B, T_max);
}

mx_status mx_kv_tables(const int32_t* old_lens, const int32_t* new_lens, int64_t B, int64_t page_size,
                       int32_t* block_table, int64_t max_blocks, int32_t* free_pages, int64_t capacity,
                       const int32_t* free_count, int32_t* free_count_out, int64_t T_max, int32_t* cu_q,
                       int64_t* slots, int32_t* positions, int32_t* status, void* workspace,
                       size_t workspace_bytes, hipStream_t stream) {
  if (B < 0 || B > kMaxBatch || T_max < 0 || T_max > kMaxRows || !page_ok(page_size) ||
      !table_ok(max_blocks, page_size) || capacity < 0 || capacity >= kMaxPages)
    return MX_ERR_SHAPE;
  if (!free_count || !free_count_out || !cu_q || !status || (B > 0 && (!old_lens || !new_lens || !block_table)) ||
      (capacity > 0 && !free_pages) || (T_max > 0 && (!slots || !positions)))
    return MX_ERR_NULL;
  if (!aligned(old_lens, 4) || !aligned(new_lens, 4) || !aligned(block_table, 4) || !aligned(free_pages, 4) ||
      !aligned(free_count, 4) || !aligned(free_count_out, 4) || !aligned(cu_q, 4) || !aligned(slots, 8) ||
      !aligned(positions, 4) || !aligned(status, 4) || !aligned(workspace, 16))
    return MX_ERR_ALIGN;
  const size_t need = mx::kv_tables_workspace_bytes(B, T_max);
  if (need && (!workspace || workspace_bytes < need)) return MX_ERR_WORKSPACE;
  const mx_status d = mx::check_device();
  if (d != MX_OK) return d;
  const mx::KvTablesArgs a = {old_lens, new_lens, block_table, free_pages, free_count, free_count_out, cu_q, slots,
                              positions, status, (int)B, (int)max_blocks, (int)capacity, (int)T_max,
                              log2_of(page_size)};
  return from_hip(mx::launch_kv_tables(a, workspace, stream));
}

mx_status mx_kv_write(const void* k_bf16, int64_t k_stride, const void* v_bf16, int64_t v_stride,
                      const int64_t* slots, int64_t T, void* cache, int64_t num_pages, int64_t page_size,
                      int64_t heads, int64_t D, hipStream_t stream) {
  if (T < 0 || T > kMaxRows || mx_kv_cache_bytes(num_pages, page_size, heads, D) == 0 || !stride_ok(k_stride, 0) ||
      !stride_ok(v_stride, 0))
    return MX_ERR_SHAPE;
  if (T == 0) return MX_OK;
  if (!k_bf16 || !v_bf16 || !slots || !cache) return MX_ERR_NULL;
  if (!aligned(k_bf16, 16) || !aligned(v_bf16, 16) || !aligned(cache, 16) || !aligned(slots, 8)) return MX_ERR_ALIGN;
  const mx_status d = mx::check_device();
  if (d != MX_OK) return d;
  return from_hip(mx::launch_kv_write(k_bf16, k_stride, v_bf16, v_stride, slots, T, cache, num_pages, page_size, heads,
                                      D, stream));
}

mx_status mx_kv_read(const void* cache, int64_t num_pages, int64_t page_size, int64_t heads, int64_t D,
                     const int64_t* slots, int64_t T, void* k_bf16, void* v_bf16, hipStream_t stream) {
  if (T < 0 || T > kMaxRows || mx_kv_cache_bytes(num_pages, page_size, heads, D) == 0) return MX_ERR_SHAPE;
  if (T == 0) return MX_OK;
  if (!k_bf16 || !v_bf16 || !slots || !cache) return MX_ERR_NULL;
  if (!aligned(k_bf16, 16) || !aligned(v_bf16, 16) || !aligned(cache, 16) || !aligned(slots, 8)) return MX_ERR_ALIGN;
  const mx_status d = mx::check_device();
  if (d != MX_OK) return d;
  return from_hip(mx::launch_kv_read(cache, num_pages, page_size, heads, D, slots, T, k_bf16, v_bf16, stream));
}

size_t mx_kv_attention_workspace_bytes(int64_t B, int64_t T, int64_t heads_q, int64_t heads, int64_t D,
                                       int64_t max_q, int64_t max_kv, int64_t window) {
  const mx::KvAttnSizes z = {B, T, heads_q, heads, D, max_q, max_kv, window};
  return attn_sizes_ok(z) && B > 0 && T > 0 ? mx::kv_attn_workspace_bytes(z) : 0;
}

mx_status mx_kv_attention(const void* q_bf16, int64_t q_stride, const void* cache, int64_t num_pages,
                          int64_t page_size, const int32_t* block_table, int64_t max_blocks,
                          const int32_t* cu_q, const int32_t* kv_lens, int64_t B, int64_t T, int64_t heads_q,
                          int64_t heads, int64_t D, int64_t max_q, int64_t max_kv, int32_t causal,
                          int64_t window, float scale, void* out_bf16, int64_t out_stride, void* workspace,
                          size_t workspace_bytes, hipStream_t stream) {
  const mx::KvAttnSizes z = {B, T, heads_q, heads, D, max_q, max_kv, window};
  if (!attn_sizes_ok(z) || mx_kv_cache_bytes(num_pages, page_size, heads, D) == 0 ||
      !table_ok(max_blocks, page_size) || (causal != 0 && causal != 1) || (window > 0 && !causal) ||
      !(scale > 0.f && scale <= kMaxScale) || !stride_ok(q_stride, 0) || !stride_ok(out_stride, heads_q * D))
    return MX_ERR_SHAPE;
  if (T == 0 || B == 0) return MX_OK;
  if (!q_bf16 || !cache || !block_table || !cu_q || !kv_lens || !out_bf16) return MX_ERR_NULL;
  if (!aligned(q_bf16, 16) || !aligned(cache, 16) || !aligned(out_bf16, 16) || !aligned(workspace, 16) ||
      !aligned(block_table, 4) || !aligned(cu_q, 4) || !aligned(kv_lens, 4))
    return MX_ERR_ALIGN;
  const mx_status d = mx::check_device();
  if (d != MX_OK) return d;
  mx::KvAttnArgs a = {};
  a.q = static_cast<const uint16_t*>(q_bf16);
  a.cache = static_cast<const uint8_t*>(cache);
  a.block_table = block_table;
  a.cu_q = cu_q;
  a.kv_lens = kv_lens;
  a.out = static_cast<uint16_t*>(out_bf16);
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.num_pages = num_pages;
  a.block_bytes = page_size * D / 16 * 17;
  a.T = (int)T;
  a.B = (int)B;
  a.max_blocks = (int)max_blocks;
  a.log2_page = log2_of(page_size);
  a.Hq = (int)heads_q;
  a.H = (int)heads;
  a.G = (int)(heads_q / heads);
  a.D = (int)D;
  a.causal = causal;
  a.window = (int)(window < max_blocks * page_size ? window : 0);  // one past every length is none
  a.scale = scale;
  return from_hip(mx::launch_kv_attn(a, z, workspace, workspace ? workspace_bytes : 0, stream));
}

mx_status mx_kv_attention_plan(int64_t B, int64_t T, int64_t heads_q, int64_t heads, int64_t D, int64_t max_q,
                               int64_t max_kv, int64_t window, size_t workspace_bytes, char* buf,
                               size_t buf_len) {
  const mx::KvAttnSizes z = {B, T, heads_q, heads, D, max_q, max_kv, window};
  if (!attn_sizes_ok(z)) return MX_ERR_SHAPE;
  if (!buf || buf_len == 0) return MX_ERR_NULL;
  mx::kv_attn_plan(z, workspace_bytes, buf, buf_len);
  return MX_OK;
}

}  // extern "C"
