// mx_moe_api.cpp - the C ABI of routing and its sorted tables: argument validation (pure host
// code, before any HIP call), the gfx950 check and dispatch to the launchers.
#include <math.h>

#include "mx.h"
#include "mx_internal.h"
#include "mx_moe.h"

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int64_t kMaxPlaces = int64_t(1) << 28;
constexpr int64_t kMaxExperts = 1024;
constexpr int64_t kMaxStride = int64_t(1) << 32;

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
mx_status from_hip(hipError_t e) { return e == hipSuccess ? MX_OK : MX_ERR_HIP; }
bool flag(int32_t x) { return x == 0 || x == 1; }

bool sort_sizes_ok(int64_t T, int64_t topk, int64_t E) {
  return T >= 0 && T <= kMaxPlaces && topk >= 1 && topk <= 1024 && T * topk <= kMaxPlaces && E >= 1 && E <= kMaxExperts;
}

}  // namespace

extern "C" {

mx_status mx_moe_route(const void* logits, int64_t logits_stride, int32_t logits_type, const float* bias,
                       int64_t T, int64_t E, int64_t topk, int32_t score, int64_t groups, int64_t topk_groups,
                       int32_t group_top, int32_t renormalize, float scale, const int32_t* num_rows,
                       int32_t* topk_ids, float* topk_weights, hipStream_t stream) {
  if (T < 0 || E < 1 || E > kMaxExperts || groups < 1 || groups > 64 || E % groups != 0 || topk_groups < 1 ||
      topk_groups > groups || topk < 1 || topk > 64 || topk > topk_groups * (E / groups) || T > kMaxRows / topk ||
      logits_stride < 0 || logits_stride >= kMaxStride || (logits_type != MX_TYPE_BF16 && logits_type != MX_TYPE_F32) ||
      (score != MX_SCORE_SOFTMAX && score != MX_SCORE_SIGMOID) || (group_top != 1 && group_top != 2) ||
      !flag(renormalize) || !isfinite(scale))
    return MX_ERR_SHAPE;
  if (T == 0) return MX_OK;
  if (!logits || !topk_ids || !topk_weights) return MX_ERR_NULL;
  if (!aligned(logits, logits_type == MX_TYPE_F32 ? 4 : 2) || !aligned(bias, 4) || !aligned(num_rows, 4) ||
      !aligned(topk_ids, 4) || !aligned(topk_weights, 4))
    return MX_ERR_ALIGN;
  const mx_status d = mx::check_device();
  if (d != MX_OK) return d;
  const mx::RouteArgs a = {logits, bias, num_rows, topk_ids, topk_weights, logits_stride, logits_type == MX_TYPE_F32, (int)T,
                           (int)E, (int)topk, score == MX_SCORE_SIGMOID, (int)groups, (int)topk_groups, group_top,
                           renormalize, scale};
  return from_hip(mx::launch_moe_route(a, stream));
}

size_t mx_moe_sort_workspace_bytes(int64_t T, int64_t topk, int64_t E) {
  return sort_sizes_ok(T, topk, E) ? mx::moe_sort_workspace_bytes(T * topk, E) : 0;
}

mx_status mx_moe_sort(const int32_t* topk_ids, int64_t T, int64_t topk, int64_t first_expert, int64_t E,
                      int32_t* expert_offsets, int32_t* row_token, int32_t* token_rows, void* workspace,
                      size_t workspace_bytes, hipStream_t stream) {
  if (!sort_sizes_ok(T, topk, E) || first_expert < 0 || first_expert >= kMaxRows) return MX_ERR_SHAPE;
  if (!expert_offsets || (T > 0 && (!topk_ids || !row_token || !token_rows))) return MX_ERR_NULL;
  if (!aligned(topk_ids, 4) || !aligned(expert_offsets, 4) || !aligned(row_token, 4) || !aligned(token_rows, 4) ||
      !aligned(workspace, 16))
    return MX_ERR_ALIGN;
  const size_t need = mx::moe_sort_workspace_bytes(T * topk, E);
  if (need && (!workspace || workspace_bytes < need)) return MX_ERR_WORKSPACE;
  const mx_status d = mx::check_device();
  if (d != MX_OK) return d;
  const mx::SortArgs a = {topk_ids, expert_offsets, row_token, token_rows, (int)(T * topk), (int)topk, (int)first_expert,
                          (int)E, E > 1 ? 64 - __builtin_clzll((unsigned long long)(E - 1)) : 0};
  return from_hip(mx::launch_moe_sort(a, workspace, stream));
}

}  // extern "C"
