// mx_moe.h - launchers behind mx_moe_route and mx_moe_sort. Sizes are validated by the caller
// (mx_moe_api.cpp) before any launcher runs.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "mx.h"

namespace mx {

struct RouteArgs {
  const void* logits;
  const float* bias;
  const int32_t* num_rows;
  int32_t* ids;
  float* weights;
  int64_t stride;
  int f32, T, E, topk, sigmoid, groups, topk_groups, group_top, renormalize;
  float scale;
};
hipError_t launch_moe_route(const RouteArgs& a, hipStream_t st);

struct SortArgs {
  const int32_t* ids;
  int32_t *offsets, *row_token, *token_rows;
  int N, topk, first, E, bits;  // bits: of an expert's number, E - 1 at most
};
size_t moe_sort_workspace_bytes(int64_t N, int64_t E);
hipError_t launch_moe_sort(const SortArgs& a, void* workspace, hipStream_t st);

}  // namespace mx
