// mx_kv_attn.hip - attention of bf16 queries over the paged MXFP4 cache.
//
// For a query q at position pos over the keys K[j] and values V[j] that it sees,
//   s_j = scale q . K[j],  out = sum_j exp(s_j - m) V[j] / sum_j exp(s_j - m),  m = max_j s_j,
// in one pass over the tokens: with the running maximum m, sum l and unscaled output o, a
// block of tokens with maximum m' multiplies l and o by exp(m - max(m, m')) and adds its own.
#include <cmath>
#include <cstdio>

#include "mx_device.h"
#include "mx_kv.h"

namespace mx {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLowest = -3.0e38f;  // the running maximum before any token: below every score

// Value of one E2M1 code: sign, two exponent bits, one mantissa bit; subnormal 0.5.
__device__ __forceinline__ float e2m1(uint32_t c) {
  const uint32_t e = (c >> 1) & 3u, m = c & 1u;
  const float v = e ? (float)((2u + m) << (e - 1)) * 0.5f : 0.5f * (float)m;
  return (c & 8u) ? -v : v;
}
__device__ __forceinline__ float e8m0(uint32_t s) {
  return __builtin_bit_cast(float, s ? s << 23 : 0x00400000u);
}

// One wave per (row, query head); lane = token in blocks of 64 for the scores, lane = elements
// lane, lane + 64, .. for the output.
__global__ __launch_bounds__(64) void k_kv_attn_row(KvAttnArgs a) {
  __shared__ float q[256], p[64];
  __shared__ int page[64];
  const int lane = threadIdx.x, t = (int)(blockIdx.x / a.Hq), hq = (int)(blockIdx.x % a.Hq), h = hq / a.G;
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.cu_q[mid] <= t) lo = mid; else hi = mid;
  }
  const int b = lo;
  const int r0 = min(max(a.cu_q[b], 0), a.T), r1 = min(max(a.cu_q[b + 1], r0), a.T);
  if (t < r0 || t >= r1) return;
  const int64_t most = (int64_t)a.max_blocks << a.log2_page;
  const int len = (int)min((int64_t)max(a.kv_lens[b], 0), most);
  const int pos = len - (r1 - r0) + (t - r0);
  const int end = a.causal ? min(len, pos + 1) : len;
  const int begin = a.window ? max(pos - a.window + 1, 0) : 0;
  for (int d = lane; d < a.D; d += 64) {
    const uint32_t x = a.q[(int64_t)t * a.q_stride + hq * a.D + d];
    q[d] = __builtin_bit_cast(float, x << 16);
  }
  __syncthreads();
  const KvLayout L = {1 << a.log2_page, a.D};
  const float c = a.scale * kLog2e;
  float m = kLowest, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int j0 = begin; j0 < end; j0 += 64) {
    const int j = j0 + lane;
    float s = -INFINITY;
    int id = -1;
    if (j < end) {
      id = a.block_table[(int64_t)b * a.max_blocks + (j >> a.log2_page)];
      if (id < 0 || id >= a.num_pages) id = -1;
    }
    if (id >= 0) {
      const uint8_t* blk = a.cache + ((int64_t)id * a.H + h) * a.block_bytes;
      const int tok = j & (L.P - 1);
      float dot = 0.f;
      for (int d = 0; d < a.D; d += 32) {
        float part = 0.f;
        for (int i = 0; i < 32; i += 2) {
          const uint32_t w = blk[L.k_code(tok, d + i)];
          part += q[d + i] * e2m1(w & 15u) + q[d + i + 1] * e2m1(w >> 4);
        }
        dot += part * e8m0(blk[L.k_scale(tok, d)]);
      }
      s = dot * c;
    }
    float top = s;
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) top = fmaxf(top, __shfl_xor(top, x));
    const float m1 = fmaxf(m, top), alpha = __builtin_amdgcn_exp2f(m - m1);
    m = m1;
    const float w = __builtin_amdgcn_exp2f(s - m);
    l = l * alpha + w;
    __syncthreads();
    p[lane] = w;
    page[lane] = id;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] *= alpha;
    for (int k = 0; k < min(64, end - j0); ++k) {
      if (page[k] < 0) continue;
      const uint8_t* blk = a.cache + ((int64_t)page[k] * a.H + h) * a.block_bytes;
      const int tok = (j0 + k) & (L.P - 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d = lane + 64 * i;
        if (d >= a.D) break;
        const uint32_t w2 = blk[L.v_code(tok, d & ~1)];
        o[i] += p[k] * (e2m1((d & 1) ? w2 >> 4 : w2 & 15u) * e8m0(blk[L.v_scale(tok, d)]));
      }
    }
  }
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) l += __shfl_xor(l, x);
  const float inv = l > 0.f ? 1.f / l : 0.f;
  for (int i = 0; lane + 64 * i < a.D; ++i)
    a.out[(int64_t)t * a.out_stride + hq * a.D + lane + 64 * i] = (uint16_t)f32_to_bf16_rne(o[i] * inv);
}

}  // namespace

size_t kv_attn_workspace_bytes(const KvAttnSizes&) { return 0; }

hipError_t launch_kv_attn(const KvAttnArgs& a, const KvAttnSizes&, void*, size_t, hipStream_t st) {
  hipLaunchKernelGGL(k_kv_attn_row, dim3((unsigned)((int64_t)a.T * a.Hq)), dim3(64), 0, st, a);
  return hipGetLastError();
}

void kv_attn_plan(const KvAttnSizes& z, size_t, char* buf, size_t len) {
  std::snprintf(buf, len, z.B == 0 || z.T == 0 ? "none" : "k_kv_attn_row");
}

}  // namespace mx
