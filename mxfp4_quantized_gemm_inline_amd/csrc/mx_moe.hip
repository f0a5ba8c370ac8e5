// mx_moe.hip - routing to experts (scores, bias, groups, top-k, weights) and the stable sort of
// the chosen experts into the tables of the grouped GEMMs and the combine.
#include "mx_moe.h"

#include "mx_device.h"

namespace mx {
namespace {

// ------------------------------------------------------------------------------- route
//
// Keys: what is compared is an FP64 number whose low 10 mantissa bits are replaced by the expert's
// number, so that the larger of two keys is the larger score or, of equal ones, the lower expert,
// and one maximum brings value and place together. The 42 bits above hold a bf16 or FP32 logit
// exactly, and a sum of score and bias to 2^-42 of it.

constexpr double kNone = -__builtin_inf();

__device__ __forceinline__ double key_of(double c, int i) {
  c = fmin(fmax(c + 0.0, -1e300), 1e300);  // -0 becomes 0; an infinite key would be a NaN with the number in it
  const uint64_t b = __builtin_bit_cast(uint64_t, c);
  return __builtin_bit_cast(double, (b & ~1023ull) | (uint64_t)(b >> 63 ? i : 1023 - i));
}
__device__ __forceinline__ int index_of(double key) {
  const uint64_t b = __builtin_bit_cast(uint64_t, key);
  return b >> 63 ? (int)(b & 1023) : 1023 - (int)(b & 1023);
}
__device__ __forceinline__ double value_of(double key) {
  return __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, key) & ~1023ull);
}

__device__ __forceinline__ double wave_max(double x) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) x = fmax(x, __shfl_xor(x, d));
  return x;
}
__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d);
  return x;
}

__device__ __forceinline__ float load_logit(const RouteArgs& a, int64_t t, int e) {
  const int64_t at = t * a.stride + e;
  if (a.f32) return static_cast<const float*>(a.logits)[at];
  return __builtin_bit_cast(float, (uint32_t)static_cast<const uint16_t*>(a.logits)[at] << 16);
}

constexpr int kRouteWaves = 4;

// A wave per token, experts spread over the lanes.
__global__ __launch_bounds__(64 * kRouteWaves) void k_moe_route(RouteArgs a) {
  __shared__ double vals[kRouteWaves][1024];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int rows = a.num_rows ? *a.num_rows : a.T;
  for (int64_t t0 = (int64_t)blockIdx.x * kRouteWaves; t0 < a.T; t0 += (int64_t)gridDim.x * kRouteWaves) {
  const int64_t t = t0 + w;
  const bool live = t < a.T && t < rows;
  constexpr int V = 16;
  double key[V];
  double top = kNone, sum = 0;
  bool ok[V];
  double x[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * 64 + lane;
    float l = live && e < a.E ? load_logit(a, t, e) : -__builtin_inff();
    if (a.bias && e < a.E && !(a.bias[e] > -__builtin_inff())) l = -__builtin_inff();
    ok[v] = l > -__builtin_inff();
    x[v] = ok[v] ? (double)fminf(l, 3.402823466e38f) : kNone;
    top = fmax(top, x[v]);
  }
  const bool scored = a.bias || (a.groups > 1 && a.group_top == 2);
  const bool whole = !a.sigmoid && (scored || !a.renormalize);  // the softmax's sum over all experts
  if (!a.sigmoid) top = wave_max(top);
  double p[V];
  if (scored || whole) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      p[v] = !ok[v] ? 0.0 : a.sigmoid ? 1 / (1 + exp(-x[v])) : exp(x[v] - top);
      sum += p[v];
    }
    if (whole) {
      sum = wave_sum(sum);
#pragma unroll
      for (int v = 0; v < V; ++v) p[v] /= sum;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * 64 + lane;
    key[v] = !ok[v] ? kNone : key_of(a.bias ? p[v] + (double)a.bias[e] : x[v], e);
  }
  if (a.groups > 1) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = v * 64 + lane;
      if (e < a.E) vals[w][e] = !ok[v] ? kNone : a.bias || a.group_top == 1 ? value_of(key[v]) : p[v];
    }
    __syncthreads();
    const int gs = a.E / a.groups;
    double best = kNone, second = kNone;
    if (lane < a.groups)
      for (int i = 0; i < gs; ++i) {
        const double y = vals[w][lane * gs + i];
        second = fmax(second, fmin(best, y));
        best = fmax(best, y);
      }
    if (a.group_top == 2 && second > kNone) best += second;
    const double mine = best > kNone ? key_of(best, lane) : kNone;
    int before = 0;
    for (int g = 0; g < a.groups; ++g) before += __shfl(mine, g) > mine;
    const uint64_t kept = __ballot(mine > kNone && before < a.topk_groups);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = v * 64 + lane;
      if (e < a.E && !(kept >> (e / gs) & 1)) key[v] = kNone;
    }
  }
  double chosen = kNone;
  for (int i = 0; i < a.topk; ++i) {
    double best = kNone;
#pragma unroll
    for (int v = 0; v < V; ++v) best = fmax(best, key[v]);
    best = wave_max(best);
    if (lane == i) chosen = best;
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = key[v] == best ? kNone : key[v];
  }
  const bool has = lane < a.topk && chosen > kNone;
  const int id = has ? index_of(chosen) : -1;
  double s = 0;
  if (has) {
    const double l = fminf(load_logit(a, t, id), 3.402823466e38f);
    s = a.sigmoid ? 1 / (1 + exp(-l)) : exp(l - top);
    if (whole) s /= sum;
  }
  if (a.renormalize) {
    const double all = wave_sum(s);
    s = all > 0 ? s / all : 0;
  }
  if (t < a.T && lane < a.topk) {
    a.ids[t * a.topk + lane] = id;
    a.weights[t * a.topk + lane] = (float)(s * (double)a.scale);
  }
  __syncthreads();
  }
}

// ------------------------------------------------------------------------------- sort
//
// A stable counting sort. Every wave of a workgroup has its own part of the places, in order, and its
// own counters in LDS: counted first, then set to where the wave's rows of each expert start, then
// advanced 64 places at a time, lanes of one expert ranked by ballots over the number's bits.
// Few places: one workgroup does it all. More: each workgroup counts its places, the counts of an
// expert are summed up over the workgroups, each workgroup places its own.

constexpr int kSortOne = 16384;    // places of a single workgroup, at most
constexpr int kSortChunk = 4096;   // places of one of several, at least
constexpr int kSortChunks = 1024;  // workgroups, at most
inline bool sort_one(int64_t N) { return N <= kSortOne; }
inline int sort_chunk(int64_t N) {
  const int64_t each = (N + kSortChunks - 1) / kSortChunks;
  return (int)(each <= kSortChunk ? kSortChunk : (each + 255) / 256 * 256);
}
inline int sort_chunks(int64_t N) { return (int)((N + sort_chunk(N) - 1) / sort_chunk(N)); }

__device__ __forceinline__ int local_expert(const SortArgs& a, int n) {
  const uint32_t e = (uint32_t)a.ids[n] - (uint32_t)a.first;
  return e < (uint32_t)a.E ? (int)e : -1;
}

// counts: [E][chunks]
__global__ __launch_bounds__(256) void k_moe_sort_count(SortArgs a, int chunk, int32_t* counts) {
  __shared__ int32_t cnt[1024];
  for (int e = threadIdx.x; e < a.E; e += 256) cnt[e] = 0;
  __syncthreads();
  const int n0 = (int)blockIdx.x * chunk, n1 = min(a.N, n0 + chunk);
  for (int n = n0 + (int)threadIdx.x; n < n1; n += 256) {
    const int e = local_expert(a, n);
    if (e >= 0) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += 256) counts[(int64_t)e * gridDim.x + blockIdx.x] = cnt[e];
}

// A wave per expert: counts become the sums before them, totals: [E] their sums.
__global__ __launch_bounds__(64) void k_moe_sort_scan(int32_t* counts, int chunks, int32_t* totals) {
  int32_t* mine = counts + (int64_t)blockIdx.x * chunks;
  int base = 0;
  for (int c0 = 0; c0 < chunks; c0 += 64) {
    const int c = c0 + (int)threadIdx.x, x = c < chunks ? mine[c] : 0;
    int s = x;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int y = __shfl_up(s, d);
      if ((int)threadIdx.x >= d) s += y;
    }
    if (c < chunks) mine[c] = base + s - x;
    base += __shfl(s, 63);
  }
  if (threadIdx.x == 0) totals[blockIdx.x] = base;
}

// counts, totals: of the two kernels above, or null where this is the only workgroup.
template <int W>
__global__ __launch_bounds__(64 * W) void k_moe_sort_place(SortArgs a, int chunk, const int32_t* counts,
                                                         const int32_t* totals) {
  constexpr int kThreads = 64 * W, kEach = 1024 / kThreads;  // experts a thread
  __shared__ int32_t cnt[W][1024];
  __shared__ int32_t start[1025];
  __shared__ int32_t part[W];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int n0 = (int)blockIdx.x * chunk, n1 = min(a.N, n0 + chunk), each = chunk / W;
  const int w0 = n0 + w * each, w1 = min(n1, w0 + each);
  for (int i = threadIdx.x; i < W * a.E; i += kThreads) cnt[i / a.E][i % a.E] = 0;
  __syncthreads();
  for (int n = w0 + lane; n < w1; n += 64) {
    const int e = local_expert(a, n);
    if (e >= 0) atomicAdd(&cnt[w][e], 1);
  }
  __syncthreads();
  // where each expert's rows start
  int x[kEach], sum = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int e = (int)threadIdx.x * kEach + i;
    x[i] = 0;
    if (e < a.E) {
      if (totals) {
        x[i] = totals[e];
      } else {
        for (int j = 0; j < W; ++j) x[i] += cnt[j][e];
      }
    }
    sum += x[i];
  }
  int run = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(run, d);
    if (lane >= d) run += y;
  }
  if (lane == 63) part[w] = run;
  __syncthreads();
  run -= sum;
  for (int i = 0; i < w; ++i) run += part[i];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int e = (int)threadIdx.x * kEach + i;
    if (e <= a.E) start[e] = run;
    run += x[i];
  }
  if (threadIdx.x == kThreads - 1 && a.E == 1024) start[1024] = run;
  __syncthreads();
  const int R = start[a.E];
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    int base = start[e] + (counts ? counts[(int64_t)e * gridDim.x + blockIdx.x] : 0);
    for (int i = 0; i < W; ++i) {
      const int c = cnt[i][e];
      cnt[i][e] = base;
      base += c;
    }
  }
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e <= a.E; e += kThreads) a.offsets[e] = start[e];
  __syncthreads();
  for (int m0 = w0; m0 < w1; m0 += 64) {
    const int n = m0 + lane;
    const int e = n < w1 ? local_expert(a, n) : -1;
    uint64_t same = __ballot(e >= 0);  // lanes of the same expert
#pragma unroll
    for (int b = 0; b < 10; ++b) {
      const uint64_t one = __ballot(e >> b & 1);
      same &= (e >> b & 1) ? one : ~one;
    }
    int row = -1;
    if (e >= 0) {
      const int rank = __popcll(same & ((1ull << lane) - 1));
      int base = 0;
      if (rank == 0) base = atomicAdd(&cnt[w][e], (int)__popcll(same));
      row = __shfl(base, __builtin_ctzll(same)) + rank;
      a.row_token[row] = n / a.topk;
    }
    if (n < w1) a.token_rows[n] = row;
  }
  for (int64_t r = (int64_t)R + blockIdx.x * kThreads + threadIdx.x; r < a.N; r += (int64_t)gridDim.x * kThreads)
    a.row_token[r] = -1;
}

}  // namespace

hipError_t launch_moe_route(const RouteArgs& a, hipStream_t st) {
  hipLaunchKernelGGL(k_moe_route, dim3((unsigned)min((a.T + (int64_t)kRouteWaves - 1) / kRouteWaves, (int64_t)1 << 20)), dim3(64 * kRouteWaves), 0,
                     st, a);
  return hipGetLastError();
}

size_t moe_sort_workspace_bytes(int64_t N, int64_t E) {
  return sort_one(N) ? 0 : (size_t)(E * (sort_chunks(N) + 1)) * 4;
}

hipError_t launch_moe_sort(const SortArgs& a, void* workspace, hipStream_t st) {
  if (sort_one(a.N)) {
    const int chunk = (a.N + 1023) / 1024 * 1024;
    hipLaunchKernelGGL(k_moe_sort_place<16>, dim3(1), dim3(1024), 0, st, a, chunk, (const int32_t*)nullptr,
                       (const int32_t*)nullptr);
    return hipGetLastError();
  }
  const int chunk = sort_chunk(a.N), chunks = sort_chunks(a.N);
  int32_t* totals = static_cast<int32_t*>(workspace);
  int32_t* counts = totals + a.E;
  hipLaunchKernelGGL(k_moe_sort_count, dim3((unsigned)chunks), dim3(256), 0, st, a, chunk, counts);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_moe_sort_scan, dim3((unsigned)a.E), dim3(64), 0, st, counts, chunks, totals);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_moe_sort_place<4>, dim3((unsigned)chunks), dim3(256), 0, st, a, chunk, (const int32_t*)counts,
                     (const int32_t*)totals);
  return hipGetLastError();
}

}  // namespace mx
