// mx_moe.hip - routing to experts (scores, bias, groups, top-k, weights) and the stable sort of
// the chosen experts into the tables of the grouped GEMMs and the combine.
#include "mx_moe.h"

#include "mx_device.h"

namespace mx {
namespace {

// ------------------------------------------------------------------------------- route
//
// A wave per token, experts over its lanes. Keys: what is compared is a number whose low bits are
// replaced by the expert's, so that the larger of two keys is the larger score or, of equal ones, the
// lower expert, and no two are equal. bf16 logits that are compared as they are: 32 bits, the logit's
// 16 in order above the expert. Otherwise FP64: the 42 bits above the expert hold an FP32 logit exactly,
// and a sum of score and bias to 2^-42 of it.
//
// The topk largest of E keys without sorting them: the lanes' largest keys are bisected for a bound that
// at least topk of them reach, and few more, so that the topk largest of all reach it too; what reaches
// it is put one to a lane, and each is ranked by comparing it with all of them. Where more than 64 reach
// the bound (rows of equal logits, the largest all in a few lanes) the largest is taken topk times
// instead.

constexpr int kRouteWaves = 4;
constexpr int kBisections = 14;  // at most: the lanes that reach the bound may be a quarter more than topk

template <int kControl, int kRows = 0xF>
__device__ __forceinline__ uint32_t dpp(uint32_t old, uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)old, (int)x, kControl, kRows, 0xF, false);
}
template <int kControl, int kRows = 0xF>
__device__ __forceinline__ double dpp(double old, double x) {
  const uint2 o = __builtin_bit_cast(uint2, old), u = __builtin_bit_cast(uint2, x);
  return __builtin_bit_cast(double, make_uint2(dpp<kControl, kRows>(o.x, u.x), dpp<kControl, kRows>(o.y, u.y)));
}
__device__ __forceinline__ uint32_t lane_value(uint32_t x, int lane) { return (uint32_t)__builtin_amdgcn_readlane((int)x, lane); }
__device__ __forceinline__ double lane_value(double x, int lane) {
  const uint2 u = __builtin_bit_cast(uint2, x);
  return __builtin_bit_cast(double, make_uint2(lane_value(u.x, lane), lane_value(u.y, lane)));
}
// op over the wave, the same in every lane: within rows of 16, then over the rows, to lane 63. `none`:
// the operation's neutral element.
template <typename T, typename Op>
__device__ __forceinline__ T wave_reduce(T x, T none, Op op) {
  x = op(x, dpp<0x111>(none, x));       // a lane 1 below
  x = op(x, dpp<0x112>(none, x));       // 2
  x = op(x, dpp<0x114>(none, x));       // 4
  x = op(x, dpp<0x118>(none, x));       // 8
  x = op(x, dpp<0x142, 0xA>(none, x));  // the row below's last lane
  x = op(x, dpp<0x143, 0xC>(none, x));  // the lower half's
  return lane_value(x, 63);
}
// The sum over the lanes up to each.
__device__ __forceinline__ uint32_t wave_scan(uint32_t x) {
  x += dpp<0x111>(0u, x);
  x += dpp<0x112>(0u, x);
  x += dpp<0x114>(0u, x);
  x += dpp<0x118>(0u, x);
  x += dpp<0x142, 0xA>(0u, x);
  return x + dpp<0x143, 0xC>(0u, x);
}
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  return wave_reduce(x, 0u, [](uint32_t a, uint32_t b) { return max(a, b); });
}
__device__ __forceinline__ double wave_max(double x) {
  return wave_reduce(x, -__builtin_inf(), [](double a, double b) { return fmax(a, b); });
}
__device__ __forceinline__ double wave_sum(double x) {
  return wave_reduce(x, 0.0, [](double a, double b) { return a + b; });
}

// exp(x) for x <= 0 (-inf gives 0), in FP64: 2^n times the series of exp(r), |r| <= log(2) / 2, up to
// r^13, whose next term is below 2^-57.
__device__ __forceinline__ double exp_of(double x) {
  x = fmax(x, -800.0);  // below the least subnormal
  const double n = rint(x * 1.44269504088896340736);
  double r = fma(-n, 0.693147180559945286227, x);
  r = fma(-n, 2.31904681384629955842e-17, r);
  double y = 1.0 / 6227020800.0;
  y = fma(y, r, 1.0 / 479001600.0);
  y = fma(y, r, 1.0 / 39916800.0);
  y = fma(y, r, 1.0 / 3628800.0);
  y = fma(y, r, 1.0 / 362880.0);
  y = fma(y, r, 1.0 / 40320.0);
  y = fma(y, r, 1.0 / 5040.0);
  y = fma(y, r, 1.0 / 720.0);
  y = fma(y, r, 1.0 / 120.0);
  y = fma(y, r, 1.0 / 24.0);
  y = fma(y, r, 1.0 / 6.0);
  y = fma(y, r, 0.5);
  y = fma(y, r, 1.0);
  y = fma(y, r, 1.0);
  return ldexp(y, (int)n);
}
__device__ __forceinline__ double sigmoid_of(double x) {
  const double e = exp_of(-fabs(x)), d = 1.0 + e;
  double r = __builtin_amdgcn_rcp(d);  // 1 <= d <= 2: two steps of Newton give all bits
  r = fma(r, fma(-d, r, 1.0), r);
  r = fma(r, fma(-d, r, 1.0), r);
  return x >= 0 ? r : e * r;
}

__device__ __forceinline__ uint32_t in_order(uint32_t bits) { return bits ^ (bits >> 31 ? 0xFFFFFFFFu : 0x80000000u); }
__device__ __forceinline__ uint32_t out_of_order(uint32_t x) { return x ^ (x >> 31 ? 0x80000000u : 0xFFFFFFFFu); }

// Keys of 32 bits. kNone is below every key, kLeast above it and none of them; coarse() keeps the order (not strictly), reaching() is the
// least key of a coarse value.
struct Key32 {
  typedef uint32_t T;
  static constexpr T kNone = 0, kLeast = 1;
  static __device__ __forceinline__ T of(float logit, int e) {  // a bf16 value above -inf
    return (in_order(__builtin_bit_cast(uint32_t, logit + 0.f)) & 0xFFFF0000u) | (uint32_t)(0xFFFF - e);
  }
  static __device__ __forceinline__ int expert(T k) { return 0xFFFF - (int)(k & 0xFFFFu); }
  static __device__ __forceinline__ float logit(T k) { return __builtin_bit_cast(float, out_of_order(k & 0xFFFF0000u) & 0xFFFF0000u); }
  static __device__ __forceinline__ T larger(T a, T b) { return max(a, b); }
  static __device__ __forceinline__ uint32_t coarse(T k) { return k; }
  static __device__ __forceinline__ T reaching(uint32_t c) { return c; }
};
struct Key64 {
  typedef double T;
  static constexpr T kNone = -__builtin_inf(), kLeast = -1e301;
  static __device__ __forceinline__ T of(double c, int e) {
    c = fmin(fmax(c + 0.0, -1e300), 1e300);  // -0 becomes 0; an infinite key would be a NaN with the number in it
    const uint64_t b = __builtin_bit_cast(uint64_t, c);
    return __builtin_bit_cast(double, (b & ~1023ull) | (uint64_t)(b >> 63 ? e : 1023 - e));
  }
  static __device__ __forceinline__ int expert(T k) {
    const uint64_t b = __builtin_bit_cast(uint64_t, k);
    return b >> 63 ? (int)(b & 1023) : 1023 - (int)(b & 1023);
  }
  static __device__ __forceinline__ double value(T k) {
    return __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, k) & ~1023ull);
  }
  static __device__ __forceinline__ float logit(T k) { return (float)value(k); }
  static __device__ __forceinline__ T larger(T a, T b) { return fmax(a, b); }
  static __device__ __forceinline__ uint32_t coarse(T k) { return in_order((uint32_t)(__builtin_bit_cast(uint64_t, k) >> 32)); }
  static __device__ __forceinline__ T reaching(uint32_t c) {
    const uint32_t hi = out_of_order(c);
    if (hi >= 0xFFF00000u) return kNone;  // the bits would be a NaN's
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | (hi >> 31 ? 0xFFFFFFFFu : 0u));
  }
};

__device__ __forceinline__ float load_logit(const uint16_t* p, int64_t at) {
  return __builtin_bit_cast(float, (uint32_t)p[at] << 16);
}
__device__ __forceinline__ float load_logit(const float* p, int64_t at) { return p[at]; }
__device__ __forceinline__ void load4(float (&x)[4], const uint16_t* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  x[0] = __builtin_bit_cast(float, u.x << 16);
  x[1] = __builtin_bit_cast(float, u.x & 0xFFFF0000u);
  x[2] = __builtin_bit_cast(float, u.y << 16);
  x[3] = __builtin_bit_cast(float, u.y & 0xFFFF0000u);
}
__device__ __forceinline__ void load4(float (&x)[4], const float* p) {
  const float4 u = *reinterpret_cast<const float4*>(p);
  x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
}

// What the host works out: each group has `lanes` neighbouring lanes, a power of two of them.
struct RouteShape {
  int lanes, size;  // of a group: lanes, experts
};

// L: the logits' type. V: experts a lane, W of them neighbours (4: loaded together). Experts of a group
// lie over its lanes in turn, W at a time; without groups (kGroups false) all over all lanes.
template <typename Key, typename L, int V, int W, bool kGroups>
__global__ __launch_bounds__(64 * kRouteWaves) void k_moe_route(RouteArgs a, RouteShape g, int first_row) {
  typedef typename Key::T T;
  constexpr bool k64 = sizeof(T) == 8;
  constexpr float kLargest = sizeof(L) == 2 ? 0x1.FEp127f : 0x1.FFFFFEp127f;  // the logits' type's
  __shared__ __attribute__((aligned(16))) T found[kRouteWaves][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int rows = a.num_rows ? min(*a.num_rows, a.T) : a.T;
  const int lanes = kGroups ? g.lanes : 64, size = kGroups ? g.size : a.E, groups = kGroups ? a.groups : 1;
  const int my_group = kGroups ? lane / lanes : 0, r = kGroups ? lane % lanes : lane;
  const L* logits = static_cast<const L*>(a.logits);
  const bool scored = k64 && (a.bias || (kGroups && a.group_top == 2));
  const bool whole = !a.sigmoid && (scored || !a.renormalize);  // the softmax's sum over all experts
  const int t = first_row + (int)blockIdx.x * kRouteWaves + w;
  if (t >= a.T) return;
  int32_t* ids = a.ids + (int64_t)t * a.topk;
  float* weights = a.weights + (int64_t)t * a.topk;
  if (t >= rows) {
    if (lane < a.topk) {
      ids[lane] = -1;
      weights[lane] = 0.f;
    }
    return;
  }
  // an expert's place in its group, and its number
  const auto place = [&](int v) { return (v / W * lanes + r) * W + v % W; };
  const auto number = [&](int v) { return my_group * size + place(v); };
  const auto has = [&](int v) { return my_group < groups && place(v) < size; };
  float x[V];  // -inf and NaN: never chosen
  const L* row = logits + t * a.stride;
#pragma unroll
  for (int v = 0; v < V; v += W) {
#pragma unroll
    for (int i = 0; i < W; ++i) x[v + i] = -__builtin_inff();
    if (has(v)) {
      if constexpr (W == 4) {
        float y[4];
        load4(y, row + number(v));
#pragma unroll
        for (int i = 0; i < 4; ++i) x[v + i] = y[i];
      } else {
        x[v] = load_logit(row, number(v));
      }
    }
  }
  float bias[V];
  if (k64 && a.bias) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      bias[v] = has(v) ? a.bias[number(v)] : 0.f;
      if (!(bias[v] > -__builtin_inff())) x[v] = -__builtin_inff();
    }
  }
  const auto masked = [&](int v) { return !(x[v] > -__builtin_inff()); };
  double top = 0, sum = 1;
  double p[V];
  if (whole || scored) {
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = masked(v) ? -__builtin_inff() : fminf(x[v], kLargest);
  }
  if (whole) {
    float m = -kLargest;
#pragma unroll
    for (int v = 0; v < V; ++v) m = fmaxf(m, x[v]);
    top = (double)__builtin_bit_cast(float, out_of_order(wave_max(in_order(__builtin_bit_cast(uint32_t, m)))));
    sum = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      p[v] = exp_of((double)x[v] - top);
      sum += p[v];
    }
    sum = wave_sum(sum);
  }
  if (scored) {
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] = a.sigmoid ? sigmoid_of((double)x[v]) : p[v] / sum;
  }
  T key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if constexpr (k64) key[v] = Key::of(a.bias ? p[v] + (double)bias[v] : (double)fminf(x[v], kLargest), number(v));
    else key[v] = Key::of(fminf(x[v], kLargest), number(v));
    if (masked(v)) key[v] = Key::kNone;
  }
  if (kGroups) {
    // each lane its group's key: the value, and of equal ones the lower group
    T best = Key::kNone;
    if constexpr (k64) {
      double one = Key64::kNone, two = Key64::kNone;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const double y = masked(v) ? Key64::kNone : a.bias || a.group_top == 1 ? Key64::value(key[v]) : p[v];
        two = fmax(two, fmin(one, y));
        one = fmax(one, y);
      }
      for (int d = 1; d < lanes; d <<= 1) {
        const double y = __shfl_xor(one, d), z = __shfl_xor(two, d);
        two = fmax(fmax(two, z), fmin(one, y));
        one = fmax(one, y);
      }
      if (a.group_top == 2 && two > Key64::kNone) one += two;
      if (one > Key64::kNone) best = Key64::of(one, my_group);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) best = max(best, key[v]);
      for (int d = 1; d < lanes; d <<= 1) best = max(best, (uint32_t)__shfl_xor((int)best, d));
      if (best) best = (best & 0xFFFF0000u) | (uint32_t)(0xFFFF - my_group);
    }
    int before = 0;
    for (int i = 0; i < a.groups; ++i) before += lane_value(best, i * lanes) > best ? 1 : 0;
    if (before >= a.topk_groups) {
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = Key::kNone;
    }
  }
  // the bound
  T mine = key[0];
#pragma unroll
  for (int v = 1; v < V; ++v) mine = Key::larger(mine, key[v]);
  const uint32_t c = Key::coarse(mine);
  uint32_t lo = 0, hi = wave_max(c);
  lo = ~wave_max(~c);
  for (int i = 0; i < kBisections && lo < hi; ++i) {
    const uint32_t mid = lo + (hi - lo + 1) / 2;
    const int n = (int)__popcll(__ballot(c >= mid));
    if (n < a.topk) {
      hi = mid - 1;
    } else {
      lo = mid;
      if (n <= a.topk + a.topk / 4) break;
    }
  }
  const T bound = Key::larger(Key::reaching(lo), Key::kLeast);
  // what reaches it: how many of each lane's, and where they go
  int mine_n = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) mine_n += key[v] >= bound ? 1 : 0;
  const int upto = (int)wave_scan((uint32_t)mine_n), n = (int)lane_value((uint32_t)upto, 63);
  T chosen = Key::kNone;
  int rank = lane;
  if (n <= 64) {
    found[w][lane] = Key::kNone;
    int at = upto - mine_n;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (key[v] >= bound) found[w][at++] = key[v];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // a wave's LDS accesses are in order
    chosen = found[w][lane];
    int before = 0;
    for (int i = 0; i < n; i += 4) {  // 16 bytes or 32 of the list, the same to every lane
      const T k0 = found[w][i], k1 = found[w][i + 1], k2 = found[w][i + 2], k3 = found[w][i + 3];
      before += (k0 > chosen) + (k1 > chosen) + (k2 > chosen) + (k3 > chosen);
    }
    if (lane < n) rank = before;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  } else {
    for (int i = 0; i < a.topk; ++i) {
      T best = key[0];
#pragma unroll
      for (int v = 1; v < V; ++v) best = Key::larger(best, key[v]);
      best = wave_max(best);
      if (lane == i) chosen = best;
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = key[v] == best ? Key::kNone : key[v];
    }
  }
  // weights
  const bool is = rank < a.topk && chosen > Key::kNone;
  int id = -1;
  double s = 0;
  double l = Key64::kNone;
  if (is) {
    id = Key::expert(chosen);
    l = (double)(k64 && a.bias ? fminf(load_logit(row, id), kLargest) : Key::logit(chosen));
  }
  if (!a.sigmoid && !whole) top = lane_value(l, __builtin_ctzll(__ballot(rank == 0)));  // of the first, or none
  if (is) {
    s = a.sigmoid ? sigmoid_of(l) : exp_of(l - top);
    if (whole) s /= sum;
  }
  if (a.renormalize) {
    const double all = wave_sum(s);
    s = all > 0 ? s / all : 0;
  }
  if (rank < a.topk) {
    ids[rank] = id;
    weights[rank] = (float)(s * (double)a.scale);
  }
}

template <typename Key, typename L, int V, int W>
hipError_t route(const RouteArgs& a, const RouteShape& g, hipStream_t st) {
  constexpr int kMost = 1 << 22;  // rows of a launch, which holds fewer than 2^32 threads
  for (int64_t first = 0; first < a.T; first += kMost) {
    const dim3 grid((unsigned)((min(a.T - first, (int64_t)kMost) + kRouteWaves - 1) / kRouteWaves)), block(64 * kRouteWaves);
    if (a.groups > 1) hipLaunchKernelGGL((k_moe_route<Key, L, V, W, true>), grid, block, 0, st, a, g, (int)first);
    else hipLaunchKernelGGL((k_moe_route<Key, L, V, W, false>), grid, block, 0, st, a, g, (int)first);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename Key, typename L>
hipError_t route(const RouteArgs& a, hipStream_t st) {
  RouteShape g = {64, a.E / a.groups};
  while (g.lanes > 64 / a.groups) g.lanes /= 2;
  const int each = (g.size + g.lanes - 1) / g.lanes, fours = (g.size + 4 * g.lanes - 1) / (4 * g.lanes);
  // four experts in one load where they lie so and it takes no more registers
  const auto on = [](uint64_t x) { return x % (4 * sizeof(L)) == 0; };
  const bool w4 = g.size % 4 == 0 && on((uint64_t)a.logits) && on((uint64_t)a.stride * sizeof(L)) && each > 2;
  if (w4 && fours <= 4) {
    if (fours == 1) return route<Key, L, 4, 4>(a, g, st);
    if (fours == 2) return route<Key, L, 8, 4>(a, g, st);
    return route<Key, L, 16, 4>(a, g, st);
  }
  if (each == 1) return route<Key, L, 1, 1>(a, g, st);
  if (each == 2) return route<Key, L, 2, 1>(a, g, st);
  if (each <= 4) return route<Key, L, 4, 1>(a, g, st);
  if (each <= 8) return route<Key, L, 8, 1>(a, g, st);
  if (each <= 16) return route<Key, L, 16, 1>(a, g, st);
  return route<Key, L, 32, 1>(a, g, st);
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
  if (a.f32) return route<Key64, float>(a, st);
  if (a.bias || (a.groups > 1 && a.group_top == 2)) return route<Key64, uint16_t>(a, st);
  return route<Key32, uint16_t>(a, st);
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
