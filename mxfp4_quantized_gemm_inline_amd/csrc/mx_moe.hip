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
// Bound: instruction issue (the floor of 16411 tokens x 896 bf16 logits is 6.4 us of HBM): 17.2 us, 1.8 TB/s,
// where the largest taken topk times took 144; 64-bit keys take 24.6 there, and 20.6 for FP32 logits, 46 with
// a bias; the bound bisected down to exactly topk lanes 0.7 us more. 64 experts 8.9 us. 256 experts in 8 groups
// with a bias 4099 tokens 9.9 us. 16 tokens 4.4 us: a launch and the chain of one token.

constexpr int kRouteWaves = 4;
constexpr int kList = 64;        // keys that are ranked, at most
// At most. 11 / 14 / 18: 4099 tokens of 256 experts in 8 groups 11.8 / 9.9 / 9.8 us, FP32 logits of 896 experts,
// 16411 tokens, 24.1 / 20.6 / 20.6 (fewer leave lists too long to rank), bf16 ones 17.2 at each.
constexpr int kBisections = 14;

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
// r^13, whose next term is below 2^-57. Its terms come from memory by scalar loads: as literals each
// would take instructions of its own in every use.
__constant__ double kExpTerms[12] = {1.0 / 6227020800.0, 1.0 / 479001600.0, 1.0 / 39916800.0, 1.0 / 3628800.0, 1.0 / 362880.0,
                                     1.0 / 40320.0, 1.0 / 5040.0, 1.0 / 720.0, 1.0 / 120.0, 1.0 / 24.0, 1.0 / 6.0, 0.5};
__device__ __forceinline__ double exp_of(double x) {
  x = fmax(x, -800.0);  // below the least subnormal
  const double n = rint(x * 1.44269504088896340736);
  const double r = fma(-n, 2.31904681384629955842e-17, fma(-n, 0.693147180559945286227, x));
  double y = kExpTerms[0];
#pragma unroll
  for (int i = 1; i < 12; ++i) y = fma(y, r, kExpTerms[i]);
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
  static constexpr T kNone = -__builtin_inf(), kLeast = -0x1p200;  // c is finite: at most a sum of two FP32 numbers and two scores
  static __device__ __forceinline__ T of(double c, int e) {
    const uint64_t b = __builtin_bit_cast(uint64_t, c + 0.0);  // -0 becomes 0
    return __builtin_bit_cast(double, (b & ~1023ull) | (uint64_t)(b >> 63 ? e : 1023 - e));
  }
  static __device__ __forceinline__ int expert(T k) {
    const uint64_t b = __builtin_bit_cast(uint64_t, k);
    return b >> 63 ? (int)(b & 1023) : 1023 - (int)(b & 1023);
  }
  static __device__ __forceinline__ double value(T k) {
    return __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, k) & ~1023ull);
  }
  // Rounded to the bits that keys hold. Sums are, where logits and biases that give equal ones in exact
  // arithmetic (sigmoids of x and -x, a bias on the one or the other) may differ by an FP64 rounding.
  static __device__ __forceinline__ double rounded(double c) {
    return __builtin_bit_cast(double, (__builtin_bit_cast(uint64_t, c) + 512) & ~1023ull);
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
  __shared__ __attribute__((aligned(16))) T found[kRouteWaves][kList];
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
      bias[v] = fminf(bias[v], 0x1.FFFFFEp127f);
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
  if (scored && a.sigmoid) {
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] = sigmoid_of((double)x[v]);
  } else if (scored) {
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] /= sum;
  }
  T key[V];
  double one = Key64::kNone, two = Key64::kNone;  // of a lane's experts the two largest that count for its group
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if constexpr (k64) {
      const double c = a.bias ? p[v] + (double)bias[v] : (double)fminf(x[v], kLargest);
      key[v] = Key::of(c, number(v));
      if (kGroups) {
        // scores or c as they are: of two c that cancel nothing may be left of their keys' 42 bits
        const double y = masked(v) ? Key64::kNone : a.bias || a.group_top == 1 ? c : p[v];
        two = fmax(two, fmin(one, y));
        one = fmax(one, y);
      }
    } else {
      key[v] = Key::of(fminf(x[v], kLargest), number(v));
    }
    if (masked(v)) key[v] = Key::kNone;
  }
  if (kGroups) {
    // each lane its group's key: the value, and of equal ones the lower group
    T best = Key::kNone;
    if constexpr (k64) {
      for (int d = 1; d < lanes; d <<= 1) {
        const double y = __shfl_xor(one, d), z = __shfl_xor(two, d);
        two = fmax(fmax(two, z), fmin(one, y));
        one = fmax(one, y);
      }
      if (a.group_top == 2 && two > Key64::kNone) one += two;
      if (one > Key64::kNone) best = Key64::of(Key64::rounded(one), my_group);
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
  // The lanes that reach the bound may be a quarter more than topk, or as many as have kList keys together. A
  // quarter alone: 64, 128, 256 experts, topk 6 to 8, 16411 tokens 12.8, 13.3, 13.7 us against 8.9, 11.5,
  // 12.7; no bound for one key a lane, longer lists, 10.0 against 8.9.
  const int most = max(a.topk + a.topk / 4, kList / V);
  for (int i = 0; i < kBisections && lo < hi; ++i) {
    const uint32_t mid = lo + (hi - lo + 1) / 2;
    const int n = (int)__popcll(__ballot(c >= mid));
    if (n < a.topk) {
      hi = mid - 1;
    } else {
      lo = mid;
      if (n <= most) break;
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
  if (n <= kList) {
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
    // 32 experts a lane only where groups, no power of two of them, leave lanes over
    if (V == 32 || a.groups > 1) hipLaunchKernelGGL((k_moe_route<Key, L, V, W, true>), grid, block, 0, st, a, g, (int)first);
    else if constexpr (V < 32) hipLaunchKernelGGL((k_moe_route<Key, L, V, W, false>), grid, block, 0, st, a, g, (int)first);
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
  // Four experts in one load where they lie so: 16411 x 896 17.2 us against 24.3 one by one, 256 tokens 5.0
  // against 5.9; 16384 of 1000 experts in 5 groups 29 against 42, with a bias 121 against 144. Of 64 and 128
  // experts (one or two a lane) one by one 8.5 against 9.7, 11.0 against 11.9.
  const auto on = [](uint64_t x) { return x % (4 * sizeof(L)) == 0; };
  const bool w4 = g.size % 4 == 0 && on((uint64_t)a.logits) && on((uint64_t)a.stride * sizeof(L)) && each > 2;
  if (w4) {
    if (fours == 1) return route<Key, L, 4, 4>(a, g, st);
    if (fours == 2) return route<Key, L, 8, 4>(a, g, st);
    if (fours <= 4) return route<Key, L, 16, 4>(a, g, st);
    return route<Key, L, 32, 4>(a, g, st);
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
// A stable counting sort. A wave has a part of the places, in order, and a row of counters in LDS, which
// it advances 64 places at a time, lanes of one expert ranked by ballots over the number's bits.
// Up to kSortAll places one launch does it: each workgroup counts all places, what lies before its own
// and behind them too, so that none waits for another. Beyond, a first launch ranks each place among its
// workgroup's of the same expert (to token_rows) and counts those, a last one adds where they start; the
// counts before a workgroup's are summed up there, or, where there are more than kSortSums workgroups,
// by a launch between the two.
// Bound: latency, a chain of loads, ballots, LDS counters and barriers a launch, and the launches. 256
// places of 896 experts 4.8 us; 65536 11.7 (5.8 + 5.6 and the gap; floor 0.2); 524296 16.0 (floor 1.3);
// 1600000 40 (15 + 4 + 18; floor 4: the rows' scattered words).
// kSortAll: 16384 places 9.9 us in one launch against 12.0 in two, 32768 13.1 against 10.8, 65536 19.9
// against 11.7 (62 where all are one expert's: LDS counters serialize). kSortSums: 131072 places (64
// workgroups) 13.7 us summed up there, 14.5 with the launch between; 160000 17.5 against 15.2.

constexpr int kSortAll = 16384;
constexpr int kSortChunk = 2048;   // places of a workgroup of the others, or a multiple
constexpr int kSortChunks = 512;   // workgroups of those, at most. 512 / 1024 / 256: 1600000 places 40.3 / 43.5 / 40.8 us, 524296 16.0 / 16.0 / 18.2
constexpr int kSortSums = 64;
constexpr int kEach = 8;           // places that a lane loads ahead in the one launch
// Waves of a workgroup that ranks, and places a lane. 8 / 4 / 16 waves: 65536 places 11.8 / 13.1 / 11.5 us,
// 320000 17.6 / 18.9 / 17.8, 1600000 43.9 / 45.3 / 46.9.
constexpr int kRankWaves = 8, kRankEach = kSortChunk / 64 / kRankWaves;
inline int sort_chunk(int64_t N) {
  const int64_t each = (N + kSortChunks - 1) / kSortChunks;
  return (int)((max(each, (int64_t)kSortChunk) + kSortChunk - 1) / kSortChunk * kSortChunk);
}
inline int sort_chunks(int64_t N) { return (int)((N + sort_chunk(N) - 1) / sort_chunk(N)); }

// The expert of place n among this call's, -1 for others'.
__device__ __forceinline__ int local_expert(const SortArgs& a, int n) {
  const uint32_t e = (uint32_t)a.ids[n] - (uint32_t)a.first;
  return e < (uint32_t)a.E ? (int)e : -1;
}

// Inclusive sum over the workgroup's threads; part: a word a wave.
template <int W>
__device__ __forceinline__ int group_scan(int x, int32_t* part) {
  const int upto = (int)wave_scan((uint32_t)x), w = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 63) part[w] = upto;
  __syncthreads();
  int base = 0;
  for (int i = 0; i < w; ++i) base += part[i];
  return upto + base;
}

// at: each one's place among those of its expert (e, or -1 for none) that the wave has had, whose number
// cnt[] holds. First lanes of the same expert by ballots over the bits of its number, then counters, then
// what they were: none waits for another's way through LDS.
template <int K>
__device__ __forceinline__ void next_places(int (&at)[K], const int (&e)[K], int bits, int32_t* cnt) {
  uint64_t same[K];
#pragma unroll
  for (int i = 0; i < K; ++i) same[i] = __ballot(e[i] >= 0);
#pragma unroll 1
  for (int b = 0; b < bits; ++b)
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const bool one = e[i] >> b & 1;
      same[i] &= __ballot(one) ^ (one ? 0 : ~0ull);
    }
  int leader[K], base[K];
#pragma unroll
  for (int i = 0; i < K; ++i) {
    at[i] = __builtin_amdgcn_mbcnt_hi((uint32_t)(same[i] >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)same[i], 0));
    leader[i] = same[i] ? (int)__builtin_ctzll(same[i]) : 0;
    base[i] = e[i] >= 0 && at[i] == 0 ? (int)__popcll(same[i]) : 0;
  }
#pragma unroll
  for (int i = 0; i < K; ++i)
    if (base[i]) base[i] = atomicAdd(&cnt[e[i]], base[i]);
#pragma unroll
  for (int i = 0; i < K; ++i) at[i] = e[i] >= 0 ? __shfl(base[i], leader[i]) + at[i] : -1;
}

__global__ __launch_bounds__(1024) void k_moe_sort(SortArgs a) {
  constexpr int W = 16, kThreads = 64 * W, kSteps = 2, each = 64 * kSteps, share = W * each;  // places of a wave, of a workgroup
  __shared__ int32_t cnt[W][1024];
  __shared__ int32_t before[1024], behind[1024];
  __shared__ int32_t part[W];
  const int w = threadIdx.x >> 6;
  const int n0 = (int)blockIdx.x * share, n1 = min(a.N, n0 + share);
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    before[e] = behind[e] = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) cnt[i][e] = 0;
  }
  __syncthreads();
  for (int b0 = 0; b0 < a.N; b0 += kThreads * kEach) {
    int e[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int n = b0 + kThreads * i + (int)threadIdx.x;
      e[i] = n < a.N ? local_expert(a, n) : -1;
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int n = b0 + kThreads * i + (int)threadIdx.x;
      if (e[i] >= 0) atomicAdd(n < n0 ? &before[e[i]] : n >= n1 ? &behind[e[i]] : &cnt[(n - n0) / each][e[i]], 1);
    }
  }
  __syncthreads();
  const int e = threadIdx.x;  // an expert a thread
  int all = 0;
  if (e < a.E) {
    all = before[e] + behind[e];
#pragma unroll
    for (int j = 0; j < W; ++j) all += cnt[j][e];
  }
  const int run = group_scan<W>(all, part) - all;
  if (e < a.E) {
    if (blockIdx.x == 0) a.offsets[e] = run;
    int base = run + before[e];
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const int c = cnt[j][e];
      cnt[j][e] = base;
      base += c;
    }
  }
  int R = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) R += part[i];
  if (blockIdx.x == 0 && e == 0) a.offsets[a.E] = R;
  __syncthreads();
  int own[kSteps], at[kSteps];
  const int m0 = n0 + w * each + (int)(threadIdx.x & 63);
#pragma unroll
  for (int i = 0; i < kSteps; ++i) own[i] = m0 + 64 * i < n1 ? local_expert(a, m0 + 64 * i) : -1;
  next_places(at, own, a.bits, cnt[w]);
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int n = m0 + 64 * i;
    if (at[i] >= 0) a.row_token[at[i]] = n / a.topk;
    if (n < n1) a.token_rows[n] = at[i];
  }
  for (int r = R + (int)(blockIdx.x * kThreads + threadIdx.x); r < a.N; r += (int)gridDim.x * kThreads) a.row_token[r] = -1;
}

// token_rows: each place's number among this workgroup's of its expert; counts: how many of each,
// [chunks][E], or with kScan [E][chunks].
template <bool kScan>
__global__ __launch_bounds__(64 * kRankWaves) void k_moe_sort_rank(SortArgs a, int chunk, int32_t* counts) {
  __shared__ int32_t cnt[kRankWaves][1024];
  __shared__ int32_t sums[1024];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  for (int e = threadIdx.x; e < a.E; e += 64 * kRankWaves) sums[e] = 0;
  const int64_t n0 = (int64_t)blockIdx.x * chunk, n1 = min((int64_t)a.N, n0 + chunk);
  for (int64_t s0 = n0; s0 < n1; s0 += kSortChunk) {
    int e[kRankEach], at[kRankEach];
#pragma unroll
    for (int i = 0; i < kRankEach; ++i) {
      const int64_t n = s0 + (w * kRankEach + i) * 64 + lane;
      e[i] = n < n1 ? local_expert(a, (int)n) : -1;
    }
    for (int i = lane; i < a.E; i += 64) cnt[w][i] = 0;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // a wave's LDS accesses are in order
    next_places(at, e, a.bits, cnt[w]);
    __syncthreads();
    for (int i = threadIdx.x; i < a.E; i += 64 * kRankWaves) {
      int base = sums[i];
#pragma unroll
      for (int j = 0; j < kRankWaves; ++j) {
        const int c = cnt[j][i];
        cnt[j][i] = base;
        base += c;
      }
      sums[i] = base;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRankEach; ++i) {
      const int64_t n = s0 + (w * kRankEach + i) * 64 + lane;
      if (n < n1) a.token_rows[n] = e[i] >= 0 ? cnt[w][e[i]] + at[i] : -1;
    }
  }
  for (int e = threadIdx.x; e < a.E; e += 64 * kRankWaves) counts[kScan ? (int64_t)e * gridDim.x + blockIdx.x : (int64_t)blockIdx.x * a.E + e] = sums[e];
}

// A wave per expert: counts become the sums before them, totals: [E] their sums.
__global__ __launch_bounds__(64) void k_moe_sort_scan(int32_t* counts, int chunks, int32_t* totals) {
  int32_t* mine = counts + (int64_t)blockIdx.x * chunks;
  int base = 0;
  for (int c0 = 0; c0 < chunks; c0 += 64) {
    const int c = c0 + (int)threadIdx.x, x = c < chunks ? mine[c] : 0;
    const int upto = (int)wave_scan((uint32_t)x);
    if (c < chunks) mine[c] = base + upto - x;
    base += (int)lane_value((uint32_t)upto, 63);
  }
  if (threadIdx.x == 0) totals[blockIdx.x] = base;
}

template <bool kScan>
__global__ __launch_bounds__(1024) void k_moe_sort_place(SortArgs a, int chunk, const int32_t* counts, const int32_t* totals) {
  __shared__ int32_t start[1024];
  __shared__ int32_t part[16];
  const int e = threadIdx.x;  // an expert a thread
  int all = 0, before = 0;
  if (e < a.E) {
    if (kScan) {
      all = totals[e];
      before = counts[(int64_t)e * gridDim.x + blockIdx.x];
    } else {
#pragma unroll 16
      for (int c = 0; c < (int)gridDim.x; ++c) {
        const int x = counts[c * a.E + e];
        before += c < (int)blockIdx.x ? x : 0;
        all += x;
      }
    }
  }
  const int run = group_scan<16>(all, part) - all;
  if (e < a.E) {
    start[e] = run + before;
    if (blockIdx.x == 0) a.offsets[e] = run;
  }
  int R = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) R += part[i];
  if (blockIdx.x == 0 && e == 0) a.offsets[a.E] = R;
  __syncthreads();
  const int64_t n0 = (int64_t)blockIdx.x * chunk, n1 = min((int64_t)a.N, n0 + chunk);
  for (int64_t n = n0 + threadIdx.x; n < n1; n += 1024) {
    const int x = local_expert(a, (int)n);
    if (x >= 0) {
      const int row = start[x] + a.token_rows[n];
      a.row_token[row] = (int)n / a.topk;
      a.token_rows[n] = row;
    }
  }
  for (int64_t r = (int64_t)R + blockIdx.x * 1024 + threadIdx.x; r < a.N; r += (int64_t)gridDim.x * 1024) a.row_token[r] = -1;
}

}  // namespace

hipError_t launch_moe_route(const RouteArgs& a, hipStream_t st) {
  if (a.f32) return route<Key64, float>(a, st);
  if (a.bias || (a.groups > 1 && a.group_top == 2)) return route<Key64, uint16_t>(a, st);
  return route<Key32, uint16_t>(a, st);
}

size_t moe_sort_workspace_bytes(int64_t N, int64_t E) {
  return N <= kSortAll ? 0 : (size_t)(E * (sort_chunks(N) + 1)) * 4;
}

hipError_t launch_moe_sort(const SortArgs& a, void* workspace, hipStream_t st) {
  if (a.N <= kSortAll) {
    hipLaunchKernelGGL(k_moe_sort, dim3((unsigned)max((a.N + 2047) / 2048, 1)), dim3(1024), 0, st, a);
    return hipGetLastError();
  }
  const int chunk = sort_chunk(a.N), chunks = sort_chunks(a.N);
  int32_t* totals = static_cast<int32_t*>(workspace);
  int32_t* counts = totals + a.E;
  const dim3 grid((unsigned)chunks), block(64 * kRankWaves);
  const bool scan = chunks > kSortSums;
  if (scan) hipLaunchKernelGGL(k_moe_sort_rank<true>, grid, block, 0, st, a, chunk, counts);
  else hipLaunchKernelGGL(k_moe_sort_rank<false>, grid, block, 0, st, a, chunk, counts);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (scan) {
    hipLaunchKernelGGL(k_moe_sort_scan, dim3((unsigned)a.E), dim3(64), 0, st, counts, chunks, totals);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_moe_sort_place<true>, grid, dim3(1024), 0, st, a, chunk, (const int32_t*)counts, (const int32_t*)totals);
  } else {
    hipLaunchKernelGGL(k_moe_sort_place<false>, grid, dim3(1024), 0, st, a, chunk, (const int32_t*)counts, (const int32_t*)nullptr);
  }
  return hipGetLastError();
}

}  // namespace mx
