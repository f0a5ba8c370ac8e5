// mx_kv_append.hip - norms of each head, rotation by position, queries out and keys and values
// into the paged MXFP4 cache, in one pass.
#include "mx_device.h"
#include "mx_kv.h"

namespace mx {
namespace {

// One launch, workgroups of three kinds: queries, a wave to a row (a load is 512 elements of it, four
// heads of 128), keys and values, a workgroup to 16 rows of a head of 128 (two heads of 64, 8 rows of a
// head of 256), so that tokens that lie side by side in the cache are written together. A thread has 8
// elements of a row, at the same place in every head that it goes through, so that its weights and angles
// are one set of registers: with A = weight * cos and B = +-(weight of the other element) * sin an element
// is r * (x A + other B), r = 1 / sqrt(mean + eps).
// Bound: HBM. 16411 rows of 32 + 8 heads of 128: 85 to 90 us, 4.0 TB/s (floor 72 at a copy's 4.9), of 16 + 4 heads
// of 256, as many bytes, 93; the queries alone 51 us, keys and values alone 25 (FP64 issue; floor 17.4).
// 101 rows 5.2 us: a launch, positions, angles, heads. 16411 rows of 1, 3, 5 query heads of 128: 11.7,
// 13.0, 16.0 us, a wave a row whatever it holds. Queries in tiles of 16 rows x 256 bytes as keys are: 75 us
// where they took 58. All three in one workgroup kind, 16 rows of all heads: 101 us, the registers of keys for all.
template <int D>
struct AppendTile {  // of keys and values
  static constexpr int kWidth = D < 128 ? 128 : D;  // elements of a row at a time
  static constexpr int kLanes = kWidth / 8;         // threads of a row
  static constexpr int kRows = 256 / kLanes;
};
constexpr int kQueryWidth = 512, kQueryRows = 4;  // elements of a row at a time, rows of a workgroup

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __builtin_bit_cast(float, w[i] << 16);
    x[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&y)[8]) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){y[2 * i], y[2 * i + 1]}, bf16x2));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int kControl>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, kControl, 0xF, 0xF, true);
}
template <int kControl>
__device__ __forceinline__ float dpp(float x) {
  return __builtin_bit_cast(float, dpp<kControl>(__builtin_bit_cast(uint32_t, x)));
}
template <int kControl>
__device__ __forceinline__ double dpp(double x) {
  const uint2 u = __builtin_bit_cast(uint2, x);
  return __builtin_bit_cast(double, make_uint2(dpp<kControl>(u.x), dpp<kControl>(u.y)));
}
constexpr int kOneApart = 0xB1, kTwoApart = 0x4E, kFlip8 = 0x141, kFlip16 = 0x140;  // lanes that DPP brings together

// The sum of a head's squares, over the D / 8 lanes that hold it.
template <int D, typename F>
__device__ __forceinline__ F sum_squares(const float (&x)[8]) {
  F s = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fma((F)x[i], (F)x[i], s);
  s += dpp<kOneApart>(s);
  s += dpp<kTwoApart>(s);
  s += dpp<kFlip8>(s);
  if (D >= 128) s += dpp<kFlip16>(s);
  if (D == 256) s += __shfl_xor(s, 16);
  return s;
}

// 1 / sqrt(mean + eps), of 2^-126 at least: finite in FP32, and a head of zeros stays 0 also without eps.
template <int D>
__device__ __forceinline__ double exact_norm(const float (&x)[8], float eps) {
  return rsqrt(fmax(sum_squares<D, double>(x) * (1.0 / D) + (double)eps, 0x1p-126));
}
// Normed and turned queries, y = (x A + o B) n, in FP32 where nothing on the way can leave its range. The norm is
// then off by at most 10 u (u = 2^-24: half of the sum's 8 + 5 roundings, the product, the sum with eps,
// the root's step). Below: with mean + eps of kLeastMean n is 2^14 at most, and what products below the normal
// numbers lose, 2^-150 each, is less than bf16 holds. Above: sums of squares under 1e38 and coefficients
// of up to kWide (wide: some are larger) give terms under 2^124. All else is FP64's: heads whose root mean square is
// below 6e-5 where eps is below 4e-9 (with such an eps also loads that a row's heads do not fill: the lanes past them
// hold zeros), or above 1e18, and weights or scales of more than 1e18.
constexpr float kLeastMean = 0x1p-28f, kWide = 0x1p60f;
template <int D>
__device__ __forceinline__ void normed(float (&y)[8], const float (&x)[8], const float (&o)[8], const float (&A)[8], const float (&B)[8],
                                       float eps, bool wide) {
  const float s = sum_squares<D, float>(x), mean = fmaf(s, 1.f / D, eps), n = __builtin_amdgcn_rsqf(mean);
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = fmaf(x[i], A[i], o[i] * B[i]) * n;
  const bool inside = mean >= kLeastMean && s < 1e38f && !wide;
  if (__any(!inside)) {  // all lanes, as they sum together
    const double m = exact_norm<D>(x, eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float z = (float)(fma((double)x[i], (double)A[i], (double)o[i] * (double)B[i]) * m);
      if (!inside) y[i] = z;
    }
  }
}

// cos and sin of pos * freq. The product is formed in FP64 and that number is the angle: it is reduced
// by multiples of pi / 2 in two steps of fused products (pi / 2 as a sum of two FP64 numbers; what is
// left is off by 2^-52 up to the largest position), then the series up to x^17 and x^16, whose next
// terms are below 2^-58 at pi / 4. Their terms come from memory by scalar loads, ahead of the position:
// as literals they are most of the code that a short call has to fetch.
struct Turn {
  double c, s;
};
__constant__ double kSeries[16] = {1.0 / 355687428096000.0, -1.0 / 1307674368000.0, 1.0 / 6227020800.0, -1.0 / 39916800.0,
                                   1.0 / 362880.0, -1.0 / 5040.0, 1.0 / 120.0, -1.0 / 6.0,
                                   1.0 / 20922789888000.0, -1.0 / 87178291200.0, 1.0 / 479001600.0, -1.0 / 3628800.0,
                                   1.0 / 40320.0, -1.0 / 720.0, 1.0 / 24.0, -0.5};
__device__ __forceinline__ Turn cos_sin(int pos, float freq) {
  const double a = (double)pos * (double)freq;
  const double n = rint(a * 0.63661977236758134308);  // below 2^31 for any position
  const double x = fma(-n, 6.12323399573676603587e-17, fma(-n, 1.57079632679489661923, a)), z = x * x;
  double s = kSeries[0], c = kSeries[8];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    s = fma(s, z, kSeries[i]);
    c = fma(c, z, kSeries[8 + i]);
  }
  s = fma(s * z, x, x);
  c = fma(c, z, 1.0);
  const int q = (int)n & 3;
  const double co = q & 1 ? s : c, si = q & 1 ? c : s;
  return {(q + 1) & 2 ? -co : co, q & 2 ? -si : si};
}

union __attribute__((aligned(16))) Shared {
  Turn turn[16 * 64];  // of each row's angles: [rows][D / 2]
  struct {
    uint32_t words[2][256 + 16];  // V's codes of a head, [kRows][kLanes + 1]; the next head's in the other half
    int64_t slot[16];             // of each row; -1: writes nothing
  } v;
};

// What a thread knows of its place.
struct Place {
  int pos;    // its row's position
  int d, od;  // its 8 elements' place in their head, and of those that they are turned with
  int other;  // the lane that has those
  int angle;  // the number of its first angle; past the angles where its elements are not turned
};
template <int D, bool kPairs>
__device__ __forceinline__ Place place_of(int c, int pos, int rot) {
  Place me = {pos, 8 * c % D, 8 * c % D, (int)threadIdx.x & 63, rot / 2};
  if (me.d < rot) {
    if (!kPairs) {
      me.od = me.d < rot / 2 ? me.d + rot / 2 : me.d - rot / 2;
      me.other += (me.od - me.d) / 8;
    }
    me.angle = kPairs ? me.d / 2 : min(me.d, me.od);
  }
  return me;
}

// Its weights, and those of the elements that its own are turned with, with the sign of the sine; 0 past
// the elements that are turned.
template <bool kPairs>
__device__ __forceinline__ void weights_of(float (&wx)[8], float (&wo)[8], const float* weight, const Place& me, int rot) {
  typedef float f32x4 __attribute__((ext_vector_type(4), aligned(4)));
  f32x4 u[4] = {{1, 1, 1, 1}, {1, 1, 1, 1}, {1, 1, 1, 1}, {1, 1, 1, 1}};
  if (weight) {
    u[0] = *reinterpret_cast<const f32x4*>(weight + me.d);
    u[1] = *reinterpret_cast<const f32x4*>(weight + me.d + 4);
    u[2] = *reinterpret_cast<const f32x4*>(weight + me.od);
    u[3] = *reinterpret_cast<const f32x4*>(weight + me.od + 4);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int j = kPairs ? i ^ 1 : i;
    wx[i] = u[i / 4][i % 4];
    wo[i] = u[2 + j / 4][j % 4];
    // of two neighbours the first takes -sin of the second; of two halves the first
    if (kPairs ? !(i & 1) : me.d < me.od) wo[i] = -wo[i];
    if (me.d >= rot) wo[i] = 0.f;
  }
}

// 8 elements and those that they are turned with (past those that are turned themselves: x * 0 of its own
// sign leaves -0 what it is).
template <bool kPairs>
__device__ __forceinline__ void elements_of(float (&x)[8], float (&o)[8], const uint4& u, const Place& me, int rot) {
  unpack8(u, x);
  if (kPairs) {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = me.d < rot ? x[i ^ 1] : x[i];
  } else {
    unpack8(make_uint4(__shfl(u.x, me.other), __shfl(u.y, me.other), __shfl(u.z, me.other), __shfl(u.w, me.other)), o);
  }
}

// A and B of the comment at the top: the `lanes` lanes of a row, all of one wave, work its angles out (past
// them cos 1 and sin 0) into `turn` and take theirs from there. F: float for queries, double for keys.
template <int D, bool kPairs, typename F>
__device__ __forceinline__ void coefficients(F (&A)[8], F (&B)[8], const KvAppendArgs& a, Turn* turn, int lane, int lanes,
                                             const float* weight, const Place& me) {
  float wx[8], wo[8];
  weights_of<kPairs>(wx, wo, weight, me, a.rot);
  for (int f = lane; f < D / 2; f += lanes) {
    Turn x = {1.0, 0.0};
    if (f < a.rot / 2) {
      x = cos_sin(me.pos, a.inv_freq[f]);
      x.c *= (double)a.rope_scale;
      x.s *= (double)a.rope_scale;
    }
    turn[f] = x;
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // a wave's LDS accesses are in order
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const Turn z = turn[me.angle + (kPairs ? i / 2 : i)];
    A[i] = (F)((double)wx[i] * z.c);
    B[i] = (F)((double)wo[i] * z.s);
  }
}

template <int D, bool kPairs>
__device__ __forceinline__ void append_queries(const KvAppendArgs& a, Shared& sh, int t, int first, int step) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  if (t >= a.T) return;
  const int pos = a.positions[t];
  const uint16_t* src = a.q + t * a.q_stride + 8 * lane;
  uint16_t* dst = a.q_out + t * a.q_out_stride + 8 * lane;
  const int limit = a.Hq * D - 8 * lane;
  int e = first * kQueryWidth;
  uint4 next = make_uint4(0, 0, 0, 0);
  if (e < limit) next = *reinterpret_cast<const uint4*>(src + e);
  if (pos < 0) return;
  const Place me = place_of<D, kPairs>(lane, pos, a.rot);
  float A[8], B[8];
  coefficients<D, kPairs, float>(A, B, a, sh.turn + w * (D / 2), lane, 64, a.q_weight, me);
  float largest = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) largest = fmaxf(largest, fmaxf(fabsf(A[i]), fabsf(B[i])));
  const bool wide = largest > kWide;
  for (; e < a.Hq * D; e += step * kQueryWidth) {
    const uint4 x4 = next;
    const int e2 = e + step * kQueryWidth;
    if (e2 < limit) next = *reinterpret_cast<const uint4*>(src + e2);
    float x[8], o[8], y[8];
    elements_of<kPairs>(x, o, x4, me, a.rot);
    if (a.q_weight) {
      normed<D>(y, x, o, A, B, a.eps, wide);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = fmaf(x[i], A[i], o[i] * B[i]);
    }
    if (e < limit) *reinterpret_cast<uint4*>(dst + e) = pack8(y);
  }
}

// 8 FP32 elements' codes at a block's scale byte, as quant8.
__device__ __forceinline__ uint32_t quant8_f32(const float (&f)[8], uint32_t s) {
  const float sc = __builtin_bit_cast(float, s ? s << 23 : 0x00400000u);
  uint32_t r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0, f[0], f[1], sc, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[2], f[3], sc, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[4], f[5], sc, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[6], f[7], sc, 3);
}
__device__ __forceinline__ uint32_t block_max(uint32_t x) {  // of four lanes, two 16-bit halves
  x = max_halves(x, dpp<kOneApart>(x));
  return max_halves(x, dpp<kTwoApart>(x));
}
__device__ __forceinline__ uint32_t field_of(float x) { return __builtin_bit_cast(uint32_t, x) >> 23; }  // of x >= 0
__device__ __forceinline__ uint32_t scale_byte(uint32_t field) { return field > 2u ? field - 2u : 0u; }

// Codes of 8 keys, and the scale byte of their block. In FP64, which this chip adds and multiplies as fast
// as FP32: a key next to a border of the quantizer goes by its exact value, and the cache's bytes do not
// turn on the order of roundings. FP32 with a bound on its error, and FP64 only for keys within it of a
// border, was slower: 30 us against 28 for 16411 rows, and 8 against 4.9 for 101, where some wave has to
// fetch the seldom path's instructions from memory.
template <int D, bool kPairs>
__device__ __forceinline__ uint32_t key_codes(const KvAppendArgs& a, const uint4& k4, const double (&A)[8], const double (&B)[8],
                                              const Place& me, uint32_t& scale) {
  float x[8], o[8], y[8];
  elements_of<kPairs>(x, o, k4, me, a.rot);
  const double n = a.k_weight ? exact_norm<D>(x, a.eps) : 1.0;
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    y[i] = (float)(fma((double)x[i], A[i], (double)o[i] * B[i]) * n);
    top = max(top, field_of(fabsf(y[i])));
  }
  scale = scale_byte(block_max(top));
  return quant8_f32(y, scale);
}

// The slot of a row, -1 where it writes nothing.
__device__ __forceinline__ int64_t slot_of(const KvAppendArgs& a, int t) {
  if (t >= a.T || a.positions[t] < 0) return -1;
  const int64_t slot = a.slots[t];
  return slot >= 0 && slot < a.num_slots ? slot : -1;
}

template <int D, bool kPairs>
__device__ __forceinline__ void append_keys(const KvAppendArgs& a, Shared& sh, int t0, int first, int step) {
  using Tile = AppendTile<D>;
  const int c = threadIdx.x % Tile::kLanes, r = threadIdx.x / Tile::kLanes, t = t0 + r;
  const int64_t slot = slot_of(a, t);
  const Place me = place_of<D, kPairs>(c, t < a.T ? a.positions[t] : 0, a.rot);
  const uint16_t* src = a.k + t * a.k_stride + 8 * c;
  const int limit = slot >= 0 ? a.H * D - 8 * c : 0;
  int e = first * Tile::kWidth;
  uint4 next = make_uint4(0, 0, 0, 0);
  if (e < limit) next = *reinterpret_cast<const uint4*>(src + e);
  double A[8], B[8];
  coefficients<D, kPairs, double>(A, B, a, sh.turn + r * (D / 2), c, Tile::kLanes, a.k_weight, me);
  const KvLayout L = {1 << a.log2_page, D};
  const int tok = (int)(slot & (L.P - 1)), code = L.k_code(tok, me.d), scale_at = L.k_scale(tok, me.d);
  uint8_t* blk = a.cache + ((slot >> a.log2_page) * a.H + (e + 8 * c) / D) * L.block_bytes();
  for (; e < a.H * D; e += step * Tile::kWidth) {
    const uint4 k4 = next;
    const int e2 = e + step * Tile::kWidth;
    if (e2 < limit) next = *reinterpret_cast<const uint4*>(src + e2);
    uint32_t scale;
    const uint32_t codes = key_codes<D, kPairs>(a, k4, A, B, me, scale);
    if (e < limit) {
      *reinterpret_cast<uint32_t*>(blk + code) = codes;
      if ((c & 3) == 0) blk[scale_at] = (uint8_t)scale;
    }
    blk += step * (Tile::kWidth / D) * L.block_bytes();
  }
}

// As k_kv_write does it: four tokens' codes to a word, where they are all here.
template <int D>
__device__ __forceinline__ void append_values(const KvAppendArgs& a, Shared& sh, int t0, int first, int step) {
  using Tile = AppendTile<D>;
  constexpr int kPad = Tile::kLanes + 1, m = D / 32;
  const int c = threadIdx.x % Tile::kLanes, r = threadIdx.x / Tile::kLanes, d = 8 * c % D, t = t0 + r;
  const int64_t slot = slot_of(a, t);
  const uint16_t* src = a.v + t * a.v_stride + 8 * c;
  const int limit = slot >= 0 ? a.H * D - 8 * c : 0;
  int e = first * Tile::kWidth;
  uint4 next = make_uint4(0, 0, 0, 0);
  if (e < limit) next = *reinterpret_cast<const uint4*>(src + e);
  if (c == 0) sh.v.slot[r] = slot;
  __syncthreads();
  const int at = (int)(slot & 3), r0 = r - at;
  bool four = r0 >= 0 && r0 + 3 < Tile::kRows;
  if (four)
#pragma unroll
    for (int i = 0; i < 4; ++i) four = four && sh.v.slot[r0 + i] == slot - at + i;
  const KvLayout L = {1 << a.log2_page, D};
  const int tok = (int)(slot & (L.P - 1)), code = L.v_code(tok, d), scale_at = L.v_scale(tok, d);
  uint8_t* blk = a.cache + ((slot >> a.log2_page) * a.H + (e + 8 * c) / D) * L.block_bytes();
  for (int turn = 0; e < a.H * D; e += step * Tile::kWidth, turn ^= 1) {
    const uint4 v4 = next;
    const int e2 = e + step * Tile::kWidth;
    if (e2 < limit) next = *reinterpret_cast<const uint4*>(src + e2);
    const uint32_t scale = scale_byte(block_max(top_field(v4))), w = quant8(v4, scale);
    uint32_t* words = sh.v.words[turn];
    words[r * kPad + c] = w;
    __syncthreads();  // and the other half's readers are past the one before
    if (e < limit) {
      if ((c & 3) == 0) blk[scale_at] = (uint8_t)scale;
      if (!four) {
#pragma unroll
        for (int b = 0; b < 4; ++b) blk[code + 4 * m * b] = (uint8_t)(w >> (8 * b));
      } else if (at == 0) {  // the first of four tokens writes for all: word b gets byte b of each
        const uint32_t w1 = words[(r + 1) * kPad + c], w2 = words[(r + 2) * kPad + c], w3 = words[(r + 3) * kPad + c];
        const uint32_t s = __builtin_amdgcn_perm(w1, w, 0x05010400), b = __builtin_amdgcn_perm(w3, w2, 0x05010400);
        const uint32_t p = __builtin_amdgcn_perm(w1, w, 0x07030602), q = __builtin_amdgcn_perm(w3, w2, 0x07030602);
        uint32_t* dst = reinterpret_cast<uint32_t*>(blk + code);
        dst[0] = __builtin_amdgcn_perm(b, s, 0x05040100);
        dst[m] = __builtin_amdgcn_perm(b, s, 0x07060302);
        dst[2 * m] = __builtin_amdgcn_perm(q, p, 0x05040100);
        dst[3 * m] = __builtin_amdgcn_perm(q, p, 0x07060302);
      }
    }
    blk += step * (Tile::kWidth / D) * L.block_bytes();
  }
}

// Workgroups of a launch over rows first_row on: `tiles` row tiles of queries times their parts, then of
// keys, then of values.
struct AppendGrid {
  int first_row, q_tiles, q_parts, kv_tiles, kv_parts;
};

template <int D, bool kPairs>
__global__ __launch_bounds__(256) void k_kv_append(KvAppendArgs a, AppendGrid g) {
  __shared__ Shared sh;
  int b = (int)blockIdx.x;
  const int nq = g.q_tiles * g.q_parts, nkv = g.kv_tiles * g.kv_parts;
  if (b < nq) {
    append_queries<D, kPairs>(a, sh, g.first_row + b % g.q_tiles * kQueryRows + (int)(threadIdx.x >> 6), b / g.q_tiles, g.q_parts);
    return;
  }
  b -= nq;
  const bool keys = b < nkv;
  if (!keys) b -= nkv;
  const int t0 = g.first_row + b % g.kv_tiles * AppendTile<D>::kRows;
  if (keys) append_keys<D, kPairs>(a, sh, t0, b / g.kv_tiles, g.kv_parts);
  else append_values<D>(a, sh, t0, b / g.kv_tiles, g.kv_parts);
}

// Ways to share `units` so that `tiles` times them come to about `want`, with equal shares.
inline int parts_of(int64_t tiles, int units, int64_t want) {
  if (units == 0) return 0;
  const int64_t ways = max(min(want / max(tiles, (int64_t)1), (int64_t)units), (int64_t)1);
  const int64_t each = (units + ways - 1) / ways;
  return (int)((units + each - 1) / each);
}

template <int D, bool kPairs>
hipError_t launch(const KvAppendArgs& a, hipStream_t st) {
  using Tile = AppendTile<D>;
  constexpr int kMost = 1 << 21;  // rows of a launch, which holds fewer than 2^32 threads
  // Workgroups of queries, and of keys or values, wanted: more share out the angles' work less, fewer leave
  // the chip idle. 512 / 256 / 1024: 1500 rows of 32 + 8 heads 10.4 / 10.3 / 12.6 us, 4000 rows 20.9 / 23.2 / 22.0,
  // 2051 of 12 + 12 heads of 64 9.0 / 11.1 / 10.1; 500 rows 6.4 / 6.0 / 7.8.
  constexpr int kGroups = 512;
  for (int64_t first = 0; first < a.T; first += kMost) {
    const int rows = (int)min(a.T - first, (int64_t)kMost);
    AppendGrid g;
    g.first_row = (int)first;
    g.q_tiles = (rows + kQueryRows - 1) / kQueryRows;
    g.q_parts = parts_of(g.q_tiles, (a.Hq * D + kQueryWidth - 1) / kQueryWidth, kGroups);
    g.kv_tiles = (rows + Tile::kRows - 1) / Tile::kRows;
    g.kv_parts = parts_of(g.kv_tiles, (a.H * D + Tile::kWidth - 1) / Tile::kWidth, kGroups);
    const unsigned groups = (unsigned)(g.q_tiles * g.q_parts + 2 * g.kv_tiles * g.kv_parts);
    hipLaunchKernelGGL((k_kv_append<D, kPairs>), dim3(groups), dim3(256), 0, st, a, g);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t st) {
  switch (a.D) {
    case 64: return a.pairs ? launch<64, true>(a, st) : launch<64, false>(a, st);
    case 128: return a.pairs ? launch<128, true>(a, st) : launch<128, false>(a, st);
    default: return a.pairs ? launch<256, true>(a, st) : launch<256, false>(a, st);
  }
}

}  // namespace mx
