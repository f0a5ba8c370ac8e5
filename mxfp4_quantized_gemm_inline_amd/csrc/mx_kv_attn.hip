// mx_kv_attn.hip - attention of bf16 queries over the paged MXFP4 cache.
//
// For a query q at position pos over the keys K[j] and values V[j] that it sees,
//   s_j = scale q . K[j],  out = sum_j exp(s_j - m) V[j] / sum_j exp(s_j - m),  m = max_j s_j,
// in one pass over the tokens: with the running maximum m, sum l and unscaled output o, a
// block of tokens with maximum m' multiplies l and o by exp(m - max(m, m')) and adds its own.
#include <algorithm>
#include <climits>
#include <cstdio>

#include "mx_device.h"
#include "mx_kv.h"

namespace mx {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLowest = -3.0e38f;  // the running maximum before any token: below every score
// How far, in powers of two, the maximum in use may lag behind the true one before the sums are
// rescaled (a published step of attention kernels): weights reach 2^8 then, which neither bf16's
// relative rounding nor an FP32 sum feels, and the rescaling of all sums is left out of nearly every
// step.
constexpr float kLag = 8.f;

// ------------------------------------------------------------------------------- row tiles
//
// The rows of one request and one key/value head: query row i and head g of the group are row
// r = i G + g of n G rows that read the same keys and values. A row tile is R of them.

struct RowTile {
  int b, q0, n, rb, rows;  // request, its first query row and count, first row of the tile, rows in it
  int len;                 // cached tokens
  int seen, hi;            // tokens that some row of the tile sees (hi <= seen: none)
  int lo;                  // seen, down to a multiple of 16: where its token tiles begin
  __device__ int pos(int r, int G) const { return len - n + r / G; }
};

__device__ __forceinline__ int clamp_int(int x, int lo, int hi) { return min(max(x, lo), hi); }

// The tokens that a row at `pos` sees.
__device__ __forceinline__ int row_end(const KvAttnArgs& a, int len, int pos) {
  return a.causal ? clamp_int(pos + 1, 0, len) : len;
}
__device__ __forceinline__ int row_begin(const KvAttnArgs& a, int pos) {
  return a.window ? max(max(pos, 0) - a.window + 1, 0) : 0;
}

// Row tile `rb` rows into request b; false where the request has no such rows.
__device__ __forceinline__ bool row_tile_of(const KvAttnArgs& a, int R, int b, int rb, RowTile& w) {
  w.b = b;
  w.q0 = clamp_int(a.cu_q[b], 0, a.T);
  w.n = clamp_int(a.cu_q[b + 1], w.q0, a.T) - w.q0;
  w.rb = rb;
  w.rows = min(R, w.n * a.G - rb);
  if (w.rows <= 0) return false;
  w.len = (int)min((int64_t)max(a.kv_lens[b], 0), (int64_t)a.max_blocks << a.log2_page);
  w.seen = row_begin(a, w.pos(rb, a.G));
  w.lo = w.seen & ~15;
  w.hi = row_end(a, w.len, w.pos(rb + w.rows - 1, a.G));
  return true;
}

// Numbering row tiles without a sum over the requests: tile b < B is request b's first; its others,
// at most floor(n G / R), are the tiles B + floor(cu_q[b] G / R) on, for which the wave searches 64
// requests at a time. Numbers without rows so come last: between the others they would leave some
// XCDs without work (256 requests of 32 rows and 4 heads over up to 4000 tokens: 176 us so).
__device__ __forceinline__ int first_tile(const KvAttnArgs& a, int R, int b) {
  return a.B + (int)((int64_t)clamp_int(a.cu_q[b], 0, a.T) * a.G / R);
}
__device__ __forceinline__ bool find_row_tile(const KvAttnArgs& a, int R, int tile, RowTile& w) {
  if (tile < a.B) return row_tile_of(a, R, tile, 0, w);
  const int lane = threadIdx.x & 63;
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int step = (hi - lo + 63) / 64, b = lo + lane * step;
    const bool at = b < hi && first_tile(a, R, b) <= tile;
    lo += (max((int)__popcll(__ballot(at)), 1) - 1) * step;
    hi = min(hi, lo + step);
  }
  lo = __builtin_amdgcn_readfirstlane(lo);
  const int i = tile - first_tile(a, R, lo) + 1;
  return i > 0 && i < (1 << 30) / R && row_tile_of(a, R, lo, i * R, w);
}
int row_tiles(const KvAttnSizes& z, int R) { return (int)(z.T * (z.Hq / z.H) / R + z.B); }

// The same with the tiles of the requests that see the most tokens first, each request's last tile
// (with a causal mask its longest) first: what is long is not left for the end. Up to 64 requests,
// one a lane: each counts those before it, and the tiles are summed in that order. Past 64 the
// order stays the requests', last tiles first.
__device__ __forceinline__ bool find_row_tile_longest(const KvAttnArgs& a, int R, int tile, int launched, RowTile& w) {
  if (a.B > 64) return find_row_tile(a, R, launched - 1 - tile, w);
  const int lane = threadIdx.x & 63;
  int tiles = 0, seen = -1;
  if (lane < a.B) {
    const int q0 = clamp_int(a.cu_q[lane], 0, a.T), n = clamp_int(a.cu_q[lane + 1], q0, a.T) - q0;
    const int len = (int)min((int64_t)max(a.kv_lens[lane], 0), (int64_t)a.max_blocks << a.log2_page);
    tiles = (n * a.G + R - 1) / R;
    seen = a.window ? min(len, a.window) : len;
  }
  int before = 0;
  for (int b = 0; b < a.B; ++b) {
    const int other = __builtin_amdgcn_readlane(seen, b);
    before += other > seen || (other == seen && b < lane);
  }
  if (lane >= a.B) before = lane;
  const int own = __builtin_amdgcn_ds_permute(before * 4, tiles), request = __builtin_amdgcn_ds_permute(before * 4, lane);
  int upto = own;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(upto, d);
    if (lane >= d) upto += y;
  }
  const uint64_t at = __ballot(tile < upto && tile >= upto - own);
  if (at == 0) return false;
  const int k = __builtin_ctzll(at);
  return row_tile_of(a, R, __builtin_amdgcn_readlane(request, k), (__builtin_amdgcn_readlane(upto, k) - 1 - tile) * R, w);
}

// The tokens [lo, hi) of a row tile in splits of C; the last of at most S takes what is left.
__device__ __forceinline__ int splits_of(const RowTile& w, int C, int S) {
  return clamp_int((w.hi - w.lo + C - 1) / C, 1, S);
}

// ------------------------------------------------------------------------------- operands

// A query row in two 8-bit floats. With 2^e the power that brings the row's largest element
// into [128, 256), hi = e4m3(q 2^-e) keeps four of bf16's eight significant bits and
// lo = e4m3((q 2^-e - hi) 2^5) the other four: together exact for elements down to 2^-13 of the
// largest and to 2^-21 of it below. So the keys enter the scaled MFMA as they lie in the cache,
// 4-bit with their scale bytes, and none is ever converted; one product more pays for that with
// the same matrix time as bf16 and no vector time.
__device__ __forceinline__ void split_fp8(const uint32_t (&x)[8], uint32_t scale, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
  typedef short s16x2 __attribute__((ext_vector_type(2)));
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  // the conversions divide by, or multiply with, a power of two
  const float by = __builtin_bit_cast(float, scale << 23), by_lo = __builtin_bit_cast(float, (scale - 5u) << 23);
  auto first = [](uint32_t pair) { return __builtin_bit_cast(float, pair << 16); };
  auto second = [](uint32_t pair) { return __builtin_bit_cast(float, pair & 0xFFFF0000u); };
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t a = x[2 * j], b = x[2 * j + 1];
    s16x2 h = {0, 0}, l = {0, 0};
    h = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(h, __builtin_bit_cast(bf16x2, a), by, false);
    h = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(h, __builtin_bit_cast(bf16x2, b), by, true);
    hi[j] = __builtin_bit_cast(uint32_t, h);
    const f32x2 p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(hi[j], by, false);
    const f32x2 q = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(hi[j], by, true);
    l = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(l, first(a) - p.x, second(a) - p.y, by_lo, false);
    l = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(l, first(b) - q.x, second(b) - q.y, by_lo, true);
    lo[j] = __builtin_bit_cast(uint32_t, l);
  }
}
// Scale byte of hi for a row whose largest exponent field is E (lo's is 5 less).
__device__ __forceinline__ uint32_t query_scale(uint32_t E) { return E > 12u ? E - 7u : 5u; }

// Largest exponent field of bf16 pairs.
__device__ __forceinline__ uint32_t top_exponent(const uint4& u, uint32_t E) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w;
    E = max(E, max((w >> 7) & 0xFFu, (w >> 23) & 0xFFu));
  }
  return E;
}

__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){x, y}, bf16x2));
}

// l + the two bf16 values of a word: the sum of the weights as the product with V takes them.
__device__ __forceinline__ float add_pair(float l, uint32_t u) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, u), __builtin_bit_cast(bf16x2, 0x3F803F80u), l, false);
}

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
__device__ __forceinline__ bf16x8 as_bf16x8(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_bit_cast(bf16x8, (u32x4){a, b, c, d});
}

// What lies at a device address that was put together from its halves.
template <typename T>
__device__ __forceinline__ T global(uint64_t at) {
  return *(const __attribute__((address_space(1))) T*)at;
}

// Byte I of a word (a pair of codes) times its scale, the scale byte J of another word.
template <int I>
__device__ __forceinline__ uint32_t decode2(uint32_t codes, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, I));
}
// Byte J of a word as the exponent of an FP32 scale, in one instruction (the compiler's own form
// for bytes 0 to 2 is a shift and a mask); shift: 23 in a register.
template <int J>
__device__ __forceinline__ float scale_at(uint32_t w, uint32_t shift) {
  uint32_t r;
  if constexpr (J == 0)
    asm("v_lshlrev_b32_sdwa %0, %1, %2 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:DWORD src1_sel:BYTE_0" : "=v"(r) : "v"(shift), "v"(w));
  else if constexpr (J == 1)
    asm("v_lshlrev_b32_sdwa %0, %1, %2 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:DWORD src1_sel:BYTE_1" : "=v"(r) : "v"(shift), "v"(w));
  else if constexpr (J == 2)
    asm("v_lshlrev_b32_sdwa %0, %1, %2 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:DWORD src1_sel:BYTE_2" : "=v"(r) : "v"(shift), "v"(w));
  else
    asm("v_lshlrev_b32_sdwa %0, %1, %2 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:DWORD src1_sel:BYTE_3" : "=v"(r) : "v"(shift), "v"(w));
  return __builtin_bit_cast(float, r);
}

// ------------------------------------------------------------------------------- few rows
//
// Decoding and drafts: a workgroup takes a tile of 16 NT rows and a run of tokens of one head,
// each wave its part of them on its own, 32 tokens a step. The next step's keys are fetched when
// this step's are in the products, its values likewise. The transposed products put a query row in
// each of the 16 columns:
//   S^T (16 tokens x 16 rows) = K Q^T    scaled 16x16x128 MFMA, A = K codes from the cache,
//   O^T (D x 16 rows)        += V^T P^T  bf16 16x16x32 MFMA, A = V decoded in registers.
// A lane's four scores of each of two token tiles (tokens 4g..4g+3) are, rounded to bf16, its
// eight elements of P^T: no exchange between lanes. (The rounding of a weight is off by 2^-8 of it
// at most, as that of the output; l sums the rounded weights, so that they still add up to one.)
// V's codes lie in the cache so that one word holds four tokens of an element pair; two
// conversions and two byte permutations make the operands of the pair's two rows of V^T.
// Bound: HBM, 17/16 D bytes a token and head, where the tokens are many: 64 requests x 8 heads x up
// to 8192 tokens, D = 128, 313 MB: 66 us and 5 of joins, 4.7 TB/s. Else the chain of loads (lengths,
// pages, tokens) and the fixed work of a segment: one request of 16 tokens 5.7 us, of 1037 11.2.

template <int D>
struct TokenTile {  // one lane's share of 16 tokens
  static constexpr int M = D / 32;
  u32x4 k[(D + 127) / 128];
  uint32_t ks[(D + 127) / 128];  // the word that holds the token's scale byte, at bit 8 (token % 4)
  uint32_t v[M];   // word j: the lane's element pair of scale block j, four tokens
  uint32_t vs[M];  // the 4 M scale bytes of its four tokens

  __device__ __forceinline__ void load_k(const uint8_t* blk, int P, int in_page, uint32_t lane) {
    const uint8_t* kc = blk + in_page * (8 * D);
    const uint8_t* kb = blk + P * D + in_page * (D / 2);
    if constexpr (D == 64) {
      k[0] = *reinterpret_cast<const u32x4*>(kc + (lane & 31u) * 16u);
      ks[0] = *reinterpret_cast<const uint32_t*>(kb + (lane & 28u));
    } else {
#pragma unroll
      for (int c = 0; c < D / 128; ++c) {
        k[c] = *reinterpret_cast<const u32x4*>(kc + (c * 1024u + lane * 16u));
        ks[c] = *reinterpret_cast<const uint32_t*>(kb + (c * 64u + (lane & 60u)));
      }
    }
  }
  __device__ __forceinline__ void load_v(const uint8_t* blk, int P, int in_page, uint32_t lane) {
    const uint8_t* vc = blk + P * (D / 2) + in_page * (8 * D);
    const uint8_t* vb = blk + P * D + P * M + in_page * (16 * M);
    typedef uint32_t words __attribute__((ext_vector_type(M)));
    const words a = *reinterpret_cast<const words*>(vc + lane * (4u * M));
    const words b = *reinterpret_cast<const words*>(vb + (lane >> 4) * (4u * M));
#pragma unroll
    for (int j = 0; j < M; ++j) {
      v[j] = a[j];
      vs[j] = b[j];
    }
  }
  // Scale of block j of the lane's token i: byte (i M + j) of vs.
  template <int I, int J>
  __device__ __forceinline__ float scale(uint32_t shift) const {
    return scale_at<(I * M + J) % 4>(vs[(I * M + J) / 4], shift);
  }
  // Scales of the tokens outside [lo, hi), which no row of the tile sees, become 0 (2^-127): bytes
  // that were never written, or are another request's, could stand for infinities or NaN, which a
  // weight of 0 does not take away. t: the lane's first token.
  __device__ __forceinline__ void mask(int t, int lo, int hi) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (t + i < lo || t + i >= hi) {
        if constexpr (M == 2) vs[i / 2] &= i % 2 ? 0x0000FFFFu : 0xFFFF0000u;
        else
#pragma unroll
          for (int j = 0; j < M / 4; ++j) vs[i * (M / 4) + j] = 0;
      }
  }
};

// Waves a SIMD that the vector registers allow without spilling (the shared kernels keep 66 to 72 scalars
// of their schedule in lanes of one).
constexpr int few_occupancy(int D, int NT) { return D == 64 ? (NT == 1 ? 4 : 3) : D == 128 ? (NT == 1 ? 3 : 2) : 2; }

constexpr int kAllRows = 0x7FFFFFFF;

// Work is cut into equal shares, however ragged the lengths are: a segment is a row tile and a
// head, of ceil(tokens / 32) + kSegmentUnits units (a segment's start and end cost about as much as
// that many units of 32 tokens: 64 requests x 8 heads x up to 8192 tokens 77, 74, 72, 72, 73 us at
// 0, 4, 8, 16, 24); the segments of all requests lie in a row, and worker i of 2^lg takes
// the units floor(i W / 2^lg) on of all W. A segment that lies in one share is written to the
// output; of one that is cut, each worker leaves an unscaled part: in its slot 0 if the segment is
// its first, else in its slot 1 (its last). The worker whose share begins in the second part of a
// segment names the parts to the join.
// Where every segment is short, or without a workspace, a workgroup takes one whole segment.
constexpr int kSegmentUnits = 8;

struct KvShares {
  int lg;         // log2 of the workers
  int rows_most;  // requests of more rows (query rows times group) are the other kernel's
  float* o;       // [workers][2][R][D]
  float2* ml;     // [workers][2][R]: maximum, sum
  int4* seams;    // [workers]: first query row; first row of the tile; head | rows << 16; parts | slot of the first << 30
};

struct KvRequest {
  int q0, n, len;
  __device__ __forceinline__ int tiles(int G, int R) const { return (n * G + R - 1) / R; }
  __device__ __forceinline__ int units(const KvAttnArgs& a) const {  // of each of its segments
    const int lo = row_begin(a, len - n) & ~15, hi = row_end(a, len, len - 1);
    return max(hi - lo + 31, 0) / 32 + kSegmentUnits;
  }
};

__device__ __forceinline__ KvRequest request_of(const KvAttnArgs& a, int b, int rows_most) {
  KvRequest r = {0, 0, 0};
  if (b < a.B) {
    r.q0 = clamp_int(a.cu_q[b], 0, a.T);
    r.n = clamp_int(a.cu_q[b + 1], r.q0, a.T) - r.q0;
    r.len = (int)min((int64_t)max(a.kv_lens[b], 0), (int64_t)a.max_blocks << a.log2_page);
    if (r.n * (int64_t)a.G > rows_most) r.n = 0;
  }
  return r;
}

constexpr int kWaves = 4, kThreads = 64 * kWaves;

template <int D, int NT, bool kShared>
__global__ __launch_bounds__(kThreads, few_occupancy(D, NT)) void k_kv_attn_few(KvAttnArgs a, KvShares sh) {
  constexpr int R = 16 * NT, M = D / 32, KC = (D + 127) / 128, LD = D + 4;
  __shared__ float o_all[kWaves][16][LD];
  __shared__ float2 ml_all[kWaves][R];
  __shared__ int64_t sums[kShared ? kThreads : 1];  // units before each thread's requests
  __shared__ KvRequest requests[kShared ? kThreads : 1];
  __shared__ int64_t wave_sum[kWaves];
  __shared__ int found;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = lane & 15, g = lane >> 4;
  const float c2 = a.scale * kLog2e;
  uint32_t shift = 23;
  asm volatile("" : "+v"(shift));  // kept in a register: scale_at
  const int P = 1 << a.log2_page, worker = (int)blockIdx.x, per = (a.B + kThreads - 1) / kThreads;
  int64_t W = 0, u = 0, u_end = 1, before = 0;
  int lg = sh.lg, b = 0, h = worker % a.H;
  RowTile w;
  auto share_at = [&](int i) { return i * (W >> lg) + ((i * (W & (((int64_t)1 << lg) - 1))) >> lg); };  // i W / 2^lg

  if constexpr (kShared) {
    // where the shares lie: a sum over the requests, each thread `per` of them
    int64_t mine = 0;
    for (int i = 0; i < per; ++i) {
      const KvRequest r = request_of(a, threadIdx.x * per + i, sh.rows_most);
      if (i == 0) requests[threadIdx.x] = r;
      if (r.n > 0) mine += (int64_t)r.tiles(a.G, R) * a.H * r.units(a);
    }
    int64_t upto = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t y = __shfl_up(upto, d);
      if (lane >= d) upto += y;
    }
    if (lane == 63) wave_sum[wave] = upto;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
      if (i == wave) upto += W;
      W += wave_sum[i];
    }
    while (lg > 0 && (W >> lg) == 0) --lg;  // a unit a worker at least
    if (W == 0 || worker >> lg) {
      if (threadIdx.x == 0) sh.seams[worker].w = 0;
      return;
    }
    u = share_at(worker);
    u_end = share_at(worker + 1);
    sums[threadIdx.x] = upto - mine;
    if (upto - mine <= u && u < upto) found = threadIdx.x;
    __syncthreads();
    b = __builtin_amdgcn_readfirstlane(found) * per;
    before = sums[__builtin_amdgcn_readfirstlane(found)];  // units before request b
  } else if (!find_row_tile(a, R, worker / a.H, w) || w.n * a.G > sh.rows_most) {
    return;
  }

  for (bool first = true; u < u_end; first = false) {
    bool whole = true;
    if constexpr (kShared) {
      // the segment of unit u
      KvRequest req;
      int units;
      for (;; ++b) {  // u < W: some request ends after it
        req = per == 1 ? requests[b] : request_of(a, b, sh.rows_most);
        units = __builtin_amdgcn_readfirstlane(req.units(a));
        const int64_t all = req.n > 0 ? (int64_t)req.tiles(a.G, R) * a.H * units : 0;
        if (u < before + all) break;
        before += all;
      }
      const int64_t in = u - before;
      const int seg = (in >> 31) ? (int)(in / units) : (int)((uint32_t)in / (uint32_t)units);  // head fastest
      const int from = (int)(in - (int64_t)seg * units);
      const int64_t seg_start = u - from, seg_end = seg_start + units;
      h = seg % a.H;
      w.b = b;
      w.q0 = __builtin_amdgcn_readfirstlane(req.q0);
      w.n = __builtin_amdgcn_readfirstlane(req.n);
      w.len = __builtin_amdgcn_readfirstlane(req.len);
      w.rb = seg / a.H * R;
      w.rows = min(R, w.n * a.G - w.rb);
      w.seen = row_begin(a, w.pos(w.rb, a.G));
      w.lo = w.seen & ~15;
      w.hi = row_end(a, w.len, w.pos(w.rb + w.rows - 1, a.G));
      const int to = (int)(min(u_end, seg_end) - seg_start), lo = w.lo;
      whole = from == 0 && to == units;
      if (first && threadIdx.x == 0) {
        const int64_t u_before = share_at(worker - 1);
        int4 seam = make_int4(w.q0, w.rb, h | (w.rows << 16), 0);
        if (from > 0 && seg_start >= u_before) {  // the share before this one holds the segment's first part
          int last = worker, past = 1 << lg;  // the last share that begins in the segment
          while (past - last > 1) {
            const int mid = (last + past) >> 1;
            if (share_at(mid) < seg_end) last = mid; else past = mid;
          }
          seam.w = (last - worker + 2) | (seg_start > u_before ? 1 << 30 : 0);
        }
        sh.seams[worker] = seam;
      }
      // the share's part of the tile's tokens; rows still see what they see
      w.lo = lo + 32 * max(from - kSegmentUnits, 0);
      if (to < units) w.hi = min(w.hi, lo + 32 * max(to - kSegmentUnits, 0));
      u = seg_end;
    } else {
      u = u_end;
    }

    // this wave's tokens
    const int share = (max(w.hi - w.lo, 0) + 32 * kWaves - 1) / (32 * kWaves) * 32;
    const int w0 = w.lo + wave * share, w1 = min(w.hi, w0 + share);
    const int32_t* table = a.block_table + (int64_t)w.b * a.max_blocks;
    int base = w0, tiles = 0, page = 0;
    uint64_t bad_tiles = 0;
    auto fetch_pages = [&]() {  // of 64 token tiles from base on, one a lane
      tiles = min(64, (w1 - base + 15) >> 4);
      page = 0;
      bool bad = false;
      if (lane < tiles) {
        page = table[(base + 16 * lane) >> a.log2_page];
        bad = page < 0 || page >= a.num_pages;
        if (bad) page = 0;
      }
      bad_tiles = __ballot(bad);
    };
    auto block_of = [&](int tile, int& in_page) {
      in_page = ((base + 16 * tile) & (P - 1)) >> 4;
      return a.cache + ((int64_t)__builtin_amdgcn_readlane(page, tile) * a.H + h) * a.block_bytes;
    };
    TokenTile<D> x[2];
    auto load_k = [&](int step) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        int in_page;
        const uint8_t* blk = block_of(max(min(2 * step + i, tiles - 1), 0), in_page);
        x[i].load_k(blk, P, in_page, lane);
      }
    };
    auto load_v = [&](int step) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        int in_page;
        const uint8_t* blk = block_of(max(min(2 * step + i, tiles - 1), 0), in_page);
        x[i].load_v(blk, P, in_page, lane);
      }
    };
    // The chain of loads is lengths, pages, tokens; the queries come meanwhile. A wave without
    // tokens fetches some of page 0, unused: without a branch the waits can tell the loads apart.
    fetch_pages();
    uint4 y[NT][D == 64 ? 2 : 4 * KC];
    int row_lo[NT], row_hi[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = w.rb + min(16 * nt + col, w.rows - 1);  // columns past the last row repeat it
      const uint16_t* src = a.q + (int64_t)(w.q0 + r / a.G) * a.q_stride + (h * a.G + r % a.G) * D;
      if constexpr (D == 64) {  // each lane group 16 elements
        y[nt][0] = reinterpret_cast<const uint4*>(src)[2 * g];
        y[nt][1] = reinterpret_cast<const uint4*>(src)[2 * g + 1];
      } else {
#pragma unroll
        for (int c = 0; c < KC; ++c)
#pragma unroll
          for (int i = 0; i < 4; ++i)  // bytes 0..15: elements 16 g, bytes 16..31: 64 + 16 g
            y[nt][4 * c + i] = reinterpret_cast<const uint4*>(src + 128 * c + 64 * (i / 2) + 16 * g)[i % 2];
      }
      const int pos = w.pos(r, a.G);
      row_lo[nt] = row_begin(a, pos);
      row_hi[nt] = row_end(a, w.len, pos);
    }
    load_k(0);
    load_v(0);

    // the queries, split in two
    v8i q_hi[NT][KC], q_lo[NT][KC];
    uint32_t q_sc[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      uint32_t E = 0;
#pragma unroll
      for (int i = 0; i < (D == 64 ? 2 : 4 * KC); ++i) E = top_exponent(y[nt][i], E);
      E = max(E, (uint32_t)__shfl_xor((int)E, 16));
      E = max(E, (uint32_t)__shfl_xor((int)E, 32));
      const uint32_t sc = query_scale(E);
      if constexpr (D == 64) {
        // one 16x16x128 product takes both parts: k < 64 is hi (bytes 0..15), k >= 64 lo, over the
        // same keys given twice (lane groups 2 and 3 load what 0 and 1 do)
        const uint32_t e[8] = {y[nt][0].x, y[nt][0].y, y[nt][0].z, y[nt][0].w, y[nt][1].x, y[nt][1].y, y[nt][1].z, y[nt][1].w};
        uint32_t hi[4], lo[4];
        split_fp8(e, sc, hi, lo);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          q_hi[nt][0][j] = (int)hi[j];
          q_hi[nt][0][4 + j] = (int)lo[j];
        }
        q_sc[nt] = g < 2 ? sc : sc - 5u;
      } else {
#pragma unroll
        for (int c = 0; c < KC; ++c)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint4 p0 = y[nt][4 * c + 2 * i], p1 = y[nt][4 * c + 2 * i + 1];
            const uint32_t e[8] = {p0.x, p0.y, p0.z, p0.w, p1.x, p1.y, p1.z, p1.w};
            uint32_t hi[4], lo[4];
            split_fp8(e, sc, hi, lo);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              q_hi[nt][c][4 * i + j] = (int)hi[j];
              q_lo[nt][c][4 * i + j] = (int)lo[j];
            }
          }
        q_sc[nt] = sc;
      }
    }
    // a step inside [all_lo, all_hi) needs no mask
    const int all_lo = row_begin(a, w.pos(w.rb + w.rows - 1, a.G)), all_hi = min(w1, row_end(a, w.len, w.pos(w.rb, a.G)));

    float m[NT], l[NT];
    v4f o[NT][2 * M];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt] = kLowest;
      l[nt] = 0.f;
#pragma unroll
      for (int j = 0; j < 2 * M; ++j) o[nt][j] = (v4f){0.f, 0.f, 0.f, 0.f};
    }

    while (base < w1) {
      const int steps = (tiles + 1) >> 1;
      for (int step = 0; step < steps; ++step) {
        const int t = base + 32 * step;
        v4f s[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            s[nt][i] = (v4f){0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < KC; ++c) {
              const int ks = (int)(x[i].ks[c] >> (8 * (lane & 3)));  // the product takes its low byte
              const v8i kv = {(int)x[i].k[c].x, (int)x[i].k[c].y, (int)x[i].k[c].z, (int)x[i].k[c].w, 0, 0, 0, 0};
              s[nt][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(kv, q_hi[nt][c], s[nt][i], 4, 0, 0, ks, 0,
                                                                          (int)q_sc[nt]);
              if constexpr (D != 64)
                s[nt][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(kv, q_lo[nt][c], s[nt][i], 4, 0, 0, ks, 0,
                                                                            (int)(q_sc[nt] - 5u));
            }
          }
        load_k(min(step + 1, steps - 1));  // the last step's loads, of what it has already, go unused
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nt][i][e] *= c2;
        const uint64_t bad2 = bad_tiles >> (2 * step);
        if (t < all_lo || t + 32 > all_hi || (bad2 & 3u)) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int tt = t + 16 * i + 4 * g;
            const bool hidden = (bad2 >> i) & 1u;
            x[i].mask(tt, w.seen, hidden ? 0 : w1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (hidden || tt + e < row_lo[nt] || tt + e >= min(row_hi[nt], w1)) s[nt][i][e] = -INFINITY;
          }
        }
        uint32_t p[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float top = fmaxf(fmaxf(fmaxf(s[nt][0][0], s[nt][0][1]), fmaxf(s[nt][0][2], s[nt][0][3])),
                            fmaxf(fmaxf(s[nt][1][0], s[nt][1][1]), fmaxf(s[nt][1][2], s[nt][1][3])));
          // The maximum in use may lag behind the true one by kLag (weights up to 2^kLag, all sums
          // in FP32); only past that are the sums rescaled.
          if (__any(top > m[nt] + kLag)) {
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const float m1 = fmaxf(m[nt], top), alpha = __builtin_amdgcn_exp2f(m[nt] - m1);
            m[nt] = m1;
            l[nt] *= alpha;
#pragma unroll
            for (int j = 0; j < 2 * M; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[nt][j][e] *= alpha;
          }
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; e += 2)
              p[nt][2 * i + e / 2] = pack_bf16(__builtin_amdgcn_exp2f(s[nt][i][e] - m[nt]),
                                               __builtin_amdgcn_exp2f(s[nt][i][e + 1] - m[nt]));
#pragma unroll
          for (int i = 0; i < 4; ++i) l[nt] = add_pair(l[nt], p[nt][i]);
        }
        static_for<M>([&](auto J) {
          constexpr int j = J;
          uint32_t even[4], odd[4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t c0 = decode2<0>(x[i].v[j], x[i].template scale<0, j>(shift));
            const uint32_t c1 = decode2<1>(x[i].v[j], x[i].template scale<1, j>(shift));
            const uint32_t c2_ = decode2<2>(x[i].v[j], x[i].template scale<2, j>(shift));
            const uint32_t c3 = decode2<3>(x[i].v[j], x[i].template scale<3, j>(shift));
            even[2 * i] = __builtin_amdgcn_perm(c1, c0, 0x05040100);
            even[2 * i + 1] = __builtin_amdgcn_perm(c3, c2_, 0x05040100);
            odd[2 * i] = __builtin_amdgcn_perm(c1, c0, 0x07060302);
            odd[2 * i + 1] = __builtin_amdgcn_perm(c3, c2_, 0x07060302);
          }
          const bf16x8 ve = as_bf16x8(even[0], even[1], even[2], even[3]), vo = as_bf16x8(odd[0], odd[1], odd[2], odd[3]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const bf16x8 pt = as_bf16x8(p[nt][0], p[nt][1], p[nt][2], p[nt][3]);
            o[nt][2 * j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ve, pt, o[nt][2 * j], 0, 0, 0);
            o[nt][2 * j + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vo, pt, o[nt][2 * j + 1], 0, 0, 0);
          }
        });
        load_v(min(step + 1, steps - 1));
      }
      base += 64 * 16;
      if (base >= w1) break;
      fetch_pages();
      load_k(0);
      load_v(0);
    }

    // join the waves: the largest maximum, every wave's sums at it, added in the waves' order
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      l[nt] += __shfl_xor(l[nt], 16);
      l[nt] += __shfl_xor(l[nt], 32);
      if (g == 0) ml_all[wave][16 * nt + col] = make_float2(m[nt], l[nt]);
    }
    __syncthreads();
    const int64_t slot = (int64_t)worker * 2 + (first ? 0 : 1);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float top = kLowest;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) top = fmaxf(top, ml_all[i][16 * nt + col].x);
      const float f = __builtin_amdgcn_exp2f(m[nt] - top);
#pragma unroll
      for (int j = 0; j < M; ++j) {
        const v4f e = o[nt][2 * j], d = o[nt][2 * j + 1];
        *reinterpret_cast<v4f*>(&o_all[wave][col][32 * j + 8 * g]) = (v4f){e[0] * f, d[0] * f, e[1] * f, d[1] * f};
        *reinterpret_cast<v4f*>(&o_all[wave][col][32 * j + 8 * g + 4]) = (v4f){e[2] * f, d[2] * f, e[3] * f, d[3] * f};
      }
      __syncthreads();
      constexpr int E = D / 16;  // a thread's elements
      const int cr = 16 * nt + threadIdx.x / 16, d0 = (threadIdx.x % 16) * E;
      if (cr < w.rows) {
        float M1 = kLowest, L = 0.f, z[E];
#pragma unroll
        for (int i = 0; i < kWaves; ++i) M1 = fmaxf(M1, ml_all[i][cr].x);
#pragma unroll
        for (int i = 0; i < kWaves; ++i) L += ml_all[i][cr].y * __builtin_amdgcn_exp2f(ml_all[i][cr].x - M1);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          z[e] = o_all[0][cr - 16 * nt][d0 + e];
#pragma unroll
          for (int i = 1; i < kWaves; ++i) z[e] += o_all[i][cr - 16 * nt][d0 + e];
        }
        if (whole) {
          const int r = w.rb + cr;
          const float inv = L > 0.f ? 1.f / L : 0.f;
          uint16_t* dst = a.out + (int64_t)(w.q0 + r / a.G) * a.out_stride + (h * a.G + r % a.G) * D + d0;
#pragma unroll
          for (int e = 0; e < E; e += 4)
            *reinterpret_cast<uint2*>(dst + e) = make_uint2(pack_bf16(z[e] * inv, z[e + 1] * inv), pack_bf16(z[e + 2] * inv, z[e + 3] * inv));
        } else {
          float* dst = sh.o + (slot * R + cr) * D + d0;
#pragma unroll
          for (int e = 0; e < E; e += 4) *reinterpret_cast<v4f*>(dst + e) = (v4f){z[e], z[e + 1], z[e + 2], z[e + 3]};
          if (threadIdx.x % 16 == 0) sh.ml[slot * R + cr] = make_float2(M1, L);
        }
      }
      __syncthreads();  // before the next rows', or the next segment's, sums take the place
    }
  }
}

// Joins the parts of the segments that shares have cut: a workgroup for `each` workers and four rows
// (more in turn), W waves a row, each every W-th part. Bound: latency, a chain of seam, maxima and
// sums: 5 us for 64 requests x 8 heads, 6.7 for 8 segments of 65 parts. The segment's first part is in the worker before,
// in the slot that the seam names; the others in the slots 0 from the worker on. The parts' weights
// are worked out 64 at a time, one a lane, so that the loads of the sums wait for nothing.
template <int D, int W>
__global__ __launch_bounds__(256 * W) void k_kv_attn_seams(KvAttnArgs a, KvShares sh, int R, int each) {
  constexpr int E = D / 64;
  typedef float vec __attribute__((ext_vector_type(E)));
  __shared__ vec o_all[4 * W][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), sub = wave % W;
  const int first = (int)blockIdx.x * each, own = first + lane;
  uint64_t with_seam = __ballot(lane < each && own < (1 << sh.lg) && sh.seams[min(own, (1 << sh.lg) - 1)].w != 0);
  for (; with_seam; with_seam &= with_seam - 1) {
    const int worker = first + __builtin_ctzll(with_seam);
    const int4 seam = sh.seams[worker];
    const int parts = seam.w & 0x3FFFFFFF, rows = seam.z >> 16, h = seam.z & 0xFFFF;
    for (int r0 = 4 * (int)blockIdx.y; r0 < rows; r0 += 4 * (int)gridDim.y) {
      const int r = r0 + wave / W;
      float l = 0.f;
      vec x;
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = 0.f;
      if (r < rows) {
        // part i's row: in the slots 2 (worker - 1 + i), the first part's one later if the seam says so
        auto at = [&](int i) { return ((int64_t)2 * (worker - 1 + i) + (i == 0 ? (seam.w >> 30) & 1 : 0)) * R + r; };
        float m = kLowest;
        for (int i = lane; i < parts; i += 64) m = fmaxf(m, sh.ml[at(i)].x);
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
        for (int i0 = 0; i0 < parts; i0 += 64) {
          float f = 0.f;
          if (i0 + lane < parts) {
            const float2 ml = sh.ml[at(i0 + lane)];
            f = __builtin_amdgcn_exp2f(ml.x - m);
            l += ml.y * f;
          }
          const int n = min(64, parts - i0);
          for (int i = sub; i < n; i += 4 * W) {  // four parts' loads at once; past the last, that one with weight 0
            vec y[4];
            float g[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int j = min(i + W * k, n - 1);
              y[k] = *reinterpret_cast<const vec*>(sh.o + at(i0 + j) * D + lane * E);
              g[k] = i + W * k < n ? __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, f), j)) : 0.f;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int e = 0; e < E; ++e) x[e] += y[k][e] * g[k];
          }
        }
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) l += __shfl_xor(l, d);
      }
      if constexpr (W > 1) {
        o_all[wave][lane] = x;
        __syncthreads();
      }
      if (r < rows && sub == 0) {
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const int row = seam.y + r;
        uint16_t* dst = a.out + (int64_t)(seam.x + row / a.G) * a.out_stride + (h * a.G + row % a.G) * D + lane * E;
        float z[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          z[e] = x[e];
#pragma unroll
          for (int k = 1; k < W; ++k) z[e] += o_all[wave + k][lane][e];
          z[e] *= inv;
        }
        if constexpr (E == 1) {
          dst[0] = (uint16_t)f32_to_bf16_rne(z[0]);
        } else {
#pragma unroll
          for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16(z[e], z[e + 1]);
        }
      }
      if constexpr (W > 1) __syncthreads();
    }
  }
}

// ------------------------------------------------------------------------------- many rows
//
// Prompts and chunks: one workgroup of four waves takes 128 rows of one head, each wave 32 of
// them, and walks the tokens 64 at a time with 32-wide products of the same form:
//   S^T (32 tokens x 32 rows) = K Q^T    scaled 32x32x64 MFMA, A = K codes from the cache,
//   O^T (32 of D x 32 rows)  += V^T P^T  bf16 32x32x16 MFMA.
// A wave reads the keys it needs itself (4-bit, no conversion, the waves' loads meet in L1). The
// values are decoded once for the workgroup: each wave decodes one token tile of the next 64
// tokens into LDS in operand order while the products of this step run; two buffers, one barrier
// a step. Bound: matrix and vector issue alike (exponentials, conversions), with two waves a SIMD:
// one prompt of 8192 tokens, 32 query heads of 128: 500 us, 1.1 PFLOP/s of products; without the
// exponentials 6% less, without V's decoding 14%, without lo's products 5%.

// How the kernel cuts: tokens of a split, most splits.
struct KvSplit {
  int C, S;
};
// Partial results of split rows in the workspace: unscaled sums o [S][T][Hq][D] with their maximum
// and sum of weights ml [S][T][Hq], and in how many splits a row is, count [T][Hq] (1: the row is
// in the output already, as a row of the other kernel's is). All null where nothing is split.
struct KvParts {
  float* o;
  float2* ml;
  int32_t* count;
  __device__ __forceinline__ int64_t at(const KvAttnArgs& a, int split, int t, int hq) const {
    return ((int64_t)split * a.T + t) * a.Hq + hq;
  }
};

constexpr int kManyWaves = 4, kManyRows = 32 * kManyWaves;
typedef float v16f __attribute__((ext_vector_type(16)));

template <int D>
__global__ __launch_bounds__(64 * kManyWaves, D == 256 ? 1 : 2) void k_kv_attn_many(KvAttnArgs a, int rows_least, KvSplit cut,
                                                                                     KvParts out) {
  constexpr int M = D / 32, KC = D / 64;
  __shared__ uint4 v_lds[2][4][M][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = lane & 31, half = lane >> 5;
  // Splits apart, then tiles, then heads: neighbours in the launch, which go to the eight XCDs in
  // turn, have like work (a split that only long requests have would load every second XCD).
  const int C = cut.C, S = cut.S, groups = (int)(gridDim.x / S), split = (int)(blockIdx.x / groups), h = (int)(blockIdx.x % a.H);
  RowTile w;
  if (!find_row_tile_longest(a, kManyRows, (int)(blockIdx.x % groups / a.H), groups / a.H, w)) return;
  if (w.n * a.G < rows_least) {  // the other kernel's
    if (split == 0 && out.count && (int)threadIdx.x < w.rows) {
      const int r = w.rb + (int)threadIdx.x;
      out.count[out.at(a, 0, w.q0 + r / a.G, h * a.G + r % a.G)] = 1;
    }
    return;
  }
  const int splits = splits_of(w, C, S);
  if (split >= splits) return;

  // this wave's rows, and its lane's
  const int wave_rows = min(32, w.rows - 32 * wave);  // may be none
  const int first = w.rb + min(32 * wave, w.rows - 1), last = w.rb + min(32 * wave + 31, w.rows - 1);
  const int r = min(first + col, last), pos = w.pos(r, a.G);
  const int row_lo = row_begin(a, pos), row_hi = row_end(a, w.len, pos);
  v8i q_hi[KC], q_lo[KC];
  uint32_t q_sc;
  {
    const uint16_t* src = a.q + (int64_t)(w.q0 + r / a.G) * a.q_stride + (h * a.G + r % a.G) * D;
    uint4 y[4 * KC];
    uint32_t E = 0;
#pragma unroll
    for (int c = 0; c < KC; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i)  // bytes 0..15: elements 16 half, bytes 16..31: 32 + 16 half
        y[4 * c + i] = reinterpret_cast<const uint4*>(src + 64 * c + 32 * (i / 2) + 16 * half)[i % 2];
#pragma unroll
    for (int i = 0; i < 4 * KC; ++i) E = top_exponent(y[i], E);
    E = max(E, (uint32_t)__shfl_xor((int)E, 32));
    q_sc = query_scale(E);
#pragma unroll
    for (int c = 0; c < KC; ++c)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 u = y[4 * c + 2 * i], v = y[4 * c + 2 * i + 1];
        const uint32_t e[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
        uint32_t hi[4], lo[4];
        split_fp8(e, q_sc, hi, lo);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          q_hi[c][4 * i + j] = (int)hi[j];
          q_lo[c][4 * i + j] = (int)lo[j];
        }
      }
  }

  // the workgroup's tokens, and where those end that some row of the wave sees
  const int t0 = w.lo + split * C;
  const int t1 = split == S - 1 ? w.hi : min(w.hi, t0 + C);
  const int tiles = (t1 - t0 + 15) >> 4, steps = (tiles + 3) >> 2;
  const int wave_hi = wave_rows > 0 ? row_end(a, w.len, w.pos(last, a.G)) : 0;
  const int all_lo = row_begin(a, w.pos(last, a.G)), all_hi = min(t1, row_end(a, w.len, w.pos(first, a.G)));
  const float c2 = a.scale * kLog2e;
  uint32_t shift = 23;
  asm volatile("" : "+v"(shift));  // kept in a register: scale_at
  const int P = 1 << a.log2_page;
  const int32_t* table = a.block_table + (int64_t)w.b * a.max_blocks;

  // Where 64 token tiles lie, one a lane: the window from tile 32 window on, moved every eight
  // steps, its pages fetched eight steps before. codes: the tile's K codes; scales: from there to
  // its K scales. V's codes and scales lie P D / 2 and P M past those. Tiles past the last repeat it.
  auto page_of = [&](int window) { return table[(t0 + 16 * clamp_int(32 * window + lane, 0, max(tiles - 1, 0))) >> a.log2_page]; };
  int window = 0, page = 0, next_page = 0, to_scales = 0;
  uint32_t codes_lo = 0, codes_hi = 0;
  uint64_t hidden_tiles = 0;
  auto place = [&]() {
    const bool bad = page < 0 || page >= a.num_pages;
    hidden_tiles = __ballot(bad);
    const int in_page = ((t0 + 16 * clamp_int(32 * window + lane, 0, max(tiles - 1, 0))) & (P - 1)) >> 4;
    const int64_t at = ((int64_t)(bad ? 0 : page) * a.H + h) * a.block_bytes + in_page * (8 * D);
    const uint64_t codes = (uint64_t)(uintptr_t)a.cache + (uint64_t)at;
    codes_lo = (uint32_t)codes;
    codes_hi = (uint32_t)(codes >> 32);
    to_scales = P * D - in_page * (8 * D - D / 2);
  };
  auto lane_of = [&](uint32_t x, int tile) { return (uint32_t)__builtin_amdgcn_readlane((int)x, tile - 32 * window); };

  u32x4 k[2][KC];
  uint32_t ks[2][KC];
  auto load_k = [&](int step, auto X) {  // half X of a step: 32 tokens
    constexpr int x = X;
    const int tile = 4 * step + 2 * x;
    const uint32_t lo0 = lane_of(codes_lo, tile), lo1 = lane_of(codes_lo, tile + 1), hi0 = lane_of(codes_hi, tile),
                   hi1 = lane_of(codes_hi, tile + 1), to0 = lane_of((uint32_t)to_scales, tile),
                   to1 = lane_of((uint32_t)to_scales, tile + 1);
    const bool second = lane & 16;
    const uint64_t codes = (uint64_t)(second ? hi1 : hi0) << 32 | (second ? lo1 : lo0);
    const uint64_t kc = codes + (uint32_t)(half * 256 + (lane & 15) * 16);
    const uint64_t kb = codes + ((second ? to1 : to0) + half * 16 + (lane & 12));
#pragma unroll
    for (int c = 0; c < KC; ++c) {
      k[x][c] = global<u32x4>(kc + c * 512);
      ks[x][c] = global<uint32_t>(kb + c * 32);
    }
  };
  auto scores = [&](v16f& s, auto X) {
    constexpr int x = X;
#pragma unroll
    for (int e = 0; e < 16; ++e) s[e] = 0.f;
#pragma unroll
    for (int c = 0; c < KC; ++c) {
      const v8i kv = {(int)k[x][c].x, (int)k[x][c].y, (int)k[x][c].z, (int)k[x][c].w, 0, 0, 0, 0};
      const int sc = (int)(ks[x][c] >> (8 * (lane & 3)));  // the product takes its low byte
      s = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(kv, q_hi[c], s, 4, 0, 0, sc, 0, (int)q_sc);
      s = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(kv, q_lo[c], s, 4, 0, 0, sc, 0, (int)(q_sc - 5u));
    }
  };
  typedef uint32_t words __attribute__((ext_vector_type(M)));
  words v, vs;  // the wave's token tile of a step: as in TokenTile
  auto load_v = [&](int step) {
    const int tile = 4 * step + wave;
    const uint64_t codes = (uint64_t)lane_of(codes_hi, tile) << 32 | lane_of(codes_lo, tile);
    v = global<words>(codes + (uint32_t)(P * (D / 2)) + (uint32_t)lane * (4u * M));
    vs = global<words>(codes + (lane_of((uint32_t)to_scales, tile) + P * M) + ((uint32_t)lane >> 4) * (4u * M));
  };
  // FIRST: of step 0, which alone can hold tokens before the first that is seen (with that bound in
  // the loop's decoding too: 6 x up to 1500 rows over up to 12001 tokens 280 us, so 271).
  auto decode_v = [&](int step, int buf, auto FIRST) {
    constexpr bool kFirst = FIRST;
    const int tile = 4 * step + wave, t = t0 + 16 * tile;
    TokenTile<D> x;
#pragma unroll
    for (int j = 0; j < M; ++j) {
      x.v[j] = v[j];
      x.vs[j] = vs[j];
    }
    const bool hidden = (hidden_tiles >> (tile - 32 * window)) & 1u;
    if ((kFirst && t < w.seen) || t + 16 > t1 || hidden) x.mask(t + 4 * (lane >> 4), kFirst ? w.seen : INT_MIN, hidden ? 0 : t1);
    uint2* dst = reinterpret_cast<uint2*>(&v_lds[buf][wave][0][((lane >> 4) & 1) * 32 + (lane & 15)]) + (lane >> 5);
    static_for<M>([&](auto J) {
      constexpr int j = J;
      const uint32_t c0 = decode2<0>(x.v[j], x.template scale<0, j>(shift));
      const uint32_t c1 = decode2<1>(x.v[j], x.template scale<1, j>(shift));
      const uint32_t c2_ = decode2<2>(x.v[j], x.template scale<2, j>(shift));
      const uint32_t c3 = decode2<3>(x.v[j], x.template scale<3, j>(shift));
      dst[j * 128] = make_uint2(__builtin_amdgcn_perm(c1, c0, 0x05040100), __builtin_amdgcn_perm(c3, c2_, 0x05040100));
      dst[j * 128 + 32] = make_uint2(__builtin_amdgcn_perm(c1, c0, 0x07060302), __builtin_amdgcn_perm(c3, c2_, 0x07060302));
    });
  };

  float m = kLowest, l = 0.f;
  v16f o[M];
#pragma unroll
  for (int j = 0; j < M; ++j)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[j][e] = 0.f;

  // Half a step at a time: the scores of the next half are in the matrix pipe while this half's
  // weights are worked out, and the next step's values are decoded under this step's products.
  constexpr std::integral_constant<int, 0> H0{};
  constexpr std::integral_constant<int, 1> H1{};
  v16f s0, s1;
  if (steps > 0) {
    page = page_of(0);
    next_page = page_of(1);
    place();
    load_v(0);
    load_k(0, H0);
    load_k(0, H1);
    decode_v(0, 0, std::true_type{});
    load_v(1);
    scores(s0, H0);
    load_k(1, H0);
  }
  __syncthreads();
  for (int st = 0; st < steps; ++st) {
    const int t = t0 + 64 * st;
    if ((st >> 3) != window) {
      ++window;
      page = next_page;
      next_page = page_of(window + 1);
      place();
    }
    const uint32_t hidden = (uint32_t)(hidden_tiles >> (4 * st - 32 * window)) & 15u;
    const bool masked = t < all_lo || t + 64 > all_hi || hidden;
    // The maximum of a half's scores, and the sums rescaled if it passes the one in use by kLag.
    auto settle = [&](v16f& s, auto X) {
      constexpr int x = X;
      if (masked) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int tok = t + 32 * x + 8 * (e / 4) + 4 * half + e % 4;
          if (tok < row_lo || tok >= min(row_hi, t1) || ((hidden >> (2 * x + e / 8)) & 1u)) s[e] = -INFINITY;
        }
      }
      float top = s[0];
#pragma unroll
      for (int e = 1; e < 16; ++e) top = fmaxf(top, s[e]);
      top *= c2;
      if (__any(top > m + kLag)) {  // as in the kernel above
        top = fmaxf(top, __shfl_xor(top, 32));
        const float m1 = fmaxf(m, top), alpha = __builtin_amdgcn_exp2f(m - m1);
        m = m1;
        l *= alpha;
#pragma unroll
        for (int j = 0; j < M; ++j)
#pragma unroll
          for (int e = 0; e < 16; ++e) o[j][e] *= alpha;
      }
    };
    uint32_t p[8];
    auto weights = [&](const v16f& s) {
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        p[e / 2] = pack_bf16(__builtin_amdgcn_exp2f(__builtin_fmaf(s[e], c2, -m)),
                             __builtin_amdgcn_exp2f(__builtin_fmaf(s[e + 1], c2, -m)));
        l = add_pair(l, p[e / 2]);
      }
    };
    // A half's values leave LDS before its weights are worked out: read where they are used, every
    // product waits for them.
    bf16x8 vt[2][M];
    auto fetch = [&](auto X) {
      constexpr int x = X;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < M; ++j) vt[i][j] = __builtin_bit_cast(bf16x8, v_lds[st & 1][2 * x + i][j][lane]);
      __builtin_amdgcn_sched_barrier(0);
    };
    auto values = [&]() {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bf16x8 pt = as_bf16x8(p[4 * i], p[4 * i + 1], p[4 * i + 2], p[4 * i + 3]);
#pragma unroll
        for (int j = 0; j < M; ++j) o[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vt[i][j], pt, o[j], 0, 0, 0);
      }
    };
    if (t < wave_hi) {  // else no row of the wave sees this or a later step
      settle(s0, H0);
      fetch(H0);
      scores(s1, H1);
      weights(s0);
      load_k(st + 1, H1);
      values();
      settle(s1, H1);
      fetch(H1);
      scores(s0, H0);
      weights(s1);
      load_k(st + 2, H0);
      decode_v(st + 1, (st + 1) & 1, std::false_type{});
      load_v(st + 2);
      values();
    } else {
      decode_v(st + 1, (st + 1) & 1, std::false_type{});
      load_v(st + 2);
    }
    __syncthreads();
  }

  // Out through LDS (the wave's quarter of the values' place), so that a row's bytes are stored
  // side by side: a row of D bf16, or half a row of FP32 sums at a time, in pieces of 16 bytes whose
  // order in LDS depends on the row (all rows' first pieces would meet in one bank).
  l += __shfl_xor(l, 32);
  constexpr int kPieces = D / 8;
  uint4* mine = reinterpret_cast<uint4*>(v_lds) + wave * 32 * kPieces;
  const int t = w.q0 + r / a.G, hq = h * a.G + r % a.G;
  const int64_t at = out.at(a, split, t, hq);
  if (32 * wave + col < w.rows && half == 0) {
    if (splits > 1) out.ml[at] = make_float2(m, l);
    if (split == 0 && out.count) out.count[at] = splits;
  }
  const float inv = splits > 1 ? 1.f : l > 0.f ? 1.f / l : 0.f;
  uint8_t* row_out = splits > 1 ? reinterpret_cast<uint8_t*>(out.o + at * D)
                                : reinterpret_cast<uint8_t*>(a.out + (int64_t)t * a.out_stride + hq * D);
  const uint64_t row_at = (uint64_t)(uintptr_t)row_out;
  auto put = [&](int piece, uint4 u) { mine[col * kPieces + (piece ^ (col & (kPieces - 1)))] = u; };
  auto store = [&](int byte) {  // rows whose pieces the wave has put, to `byte` of each
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPieces / 2; ++i) {
      const int row = (64 * i + lane) / kPieces, piece = lane % kPieces;
      const uint64_t to = (uint64_t)(uint32_t)__shfl((int)(row_at >> 32), row) << 32 | (uint32_t)__shfl((int)row_at, row);
      const uint4 u = mine[row * kPieces + (piece ^ (row & (kPieces - 1)))];
      if (32 * wave + row < w.rows) *(__attribute__((address_space(1))) u32x4*)(to + byte + 16 * piece) = (u32x4){u.x, u.y, u.z, u.w};
    }
    __syncthreads();
  };
  if (splits == 1) {
#pragma unroll
    for (int j = 0; j < M; ++j)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        uint32_t f[4];  // elements 32 j + 16 x + 8 half on: even ones from rows 0 .. 15 of V^T, odd ones from 16 on
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = pack_bf16(o[j][4 * x + e] * inv, o[j][8 + 4 * x + e] * inv);
        put(4 * j + 2 * x + half, make_uint4(f[0], f[1], f[2], f[3]));
      }
    store(0);
  } else {
#pragma unroll
    for (int part = 0; part < 2; ++part) {
#pragma unroll
      for (int j = 0; j < M / 2; ++j)
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const v16f& y = o[part * (M / 2) + j];
            const v4f z = {y[4 * x + e], y[8 + 4 * x + e], y[4 * x + e + 1], y[8 + 4 * x + e + 1]};
            put(8 * j + 4 * x + 2 * half + e / 2, __builtin_bit_cast(uint4, z));
          }
      store(part * 2 * D);
    }
  }
}

// Joins the splits of the many-rows kernel, a wave a row and query head (bound: the FP32 sums' bytes). Whether a row is split,
// and in how many, is read with the maxima: two dependent loads to the first sums.
template <int D>
__global__ __launch_bounds__(256) void k_kv_attn_join(KvAttnArgs a, int S, KvParts in) {
  constexpr int E = D / 64;
  typedef float vec __attribute__((ext_vector_type(E)));
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), each = (int64_t)a.T * a.Hq;
  const int lane = threadIdx.x & 63;
  if (row >= each) return;
  const int t = (int)(row / a.Hq), hq = (int)(row % a.Hq);
  if (t < a.cu_q[0] || t >= a.cu_q[a.B]) return;  // no request's
  const int splits = min(in.count[row], S);
  if (splits <= 1) return;  // written already
  float m = kLowest, l = 0.f, x[E];
#pragma unroll
  for (int e = 0; e < E; ++e) x[e] = 0.f;
  for (int s = lane; s < splits; s += 64) m = fmaxf(m, in.ml[s * each + row].x);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
#pragma unroll 4
  for (int s = 0; s < splits; ++s) {
    const float2 ml = in.ml[s * each + row];
    const vec y = *reinterpret_cast<const vec*>(in.o + (s * each + row) * D + lane * E);
    const float f = __builtin_amdgcn_exp2f(ml.x - m);
    l += ml.y * f;
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] += y[e] * f;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  uint16_t* dst = a.out + (int64_t)t * a.out_stride + hq * D + lane * E;
  if constexpr (E == 1) {
    dst[0] = (uint16_t)f32_to_bf16_rne(x[0] * inv);
  } else {
#pragma unroll
    for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16(x[e] * inv, x[e + 1] * inv);
  }
}

// ------------------------------------------------------------------------------- the launch

// Workers that share the few-rows work: two a CU, twice that at D = 64 (whose registers let four run)
// for kManySegments and more. 960 / 32 segments of D = 64: 91 / 22 us at 512 workers, 75 / 25 at 1024;
// 128 x 8 heads x up to 8192 tokens at D = 128: 133 at 512, 152 at 1024. At least kLeastUnits units
// each: 1 x 8 heads x 8192 tokens 15 us with 12, 19 with 4.
constexpr int64_t kWorkers = 512, kManySegments = 256, kLeastUnits = 12;
// Segments stay whole up to kWholeTokens tokens, or kWholeTimes of them for each segment there is (the
// chip's workgroups then even out by their number). Whole / shared at D = 128, lengths from an eighth to
// all of so many tokens. The rule keeps whole: 1 x 8 heads x 1200 12.8 / 14.4 us, 8 x 8 x 1200 14.5 / 17.3,
// 64 x 8 x 2000 25.5 / 31.2, 128 x 8 x 4000 79 / 84, 256 x 8 x 700 37 / 53, 256 x 8 x 4000 145 / 145. It
// shares: 1 x 8 x 1500 14.2 / 13.4, 1 x 8 x 2400 19.4 / 14.6, 8 x 8 x 2400 23.9 / 18.1, 64 x 8 x 4000 49 / 48,
// x 8192 90 / 74, 128 x 8 x 8192 149 / 141, 256 x 1 x 4000 36.5 / 29.5. Near the border it can take the slower
// side: 64 x 8 x 2400 33.9 / 36.7 (shared; 51.5 / 58.2 at D = 256, 22.1 / 29.5 at 64), 256 x 1 x 2000
// 22.2 / 24.6 (shared), 256 x 8 x 8192 277 / 254 and 512 x 8 x 8192 494 / 476 (whole).
constexpr int64_t kWholeTokens = 1280, kWholeTimes = 4;
constexpr int64_t kManySlots = 512, kLeastTokens = 512;
// All requests in the few-rows kernel, in tiles of 32 rows (16 at D = 256, or where no request has more):
// up to kFewRows rows each and kFewAverage on average. Otherwise requests of more rows than a tile go to the
// many-rows kernel. This way / otherwise, 4 heads over up to 4000 tokens, rows from an eighth to all of so
// many: 64 requests of 16 rows 30 / 49 us, 32 38 / 87, 64 53 / 95; 8 requests of 16 rows 19.6 / 24.4, 64
// 29.5 / 54; 1 of 64 rows 17.4 / 24.1; 16 of 128 rows, 63 on average, 33 / 69, 4 of 128, 64, 30 / 31; at
// D = 256 64 of 32 rows 62 / 160, 8 of 64 31 / 66. But 64 requests of 128 rows each 142 this way, 107
// otherwise. Beside requests of more rows the few-rows kernel takes those of one tile of 16 rows (32 where
// 16 heads are not enough for one): 20 requests, most of one row, 14 us in tiles of 16, 17.5 in tiles of 32.
constexpr int64_t kFewRows = 128, kFewAverage = 64;

// Which kernels run: requests of at most rows_most rows in the few-rows kernel (0: it is not
// launched), the others in the many-rows kernel (rows_most == kAllRows: not launched).
struct KvPlan {
  int rows_most;
  int R, lg;  // few rows: rows of a tile, log2 of the workers
  bool cut;   // whether shares cut segments, and if so
  int parts, row_groups;  // how many parts a long segment has, fours of rows in a tile
  KvSplit many;
};

// Row tiles of the few-rows kernel: beside the other kernel each request's first.
int64_t few_tiles(const KvAttnSizes& z, const KvPlan& p) { return p.rows_most == kAllRows ? row_tiles(z, p.R) : z.B; }
size_t few_bytes(const KvAttnSizes& z, const KvPlan& p) {
  return p.rows_most > 0 && p.cut ? ((size_t)1 << p.lg) * (2 * p.R * (z.D + 2) * 4 + 16) : 0;
}
size_t many_bytes(const KvAttnSizes& z, const KvPlan& p) {
  return p.rows_most < kAllRows && p.many.S > 1 ? (size_t)(z.T * z.Hq * (p.many.S * (z.D + 2) + 1) * 4) : 0;
}

KvPlan plan_of(const KvAttnSizes& z, size_t workspace_bytes) {
  KvPlan p;
  const int64_t G = z.Hq / z.H, max_q = std::min(z.max_q, z.T), rows = max_q * G, all = std::min(z.T, z.B * max_q) * G;
  const bool few = rows <= kFewRows && all <= kFewAverage * z.B;
  p.R = rows <= 16 || (!few && G <= 16) || z.D == 256 ? 16 : 32;
  if (few && (z.T * G / p.R + z.B) * z.H <= (1 << 23)) p.rows_most = kAllRows;  // a launch holds under 2^32 threads
  else if (z.T == z.B * max_q || G > p.R) p.rows_most = 0;  // no request has so few rows
  else p.rows_most = p.R;
  const int64_t longest = std::min(z.max_kv, (int64_t)1 << 30);
  // tokens that a tile of R rows sees at most
  auto span = [&](int64_t R) { return z.window && z.window < longest ? std::min(longest, z.window + R / G + 16) : longest; };

  // few rows
  const int64_t segments = z.H * z.B * (p.rows_most == kAllRows ? (rows + p.R - 1) / p.R : 1);
  const int64_t units = segments * ((span(p.R) + 31) / 32 + kSegmentUnits);
  p.cut = span(p.R) > std::max(kWholeTokens, kWholeTimes * segments);
  const int64_t most = z.D == 64 && segments >= kManySegments ? 2 * kWorkers : kWorkers;
  for (p.lg = 0; ((int64_t)2 << p.lg) <= std::min<int64_t>(most, units / kLeastUnits); ++p.lg) {
  }
  p.parts = (int)(((int64_t)1 << p.lg) / std::max<int64_t>(segments, 1)) + 1;
  p.row_groups = (int)((std::min<int64_t>(rows, p.R) + 3) / 4);

  // Many rows: as many splits as the groups with rows leave room for on the chip (kManySlots of them
  // run at once, half as many at D = 256), at least kLeastTokens each. More cost the joins more than
  // they even out: 3 requests of up to 2049 rows at D = 256 65 us unsplit, 113 in 3; 4 x up to 300 rows
  // over up to 16000 tokens 59 us by this rule, 74 with more.
  const int64_t tiles = z.H * std::max<int64_t>(z.T * G / kManyRows, 1), launched = z.H * row_tiles(z, kManyRows);
  const int64_t slots = z.D == 256 ? kManySlots / 2 : kManySlots, seen = span(kManyRows);
  const int64_t S = std::max<int64_t>(1, std::min({slots / tiles, seen / kLeastTokens, ((int64_t)1 << 20) / launched}));
  p.many.C = (int)((seen + 64 * S - 1) / (64 * S) * 64);
  p.many.S = (int)std::max<int64_t>(1, (seen + p.many.C - 1) / p.many.C);

  if (few_bytes(z, p) + many_bytes(z, p) > workspace_bytes) p.many = {1 << 30, 1};
  if (few_bytes(z, p) > workspace_bytes) p.cut = false;
  return p;
}

template <int D>
hipError_t launch(const KvAttnArgs& a, const KvAttnSizes& z, const KvPlan& p, void* ws, hipStream_t st) {
  hipError_t e = hipSuccess;
  if (p.rows_most > 0) {
    const size_t slots = ((size_t)2 << p.lg) * p.R;
    KvShares sh = {p.lg, p.rows_most, nullptr, nullptr, nullptr};
    constexpr int D2 = D == 256 ? 64 : D;  // R is 16 at D = 256
    const dim3 block(kThreads);
    if (p.cut) {
      sh.o = static_cast<float*>(ws);
      sh.ml = reinterpret_cast<float2*>(sh.o + slots * D);
      sh.seams = reinterpret_cast<int4*>(sh.ml + slots);
      const dim3 grid(1u << p.lg);
      if (p.R == 16) hipLaunchKernelGGL((k_kv_attn_few<D, 1, true>), grid, block, 0, st, a, sh);
      else hipLaunchKernelGGL((k_kv_attn_few<D2, 2, true>), grid, block, 0, st, a, sh);
    } else {
      const dim3 grid((unsigned)(few_tiles(z, p) * z.H));
      if (p.R == 16) hipLaunchKernelGGL((k_kv_attn_few<D, 1, false>), grid, block, 0, st, a, sh);
      else hipLaunchKernelGGL((k_kv_attn_few<D2, 2, false>), grid, block, 0, st, a, sh);
    }
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (p.cut) {
      // Many parts: four waves a row, and few segments, so of eight neighbouring workers one or two have a
      // seam at most. Four waves / one: 65 parts 6.7 / 16 us, 33 parts 5.9 / 9.0, 17 parts 7.0 / 6.6, 9 parts 8.1 / 5.6.
      const unsigned workers = 1u << p.lg;
      if (p.parts > 24)
        hipLaunchKernelGGL((k_kv_attn_seams<D, 4>), dim3((workers + 7) / 8, p.row_groups), dim3(1024), 0, st, a, sh, p.R, 8);
      else
        hipLaunchKernelGGL((k_kv_attn_seams<D, 1>), dim3(workers, p.row_groups), dim3(256), 0, st, a, sh, p.R, 1);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  if (p.rows_most < kAllRows) {
    const size_t each = (size_t)a.T * a.Hq;
    KvParts parts = {nullptr, nullptr, nullptr};
    if (p.many.S > 1) {
      parts.o = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + few_bytes(z, p));
      parts.ml = reinterpret_cast<float2*>(parts.o + p.many.S * each * D);
      parts.count = reinterpret_cast<int32_t*>(parts.ml + p.many.S * each);
    }
    const dim3 grid((unsigned)((int64_t)row_tiles(z, kManyRows) * a.H * p.many.S)), block(64 * kManyWaves);
    hipLaunchKernelGGL((k_kv_attn_many<D>), grid, block, 0, st, a, p.rows_most + 1, p.many, parts);
    e = hipGetLastError();
    if (e != hipSuccess || p.many.S == 1) return e;
    hipLaunchKernelGGL((k_kv_attn_join<D>), dim3((unsigned)((each + 3) / 4)), dim3(256), 0, st, a, p.many.S, parts);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace

size_t kv_attn_workspace_bytes(const KvAttnSizes& z) {
  const KvPlan p = plan_of(z, ~(size_t)0);
  return few_bytes(z, p) + many_bytes(z, p);
}

hipError_t launch_kv_attn(const KvAttnArgs& a, const KvAttnSizes& z, void* workspace, size_t workspace_bytes,
                          hipStream_t st) {
  const KvPlan p = plan_of(z, workspace_bytes);
  if (a.D == 64) return launch<64>(a, z, p, workspace, st);
  if (a.D == 128) return launch<128>(a, z, p, workspace, st);
  return launch<256>(a, z, p, workspace, st);
}

void kv_attn_plan(const KvAttnSizes& z, size_t workspace_bytes, char* buf, size_t len) {
  if (z.B == 0 || z.T == 0) {
    std::snprintf(buf, len, "none");
    return;
  }
  const KvPlan p = plan_of(z, workspace_bytes);
  char few[96] = "", many[96] = "";
  if (p.rows_most > 0)
    std::snprintf(few, sizeof few, p.cut ? "k_kv_attn_few<%d, %d, true> workers=%d + k_kv_attn_seams" : "k_kv_attn_few<%d, %d, false>",
                  (int)z.D, p.R / 16, 1 << p.lg);
  if (p.rows_most < kAllRows)
    std::snprintf(many, sizeof many, "k_kv_attn_many<%d> C=%d S=%d%s", (int)z.D, p.many.C, p.many.S,
                  p.many.S > 1 ? " + k_kv_attn_join" : "");
  std::snprintf(buf, len, "%s%s%s", few, few[0] && many[0] ? " + " : "", many);
}

}  // namespace mx
