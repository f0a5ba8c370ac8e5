// mx_kv.hip - the paged MXFP4 key/value cache: block tables and slots from the requests'
// lengths, the write (quantizing) and the read back.
#include "mx_kv.h"

#include "mx_device.h"

namespace mx {
namespace {

// ------------------------------------------------------------------------------- tables
//
// Three running sums over the requests decide everything: new rows, pages taken, pages given
// back. With cnt pages on the stack, `back` given back and `take` taken, the stack after the
// pushes is virtual[i] = free_pages[i] (i < cnt) or the (i - cnt)-th page given back, and the
// k-th page taken is virtual[cnt + back - 1 - k]. No step needs another's writes: entries
// below cnt are only read, those from cnt on only written, rows of the table either give
// (read) or take (written), so every row and page is worked out on its own from the sums.
// Bound: launch latency at decoding sizes; one dependent chain of searches per row beyond. 96
// requests, a new row each: 5.4 us, 8.0 where some give pages back (a second search); 48 prompts,
// 402000 rows: 4.6 us of sums and 5.4 of rows.

constexpr int kScanThreads = 1024;
constexpr int kOneGroupRequests = 1024;  // whose sums fit 12 KB of LDS
// Rows that one workgroup fills by itself; past them the sums go through the workspace to a
// second launch over the whole chip. 96 requests, one launch / two: 96 rows 5.4 / 6.8 us, 1900 rows
// 6.7 / 8.5, 4900 9.4 / 8.6, 7600 11.6 / 8.9; 1000 requests and 11100 rows 18.2 / 9.8.
constexpr int kOneGroupRows = 4096;
constexpr uint32_t kCap = (1u << 31) - 1;  // sums saturate here: larger than any valid one

__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, kCap); }  // a, b <= kCap

struct KvSums {
  int ok, cnt, back, take, rows;
};

__device__ __forceinline__ int pages_of(int len, int lg) { return (int)(((int64_t)len + (1 << lg) - 1) >> lg); }

// The largest b < n with sums[b] <= x, sums non-decreasing with sums[0] = 0 and x >= 0.
__device__ __forceinline__ int find(const int32_t* sums, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// Inclusive scan over the workgroup of three saturating sums.
__device__ __forceinline__ void scan3(uint32_t (&x)[3], uint32_t (*wave)[3]) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1)
#pragma unroll
    for (int c = 0; c < 3; ++c) {
      const uint32_t y = __shfl_up(x[c], d);
      if (lane >= d) x[c] = sat_add(x[c], y);
    }
  __syncthreads();  // the previous round's reads of wave[] are over
  if (lane == 63)
#pragma unroll
    for (int c = 0; c < 3; ++c) wave[w][c] = x[c];
  __syncthreads();
#pragma unroll
  for (int c = 0; c < 3; ++c) {
    uint32_t base = 0;
    for (int i = 0; i < w; ++i) base = sat_add(base, wave[i][c]);
    x[c] = sat_add(x[c], base);
  }
}

// The sums by one workgroup, to rows/take/back[0 .. B] (LDS or workspace; entry 0 is 0), and
// what they come to.
__device__ KvSums tables_scan(const KvTablesArgs& a, int32_t* rows, int32_t* take, int32_t* back) {
  __shared__ uint32_t wave[kScanThreads / 64][3];
  __shared__ uint32_t total[3];
  __shared__ int bad;
  if (threadIdx.x == 0) {
    rows[0] = take[0] = back[0] = 0;
    bad = 0;
    total[0] = total[1] = total[2] = 0;
  }
  __syncthreads();
  for (int b0 = 0; b0 < a.B; b0 += kScanThreads) {
    const int b = b0 + (int)threadIdx.x;
    uint32_t x[3] = {0, 0, 0};
    if (b < a.B) {
      const int o = a.old_lens[b], n = a.new_lens[b];
      if (o < 0 || n < 0 || pages_of(max(o, n), a.log2_page) > a.max_blocks) {
        bad = 1;
      } else {
        const int held = pages_of(o, a.log2_page), want = pages_of(n, a.log2_page);
        x[0] = (uint32_t)max(n - o, 0);
        x[1] = (uint32_t)max(want - held, 0);
        x[2] = (uint32_t)max(held - want, 0);
      }
    }
    scan3(x, wave);
#pragma unroll
    for (int c = 0; c < 3; ++c) x[c] = sat_add(x[c], total[c]);
    if (b < a.B) {
      rows[b + 1] = (int32_t)x[0];
      take[b + 1] = (int32_t)x[1];
      back[b + 1] = (int32_t)x[2];
    }
    __syncthreads();
    if (threadIdx.x == kScanThreads - 1)
#pragma unroll
      for (int c = 0; c < 3; ++c) total[c] = x[c];
    __syncthreads();
  }
  KvSums s;
  s.cnt = *a.free_count;
  s.rows = (int)total[0];
  s.take = (int)total[1];
  s.back = (int)total[2];
  const bool valid = !bad && s.cnt >= 0 && s.cnt <= a.capacity && s.rows <= a.T_max &&
                     (int64_t)s.cnt + s.back - s.take <= a.capacity;
  const int64_t lacks = (int64_t)s.take - s.back - s.cnt;
  s.ok = valid && lacks <= 0;
  __syncthreads();  // everybody has read free_count, which may be free_count_out
  if (threadIdx.x == 0) {
    *a.status = !valid ? -1 : lacks > 0 ? (int)lacks : 0;
    *a.free_count_out = s.ok ? s.cnt + s.back - s.take : s.cnt;
  }
  for (int b = (int)threadIdx.x; b <= a.B; b += kScanThreads) a.cu_q[b] = s.ok ? rows[b] : 0;
  return s;
}

// The i-th page given back.
__device__ __forceinline__ int given_back(const KvTablesArgs& a, const int32_t* back, int i) {
  const int b = find(back, a.B, i);
  return a.block_table[(int64_t)b * a.max_blocks + pages_of(a.new_lens[b], a.log2_page) + i - back[b]];
}

__device__ __forceinline__ void tables_fill(const KvTablesArgs& a, const KvSums& s, const int32_t* rows,
                                            const int32_t* take, const int32_t* back, int first, int step) {
  const int P = 1 << a.log2_page;
  for (int t = first; t < a.T_max; t += step) {
    int64_t slot = -1;
    int pos = -1;
    if (s.ok && t < s.rows) {
      const int b = find(rows, a.B, t);
      pos = a.old_lens[b] + t - rows[b];
      const int blk = pos >> a.log2_page, held = pages_of(a.old_lens[b], a.log2_page);
      int32_t* entry = a.block_table + (int64_t)b * a.max_blocks + blk;
      int page;
      if (blk < held) {
        page = *entry;
      } else {
        const int v = s.cnt + s.back - 1 - (take[b] + blk - held);
        page = v < s.cnt ? a.free_pages[v] : given_back(a, back, v - s.cnt);
        if ((pos & (P - 1)) == 0) *entry = page;  // a new page's first token is always a new row
      }
      slot = ((int64_t)page << a.log2_page) + (pos & (P - 1));
    }
    a.slots[t] = slot;
    a.positions[t] = pos;
  }
  if (s.ok)
    for (int i = first; i < s.back - s.take; i += step) a.free_pages[s.cnt + i] = given_back(a, back, i);
}

__global__ __launch_bounds__(kScanThreads) void k_kv_tables(KvTablesArgs a) {
  __shared__ int32_t rows[kOneGroupRequests + 1], take[kOneGroupRequests + 1], back[kOneGroupRequests + 1];
  const KvSums s = tables_scan(a, rows, take, back);
  tables_fill(a, s, rows, take, back, (int)threadIdx.x, kScanThreads);
}

// workspace: KvSums, padded to 32 bytes, then rows, take and back of B + 1 entries each
__global__ __launch_bounds__(kScanThreads) void k_kv_tables_scan(KvTablesArgs a, int32_t* ws) {
  int32_t* sums = ws + 8;
  const KvSums s = tables_scan(a, sums, sums + a.B + 1, sums + 2 * (a.B + 1));
  if (threadIdx.x == 0) *reinterpret_cast<KvSums*>(ws) = s;
}

__global__ __launch_bounds__(256) void k_kv_tables_fill(KvTablesArgs a, const int32_t* ws) {
  const KvSums s = *reinterpret_cast<const KvSums*>(ws);
  const int32_t* sums = ws + 8;
  tables_fill(a, s, sums, sums + a.B + 1, sums + 2 * (a.B + 1), (int)(blockIdx.x * 256 + threadIdx.x),
              (int)(gridDim.x * 256));
}

bool one_group(int64_t B, int64_t T_max) { return B <= kOneGroupRequests && T_max <= kOneGroupRows; }

// ------------------------------------------------------------------------------- write, read

// The largest bf16 exponent field of 8 elements.
__device__ __forceinline__ uint32_t top_field(const uint4& u) {
  const uint32_t x[4] = {u.x, u.y, u.z, u.w};
  u16x2 m = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, x[i] & 0x7F807F80u));
  return (uint32_t)(m.x > m.y ? m.x : m.y) >> 7;
}
__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}
// 8 elements' codes at a block's scale byte: as quant_block, a scale byte of 0 is passed as 2^-127.
__device__ __forceinline__ uint32_t quant8(const uint4& x, uint32_t s) {
  const float sc = __builtin_bit_cast(float, s ? s << 23 : 0x00400000u);
  uint32_t r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(0, __builtin_bit_cast(bf16x2, x.x), sc, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, x.y), sc, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, x.z), sc, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, x.w), sc, 3);
}

// A workgroup quantizes 16 rows of 128 elements (two heads of 64, a head of 128 or half a head of
// 256): a thread has 8 elements of a row, four neighbours a block. K's codes go out as they come, 16
// bytes a block. V's lie four tokens to a word in the cache: its bytes meet in LDS, and wherever four
// rows of the workgroup are the four tokens of a word, whatever row the first of them is, whole words
// are written; other rows' bytes one by one.
// Bound: HBM, 4 bytes read and 17/16 written per element of K and V; at decoding sizes the launch.
// 16411 rows x 8 x 128: 21.4 us (4.0 TB/s); 96 rows 3.7. With 64 rows a workgroup, fewer of whose
// words are incomplete, 22.7 us (1024 rows 7.2 against 4.6): the L2 puts the words together as well.
constexpr int kWriteRows = 16;
__global__ __launch_bounds__(256) void k_kv_write(const uint16_t* __restrict__ k, int64_t k_stride,
                                                  const uint16_t* __restrict__ v, int64_t v_stride,
                                                  const int64_t* __restrict__ slots, int64_t T,
                                                  uint8_t* __restrict__ cache, int64_t num_slots, int lg, int heads,
                                                  int D) {
  __shared__ uint32_t v_words[kWriteRows][17];  // a row's 16 words of codes (one more spreads rows over the banks)
  __shared__ int64_t row_slot[kWriteRows];      // -1: writes nothing
  const KvLayout L = {1 << lg, D};
  const int m = D / 32, c = threadIdx.x & 15, r = threadIdx.x >> 4;
  const int e = (int)blockIdx.y * 128 + 8 * c, h = e / D, d = e % D;  // this thread's 8 elements of row r
  for (int64_t t0 = (int64_t)blockIdx.x * kWriteRows; t0 < T; t0 += (int64_t)gridDim.x * kWriteRows) {
    const int64_t t = t0 + r;
    int64_t slot = t < T ? slots[t] : -1;
    if (slot >= num_slots) slot = -1;
    const bool has = h < heads && slot >= 0;
    const int tok = (int)(slot & (L.P - 1));
    uint8_t* blk = cache + ((slot >> lg) * heads + h) * L.block_bytes();
    uint4 kx = make_uint4(0, 0, 0, 0), vx = kx;
    if (has) {
      kx = *reinterpret_cast<const uint4*>(k + t * k_stride + e);
      vx = *reinterpret_cast<const uint4*>(v + t * v_stride + e);
    }
    uint32_t top = top_field(kx) | top_field(vx) << 16;  // both largest exponents
    top = max_halves(top, (uint32_t)__shfl_xor((int)top, 1));
    top = max_halves(top, (uint32_t)__shfl_xor((int)top, 2));
    const uint32_t ek = top & 0xFFFFu, ev = top >> 16, sk = ek > 2u ? ek - 2u : 0u, sv = ev > 2u ? ev - 2u : 0u;
    v_words[r][c] = quant8(vx, sv);
    if (c == 0) row_slot[r] = slot;
    if (has) {
      *reinterpret_cast<uint32_t*>(blk + L.k_code(tok, d)) = quant8(kx, sk);
      if ((c & 3) == 0) {
        blk[L.k_scale(tok, d)] = (uint8_t)sk;
        blk[L.v_scale(tok, d)] = (uint8_t)sv;
      }
    }
    __syncthreads();
    if (has) {  // V's codes: the first of four tokens writes for all
      const int at = (int)(slot & 3), first = r - at;
      bool four = first >= 0 && first + 3 < kWriteRows;
      if (four)
#pragma unroll
        for (int x = 0; x < 4; ++x) four = four && row_slot[first + x] == slot - at + x;
      if (!four) {
        const uint32_t w = v_words[r][c];
#pragma unroll
        for (int b = 0; b < 4; ++b) blk[L.v_code(tok, d + 2 * b)] = (uint8_t)(w >> (8 * b));
      } else if (at == 0) {
        // bytes of four tokens, transposed: word b gets byte b of each
        const uint32_t w0 = v_words[r][c], w1 = v_words[r + 1][c], w2 = v_words[r + 2][c], w3 = v_words[r + 3][c];
        const uint32_t a = __builtin_amdgcn_perm(w1, w0, 0x05010400), b = __builtin_amdgcn_perm(w3, w2, 0x05010400);
        const uint32_t p = __builtin_amdgcn_perm(w1, w0, 0x07030602), q = __builtin_amdgcn_perm(w3, w2, 0x07030602);
        uint32_t* dst = reinterpret_cast<uint32_t*>(blk + L.v_code(tok, d));
        dst[0] = __builtin_amdgcn_perm(b, a, 0x05040100);
        dst[m] = __builtin_amdgcn_perm(b, a, 0x07060302);
        dst[2 * m] = __builtin_amdgcn_perm(q, p, 0x05040100);
        dst[3 * m] = __builtin_amdgcn_perm(q, p, 0x07060302);
      }
    }
    __syncthreads();  // before the next rows take their place
  }
}

// 8 codes of one scale, as bf16 (an E2M1 value times a power of two is exact in bf16).
__device__ __forceinline__ uint4 decode8(uint32_t codes, uint32_t scale) {
  const float sc = __builtin_bit_cast(float, scale << 23);  // 0 acts as 2^-127
  return make_uint4(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, sc, 0)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, sc, 1)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, sc, 2)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, sc, 3)));
}

// One thread per 8 elements of one head of one row; its V codes are four bytes of as many words,
// which the rows beside it find in L1. Bound: HBM, 17/16 bytes read and 4 written per element of K
// and V: 16411 rows x 8 x 128 24.6 us (3.5 TB/s); 96 rows 3.2.
__global__ __launch_bounds__(256) void k_kv_read(const uint8_t* __restrict__ cache, int64_t num_slots, int lg,
                                                 int heads, int D, const int64_t* __restrict__ slots, int64_t units,
                                                 uint16_t* __restrict__ k, uint16_t* __restrict__ v) {
  const int m = D / 8, per = heads * m;
  const KvLayout L = {1 << lg, D};
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < units; u += (int64_t)gridDim.x * 256) {
    const int64_t t = u / per;
    const int h = (int)(u % per) / m, d = (int)(u % m) * 8;
    const int64_t slot = slots[t];
    if (slot < 0 || slot >= num_slots) continue;
    const int tok = (int)(slot & (L.P - 1));
    const uint8_t* blk = cache + ((slot >> lg) * heads + h) * L.block_bytes();
    *reinterpret_cast<uint4*>(k + u * 8) =
        decode8(*reinterpret_cast<const uint32_t*>(blk + L.k_code(tok, d)), blk[L.k_scale(tok, d)]);
    uint32_t c = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) c |= (uint32_t)blk[L.v_code(tok, d + 2 * b)] << (8 * b);
    *reinterpret_cast<uint4*>(v + u * 8) = decode8(c, blk[L.v_scale(tok, d)]);
  }
}

}  // namespace

// Workgroups of 256 threads for `units` threads' worth of work; past 2^20 they loop (a launch
// holds fewer than 2^32 threads).
static unsigned groups_of(int64_t units) { return (unsigned)min((units + 255) / 256, (int64_t)1 << 20); }

size_t kv_tables_workspace_bytes(int64_t B, int64_t T_max) {
  return one_group(B, T_max) ? 0 : (size_t)(32 + 12 * (B + 1));
}

hipError_t launch_kv_tables(const KvTablesArgs& a, void* workspace, hipStream_t st) {
  if (one_group(a.B, a.T_max)) {
    hipLaunchKernelGGL(k_kv_tables, dim3(1), dim3(kScanThreads), 0, st, a);
    return hipGetLastError();
  }
  int32_t* ws = static_cast<int32_t*>(workspace);
  hipLaunchKernelGGL(k_kv_tables_scan, dim3(1), dim3(kScanThreads), 0, st, a, ws);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // one row per thread up to a few rounds of the chip; pages given back beyond that loop
  const int groups = min(max((a.T_max + 255) / 256, 64), 4096);
  hipLaunchKernelGGL(k_kv_tables_fill, dim3((unsigned)groups), dim3(256), 0, st, a, (const int32_t*)ws);
  return hipGetLastError();
}

hipError_t launch_kv_write(const void* k, int64_t k_stride, const void* v, int64_t v_stride, const int64_t* slots,
                           int64_t T, void* cache, int64_t num_pages, int64_t P, int64_t heads, int64_t D,
                           hipStream_t st) {
  const int lg = __builtin_ctzll((unsigned long long)P);
  const dim3 grid((unsigned)min((T + kWriteRows - 1) / kWriteRows, (int64_t)1 << 20), (unsigned)((heads * D + 127) / 128));
  hipLaunchKernelGGL(k_kv_write, grid, dim3(256), 0, st, static_cast<const uint16_t*>(k), k_stride,
                     static_cast<const uint16_t*>(v), v_stride, slots, T, static_cast<uint8_t*>(cache), num_pages * P, lg,
                     (int)heads, (int)D);
  return hipGetLastError();
}

hipError_t launch_kv_read(const void* cache, int64_t num_pages, int64_t P, int64_t heads, int64_t D,
                          const int64_t* slots, int64_t T, void* k, void* v, hipStream_t st) {
  const int64_t units = T * heads * (D / 8);
  const int lg = __builtin_ctzll((unsigned long long)P);
  hipLaunchKernelGGL(k_kv_read, dim3(groups_of(units)), dim3(256), 0, st,
                     static_cast<const uint8_t*>(cache), num_pages * P, lg, (int)heads, (int)D, slots, units,
                     static_cast<uint16_t*>(k), static_cast<uint16_t*>(v));
  return hipGetLastError();
}

}  // namespace mx
