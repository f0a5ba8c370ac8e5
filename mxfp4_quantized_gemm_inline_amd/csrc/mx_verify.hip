// mx_verify.hip - verification of drafted tokens against given probabilities and random numbers,
// and the next token by inverse transform.
#include "mx_device.h"
#include "mx_kv.h"

namespace mx {
namespace {

// Two launches. The first finds each request's first refused draft, every workgroup for itself (it is a
// handful of numbers), and sums the row that the next token is drawn from, a chunk a wave; the second
// finds the chunk and then the token at which the running sum passes its number. Sums are FP64, in a
// fixed order.
// Bound: HBM where requests are many (64 rows of 131072 of p, and of q for the 25 to 29 of them where a draft
// is refused, 48 MB: 11.4 us, 4.2 TB/s, + 4.6; floor 9.7), else latency: one request 3.9 + 3.8 us, chains of
// four and five loads. 150 rows of 50021 of p alone, 30 MB: 8.8 + 4.6 us, of which the way to the row (cu_q,
// tokens, p) is 1.0; rows that begin at whole lines take as long. kStep 1024 / 2048 / 512: 64 x 131072
// 16.7 / 18.9 / 17.6 us, one request 7.6 / 9.3 / 8.2, 500 x 5000 12.3 / 15.1 / 11.2.

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kChunks = kThreads;  // of a row, at most: one a thread of the second launch
constexpr int kStep = 1024;        // elements that a wave, or the second launch's workgroup, takes at a time
constexpr int kAhead = kStep / 64, kEach = kStep / kThreads;

// Elements of a chunk: a multiple of kStep. A row's first chunk begins up to 63 elements before it, where
// a wave's loads are of whole lines also in rows of an odd length.
inline int chunk_of(int64_t V) { return (int)(((V + 63 + kChunks - 1) / kChunks + kStep - 1) / kStep * kStep); }
inline int chunks_of(int64_t V) { return (int)((V + 63 + chunk_of(V) - 1) / chunk_of(V)); }

// The workspace: accepted drafts [B], padded to 16 bytes, then the sums of chunks [B][chunks].
inline int64_t sums_at(int64_t B) { return (B * 4 + 15) / 16 * 16; }

__device__ __forceinline__ float positive(float x) { return fmaxf(x, 0.f); }  // NaN becomes 0

struct Request {
  int r0, n;  // its rows
};
__device__ __forceinline__ Request request_of(const VerifyArgs& a, int b) {
  const int lo = min(max(a.cu_q[b], 0), a.T), hi = min(max(a.cu_q[b + 1], lo), a.T);
  return {lo, hi - lo};
}

// Accepted drafts of a request (by one wave; the same in every lane).
__device__ __forceinline__ int accepted_of(const VerifyArgs& a, const Request& x, int lane) {
  for (int i0 = 0; i0 < x.n - 1; i0 += 64) {
    const int i = i0 + lane;
    bool refused = false;
    if (i < x.n - 1) {
      const int64_t row = x.r0 + i;
      const int tok = a.tokens[row + 1];
      refused = true;
      if (tok >= 0 && tok < a.V) {
        const float p = positive(a.p[row * a.p_stride + tok]), q = a.q ? positive(a.q[row * a.q_stride + tok]) : 1.f;
        refused = !((double)a.accept[row] * (double)q < (double)p);
      }
    }
    const uint64_t at = __ballot(refused);
    if (at) return i0 + (int)__builtin_ctzll(at);
  }
  return x.n - 1;
}

// What the token is drawn from: max(p - q, 0), p without the refused draft, or p.
struct Weights {
  const float *p, *q;
  int without, V;
  int before;  // elements from the last whole line's begin to the row's
  __device__ __forceinline__ double weigh(float x, float y, int j) const {
    if (j < 0 || j >= V || j == without) return 0.0;
    return fmax((double)positive(x) - (double)positive(y), 0.0);
  }
};
__device__ __forceinline__ Weights weights_of(const VerifyArgs& a, const Request& x, int acc, bool whole) {
  const int64_t row = x.r0 + acc;
  const bool refused = acc < x.n - 1 && !whole;
  const float* p = a.p + row * a.p_stride;
  return {p, refused && a.q ? a.q + row * a.q_stride : nullptr, refused && !a.q ? a.tokens[row + 1] : -1, a.V,
          (int)(reinterpret_cast<uintptr_t>(p) >> 2 & 63)};
}

// The sum over the threads before this one, and over all.
__device__ __forceinline__ double group_before(double x, double* part, double& all) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  double upto = x;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double y = __shfl_up(upto, d);
    if (lane >= d) upto += y;
  }
  if (lane == 63) part[w] = upto;
  double before = __shfl_up(upto, 1);
  if (lane == 0) before = 0;
  __syncthreads();
  double base = 0;
  all = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    if (i < w) base += part[i];
    all += part[i];
  }
  return base + before;
}

constexpr int kNone = 0x7FFFFFFF;
struct Found {
  int first, last;  // of each wave: the first past the goal (kNone: none), the last with a weight (-1)
};
// Over the workgroup, of numbers that grow with the thread. found: one a wave.
__device__ __forceinline__ Found group_found(int hit, int last, Found* found) {
  const int w = threadIdx.x >> 6;
  const uint64_t hits = __ballot(hit != kNone), lasts = __ballot(last >= 0);
  const int h = hits ? __builtin_amdgcn_readlane(hit, (int)__builtin_ctzll(hits)) : kNone;
  const int l = lasts ? __builtin_amdgcn_readlane(last, 63 - (int)__builtin_clzll(lasts)) : -1;
  if ((threadIdx.x & 63) == 0) found[w] = {h, l};
  __syncthreads();
  Found f = found[0];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) {
    f.first = min(f.first, found[i].first);
    f.last = max(f.last, found[i].last);
  }
  return f;
}

// The sum of a chunk, by one wave; the same in every lane.
__device__ __forceinline__ double chunk_sum(const Weights& w, int c, int chunk) {
  const int lane = threadIdx.x & 63, j0 = c * chunk - w.before;
  double s = 0;
  for (int b0 = j0; b0 < min(w.V, j0 + chunk); b0 += kStep) {
    float p[kAhead], q[kAhead];
    if (b0 >= 0 && b0 + kStep <= w.V) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) p[i] = w.p[b0 + 64 * i + lane];
      if (w.q) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) q[i] = w.q[b0 + 64 * i + lane];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) s += fmax((double)positive(p[i]) - (double)positive(q[i]), 0.0);
      } else {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) s += b0 + 64 * i + lane == w.without ? 0.0 : (double)positive(p[i]);
      }
    } else {
      int at[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) at[i] = min(max(b0 + 64 * i + lane, 0), w.V - 1);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) p[i] = w.p[at[i]];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) q[i] = 0.f;
      if (w.q) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) q[i] = w.q[at[i]];
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) s += w.weigh(p[i], q[i], b0 + 64 * i + lane);
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d);
  return s;
}

__global__ __launch_bounds__(kThreads) void k_verify_sums(VerifyArgs a, int chunk, int chunks, int32_t* accepted, double* sums) {
  const int b = blockIdx.y, lane = threadIdx.x & 63;
  const Request x = request_of(a, b);
  if (x.n == 0) return;
  const int acc = accepted_of(a, x, lane);
  const int c = (int)blockIdx.x * kWaves + (int)(threadIdx.x >> 6);
  if (c >= chunks) return;
  const double s = chunk_sum(weights_of(a, x, acc, false), c, chunk);
  if (lane == 0) {
    sums[(int64_t)b * chunks + c] = s;
    if (c == 0) accepted[b] = acc;
  }
}

__global__ __launch_bounds__(kThreads) void k_verify_draw(VerifyArgs a, int chunk, int chunks, const int32_t* accepted,
                                                          const double* sums) {
  __shared__ double part[kWaves], part2[kWaves], run_of;
  __shared__ Found found[2][kWaves];
  __shared__ double again[kChunks];
  const int b = blockIdx.x, i = threadIdx.x;
  if (b == a.B) {  // rows behind the last request
    const int end = min(max(a.cu_q[a.B], 0), a.T);
    for (int64_t t = end + (int64_t)i; t < a.T; t += kThreads) a.out[t] = -1;
    return;
  }
  const Request x = request_of(a, b);
  const int kv = a.kv_lens[b];
  if (x.n == 0) {
    if (i == 0) {
      a.accepted[b] = 0;
      a.new_lens[b] = kv;
    }
    return;
  }
  const int acc = accepted[b];
  const float u = a.sample[b];
  double mine = i < chunks ? sums[(int64_t)b * chunks + i] : 0.0, total;
  double before = group_before(mine, part, total);
  const bool whole = !(total > 0);  // nothing is left of p: p itself
  const Weights w = weights_of(a, x, acc, whole);
  if (whole && acc < x.n - 1) {
    for (int c = i / 64; c < chunks; c += kWaves) {
      const double y = chunk_sum(w, c, chunk);
      if (i % 64 == 0) again[c] = y;
    }
    __syncthreads();
    mine = i < chunks ? again[i] : 0.0;
    before = group_before(mine, part, total);
  }
  const double goal = fmin(fmax((double)u, 0.0), 1.0) * total;
  Found f = group_found(mine > 0 && before + mine > goal ? i : kNone, mine > 0 ? i : -1, found[0]);
  int token = -1;
  const int at = f.first != kNone ? f.first : f.last;  // the chunk; -1: no weight anywhere
  if (at >= 0) {
    if (i == at) run_of = before;
    __syncthreads();
    const int start = at * chunk - w.before, end = min(a.V, start + chunk);
    for (int b0 = start; b0 < end; b0 += kStep) {
      const int j = b0 + i * kEach;
      double y[kEach], s = 0, block;
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        const int at = min(max(j + k, 0), a.V - 1);
        y[k] = w.weigh(w.p[at], w.q ? w.q[at] : 0.f, j + k);
      }
#pragma unroll
      for (int k = 0; k < kEach; ++k) s += y[k];
      const double run = run_of;
      double upto = run + group_before(s, part2, block);
      int hit = kNone, last = -1;
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        upto += y[k];
        if (y[k] > 0) {
          last = j + k;
          if (upto > goal && hit == kNone) hit = last;
        }
      }
      f = group_found(hit, last, found[1]);
      if (f.last >= 0) token = f.last;
      if (f.first != kNone) {
        token = f.first;
        break;
      }
      if (i == 0) run_of = run + block;  // every thread has read it
      __syncthreads();
    }
  }
  if (i == 0) {
    a.accepted[b] = acc;
    a.new_lens[b] = kv - (x.n - 1 - acc);
  }
  for (int r = i; r < x.n; r += kThreads) a.out[x.r0 + r] = r < acc ? a.tokens[x.r0 + r + 1] : r == acc ? token : -1;
}

}  // namespace

size_t verify_workspace_bytes(int64_t B, int64_t V) { return (size_t)(sums_at(B) + B * chunks_of(V) * 8); }

hipError_t launch_verify(const VerifyArgs& a, void* workspace, hipStream_t st) {
  int32_t* accepted = static_cast<int32_t*>(workspace);
  double* sums = reinterpret_cast<double*>(static_cast<uint8_t*>(workspace) + sums_at(a.B));
  const int chunk = chunk_of(a.V), chunks = chunks_of(a.V);
  if (a.B > 0) {
    const dim3 grid((unsigned)((chunks + kWaves - 1) / kWaves), (unsigned)a.B);
    hipLaunchKernelGGL(k_verify_sums, grid, dim3(kThreads), 0, st, a, chunk, chunks, accepted, sums);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(k_verify_draw, dim3((unsigned)a.B + 1), dim3(kThreads), 0, st, a, chunk, chunks, (const int32_t*)accepted,
                     (const double*)sums);
  return hipGetLastError();
}

}  // namespace mx
