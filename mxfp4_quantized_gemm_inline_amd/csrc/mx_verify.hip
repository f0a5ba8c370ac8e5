// mx_verify.hip - verification of drafted tokens against given probabilities and random numbers,
// and the next token by inverse transform.
#include "mx_device.h"
#include "mx_kv.h"

namespace mx {
namespace {

// Two launches. The first finds each request's first refused draft, every workgroup for itself (it is a
// handful of numbers), and sums a slice of the row that the next token is drawn from; the second finds
// the slice and then the token at which the running sum passes its number. Sums are FP64, in a fixed
// order.

constexpr int kThreads = 256;
constexpr int kAhead = 8;  // elements that a thread loads at once
constexpr int kStep = kThreads * kAhead;
constexpr int kMaxSlices = kThreads;  // one a thread of the second launch
constexpr int kGroups = 1024;         // workgroups of the first, at least, where the slices are long enough
constexpr int kBlock = 4096;          // elements that the second takes at a time: a slice, as a rule
constexpr int kEach = kBlock / kThreads;

// Elements of a slice: a multiple of kStep.
inline int slice_of(int64_t B, int64_t V) {
  const int64_t want = min(max(kGroups / B, (V + kBlock - 1) / kBlock), (int64_t)kMaxSlices);
  const int64_t each = (V + want - 1) / want;
  return (int)((each + kStep - 1) / kStep * kStep);
}
inline int slices_of(int64_t B, int64_t V) { return (int)((V + slice_of(B, V) - 1) / slice_of(B, V)); }

// The workspace: accepted drafts [B], padded to 16 bytes, then the sums of slices [B][slices].
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
  int without;
  __device__ __forceinline__ double at(int j) const {
    const double x = (double)positive(p[j]);
    if (q) return fmax(x - (double)positive(q[j]), 0.0);
    return j == without ? 0.0 : x;
  }
};
__device__ __forceinline__ Weights weights_of(const VerifyArgs& a, const Request& x, int acc, bool whole) {
  const int64_t row = x.r0 + acc;
  const bool refused = acc < x.n - 1 && !whole;
  return {a.p + row * a.p_stride, refused && a.q ? a.q + row * a.q_stride : nullptr, refused ? a.tokens[row + 1] : -1};
}

// The sum over the workgroup; part: a number a wave.
__device__ __forceinline__ double group_sum(double s, double* part) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
  __syncthreads();
  s = part[0];
#pragma unroll
  for (int i = 1; i < kThreads / 64; ++i) s += part[i];
  return s;
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
  for (int i = 0; i < kThreads / 64; ++i) {
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
  for (int i = 1; i < kThreads / 64; ++i) {
    f.first = min(f.first, found[i].first);
    f.last = max(f.last, found[i].last);
  }
  return f;
}

__device__ __forceinline__ double slice_sum(const Weights& w, int j0, int j1) {
  double s = 0;
  for (int j = j0 + (int)threadIdx.x; j < j1; j += kStep) {
    if (j - (int)threadIdx.x + kStep <= j1) {
      float p[kAhead], q[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) p[i] = w.p[j + kThreads * i];
      if (w.q) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) q[i] = w.q[j + kThreads * i];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) s += fmax((double)positive(p[i]) - (double)positive(q[i]), 0.0);
      } else {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) s += j + kThreads * i == w.without ? 0.0 : (double)positive(p[i]);
      }
    } else {
      for (int i = j; i < j1; i += kThreads) s += w.at(i);
    }
  }
  return s;
}

__global__ __launch_bounds__(kThreads) void k_verify_sums(VerifyArgs a, int slice, int32_t* accepted, double* sums) {
  __shared__ double part[kThreads / 64];
  const int b = blockIdx.y;
  const Request x = request_of(a, b);
  if (x.n == 0) return;
  const int acc = accepted_of(a, x, threadIdx.x & 63);
  const int j0 = (int)blockIdx.x * slice, j1 = min(a.V, j0 + slice);
  const double s = group_sum(slice_sum(weights_of(a, x, acc, false), j0, j1), part);
  if (threadIdx.x == 0) {
    sums[(int64_t)b * gridDim.x + blockIdx.x] = s;
    if (blockIdx.x == 0) accepted[b] = acc;
  }
}

__global__ __launch_bounds__(kThreads) void k_verify_draw(VerifyArgs a, int slice, int slices, const int32_t* accepted,
                                                          const double* sums) {
  __shared__ double part[kThreads / 64], part2[kThreads / 64], run_of;
  __shared__ Found found[2][kThreads / 64];
  __shared__ double row[kBlock + kThreads];  // 17 places for 16: threads side by side use different banks
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
  double mine = i < slices ? sums[(int64_t)b * slices + i] : 0.0, total;
  double before = group_before(mine, part, total);
  const bool whole = !(total > 0);  // nothing is left of p: p itself
  const Weights w = weights_of(a, x, acc, whole);
  if (whole && acc < x.n - 1) {
    for (int s = 0; s < slices; ++s) {
      __syncthreads();
      const double y = group_sum(slice_sum(w, s * slice, min(a.V, (s + 1) * slice)), part);
      if (i == s) mine = y;
    }
    __syncthreads();
    before = group_before(mine, part, total);
  }
  const double goal = fmin(fmax((double)u, 0.0), 1.0) * total;
  Found f = group_found(mine > 0 && before + mine > goal ? i : kNone, mine > 0 ? i : -1, found[0]);
  int token = -1;
  const int at = f.first != kNone ? f.first : f.last;  // the slice; -1: no weight anywhere
  if (at >= 0) {
    if (i == at) run_of = before;
    const int end = min(a.V, (at + 1) * slice);
    for (int b0 = at * slice; b0 < end; b0 += kBlock) {
      // loaded side by side, taken 16 to a thread
      double y[kEach];
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        const int j = b0 + k * kThreads + i;
        y[k] = j < end ? w.at(j) : 0.0;
      }
#pragma unroll
      for (int k = 0; k < kEach; ++k) row[k * kThreads + i + (k * kThreads + i) / kEach] = y[k];
      __syncthreads();
      double s = 0, block;
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        y[k] = row[i * (kEach + 1) + k];
        s += y[k];
      }
      const double run = run_of;
      double upto = run + group_before(s, part2, block);
      int hit = kNone, last = -1;
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        upto += y[k];
        if (y[k] > 0) {
          last = b0 + i * kEach + k;
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

size_t verify_workspace_bytes(int64_t B, int64_t V) { return (size_t)(sums_at(B) + B * slices_of(B, V) * 8); }

hipError_t launch_verify(const VerifyArgs& a, void* workspace, hipStream_t st) {
  int32_t* accepted = static_cast<int32_t*>(workspace);
  double* sums = reinterpret_cast<double*>(static_cast<uint8_t*>(workspace) + sums_at(a.B));
  int slice = kStep, slices = 0;
  if (a.B > 0) {
    slice = slice_of(a.B, a.V);
    slices = slices_of(a.B, a.V);
    hipLaunchKernelGGL(k_verify_sums, dim3((unsigned)slices, (unsigned)a.B), dim3(kThreads), 0, st, a, slice, accepted, sums);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(k_verify_draw, dim3((unsigned)a.B + 1), dim3(kThreads), 0, st, a, slice, slices, (const int32_t*)accepted,
                     (const double*)sums);
  return hipGetLastError();
}

}  // namespace mx
