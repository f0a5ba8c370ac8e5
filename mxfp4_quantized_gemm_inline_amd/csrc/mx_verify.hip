// mx_verify.hip - verification of drafted tokens against given probabilities and random numbers,
// and the next token by inverse transform.
#include "mx_device.h"
#include "mx_kv.h"

namespace mx {
namespace {

// Two launches. The first finds each request's first refused draft, every workgroup for itself (it
// is a handful of numbers), and sums a slice of the row that the next token is drawn from; the second
// finds the slice and then the token at which the running sum passes its number. Sums are FP64, in a
// fixed order.

constexpr int kThreads = 256;
constexpr int kMaxSlices = 256;

// Elements of a slice: a multiple of 1024.
__host__ __device__ inline int slice_of(int64_t B, int64_t V) {
  const int64_t want = min(max((int64_t)1024 / B, (int64_t)1), (int64_t)kMaxSlices);  // slices
  const int64_t each = (V + want - 1) / want;
  return (int)(max((each + 1023) / 1024, (int64_t)2) * 1024);
}

struct Slice {
  double rest, all;  // sums of max(p - q, 0) and of p
};

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

// What the token is drawn from, at element j: max(p - q, 0), p without the refused draft, or p.
struct Weights {
  const float *p, *q;
  int without;
  __device__ __forceinline__ double all(int j) const { return (double)positive(p[j]); }
  __device__ __forceinline__ double rest(int j) const {
    if (q) return fmax((double)positive(p[j]) - (double)positive(q[j]), 0.0);
    return j == without ? 0.0 : all(j);
  }
};
__device__ __forceinline__ Weights weights_of(const VerifyArgs& a, const Request& x, int acc) {
  const int64_t row = x.r0 + acc;
  const bool refused = acc < x.n - 1;
  return {a.p + row * a.p_stride, refused && a.q ? a.q + row * a.q_stride : nullptr, refused ? a.tokens[row + 1] : -1};
}

__global__ __launch_bounds__(kThreads) void k_verify_sums(VerifyArgs a, int slice, Slice* sums) {
  __shared__ Slice part[kThreads / 64];
  const int b = blockIdx.y, lane = threadIdx.x & 63;
  const Request x = request_of(a, b);
  if (x.n == 0) return;
  const Weights w = weights_of(a, x, accepted_of(a, x, lane));
  const int j0 = (int)blockIdx.x * slice, j1 = min(a.V, j0 + slice);
  Slice s = {0, 0};
  for (int j = j0 + (int)threadIdx.x; j < j1; j += kThreads) {
    s.rest += w.rest(j);
    s.all += w.all(j);
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    s.rest += __shfl_xor(s.rest, d);
    s.all += __shfl_xor(s.all, d);
  }
  if (lane == 0) part[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kThreads / 64; ++i) {
      s.rest += part[i].rest;
      s.all += part[i].all;
    }
    sums[(int64_t)b * gridDim.x + blockIdx.x] = s;
  }
}

__global__ __launch_bounds__(kThreads) void k_verify_draw(VerifyArgs a, int slice, int slices, const Slice* sums) {
  __shared__ double part[kThreads];
  __shared__ double base_of, goal_of;
  __shared__ int at[4];  // the slice (-1: nothing to draw from), the token, the last with a weight, whether the rest is drawn from
  const int b = blockIdx.x, lane = threadIdx.x & 63;
  if (b == a.B) {  // rows behind the last request
    const int end = min(max(a.cu_q[a.B], 0), a.T);
    for (int64_t t = end + (int64_t)threadIdx.x; t < a.T; t += kThreads) a.out[t] = -1;
    return;
  }
  const Request x = request_of(a, b);
  if (x.n == 0) {
    if (threadIdx.x == 0) {
      a.accepted[b] = 0;
      a.new_lens[b] = a.kv_lens[b];
    }
    return;
  }
  const int acc = accepted_of(a, x, lane);
  const Weights w = weights_of(a, x, acc);
  const Slice* mine = sums + (int64_t)b * slices;
  if (threadIdx.x == 0) {
    Slice total = {0, 0};
    for (int i = 0; i < slices; ++i) {
      total.rest += mine[i].rest;
      total.all += mine[i].all;
    }
    const bool rest = total.rest > 0;
    const double goal = fmin(fmax((double)a.sample[b], 0.0), 1.0) * (rest ? total.rest : total.all);
    double run = 0, base = 0;
    int found = -1;
    for (int i = 0; i < slices; ++i) {
      const double s = rest ? mine[i].rest : mine[i].all;
      if (s > 0) {
        found = i;
        base = run;
        if (run + s > goal) break;
      }
      run += s;
    }
    at[0] = found;
    at[1] = 0x7FFFFFFF;
    at[2] = -1;
    at[3] = rest;
    base_of = base;
    goal_of = goal;
  }
  __syncthreads();
  if (at[0] >= 0) {
    const bool rest = at[3];
    const double goal = goal_of;
    const int each = slice / kThreads, j0 = at[0] * slice + (int)threadIdx.x * each, j1 = min(a.V, j0 + each);
    double s = 0;
    for (int j = j0; j < j1; ++j) s += rest ? w.rest(j) : w.all(j);
    part[threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
      double run = base_of;
      for (int i = 0; i < kThreads; ++i) {
        const double y = part[i];
        part[i] = run;
        run += y;
      }
    }
    __syncthreads();
    double run = part[threadIdx.x];
    int hit = 0x7FFFFFFF, last = -1;
    for (int j = j0; j < j1; ++j) {
      const double y = rest ? w.rest(j) : w.all(j);
      run += y;
      if (y > 0) {
        last = j;
        if (run > goal && hit == 0x7FFFFFFF) hit = j;
      }
    }
    if (hit != 0x7FFFFFFF) atomicMin(&at[1], hit);
    if (last >= 0) atomicMax(&at[2], last);
    __syncthreads();
  }
  const int token = at[0] < 0 ? -1 : at[1] != 0x7FFFFFFF ? at[1] : at[2];
  if (threadIdx.x == 0) {
    a.accepted[b] = acc;
    a.new_lens[b] = a.kv_lens[b] - (x.n - 1 - acc);
  }
  for (int i = threadIdx.x; i < x.n; i += kThreads)
    a.out[x.r0 + i] = i < acc ? a.tokens[x.r0 + i + 1] : i == acc ? token : -1;
}

}  // namespace

size_t verify_workspace_bytes(int64_t B, int64_t V) {
  const int64_t slice = slice_of(B, V);
  return (size_t)(B * ((V + slice - 1) / slice)) * sizeof(Slice);
}

hipError_t launch_verify(const VerifyArgs& a, void* workspace, hipStream_t st) {
  Slice* sums = static_cast<Slice*>(workspace);
  int slice = 1024, slices = 0;
  if (a.B > 0) {
    slice = slice_of(a.B, a.V);
    slices = (a.V + slice - 1) / slice;
    hipLaunchKernelGGL(k_verify_sums, dim3((unsigned)slices, (unsigned)a.B), dim3(kThreads), 0, st, a, slice, sums);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(k_verify_draw, dim3((unsigned)a.B + 1), dim3(kThreads), 0, st, a, slice, slices, (const Slice*)sums);
  return hipGetLastError();
}

}  // namespace mx
