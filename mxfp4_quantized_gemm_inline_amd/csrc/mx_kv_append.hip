// mx_kv_append.hip - norms of each head, rotation by position, queries out and keys and values
// into the paged MXFP4 cache, in one pass.
#include "mx_device.h"
#include "mx_kv.h"

namespace mx {
namespace {

// A workgroup has kTile / D heads (one of 256 elements, one of 128, two of 64) of kRows rows at a
// time: a thread 8 elements of a row. What a thread's 8 elements are turned by depends on its row and
// place alone, so the angles are worked out once, each by one thread, and shared through LDS; the
// workgroup then goes through its heads with them in registers.
template <int D>
struct AppendTile {
  static constexpr int kWidth = D < 128 ? 128 : D;  // elements of a row at a time
  static constexpr int kLanes = kWidth / 8;         // threads of a row
  static constexpr int kRows = 256 / kLanes;        // 16, or 8 for heads of 256
};

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __builtin_bit_cast(float, w[i] << 16);
    x[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xFFFF0000u);
  }
}

// 1 / sqrt(mean of a head's squares + eps); in FP64, where no bf16 square leaves the range.
template <int D>
__device__ __forceinline__ double inverse_norm(const float (&x)[8], float eps) {
  double s = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fma((double)x[i], (double)x[i], s);
#pragma unroll
  for (int d = 1; d < D / 8; d <<= 1) s += __shfl_xor(s, d);
  return 1.0 / sqrt(s / D + (double)eps);
}

// F: float for queries, double for keys. x: 8 elements of a head from element d on, o: those that
// they are turned with (halves: those rot / 2 away; pairs: unused), with their weights.
template <typename F>
__device__ __forceinline__ void turn8(F (&y)[8], const float (&x)[8], const float (&o)[8], const float (&wx)[8],
                                      const float (&wo)[8], F r, const F (&cs)[8], const F (&sn)[8], int d, int rot,
                                      int pairs) {
  F a[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = (F)x[i] * r * (F)wx[i];
  if (d >= rot) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = a[i];
  } else if (pairs) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[2 * i] = a[2 * i] * cs[i] - a[2 * i + 1] * sn[i];
      y[2 * i + 1] = a[2 * i] * sn[i] + a[2 * i + 1] * cs[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const F b = (F)o[i] * r * (F)wo[i];
      y[i] = a[i] * cs[i] + b * sn[i];  // sn is negated for the first half
    }
  }
}

template <int D>
__global__ __launch_bounds__(256) void k_kv_append(KvAppendArgs a, int q_units, int units) {
  using Tile = AppendTile<D>;
  __shared__ double2 turn[Tile::kRows][D / 2];              // cos and sin of each row's angles
  __shared__ uint32_t v_words[Tile::kRows][Tile::kLanes + 1];
  __shared__ int64_t row_slot[Tile::kRows];                 // -1: writes nothing
  const int c = threadIdx.x % Tile::kLanes, r = threadIdx.x / Tile::kLanes;
  const int d = 8 * c % D;       // this thread's elements of its head
  for (int64_t t0 = (int64_t)blockIdx.x * Tile::kRows; t0 < a.T; t0 += (int64_t)gridDim.x * Tile::kRows) {
    const int64_t t = t0 + r;
    const int pos = t < a.T ? a.positions[t] : -1;
    const int half = a.rot / 2;
    for (int i = threadIdx.x; i < Tile::kRows * half; i += 256) {
      const int rr = i / half, f = i % half;
      const int p = t0 + rr < a.T ? a.positions[t0 + rr] : -1;
      double s, co;
      sincos((double)p * (double)a.inv_freq[f], &s, &co);
      turn[rr][f] = make_double2(co * (double)a.rope_scale, s * (double)a.rope_scale);
    }
    int64_t slot = -1;
    if (a.H > 0 && pos >= 0) {
      slot = a.slots[t];
      if (slot >= a.num_slots) slot = -1;
    }
    if (c == 0) row_slot[r] = slot;
    __syncthreads();
    // this thread's cos and sin, and the lane that has the elements that its own are turned with
    double cs[8], sn[8];
    int other = threadIdx.x & 63, od = d;
    const bool second = d >= half;
    if (d < a.rot && !a.pairs) {
      od = second ? d - half : d + half;
      other += (od - d) / 8;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      cs[i] = 1;
      sn[i] = 0;
      if (d < a.rot && (!a.pairs || i < 4)) {
        const double2 x = turn[r][a.pairs ? d / 2 + i : (second ? od : d) + i];
        cs[i] = x.x;
        sn[i] = a.pairs || second ? x.y : -x.y;
      }
    }
    for (int u = blockIdx.y; u < units; u += gridDim.y) {
      const bool is_q = u < q_units;
      const int e = (is_q ? u : u - q_units) * Tile::kWidth + 8 * c, h = e / D;
      const float* weight = is_q ? a.q_weight : a.k_weight;
      float wx[8], wo[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        wx[i] = weight ? weight[d + i] : 1.f;
        wo[i] = weight ? weight[od + i] : 1.f;
      }
      if (is_q) {
        const bool has = pos >= 0 && h < a.Hq;
        uint4 u4 = make_uint4(0, 0, 0, 0), o4;
        if (has) u4 = *reinterpret_cast<const uint4*>(a.q + t * a.q_stride + e);
        o4.x = __shfl(u4.x, other); o4.y = __shfl(u4.y, other); o4.z = __shfl(u4.z, other); o4.w = __shfl(u4.w, other);
        float x[8], o[8], y[8], fc[8], fs[8];
        unpack8(u4, x);
        unpack8(o4, o);
#pragma unroll
        for (int i = 0; i < 8; ++i) fc[i] = (float)cs[i], fs[i] = (float)sn[i];
        const float n = weight ? (float)inverse_norm<D>(x, a.eps) : 1.f;
        turn8<float>(y, x, o, wx, wo, n, fc, fs, d, a.rot, a.pairs);
        if (has) {
          const uint2 lo = pack4_bf16(y[0], y[1], y[2], y[3]), hi = pack4_bf16(y[4], y[5], y[6], y[7]);
          *reinterpret_cast<uint4*>(a.q_out + t * a.q_out_stride + e) = make_uint4(lo.x, lo.y, hi.x, hi.y);
        }
        continue;
      }
      const bool has = slot >= 0 && h < a.H;
      const KvLayout L = {1 << a.log2_page, D};
      const int tok = (int)(slot & (L.P - 1)), m = D / 32;
      uint8_t* blk = a.cache + ((slot >> a.log2_page) * a.H + h) * L.block_bytes();
      uint4 k4 = make_uint4(0, 0, 0, 0), v4 = k4, o4;
      if (has) {
        k4 = *reinterpret_cast<const uint4*>(a.k + t * a.k_stride + e);
        v4 = *reinterpret_cast<const uint4*>(a.v + t * a.v_stride + e);
      }
      o4.x = __shfl(k4.x, other); o4.y = __shfl(k4.y, other); o4.z = __shfl(k4.z, other); o4.w = __shfl(k4.w, other);
      float x[8], o[8];
      unpack8(k4, x);
      unpack8(o4, o);
      double y[8];
      turn8<double>(y, x, o, wx, wo, weight ? inverse_norm<D>(x, a.eps) : 1.0, cs, sn, d, a.rot, a.pairs);
      float f[8];
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        f[i] = (float)y[i];
        top = max(top, __builtin_bit_cast(uint32_t, f[i]) << 1 >> 24);
      }
      top |= top_field(v4) << 16;
      top = max_halves(top, (uint32_t)__shfl_xor((int)top, 1));
      top = max_halves(top, (uint32_t)__shfl_xor((int)top, 2));
      const uint32_t ek = top & 0xFFFFu, ev = top >> 16, sk = ek > 2u ? ek - 2u : 0u, sv = ev > 2u ? ev - 2u : 0u;
      v_words[r][c] = quant8(v4, sv);
      if (has) {
        const float sc = __builtin_bit_cast(float, sk ? sk << 23 : 0x00400000u);
        uint32_t kq = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0, f[0], f[1], sc, 0);
        kq = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(kq, f[2], f[3], sc, 1);
        kq = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(kq, f[4], f[5], sc, 2);
        kq = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(kq, f[6], f[7], sc, 3);
        *reinterpret_cast<uint32_t*>(blk + L.k_code(tok, d)) = kq;
        if ((c & 3) == 0) {
          blk[L.k_scale(tok, d)] = (uint8_t)sk;
          blk[L.v_scale(tok, d)] = (uint8_t)sv;
        }
      }
      __syncthreads();
      if (has) {  // V's codes: the first of four tokens writes for all
        const int at = (int)(slot & 3), first = r - at;
        bool four = first >= 0 && first + 3 < Tile::kRows;
        if (four)
#pragma unroll
          for (int i = 0; i < 4; ++i) four = four && row_slot[first + i] == slot - at + i;
        if (!four) {
          const uint32_t w = v_words[r][c];
#pragma unroll
          for (int b = 0; b < 4; ++b) blk[L.v_code(tok, d + 2 * b)] = (uint8_t)(w >> (8 * b));
        } else if (at == 0) {
          const uint32_t w0 = v_words[r][c], w1 = v_words[r + 1][c], w2 = v_words[r + 2][c], w3 = v_words[r + 3][c];
          const uint32_t s = __builtin_amdgcn_perm(w1, w0, 0x05010400), b = __builtin_amdgcn_perm(w3, w2, 0x05010400);
          const uint32_t p = __builtin_amdgcn_perm(w1, w0, 0x07030602), q = __builtin_amdgcn_perm(w3, w2, 0x07030602);
          uint32_t* dst = reinterpret_cast<uint32_t*>(blk + L.v_code(tok, d));
          dst[0] = __builtin_amdgcn_perm(b, s, 0x05040100);
          dst[m] = __builtin_amdgcn_perm(b, s, 0x07060302);
          dst[2 * m] = __builtin_amdgcn_perm(q, p, 0x05040100);
          dst[3 * m] = __builtin_amdgcn_perm(q, p, 0x07060302);
        }
      }
      __syncthreads();  // before the next heads take their place
    }
    __syncthreads();  // before the next rows' angles take their place
  }
}

template <int D>
hipError_t launch(const KvAppendArgs& a, hipStream_t st) {
  using Tile = AppendTile<D>;
  const int per = Tile::kWidth / D;
  const int q_units = (a.Hq + per - 1) / per, units = q_units + (a.H + per - 1) / per;
  const int64_t rows = ((int64_t)a.T + Tile::kRows - 1) / Tile::kRows;
  // a workgroup per unit until the chip is full, then more units a workgroup
  const int split = (int)max((int64_t)1, min((int64_t)units, 2048 / rows));
  const unsigned groups = (unsigned)min(rows, (int64_t)1 << 20);  // past them they loop (a launch holds fewer than 2^32 threads)
  hipLaunchKernelGGL(k_kv_append<D>, dim3(groups, (unsigned)split), dim3(256), 0, st, a, q_units, units);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t st) {
  switch (a.D) {
    case 64: return launch<64>(a, st);
    case 128: return launch<128>(a, st);
    default: return launch<256>(a, st);
  }
}

}  // namespace mx
