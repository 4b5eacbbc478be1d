// Head norms and rotary positions, as the kernels that read or write queries
// and keys share them.
//
// A half-warp holds one head: 8 of its 128 elements a lane, in two chunks of
// four.  With the rotated part's pairs (i, i + rot/2), lane l < rot/8 holds
// elements 4l.. and rot/2 + 4l.., with neighbours (2i, 2i + 1) elements 8l..:
// either way a lane has its four pairs whole and nothing is exchanged.  Lanes
// from rot/8 on hold the elements 8l.. that are not rotated (angle zero).
//
// The angle of pair i at position p is p f_i.  Frequencies come as turns a
// token times 2^64, so the low 64 bits of p F are the angle in turns modulo
// one, exact for every 32-bit position: nothing is lost at far ones, where
// a product in fp32 is off by 2^-24 of hundreds of thousands of radians.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>

#include "gdn_internal.cuh"
#include "sm103_ptx.cuh"

namespace gdn {

constexpr int kRopeD = 128;   // elements of a head
constexpr int kNormNone = 0, kNormRms = 1, kNormUnit = 2;

struct RopeArgs {
  const uint64_t* turns;  // [rot / 2]
  int rot, interleaved;
  float magnitude;
  int norm;
  float eps, inv_n;       // 1 / sqrt(inv_n sum x^2 + eps)
};

// Where a packed token stands: given, counted from its sequence's start, or
// from its row's.
struct PosArgs {
  const int32_t* positions;  // [T] or null
  const int32_t* cu;         // [n_seqs + 1] or null
  int n_seqs, T, n_each;
};

// The last sequence that begins at t or before, within [0, n).
__device__ __forceinline__ int seq_of(const int32_t* cu, int n, int t) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}
// False for a token outside every sequence.
__device__ __forceinline__ bool token_position(const PosArgs& a, int t, int& pos) {
  if (a.positions) {
    pos = a.positions[t];
  } else if (a.cu) {
    const int seq = seq_of(a.cu, a.n_seqs, t), begin = a.cu[seq];
    pos = (int)((unsigned)t - (unsigned)begin);
    return t >= begin && t < a.cu[seq + 1];
  } else {
    pos = t % a.n_each;
  }
  return true;
}

struct RopeLane {
  int o0, o1;    // first elements of the lane's chunks
  bool turned;
};
__device__ __forceinline__ RopeLane rope_lane(const RopeArgs& r, int l) {
  RopeLane p;
  p.turned = l < (r.rot >> 3);
  const bool halves = p.turned && !r.interleaved;
  p.o0 = halves ? 4 * l : 8 * l;
  p.o1 = halves ? (r.rot >> 1) + 4 * l : 8 * l + 4;
  return p;
}

struct RopeFreq {
  uint64_t f[4];
};
__device__ __forceinline__ RopeFreq rope_freq(const RopeArgs& r, const RopeLane& p, int l) {
  RopeFreq q = {{0, 0, 0, 0}};
  if (p.turned) {
    const ulonglong2* t = reinterpret_cast<const ulonglong2*>(r.turns + 4 * l);
    const ulonglong2 a = __ldg(t), b = __ldg(t + 1);
    q.f[0] = a.x; q.f[1] = a.y; q.f[2] = b.x; q.f[3] = b.y;
  }
  return q;
}

// magnitude times cos and sin of the lane's pairs at position p.  The phase
// enters as its upper 32 bits, a signed fraction of half a turn, whose
// conversion to fp32 is off by 2^-25 of a half turn at most.
__device__ __forceinline__ void rope_angles(const RopeArgs& r, const RopeLane& p, const RopeFreq& q, int pos, float (&c)[4],
                                            float (&s)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    c[e] = 1.f;
    s[e] = 0.f;
  }
  if (!p.turned) return;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint64_t phase = (uint64_t)(int64_t)pos * q.f[e];
    sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &s[e], &c[e]);
    c[e] *= r.magnitude;
    s[e] *= r.magnitude;
  }
}

// Rotates the lane's pairs; sign -1: by the transposed rotation.
template <bool kInterleaved>
__device__ __forceinline__ void rope_turn(float (&x)[8], const float (&c)[4], const float (&s)[4], float sign = 1.f) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float& a = x[kInterleaved ? 2 * e : e];
    float& b = x[kInterleaved ? 2 * e + 1 : e + 4];
    const float se = sign * s[e];
    const float ya = a * c[e] - b * se, yb = b * c[e] + a * se;
    a = ya;
    b = yb;
  }
}

// ---- a lane's 8 elements in memory ----
struct Row8f {
  float4 a, b;
};
struct Row8h {
  uint2 a, b;
};
template <typename T>
struct RowOf;
template <>
struct RowOf<float> {
  using type = Row8f;
};
template <>
struct RowOf<__nv_bfloat16> {
  using type = Row8h;
};
__device__ __forceinline__ Row8f load_row(const float* p, const RopeLane& l) {
  return {*reinterpret_cast<const float4*>(p + l.o0), *reinterpret_cast<const float4*>(p + l.o1)};
}
__device__ __forceinline__ Row8h load_row(const __nv_bfloat16* p, const RopeLane& l) {
  return {*reinterpret_cast<const uint2*>(p + l.o0), *reinterpret_cast<const uint2*>(p + l.o1)};
}
__device__ __forceinline__ void unpack_row(const Row8f& r, float (&x)[8]) {
  x[0] = r.a.x; x[1] = r.a.y; x[2] = r.a.z; x[3] = r.a.w;
  x[4] = r.b.x; x[5] = r.b.y; x[6] = r.b.z; x[7] = r.b.w;
}
__device__ __forceinline__ void unpack_row(const Row8h& r, float (&x)[8]) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.b.x, r.b.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store_row(float* p, const RopeLane& l, const float (&x)[8]) {
  *reinterpret_cast<float4*>(p + l.o0) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(p + l.o1) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void store_row(__nv_bfloat16* p, const RopeLane& l, const float (&x)[8]) {
  *reinterpret_cast<uint2*>(p + l.o0) = make_uint2(pack2(x[0], x[1]), pack2(x[2], x[3]));
  *reinterpret_cast<uint2*>(p + l.o1) = make_uint2(pack2(x[4], x[5]), pack2(x[6], x[7]));
}

// ---- the norm ----
// Sum over the calling half-warp; `mask` is its lanes.
__device__ __forceinline__ unsigned half_mask() { return 0xffffu << (threadIdx.x & 16); }
__device__ __forceinline__ float half_sum(float v, unsigned mask) {
#pragma unroll
  for (int d = 8; d; d >>= 1) v += __shfl_xor_sync(mask, v, d);
  return v;
}
__device__ __forceinline__ float sum_squares(const float (&x)[8]) {
  return ((x[0] * x[0] + x[1] * x[1]) + (x[2] * x[2] + x[3] * x[3])) +
         ((x[4] * x[4] + x[5] * x[5]) + (x[6] * x[6] + x[7] * x[7]));
}
// 1 / sqrt(inv_n ss + eps), ss the head's sum of squares.  Past fp32's range
// (elements of 2^60 and more) x is scaled by `unit` = 2^-68, beside which eps
// is nothing, and the result belongs to the scaled x.
__device__ __forceinline__ float head_scale(float ss, float (&x)[8], float inv_n, float eps, unsigned mask, float& unit) {
  unit = 1.f;
  if (ss <= 3e38f) return rsqrtf(fmaf(ss, inv_n, eps));
  unit = 0x1p-68f;
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] *= unit;
  return rsqrtf(half_sum(sum_squares(x), mask) * inv_n);
}

__device__ __forceinline__ void load_weight(const float* w, const RopeLane& l, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(w + l.o0)), b = __ldg(reinterpret_cast<const float4*>(w + l.o1));
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

constexpr int kRopeBatch = 4;  // heads whose loads are in flight together

// n heads of a token: in -> out.
template <typename T, bool kInterleaved>
__device__ __forceinline__ void turn_heads(const RopeArgs& r, const RopeLane& l, const float (&c)[4], const float (&s)[4],
                                           const T* in, T* out, int n, const float* weight, unsigned mask) {
  if (n <= 0) return;
  float w[8];
  if (weight) load_weight(weight, l, w);
  for (int h0 = 0; h0 < n; h0 += kRopeBatch) {
    typename RowOf<T>::type raw[kRopeBatch];
#pragma unroll
    for (int i = 0; i < kRopeBatch; ++i)
      if (h0 + i < n) raw[i] = load_row(in + (h0 + i) * kRopeD, l);
#pragma unroll
    for (int i = 0; i < kRopeBatch; ++i) {
      if (h0 + i >= n) break;
      float x[8];
      unpack_row(raw[i], x);
      if (r.norm != kNormNone) {
        float unit;
        const float f = head_scale(half_sum(sum_squares(x), mask), x, r.inv_n, r.eps, mask, unit);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= f;
        if (weight) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] *= w[e];
        }
      }
      rope_turn<kInterleaved>(x, c, s);
      store_row(out + (h0 + i) * kRopeD, l, x);
    }
  }
}

// Arguments of gdn_qk_rope and its gradient.
struct QkRopeArgs {
  RopeArgs r;
  PosArgs pos;
  const void* q;
  const void* k;
  const float* q_weight;   // [128] or null
  const float* k_weight;
  void* q_out;             // backward: the gradient of q_out, read
  void* k_out;
  int64_t q_stride, k_stride, q_out_stride, k_out_stride;
  int h_q, h_k;
  int splits;              // half-warps that share a token's heads
  // backward
  void* dq;
  void* dk;
  int64_t dq_stride, dk_stride;
  float* part;             // [CTAs, 2, 128] sums of the weights' gradients, or null
  float* dq_weight;
  float* dk_weight;
};

cudaError_t launch_qk_rope(const QkRopeArgs& a, bool f32, cudaStream_t st);
cudaError_t launch_qk_rope_bwd(const QkRopeArgs& a, bool f32, int ctas, cudaStream_t st);
cudaError_t launch_qk_rope_weights(const QkRopeArgs& a, int ctas, cudaStream_t st);

}  // namespace gdn
