// Queries and keys of every head, normalised and rotated in one pass, and the
// gradients of that.
//
// Forward, per token and head (x: 128 elements, R: the rotation at the
// token's position, m: magnitude): r = 1 / sqrt(inv_n sum x^2 + eps),
// y = m R (x r w).  Backward, from dy: du = m R^T dy, n = x r,
//   dw = sum over tokens and heads of du n,  dn = du w,
//   dx = r (dn - n inv_n sum(dn n)).
// (From d(r) = -r^3 inv_n sum x dx, with n = x r.)
//
// Each element is read and written once and both are bound by that.  A
// half-warp takes a token's heads, or a part of them, one after another with
// the cosines in registers, so they are computed once a token.
#include "gdn_rope.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kTasks = kThreads / 16;   // half-warps of a CTA

template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) rope_kernel(const QkRopeArgs a) {
  const int lane = threadIdx.x & 15;
  const unsigned mask = half_mask();
  const int64_t task = (int64_t)blockIdx.x * kTasks + (threadIdx.x >> 4);
  const int t = (int)(task / a.splits), part = (int)(task % a.splits);
  grid_dependency_wait();
  grid_launch_dependents();
  if (t >= a.pos.T) return;
  const RopeLane l = rope_lane(a.r, lane);
  int pos;
  if (!token_position(a.pos, t, pos)) return;
  float c[4], s[4];
  rope_angles(a.r, l, rope_freq(a.r, l, lane), pos, c, s);
  const int heads = a.h_q + a.h_k;
  const int h0 = (int)((int64_t)part * heads / a.splits), h1 = (int)((int64_t)(part + 1) * heads / a.splits);
  const int q0 = min(h0, a.h_q), q1 = min(h1, a.h_q), k0 = max(h0 - a.h_q, 0), k1 = max(h1 - a.h_q, 0);
  turn_heads<T, kInterleaved>(a.r, l, c, s, static_cast<const T*>(a.q) + t * a.q_stride + q0 * kRopeD,
                              static_cast<T*>(a.q_out) + t * a.q_out_stride + q0 * kRopeD, q1 - q0, a.q_weight, mask);
  turn_heads<T, kInterleaved>(a.r, l, c, s, static_cast<const T*>(a.k) + t * a.k_stride + k0 * kRopeD,
                              static_cast<T*>(a.k_out) + t * a.k_out_stride + k0 * kRopeD, k1 - k0, a.k_weight, mask);
}

// The gradients of n heads of a token; dw takes their share of the weight's.
template <typename T, bool kInterleaved>
__device__ __forceinline__ void turn_heads_bwd(const RopeArgs& r, const RopeLane& l, const float (&c)[4], const float (&s)[4],
                                               const T* in, const T* dy, T* dx, int n, const float* weight, float (&dw)[8],
                                               unsigned mask) {
  if (n <= 0) return;
  float w[8];
  if (weight) load_weight(weight, l, w);
  constexpr int kHeads = 2;
  for (int h0 = 0; h0 < n; h0 += kHeads) {
    typename RowOf<T>::type rx[kHeads], rg[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
      if (h0 + i < n) {
        rg[i] = load_row(dy + (h0 + i) * kRopeD, l);
        if (r.norm != kNormNone) rx[i] = load_row(in + (h0 + i) * kRopeD, l);
      }
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      if (h0 + i >= n) break;
      float g[8];
      unpack_row(rg[i], g);
      rope_turn<kInterleaved>(g, c, s, -1.f);
      if (r.norm != kNormNone) {
        float x[8];
        unpack_row(rx[i], x);
        float unit, dot = 0.f;
        const float f = head_scale(half_sum(sum_squares(x), mask), x, r.inv_n, r.eps, mask, unit);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] *= f;
          if (weight) {
            dw[e] = fmaf(g[e], x[e], dw[e]);
            g[e] *= w[e];
          }
          dot = fmaf(g[e], x[e], dot);
        }
        dot = half_sum(dot, mask) * r.inv_n;
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = f * (g[e] - x[e] * dot) * unit;
      }
      store_row(dx + (h0 + i) * kRopeD, l, g);
    }
  }
}

// A fixed number of CTAs, each with every gridDim-th group of tasks, so that
// the weights' gradients are summed in registers and leave a CTA once.
template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) rope_bwd_kernel(const QkRopeArgs a) {
  __shared__ float sum[kTasks][2][kRopeD];
  const int lane = threadIdx.x & 15, hw = threadIdx.x >> 4;
  const unsigned mask = half_mask();
  grid_dependency_wait();
  grid_launch_dependents();
  const RopeLane l = rope_lane(a.r, lane);
  const RopeFreq f = rope_freq(a.r, l, lane);
  const int heads = a.h_q + a.h_k;
  const int64_t tasks = (int64_t)a.pos.T * a.splits;
  float dwq[8] = {}, dwk[8] = {};
  for (int64_t task = (int64_t)blockIdx.x * kTasks + hw; task < tasks; task += (int64_t)gridDim.x * kTasks) {
    const int t = (int)(task / a.splits), part = (int)(task % a.splits);
    int pos;
    if (!token_position(a.pos, t, pos)) continue;
    float c[4], s[4];
    rope_angles(a.r, l, f, pos, c, s);
    const int h0 = (int)((int64_t)part * heads / a.splits), h1 = (int)((int64_t)(part + 1) * heads / a.splits);
    const int q0 = min(h0, a.h_q), q1 = min(h1, a.h_q), k0 = max(h0 - a.h_q, 0), k1 = max(h1 - a.h_q, 0);
    turn_heads_bwd<T, kInterleaved>(a.r, l, c, s, static_cast<const T*>(a.q) + t * a.q_stride + q0 * kRopeD,
                                    static_cast<const T*>(a.q_out) + t * a.q_out_stride + q0 * kRopeD,
                                    static_cast<T*>(a.dq) + t * a.dq_stride + q0 * kRopeD, q1 - q0, a.q_weight, dwq, mask);
    turn_heads_bwd<T, kInterleaved>(a.r, l, c, s, static_cast<const T*>(a.k) + t * a.k_stride + k0 * kRopeD,
                                    static_cast<const T*>(a.k_out) + t * a.k_out_stride + k0 * kRopeD,
                                    static_cast<T*>(a.dk) + t * a.dk_stride + k0 * kRopeD, k1 - k0, a.k_weight, dwk, mask);
  }
  if (!a.part) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int at = (e < 4 ? l.o0 : l.o1 - 4) + e;
    sum[hw][0][at] = dwq[e];
    sum[hw][1][at] = dwk[e];
  }
  __syncthreads();
  const int side = threadIdx.x >> 7, at = threadIdx.x & 127;
  float v = 0.f;
#pragma unroll
  for (int i = 0; i < kTasks; ++i) v += sum[i][side][at];
  a.part[((int64_t)blockIdx.x * 2 + side) * kRopeD + at] = v;
}

// The CTAs' sums to one, in a fixed order: CTA (side, 32 elements), a row a warp.
__global__ void __launch_bounds__(1024) rope_weight_kernel(const float* part, int n, float* dq_weight, float* dk_weight) {
  __shared__ double sum[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int side = blockIdx.x >> 2, at = (blockIdx.x & 3) * 32 + lane;
  grid_dependency_wait();
  grid_launch_dependents();
  float* out = side ? dk_weight : dq_weight;
  if (!out) return;
  double v = 0.0;
#pragma unroll 8
  for (int i = warp; i < n; i += 32) v += part[((int64_t)i * 2 + side) * kRopeD + at];
  sum[warp][lane] = v;
  __syncthreads();
  if (warp == 0) {
    v = 0.0;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += sum[i][lane];
    out[at] = (float)v;
  }
}

}  // namespace

cudaError_t launch_qk_rope(const QkRopeArgs& a, bool f32, cudaStream_t st) {
  const dim3 grid((unsigned)(((int64_t)a.pos.T * a.splits + kTasks - 1) / kTasks));
  const dim3 block(kThreads);
  if (f32)
    return a.r.interleaved ? launch_kernel(rope_kernel<float, true>, grid, block, 0, st, true, a)
                           : launch_kernel(rope_kernel<float, false>, grid, block, 0, st, true, a);
  return a.r.interleaved ? launch_kernel(rope_kernel<__nv_bfloat16, true>, grid, block, 0, st, true, a)
                         : launch_kernel(rope_kernel<__nv_bfloat16, false>, grid, block, 0, st, true, a);
}

cudaError_t launch_qk_rope_bwd(const QkRopeArgs& a, bool f32, int ctas, cudaStream_t st) {
  const dim3 grid(ctas), block(kThreads);
  if (f32)
    return a.r.interleaved ? launch_kernel(rope_bwd_kernel<float, true>, grid, block, 0, st, true, a)
                           : launch_kernel(rope_bwd_kernel<float, false>, grid, block, 0, st, true, a);
  return a.r.interleaved ? launch_kernel(rope_bwd_kernel<__nv_bfloat16, true>, grid, block, 0, st, true, a)
                         : launch_kernel(rope_bwd_kernel<__nv_bfloat16, false>, grid, block, 0, st, true, a);
}

cudaError_t launch_qk_rope_weights(const QkRopeArgs& a, int ctas, cudaStream_t st) {
  return launch_kernel(rope_weight_kernel, dim3(8), dim3(1024), 0, st, true, (const float*)a.part, ctas, a.dq_weight,
                       a.dk_weight);
}

}  // namespace gdn
