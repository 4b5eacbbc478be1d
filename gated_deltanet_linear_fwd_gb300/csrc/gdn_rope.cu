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
// Each element is read and written once and both are bound by that; what
// comes next is issue slots, so the arithmetic is on pairs of fp32.
#include "gdn_rope.cuh"

namespace gdn {
namespace {

template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads, sizeof(T) == 2 ? 4 : 3) rope_kernel(const QkRopeArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  const unsigned task = blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
  if ((task >> a.shares_log2) * 2 < (unsigned)a.pos.T) turn_tokens<T, kInterleaved>(a, task);
}

// As turn_tokens with two inputs, one side a CTA (of q's come first), so that one
// weight's gradient is summed in registers and leaves a CTA once.
template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads, 3) rope_bwd_kernel(const QkRopeArgs a) {
  constexpr int kBatch = kRopeBatch<T> / 2, kGroups = 2 * kRopeWarps, kStep = kRopeD * sizeof(T);
  __shared__ float sum[kGroups][kRopeD];
  const int lane = threadIdx.x & 15, hw = threadIdx.x >> 4;
  const RopeLane l = rope_lane(a.r, lane);
  const bool norm = a.r.norm != kNormNone, key = (int)blockIdx.x >= a.side[0].ctas;
  const RopeSide& s = a.side[key];
  const float inv_n = a.r.inv_n, eps = a.r.eps;
  const int gap = (l.o1 - l.o0) * (int)sizeof(T), share = s.share, log2 = s.shares_log2;
  grid_dependency_wait();
  grid_launch_dependents();
  F2 dw[4], w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) dw[e] = f2(0.f);
  load_weight(s.weight, l, w);
  const unsigned tasks = (((unsigned)a.pos.T + 1) / 2) << log2;
  for (unsigned task = (blockIdx.x - (key ? a.side[0].ctas : 0)) * kRopeWarps + (threadIdx.x >> 5); task < tasks;
       task += s.ctas * kRopeWarps) {
    const int t2 = (int)(task >> log2) * 2 + (hw & 1), t = min(t2, a.pos.T - 1);
    const int h = (int)(task & ((1u << log2) - 1)) * share;
    int n = min(share, s.heads - h);
    if (n <= 0) continue;
    const char* x0 = head_at<T>(s.in, s.in_stride, t, h, l);
    const char* g0 = head_at<T>(s.out, s.out_stride, t, h, l);
    char* y0 = const_cast<char*>(head_at<T>(s.dx, s.dx_stride, t, h, l));
    typename RowOf<T>::type rx[kBatch], rg[kBatch];
    load_batch<T, kBatch>(rg, g0, gap, n);
    if (norm) load_batch<T, kBatch>(rx, x0, gap, n);
    int pos = 0;
    const bool in = token_position(a.pos, t, pos) && t == t2;
    const Angles angle = rope_angles(a.r, l, rope_freq(a.r, l, lane), pos);
    while (true) {
      char* y1 = y0 + gap;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (i >= n) break;
        F2 g[4];
        unpack_row(rg[i], g);
        turn_row<kInterleaved, true>(l, angle, g);
        if (norm) {
          F2 x[4];
          unpack_row(rx[i], x);
          float unit;
          const float f = head_scale(x, inv_n, eps, unit);
          scale_row(x, f);
          if (in) {
#pragma unroll
            for (int e = 0; e < 4; ++e) dw[e] = fma2(g[e], x[e], dw[e]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) g[e] = mul2(g[e], w[e]);
          const F2 m = f2(-half_sum(dot_row(g, x)) * inv_n);
#pragma unroll
          for (int e = 0; e < 4; ++e) g[e] = mul2(fma2(x[e], m, g[e]), f2(f));
          if (unit != 1.f) scale_row(g, unit);
        }
        if (in) store_row<T>(y0 + i * kStep, y1 + i * kStep, g);
      }
      n -= kBatch;
      if (n <= 0) break;
      x0 += kBatch * kStep;
      g0 += kBatch * kStep;
      y0 += kBatch * kStep;
      load_batch<T, kBatch>(rg, g0, gap, n);
      if (norm) load_batch<T, kBatch>(rx, x0, gap, n);
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int at = (e < 2 ? l.o0 : l.o1 - 4) + 2 * e;
    const float2 x = parts(dw[e]);
    sum[hw][at] = x.x;
    sum[hw][at + 1] = x.y;
  }
  __syncthreads();
  if (threadIdx.x < kRopeD) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) v += sum[i][threadIdx.x];
    a.part[(int64_t)blockIdx.x * kRopeD + threadIdx.x] = v;
  }
}

// The CTAs' sums to one, in a fixed order: CTA (side, 32 elements), a row a warp.
__global__ void __launch_bounds__(1024) rope_weight_kernel(const QkRopeArgs a) {
  __shared__ double sum[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int side = blockIdx.x >> 2, at = (blockIdx.x & 3) * 32 + lane;
  grid_dependency_wait();
  grid_launch_dependents();
  float* out = a.side[side].d_weight;
  if (!out) return;
  const float* part = a.part + (int64_t)(side ? a.side[0].ctas : 0) * kRopeD;
  double v = 0.0;
#pragma unroll 8
  for (int i = warp; i < a.side[side].ctas; i += 32) v += part[(int64_t)i * kRopeD + at];
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
  const dim3 grid((unsigned)((rope_tasks(a) + kRopeWarps - 1) / kRopeWarps)), block(kRopeThreads);
  if (f32)
    return a.r.interleaved ? launch_kernel(rope_kernel<float, true>, grid, block, 0, st, true, a)
                           : launch_kernel(rope_kernel<float, false>, grid, block, 0, st, true, a);
  return a.r.interleaved ? launch_kernel(rope_kernel<__nv_bfloat16, true>, grid, block, 0, st, true, a)
                         : launch_kernel(rope_kernel<__nv_bfloat16, false>, grid, block, 0, st, true, a);
}

cudaError_t launch_qk_rope_bwd(const QkRopeArgs& a, bool f32, cudaStream_t st) {
  const dim3 grid(a.side[0].ctas + a.side[1].ctas), block(kRopeThreads);
  if (f32)
    return a.r.interleaved ? launch_kernel(rope_bwd_kernel<float, true>, grid, block, 0, st, true, a)
                           : launch_kernel(rope_bwd_kernel<float, false>, grid, block, 0, st, true, a);
  return a.r.interleaved ? launch_kernel(rope_bwd_kernel<__nv_bfloat16, true>, grid, block, 0, st, true, a)
                         : launch_kernel(rope_bwd_kernel<__nv_bfloat16, false>, grid, block, 0, st, true, a);
}

cudaError_t launch_qk_rope_weights(const QkRopeArgs& a, cudaStream_t st) {
  return launch_kernel(rope_weight_kernel, dim3(8), dim3(1024), 0, st, true, a);
}

}  // namespace gdn
