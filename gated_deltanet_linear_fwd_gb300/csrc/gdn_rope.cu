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
// Each element is read and written once; what comes next to that is issue
// slots, so the arithmetic is on pairs of fp32.  Measured, 8 + 2 heads of bf16:
// 32768 tokens 31.0 us, 5.4 TB/s, 81 % of what a copy reaches, with issue slots
// 74 % busy; the gradient of 34150 packed tokens, weights' sums with it, 52.5
// us, 5.0 TB/s (75 %).  32768 tokens of fp32 57.7 us (87 %), their gradient 87.9
// (86 %).  One token 2.0 us, back to back in a graph.
// First versions, a block a tile of tokens: 33.8 and 91.7 us.
#include "gdn_rope.cuh"

namespace gdn {
namespace {

template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_kernel(const QkRopeArgs a) {
  __shared__ RopeRing ring;
  grid_dependency_wait();
  grid_launch_dependents();
  turn_run<T, kInterleaved>(a, blockIdx.x, ring);
}

// The gradient of a row, in g, from it and the input x; dw: of the weight.
template <bool kInterleaved>
__device__ __forceinline__ void row_back(const QkRopeArgs& a, const RopeLane& l, const Angles& angle, bool all, bool norm, bool in,
                                         F2 (&x)[4], F2 (&g)[4], const F2 (&w)[4], F2 (&dw)[4]) {
  turn_row<kInterleaved, true>(all, l, angle, g);
  if (!norm) return;
  const float ss = half_sum(dot_row(x, x));
  float f = rsqrt_approx(fmaf(ss, a.r.inv_n, a.r.eps)), unit = 1.f;
  const bool large = large_heads(ss);
  if (large) f = scaled_head(x, ss, a.r.inv_n, a.r.eps, unit);
  scale_row(x, f);
  if (in) {
#pragma unroll
    for (int e = 0; e < 4; ++e) dw[e] = fma2(g[e], x[e], dw[e]);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) g[e] = mul2(g[e], w[e]);
  const F2 m = f2(-half_sum(dot_row(g, x)) * a.r.inv_n);
  // unit comes in halves, one with f: f unit may be below fp32's normal numbers, and
  // a gradient times f past the largest
  const float root = large && unit != 1.f ? kHeadUnitRoot : 1.f;
  f *= root;
#pragma unroll
  for (int e = 0; e < 4; ++e) g[e] = mul2(fma2(x[e], m, g[e]), f2(f));
  if (large) scale_row(g, root);
}

// A lane's sums of the weights' gradients go to its pairs of fp32, [16][threads].
// 5500 equal terms a lane: without this off by 800 roundings of 2^-24.  2^20 tokens of
// 8 + 2 heads, 2100 terms a lane, take 1356 us, and took 1350.
constexpr int kKept = 16, kKeptBytes = kKept * kRopeThreads * sizeof(float2);
__device__ __forceinline__ void put_away(float2* kept, F2 (&dwq)[4], F2 (&dwk)[4]) {
#pragma unroll
  for (int i = 0; i < kKept; ++i) {
    const F2 pair = i < 8 ? dwq[i / 2] : dwk[i / 2 - 4];
    float2& at = kept[i * kRopeThreads + threadIdx.x];
    Sum2 s = {at.x, at.y};
    s.add(i % 2 ? parts(pair).y : parts(pair).x);
    at = make_float2(s.hi, s.lo);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) dwq[e] = dwk[e] = f2(0.f);
}

// As turn_run, with two inputs; the weights' gradients are summed in registers.
// 105 to 119 registers, 16 warps an SM: a row's instructions wait for one another,
// and at 59 % of issue slots neither those nor memory (75 % of a copy's) is full.
// Taking both sums of a row at once, in 5 shuffles and not 8, changed nothing.
template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads, 2) rope_bwd_kernel(const QkRopeArgs a) {
  constexpr int kBatch = sizeof(T) == 2 ? 2 : 1, kGroups = 2 * kRopeWarps, kRow = kRopeD * sizeof(T);
  constexpr int kStage = kBatch * 4 * kRow, kStages = 3;  // 2 KB: of each head rows of x and g of two tokens
  __shared__ union {
    alignas(16) char ring[kRopeWarps][kStages * kStage];
    float sum[kGroups][2][kRopeD];
  } sh;
  const int lane = threadIdx.x & 15, half = threadIdx.x >> 4 & 1, hw = threadIdx.x >> 4;
  const RopeLane l = rope_lane(a.r, lane);
  const bool norm = a.r.norm != kNormNone, all = a.r.rot == kRopeD;
  const int T_all = a.pos.T, h_q = a.side[0].heads, heads = h_q + a.side[1].heads, gap = (l.o1 - l.o0) * (int)sizeof(T);
  const unsigned warp = warp_index();
  grid_dependency_wait();
  grid_launch_dependents();
  F2 dwq[4], dwk[4], w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) dwq[e] = dwk[e] = w[e] = f2(0.f);
  char* ring = sh.ring[warp];
  Walk now = rope_run(a, (int64_t)blockIdx.x * kRopeWarps + warp), next = now;
  extern __shared__ float2 kept[];
  int mark = -1;  // what is left of a long run when the sums are put away next
  if (a.fold && now.left > kRopeFold) {
    mark = now.left - kRopeFold;
    for (int i = 0; i < kKept; ++i) kept[i * kRopeThreads + threadIdx.x] = make_float2(0.f, 0.f);
  }
  const char *x = nullptr, *g = nullptr;  // the lane's 16 bytes of the next head's rows
  auto place = [&] {
    const bool key = next.h >= h_q;
    const RopeSide& s = a.side[key];
    x = head_at<T>(s.in, s.in_stride, T_all, next.pair, next.h - (key ? h_q : 0)) + lane * 16;
    g = head_at<T>(s.out, s.out_stride, T_all, next.pair, next.h - (key ? h_q : 0)) + lane * 16;
  };
  auto copy_batch = [&](int slot) {
    if (next.left > 0) {
      const int n = next.batch(h_q, heads, kBatch);
      char* to = ring + slot * kStage + half * kRow + lane * 16;
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (i < n) {
#pragma unroll
          for (int j = 0; j < kRow; j += 256) {
            copy16(to + i * 4 * kRow + j, g + i * kRow + j);
            if (norm) copy16(to + (i * 4 + 2) * kRow + j, x + i * kRow + j);
          }
        }
      x += n * kRow;
      g += n * kRow;
      if (next.step(n, h_q, heads)) place();
    }
    copy_commit();
  };
  place();
#pragma unroll
  for (int i = 0; i < kStages; ++i) copy_batch(i);
  int slot = 0;
  bool in = false, all_in = false, new_pair = true, new_side = true;
  TokenSeq seq;
  Angles angle;
  char* y = nullptr;
  while (now.left > 0) {
    const bool key = now.h >= h_q;
    if (new_pair) {
      const int t2 = 2 * now.pair + half, t = min(t2, T_all - 1);
      int pos = 0;
      in = token_position(a.pos, t, seq, pos) && t == t2;
      all_in = __all_sync(0xffffffffu, in);
      angle = rope_angles(a.r, l, rope_freq(a.r, l, lane), pos);
    }
    if (new_side) {
      const RopeSide& s = a.side[key];
      y = const_cast<char*>(head_at<T>(s.dx, s.dx_stride, T_all, now.pair, now.h - (key ? h_q : 0))) + l.o0 * (int)sizeof(T);
      load_weight(s.weight, l, w);
    }
    const int n = now.batch(h_q, heads, kBatch);
    copy_wait<kStages - 1>();
    __syncwarp();
    const char* from = ring + slot * kStage + half * kRow + l.o0 * (int)sizeof(T);
    typename RowOf<T>::type rx[kBatch], rg[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      rg[i] = load_row<T>(from + i * 4 * kRow, from + i * 4 * kRow + gap);
      rx[i] = load_row<T>(from + (i * 4 + 2) * kRow, from + (i * 4 + 2) * kRow + gap);
    }
    __syncwarp();
    copy_batch(slot);
    slot = slot + 1 == kStages ? 0 : slot + 1;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (i >= n) break;
      F2 gr[4], xr[4];
      unpack_row(rg[i], gr);
      unpack_row(rx[i], xr);
      if (key) row_back<kInterleaved>(a, l, angle, all, norm, all_in || in, xr, gr, w, dwk);
      else row_back<kInterleaved>(a, l, angle, all, norm, all_in || in, xr, gr, w, dwq);
      if (all_in || in) store_row<T>(y + i * kRow, y + i * kRow + gap, gr);
    }
    y += n * kRow;
    new_side = now.step(n, h_q, heads);
    new_pair = now.h == 0;
    if (now.left <= mark) {
      put_away(kept, dwq, dwk);
      mark = max(now.left - kRopeFold, 0);
    }
  }
  copy_wait<0>();
  if (!a.part) return;
  if (mark >= 0) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      auto value = [&](int i) {
        const float2 v = kept[i * kRopeThreads + threadIdx.x];
        return Sum2{v.x, v.y}.value();
      };
      dwq[e] = f2(value(2 * e), value(2 * e + 1));
      dwk[e] = f2(value(8 + 2 * e), value(9 + 2 * e));
    }
  }
  __syncthreads();  // the rings are done with
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int at = (e < 2 ? l.o0 : l.o1 - 4) + 2 * e;
    const float2 p = parts(dwq[e]), q = parts(dwk[e]);
    sh.sum[hw][0][at] = p.x;
    sh.sum[hw][0][at + 1] = p.y;
    sh.sum[hw][1][at] = q.x;
    sh.sum[hw][1][at + 1] = q.y;
  }
  __syncthreads();
  const int side = threadIdx.x >> 7, at = threadIdx.x & 127;
  float v = 0.f;
#pragma unroll
  for (int i = 0; i < kGroups; ++i) v += sh.sum[i][side][at];
  a.part[((int64_t)blockIdx.x * 2 + side) * kRopeD + at] = v;
}

// The CTAs' sums to one, in a fixed order: CTA (side, 8 elements), a row of them
// a quarter of a warp.  So small that it is there, and waiting, before the kernel
// that writes the sums has ended: with 8 CTAs of 1024 threads, which begin after
// it, the gradient took 58.2 us and not 54.2; with 64-bit additions 1.5 us more.
constexpr int kSumThreads = 128, kSumWidth = 8, kSumRows = kSumThreads / kSumWidth;
__global__ void __launch_bounds__(kSumThreads) rope_weight_kernel(const QkRopeArgs a) {
  __shared__ float2 sum[kSumRows][kSumWidth];
  const int e = threadIdx.x % kSumWidth, row = threadIdx.x / kSumWidth;
  const int side = blockIdx.x / (kRopeD / kSumWidth), at = blockIdx.x % (kRopeD / kSumWidth) * kSumWidth + e;
  grid_dependency_wait();
  grid_launch_dependents();
  float* out = a.side[side].d_weight;
  if (!out) return;
  constexpr int kEach = (kRopeBwdCtas + kSumRows - 1) / kSumRows;
  float x[kEach];  // all at once: one after another they would be waited for
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int cta = row + i * kSumRows;
    x[i] = cta < a.ctas ? a.part[((int64_t)cta * 2 + side) * kRopeD + at] : 0.f;
  }
  Sum2 v;
#pragma unroll
  for (int i = 0; i < kEach; ++i) v.add(x[i]);
  sum[row][e] = make_float2(v.hi, v.lo);
  __syncthreads();
  if (row == 0) {
    v = {};
#pragma unroll
    for (int i = 0; i < kSumRows; ++i) v.add({sum[i][e].x, sum[i][e].y});
    out[at] = v.value();
  }
}

}  // namespace

cudaError_t launch_qk_rope(const QkRopeArgs& a, bool f32, cudaStream_t st) {
  const dim3 grid(a.ctas), block(kRopeThreads);
  if (f32)
    return a.r.interleaved ? launch_kernel(rope_kernel<float, true>, grid, block, 0, st, true, a)
                           : launch_kernel(rope_kernel<float, false>, grid, block, 0, st, true, a);
  return a.r.interleaved ? launch_kernel(rope_kernel<__nv_bfloat16, true>, grid, block, 0, st, true, a)
                         : launch_kernel(rope_kernel<__nv_bfloat16, false>, grid, block, 0, st, true, a);
}

cudaError_t rope_bwd_setup() {
  auto allow = [](auto kernel) { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kKeptBytes); };
  cudaError_t e = allow(rope_bwd_kernel<float, true>);
  if (e == cudaSuccess) e = allow(rope_bwd_kernel<float, false>);
  if (e == cudaSuccess) e = allow(rope_bwd_kernel<__nv_bfloat16, true>);
  if (e == cudaSuccess) e = allow(rope_bwd_kernel<__nv_bfloat16, false>);
  return e;
}

cudaError_t launch_qk_rope_bwd(const QkRopeArgs& a, bool f32, cudaStream_t st) {
  const dim3 grid(a.ctas), block(kRopeThreads);
  const size_t smem = a.fold ? kKeptBytes : 0;
  if (f32)
    return a.r.interleaved ? launch_kernel(rope_bwd_kernel<float, true>, grid, block, smem, st, true, a)
                           : launch_kernel(rope_bwd_kernel<float, false>, grid, block, smem, st, true, a);
  return a.r.interleaved ? launch_kernel(rope_bwd_kernel<__nv_bfloat16, true>, grid, block, smem, st, true, a)
                         : launch_kernel(rope_bwd_kernel<__nv_bfloat16, false>, grid, block, smem, st, true, a);
}

cudaError_t launch_qk_rope_weights(const QkRopeArgs& a, cudaStream_t st) {
  return launch_kernel(rope_weight_kernel, dim3(2 * kRopeD / kSumWidth), dim3(kSumThreads), 0, st, true, a);
}

}  // namespace gdn
