// The short causal convolution before the gated delta rule: per channel c of
// the projection and token t of a sequence, with taps w and kept inputs before
// the sequence's first token,
//   u_t = b + sum_{j < W} w_j x_{t - W + 1 + j},   y = u sigmoid(u)  (or u),
// heads of 128 channels, q's, then k's, then v's; those of q and k scaled to
// unit length, y / sqrt(sum y^2 + eps).  And its gradients, and its form for
// one new token of each sequence.
//
// All of it moves each element once and is bound by that or, in the gradient, by
// what it computes meanwhile.  A warp owns a head's channels over a run of tokens
// and keeps the last W - 1 inputs in registers, so an input is read once but for
// the W - 1 before each run.  Measured, 2 + 2 + 8 heads, 4 taps, bf16: 32768
// tokens 35.5 us, 5.7 TB/s, 85 % of what a copy reaches; 348160 tokens 331 us, 97
// %; the gradient of 32768 tokens 69.6 us, 4.3 TB/s (65 %); one token for 256
// sequences 2.6 us, back to back in a graph.  First versions: 78.6, 662 and 165.
#include <type_traits>

#include "gdn_conv.cuh"
#include "gdn_pair.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// First token and end of the sequence that token t is in, within [0, T]; seq -1
// where it is outside every one, then with the end of such tokens.
struct ConvSeq {
  int seq, begin, end;
};
__device__ __forceinline__ ConvSeq conv_seq(const ConvArgs& a, int t) {
  ConvSeq s;
  if (!a.cu) {
    s.seq = t / a.n_each;
    s.begin = s.seq * a.n_each;
    s.end = s.begin + a.n_each;
    return s;
  }
  int lo = 0, hi = a.n_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.cu[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  s.seq = lo;
  s.begin = a.cu[lo];
  s.end = a.cu[lo + 1];
  if (s.begin < 0 || s.begin > t || s.end <= t || s.end > a.T) {
    s.seq = -1;
    s.end = s.begin > t ? min(s.begin, a.T) : a.T;
    s.begin = t;
  }
  return s;
}

// The sequence of token t, which is where s ends: mostly the next one.
__device__ __forceinline__ ConvSeq conv_seq_after(const ConvArgs& a, const ConvSeq& s, int t) {
  if (a.cu && s.seq >= 0 && s.seq + 2 <= a.n_seqs) {
    const ConvSeq n = {s.seq + 1, a.cu[s.seq + 1], a.cu[s.seq + 2]};
    if (n.begin == t && n.end > t && n.end <= a.T) return n;
  }
  return conv_seq(a, t);
}

// ---- four consecutive channels of a lane, as two pairs of fp32 ----
// A warp holds a head of 128 channels.
template <typename T>
struct RawOf;
template <>
struct RawOf<float> {
  using type = float4;
};
template <>
struct RawOf<__nv_bfloat16> {
  using type = uint2;
};
template <typename T>
using Raw = typename RawOf<T>::type;
template <typename T>
__device__ __forceinline__ Raw<T> load_raw(const T* p) {
  return *reinterpret_cast<const Raw<T>*>(p);
}
__device__ __forceinline__ void unpack(const float4& r, F2 (&x)[2]) {
  x[0] = f2(r.x, r.y);
  x[1] = f2(r.z, r.w);
}
__device__ __forceinline__ void unpack(const uint2& r, F2 (&x)[2]) {
  x[0] = bf16_pair(r.x);
  x[1] = bf16_pair(r.y);
}
__device__ __forceinline__ void store4(float* p, const F2 (&x)[2]) {
  const float2 a = parts(x[0]), b = parts(x[1]);
  *reinterpret_cast<float4*>(p) = make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const F2 (&x)[2]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pair_bf16(x[0]), pair_bf16(x[1]));
}
template <typename T>
__device__ __forceinline__ void load4(const T* p, F2 (&x)[2]) {
  unpack(load_raw(p), x);
}

// 1 / (1 + e^-u).  u log2 e is rounded once, so e^-u is off by 1.2 |u| of 2^-24 next to
// the power's 2 ulp, and s by 1 - s times that: above 0 no more than 0.4 roundings; below,
// where s is small, 1.2 |u| of them, which moves u s by less than 2^-24.
__device__ __forceinline__ F2 sigmoid(F2 u) {
  const float2 t = parts(mul2(u, f2(-1.4426950408889634f)));
  const float2 d = parts(add2(f2(ex2_approx(t.x), ex2_approx(t.y)), f2(1.f)));
  return f2(rcp_approx(d.x), rcp_approx(d.y));
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}
__device__ __forceinline__ float dot(const F2 (&x)[2], const F2 (&y)[2]) { return both(fma2(x[1], y[1], mul2(x[0], y[0]))); }
// 1 / sqrt(sum y^2 + eps) of a head; past fp32's range y is scaled by 2^-68
// (unit), beside which eps is nothing, and the result belongs to the scaled y.
__device__ __forceinline__ float unit_scale(F2 (&y)[2], float eps, float& unit) {
  const float ss = warp_sum(dot(y, y));
  unit = 1.f;
  if (ss <= 3e38f) return rsqrt_approx(ss + eps);  // all lanes have the same sum
  unit = 0x1p-68f;
  y[0] = mul2(y[0], f2(unit));
  y[1] = mul2(y[1], f2(unit));
  return rsqrt_approx(warp_sum(dot(y, y)));
}

// Sums over the warp of N values a lane, N a power of two: in the first rounds a
// lane gives half of its values away and keeps the other half's sums, so that
// 4 (8) values take 6 (9) shuffles and not 20 (40).  The lane ends with the sum of
// value lane / (32 / N); group_value hands it to all.
template <int N>
__device__ __forceinline__ float group_sums(float (&v)[N]) {
  const int lane = threadIdx.x & 31;
  int d = 16;
#pragma unroll
  for (int n = N / 2; n; n >>= 1, d >>= 1) {
    const bool upper = lane & d;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = upper ? v[i] : v[i + n], keep = upper ? v[i + n] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, d);
    }
  }
#pragma unroll
  for (; d; d >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], d);
  return v[0];
}
template <int N>
__device__ __forceinline__ float group_value(float sum, int i) {
  return __shfl_sync(0xffffffffu, sum, i * (32 / N));
}
// Heads of G tokens to unit length at once, or one by one where a sum of
// squares passes fp32's range.
template <int G>
__device__ __forceinline__ void unit_group(F2 (&y)[G][2], float eps) {
  float v[G];
#pragma unroll
  for (int i = 0; i < G; ++i) v[i] = dot(y[i], y[i]);
  const float ss = group_sums<G>(v);
  if (__any_sync(0xffffffffu, !(ss <= 3e38f))) {
#pragma unroll
    for (int i = 0; i < G; ++i) {
      float unit;
      const F2 r = f2(unit_scale(y[i], eps, unit));
      y[i][0] = mul2(y[i][0], r);
      y[i][1] = mul2(y[i][1], r);
    }
    return;
  }
  const float mine = rsqrt_approx(ss + eps);
#pragma unroll
  for (int i = 0; i < G; ++i) {
    const F2 r = f2(group_value<G>(mine, i));
    y[i][0] = mul2(y[i][0], r);
    y[i][1] = mul2(y[i][1], r);
  }
}

// A lane's taps from [C, W], by tap.
template <int W>
__device__ __forceinline__ void load_taps(const float* weight, int c, F2 (&w)[W][2]) {
  const float4* p = reinterpret_cast<const float4*>(weight + (int64_t)c * W);
  float f[W * 4];
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const float4 v = __ldg(p + i);
    f[4 * i] = v.x; f[4 * i + 1] = v.y; f[4 * i + 2] = v.z; f[4 * i + 3] = v.w;
  }
#pragma unroll
  for (int j = 0; j < W; ++j) {
    w[j][0] = f2(f[j], f[W + j]);
    w[j][1] = f2(f[2 * W + j], f[3 * W + j]);
  }
}

// A head's rows of the output: q, k or v.
template <typename T>
struct HeadRows {
  T* p;
  int64_t stride;
};
template <typename T>
__device__ __forceinline__ HeadRows<T> head_rows(const ConvArgs& a, int head) {
  if (head < a.h_qk) return {static_cast<T*>(a.q) + head * kConvD, (int64_t)a.h_qk * kConvD};
  if (head < 2 * a.h_qk) return {static_cast<T*>(a.k) + (head - a.h_qk) * kConvD, (int64_t)a.h_qk * kConvD};
  return {static_cast<T*>(a.v) + (head - 2 * a.h_qk) * kConvD, (int64_t)a.h_v * kConvD};
}

// The W - 1 inputs before token t: earlier tokens, then the kept state.
template <typename T, int W>
__device__ __forceinline__ void load_window(const ConvArgs& a, const ConvSeq& s, int t, int c, int C, F2 (&win)[W - 1][2]) {
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    const int at = t - (W - 1) + j;
    if (at >= s.begin) {
      load4(static_cast<const T*>(a.x) + at * a.x_stride + c, win[j]);
    } else if (a.state && s.seq >= 0) {
      load4(static_cast<const T*>(a.state) + ((int64_t)s.seq * (W - 1) + (W - 1) + at - s.begin) * C + c, win[j]);
    } else {
      win[j][0] = win[j][1] = f2(0.f);
    }
  }
}

// u of the token whose inputs are x[0] .. x[W - 1].
template <int W>
__device__ __forceinline__ void taps(const F2 (*x)[2], const F2 (&w)[W][2], const F2 (&b)[2], F2 (&u)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    u[i] = b[i];
#pragma unroll
    for (int j = 0; j < W; ++j) u[i] = fma2(w[j][i], x[j][i], u[i]);
  }
}
__device__ __forceinline__ void load_bias(const float* bias, int c, F2 (&b)[2]) {
  b[0] = b[1] = f2(0.f);
  if (bias) load4(bias + c, b);
}
template <bool kSilu>
__device__ __forceinline__ void activate(F2 (&u)[2]) {
  if (kSilu) {
    u[0] = mul2(u[0], sigmoid(u[0]));
    u[1] = mul2(u[1], sigmoid(u[1]));
  }
}
template <bool kSilu>
__device__ __forceinline__ void finish(F2 (&u)[2], bool unit_head, float eps) {
  activate<kSilu>(u);
  if (unit_head) {
    float unit;
    const F2 r = f2(unit_scale(u, eps, unit));
    u[0] = mul2(u[0], r);
    u[1] = mul2(u[1], r);
  }
}

// A warp's (backward: a CTA's) head and which of its runs (groups of runs).
struct ConvTask {
  int head, place, run;
  bool unit_head;
};
__device__ __forceinline__ ConvTask conv_task(const ConvArgs& a, unsigned i) {
  const unsigned n_unit = a.n_unit, first = n_unit * (unsigned)a.runs[0];
  ConvTask t;
  t.unit_head = i < first;
  const unsigned heads = t.unit_head ? n_unit : (unsigned)(2 * a.h_qk + a.h_v) - n_unit;
  if (!t.unit_head) i -= first;
  t.place = (int)(i / heads);
  t.head = (int)(i % heads) + (t.unit_head ? 0 : (int)n_unit);
  t.run = a.run[t.unit_head ? 0 : 1];
  return t;
}

// The state after the call of a sequence's head, a warp each: row r is the padded
// row len + r of (state, tokens).
template <typename T, int W>
__device__ __forceinline__ void final_state(const ConvArgs& a, unsigned task, int heads) {
  const unsigned seq = task / (unsigned)heads;
  if (seq >= (unsigned)a.n_seqs) return;
  const int C = heads * kConvD, c = (int)(task - seq * heads) * kConvD + 4 * (threadIdx.x & 31);
  int begin, end;
  if (a.cu) {
    begin = min(max(a.cu[seq], 0), a.T);
    end = min(max(a.cu[seq + 1], begin), a.T);
  } else {
    begin = (int)seq * a.n_each;
    end = begin + a.n_each;
  }
  const int64_t row = (int64_t)seq * (W - 1);
  Raw<T> v[W - 1];
#pragma unroll
  for (int r = 0; r < W - 1; ++r) {
    const int at = end - (W - 1) + r;
    v[r] = {};
    if (at >= begin) v[r] = load_raw(static_cast<const T*>(a.x) + at * a.x_stride + c);
    else if (a.state) v[r] = load_raw(static_cast<const T*>(a.state) + (row + (W - 1) + at - begin) * C + c);
  }
#pragma unroll
  for (int r = 0; r < W - 1; ++r) *reinterpret_cast<Raw<T>*>(static_cast<T*>(a.final_state) + (row + r) * C + c) = v[r];
}

// A warp a (run, head); then CTAs for the final states.  A warp's next tokens are
// copied into a ring of shared memory of its own: in registers there is room
// for too few (with four tokens ahead warps waited for memory three times as
// long as they computed).  Groups of four tokens
// within a sequence go through straight code, the groups at its ends token by
// token.
template <typename T, int W, bool kSilu>
__global__ void __launch_bounds__(kThreads, 3) conv_kernel(const ConvArgs a) {
  constexpr int G = 4, kRowBytes = kConvD * sizeof(T), kRing = 4096 / kRowBytes;  // 16 tokens, or 8 of fp32
  __shared__ alignas(16) char ring_all[kWarps][kRing * kRowBytes];
  const int lane = threadIdx.x & 31;
  grid_dependency_wait();
  grid_launch_dependents();
  const int heads = 2 * a.h_qk + a.h_v, C = heads * kConvD;
  const unsigned warp = warp_index();
  if (blockIdx.x >= (unsigned)a.blocks) {
    final_state<T, W>(a, (blockIdx.x - a.blocks) * kWarps + warp, heads);
    return;
  }
  const ConvTask task = conv_task(a, blockIdx.x * kWarps + warp);
  const int head = task.head, c = head * kConvD + 4 * lane;
  const int64_t first = (int64_t)task.place * task.run;
  if (head >= heads || first >= a.T) return;
  const int t0 = (int)first, t1 = (int)min((int64_t)a.T, first + task.run);
  const bool unit_head = task.unit_head;
  const float eps = a.eps;
  char* ring = ring_all[warp];
  // the lane's part of a copy: kRows tokens at a time, 16 bytes of one of them
  constexpr int kLanes = kRowBytes / 16, kRows = 32 / kLanes;
  const int64_t step = kRows * a.x_stride * (int64_t)sizeof(T);
  const char* from = static_cast<const char*>(a.x) + (((int64_t)t0 + lane / kLanes) * a.x_stride + head * kConvD) * (int64_t)sizeof(T) +
                     lane % kLanes * 16;
  int slot = 0;  // of the group that comes next
  auto copy_group = [&](int at, int left) {  // left: tokens of the run from the group on
    char* to = ring + at * kRowBytes + lane * 16;
    if (left >= G) {
#pragma unroll
      for (int i = 0; i < G; i += kRows) {
        copy16(to + i * kRowBytes, from);
        from += step;
      }
    } else {
#pragma unroll
      for (int i = 0; i < G; i += kRows) {
        if (i + lane / kLanes < left) copy16(to + i * kRowBytes, from);
        from += step;
      }
    }
    copy_commit();
  };
#pragma unroll
  for (int i = 0; i < kRing; i += G) copy_group(i, t1 - t0 - i);
  F2 w[W][2], b[2], win[W - 1][2];
  load_taps<W>(a.weight, c, w);
  load_bias(a.bias, c, b);
  const HeadRows<T> rows = head_rows<T>(a, head);
  T* y = rows.p + t0 * rows.stride + 4 * lane;
  ConvSeq s = {-1, 0, t0};
  int straight = 0;  // where the current sequence, and straight code, ends
  auto begin_sequence = [&](int t) {
    s = conv_seq_after(a, s, t);
    load_window<T, W>(a, s, t, c, C, win);
    straight = s.seq >= 0 ? min(s.end, t1) : -1;
  };
  for (int g = t0; g < t1; g += G) {
    if (g == s.end) begin_sequence(g);
    copy_wait<kRing / G - 1>();
    __syncwarp();
    const T* x = reinterpret_cast<const T*>(ring + slot * kRowBytes) + 4 * lane;
    F2 in[W - 1 + G][2];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      in[j][0] = win[j][0];
      in[j][1] = win[j][1];
    }
    if (g + G <= straight) {
      Raw<T> raw[G];
#pragma unroll
      for (int i = 0; i < G; ++i) raw[i] = load_raw(x + i * kConvD);
      __syncwarp();
      copy_group(slot, t1 - g - kRing);
      F2 u[G][2];
#pragma unroll
      for (int i = 0; i < G; ++i) {
        unpack(raw[i], in[W - 1 + i]);
        taps<W>(in + i, w, b, u[i]);
        activate<kSilu>(u[i]);
      }
      if (unit_head) unit_group<G>(u, eps);
#pragma unroll
      for (int i = 0; i < G; ++i) {
        store4(y, u[i]);
        y += rows.stride;
      }
#pragma unroll
      for (int j = 0; j < W - 1; ++j) {
        win[j][0] = in[G + j][0];
        win[j][1] = in[G + j][1];
      }
    } else {
#pragma unroll 1
      for (int i = 0; i < min(G, t1 - g); ++i, y += rows.stride) {
        if (g + i == s.end) begin_sequence(g + i);
        if (s.seq < 0) continue;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
          in[j][0] = win[j][0];
          in[j][1] = win[j][1];
        }
        load4(x + i * kConvD, in[W - 1]);
        F2 u[2];
        taps<W>(in, w, b, u);
        finish<kSilu>(u, unit_head, eps);
        store4(y, u);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
          win[j][0] = in[j + 1][0];
          win[j][1] = in[j + 1][1];
        }
      }
      __syncwarp();
      copy_group(slot, t1 - g - kRing);
    }
    slot = slot + G == kRing ? 0 : slot + G;
  }
  copy_wait<0>();
}

// One token a sequence: a warp a (sequence, head); the state moves on.
template <typename T, int W, bool kSilu>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(const ConvArgs a) {
  const int lane = threadIdx.x & 31;
  const int heads = 2 * a.h_qk + a.h_v, C = heads * kConvD;
  const unsigned task = blockIdx.x * kWarps + warp_index(), t = task / (unsigned)heads;
  const int head = (int)(task - t * heads), c = head * kConvD + 4 * lane;
  F2 w[W][2];
  grid_dependency_wait();
  grid_launch_dependents();
  if (t >= (unsigned)a.n_seqs) return;
  T* state = static_cast<T*>(a.final_state) + (int64_t)t * (W - 1) * C + c;
  Raw<T> raw[W];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) raw[j] = load_raw(state + (int64_t)j * C);
  raw[W - 1] = load_raw(static_cast<const T*>(a.x) + t * a.x_stride + c);
  load_taps<W>(a.weight, c, w);
  F2 in[W][2], u[2], b[2];
  load_bias(a.bias, c, b);
#pragma unroll
  for (int j = 0; j < W; ++j) unpack(raw[j], in[j]);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) *reinterpret_cast<Raw<T>*>(state + (int64_t)j * C) = raw[j + 1];
  taps<W>(in, w, b, u);
  finish<kSilu>(u, a.norm && head < 2 * a.h_qk, a.eps);
  const HeadRows<T> rows = head_rows<T>(a, head);
  store4(rows.p + t * rows.stride + 4 * lane, u);
}

// ---- backward ----
// Sum of tap j and channel c over group `group` of runs, in the workspace.
__device__ __forceinline__ float* conv_part(const ConvArgs& a, bool unit_head, int group, int j, int c) {
  const int64_t n_unit = (int64_t)a.n_unit * kConvD, others = (int64_t)(2 * a.h_qk + a.h_v) * kConvD - n_unit, rows = a.width + 1;
  return unit_head ? a.part + (group * rows + j) * n_unit + c
                   : a.part + a.runs[0] * rows * n_unit + (group * rows + j) * others + (c - n_unit);
}

// With g the gradient of a head's output, n = y r its unit vector:
//   dy = r (g - n sum(g n)),  du = dy (s + u s (1 - s)),  s = sigmoid(u),
//   dx_t = sum_j w_j du_{t + W - 1 - j},  dw_j = sum_t du_t x_{t - W + 1 + j}.
// A warp walks a run of tokens of one head, 4 channels a lane, and W - 1
// tokens past it, whose du belong to the run's last dx; `acc` holds the W - 1
// gradients that wait for later tokens.  The gradient before a sequence's
// first token is its state's.  With taps, their sums, inputs and waiting
// gradients of 4 channels in 128 registers, 16 warps fit an SM; issue slots are 57 %
// busy, the packed arithmetic's pipe 47 %.  A run
// length that makes two waves or more lost (84 to 99 us), and so did windows
// that turn in registers instead of being moved (83).
template <typename T, int W>
__device__ __forceinline__ void put_dx(const ConvArgs& a, const ConvSeq& s, int at, int t0, int t1, int c, int C,
                                       const F2 (&v)[2]) {
  if (at >= s.begin) {
    if (at >= t0 && at < t1) store4(static_cast<T*>(a.dx) + at * a.dx_stride + c, v);
  } else if (a.d_state && s.begin >= t0 && s.begin < t1) {
    store4(static_cast<T*>(a.d_state) + ((int64_t)s.seq * (W - 1) + (W - 1) + at - s.begin) * C + c, v);
  }
}

// The end of a sequence: nothing later adds to its last W - 1 gradients but
// those of its final state, which are its last inputs.
template <typename T, int W>
__device__ __forceinline__ void end_sequence(const ConvArgs& a, const ConvSeq& s, int t0, int t1, int c, int C,
                                             F2 (&acc)[W - 1][2]) {
  if (s.seq < 0) return;
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    if (a.d_final) {
      F2 f[2];
      load4(static_cast<const T*>(a.d_final) + ((int64_t)s.seq * (W - 1) + j) * C + c, f);
      acc[j][0] = add2(acc[j][0], f[0]);
      acc[j][1] = add2(acc[j][1], f[1]);
    }
    put_dx<T, W>(a, s, s.end - (W - 1) + j, t0, t1, c, C, acc[j]);
    acc[j][0] = acc[j][1] = f2(0.f);
  }
}

// du of a token from the gradient g of its output, in g, with y and the
// slope s + y (1 - s) of the activation.
template <bool kSilu>
__device__ __forceinline__ void slope_of(const F2 (&u)[2], F2 (&y)[2], F2 (&slope)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (kSilu) {
      const F2 sg = sigmoid(u[i]);
      y[i] = mul2(u[i], sg);
      slope[i] = fma2(y[i], fma2(sg, f2(-1.f), f2(1.f)), sg);
    } else {
      y[i] = u[i];
    }
  }
}
template <bool kSilu>
__device__ __forceinline__ void times_slope(F2 (&g)[2], const F2 (&slope)[2]) {
  if (kSilu) {
    g[0] = mul2(g[0], slope[0]);
    g[1] = mul2(g[1], slope[1]);
  }
}
// The gradients of the y of G tokens of a head from those of its unit vectors,
// in g: dy = r (g - y r^2 sum(g y)).  The same for each token whatever G is.
template <int G>
__device__ __forceinline__ void unit_back(F2 (&y)[G][2], F2 (&g)[G][2], float eps) {
  float v[2 * G];
#pragma unroll
  for (int i = 0; i < G; ++i) {
    v[i] = dot(y[i], y[i]);
    v[G + i] = dot(g[i], y[i]);
  }
  const float sum = group_sums<2 * G>(v);
  if (__any_sync(0xffffffffu, !(fabsf(sum) <= 3e38f))) {  // past fp32's range: of scaled y, one by one
#pragma unroll
    for (int i = 0; i < G; ++i) {
      float unit;
      const float r = unit_scale(y[i], eps, unit);
      y[i][0] = mul2(y[i][0], f2(r));
      y[i][1] = mul2(y[i][1], f2(r));
      const F2 m = f2(-warp_sum(dot(g[i], y[i])));
      const float root = unit == 1.f ? 1.f : 0x1p-34f;  // by halves: g r may leave fp32's range, and so may r unit
#pragma unroll
      for (int e = 0; e < 2; ++e) g[i][e] = mul2(mul2(fma2(y[i][e], m, g[i][e]), f2(r * root)), f2(root));
    }
    return;
  }
  const float r_mine = rsqrt_approx(sum + eps);  // of the lanes that hold a sum of squares
#pragma unroll
  for (int i = 0; i < G; ++i) {
    const float r = group_value<2 * G>(r_mine, i), m = -r * (r * group_value<2 * G>(sum, G + i));
#pragma unroll
    for (int e = 0; e < 2; ++e) g[i][e] = mul2(fma2(y[i][e], f2(m), g[i][e]), f2(r));
  }
}

template <typename T, int W, bool kSilu>
__global__ void __launch_bounds__(kThreads, 2) conv_bwd_kernel(const ConvArgs a) {
  // groups of 4 tokens, 2 of fp32, done 2 at a time (with more the registers run out); a ring of 3 groups
  constexpr int H = 2, G = sizeof(T) == 2 ? 4 : 2, kRowBytes = kConvD * sizeof(T), kRing = 3 * G;
  __shared__ union {
    alignas(16) char ring[kWarps][2 * kRing * kRowBytes];
    float sum[kWarps][W + 1][kConvD];
  } sh;
  const int lane = threadIdx.x & 31, warp = (int)warp_index();
  grid_dependency_wait();
  grid_launch_dependents();
  const int heads = 2 * a.h_qk + a.h_v, C = heads * kConvD;
  const ConvTask task = conv_task(a, blockIdx.x);
  const int head = task.head, c = head * kConvD + 4 * lane;
  F2 dw[W + 1][2];
#pragma unroll
  for (int j = 0; j <= W; ++j) dw[j][0] = dw[j][1] = f2(0.f);
  const int64_t first = ((int64_t)task.place * kWarps + warp) * task.run;
  if (first < a.T) {
    const int t0 = (int)first, t1 = (int)min((int64_t)a.T, first + task.run);
    const int stop = (int)min((int64_t)a.T, first + task.run + W - 1);  // tokens past the run, while its last sequence goes on
    const bool unit_head = task.unit_head;
    const float eps = a.eps;
    const int64_t dxs = a.dx_stride;
    const HeadRows<T> rows = head_rows<T>(a, head);
    // a token's row of x, then its row of g, in the ring; bf16: a half of the warp copies either, fp32: all lanes both
    char* ring = sh.ring[warp];
    constexpr int kLanes = kRowBytes / 16;
    const bool copies_g = kLanes == 16 && lane >= 16;
    const char* from_x = reinterpret_cast<const char*>(static_cast<const T*>(a.x) + t0 * a.x_stride + head * kConvD) + lane % kLanes * 16;
    const char* from_g = reinterpret_cast<const char*>(rows.p + t0 * rows.stride) + lane % kLanes * 16;
    const int64_t step_x = a.x_stride * (int64_t)sizeof(T), step_g = rows.stride * (int64_t)sizeof(T);
    const char* from = copies_g ? from_g : from_x;
    const int64_t step = copies_g ? step_g : step_x;
    int slot = 0;
    auto copy_group = [&](int at, int left) {  // left: tokens from the group on
      char* to = ring + at * 2 * kRowBytes + lane * 16;
#pragma unroll
      for (int i = 0; i < G; ++i) {
        if (left >= G || i < left) {
          copy16(to + i * 2 * kRowBytes, from);
          if (kLanes == 32) copy16(to + (i * 2 + 1) * kRowBytes, from_g);
        }
        from += step;
        if (kLanes == 32) from_g += step_g;
      }
      copy_commit();
    };
#pragma unroll
    for (int i = 0; i < kRing; i += G) copy_group(i, stop - t0 - i);
    T* dx = static_cast<T*>(a.dx) + (t0 - (W - 1)) * dxs + c;  // of the token whose gradient is whole after the group's first
    F2 w[W][2], b[2], win[W - 1][2], acc[W - 1][2];
    load_taps<W>(a.weight, c, w);
    load_bias(a.bias, c, b);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) acc[j][0] = acc[j][1] = f2(0.f);
    ConvSeq s = {-1, 0, t0};
    int straight = 0, from_t = 0;  // groups from `from_t` on that end by `straight` go through straight code
    auto begin_sequence = [&](int t) {
      s = conv_seq_after(a, s, t);
      load_window<T, W>(a, s, t, c, C, win);
      straight = s.seq >= 0 ? min(s.end, t1) : -1;
      from_t = max(s.begin, t0) + W - 1;
    };
    bool done = false;
    for (int g0 = t0; g0 < stop && !done; g0 += G) {
      copy_wait<kRing / G - 1>();
      __syncwarp();
      const T* x = reinterpret_cast<const T*>(ring + slot * 2 * kRowBytes) + 4 * lane;
      if (g0 + G <= straight && g0 >= from_t) {
#pragma unroll
        for (int h = 0; h < G; h += H) {
          F2 in[W - 1 + H][2], out[W - 1 + H][2], g[H][2], slope[H][2];
#pragma unroll
          for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              in[j][e] = win[j][e];
              out[j][e] = acc[j][e];
            }
          {
            F2 y[H][2];
#pragma unroll
            for (int i = 0; i < H; ++i) {
              F2 u[2];
              load4(x + 2 * (h + i) * kConvD, in[W - 1 + i]);
              load4(x + (2 * (h + i) + 1) * kConvD, g[i]);
              taps<W>(in + i, w, b, u);
              slope_of<kSilu>(u, y[i], slope[i]);
            }
            if (unit_head) unit_back<H>(y, g, eps);
          }
#pragma unroll
          for (int i = 0; i < H; ++i) {
            times_slope<kSilu>(g[i], slope[i]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
              for (int j = 0; j < W; ++j) {
                out[i + j][e] = j < W - 1 ? fma2(w[j][e], g[i][e], out[i + j][e]) : mul2(w[j][e], g[i][e]);
                dw[j][e] = fma2(g[i][e], in[i + j][e], dw[j][e]);
              }
              dw[W][e] = add2(dw[W][e], g[i][e]);
            }
            store4(dx, out[i]);
            dx += dxs;
          }
#pragma unroll
          for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              win[j][e] = in[H + j][e];
              acc[j][e] = out[H + j][e];
            }
        }
      } else {
        dx += G * dxs;
#pragma unroll 1
        for (int i = 0; i < min(G, stop - g0); ++i) {
          const int t = g0 + i;
          if (t == s.end) {
            end_sequence<T, W>(a, s, t0, t1, c, C, acc);
            if (t >= t1) {
              done = true;
              break;
            }
            begin_sequence(t);
          }
          if (s.seq < 0) continue;
          F2 in[W][2];
#pragma unroll
          for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) in[j][e] = win[j][e];
          load4(x + 2 * i * kConvD, in[W - 1]);
          F2 u[2], one[1][2], y[1][2], slope[2], d[W][2];
          F2(&g)[2] = one[0];
          taps<W>(in, w, b, u);
          load4(x + (2 * i + 1) * kConvD, g);
          slope_of<kSilu>(u, y[0], slope);
          if (unit_head) unit_back<1>(y, one, eps);
          times_slope<kSilu>(g, slope);
          const bool own = t < t1;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int j = 0; j < W; ++j) {
              d[j][e] = j < W - 1 ? fma2(w[j][e], g[e], acc[j][e]) : mul2(w[j][e], g[e]);
              if (own) dw[j][e] = fma2(g[e], in[j][e], dw[j][e]);
            }
            if (own) dw[W][e] = add2(dw[W][e], g[e]);
          }
          put_dx<T, W>(a, s, t - (W - 1), t0, t1, c, C, d[0]);
#pragma unroll
          for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              win[j][e] = in[j + 1][e];
              acc[j][e] = d[j + 1][e];
            }
        }
      }
      __syncwarp();
      copy_group(slot, stop - g0 - kRing);
      slot = slot + G == kRing ? 0 : slot + G;
    }
    if (!done && stop == s.end) end_sequence<T, W>(a, s, t0, t1, c, C, acc);
    copy_wait<0>();
  }
  if (!a.sums) return;
  __syncthreads();  // the rings are done with
#pragma unroll
  for (int j = 0; j <= W; ++j) {
    const float2 p = parts(dw[j][0]), q = parts(dw[j][1]);
    *reinterpret_cast<float4*>(&sh.sum[warp][j][4 * lane]) = make_float4(p.x, p.y, q.x, q.y);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < (W + 1) * kConvD; i += kThreads) {
    const int j = i / kConvD, at = i % kConvD;
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) v += sh.sum[k][j][at];
    *conv_part(a, task.unit_head, task.place, j, c - 4 * lane + at) = v;
  }
}

// The CTAs' sums to one, in a fixed order, 32 channels of a tap a CTA; and the
// state gradients of sequences without tokens, which are their final state's.
template <typename T>
__global__ void __launch_bounds__(1024) conv_bwd_sum_kernel(const ConvArgs a) {
  __shared__ float2 sum[32][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int W = a.width, C = (2 * a.h_qk + a.h_v) * kConvD;
  grid_dependency_wait();
  grid_launch_dependents();
  const int blocks = a.sums ? (W + 1) * (C / 32) : 0;
  if ((int)blockIdx.x >= blocks) {
    const int64_t seq = ((int64_t)blockIdx.x - blocks) * 32 + warp;  // a warp a sequence
    if (seq >= a.n_seqs || (a.cu ? a.cu[seq + 1] > a.cu[seq] : a.n_each > 0)) return;
    const int64_t n = (int64_t)(W - 1) * C;
    for (int64_t i = 4 * lane; i < n; i += 4 * 32) {
      Raw<T> v = {};
      if (a.d_final) v = load_raw(static_cast<const T*>(a.d_final) + seq * n + i);
      *reinterpret_cast<Raw<T>*>(static_cast<T*>(a.d_state) + seq * n + i) = v;
    }
    return;
  }
  const int j = blockIdx.x % (W + 1), at = (int)(blockIdx.x / (W + 1)) * 32 + lane;
  if (j == W && !a.d_bias) return;
  if (j < W && !a.d_weight) return;
  const bool unit_head = at < a.n_unit * kConvD;
  const int groups = a.runs[unit_head ? 0 : 1];
  const float* part = conv_part(a, unit_head, 0, j, at);
  const int64_t step = conv_part(a, unit_head, 1, j, at) - part;
  Sum2 v;
#pragma unroll 8
  for (int i = warp; i < groups; i += 32) v.add(part[i * step]);
  sum[warp][lane] = make_float2(v.hi, v.lo);
  __syncthreads();
  if (warp == 0) {
    v = {};
#pragma unroll
    for (int i = 0; i < 32; ++i) v.add({sum[i][lane].x, sum[i][lane].y});
    if (j == W) a.d_bias[at] = v.value();
    else a.d_weight[(int64_t)at * W + j] = v.value();
  }
}

// f(type, taps, activation) of a call.
template <typename F>
cudaError_t by_kind(const ConvArgs& a, bool f32, F&& f) {
  auto width = [&](auto type, auto silu) {
    return a.width == 2   ? f(type, std::integral_constant<int, 2>(), silu)
           : a.width == 3 ? f(type, std::integral_constant<int, 3>(), silu)
                          : f(type, std::integral_constant<int, 4>(), silu);
  };
  auto activation = [&](auto type) { return a.silu ? width(type, std::true_type()) : width(type, std::false_type()); };
  return f32 ? activation(float()) : activation(__nv_bfloat16());
}

}  // namespace

cudaError_t launch_conv(const ConvArgs& args, bool f32, cudaStream_t st) {
  ConvArgs a = args;
  const int64_t heads = 2 * a.h_qk + a.h_v, tasks = (int64_t)a.n_unit * a.runs[0] + (heads - a.n_unit) * a.runs[1];
  a.blocks = (int)((tasks + kWarps - 1) / kWarps);
  int64_t blocks = a.blocks;
  if (a.final_state) blocks += ((int64_t)a.n_seqs * heads + kWarps - 1) / kWarps;
  if (blocks == 0) return cudaSuccess;
  return by_kind(a, f32, [&](auto type, auto w, auto silu) {
    return launch_kernel(conv_kernel<decltype(type), decltype(w)::value, decltype(silu)::value>, dim3((unsigned)blocks),
                         dim3(kThreads), 0, st, true, a);
  });
}

cudaError_t launch_conv_step(const ConvArgs& a, bool f32, cudaStream_t st) {
  const int64_t blocks = ((int64_t)a.n_seqs * (2 * a.h_qk + a.h_v) + kWarps - 1) / kWarps;
  return by_kind(a, f32, [&](auto type, auto w, auto silu) {
    return launch_kernel(conv_step_kernel<decltype(type), decltype(w)::value, decltype(silu)::value>, dim3((unsigned)blocks),
                         dim3(kThreads), 0, st, true, a);
  });
}

cudaError_t launch_conv_bwd(const ConvArgs& a, bool f32, cudaStream_t st) {
  const int64_t blocks = (int64_t)a.n_unit * a.runs[0] + (int64_t)(2 * a.h_qk + a.h_v - a.n_unit) * a.runs[1];
  return by_kind(a, f32, [&](auto type, auto w, auto silu) {
    return launch_kernel(conv_bwd_kernel<decltype(type), decltype(w)::value, decltype(silu)::value>, dim3((unsigned)blocks),
                         dim3(kThreads), 0, st, true, a);
  });
}

cudaError_t launch_conv_bwd_sums(const ConvArgs& a, bool f32, cudaStream_t st) {
  const int64_t C = (int64_t)(2 * a.h_qk + a.h_v) * kConvD;
  int64_t blocks = a.sums ? (a.width + 1) * (C / 32) : 0;
  if (a.d_state) blocks += ((int64_t)a.n_seqs + 31) / 32;
  if (blocks == 0) return cudaSuccess;
  return f32 ? launch_kernel(conv_bwd_sum_kernel<float>, dim3((unsigned)blocks), dim3(1024), 0, st, true, a)
             : launch_kernel(conv_bwd_sum_kernel<__nv_bfloat16>, dim3((unsigned)blocks), dim3(1024), 0, st, true, a);
}

}  // namespace gdn
