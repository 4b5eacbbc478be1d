// The short causal convolution before the gated delta rule: per channel c of
// the projection and token t of a sequence, with taps w and kept inputs before
// the sequence's first token,
//   u_t = b + sum_{j < W} w_j x_{t - W + 1 + j},   y = u sigmoid(u)  (or u),
// heads of 128 channels, q's, then k's, then v's; those of q and k scaled to
// unit length, y / sqrt(sum y^2 + eps).  And its gradients, and its form for
// one new token of each sequence.
//
// All of it moves each element once and is bound by that.  A group of lanes
// owns a head's channels over a run of tokens and keeps the last W - 1 inputs
// in registers, so an input is read once but for the W - 1 before each run.
#include <type_traits>

#include "gdn_conv.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kGroups = kThreads / 16;

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

// ---- N elements of a lane, N consecutive channels ----
template <typename T, int N>
struct Raw {
  uint32_t w[N * sizeof(T) / 4];
};
template <typename T, int N>
__device__ __forceinline__ Raw<T, N> load_raw(const void* p) {
  Raw<T, N> r;
  if constexpr (N * sizeof(T) == 8) {
    const uint2 v = *static_cast<const uint2*>(p);
    r.w[0] = v.x; r.w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < (int)(N * sizeof(T) / 16); ++i) {
      const uint4 v = static_cast<const uint4*>(p)[i];
      r.w[4 * i] = v.x; r.w[4 * i + 1] = v.y; r.w[4 * i + 2] = v.z; r.w[4 * i + 3] = v.w;
    }
  }
  return r;
}
template <typename T, int N>
__device__ __forceinline__ void store_raw(void* p, const Raw<T, N>& r) {
  if constexpr (N * sizeof(T) == 8) {
    *static_cast<uint2*>(p) = make_uint2(r.w[0], r.w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < (int)(N * sizeof(T) / 16); ++i)
      static_cast<uint4*>(p)[i] = make_uint4(r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]);
  }
}
template <typename T, int N>
__device__ __forceinline__ void unpack(const Raw<T, N>& r, float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < (int)(N * sizeof(T) / 4); ++i) {
    if constexpr (sizeof(T) == 4) {
      x[i] = __uint_as_float(r.w[i]);
    } else {
      x[2 * i] = __uint_as_float(r.w[i] << 16);
      x[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
    }
  }
}
template <typename T, int N>
__device__ __forceinline__ Raw<T, N> pack(const float (&x)[N]) {
  Raw<T, N> r;
#pragma unroll
  for (int i = 0; i < (int)(N * sizeof(T) / 4); ++i) {
    if constexpr (sizeof(T) == 4) r.w[i] = __float_as_uint(x[i]);
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r.w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
  }
  return r;
}
template <typename T, int N>
__device__ __forceinline__ void load_f32(const T* p, float (&x)[N]) {
  unpack<T, N>(load_raw<T, N>(p), x);
}

__device__ __forceinline__ float sigmoid(float u) { return __fdividef(1.f, 1.f + __expf(-u)); }

template <int kLanes>
__device__ __forceinline__ float group_sum(float v, unsigned mask) {
#pragma unroll
  for (int d = kLanes / 2; d; d >>= 1) v += __shfl_xor_sync(mask, v, d);
  return v;
}
template <int N>
__device__ __forceinline__ float dot(const float (&x)[N], const float (&y)[N]) {
  float a = 0.f, b = 0.f;
#pragma unroll
  for (int e = 0; e < N; e += 2) {
    a = fmaf(x[e], y[e], a);
    b = fmaf(x[e + 1], y[e + 1], b);
  }
  return a + b;
}
// 1 / sqrt(sum y^2 + eps) of a head; past fp32's range y is scaled by 2^-68
// (unit), beside which eps is nothing, and the result belongs to the scaled y.
template <int kLanes, int N>
__device__ __forceinline__ float unit_scale(float (&y)[N], float eps, unsigned mask, float& unit) {
  const float ss = group_sum<kLanes>(dot(y, y), mask);
  unit = 1.f;
  if (ss <= 3e38f) return rsqrtf(ss + eps);
  unit = 0x1p-68f;
#pragma unroll
  for (int e = 0; e < N; ++e) y[e] *= unit;
  return rsqrtf(group_sum<kLanes>(dot(y, y), mask));
}

// A lane's taps, channel by channel as they are in memory, by tap.
template <int W, int N>
__device__ __forceinline__ void load_taps(const float* weight, int c, float (&w)[W][N]) {
  const float4* p = reinterpret_cast<const float4*>(weight + (int64_t)c * W);
  float f[W * N];
#pragma unroll
  for (int i = 0; i < W * N / 4; ++i) {
    const float4 v = __ldg(p + i);
    f[4 * i] = v.x; f[4 * i + 1] = v.y; f[4 * i + 2] = v.z; f[4 * i + 3] = v.w;
  }
#pragma unroll
  for (int e = 0; e < N; ++e)
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][e] = f[e * W + j];
}

// The output row of a head: q, k or v.
template <typename T>
__device__ __forceinline__ T* head_row(const ConvArgs& a, int head, int64_t t) {
  if (head < a.h_qk) return static_cast<T*>(a.q) + (t * a.h_qk + head) * kConvD;
  if (head < 2 * a.h_qk) return static_cast<T*>(a.k) + (t * a.h_qk + head - a.h_qk) * kConvD;
  return static_cast<T*>(a.v) + (t * a.h_v + head - 2 * a.h_qk) * kConvD;
}

// The W - 1 inputs before token t: earlier tokens, then the kept state.
template <typename T, int W, int N>
__device__ __forceinline__ void load_window(const ConvArgs& a, const ConvSeq& s, int t, int c, int C, float (&win)[W][N]) {
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    const int at = t - (W - 1) + j;
    if (at >= s.begin) {
      load_f32<T, N>(static_cast<const T*>(a.x) + at * a.x_stride + c, win[j]);
    } else if (a.state && s.seq >= 0) {
      load_f32<T, N>(static_cast<const T*>(a.state) + ((int64_t)s.seq * (W - 1) + (W - 1) + at - s.begin) * C + c, win[j]);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) win[j][e] = 0.f;
    }
  }
}

// y of one token from its window; the window moves on.
template <int W, int N>
__device__ __forceinline__ void taps(const float (&win)[W][N], const float (&w)[W][N], const float (&b)[N], float (&u)[N]) {
#pragma unroll
  for (int e = 0; e < N; ++e) {
    float v = b[e];
#pragma unroll
    for (int j = 0; j < W; ++j) v = fmaf(w[j][e], win[j][e], v);
    u[e] = v;
  }
}
template <int W, int N>
__device__ __forceinline__ void shift(float (&win)[W][N]) {
#pragma unroll
  for (int j = 0; j < W - 1; ++j)
#pragma unroll
    for (int e = 0; e < N; ++e) win[j][e] = win[j + 1][e];
}

// Element i of the states after the call: row r of sequence s is the padded
// row len + r of (state, tokens).
template <typename T>
__device__ __forceinline__ void final_states(const ConvArgs& a, int64_t i, int C) {
  const int W1 = a.width - 1;
  const int64_t row = i / (C / 8);
  const int c = (int)(i % (C / 8)) * 8;
  if (row >= (int64_t)a.n_seqs * W1) return;
  const int seq = (int)(row / W1), r = (int)(row % W1);
  int begin = 0, end = 0;
  if (a.cu) {
    begin = min(max(a.cu[seq], 0), a.T);
    end = min(max(a.cu[seq + 1], begin), a.T);
  } else {
    begin = seq * a.n_each;
    end = begin + a.n_each;
  }
  const int at = end - W1 + r;
  Raw<T, 8> v;
  if (at >= begin) {
    v = load_raw<T, 8>(static_cast<const T*>(a.x) + at * a.x_stride + c);
  } else if (a.state) {
    v = load_raw<T, 8>(static_cast<const T*>(a.state) + ((int64_t)seq * W1 + W1 + at - begin) * C + c);
  } else {
#pragma unroll
    for (auto& w : v.w) w = 0;
  }
  store_raw<T, 8>(static_cast<T*>(a.final_state) + row * C + c, v);
}

// A half-warp a (run, head), 8 channels a lane; then CTAs for the final states.
template <typename T, int W>
__global__ void __launch_bounds__(kThreads) conv_kernel(const ConvArgs a) {
  constexpr int N = 8, kAhead = 4;
  const int lane = threadIdx.x & 15;
  const unsigned mask = 0xffffu << (threadIdx.x & 16);
  grid_dependency_wait();
  grid_launch_dependents();
  const int heads = 2 * a.h_qk + a.h_v, C = heads * kConvD;
  const int64_t runs = ((int64_t)a.T + a.run - 1) / a.run, tasks = runs * heads;
  const int64_t blocks = (tasks + kGroups - 1) / kGroups;
  if (blockIdx.x >= blocks) {
    final_states<T>(a, (blockIdx.x - blocks) * kThreads + threadIdx.x, C);
    return;
  }
  const int64_t task = (int64_t)blockIdx.x * kGroups + (threadIdx.x >> 4);
  if (task >= tasks) return;
  const int head = (int)(task % heads), c = head * kConvD + lane * N;
  const int t0 = (int)(task / heads) * a.run, t1 = (int)min((int64_t)a.T, (int64_t)t0 + a.run);
  float w[W][N], b[N] = {}, win[W][N];
  load_taps<W, N>(a.weight, c, w);
  if (a.bias) load_f32<float, N>(a.bias + c, b);
  ConvSeq s = conv_seq(a, t0);
  load_window<T, W, N>(a, s, t0, c, C, win);
  const bool unit_heads = a.norm && head < 2 * a.h_qk;
  const T* x = static_cast<const T*>(a.x) + c;
  for (int g = t0; g < t1; g += kAhead) {
    Raw<T, N> raw[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (g + i < t1) raw[i] = load_raw<T, N>(x + (g + i) * a.x_stride);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int t = g + i;
      if (t >= t1) break;
      if (t == s.end) {
        s = conv_seq(a, t);
        load_window<T, W, N>(a, s, t, c, C, win);
      }
      if (s.seq < 0) continue;
      unpack<T, N>(raw[i], win[W - 1]);
      float y[N];
      taps<W, N>(win, w, b, y);
      shift<W, N>(win);
      if (a.silu) {
#pragma unroll
        for (int e = 0; e < N; ++e) y[e] *= sigmoid(y[e]);
      }
      if (unit_heads) {
        float unit;
        const float r = unit_scale<16, N>(y, a.eps, mask, unit);
#pragma unroll
        for (int e = 0; e < N; ++e) y[e] *= r;
      }
      store_raw<T, N>(head_row<T>(a, head, t) + lane * N, pack<T, N>(y));
    }
  }
}

// One token a sequence: a half-warp a (sequence, head); the state moves on.
template <typename T, int W>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(const ConvArgs a) {
  constexpr int N = 8;
  const int lane = threadIdx.x & 15;
  const unsigned mask = 0xffffu << (threadIdx.x & 16);
  const int heads = 2 * a.h_qk + a.h_v, C = heads * kConvD;
  const int64_t task = (int64_t)blockIdx.x * kGroups + (threadIdx.x >> 4);
  grid_dependency_wait();
  grid_launch_dependents();
  if (task >= (int64_t)a.n_seqs * heads) return;
  const int head = (int)(task % heads), c = head * kConvD + lane * N, t = (int)(task / heads);
  T* state = static_cast<T*>(a.final_state) + (int64_t)t * (W - 1) * C + c;
  Raw<T, N> raw[W];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) raw[j] = load_raw<T, N>(state + (int64_t)j * C);
  raw[W - 1] = load_raw<T, N>(static_cast<const T*>(a.x) + t * a.x_stride + c);
  float w[W][N], b[N] = {}, win[W][N], y[N];
  load_taps<W, N>(a.weight, c, w);
  if (a.bias) load_f32<float, N>(a.bias + c, b);
#pragma unroll
  for (int j = 0; j < W; ++j) unpack<T, N>(raw[j], win[j]);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) store_raw<T, N>(state + (int64_t)j * C, raw[j + 1]);
  taps<W, N>(win, w, b, y);
  if (a.silu) {
#pragma unroll
    for (int e = 0; e < N; ++e) y[e] *= sigmoid(y[e]);
  }
  if (a.norm && head < 2 * a.h_qk) {
    float unit;
    const float r = unit_scale<16, N>(y, a.eps, mask, unit);
#pragma unroll
    for (int e = 0; e < N; ++e) y[e] *= r;
  }
  store_raw<T, N>(head_row<T>(a, head, t) + lane * N, pack<T, N>(y));
}

// ---- backward ----
// With g the gradient of a head's output, n = y r its unit vector:
//   dy = r (g - n sum(g n)),  du = dy (s + u s (1 - s)),  s = sigmoid(u),
//   dx_t = sum_j w_j du_{t + W - 1 - j},  dw_j = sum_t du_t x_{t - W + 1 + j}.
// A warp walks a run of tokens of one head, 4 channels a lane, and W - 1
// tokens past it, whose du belong to the run's last dx; `acc` holds the W - 1
// gradients that wait for later tokens.  The gradient before a sequence's
// first token is its state's.
constexpr int kWarps = kThreads / 32;

template <typename T, int W, int N>
__device__ __forceinline__ void put_dx(const ConvArgs& a, const ConvSeq& s, int at, int t0, int t1, int c, int C,
                                       const float (&v)[N]) {
  if (at >= s.begin) {
    if (at >= t0 && at < t1) store_raw<T, N>(static_cast<T*>(a.dx) + at * a.dx_stride + c, pack<T, N>(v));
  } else if (a.d_state && s.begin >= t0 && s.begin < t1) {
    store_raw<T, N>(static_cast<T*>(a.d_state) + ((int64_t)s.seq * (W - 1) + (W - 1) + at - s.begin) * C + c, pack<T, N>(v));
  }
}

// The end of a sequence: nothing later adds to its last W - 1 gradients but
// those of its final state, which are its last inputs.
template <typename T, int W, int N>
__device__ __forceinline__ void end_sequence(const ConvArgs& a, const ConvSeq& s, int t0, int t1, int c, int C,
                                             float (&acc)[W][N]) {
  if (s.seq < 0) return;
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    if (a.d_final) {
      float f[N];
      load_f32<T, N>(static_cast<const T*>(a.d_final) + ((int64_t)s.seq * (W - 1) + j) * C + c, f);
#pragma unroll
      for (int e = 0; e < N; ++e) acc[j][e] += f[e];
    }
    put_dx<T, W, N>(a, s, s.end - (W - 1) + j, t0, t1, c, C, acc[j]);
  }
#pragma unroll
  for (int j = 0; j < W; ++j)
#pragma unroll
    for (int e = 0; e < N; ++e) acc[j][e] = 0.f;
}

template <typename T, int W>
__global__ void __launch_bounds__(kThreads) conv_bwd_kernel(const ConvArgs a) {
  constexpr int N = 4, kAhead = 4;
  __shared__ float sum[kWarps][W + 1][kConvD];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr unsigned mask = 0xffffffffu;
  grid_dependency_wait();
  grid_launch_dependents();
  const int heads = 2 * a.h_qk + a.h_v, C = heads * kConvD;
  const int head = (int)(blockIdx.x % (unsigned)heads), group = (int)(blockIdx.x / (unsigned)heads);
  const int c = head * kConvD + lane * N;
  float dw[W + 1][N] = {};
  const int64_t first = ((int64_t)group * kWarps + warp) * a.run;
  if (first < a.T) {
    const int t0 = (int)first, t1 = (int)min((int64_t)a.T, first + a.run);
    float w[W][N], b[N] = {}, win[W][N], acc[W][N] = {};
    load_taps<W, N>(a.weight, c, w);
    if (a.bias) load_f32<float, N>(a.bias + c, b);
    ConvSeq s = conv_seq(a, t0);
    load_window<T, W, N>(a, s, t0, c, C, win);
    const bool unit_heads = a.norm && head < 2 * a.h_qk;
    const T* x = static_cast<const T*>(a.x) + c;
    // tokens past the run belong to it while its last sequence goes on
    const int stop = min(t1 + W - 1, a.T);
    bool done = false;
    for (int g0 = t0; g0 < stop && !done; g0 += kAhead) {
      Raw<T, N> rx[kAhead], rg[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (g0 + i < stop) {
          rx[i] = load_raw<T, N>(x + (g0 + i) * a.x_stride);
          rg[i] = load_raw<T, N>(head_row<T>(a, head, g0 + i) + lane * N);
        }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int t = g0 + i;
        if (t >= stop) break;
        if (t == s.end) {
          end_sequence<T, W, N>(a, s, t0, t1, c, C, acc);
          if (t >= t1) {
            done = true;
            break;
          }
          s = conv_seq(a, t);
          load_window<T, W, N>(a, s, t, c, C, win);
        }
        if (s.seq < 0) continue;
        unpack<T, N>(rx[i], win[W - 1]);
        float u[N], sg[N], y[N], g[N];
        taps<W, N>(win, w, b, u);
        unpack<T, N>(rg[i], g);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          sg[e] = a.silu ? sigmoid(u[e]) : 1.f;
          y[e] = u[e] * sg[e];
        }
        if (unit_heads) {
          float ys[N], unit;
#pragma unroll
          for (int e = 0; e < N; ++e) ys[e] = y[e];
          const float r = unit_scale<32, N>(ys, a.eps, mask, unit);
#pragma unroll
          for (int e = 0; e < N; ++e) ys[e] *= r;
          const float gn = group_sum<32>(dot(g, ys), mask);
#pragma unroll
          for (int e = 0; e < N; ++e) g[e] = r * (g[e] - ys[e] * gn) * unit;
        }
        if (a.silu) {
#pragma unroll
          for (int e = 0; e < N; ++e) g[e] *= sg[e] + y[e] * (1.f - sg[e]);
        }
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
          for (int e = 0; e < N; ++e) acc[j][e] = fmaf(w[j][e], g[e], acc[j][e]);
        if (t < t1) {
#pragma unroll
          for (int j = 0; j < W; ++j)
#pragma unroll
            for (int e = 0; e < N; ++e) dw[j][e] = fmaf(g[e], win[j][e], dw[j][e]);
#pragma unroll
          for (int e = 0; e < N; ++e) dw[W][e] += g[e];
        }
        put_dx<T, W, N>(a, s, t - (W - 1), t0, t1, c, C, acc[0]);
        shift<W, N>(acc);
#pragma unroll
        for (int e = 0; e < N; ++e) acc[W - 1][e] = 0.f;
        shift<W, N>(win);
      }
    }
    if (!done && stop == s.end) end_sequence<T, W, N>(a, s, t0, t1, c, C, acc);
  }
  if (!a.sums) return;
#pragma unroll
  for (int j = 0; j <= W; ++j)
#pragma unroll
    for (int e = 0; e < N; ++e) sum[warp][j][lane * N + e] = dw[j][e];
  __syncthreads();
  for (int i = threadIdx.x; i < (W + 1) * kConvD; i += kThreads) {
    const int j = i / kConvD, at = i % kConvD;
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) v += sum[k][j][at];
    a.part[((int64_t)group * (W + 1) + j) * C + head * kConvD + at] = v;
  }
}

// The CTAs' sums to one, in a fixed order, 32 channels of a tap a CTA; and the
// state gradients of sequences without tokens, which are their final state's.
template <typename T>
__global__ void __launch_bounds__(1024) conv_bwd_sum_kernel(const ConvArgs a) {
  __shared__ double sum[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int W = a.width, C = (2 * a.h_qk + a.h_v) * kConvD;
  grid_dependency_wait();
  grid_launch_dependents();
  const int blocks = a.sums ? (W + 1) * (C / 32) : 0;
  if ((int)blockIdx.x >= blocks) {
    const int64_t i = ((int64_t)blockIdx.x - blocks) * 1024 + threadIdx.x;
    const int64_t row = i / (C / 8);
    const int c = (int)(i % (C / 8)) * 8;
    if (row >= (int64_t)a.n_seqs * (W - 1)) return;
    const int seq = (int)(row / (W - 1));
    const bool empty = a.cu ? a.cu[seq + 1] <= a.cu[seq] : a.n_each == 0;
    if (!empty) return;
    Raw<T, 8> v;
#pragma unroll
    for (auto& w : v.w) w = 0;
    if (a.d_final) v = load_raw<T, 8>(static_cast<const T*>(a.d_final) + row * C + c);
    store_raw<T, 8>(static_cast<T*>(a.d_state) + row * C + c, v);
    return;
  }
  const int j = blockIdx.x % (W + 1), at = (int)(blockIdx.x / (W + 1)) * 32 + lane;
  if (j == W && !a.d_bias) return;
  if (j < W && !a.d_weight) return;
  double v = 0.0;
#pragma unroll 8
  for (int i = warp; i < a.groups; i += 32) v += a.part[((int64_t)i * (W + 1) + j) * C + at];
  sum[warp][lane] = v;
  __syncthreads();
  if (warp == 0) {
    v = 0.0;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += sum[i][lane];
    if (j == W) a.d_bias[at] = (float)v;
    else a.d_weight[(int64_t)at * W + j] = (float)v;
  }
}

template <typename F>
cudaError_t by_width(int width, F&& f) {
  return width == 2 ? f(std::integral_constant<int, 2>()) : width == 3 ? f(std::integral_constant<int, 3>())
                                                                       : f(std::integral_constant<int, 4>());
}

}  // namespace

cudaError_t launch_conv(const ConvArgs& a, bool f32, cudaStream_t st) {
  const int64_t heads = 2 * a.h_qk + a.h_v, runs = ((int64_t)a.T + a.run - 1) / a.run;
  int64_t blocks = (runs * heads + kGroups - 1) / kGroups;
  if (a.final_state) blocks += ((int64_t)a.n_seqs * (a.width - 1) * heads * 16 + kThreads - 1) / kThreads;
  if (blocks == 0) return cudaSuccess;
  return by_width(a.width, [&](auto w) {
    return f32 ? launch_kernel(conv_kernel<float, decltype(w)::value>, dim3((unsigned)blocks), dim3(kThreads), 0, st, true, a)
               : launch_kernel(conv_kernel<__nv_bfloat16, decltype(w)::value>, dim3((unsigned)blocks), dim3(kThreads), 0, st, true, a);
  });
}

cudaError_t launch_conv_step(const ConvArgs& a, bool f32, cudaStream_t st) {
  const int64_t blocks = ((int64_t)a.n_seqs * (2 * a.h_qk + a.h_v) + kGroups - 1) / kGroups;
  return by_width(a.width, [&](auto w) {
    return f32 ? launch_kernel(conv_step_kernel<float, decltype(w)::value>, dim3((unsigned)blocks), dim3(kThreads), 0, st, true, a)
               : launch_kernel(conv_step_kernel<__nv_bfloat16, decltype(w)::value>, dim3((unsigned)blocks), dim3(kThreads), 0, st, true, a);
  });
}

cudaError_t launch_conv_bwd(const ConvArgs& a, bool f32, cudaStream_t st) {
  const int64_t blocks = (int64_t)a.groups * (2 * a.h_qk + a.h_v);
  return by_width(a.width, [&](auto w) {
    return f32 ? launch_kernel(conv_bwd_kernel<float, decltype(w)::value>, dim3((unsigned)blocks), dim3(kThreads), 0, st, true, a)
               : launch_kernel(conv_bwd_kernel<__nv_bfloat16, decltype(w)::value>, dim3((unsigned)blocks), dim3(kThreads), 0, st, true, a);
  });
}

cudaError_t launch_conv_bwd_sums(const ConvArgs& a, bool f32, cudaStream_t st) {
  const int64_t C = (int64_t)(2 * a.h_qk + a.h_v) * kConvD;
  int64_t blocks = a.sums ? (a.width + 1) * (C / 32) : 0;
  if (a.d_state) blocks += ((int64_t)a.n_seqs * (a.width - 1) * (C / 8) + 1023) / 1024;
  if (blocks == 0) return cudaSuccess;
  return f32 ? launch_kernel(conv_bwd_sum_kernel<float>, dim3((unsigned)blocks), dim3(1024), 0, st, true, a)
             : launch_kernel(conv_bwd_sum_kernel<__nv_bfloat16>, dim3((unsigned)blocks), dim3(1024), 0, st, true, a);
}

}  // namespace gdn
