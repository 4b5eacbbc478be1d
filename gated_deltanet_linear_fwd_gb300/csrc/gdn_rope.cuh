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
// one, and that product is exact for every 32-bit position.  What is off is the
// table (fp64 frequencies to a few of 2^-53 of themselves, to 2^-65 turns: 2^-34
// turns at position 2^31) and the cut to the top 32 bits (2^-32 turns): less
// than fp32 can hold of a cosine.  A product in fp32 would be off by 2^-24 of
// hundreds of thousands of radians at far positions.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>

#include "gdn_internal.cuh"
#include "gdn_pair.cuh"
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

// Where a packed token stands: given, counted from its sequence's start or its
// row's, or, the tokens being the last of lens[i], in the cache.
struct PosArgs {
  const int32_t* positions;  // [T] or null
  const int32_t* cu;         // [n_seqs + 1] or null
  const int32_t* lens;       // [n_seqs] or null
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
// The sequence of the last token asked for: token t of it is at t - shift.
struct TokenSeq {
  int begin = 0, end = 0, shift = 0;
};
// False for a token outside every sequence.  Searches only where s is not the token's.
__device__ __forceinline__ bool token_position(const PosArgs& a, int t, TokenSeq& s, int& pos) {
  if (a.positions) {
    pos = a.positions[t];
    return true;
  }
  if (t < s.begin || t >= s.end) {
    int seq;
    if (a.cu) {
      seq = seq_of(a.cu, a.n_seqs, t);
      s.begin = a.cu[seq];
      s.end = a.cu[seq + 1];
    } else {
      seq = t / a.n_each;
      s.begin = seq * a.n_each;
      s.end = s.begin + a.n_each;
    }
    s.shift = a.lens ? (int)((unsigned)s.end - (unsigned)a.lens[seq]) : s.begin;
  }
  pos = (int)((unsigned)t - (unsigned)s.shift);
  return t >= s.begin && t < s.end;
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

// Cos and sin of two angles of phase / 2^32 turns.  The nearest quarter turn
// comes off in integers; what remains, u halves of a quarter turn, |u| <= 1,
// goes into polynomials of u^2 whose coefficients are the minimax ones on [0, 1]
// (Remez's exchange): u A(u^2) for sin(pi u / 4) and B(u^2) for cos.  With the
// coefficients rounded to fp32 and as computed here, all u on a grid of 2^-22: sine
// to 2^-22.9 and cosine to 2^-23.5 of themselves, within 2 ulp.  Some 25
// instructions an angle; with sincospif an angle took 94, a fifth of the forward's.
__device__ __forceinline__ void sincos_turns(uint32_t p0, uint32_t p1, F2& c, F2& s) {
  const uint32_t q0 = (p0 + 0x20000000u) >> 30, q1 = (p1 + 0x20000000u) >> 30;
  const F2 u = mul2(f2((float)(int32_t)(p0 - (q0 << 30)), (float)(int32_t)(p1 - (q1 << 30))), f2(0x1p-29f)), v = mul2(u, u);
  const F2 sn = mul2(u, fma2(v, fma2(v, fma2(v, f2(-3.5950452e-5f), f2(2.4900010e-3f)), f2(-8.0745433e-2f)), f2(7.8539816e-1f)));
  const F2 cs = fma2(
      v, fma2(v, fma2(v, fma2(v, f2(3.5298113e-6f), f2(-3.2593861e-4f)), f2(1.5854325e-2f)), f2(-3.0842514e-1f)), f2(1.0f));
  const float2 a = parts(sn), b = parts(cs);
  auto sign = [](float x, uint32_t q) { return __uint_as_float(__float_as_uint(x) ^ (q << 30 & 0x80000000u)); };
  s = f2(sign(q0 & 1 ? b.x : a.x, q0), sign(q1 & 1 ? b.y : a.y, q1));
  c = f2(sign(q0 & 1 ? a.x : b.x, q0 + 1), sign(q1 & 1 ? a.y : b.y, q1 + 1));
}

// The frequencies of a lane's four pairs, and magnitude times their cosines and
// sines at position p; of lanes that do not turn, ones and zeros.
struct RopeFreq {
  uint64_t f[4];
};
__device__ __forceinline__ RopeFreq rope_freq(const RopeArgs& r, const RopeLane& p, int lane) {
  RopeFreq q = {{0, 0, 0, 0}};
  if (p.turned) {
    const ulonglong2* t = reinterpret_cast<const ulonglong2*>(r.turns + 4 * lane);
    const ulonglong2 a = __ldg(t), b = __ldg(t + 1);
    q.f[0] = a.x; q.f[1] = a.y; q.f[2] = b.x; q.f[3] = b.y;
  }
  return q;
}
struct Angles {
  F2 c[2], s[2], minus_s[2];
};
__device__ __forceinline__ Angles rope_angles(const RopeArgs& r, const RopeLane& l, const RopeFreq& q, int pos) {
  Angles a;
  const F2 m = f2(l.turned ? r.magnitude : 1.f);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    sincos_turns((uint32_t)(((uint64_t)(int64_t)pos * q.f[2 * i]) >> 32),
                 (uint32_t)(((uint64_t)(int64_t)pos * q.f[2 * i + 1]) >> 32), a.c[i], a.s[i]);
    a.c[i] = mul2(a.c[i], m);
    a.s[i] = mul2(a.s[i], m);
    a.minus_s[i] = mul2(a.s[i], f2(-1.f));
  }
  return a;
}

// A lane's 8 elements are four pairs of fp32: x[0], x[1] the first chunk, x[2],
// x[3] the second.  Rotates them, kBack by the transposed rotation.
template <bool kInterleaved, bool kBack>
__device__ __forceinline__ void turn_lane(const Angles& a, F2 (&x)[4]) {
  if (kInterleaved) {  // the partners are the neighbours
    const float2 c0 = parts(a.c[0]), c1 = parts(a.c[1]), s0 = parts(a.s[0]), s1 = parts(a.s[1]);
    const float c[4] = {c0.x, c0.y, c1.x, c1.y}, s[4] = {s0.x, s0.y, s1.x, s1.y};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = fma2(swapped(x[i]), kBack ? f2(s[i], -s[i]) : f2(-s[i], s[i]), mul2(x[i], f2(c[i])));
  } else {  // the other chunk
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const F2 y = fma2(x[i + 2], kBack ? a.s[i] : a.minus_s[i], mul2(x[i], a.c[i]));
      x[i + 2] = fma2(x[i], kBack ? a.minus_s[i] : a.s[i], mul2(x[i + 2], a.c[i]));
      x[i] = y;
    }
  }
}
// A lane that does not turn leaves what it has, infinities too.  `all`: every one
// turns, the same for the whole grid, so that most calls branch without dividing.
template <bool kInterleaved, bool kBack = false>
__device__ __forceinline__ void turn_row(bool all, const RopeLane& l, const Angles& a, F2 (&x)[4]) {
  if (all) turn_lane<kInterleaved, kBack>(a, x);
  else if (l.turned) turn_lane<kInterleaved, kBack>(a, x);
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
// From the addresses of its chunks.
template <typename T>
__device__ __forceinline__ typename RowOf<T>::type load_row(const char* a, const char* b) {
  using V = decltype(RowOf<T>::type::a);
  return {*reinterpret_cast<const V*>(a), *reinterpret_cast<const V*>(b)};
}
__device__ __forceinline__ void unpack_row(const Row8f& r, F2 (&x)[4]) {
  x[0] = f2(r.a.x, r.a.y);
  x[1] = f2(r.a.z, r.a.w);
  x[2] = f2(r.b.x, r.b.y);
  x[3] = f2(r.b.z, r.b.w);
}
__device__ __forceinline__ void unpack_row(const Row8h& r, F2 (&x)[4]) {
  x[0] = bf16_pair(r.a.x);
  x[1] = bf16_pair(r.a.y);
  x[2] = bf16_pair(r.b.x);
  x[3] = bf16_pair(r.b.y);
}
template <typename T>
__device__ __forceinline__ void store_row(char* a, char* b, const F2 (&x)[4]) {
  if constexpr (sizeof(T) == 4) {
    const float2 p = parts(x[0]), q = parts(x[1]), r = parts(x[2]), s = parts(x[3]);
    *reinterpret_cast<float4*>(a) = make_float4(p.x, p.y, q.x, q.y);
    *reinterpret_cast<float4*>(b) = make_float4(r.x, r.y, s.x, s.y);
  } else {
    *reinterpret_cast<uint2*>(a) = make_uint2(pair_bf16(x[0]), pair_bf16(x[1]));
    *reinterpret_cast<uint2*>(b) = make_uint2(pair_bf16(x[2]), pair_bf16(x[3]));
  }
}

// ---- the norm ----
// Whole warps run all of this, two heads at a time: shuffles by less than 16
// stay within a half, and with all lanes named they cost one instruction.
__device__ __forceinline__ float half_sum(float v) {
#pragma unroll
  for (int d = 8; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}
__device__ __forceinline__ float dot_row(const F2 (&x)[4], const F2 (&y)[4]) {
  return both(add2(fma2(x[1], y[1], mul2(x[0], y[0])), fma2(x[3], y[3], mul2(x[2], y[2]))));
}
__device__ __forceinline__ void scale_row(F2 (&x)[4], float f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = mul2(x[i], f2(f));
}
// A head's sum of squares, and whether it passes fp32's range in either half
// (elements of 2^60 and more): then scaled_head takes it again of x 2^-68, which x
// becomes and its 1 / sqrt(inv_n ss) belongs to; eps is nothing beside it.
constexpr float kHeadUnit = 0x1p-68f, kHeadUnitRoot = 0x1p-34f;
__device__ __forceinline__ bool large_heads(float ss) { return __any_sync(0xffffffffu, !(ss <= 3e38f)); }
// Also whether this half's is the large one: unit is then kHeadUnit, else 1.
__device__ __forceinline__ float scaled_head(F2 (&x)[4], float ss, float inv_n, float eps, float& unit) {
  const bool large = !(ss <= 3e38f);
  unit = large ? kHeadUnit : 1.f;
  scale_row(x, unit);
  ss = half_sum(dot_row(x, x));
  return rsqrt_approx(fmaf(ss, inv_n, large ? 0.f : eps));
}

// The lane's part of a weight, or ones.
__device__ __forceinline__ void load_weight(const float* w, const RopeLane& l, F2 (&x)[4]) {
  if (w) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(w + l.o0)), b = __ldg(reinterpret_cast<const float4*>(w + l.o1));
    x[0] = f2(a.x, a.y);
    x[1] = f2(a.z, a.w);
    x[2] = f2(b.x, b.y);
    x[3] = f2(b.z, b.w);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = f2(1.f);
  }
}

// ---- runs of heads ----
// The heads of all tokens are cut into equal runs, one a warp, so that all end
// together.  A warp takes two tokens at a time, one a half, and their heads one
// after another, with the cosines and sines in registers, and copies the rows
// that come next into a ring of shared memory of its own.  Heads are at constant
// distances from one another: with an address each, or a table of cosines in
// shared memory, 220 instructions went into a row of two heads.
constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;
constexpr int kRopeBwdCtas = 2 * 152;  // what is resident of the gradient; rows of its workspace
// Heads of the weights' gradients that a lane adds up in one fp32 number, and one
// more: longer runs put them away in pairs of fp32, so that sums lose no more the
// longer the call is.  The pairs take shared memory, which shorter calls go without.
constexpr int kRopeFold = 255;

// Queries or keys.
struct RopeSide {
  const void* in;
  void* out;               // backward: the gradient of the output, read
  void* dx;                // backward
  const float* weight;     // [128] or null
  float* d_weight;         // backward
  int64_t in_stride, out_stride, dx_stride;
  int heads;
};

// Arguments of gdn_qk_rope and its gradient, and the queries' of gdn_kv_append_rope.
struct QkRopeArgs {
  RopeArgs r;
  PosArgs pos;
  RopeSide side[2];        // q, then k
  int ctas;                // whose warps take a run each
  float* part;             // backward: [CTAs, 2, 128] sums of the weights' gradients, or null
  int fold;                // backward: a run is longer than kRopeFold, and part is wanted
};

// A place in a warp's heads, which it takes two tokens at a time, one a half of
// the warp, q's heads first: `left` more heads from head h of token pair `pair` on.
struct Walk {
  int pair, h, left;
  // heads that come next and are of one side, at most `most`
  __device__ __forceinline__ int batch(int h_q, int heads, int most) const {
    return min(min(most, left), (h < h_q ? h_q : heads) - h);
  }
  // past n heads; true at the beginning of a side
  __device__ __forceinline__ bool step(int n, int h_q, int heads) {
    left -= n;
    h += n;
    if (h == heads) {
      h = 0;
      ++pair;
      return true;
    }
    return h == h_q;
  }
};

// The runs of a call: this warp's, of warp `me` of the call's.
__device__ __forceinline__ Walk rope_run(const QkRopeArgs& a, int64_t me) {
  const int heads = a.side[0].heads + a.side[1].heads;
  const int64_t units = ((int64_t)a.pos.T + 1) / 2 * heads, warps = (int64_t)a.ctas * kRopeWarps;
  const int64_t first = me * units / warps, last = (me + 1) * units / warps;
  return {(int)(first / heads), (int)(first % heads), (int)(last - first)};
}

// Address of head h of a side's tensor, for this half of the warp.
template <typename T>
__device__ __forceinline__ const char* head_at(const void* base, int64_t stride, int T_all, int pair, int h) {
  const int64_t t = min(2 * pair + (int)(threadIdx.x >> 4 & 1), T_all - 1);
  return reinterpret_cast<const char*>(static_cast<const T*>(base) + t * stride + (int64_t)h * kRopeD);
}

// 4 KB a warp: two stages of four heads (fp32: two) of two tokens.
struct RopeRing {
  alignas(16) char bytes[kRopeWarps][4096];
};

// One warp's run: in -> out.
template <typename T, bool kInterleaved>
__device__ __forceinline__ void turn_run(const QkRopeArgs& a, unsigned block, RopeRing& rings) {
  constexpr int kRow = kRopeD * sizeof(T), kStages = 2, kStage = 4096 / kStages, kBatch = kStage / (2 * kRow);
  const int lane = threadIdx.x & 15, half = threadIdx.x >> 4 & 1;
  const RopeLane l = rope_lane(a.r, lane);
  const bool norm = a.r.norm != kNormNone, all = a.r.rot == kRopeD;
  const int T_all = a.pos.T, h_q = a.side[0].heads, heads = h_q + a.side[1].heads, gap = (l.o1 - l.o0) * (int)sizeof(T);
  const unsigned warp = warp_index();
  char* ring = rings.bytes[warp];
  Walk now = rope_run(a, (int64_t)block * kRopeWarps + warp), next = now;
  const char* x = nullptr;  // the lane's 16 bytes of the next head's row
  auto place = [&] {
    const bool key = next.h >= h_q;
    const RopeSide& s = a.side[key];
    x = head_at<T>(s.in, s.in_stride, T_all, next.pair, next.h - (key ? h_q : 0)) + lane * 16;
  };
  auto copy_batch = [&](int slot) {
    if (next.left > 0) {
      const int n = next.batch(h_q, heads, kBatch);
      char* to = ring + slot * kStage + half * kRow + lane * 16;
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (i < n) {
#pragma unroll
          for (int j = 0; j < kRow; j += 256) copy16(to + i * 2 * kRow + j, x + i * kRow + j);
        }
      x += n * kRow;
      if (next.step(n, h_q, heads)) place();
    }
    copy_commit();
  };
  place();
#pragma unroll
  for (int i = 0; i < kStages; ++i) copy_batch(i);
  int slot = 0;
  bool in = false, new_pair = true, new_side = true;
  TokenSeq seq;
  Angles angle;
  F2 w[4];
  char* y = nullptr;
  while (now.left > 0) {
    if (new_pair) {
      const int t2 = 2 * now.pair + half, t = min(t2, T_all - 1);
      int pos = 0;
      in = token_position(a.pos, t, seq, pos) && t == t2;
      angle = rope_angles(a.r, l, rope_freq(a.r, l, lane), pos);
    }
    if (new_side) {
      const bool key = now.h >= h_q;
      const RopeSide& s = a.side[key];
      y = const_cast<char*>(head_at<T>(s.out, s.out_stride, T_all, now.pair, now.h - (key ? h_q : 0))) + l.o0 * (int)sizeof(T);
      load_weight(s.weight, l, w);
    }
    const int n = now.batch(h_q, heads, kBatch);
    copy_wait<kStages - 1>();
    __syncwarp();
    const char* from = ring + slot * kStage + half * kRow + l.o0 * (int)sizeof(T);
    typename RowOf<T>::type raw[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) raw[i] = load_row<T>(from + i * 2 * kRow, from + i * 2 * kRow + gap);
    __syncwarp();
    copy_batch(slot);
    slot = slot + 1 == kStages ? 0 : slot + 1;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (i >= n) break;
      F2 row[4];
      unpack_row(raw[i], row);
      if (norm) {
        const float ss = half_sum(dot_row(row, row));
        float f = rsqrt_approx(fmaf(ss, a.r.inv_n, a.r.eps)), unit;
        if (large_heads(ss)) f = scaled_head(row, ss, a.r.inv_n, a.r.eps, unit);
        scale_row(row, f);
#pragma unroll
        for (int e = 0; e < 4; ++e) row[e] = mul2(row[e], w[e]);
      }
      turn_row<kInterleaved>(all, l, angle, row);
      if (in) store_row<T>(y + i * kRow, y + i * kRow + gap, row);
    }
    y += n * kRow;
    new_side = now.step(n, h_q, heads);
    new_pair = now.h == 0;
  }
  copy_wait<0>();
}

cudaError_t rope_bwd_setup();  // before calls with fold
cudaError_t launch_qk_rope(const QkRopeArgs& a, bool f32, cudaStream_t st);
cudaError_t launch_qk_rope_bwd(const QkRopeArgs& a, bool f32, cudaStream_t st);
cudaError_t launch_qk_rope_weights(const QkRopeArgs& a, cudaStream_t st);

}  // namespace gdn
