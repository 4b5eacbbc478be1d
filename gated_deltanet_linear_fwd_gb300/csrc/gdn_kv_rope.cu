// New keys normalised and rotated on their way into the 8-bit key/value cache,
// values beside them, and the queries of the same tokens: what a layer does
// between its projection and its attention, in one launch.
//
// Keys go through y = m R (x r w) (gdn_rope.cuh) in fp32 and from there into
// the codes, without a rounding in between; pages, scales and codes are those
// of gdn_kv.cu.  Blocks: queries, 8 warps' runs each, then keys of a (page
// slot, head) each, then values; with few tokens a sequence, warps of keys and
// values.  Measured, 32768 tokens of 8 heads on 2, bf16: 35.7 us, 5.2 TB/s, 78 % of
// what a copy reaches, with issue slots 73 % busy (norm, rotation, codes).
#include <type_traits>

#include "gdn_kv_page.cuh"
#include "gdn_rope.cuh"

namespace gdn {
namespace {

constexpr int kThreads = kPageThreads;
static_assert(kThreads == kRopeThreads, "a block does either");
constexpr int kTasks = kThreads / 16;
constexpr int kRows = kPage / kTasks;   // rows of a page that a half-warp holds

// e4m3 codes of four elements.
__device__ __forceinline__ uint32_t encode4(F2 x, F2 y, float inv_s) {
  const float2 a = parts(mul2(x, f2(inv_s))), b = parts(mul2(y, f2(inv_s)));
  return f32x2_to_e4m3x2(a.x, a.y) | f32x2_to_e4m3x2(b.x, b.y) << 16;
}
__device__ __forceinline__ uint32_t recode4(uint32_t c, float s, float inv_s) {
  const float2 a = e4m3x2_to_f32x2(c), b = e4m3x2_to_f32x2(c >> 16);
  return encode4(f2(a.x * s, a.y * s), f2(b.x * s, b.y * s), inv_s);
}
__device__ __forceinline__ uint32_t magnitude_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }
__device__ __forceinline__ float or_nan(float x) { return magnitude_bits(x) < 0x7f800000u ? x : __uint_as_float(0x7fffffffu); }

// The rotations by 16, 32 and 48 tokens: a half-warp's rows are 16 apart, and all
// but the first turn by the first's angles and then by these, a product a
// pair instead of a cosine and a sine.
struct alignas(16) PageSteps {
  float c[kRows - 1][kRopeD / 2], s[kRows - 1][kRopeD / 2];
};
__device__ __forceinline__ void page_steps(const RopeArgs& r, PageSteps& sh) {
  const int pair = threadIdx.x & 31, step = threadIdx.x >> 5;  // two pairs of 64 a thread
  if (step >= kRows - 1 || 4 * pair >= r.rot) return;
  const ulonglong2 f = __ldg(reinterpret_cast<const ulonglong2*>(r.turns) + pair);
  const uint64_t p = (uint64_t)(kTasks * (step + 1));
  F2 c, s;
  sincos_turns((uint32_t)(p * f.x >> 32), (uint32_t)(p * f.y >> 32), c, s);
  *reinterpret_cast<float2*>(&sh.c[step][2 * pair]) = parts(c);
  *reinterpret_cast<float2*>(&sh.s[step][2 * pair]) = parts(s);
}
__device__ __forceinline__ Angles further(const Angles& a, const float4& c, const float4& s) {
  const F2 cc[2] = {f2(c.x, c.y), f2(c.z, c.w)}, ss[2] = {f2(s.x, s.y), f2(s.z, s.w)};
  Angles r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    r.c[i] = fma2(a.minus_s[i], ss[i], mul2(a.c[i], cc[i]));
    r.s[i] = fma2(a.c[i], ss[i], mul2(a.s[i], cc[i]));
    r.minus_s[i] = mul2(r.s[i], f2(-1.f));
  }
  return r;
}

// A row of keys, normalised and rotated.  Whole warps run this.
template <bool kInterleaved>
__device__ __forceinline__ void key_row(const KvRopeArgs& a, const RopeLane& l, const F2 (&w)[4], const Angles& angle, F2 (&y)[4]) {
  if (a.q.r.norm != kNormNone) {
    const float ss = half_sum(dot_row(y, y));
    float n = rsqrt_approx(fmaf(ss, a.q.r.inv_n, a.q.r.eps)), unit;
    if (large_heads(ss)) n = scaled_head(y, ss, a.q.r.inv_n, a.q.r.eps, unit);
    scale_row(y, n);
    if (a.k_weight) {
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = mul2(y[e], w[e]);
    }
  }
  turn_row<kInterleaved>(a.q.r.rot == kRopeD, l, angle, y);
}
// The largest magnitude of a lane's part of a row, as bits.
__device__ __forceinline__ uint32_t row_bits(const F2 (&y)[4]) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 p = parts(y[e]);
    m = max(m, max(magnitude_bits(p.x), magnitude_bits(p.y)));
  }
  return m;
}
// What is not finite becomes NaN and does not count: the largest of the others.
template <int N>
__device__ __forceinline__ uint32_t finite_rows(F2 (&y)[N][4]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 p = parts(y[i][e]);
      if (magnitude_bits(p.x) < 0x7f800000u) m = max(m, magnitude_bits(p.x));
      if (magnitude_bits(p.y) < 0x7f800000u) m = max(m, magnitude_bits(p.y));
      y[i][e] = f2(or_nan(p.x), or_nan(p.y));
    }
  }
  return m;
}

template <typename T, bool kInterleaved>
__device__ __forceinline__ void append_turned_page(const KvRopeArgs& a, const Entry& en, int h, uint32_t& top,
                                                   PageSteps& sh) {
  const int tid = threadIdx.x, lane = tid & 15, hw = tid >> 4;
  const int past = en.s.len - en.s.n, pos0 = en.slot * kPage;
  const int lo = max(past - pos0, 0), hi = min(en.s.len - pos0, kPage);  // rows of the page that are new
  if (hi <= lo) return;
  const RopeLane l = rope_lane(a.q.r, lane);
  const int64_t stride = a.p.k_stride;
  const T* src = static_cast<const T*>(a.p.k) + ((int64_t)en.s.tok0 + pos0 - past) * stride + h * kHeadDim;
  const char* first = reinterpret_cast<const char*>(src + l.o0);
  const uint32_t gap = (l.o1 - l.o0) * sizeof(T);
  typename RowOf<T>::type raw[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = hw + kTasks * i;
    raw[i] = {};
    const char* p = first + r * stride * (int64_t)sizeof(T);
    if (r >= lo && r < hi) raw[i] = load_row<T>(p, p + gap);
  }
  const int page = kv_page(a.p.c, en.seq, en.slot);
  if (page < 0) return;
  const size_t head = (size_t)page * a.p.c.h_kv + h;
  float* scale = a.p.c.k_scale + head;
  const float old_s = lo > 0 ? *scale : 0.f;
  page_steps(a.q.r, sh);
  F2 y[kRows][4], w[4];
  load_weight(a.k_weight, l, w);
  const Angles angle = rope_angles(a.q.r, l, rope_freq(a.q.r, l, lane), pos0 + hw);
  __syncthreads();
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    unpack_row(raw[i], y[i]);  // zeros where the row is not new
    if (kTasks * i >= hi || kTasks * (i + 1) <= lo) continue;
    Angles here = angle;
    if (i > 0 && l.turned)
      here = further(angle, *reinterpret_cast<const float4*>(&sh.c[max(i - 1, 0)][4 * lane]),
                     *reinterpret_cast<const float4*>(&sh.s[max(i - 1, 0)][4 * lane]));
    key_row<kInterleaved>(a, l, w, here, y[i]);
    m = max(m, row_bits(y[i]));
  }
  if (m >= 0x7f800000u) m = finite_rows(y);
  m = __reduce_max_sync(0xffffffffu, m);
  __syncthreads();  // top is zero; everyone has read the scale
  if ((tid & 31) == 0 && m) atomicMax(&top, m);
  __syncthreads();
  const float s = fmaxf(pow2f(min(e4m3_scale_exp(top, kScaleMinExp), kScaleMaxExp)), old_s);
  const float inv = 1.0f / s;  // exact: a power of two
  uint8_t* codes = a.p.c.k + head * kPageBytes;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = hw + kTasks * i;
    uint32_t* c0 = reinterpret_cast<uint32_t*>(codes + r * kHeadDim + l.o0);
    uint32_t* c1 = reinterpret_cast<uint32_t*>(codes + r * kHeadDim + l.o1);
    if (r >= lo && r < hi) {
      *c0 = encode4(y[i][0], y[i][1], inv);
      *c1 = encode4(y[i][2], y[i][3], inv);
    } else if (r < lo && s > old_s) {
      *c0 = recode4(*c0, old_s, inv);
      *c1 = recode4(*c1, old_s, inv);
    }
  }
  if (tid == 0) *scale = s;
}

// ---- few tokens a sequence ----
// A page slot and head of keys or values, with at most kFewTokens new rows, by
// one warp: two rows at a time, a half each.  Of a block's 16 half-warps most
// would have no row, and a block's start and barriers are what it costs.  Back to
// back in a graph, 8 + 2 heads, 256 sequences, with 1 / 4 / 8 tokens each: 2.8 /
// 4.9 / 6.1 us, by blocks 6.6 / 9.7 / 10.7; 1024 sequences of 32 + 8 heads: 12.3
// / 22.4 / 37.1 and 73 / 104 / 121.  With 16 rows a warp a single sequence takes
// twice as long (5.9 and 3.1).
template <typename T, bool kInterleaved, int kFewTokens>
__device__ __forceinline__ void append_few(const KvRopeArgs& a, unsigned task) {
  const unsigned h_kv = a.p.c.h_kv, pages = a.entries * h_kv;  // the grid is below 2^31
  const bool values = task >= pages;
  if (values) task -= pages;
  if (task >= pages) return;
  const int h = (int)(task % h_kv), e = (int)(task / h_kv), seq = e / a.p.pages_each, j = e % a.p.pages_each;
  const KvSeq s = kv_seq(a.p.c, seq);
  if (j >= seq_slots(s)) return;
  const int past = s.len - s.n, slot = max(past, 0) / kPage + j, pos0 = slot * kPage;
  const int lo = max(past - pos0, 0), hi = min(s.len - pos0, kPage);  // rows of the page that are new
  if (hi <= lo) return;
  const int lane = threadIdx.x & 15, half = threadIdx.x >> 4 & 1;
  const RopeLane l = values ? RopeLane{8 * lane, 8 * lane + 4, false} : rope_lane(a.q.r, lane);
  const int64_t stride = values ? a.p.v_stride : a.p.k_stride;
  const T* src = static_cast<const T*>(values ? a.p.v : a.p.k) + ((int64_t)s.tok0 + pos0 - past) * stride + h * kHeadDim;
  const char* first = reinterpret_cast<const char*>(src + l.o0);
  const uint32_t gap = (l.o1 - l.o0) * sizeof(T);
  typename RowOf<T>::type raw[kFewTokens / 2];
#pragma unroll
  for (int i = 0; i < kFewTokens / 2; ++i) {
    const int r = lo + 2 * i + half;
    raw[i] = {};
    const char* p = first + r * stride * (int64_t)sizeof(T);
    if (r < hi) raw[i] = load_row<T>(p, p + gap);
  }
  const int page = kv_page(a.p.c, seq, slot);
  if (page < 0) return;
  const size_t head = (size_t)page * h_kv + h;
  float* scale = (values ? a.p.c.v_scale : a.p.c.k_scale) + head;
  const float old_s = lo > 0 ? *scale : 0.f;
  F2 y[kFewTokens / 2][4], w[4];
  load_weight(values ? nullptr : a.k_weight, l, w);
  const RopeFreq freq = rope_freq(a.q.r, l, lane);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kFewTokens / 2; ++i) {
    unpack_row(raw[i], y[i]);
    if (lo + 2 * i >= hi) continue;
    if (!values) key_row<kInterleaved>(a, l, w, rope_angles(a.q.r, l, freq, pos0 + lo + 2 * i + half), y[i]);
    m = max(m, row_bits(y[i]));
  }
  if (m >= 0x7f800000u) m = finite_rows(y);
  m = __reduce_max_sync(0xffffffffu, m);
  const float now_s = fmaxf(pow2f(min(e4m3_scale_exp(m, kScaleMinExp), kScaleMaxExp)), old_s);
  const float inv = 1.0f / now_s;  // exact: a power of two
  uint8_t* codes = (values ? a.p.c.v : a.p.c.k) + head * kPageBytes;
#pragma unroll
  for (int i = 0; i < kFewTokens / 2; ++i) {
    const int r = lo + 2 * i + half;
    if (r >= hi) continue;
    *reinterpret_cast<uint32_t*>(codes + r * kHeadDim + l.o0) = encode4(y[i][0], y[i][1], inv);
    *reinterpret_cast<uint32_t*>(codes + r * kHeadDim + l.o1) = encode4(y[i][2], y[i][3], inv);
  }
  if (now_s > old_s)  // the earlier rows follow
    for (uint32_t* c = reinterpret_cast<uint32_t*>(codes) + (threadIdx.x & 31); c < reinterpret_cast<uint32_t*>(codes + lo * kHeadDim); c += 32)
      *c = recode4(*c, old_s, inv);
  if ((threadIdx.x & 31) == 0) *scale = now_s;
}

template <typename T, bool kInterleaved, int kFewTokens>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 2) append_few_kernel(const KvRopeArgs a) {
  __shared__ RopeRing ring;
  grid_dependency_wait();
  grid_launch_dependents();
  if (blockIdx.x < (unsigned)a.q.ctas) turn_run<T, kInterleaved>(a.q, blockIdx.x, ring);
  else append_few<T, kInterleaved, kFewTokens>(a, (blockIdx.x - a.q.ctas) * kRopeWarps + warp_index());
}

template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 2) append_rope_kernel(const KvRopeArgs a) {
  __shared__ int part[kThreads / 32];
  __shared__ Entry found;
  __shared__ uint32_t top;
  __shared__ union {
    PageSteps steps;
    RopeRing ring;
  } sh;
  const int tid = threadIdx.x;
  if (tid == 0) top = 0;
  grid_dependency_wait();
  grid_launch_dependents();
  // queries first: theirs are long runs, beside which the pages' blocks come and go
  if (blockIdx.x < (unsigned)a.q.ctas) {
    turn_run<T, kInterleaved>(a.q, blockIdx.x, sh.ring);
    return;
  }
  unsigned b = blockIdx.x - a.q.ctas;
  const unsigned pages = a.entries * (unsigned)a.p.c.h_kv;  // the grid is below 2^31
  const bool values = b >= pages;
  if (values) b -= pages;
  const int h = (int)(b % (unsigned)a.p.c.h_kv);
  const Entry en = find_entry(a.p, (int)(b / (unsigned)a.p.c.h_kv), part, &found);
  if (en.seq < 0) return;
  if (values) append_page<T>(a.p, en, h, true, top);
  else append_turned_page<T, kInterleaved>(a, en, h, top, sh.steps);
}

}  // namespace

cudaError_t launch_kv_append_rope(const KvRopeArgs& a, bool f32, cudaStream_t st) {
  const unsigned tasks = 2 * a.entries * (unsigned)a.p.c.h_kv;
  const int most = a.p.c.cu ? kPage : a.p.c.n_each;  // new rows of a page
  const bool few = most <= 8;
  const dim3 grid(a.q.ctas + (few ? (tasks + kRopeWarps - 1) / kRopeWarps : tasks)), block(kThreads);
  auto run = [&](auto type, auto interleaved) {
    using T = decltype(type);
    constexpr bool kInterleaved = decltype(interleaved)::value;
    return most <= 4 ? launch_kernel(append_few_kernel<T, kInterleaved, 4>, grid, block, 0, st, true, a)
           : few     ? launch_kernel(append_few_kernel<T, kInterleaved, 8>, grid, block, 0, st, true, a)
                     : launch_kernel(append_rope_kernel<T, kInterleaved>, grid, block, 0, st, true, a);
  };
  auto typed = [&](auto type) { return a.q.r.interleaved ? run(type, std::true_type()) : run(type, std::false_type()); };
  return f32 ? typed(float()) : typed(__nv_bfloat16());
}

}  // namespace gdn
