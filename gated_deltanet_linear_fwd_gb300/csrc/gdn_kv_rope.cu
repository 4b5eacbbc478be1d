// New keys normalised and rotated on their way into the 8-bit key/value cache,
// values beside them, and the queries of the same tokens: what a layer does
// between its projection and its attention, in one launch.
//
// Keys go through y = m R (x r w) (gdn_rope.cuh) in fp32 and from there into
// the codes, without a rounding in between; pages, scales and codes are those
// of gdn_kv.cu.  Blocks: queries, 8 warps' runs each, then keys of a (page
// slot, head) each, then values; with few tokens a sequence, warps of keys and
// values.  Measured, 32768 tokens of 8 heads on 2, bf16: 35.7 us, 5.2 TB/s, 77 % of
// what a copy reaches, with issue slots 73 % busy (norm, rotation, codes); of
// fp32 58.9 us, 90 %.
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
// pair instead of a cosine and a sine.  A cosine is then off by both factors'
// errors and two roundings more, 13 of 2^-24 and not 6, and a key by up to 27 and not
// 19 in all; its e4m3 code rounds to 2^-4.
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
// The new rows of a page slot.  Without offsets entry e is slot e % pages_each of
// sequence e / pages_each's; with offsets it is token e's, if that is the slot's
// first new one.
struct PageRows {
  Entry en;
  int lo, hi;  // hi <= lo: none
};
template <bool kRagged>
__device__ __forceinline__ PageRows page_rows(const KvAppendArgs& a, int e) {
  PageRows p;
  p.lo = p.hi = 0;
  KvSeq& s = p.en.s;
  if (kRagged) {
    p.en.seq = seq_of(a.c.cu, a.c.n_seqs, e);
    s = kv_seq(a.c, p.en.seq);
    const int at = e - s.tok0, pos = s.len - s.n + at;
    if (at < 0 || at >= s.n || pos < 0 || (at > 0 && pos % kPage)) return p;
    p.en.slot = pos / kPage;
  } else {
    p.en.seq = e / a.pages_each;
    s = kv_seq(a.c, p.en.seq);
    const int j = e % a.pages_each;
    if (j >= seq_slots(s)) return p;
    p.en.slot = max(s.len - s.n, 0) / kPage + j;
  }
  p.lo = max(s.len - s.n - p.en.slot * kPage, 0);
  p.hi = min(s.len - p.en.slot * kPage, kPage);
  return p;
}

// A page slot and head of keys or values, with at most kFew new rows, by one
// warp: two rows at a time, a half each.
template <typename T, bool kInterleaved, int kFew>
__device__ __forceinline__ void append_few(const KvRopeArgs& a, const PageRows& p, int h, bool values) {
  const int lane = threadIdx.x & 15, half = threadIdx.x >> 4 & 1, pos0 = p.en.slot * kPage;
  const RopeLane l = values ? RopeLane{8 * lane, 8 * lane + 4, false} : rope_lane(a.q.r, lane);
  const int64_t stride = values ? a.p.v_stride : a.p.k_stride;
  // packed token of row r: tok0 + pos0 + r - (len - n)
  const T* src = static_cast<const T*>(values ? a.p.v : a.p.k) +
                 ((int64_t)p.en.s.tok0 + pos0 - (p.en.s.len - p.en.s.n)) * stride + h * kHeadDim;
  const char* first = reinterpret_cast<const char*>(src + l.o0);
  const uint32_t gap = (l.o1 - l.o0) * sizeof(T);
  typename RowOf<T>::type raw[kFew / 2];
#pragma unroll
  for (int i = 0; i < kFew / 2; ++i) {
    const int r = p.lo + 2 * i + half;
    raw[i] = {};
    const char* at = first + r * stride * (int64_t)sizeof(T);
    if (r < p.hi) raw[i] = load_row<T>(at, at + gap);
  }
  const int page = kv_page(a.p.c, p.en.seq, p.en.slot);
  if (page < 0) return;
  const size_t head = (size_t)page * a.p.c.h_kv + h;
  float* scale = (values ? a.p.c.v_scale : a.p.c.k_scale) + head;
  const float old_s = p.lo > 0 ? *scale : 0.f;
  F2 y[kFew / 2][4], w[4];
  load_weight(values ? nullptr : a.k_weight, l, w);
  const RopeFreq freq = rope_freq(a.q.r, l, lane);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kFew / 2; ++i) {
    unpack_row(raw[i], y[i]);
    if (p.lo + 2 * i >= p.hi) continue;
    if (!values) key_row<kInterleaved>(a, l, w, rope_angles(a.q.r, l, freq, pos0 + p.lo + 2 * i + half), y[i]);
    m = max(m, row_bits(y[i]));
  }
  if (m >= 0x7f800000u) m = finite_rows(y);
  m = __reduce_max_sync(0xffffffffu, m);
  const float s = fmaxf(pow2f(min(e4m3_scale_exp(m, kScaleMinExp), kScaleMaxExp)), old_s);
  const float inv = 1.0f / s;  // exact: a power of two
  uint8_t* codes = (values ? a.p.c.v : a.p.c.k) + head * kPageBytes;
#pragma unroll
  for (int i = 0; i < kFew / 2; ++i) {
    const int r = p.lo + 2 * i + half;
    if (r >= p.hi) continue;
    *reinterpret_cast<uint32_t*>(codes + r * kHeadDim + l.o0) = encode4(y[i][0], y[i][1], inv);
    *reinterpret_cast<uint32_t*>(codes + r * kHeadDim + l.o1) = encode4(y[i][2], y[i][3], inv);
  }
  if (s > old_s)  // the earlier rows follow
    for (int i = threadIdx.x & 31; i < p.lo * kHeadDim / 4; i += 32) {
      uint32_t* c = reinterpret_cast<uint32_t*>(codes) + i;
      *c = recode4(*c, old_s, inv);
    }
  if ((threadIdx.x & 31) == 0) *scale = s;
}

// Of a block's 16 half-warps most would have no row here, and a block's start,
// barriers and, with offsets, its search for the slot cost more than the rows: so a
// warp takes a page slot and head.  With offsets a slot may have more than kFew
// rows after all: those the block does, one after another.  Used where a sequence has
// up to 8 tokens, with offsets on average.  Back to back in a graph, in us, bf16:
//   8 + 2 heads, 256 sequences of 1 / 4 / 8 tokens  2.7 / 4.9 / 6.1, by blocks 6.6 / 9.7 / 10.7
//     the same with offsets                         3.9 / 7.0 / 11.4,          8.5 / 10.6 / 12.1
//   32 + 8 heads, 1024 sequences                    12.6 / 23 / 38,            73 / 104 / 121
//     the same with offsets                         18 / 54 / 119,             178 / 193 / 214
//   8 + 2 (32 + 8) heads, 255 of 1 token and one of 1700  10.4 (23),           12.0 (36)
//     63 of 1 token and one of 448                  7.0 (10),                  5.5 (11)
// With 16 rows a warp a single sequence takes twice as long (5.9 and 3.1).  At
// 64 registers bf16 spills 16 to 124 bytes a thread of 8 rows, and 36 to 72 of 4 with offsets;
// three CTAs an SM, without spills, are slower.
template <typename T, bool kInterleaved, int kFew, bool kRagged>
__global__ void __launch_bounds__(kThreads, kAppendRopeCtas<T>) append_few_kernel(const KvRopeArgs a) {
  __shared__ uint32_t top;
  __shared__ Entry many[kRopeWarps];  // seq < 0: none
  __shared__ union {
    PageSteps steps;
    RopeRing ring;
  } sh;
  grid_dependency_wait();
  grid_launch_dependents();
  if (blockIdx.x < (unsigned)a.q.ctas) {
    turn_run<T, kInterleaved>(a.q, blockIdx.x, sh.ring);
    return;
  }
  const unsigned block = blockIdx.x - a.q.ctas, warp = warp_index(), h_kv = a.p.c.h_kv;
  const unsigned slots = kRagged ? (unsigned)a.p.c.T : a.entries, pages = slots * h_kv;  // of keys; as many of values
  // with offsets heads come after one another: slots of many rows are then in different blocks
  auto values = [&](unsigned w) { return block * kRopeWarps + w >= pages; };
  auto place = [&](unsigned w) { return block * kRopeWarps + w - (values(w) ? pages : 0u); };
  auto head = [&](unsigned w) { return (int)(kRagged ? place(w) / slots : place(w) % h_kv); };
  PageRows p;
  p.lo = p.hi = 0;
  if (place(warp) < pages) p = page_rows<kRagged>(a.p, (int)(kRagged ? place(warp) % slots : place(warp) / h_kv));
  if (p.hi > p.lo && p.hi - p.lo <= kFew) append_few<T, kInterleaved, kFew>(a, p, head(warp), values(warp));
  if constexpr (kRagged) {
    if (block == 0)  // the lengths of sequences without tokens are checked too
      for (int i = threadIdx.x; i < a.p.c.n_seqs; i += kThreads) kv_seq(a.p.c, i);
    const bool more = p.hi - p.lo > kFew;
    if ((threadIdx.x & 31) == 0) {
      many[warp] = p.en;
      if (!more) many[warp].seq = -1;
    }
    if (!__syncthreads_or(more)) return;
    for (unsigned w = 0; w < kRopeWarps; ++w) {
      const Entry en = many[w];
      if (en.seq < 0) continue;
      if (threadIdx.x == 0) top = 0;
      if (values(w)) append_page<T>(a.p, en, head(w), true, top);
      else append_turned_page<T, kInterleaved>(a, en, head(w), top, sh.steps);
      __syncthreads();
    }
  }
}

// bf16: at the 64 registers of four CTAs an SM some 50 bytes a thread are spilled;
// with three and none 38.0 us for 32768 tokens, with four 35.4.
template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, kAppendRopeCtas<T>) append_rope_kernel(const KvRopeArgs a) {
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
  const int64_t each = append_each(a.p.c);
  const bool few = append_by_warps(a.p.c);
  const unsigned tasks = (unsigned)append_tasks(a);  // below 2^31
  const dim3 grid(a.q.ctas + (few ? (tasks + kRopeWarps - 1) / kRopeWarps : tasks)), block(kThreads);
  auto run = [&](auto type, auto interleaved) {
    using T = decltype(type);
    constexpr bool kInterleaved = decltype(interleaved)::value;
    auto launch = [&](auto kernel) { return launch_kernel(kernel, grid, block, 0, st, true, a); };
    if (!few) return launch(append_rope_kernel<T, kInterleaved>);
    if (a.p.c.cu)
      return each <= 4 ? launch(append_few_kernel<T, kInterleaved, 4, true>) : launch(append_few_kernel<T, kInterleaved, 8, true>);
    return each <= 4 ? launch(append_few_kernel<T, kInterleaved, 4, false>) : launch(append_few_kernel<T, kInterleaved, 8, false>);
  };
  auto typed = [&](auto type) { return a.q.r.interleaved ? run(type, std::true_type()) : run(type, std::false_type()); };
  return f32 ? typed(float()) : typed(__nv_bfloat16());
}

}  // namespace gdn
