// New keys normalised and rotated on their way into the 8-bit key/value cache,
// values beside them, and the queries of the same tokens: what a layer does
// between its projection and its attention, in one launch.
//
// Keys go through y = m R (x r w) (gdn_rope.cuh) in fp32 and from there into
// the codes, without a rounding in between; pages, scales and codes are those
// of gdn_kv.cu.  Blocks: queries, 8 warps' runs each, then keys of a (page
// slot, head) each, then values.
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
  const bool norm = a.q.r.norm != kNormNone;
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    unpack_row(raw[i], y[i]);  // zeros where the row is not new
    if (kTasks * i >= hi || kTasks * (i + 1) <= lo) continue;
    if (norm) {
      const float ss = half_sum(dot_row(y[i], y[i]));
      float n = rsqrt_approx(fmaf(ss, a.q.r.inv_n, a.q.r.eps)), unit;
      if (large_heads(ss)) n = scaled_head(y[i], ss, a.q.r.inv_n, a.q.r.eps, unit);
      scale_row(y[i], n);
      if (a.k_weight) {
#pragma unroll
        for (int e = 0; e < 4; ++e) y[i][e] = mul2(y[i][e], w[e]);
      }
    }
    Angles here = angle;
    if (i > 0 && l.turned)
      here = further(angle, *reinterpret_cast<const float4*>(&sh.c[max(i - 1, 0)][4 * lane]),
                     *reinterpret_cast<const float4*>(&sh.s[max(i - 1, 0)][4 * lane]));
    turn_row<kInterleaved>(a.q.r.rot == kRopeD, l, here, y[i]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 p = parts(y[i][e]);
      m = max(m, max(magnitude_bits(p.x), magnitude_bits(p.y)));
    }
  }
  if (m >= 0x7f800000u) {  // what is not finite becomes NaN codes and does not count
    m = 0;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 p = parts(y[i][e]);
        if (magnitude_bits(p.x) < 0x7f800000u) m = max(m, magnitude_bits(p.x));
        if (magnitude_bits(p.y) < 0x7f800000u) m = max(m, magnitude_bits(p.y));
        y[i][e] = f2(or_nan(p.x), or_nan(p.y));
      }
    }
  }
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
  const dim3 grid(a.q.ctas + 2 * a.entries * (unsigned)a.p.c.h_kv), block(kThreads);
  if (f32)
    return a.q.r.interleaved ? launch_kernel(append_rope_kernel<float, true>, grid, block, 0, st, true, a)
                           : launch_kernel(append_rope_kernel<float, false>, grid, block, 0, st, true, a);
  return a.q.r.interleaved ? launch_kernel(append_rope_kernel<__nv_bfloat16, true>, grid, block, 0, st, true, a)
                         : launch_kernel(append_rope_kernel<__nv_bfloat16, false>, grid, block, 0, st, true, a);
}

}  // namespace gdn
