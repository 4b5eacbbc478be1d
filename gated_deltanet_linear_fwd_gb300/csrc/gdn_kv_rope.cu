// New keys normalised and rotated on their way into the 8-bit key/value cache,
// values beside them, and the queries of the same tokens: what a layer does
// between its projection and its attention, in one launch.
//
// Keys go through y = m R (x r w) (gdn_rope.cuh) in fp32 and from there into
// the codes, without a rounding in between; pages, scales and codes are those
// of gdn_kv.cu.  Blocks: keys of a (page slot, head) each, then values, then
// queries, 16 half-warps' worth of heads each.
#include "gdn_kv_page.cuh"
#include "gdn_rope.cuh"

namespace gdn {
namespace {

constexpr int kThreads = kPageThreads;
constexpr int kTasks = kThreads / 16;
constexpr int kRows = kPage / kTasks;   // rows of a page that a half-warp holds

// e4m3 codes of four elements.
__device__ __forceinline__ uint32_t encode4(const float* x, float inv_s) {
  return f32x2_to_e4m3x2(x[0] * inv_s, x[1] * inv_s) | f32x2_to_e4m3x2(x[2] * inv_s, x[3] * inv_s) << 16;
}
__device__ __forceinline__ uint32_t recode4(uint32_t c, float s, float inv_s) {
  const float2 a = e4m3x2_to_f32x2(c), b = e4m3x2_to_f32x2(c >> 16);
  const float x[4] = {a.x * s, a.y * s, b.x * s, b.y * s};
  return encode4(x, inv_s);
}

template <typename T, bool kInterleaved>
__device__ __forceinline__ void append_turned_page(const KvRopeArgs& a, const Entry& en, int h, uint32_t& top) {
  const int tid = threadIdx.x, lane = tid & 15, hw = tid >> 4;
  const unsigned mask = half_mask();
  const int past = en.s.len - en.s.n, pos0 = en.slot * kPage;
  const int lo = max(past - pos0, 0), hi = min(en.s.len - pos0, kPage);  // rows of the page that are new
  if (hi <= lo) return;
  const RopeLane l = rope_lane(a.r, lane);
  const int64_t stride = a.p.k_stride;
  const T* src = static_cast<const T*>(a.p.k) + ((int64_t)en.s.tok0 + pos0 - past) * stride + h * kHeadDim;
  typename RowOf<T>::type raw[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = hw + kTasks * i;
    if (r >= lo && r < hi) raw[i] = load_row(src + r * stride, l);
  }
  const int page = kv_page(a.p.c, en.seq, en.slot);
  if (page < 0) return;
  const size_t head = (size_t)page * a.p.c.h_kv + h;
  float* scale = a.p.c.k_scale + head;
  const float old_s = lo > 0 ? *scale : 0.f;
  const RopeFreq f = rope_freq(a.r, l, lane);
  float y[kRows][8], w[8];
  if (a.k_weight) load_weight(a.k_weight, l, w);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = hw + kTasks * i;
    if (r < lo || r >= hi) continue;
    float c[4], s[4];
    rope_angles(a.r, l, f, pos0 + r, c, s);
    unpack_row(raw[i], y[i]);
    if (a.r.norm != kNormNone) {
      float unit;
      const float n = head_scale(half_sum(sum_squares(y[i]), mask), y[i], a.r.inv_n, a.r.eps, mask, unit);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[i][e] *= n;
      if (a.k_weight) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[i][e] *= w[e];
      }
    }
    rope_turn<kInterleaved>(y[i], c, s);
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(y[i][e]) & 0x7fffffffu);
  }
  if (m >= 0x7f800000u) {  // what is not finite becomes NaN codes and does not count
    m = 0;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int r = hw + kTasks * i;
      if (r < lo || r >= hi) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t b = __float_as_uint(y[i][e]) & 0x7fffffffu;
        if (b < 0x7f800000u) m = max(m, b);
        else y[i][e] = __uint_as_float(0x7fffffffu);
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
      *c0 = encode4(y[i], inv);
      *c1 = encode4(y[i] + 4, inv);
    } else if (r < lo && s > old_s) {
      *c0 = recode4(*c0, old_s, inv);
      *c1 = recode4(*c1, old_s, inv);
    }
  }
  if (tid == 0) *scale = s;
}

// A task: some of the query heads of a token.
template <typename T, bool kInterleaved>
__device__ __forceinline__ void turn_queries(const KvRopeArgs& a, int64_t task) {
  const int lane = threadIdx.x & 15;
  const int t = (int)(task / a.splits), part = (int)(task % a.splits);
  if (t >= a.p.c.T) return;
  const int seq = a.p.c.cu ? seq_of(a.p.c.cu, a.p.c.n_seqs, t) : t / a.p.c.n_each;
  const KvSeq s = kv_seq(a.p.c, seq);
  if (t < s.tok0 || t - s.tok0 >= s.n) return;  // a token outside every sequence
  const RopeLane l = rope_lane(a.r, lane);
  float c[4], sn[4];
  rope_angles(a.r, l, rope_freq(a.r, l, lane), s.len - s.n + t - s.tok0, c, sn);
  const int h0 = (int)((int64_t)part * a.p.c.h_q / a.splits), h1 = (int)((int64_t)(part + 1) * a.p.c.h_q / a.splits);
  turn_heads<T, kInterleaved>(a.r, l, c, sn, static_cast<const T*>(a.q) + t * a.q_stride + h0 * kRopeD,
                              static_cast<T*>(a.q_out) + t * a.q_out_stride + h0 * kRopeD, h1 - h0, a.q_weight, half_mask());
}

template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) append_rope_kernel(const KvRopeArgs a) {
  __shared__ int part[kThreads / 32];
  __shared__ Entry found;
  __shared__ uint32_t top;
  const int tid = threadIdx.x;
  if (tid == 0) top = 0;
  grid_dependency_wait();
  grid_launch_dependents();
  unsigned b = blockIdx.x;
  const unsigned pages = a.entries * (unsigned)a.p.c.h_kv;  // the grid, 2 pages and more, is below 2^31
  if (b >= 2 * pages) {
    turn_queries<T, kInterleaved>(a, (int64_t)(b - 2 * pages) * kTasks + (tid >> 4));
    return;
  }
  const bool values = b >= pages;
  if (values) b -= pages;
  const int h = (int)(b % (unsigned)a.p.c.h_kv);
  const Entry en = find_entry(a.p, (int)(b / (unsigned)a.p.c.h_kv), part, &found);
  if (en.seq < 0) return;
  if (values) append_page<T>(a.p, en, h, true, top);
  else append_turned_page<T, kInterleaved>(a, en, h, top);
}

}  // namespace

cudaError_t launch_kv_append_rope(const KvRopeArgs& a, bool f32, cudaStream_t st) {
  const int64_t tasks = a.q ? (int64_t)a.p.c.T * a.splits : 0;
  const dim3 grid((unsigned)(2 * (int64_t)a.entries * a.p.c.h_kv + (tasks + kTasks - 1) / kTasks)), block(kThreads);
  if (f32)
    return a.r.interleaved ? launch_kernel(append_rope_kernel<float, true>, grid, block, 0, st, true, a)
                           : launch_kernel(append_rope_kernel<float, false>, grid, block, 0, st, true, a);
  return a.r.interleaved ? launch_kernel(append_rope_kernel<__nv_bfloat16, true>, grid, block, 0, st, true, a)
                         : launch_kernel(append_rope_kernel<__nv_bfloat16, false>, grid, block, 0, st, true, a);
}

}  // namespace gdn
