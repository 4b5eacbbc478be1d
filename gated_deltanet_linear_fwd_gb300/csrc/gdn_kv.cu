// Writing the 8-bit key/value cache and reading it back.
//
// A page of one key/value head is 64 tokens of 128 e4m3 codes c with one
// power-of-two scale s for its keys and one for its values, x = c s.  With a
// the largest finite magnitude among the new tokens of the page, s(a) is the
// smallest power of two with a / s <= 448 (e4m3's largest value).  A page
// that holds earlier tokens keeps the larger of its scale and s(a); when the
// scale grows, the earlier codes are divided by the (power of two) ratio,
// which only moves their exponents unless they become subnormal.  Because s
// is a power of two, x / s and c s are exact in fp32 and the one rounding is
// that to e4m3.
//
// One CTA per (page slot that receives tokens, head).  Both operators move
// each byte once and are bound by that.
#include "gdn_kv.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kChunks = kPage * kHeadDim / 8 / kThreads;  // 8-element chunks a thread holds

constexpr int kScaleMinExp = -40, kScaleMaxExp = 40;

// 8 elements of a row as they are in memory, and as fp32.
struct Raw8f {
  float4 a, b;
};
__device__ __forceinline__ Raw8f load_raw(const float* p) {
  return {__ldg(reinterpret_cast<const float4*>(p)), __ldg(reinterpret_cast<const float4*>(p) + 1)};
}
__device__ __forceinline__ uint4 load_raw(const __nv_bfloat16* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ void zero_raw(Raw8f& r) { r.a = r.b = make_float4(0.f, 0.f, 0.f, 0.f); }
__device__ __forceinline__ void zero_raw(uint4& r) { r = make_uint4(0, 0, 0, 0); }
__device__ __forceinline__ void unpack8(const Raw8f& r, float (&x)[8]) {
  x[0] = r.a.x; x[1] = r.a.y; x[2] = r.a.z; x[3] = r.a.w;
  x[4] = r.b.x; x[5] = r.b.y; x[6] = r.b.z; x[7] = r.b.w;
}
__device__ __forceinline__ void unpack8(const uint4& r, float (&x)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
// The largest magnitude of n chunks (fp32 bits), with infinities and NaN as
// they are, the larger; on bf16 pairs as they are in memory.
template <int N>
__device__ __forceinline__ uint32_t max_bits(const Raw8f (&r)[N]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float x[8];
    unpack8(r[i], x);
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(x[e]) & 0x7fffffffu);
  }
  return m;
}
template <int N>
__device__ __forceinline__ uint32_t max_bits(const uint4 (&r)[N]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i)
    m = __vmaxu2(m, __vmaxu2(__vmaxu2(r[i].x & 0x7fff7fffu, r[i].y & 0x7fff7fffu), __vmaxu2(r[i].z & 0x7fff7fffu, r[i].w & 0x7fff7fffu)));
  return max(m << 16, m & 0xffff0000u);
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
// Exact: a value with four significant bits times a power of two.
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = (__float_as_uint(x[2 * i]) >> 16) | (__float_as_uint(x[2 * i + 1]) & 0xffff0000u);
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void decode8(uint2 c, float s, float (&x)[8]) {
  const uint32_t w[4] = {c.x, c.x >> 16, c.y, c.y >> 16};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = e4m3x2_to_f32x2(w[i]);
    x[2 * i] = f.x * s;
    x[2 * i + 1] = f.y * s;
  }
}
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv_s) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = f32x2_to_e4m3x2(x[2 * i] * inv_s, x[2 * i + 1] * inv_s);
  return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

// Which page slot of which sequence entry `e` of the call is.  Every sequence
// with tokens has the slots from its first new token's to its last one's.
struct Entry {
  KvSeq s;
  int seq, slot;  // seq < 0: none
};
__device__ __forceinline__ int seq_slots(const KvSeq& s) {
  if (s.n == 0) return 0;
  const int first = max(s.len - s.n, 0);
  return max(1, (s.len + kPage - 1) / kPage - first / kPage);
}
__device__ __forceinline__ Entry find_entry(const KvAppendArgs& a, int e, int (&part)[kThreads / 32], Entry* found) {
  Entry r;
  r.seq = -1;
  if (a.c.cu == nullptr) {
    const int seq = e / a.pages_each, j = e % a.pages_each;
    r.s = kv_seq(a.c, seq);
    if (j < seq_slots(r.s)) {
      r.seq = seq;
      r.slot = max(r.s.len - r.s.n, 0) / kPage + j;
    }
    return r;
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) found->seq = -1;
  int base = 0;
  for (int s0 = 0; s0 < a.c.n_seqs && base <= e; s0 += kThreads) {
    KvSeq s = {0, 0, 0};
    if (s0 + tid < a.c.n_seqs) s = kv_seq(a.c, s0 + tid);
    const int n = seq_slots(s);
    int v = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v += u;
    }
    __syncthreads();
    if (lane == 31) part[warp] = v;
    __syncthreads();
    int total = 0;
    v += base;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      const int p = part[w];
      if (w < warp) v += p;
      total += p;
    }
    if (v - n <= e && e < v) {
      Entry f;
      f.s = s;
      f.seq = s0 + tid;
      f.slot = max(s.len - s.n, 0) / kPage + e - (v - n);
      *found = f;
    }
    base += total;
  }
  __syncthreads();
  return *found;
}

// z of the grid: 0 keys, 1 values.  32 elements a thread, as they are in
// memory, between the maximum and the conversion: 16 registers in bf16, so eight
// CTAs an SM have their 16 KB in flight.  What is not finite is looked for once
// a thread, on pairs, and handled apart: with a test an element the integer
// pipe was busy 79 % of the time.  32768 tokens of 8 heads (201 MB): bf16 32 us,
// 6.3 TB/s (39 with a test an element and six CTAs, 76 with keys and values in
// one CTA, as fp32, 128 registers a thread); fp32 (335 MB) 52 us, 6.4 TB/s.
template <typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 8 : 4) append_kernel(const KvAppendArgs a) {
  __shared__ int part[kThreads / 32];
  __shared__ Entry found;
  __shared__ uint32_t top;
  const int tid = threadIdx.x, h = blockIdx.y;
  const bool values = blockIdx.z != 0;
  if (tid == 0) top = 0;
  grid_dependency_wait();
  grid_launch_dependents();
  const Entry en = find_entry(a, blockIdx.x, part, &found);
  if (en.seq < 0) return;
  const int past = en.s.len - en.s.n;              // position of the first new token
  const int pos0 = en.slot * kPage;
  const int lo = max(past - pos0, 0), hi = min(en.s.len - pos0, kPage);  // rows of the page that are new
  if (hi <= lo) return;  // a sequence of length zero
  // packed token of row r: tok0 + pos0 + r - past
  const int64_t stride = values ? a.v_stride : a.k_stride;
  const T* src = reinterpret_cast<const T*>(values ? a.v : a.k) + ((int64_t)en.s.tok0 + pos0 - past) * stride + h * kHeadDim;
  decltype(load_raw(src)) x[kChunks];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int c = i * kThreads + tid, r = c >> 4;
    zero_raw(x[i]);
    if (r >= lo && r < hi) x[i] = load_raw(src + r * stride + (c & 15) * 8);
  }
  const int page = kv_page(a.c, en.seq, en.slot);
  if (page < 0) return;
  const size_t head = (size_t)page * a.c.h_kv + h;
  float* scale = (values ? a.c.v_scale : a.c.k_scale) + head;
  const float old_s = lo > 0 ? *scale : 0.f;
  uint32_t m = max_bits(x);
  const bool finite = m < 0x7f800000u;
  if (!finite) {  // the finite ones' only
    m = 0;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      float y[8];
      unpack8(x[i], y);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t b = __float_as_uint(y[e]) & 0x7fffffffu;
        m = b < 0x7f800000u ? max(m, b) : m;
      }
    }
  }
  m = __reduce_max_sync(0xffffffffu, m);
  __syncthreads();  // top is zero; everyone has read the scale
  if ((tid & 31) == 0 && m) atomicMax(&top, m);
  __syncthreads();
  const float s = fmaxf(pow2f(min(e4m3_scale_exp(top, kScaleMinExp), kScaleMaxExp)), old_s);
  const float inv = 1.0f / s;  // exact: a power of two
  uint2* codes = reinterpret_cast<uint2*>((values ? a.c.v : a.c.k) + head * kPageBytes);
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int c = i * kThreads + tid, r = c >> 4;
    float y[8];
    if (r >= lo && r < hi) {
      unpack8(x[i], y);
      if (!finite) {
#pragma unroll
        for (int e = 0; e < 8; ++e)  // infinities too become NaN codes
          y[e] = (__float_as_uint(y[e]) & 0x7fffffffu) < 0x7f800000u ? y[e] : __uint_as_float(0x7fffffffu);
      }
      codes[c] = encode8(y, inv);
    } else if (r < lo && s > old_s) {
      decode8(codes[c], old_s, y);
      codes[c] = encode8(y, inv);
    }
  }
  if (tid == 0) *scale = s;
}

// A code and its scale to a value, both exact; each CTA keys and values of one
// (page, head), whose loads are all in flight.  348160 tokens of 2 heads (535 MB):
// 83 us, 6.5 TB/s.
template <typename T>
__global__ void __launch_bounds__(kThreads) read_kernel(const KvAppendArgs a) {
  __shared__ int part[kThreads / 32];
  __shared__ Entry found;
  const int tid = threadIdx.x, h = blockIdx.y;
  grid_dependency_wait();
  grid_launch_dependents();
  const Entry en = find_entry(a, blockIdx.x, part, &found);
  if (en.seq < 0) return;
  const int past = en.s.len - en.s.n, pos0 = en.slot * kPage;
  const int lo = max(past - pos0, 0), hi = min(en.s.len - pos0, kPage);
  const int64_t row0 = (int64_t)en.s.tok0 + pos0 - past;
  if (past < 0 && en.slot == 0) {  // tokens before position 0 read as zeros
    float z[8] = {};
    for (int64_t c = tid; c < (int64_t)(-past) * 16; c += kThreads) {
      const int64_t row = en.s.tok0 + (c >> 4);
      const int col = (int)(c & 15) * 8;
      store8(reinterpret_cast<T*>(a.k) + row * a.k_stride + h * kHeadDim + col, z);
      store8(reinterpret_cast<T*>(a.v) + row * a.v_stride + h * kHeadDim + col, z);
    }
  }
  if (hi <= lo) return;
  const int page = kv_page(a.c, en.seq, en.slot);
  if (page < 0) return;
  const size_t head = (size_t)page * a.c.h_kv + h;
  const float sk = a.c.k_scale[head], sv = a.c.v_scale[head];
  const uint2* ck = reinterpret_cast<const uint2*>(a.c.k + head * kPageBytes);
  const uint2* cv = reinterpret_cast<const uint2*>(a.c.v + head * kPageBytes);
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int c = i * kThreads + tid, r = c >> 4, col = (c & 15) * 8;
    if (r < lo || r >= hi) continue;
    float x[8];
    decode8(__ldg(ck + c), sk, x);
    store8(reinterpret_cast<T*>(a.k) + (row0 + r) * a.k_stride + h * kHeadDim + col, x);
    decode8(__ldg(cv + c), sv, x);
    store8(reinterpret_cast<T*>(a.v) + (row0 + r) * a.v_stride + h * kHeadDim + col, x);
  }
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& a, bool f32, unsigned entries, cudaStream_t st) {
  const dim3 grid(entries, a.c.h_kv, 2);
  return f32 ? launch_kernel(append_kernel<float>, grid, dim3(kThreads), 0, st, true, a)
             : launch_kernel(append_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, st, true, a);
}

cudaError_t launch_kv_read(const KvAppendArgs& a, bool f32, unsigned entries, cudaStream_t st) {
  const dim3 grid(entries, a.c.h_kv);
  return f32 ? launch_kernel(read_kernel<float>, grid, dim3(kThreads), 0, st, true, a)
             : launch_kernel(read_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, st, true, a);
}

}  // namespace gdn
