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
// each byte once: a CTA holds its page's new tokens in registers between the
// maximum and the conversion.
#include "gdn_kv.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kChunks = kPage * kHeadDim / 8 / kThreads;  // 8-element chunks a thread holds

constexpr int kScaleMinExp = -40, kScaleMaxExp = 40;

// 8 elements of a row as fp32.
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
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

template <typename T>
__global__ void __launch_bounds__(kThreads) append_kernel(const KvAppendArgs a) {
  __shared__ int part[kThreads / 32];
  __shared__ Entry found;
  __shared__ uint32_t top[2];
  const int tid = threadIdx.x, h = blockIdx.y;
  if (tid < 2) top[tid] = 0;
  grid_dependency_wait();
  grid_launch_dependents();
  const Entry en = find_entry(a, blockIdx.x, part, &found);
  if (en.seq < 0) return;
  const int past = en.s.len - en.s.n;              // position of the first new token
  const int pos0 = en.slot * kPage;
  const int lo = max(past - pos0, 0), hi = min(en.s.len - pos0, kPage);  // rows of the page that are new
  if (hi <= lo) return;  // a sequence of length zero
  const int page = kv_page(a.c, en.seq, en.slot);
  if (page < 0) return;
  const size_t head = (size_t)page * a.c.h_kv + h;
  const float old_k = a.c.k_scale[head], old_v = a.c.v_scale[head];
  __syncthreads();  // top is zero

  // packed token of row r: tok0 + pos0 + r - past
  const int64_t row0 = (int64_t)en.s.tok0 + pos0 - past;
  float x[2][kChunks][8];
  uint32_t m[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int c = i * kThreads + tid, r = c >> 4, col = (c & 15) * 8;
    if (r >= lo && r < hi) {
      load8(reinterpret_cast<const T*>(a.k) + (row0 + r) * a.k_stride + h * kHeadDim + col, x[0][i]);
      load8(reinterpret_cast<const T*>(a.v) + (row0 + r) * a.v_stride + h * kHeadDim + col, x[1][i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[0][i][e] = x[1][i][e] = 0.f;
    }
  }
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t b = __float_as_uint(x[w][i][e]) & 0x7fffffffu;
        if (b < 0x7f800000u)
          m[w] = max(m[w], b);
        else
          x[w][i][e] = __uint_as_float(0x7fffffffu);  // infinities too become NaN codes
      }
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const uint32_t mw = __reduce_max_sync(0xffffffffu, m[w]);
    if ((tid & 31) == 0 && mw) atomicMax(&top[w], mw);
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const float old_s = w ? old_v : old_k;
    uint8_t* codes = (w ? a.c.v : a.c.k) + head * kPageBytes;
    float s = pow2f(min(e4m3_scale_exp(top[w], kScaleMinExp), kScaleMaxExp));
    if (lo > 0) s = fmaxf(s, old_s);
    const float inv = 1.0f / s;  // exact: a power of two
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int c = i * kThreads + tid, r = c >> 4;
      if (r >= lo && r < hi) {
        *reinterpret_cast<uint2*>(codes + (size_t)c * 8) = encode8(x[w][i], inv);
      } else if (r < lo && s > old_s) {
        float y[8];
        uint2* at = reinterpret_cast<uint2*>(codes + (size_t)c * 8);
        decode8(*at, old_s, y);
        *at = encode8(y, inv);
      }
    }
    if (tid == 0) (w ? a.c.v_scale : a.c.k_scale)[head] = s;
  }
}

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
  const dim3 grid(entries, a.c.h_kv);
  return f32 ? launch_kernel(append_kernel<float>, grid, dim3(kThreads), 0, st, true, a)
             : launch_kernel(append_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, st, true, a);
}

cudaError_t launch_kv_read(const KvAppendArgs& a, bool f32, unsigned entries, cudaStream_t st) {
  const dim3 grid(entries, a.c.h_kv);
  return f32 ? launch_kernel(read_kernel<float>, grid, dim3(kThreads), 0, st, true, a)
             : launch_kernel(read_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, st, true, a);
}

}  // namespace gdn
