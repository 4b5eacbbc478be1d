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
#include "gdn_kv_page.cuh"

namespace gdn {
namespace {

constexpr int kThreads = kPageThreads;

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
  append_page<T>(a, en, h, values, top);
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
  for (int i = 0; i < kPageChunks; ++i) {
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
