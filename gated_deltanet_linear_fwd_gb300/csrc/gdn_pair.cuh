// Pairs of fp32 values in one 64-bit register: the packed instructions do two
// multiply-adds an issue slot, and the kernels that use them are otherwise bound
// by issue slots before memory.  Also the approximate functions they use.
#pragma once
#include <cmath>
#include <cstdint>

namespace gdn {

struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ F2 f2(float x) { return f2(x, x); }
__device__ __forceinline__ float2 parts(F2 x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x.v));
  return r;
}
__device__ __forceinline__ F2 swapped(F2 x) {
  const float2 p = parts(x);
  return f2(p.y, p.x);
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ float both(F2 x) {
  const float2 p = parts(x);
  return p.x + p.y;
}

// To 2 ulp; their arguments here are normal numbers (or, of ex2 and rcp, results
// below the normal numbers may become zero).
__device__ __forceinline__ float ex2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rsqrt_approx(float x) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// A sum in two fp32, what the additions round off in the second [Knuth's sum of two
// numbers and its exact error]: 64-bit additions issue at a small fraction of the rate.
struct Sum2 {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float x) {
    const float t = __fadd_rn(hi, x), z = __fsub_rn(t, hi);
    lo += __fsub_rn(hi, __fsub_rn(t, z)) + __fsub_rn(x, z);
    hi = t;
  }
  __device__ __forceinline__ void add(const Sum2& s) {
    add(s.hi);
    lo += s.lo;
  }
  __device__ __forceinline__ float value() const { return fabsf(hi) < INFINITY ? hi + lo : hi; }
};

// Two bf16 in a word as fp32 (exact), and back (nearest even).
__device__ __forceinline__ F2 bf16_pair(uint32_t w) { return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
__device__ __forceinline__ uint32_t pair_bf16(F2 x) {
  const float2 p = parts(x);
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(p.y), "f"(p.x));
  return r;
}

// The thread's warp in its block, in a way that the compiler sees is the same for
// all lanes: what follows from it alone is then done once a warp.
__device__ __forceinline__ unsigned warp_index() { return __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0); }

// ---- 16 bytes a lane into shared memory, asynchronously, in groups ----
__device__ __forceinline__ void copy16(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)),
               "l"(reinterpret_cast<uint64_t>(from))
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLater>
__device__ __forceinline__ void copy_wait() {  // all groups but the last kLater are there
  asm volatile("cp.async.wait_group %0;" ::"n"(kLater) : "memory");
}

}  // namespace gdn
