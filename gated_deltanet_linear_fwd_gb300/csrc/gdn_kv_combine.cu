// The second kernel of an attention call whose key tiles were shared out in
// runs: it joins the parts of items several CTAs worked on.
#include "gdn_kv.cuh"
#include "sm103_ptx.cuh"

namespace gdn {
namespace {

__device__ __forceinline__ void store4(float* p, float a, float b, float c, float d) {
  *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, float a, float b, float c, float d) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(a, b), pack_bf16x2(c, d));
}

constexpr float kNegInf = -__builtin_huge_valf();

// Joins the parts of an item: with M the largest of their maxima m_i and
// f_i = 2^(m_i - M), out = sum f_i o_i / sum f_i l_i.  Block (c, y) looks after
// the item whose first part CTA c made and its rows y, y + gridDim.y, ... at
// kWarps warps a row, a lane four columns.  A warp takes every kWarps-th part,
// in batches of 32 whose maxima and sums are loaded a part a lane, the first
// eight outputs with them; the warps' sums are joined in shared memory.  Reads
// each part once, in a fixed order.  Bound by the latency of its four loads in
// turn (item, maxima, outputs; 6 us with a cold start); 114 parts of 8 rows each,
// four warps a row, took 15 us where every warp read all maxima, batch by batch.
template <typename T, int kWarps>
__global__ void __launch_bounds__(256) combine_kernel(const KvAttnArgs a) {
  __shared__ float4 so[8][32];
  __shared__ float2 sml[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, w = warp % kWarps;
  const int rows_per_pass = (blockDim.x >> 5) / kWarps;
  grid_dependency_wait();
  const int4 d = a.desc[2 * blockIdx.x], seq = a.desc[2 * blockIdx.x + 1];
  if (d.x < 0) return;
  const int head0 = kv_first_q_head(a.c, d.z), group = kv_first_q_head(a.c, d.z + 1) - head0;
  const int rows = min(a.rows, a.max_rows);
  const int parts = d.x - (int)blockIdx.x + 1, mine = (parts - w + kWarps - 1) / kWarps;
  // part i: slot 2 c + 1 of the first CTA, slot 2 (c + i) of the others; this warp's k-th is part w + k kWarps
  auto slot = [&](int k) {
    const int i = w + k * kWarps;
    return (size_t)(2 * (blockIdx.x + i) + (i == 0 ? 1 : 0));
  };
  for (int row0 = blockIdx.y * rows_per_pass; row0 < rows; row0 += gridDim.y * rows_per_pass) {
    const int row = row0 + warp / kWarps, rr = d.y * a.rows + row, t = rr / a.group, g = rr - t * a.group;
    const bool live = row < rows && t < seq.y && g < group;
    float m = kNegInf, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (live) {
      auto part = [&](int k) {
        return __ldcg(reinterpret_cast<const float4*>(a.o + (slot(k) * a.rows + row) * kHeadDim) + lane);
      };
      for (int k0 = 0; k0 < mine; k0 += 32) {
        const int n = min(32, mine - k0);
        float2 ml = make_float2(kNegInf, 0.f);
        if (lane < n) ml = __ldcg(a.ml + slot(k0 + lane) * a.rows + row);
        float4 x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = e < n ? part(k0 + e) : make_float4(0.f, 0.f, 0.f, 0.f);
        float top = ml.x;
#pragma unroll
        for (int e = 16; e > 0; e >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, e));
        top = fmaxf(top, m);
        const float ref = top == kNegInf ? 0.f : top, alpha = exp2f(m - ref), f = exp2f(ml.x - ref);
        m = top;
        l = fmaf(l, alpha, f * ml.y);  // a lane's share
        o = make_float4(o.x * alpha, o.y * alpha, o.z * alpha, o.w * alpha);
#pragma unroll 1
        for (int k = 0; k < n; k += 8) {
          if (k > 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = k + e < n ? part(k0 + k + e) : make_float4(0.f, 0.f, 0.f, 0.f);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float fi = __shfl_sync(0xffffffffu, f, k + e);  // zero past the last
            o.x = fmaf(x[e].x, fi, o.x);
            o.y = fmaf(x[e].y, fi, o.y);
            o.z = fmaf(x[e].z, fi, o.z);
            o.w = fmaf(x[e].w, fi, o.w);
          }
        }
      }
#pragma unroll
      for (int e = 16; e > 0; e >>= 1) l += __shfl_xor_sync(0xffffffffu, l, e);
    }
    if (kWarps > 1) {
      so[warp][lane] = o;
      if (lane == 0) sml[warp] = make_float2(m, l);
      __syncthreads();
      if (w == 0) {
        float top = m;
#pragma unroll
        for (int i = 1; i < kWarps; ++i) top = fmaxf(top, sml[warp + i].x);
        const float ref = top == kNegInf ? 0.f : top, f0 = exp2f(m - ref);
        m = top;
        l *= f0;
        o = make_float4(o.x * f0, o.y * f0, o.z * f0, o.w * f0);
#pragma unroll
        for (int i = 1; i < kWarps; ++i) {
          const float f = exp2f(sml[warp + i].x - ref);
          const float4 x = so[warp + i][lane];
          l = fmaf(sml[warp + i].y, f, l);
          o = make_float4(fmaf(x.x, f, o.x), fmaf(x.y, f, o.y), fmaf(x.z, f, o.z), fmaf(x.w, f, o.w));
        }
      }
      __syncthreads();
      if (w != 0) continue;
    }
    if (!live) continue;
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    T* dst = reinterpret_cast<T*>(a.out) + (int64_t)(seq.x + t) * a.out_stride + (head0 + g) * kHeadDim + 4 * lane;
    store4(dst, o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    if (a.lse && lane == 0) a.lse[(int64_t)(seq.x + t) * a.c.h_q + head0 + g] = kv_lse(m, l);
  }
}

}  // namespace

cudaError_t launch_kv_combine(const KvAttnArgs& a, bool f32, cudaStream_t st) {
  // Few rows: one wave of blocks of four warps (16 fit an SM) over all CTAs'
  // items, and several warps a row, since there the parts are what there is to spread.
  const int rows = a.rows < a.max_rows ? a.rows : a.max_rows;
  const int threads = rows <= 16 ? 128 : 256, y = rows <= 8 ? rows : rows <= 16 ? 8 : (rows + 7) / 8;
  const dim3 grid(a.n_ctas, y), block(threads);
  if (rows <= 8)
    return f32 ? launch_kernel(combine_kernel<float, 4>, grid, block, 0, st, true, a)
               : launch_kernel(combine_kernel<__nv_bfloat16, 4>, grid, block, 0, st, true, a);
  if (rows <= 16)
    return f32 ? launch_kernel(combine_kernel<float, 2>, grid, block, 0, st, true, a)
               : launch_kernel(combine_kernel<__nv_bfloat16, 2>, grid, block, 0, st, true, a);
  return f32 ? launch_kernel(combine_kernel<float, 1>, grid, block, 0, st, true, a)
             : launch_kernel(combine_kernel<__nv_bfloat16, 1>, grid, block, 0, st, true, a);
}

}  // namespace gdn
