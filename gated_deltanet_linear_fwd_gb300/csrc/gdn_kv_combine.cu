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

// Joins the parts of an item: with M the largest of their maxima m_i and
// f_i = 2^(m_i - M), out = sum f_i o_i / sum f_i l_i.  Block (c, y) looks after
// the item whose first part CTA c made and its rows y, y + gridDim.y, ... a
// warp (or kWarps of them when few rows meet many parts) a row, a lane four
// columns.  The factors come first, a part a lane, so that the outputs' loads
// do not wait for one another.  Reads each part once.
template <typename T, int kWarps>
__global__ void __launch_bounds__(256) combine_kernel(const KvAttnArgs a) {
  constexpr int kRowsPerPass = 8 / kWarps;
  __shared__ float4 so[8][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, w = warp % kWarps;
  grid_dependency_wait();
  const int4 d = a.desc[blockIdx.x];
  if (d.x < 0) return;
  const KvSeq s = kv_seq(a.c, d.x);
  const int head0 = kv_first_q_head(a.c, d.z), group = kv_first_q_head(a.c, d.z + 1) - head0;
  const int rows = min(a.rows, a.max_rows);
  const int parts = d.w - (int)blockIdx.x + 1;
  // part i: slot 2 c + 1 of the first CTA, slot 2 (c + i) of the others
  auto slot = [&](int i) { return (size_t)(2 * (blockIdx.x + i) + (i == 0 ? 1 : 0)); };
  for (int row0 = blockIdx.y * kRowsPerPass; row0 < rows; row0 += gridDim.y * kRowsPerPass) {
    const int row = row0 + warp / kWarps, rr = d.y * a.rows + row, t = rr / a.group, g = rr - t * a.group;
    const bool live = row < rows && t < s.n && g < group;
    float m = -__int_as_float(0x7f800000), l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (live) {
      for (int i = lane; i < parts; i += 32) m = fmaxf(m, a.ml[slot(i) * a.rows + row].x);
#pragma unroll
      for (int e = 16; e > 0; e >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, e));
      const float ref = m == -__int_as_float(0x7f800000) ? 0.f : m;
      for (int i0 = 0; i0 < parts; i0 += 32) {
        float f = 0.f;
        if (i0 + lane < parts) {
          const float2 ml = a.ml[slot(i0 + lane) * a.rows + row];
          f = exp2f(ml.x - ref);
          l += f * ml.y;
        }
        const int n = min(32, parts - i0);
#pragma unroll 8
        for (int i = w; i < n; i += kWarps) {
          const float4 x = __ldcg(reinterpret_cast<const float4*>(a.o + (slot(i0 + i) * a.rows + row) * kHeadDim) + lane);
          const float fi = __shfl_sync(0xffffffffu, f, i);
          o.x = fmaf(x.x, fi, o.x);
          o.y = fmaf(x.y, fi, o.y);
          o.z = fmaf(x.z, fi, o.z);
          o.w = fmaf(x.w, fi, o.w);
        }
      }
#pragma unroll
      for (int e = 16; e > 0; e >>= 1) l += __shfl_xor_sync(0xffffffffu, l, e);
    }
    if (kWarps > 1) {
      so[warp][lane] = o;
      __syncthreads();
      if (w == 0) {
#pragma unroll
        for (int i = 1; i < kWarps; ++i) {
          const float4 x = so[warp + i][lane];
          o = make_float4(o.x + x.x, o.y + x.y, o.z + x.z, o.w + x.w);
        }
      }
      __syncthreads();
      if (w != 0) continue;
    }
    if (!live) continue;
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    T* dst = reinterpret_cast<T*>(a.out) + (int64_t)(s.tok0 + t) * a.out_stride + (head0 + g) * kHeadDim + 4 * lane;
    store4(dst, o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    if (a.lse && lane == 0) a.lse[(int64_t)(s.tok0 + t) * a.c.h_q + head0 + g] = kv_lse(m, l);
  }
}

}  // namespace

cudaError_t launch_kv_combine(const KvAttnArgs& a, bool f32, cudaStream_t st) {
  // Few rows: one wave of blocks (8 fit an SM) over all CTAs' items, and several
  // warps a row, since there the parts are what there is to spread.
  const int rows = a.rows < a.max_rows ? a.rows : a.max_rows;
  const int y = rows <= 16 ? 4 : (rows + 7) / 8;
  const dim3 grid(a.n_ctas, y), block(256);
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
