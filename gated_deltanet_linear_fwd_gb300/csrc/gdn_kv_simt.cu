// Attention over the 8-bit key/value cache on the CUDA cores in fp32, and
// the kernel that joins the parts of items several CTAs worked on.
//
// For a row (token at position p, query head) and the keys j its masks leave,
// with x_j = scale log2(e) q . k_j: running maximum m and sum l = sum
// 2^(x_j - m), output sum 2^(x_j - m) v_j / l, one pass over the keys, both
// rescaled by 2^(m_old - m) when m grows.
//
// A CTA takes 16 rows of a key/value head's group and one page (64 keys) at a
// time: thread (r, c) forms the scores of row r with keys c, c + 16, ...,
// then columns 8 c .. 8 c + 7 of row r's output.  Bound by shared-memory reads
// (a key or value element feeds 16 rows) and fp32 FMAs.
#include "gdn_kv.cuh"
#include "sm103_ptx.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 16;
constexpr int kKeyStride = kHeadDim + 4;  // floats; rows 4 banks apart
constexpr int kSStride = kPage + 4;

struct SimtSmem {
  float q[kRows][kHeadDim];
  float k[kPage][kKeyStride];
  float v[kPage][kHeadDim];
  float s[kRows][kSStride];
  KvRunScratch run;
};

__device__ __forceinline__ void store4(float* p, float a, float b, float c, float d) {
  *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, float a, float b, float c, float d) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(a, b), pack_bf16x2(c, d));
}

__global__ void __launch_bounds__(kThreads) attn_simt_kernel(const KvAttnArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SimtSmem& sm = *reinterpret_cast<SimtSmem*>(smem_raw);
  const int tid = threadIdx.x, r = tid >> 4, c = tid & 15;
  grid_dependency_wait();
  kv_run<kThreads>(a, &sm.run);
  const KvRun& run = sm.run.run;
  if (a.n_ctas && tid == 0) a.desc[blockIdx.x] = make_int4(-1, 0, 0, 0);
  KvCursor cur;
#pragma unroll 1
  for (cur.start(a, run); cur.valid(); cur.next(a)) {
    const KvItem& it = cur.it;
    // row r of the item: token t of the sequence, query head j
    const int rr = cur.rt * kRows + r, t = rr / a.group;
    const int j = kv_first_q_head(a.c, cur.head) + rr % a.group;
    const bool live = t < it.n && j < kv_first_q_head(a.c, cur.head + 1);
    const int p = it.len - it.n + t;
    const int key_end = live ? (a.causal ? min(p + 1, it.len) : it.len) : 0;
    const int key_begin = a.window > 0 ? max(0, p - a.window + 1) : 0;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e)
      sm.q[r][c + 16 * e] =
          live ? reinterpret_cast<const float*>(a.q)[(int64_t)(it.tok0 + t) * a.q_stride + j * kHeadDim + c + 16 * e]
               : 0.f;
    float m = -__int_as_float(0x7f800000), l = 0.f, o[8] = {};
    const int page_begin = 2 * cur.tile_begin(), page_end = min(page_begin + 2 * cur.tiles(), (it.len + kPage - 1) / kPage);
    for (int pg = page_begin; pg < page_end; ++pg) {
      __syncthreads();
      const int page = kv_page(a.c, cur.seq, pg);
      const size_t head = (size_t)max(page, 0) * a.c.h_kv + cur.head;
      const float sk = a.c.k_scale[head], sv = a.c.v_scale[head];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int ch = i * kThreads + tid, row = ch >> 3, col = (ch & 7) * 16;
        const bool in = pg * kPage + row < it.len;  // rows past the sequence may hold anything
        const uint4 zero = make_uint4(0, 0, 0, 0);
        const uint4 wk = in ? __ldg(reinterpret_cast<const uint4*>(a.c.k + head * kPageBytes) + ch) : zero;
        const uint4 wv = in ? __ldg(reinterpret_cast<const uint4*>(a.c.v + head * kPageBytes) + ch) : zero;
        const uint32_t kk[4] = {wk.x, wk.y, wk.z, wk.w}, vv[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float2 k0 = e4m3x2_to_f32x2(kk[w]), k1 = e4m3x2_to_f32x2(kk[w] >> 16);
          const float2 v0 = e4m3x2_to_f32x2(vv[w]), v1 = e4m3x2_to_f32x2(vv[w] >> 16);
          *reinterpret_cast<float4*>(&sm.k[row][col + 4 * w]) = make_float4(k0.x * sk, k0.y * sk, k1.x * sk, k1.y * sk);
          *reinterpret_cast<float4*>(&sm.v[row][col + 4 * w]) = make_float4(v0.x * sv, v0.y * sv, v1.x * sv, v1.y * sv);
        }
      }
      __syncthreads();
      float x[4] = {};
#pragma unroll 4
      for (int d = 0; d < kHeadDim; d += 4) {
        const float4 q4 = *reinterpret_cast<const float4*>(&sm.q[r][d]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 k4 = *reinterpret_cast<const float4*>(&sm.k[c + 16 * i][d]);
          x[i] = fmaf(q4.x, k4.x, fmaf(q4.y, k4.y, fmaf(q4.z, k4.z, fmaf(q4.w, k4.w, x[i]))));
        }
      }
      float top = m;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = pg * kPage + c + 16 * i;
        x[i] = key >= key_begin && key < key_end ? x[i] * a.scale_log2 : -__int_as_float(0x7f800000);
        top = fmaxf(top, x[i]);
      }
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      const float ref = top == -__int_as_float(0x7f800000) ? 0.f : top;
      const float alpha = exp2f(m - ref);
      l *= alpha;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float w = exp2f(x[i] - ref);
        l += w;
        sm.s[r][c + 16 * i] = w;
      }
      m = top;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] *= alpha;
      __syncwarp();  // a row's 16 threads are in one warp
#pragma unroll 4
      for (int i = 0; i < kPage; ++i) {
        const float w = sm.s[r][i];
        if (w == 0.f) continue;  // a masked value may be NaN
        const float4 v0 = *reinterpret_cast<const float4*>(&sm.v[i][8 * c]);
        const float4 v1 = *reinterpret_cast<const float4*>(&sm.v[i][8 * c + 4]);
        o[0] = fmaf(w, v0.x, o[0]);
        o[1] = fmaf(w, v0.y, o[1]);
        o[2] = fmaf(w, v0.z, o[2]);
        o[3] = fmaf(w, v0.w, o[3]);
        o[4] = fmaf(w, v1.x, o[4]);
        o[5] = fmaf(w, v1.y, o[5]);
        o[6] = fmaf(w, v1.z, o[6]);
        o[7] = fmaf(w, v1.w, o[7]);
      }
    }
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    if (cur.whole()) {
      if (live) {
        const float inv = l == 0.f ? 0.f : 1.0f / l;
        float* dst = reinterpret_cast<float*>(a.out) + (int64_t)(it.tok0 + t) * a.out_stride + j * kHeadDim + 8 * c;
        store4(dst, o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
        store4(dst + 4, o[4] * inv, o[5] * inv, o[6] * inv, o[7] * inv);
        if (a.lse && c == 0) a.lse[(int64_t)(it.tok0 + t) * a.c.h_q + j] = kv_lse(m, l);
      }
    } else {
      const size_t row = (size_t)cur.slot() * kRows + r;
#pragma unroll
      for (int e = 0; e < 8; ++e) a.o[row * kHeadDim + 8 * c + e] = o[e];
      if (c == 0) a.ml[row] = make_float2(m, l);
      if (tid == 0 && cur.off == 0)
        a.desc[blockIdx.x] = make_int4(cur.seq, cur.rt, cur.head, kv_last_cta(a, run, cur));
    }
  }
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
  const int parts = d.w - (int)blockIdx.x + 1;
  // part i: slot 2 c + 1 of the first CTA, slot 2 (c + i) of the others
  auto slot = [&](int i) { return (size_t)(2 * (blockIdx.x + i) + (i == 0 ? 1 : 0)); };
  for (int row0 = blockIdx.y * kRowsPerPass; row0 < a.rows; row0 += gridDim.y * kRowsPerPass) {
    const int row = row0 + warp / kWarps, rr = d.y * a.rows + row, t = rr / a.group, g = rr - t * a.group;
    const bool live = row < a.rows && t < s.n && g < group;
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

cudaError_t kv_simt_setup() {
  return cudaFuncSetAttribute(attn_simt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(SimtSmem));
}

cudaError_t launch_kv_attn_simt(const KvAttnArgs& a, unsigned grid, cudaStream_t st) {
  return launch_kernel(attn_simt_kernel, dim3(grid), dim3(kThreads), sizeof(SimtSmem), st, true, a);
}

cudaError_t launch_kv_combine(const KvAttnArgs& a, bool f32, cudaStream_t st) {
  // Few rows: one wave of blocks (8 fit an SM) over all CTAs' items, and several
  // warps a row, since there the parts are what there is to spread.
  const int y = a.rows <= 16 ? 4 : (a.rows + 7) / 8;
  const dim3 grid(a.n_ctas, y), block(256);
  if (a.rows <= 8)
    return f32 ? launch_kernel(combine_kernel<float, 4>, grid, block, 0, st, true, a)
               : launch_kernel(combine_kernel<__nv_bfloat16, 4>, grid, block, 0, st, true, a);
  if (a.rows <= 16)
    return f32 ? launch_kernel(combine_kernel<float, 2>, grid, block, 0, st, true, a)
               : launch_kernel(combine_kernel<__nv_bfloat16, 2>, grid, block, 0, st, true, a);
  return f32 ? launch_kernel(combine_kernel<float, 1>, grid, block, 0, st, true, a)
             : launch_kernel(combine_kernel<__nv_bfloat16, 1>, grid, block, 0, st, true, a);
}

}  // namespace gdn
