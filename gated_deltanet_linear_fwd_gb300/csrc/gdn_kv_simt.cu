// Attention over the 8-bit key/value cache on the CUDA cores in fp32, and
// the kernel that joins the parts of items several CTAs worked on.
//
// For a row (token at position p, query head) and the keys j its masks leave,
// with x_j = scale log2(e) q . k_j: running maximum m and sum l = sum
// 2^(x_j - m), output sum 2^(x_j - m) v_j / l, one pass over the keys, both
// rescaled by 2^(m_old - m) when m grows.
//
// A CTA takes 16 kR rows of a key/value head's group and one page (64 keys) at
// a time: thread (y, x) forms the scores of rows y, y + 16, ... with keys x,
// x + 16, x + 32, x + 48, then columns 4 x .. and 64 + 4 x .. of those rows' output.
// Bound by shared-memory reads, and those by kR: 4 + kR 16-byte reads feed 16 kR
// FMAs.  kR is 4 where there are the rows for it, 1 for a few (one token's
// group, a long axis).  Keys and values take turns in one buffer, so two CTAs
// fit an SM.
#include "gdn_kv.cuh"
#include "sm103_ptx.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kKeyStride = kHeadDim + 4;  // floats; rows 4 banks apart
constexpr int kSStride = kPage + 4;

template <int kR>
struct SimtSmem {
  float q[16 * kR][kHeadDim];
  float kv[kPage][kKeyStride];
  float s[16 * kR][kSStride];
  KvRunScratch run;
};

constexpr float kNegInf = -__builtin_huge_valf();

// A page's codes of one head as fp32; rows past the sequence, which may hold anything, as zeros.
__device__ __forceinline__ void load_page(float (&dst)[kPage][kKeyStride], const uint8_t* codes, float scale, int rows) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int ch = i * kThreads + (int)threadIdx.x, row = ch >> 3, col = (ch & 7) * 16;
    const uint4 w4 = row < rows ? __ldg(reinterpret_cast<const uint4*>(codes) + ch) : make_uint4(0, 0, 0, 0);
    const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 a = e4m3x2_to_f32x2(w[e]), b = e4m3x2_to_f32x2(w[e] >> 16);
      *reinterpret_cast<float4*>(&dst[row][col + 4 * e]) = make_float4(a.x * scale, a.y * scale, b.x * scale, b.y * scale);
    }
  }
}

__device__ __forceinline__ void store4(float* p, float a, float b, float c, float d) {
  *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, float a, float b, float c, float d) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(a, b), pack_bf16x2(c, d));
}

template <int kR>
__global__ void __launch_bounds__(kThreads, 2) attn_simt_kernel(const KvAttnArgs a) {
  constexpr int kRows = 16 * kR;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SimtSmem<kR>& sm = *reinterpret_cast<SimtSmem<kR>*>(smem_raw);
  const int tid = threadIdx.x, y = tid >> 4, x = tid & 15;
  grid_dependency_wait();
  kv_run<kThreads>(a, &sm.run);
  const KvRun& run = sm.run.run;
  if (a.n_ctas && tid == 0) a.desc[blockIdx.x] = make_int4(-1, 0, 0, 0);
  KvCursor cur;
#pragma unroll 1
  for (cur.start(a, run); cur.valid(); cur.next(a)) {
    const KvItem it = cur.it;
    const int head0 = kv_first_q_head(a.c, cur.head), group = kv_first_q_head(a.c, cur.head + 1) - head0;
    // row y + 16 i of the item: token t of the sequence, query head head0 + g
    int t[kR], g[kR], key_begin[kR], key_end[kR];
    bool live[kR];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      const int rr = cur.rt * kRows + y + 16 * i;
      t[i] = rr / a.group;
      g[i] = rr - t[i] * a.group;
      live[i] = t[i] < it.n && g[i] < group;
      const int p = it.len - it.n + t[i];
      key_end[i] = live[i] ? (a.causal ? min(p + 1, it.len) : it.len) : 0;
      key_begin[i] = a.window > 0 ? max(0, p - a.window + 1) : 0;
      const float* src = reinterpret_cast<const float*>(a.q) + (int64_t)(it.tok0 + t[i]) * a.q_stride + (head0 + g[i]) * kHeadDim;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        *reinterpret_cast<float4*>(&sm.q[y + 16 * i][4 * x + 64 * e]) =
            live[i] ? __ldg(reinterpret_cast<const float4*>(src + 4 * x + 64 * e)) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float m[kR], l[kR], o[kR][8];
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      m[i] = kNegInf;
      l[i] = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[i][e] = 0.f;
    }
    const int page_begin = 2 * cur.tile_begin(), page_end = min(page_begin + 2 * cur.tiles(), (it.len + kPage - 1) / kPage);
#pragma unroll 1
    for (int pg = page_begin; pg < page_end; ++pg) {
      const int page = kv_page(a.c, cur.seq, pg), rows = it.len - pg * kPage;
      const size_t head = (size_t)max(page, 0) * a.c.h_kv + cur.head;
      __syncthreads();
      load_page(sm.kv, a.c.k + head * kPageBytes, a.c.k_scale[head], rows);
      __syncthreads();
      float s[kR][4];
#pragma unroll
      for (int i = 0; i < kR; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[i][c] = 0.f;
#pragma unroll 2
      for (int d = 0; d < kHeadDim; d += 4) {
        float4 k4[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) k4[c] = *reinterpret_cast<const float4*>(&sm.kv[x + 16 * c][d]);
#pragma unroll
        for (int i = 0; i < kR; ++i) {
          const float4 q4 = *reinterpret_cast<const float4*>(&sm.q[y + 16 * i][d]);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            s[i][c] = fmaf(q4.x, k4[c].x, fmaf(q4.y, k4[c].y, fmaf(q4.z, k4[c].z, fmaf(q4.w, k4[c].w, s[i][c]))));
        }
      }
#pragma unroll
      for (int i = 0; i < kR; ++i) {
        float top = m[i];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int key = pg * kPage + x + 16 * c;
          s[i][c] = key >= key_begin[i] && key < key_end[i] ? s[i][c] * a.scale_log2 : kNegInf;
          top = fmaxf(top, s[i][c]);
        }
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float ref = top == kNegInf ? 0.f : top, alpha = exp2f(m[i] - ref);
        m[i] = top;
        l[i] *= alpha;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float w = exp2f(s[i][c] - ref);
          l[i] += w;
          sm.s[y + 16 * i][x + 16 * c] = w;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) o[i][e] *= alpha;
      }
      __syncthreads();  // the keys are read; a row's weights are its half warp's own
      load_page(sm.kv, a.c.v + head * kPageBytes, a.c.v_scale[head], rows);
      __syncthreads();
#pragma unroll 1
      for (int k = 0; k < kPage; k += 4) {
        float w[kR][4];
#pragma unroll
        for (int i = 0; i < kR; ++i) *reinterpret_cast<float4*>(w[i]) = *reinterpret_cast<const float4*>(&sm.s[y + 16 * i][k]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float4 v0 = *reinterpret_cast<const float4*>(&sm.kv[k + c][4 * x]);
          const float4 v1 = *reinterpret_cast<const float4*>(&sm.kv[k + c][64 + 4 * x]);
#pragma unroll
          for (int i = 0; i < kR; ++i) {
            if (w[i][c] == 0.f) continue;  // a masked value may be NaN
            o[i][0] = fmaf(w[i][c], v0.x, o[i][0]);
            o[i][1] = fmaf(w[i][c], v0.y, o[i][1]);
            o[i][2] = fmaf(w[i][c], v0.z, o[i][2]);
            o[i][3] = fmaf(w[i][c], v0.w, o[i][3]);
            o[i][4] = fmaf(w[i][c], v1.x, o[i][4]);
            o[i][5] = fmaf(w[i][c], v1.y, o[i][5]);
            o[i][6] = fmaf(w[i][c], v1.z, o[i][6]);
            o[i][7] = fmaf(w[i][c], v1.w, o[i][7]);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kR; ++i) {
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
      if (cur.whole()) {
        if (live[i]) {
          const float inv = l[i] == 0.f ? 0.f : 1.0f / l[i];
          const int64_t tok = it.tok0 + t[i];
          float* dst = reinterpret_cast<float*>(a.out) + tok * a.out_stride + (head0 + g[i]) * kHeadDim + 4 * x;
          store4(dst, o[i][0] * inv, o[i][1] * inv, o[i][2] * inv, o[i][3] * inv);
          store4(dst + 64, o[i][4] * inv, o[i][5] * inv, o[i][6] * inv, o[i][7] * inv);
          if (a.lse && x == 0) a.lse[tok * a.c.h_q + head0 + g[i]] = kv_lse(m[i], l[i]);
        }
      } else {
        const size_t row = (size_t)cur.slot() * kRows + y + 16 * i;
        store4(a.o + row * kHeadDim + 4 * x, o[i][0], o[i][1], o[i][2], o[i][3]);
        store4(a.o + row * kHeadDim + 4 * x + 64, o[i][4], o[i][5], o[i][6], o[i][7]);
        if (x == 0) a.ml[row] = make_float2(m[i], l[i]);
      }
    }
    if (tid == 0 && !cur.whole() && cur.off == 0)
      a.desc[blockIdx.x] = make_int4(cur.seq, cur.rt, cur.head, kv_last_cta(a, run, cur));
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
  cudaError_t e = cudaFuncSetAttribute(attn_simt_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(SimtSmem<1>));
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(attn_simt_kernel<4>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(SimtSmem<4>));
}

cudaError_t launch_kv_attn_simt(const KvAttnArgs& a, unsigned grid, cudaStream_t st) {
  return a.rows == 16 ? launch_kernel(attn_simt_kernel<1>, dim3(grid), dim3(kThreads), sizeof(SimtSmem<1>), st, true, a)
                      : launch_kernel(attn_simt_kernel<4>, dim3(grid), dim3(kThreads), sizeof(SimtSmem<4>), st, true, a);
}

cudaError_t launch_kv_combine(const KvAttnArgs& a, bool f32, cudaStream_t st) {
  // Few rows: one wave of blocks (8 fit an SM) over all CTAs' items, and several
  // warps a row, since there the parts are what there is to spread.
  const int y = a.rows <= 16 ? 4 : (a.rows + 7) / 8;
  const dim3 grid(a.n_ctas, y), block(256);
  if (a.rows <= 8) return launch_kernel(combine_kernel<__nv_bfloat16, 4>, grid, block, 0, st, true, a);  // bf16 only
  if (a.rows <= 16)
    return f32 ? launch_kernel(combine_kernel<float, 2>, grid, block, 0, st, true, a)
               : launch_kernel(combine_kernel<__nv_bfloat16, 2>, grid, block, 0, st, true, a);
  return f32 ? launch_kernel(combine_kernel<float, 1>, grid, block, 0, st, true, a)
             : launch_kernel(combine_kernel<__nv_bfloat16, 1>, grid, block, 0, st, true, a);
}

}  // namespace gdn
