// Attention over the 8-bit key/value cache for fp32 queries and outputs.
//
// On the tensor cores, with operands split so that nothing of fp32 is lost
// that its own sums would not lose:
//   S [128 rows, 128 keys] = Q K^T, fp16 operands, fp32 sums.  The keys' codes
//     are exact in fp16.  A query row, scaled by a power of two so that its
//     largest magnitude is in [2^14, 2^15), is the sum of two fp16 rows: the
//     rounded one and the rounded rest, exact to 2^-24 of each element (to
//     2^-39 of the row's largest).
//   O [128 rows, 128 d] = P V, the weights P <= 2^14 split the same way: 22 bits
//     down to 2^-17 of the tile's largest, 2^-39 of that below.
// The low parts come first: the tensor cores' sums lose a little at every step,
// in proportion to what is in them (2000 to 4000 keys, unit queries: relative error
// 4e-7 against 64 bits, 1.1e-6 with the high parts first, 1.2e-6 for fp32 products
// and softmax).
//
// That is twice the products of a bf16 call.  Prompts over themselves, 8 query
// heads on 2: 16384 tokens 1591 us (345 TFLOP/s of the formula), 2048 tokens 53 us;
// as fp32 FMAs on the CUDA cores 2048 tokens took 278 us.  64 sequences of 1024 to
// 8192 tokens, 4 heads: 209 us for 8 rows (1.27 TB/s of codes; 598 with FMAs).
// Bound by the chain of a tile, some 6200 cycles: converting keys 650, scores and
// maximum 700, weights 1200, 2000 in which warp 0 issues the products as they
// run, join and converting values 1100.  With 512 threads, half as much for each,
// the same chain was longer (16384 tokens 1950 us).
//
// Softmax as in the kernel for few rows: x_j = scale log2(e) q . k_j plus the
// log2 of the values' page scale; weights count from their own tile's maximum,
// and tiles are joined in fp32 registers, o <- o 2^(m - m') + O_t 2^(m_t - m').
//
// A CTA of 256 threads takes 128 rows (token, query head of one group) and 128
// keys (two pages) at a time.  Warp w holds rows 32 (w & 3) + lane: their scores
// with the keys of page w >> 2 of the tile, and columns 64 (w >> 2) .. of their
// output.  The threads convert codes as well (thread = half a key's row, a
// register copy of the next tile's codes in flight); warp 0 issues the
// products.  S of the next tile runs under this tile's join and the values'
// conversion.  Rows are taken 128 at a time however few there are; warps without
// rows skip the softmax.
#include <cuda_fp16.h>

#include "gdn_dev.cuh"
#include "gdn_kv.cuh"

namespace gdn {
namespace {

constexpr int kRows = 128;
constexpr int kThreads = 256;
constexpr int kPanel = 128 * 128;  // bytes of 128 rows of 64 fp16

constexpr uint32_t kOffQ = 0;                    // part (high, low), panel of 64 columns
constexpr uint32_t kOffK = kOffQ + 4 * kPanel;   // two tiles
constexpr uint32_t kOffV = kOffK + 4 * kPanel;
constexpr uint32_t kSmem = kOffV + 2 * kPanel + 1024;

constexpr uint32_t kColS = 0, kColO = 128, kColP = 256;  // P: high parts, two a column, then low parts
constexpr uint32_t kTmemCols = 512;
constexpr float kLift = 14.f;  // weights are up to 2^kLift

enum { kBarS = 1, kBarO };

struct F32Ctl {
  uint64_t s_full, o_full;
  uint32_t nan_keys[2][2][4];  // tile, half of the row: keys of a masked tile whose values hold a NaN code
  float top[2][kRows];         // of a row, from either half
  KvRunScratch run;
  uint32_t tmem;
  int abort;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// (x0, x1) = high + low in fp16.
__device__ __forceinline__ void split_f16(float x0, float x1, uint32_t& high, uint32_t& low) {
  high = pack_f16x2(x0, x1);
  const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&high));
  low = pack_f16x2(x0 - h.x, x1 - h.y);
}

constexpr float kNegInf = -__builtin_huge_valf();

// 64 codes of a key, half its row, to a row of an fp16 panel.
__device__ __forceinline__ void convert_row(uint8_t* panel, int row, const uint4 (&w)[4], uint32_t keep) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const uint32_t u[4] = {w[c].x & keep, w[c].y & keep, w[c].z & keep, w[c].w & keep};
    uint32_t f[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f[2 * e]) : "h"((uint16_t)u[e]));
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f[2 * e + 1]) : "h"((uint16_t)(u[e] >> 16)));
    }
    *reinterpret_cast<uint4*>(panel + sw128_offset(row, 2 * c)) = make_uint4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<uint4*>(panel + sw128_offset(row, 2 * c + 1)) = make_uint4(f[4], f[5], f[6], f[7]);
  }
}
__device__ __forceinline__ bool has_nan(const uint4 (&w)[4]) {
  uint32_t carry = 0;
#pragma unroll
  for (int c = 0; c < 4; ++c)  // b & 0x7f = 0x7f: adding 1 to the low seven bits carries into the eighth
    carry |= ((w[c].x & 0x7f7f7f7fu) + 0x01010101u) | ((w[c].y & 0x7f7f7f7fu) + 0x01010101u) |
             ((w[c].z & 0x7f7f7f7fu) + 0x01010101u) | ((w[c].w & 0x7f7f7f7fu) + 0x01010101u);
  return (carry & 0x80808080u) != 0;
}

__global__ void __launch_bounds__(kThreads, 1) attn_f32_kernel(const __grid_constant__ KvAttnArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ F32Ctl ctl;
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int half = warp >> 2, row = tid & 127;  // as a softmax thread
  const int key_row = tid & 127;                // as a converting one: half `half` of this key's row
  if (tid == 0) {
    mbar_init(&ctl.s_full, 1);
    mbar_init(&ctl.o_full, 1);
    fence_mbar_init();
    ctl.abort = 0;
  }
  if (warp == 0) {
    tmem_alloc(&ctl.tmem, kTmemCols);
    tmem_relinquish();
  }
  grid_dependency_wait();
  if (tid == 0) kv_desc_none(a);
  kv_run<kThreads>(a, &ctl.run);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const KvRun& run = ctl.run.run;
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl.tmem, 0);
  const uint32_t t_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
  constexpr uint32_t kIdS = idesc_f16(128, 128, false, false), kIdO = idesc_f16(128, 128, false, true);
  const uint32_t sm32 = smem_u32(sm);
  const uint64_t dq = sdesc_sw128(sm32 + kOffQ, 0, 1024), dk = sdesc_sw128(sm32 + kOffK, 0, 1024);
  const uint64_t dv = sdesc_sw128(sm32 + kOffV, kPanel, 1024);

  uint32_t par = 0;  // of both barriers: one phase a tile
  bool bad = false;
  KvCursor cur;
#pragma unroll 1
  for (cur.start(a, run); cur.valid() && !bad; cur.next(a)) {
    const KvItem& it = cur.it;
    const int past = it.len - it.n, tiles = cur.tiles();
    const int head0 = kv_first_q_head(a.c, cur.head), group = kv_first_q_head(a.c, cur.head + 1) - head0;
    const int r0 = cur.rt * kRows, rows = it.n * a.group - r0;  // rows of the tile: the first min(rows, 128)
    const int rr = r0 + row, t = rr / a.group, g = rr - t * a.group;
    const bool live = t < it.n && g < group;
    const bool idle = (warp & 3) * 32 >= rows;  // no row of this warp
    const int p = past + t;
    const int key_hi = live ? (a.causal ? min(max(p + 1, 0), it.len) : it.len) : 0;
    const int key_lo = kv_window_begin(p, a.window);
    // tiles within every live row's keys need no mask
    const int t0 = r0 / a.group, t1 = min(it.n - 1, (r0 + kRows - 1) / a.group);
    const int all_lo = kv_window_begin(past + t1, a.window), all_hi = a.causal ? min(past + t0 + 1, it.len) : it.len;
    auto masked = [&](int j) {
      const int k0 = (cur.tile_begin() + j) * kKvTile;
      return k0 < all_lo || k0 + kKvTile > all_hi;
    };

    float o[64], l = 0.f, m = kNegInf, f = 0.f;
#pragma unroll
    for (int d = 0; d < 64; ++d) o[d] = 0.f;

    if (tiles > 0) {
      // ---- the codes of a tile on their way: a tile ahead of their use, their pages another tile ahead ----
      int page0 = -1, page1 = -1, next0, next1;  // times heads; -1: past the sequence
      uint4 kc[4], vc[4];
      float sk, sv, next_sk = 1.f, next_sv = 1.f;  // scales of this warp's page
      auto fetch_pages = [&](int j) {
        const int slot = 2 * (cur.tile_begin() + j);
        next0 = j < tiles && slot * kPage < it.len ? max(kv_page(a.c, cur.seq, slot), 0) * a.c.h_kv + cur.head : -1;
        next1 = j < tiles && (slot + 1) * kPage < it.len ? max(kv_page(a.c, cur.seq, slot + 1), 0) * a.c.h_kv + cur.head : -1;
      };
      auto fetch = [&](uint4 (&w)[4], const uint8_t* codes) {
        const int mine = key_row < kPage ? page0 : page1;
        const size_t at = (size_t)max(mine, 0) * kPageBytes + (key_row & (kPage - 1)) * kHeadDim + half * 64;
#pragma unroll
        for (int c = 0; c < 4; ++c) w[c] = mine >= 0 ? __ldg(reinterpret_cast<const uint4*>(codes + at) + c) : make_uint4(0, 0, 0, 0);
      };
      auto fetch_values = [&]() {  // and the scales
        fetch(vc, a.c.v);
        const int of_scale = half ? page1 : page0;
        next_sk = of_scale >= 0 ? a.c.k_scale[of_scale] : 1.f;
        next_sv = of_scale >= 0 ? a.c.v_scale[of_scale] : 1.f;
        page0 = next0;
        page1 = next1;
      };
      uint32_t keep;  // of the values in vc
      // keys of tile j to shared memory; which of its values may be used
      auto convert_keys = [&](int j) {
        uint8_t* panel = sm + kOffK + ((j & 1) * 2 + half) * kPanel;
        convert_row(panel, key_row, kc, 0xffffffffu);
        keep = 0xffffffffu;
        if (masked(j)) {
          // Values no row may use must not meet a zero weight as NaN: a key
          // past the sequence, or half a row that holds a NaN code, becomes
          // zeros; the rows that do attend to the latter become NaN.
          const bool in = (cur.tile_begin() + j) * kKvTile + key_row < it.len, nan = has_nan(vc);
          const uint32_t word = __ballot_sync(0xffffffffu, nan && in);
          if (lane == 0) ctl.nan_keys[j & 1][half][warp & 3] = word;
          if (nan || !in) keep = 0;
        }
      };
      fetch_pages(0);
      page0 = next0;
      page1 = next1;
      fetch_pages(1);
      fetch(kc, a.c.k);
      fetch_values();

      // ---- query rows: thread = 64 columns of one ----
      {
        const float4* src = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(a.q) +
                                                            (int64_t)(it.tok0 + t) * a.q_stride + (head0 + g) * kHeadDim + half * 64);
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float4 w = live ? __ldg(src + c) : make_float4(0.f, 0.f, 0.f, 0.f);
          o[4 * c] = w.x;
          o[4 * c + 1] = w.y;
          o[4 * c + 2] = w.z;
          o[4 * c + 3] = w.w;
        }
#pragma unroll
        for (int d = 0; d < 64; ++d) top = max(top, __float_as_uint(o[d]) & 0x7fffffffu);
        ctl.top[half][row] = __uint_as_float(top);
        __syncthreads();
        top = max(top, __float_as_uint(ctl.top[half ^ 1][row]));
        // below 2^-96 a row's scores are zero for any key the cache can hold
        const int ex = top < 0x7f800000u ? max((int)(top >> 23) - 127 - 14, -110) : 0;
        f = top < 0x7f800000u ? pow2f(ex) * a.scale_log2 : __int_as_float(0x7fffffff);  // a row that is not finite gives NaN
        const float inv = pow2f(-ex);
        uint8_t* panel = sm + kOffQ + half * kPanel;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t high[4], low[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) split_f16(o[8 * c + 2 * e] * inv, o[8 * c + 2 * e + 1] * inv, high[e], low[e]);
          *reinterpret_cast<uint4*>(panel + sw128_offset(row, c)) = make_uint4(high[0], high[1], high[2], high[3]);
          *reinterpret_cast<uint4*>(panel + 2 * kPanel + sw128_offset(row, c)) = make_uint4(low[0], low[1], low[2], low[3]);
        }
#pragma unroll
        for (int d = 0; d < 64; ++d) o[d] = 0.f;
      }
      // products of the elected lane
      auto issue_s = [&](uint32_t buf) {
        const uint64_t k = dk + buf * (2 * kPanel >> 4);
#pragma unroll
        for (int s = 0; s < 16; ++s)  // part (low first), panel, 16 columns
          mma_bf16(tmem + kColS, dq + ((s >> 2) ^ 2) * (kPanel >> 4) + (s & 3) * 2, k + ((s >> 2) & 1) * (kPanel >> 4) + (s & 3) * 2,
                   kIdS, s > 0);
        mma_commit(&ctl.s_full);
      };
      auto issue_o = [&]() {
#pragma unroll
        for (int s = 0; s < 16; ++s)  // part (low first), 16 keys
          mma_f16_ts(tmem + kColO, tmem + kColP + 8 * (s ^ 8), dv + (s & 7) * 128, kIdO, s > 0);
        mma_commit(&ctl.o_full);
      };
      convert_keys(0);
      convert_row(sm + kOffV + half * kPanel, key_row, vc, keep);
      sk = next_sk;
      sv = next_sv;
      fetch_pages(2);
      fetch(kc, a.c.k);
      fetch_values();
      fence_proxy_async_smem();
      tc_fence_before();
      __syncthreads();
      tc_fence_after();
      if (warp == 0) {
        if (elect_one()) issue_s(0);
        __syncwarp();
      }

#pragma unroll 1
      for (int j = 0; j < tiles; ++j) {
        if (j + 1 < tiles) {
          convert_keys(j + 1);
          fetch(kc, a.c.k);
          fetch_pages(j + 3);
        }
        // a warp's lanes agree on what they waited for: its tensor-memory accesses are the whole warp's
        bad |= !kv_wait_warp([&] { return kv_wait(&ctl.s_full, par, &ctl.abort, 100 + kBarS); });
        tc_fence_after();
        const float ev = (float)((int)(__float_as_uint(sv) >> 23) - 127);  // log2 of a power of two
        const float inv_sv = __int_as_float((254 << 23) - __float_as_int(sv));
        float x[64], top = kNegInf;
        if (!idle && !bad) {
#pragma unroll
          for (int c = 0; c < 64; c += 32) {
            uint32_t s0[16], s1[16];
            tmem_ld16(t_lane + kColS + half * 64 + c, s0);
            tmem_ld16(t_lane + kColS + half * 64 + c + 16, s1);
            tmem_ld_wait(s0, s1);
            const float fs = f * sk;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              x[c + e] = fmaf(__uint_as_float(s0[e]), fs, ev);
              x[c + 16 + e] = fmaf(__uint_as_float(s1[e]), fs, ev);
            }
          }
          if (masked(j)) {
            const int k0 = (cur.tile_begin() + j) * kKvTile + half * 64;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const uint32_t nan = ctl.nan_keys[j & 1][0][2 * half + c] | ctl.nan_keys[j & 1][1][2 * half + c];
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const int key = k0 + 32 * c + e;
                const float y = (nan >> e) & 1 ? __int_as_float(0x7fffffff) : x[32 * c + e];
                x[32 * c + e] = key >= key_lo && key < key_hi ? y : kNegInf;
              }
            }
          }
#pragma unroll
          for (int e = 0; e < 64; ++e) top = fmaxf(top, x[e]);
          ctl.top[half][row] = top;
        }
        named_bar_sync(1 + (warp & 3), 64);  // the two warps of these rows
        float alpha = 0.f, beta = 0.f;
        if (!idle && !bad) {
          top = fmaxf(top, ctl.top[half ^ 1][row]);
          const float both = fmaxf(m, top), at = both == kNegInf ? 0.f : both;
          alpha = ex2(m - at);
          beta = ex2(top - at);
          m = both;
          const float ref = kLift - (top == kNegInf ? 0.f : top);
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < 64; c += 32) {
            uint32_t high[16], low[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float w0 = ex2(x[c + 2 * e] + ref), w1 = ex2(x[c + 2 * e + 1] + ref);
              sum[e & 3] += w0 + w1;
              split_f16(w0, w1, high[e], low[e]);
            }
            tmem_st16(t_lane + kColP + half * 32 + c / 2, high);
            tmem_st16(t_lane + kColP + 64 + half * 32 + c / 2, low);
          }
          l = fmaf(l, alpha, ((sum[0] + sum[1]) + (sum[2] + sum[3])) * inv_sv * beta);
          tmem_st_wait();
        }
        sk = next_sk;
        sv = next_sv;
        fence_proxy_async_smem();
        tc_fence_before();
        bad = __syncthreads_or(bad);
        if (bad) break;
        tc_fence_after();
        if (warp == 0) {
          const uint32_t buf = __shfl_sync(0xffffffffu, (j + 1) & 1, 0), more = __shfl_sync(0xffffffffu, j + 1 < tiles, 0);
          if (elect_one()) {
            issue_o();
            if (more) issue_s(buf);
          }
          __syncwarp();
        }
        // values of the next tile, in registers until this tile's product has read its own; then on to the codes after
        bad = !kv_wait_warp([&] { return kv_wait(&ctl.o_full, par, &ctl.abort, 100 + kBarO); });
        par ^= 1;
        tc_fence_after();
        if (j + 1 < tiles) {
          if (!bad) convert_row(sm + kOffV + half * kPanel, key_row, vc, keep);
          fetch_values();
        }
        if (!idle && !bad) {
#pragma unroll
          for (int c = 0; c < 64; c += 32) {
            uint32_t s0[16], s1[16];
            tmem_ld16(t_lane + kColO + half * 64 + c, s0);
            tmem_ld16(t_lane + kColO + half * 64 + c + 16, s1);
            tmem_ld_wait(s0, s1);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              o[c + e] = fmaf(o[c + e], alpha, __uint_as_float(s0[e]) * beta);
              o[c + 16 + e] = fmaf(o[c + 16 + e], alpha, __uint_as_float(s1[e]) * beta);
            }
          }
        }
        tc_fence_before();
      }
      ctl.top[half][row] = l;  // the sum of this half's weights
      bad = __syncthreads_or(bad);
      if (bad) break;
      l = half ? ctl.top[0][row] + l : l + ctl.top[1][row];
      __syncthreads();
    }
    if (live) {
      float4* dst;
      float by = 1.f;
      if (cur.whole()) {
        dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + (int64_t)(it.tok0 + t) * a.out_stride +
                                        (head0 + g) * kHeadDim + half * 64);
        by = l == 0.f ? 0.f : 1.0f / l;
        if (a.lse && half == 0) a.lse[(int64_t)(it.tok0 + t) * a.c.h_q + head0 + g] = kv_lse(m - kLift, l);
      } else {
        const size_t at = (size_t)cur.slot() * kRows + row;
        dst = reinterpret_cast<float4*>(a.o + at * kHeadDim + half * 64);
        if (half == 0) a.ml[at] = make_float2(m - kLift, l);
      }
#pragma unroll
      for (int c = 0; c < 16; ++c)
        dst[c] = make_float4(o[4 * c] * by, o[4 * c + 1] * by, o[4 * c + 2] * by, o[4 * c + 3] * by);
    }
    if (tid == 0 && !cur.whole() && cur.off == 0)
      kv_desc_put(a, run, cur);
  }
  __syncwarp();
  grid_launch_dependents();
  tc_fence_before();
  __syncthreads();
  if (ctl.abort) {
    if (tid == 0) report(a.c.status, kDevTimeout, ctl.abort);
    // let MMAs already in flight land before the memory is released
    const uint64_t start = globaltimer_ns();
    while (globaltimer_ns() - start < 2000000ull) {
    }
  }
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace

cudaError_t kv_f32_setup() {
  return cudaFuncSetAttribute(attn_f32_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
}

cudaError_t launch_kv_attn_f32(const KvAttnArgs& a, unsigned grid, cudaStream_t st) {
  return launch_kernel(attn_f32_kernel, dim3(grid), dim3(kThreads), kSmem, st, true, a);
}

}  // namespace gdn
