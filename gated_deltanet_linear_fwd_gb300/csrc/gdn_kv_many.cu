// Attention over the 8-bit key/value cache for many query rows (prompts and
// pieces of prompts): bound by the tensor cores, 4 x 128 operations a row and
// key, with the exponentials next.
//
// A CTA takes 256 rows (token, query head of one group) as two tiles of 128
// and walks the keys in tiles of 128 (two pages); each key tile serves both.
//   S [128 rows, 128 keys] = Q K^T: e4m3 operands.  The keys' codes enter as
//     they are; a bf16 query row, scaled by a power of two so that its largest
//     magnitude is in (224, 448], is the sum of two e4m3 rows (four leading
//     bits, then the remaining four, exact to 2^-17.8 of the row's largest, so
//     that elements below 2^-10 of it keep fewer than their eight bits: the low
//     part has no factor of its own, since both share one accumulator).
//     Both accumulate into one S: as many steps as one bf16 product.
//   O [128 rows, 128 d] += P V: fp16 operands.  The values' codes are exact in
//     fp16 and converted once per CTA by a warpgroup of their own; the weights
//     P are rounded to fp16's 11 bits.
// Converting only the values keeps the conversion (48 KB of shared-memory
// traffic a tile) beside the products' own reads; splitting P into two e4m3
// parts instead would cost the softmax warps four more instructions a weight.
//
// Softmax: a thread owns a row.  x_j = scale log2(e) q . k_j; the values' page
// scale 2^e_v is folded into the exponent, P_j = 2^(x_j + e_v - m + 3), so P times
// the codes is the output in units of 2^(m - 3); the softmax's sum is of P_j 2^-e_v in
// fp32.  m follows the running maximum of x + e_v only when that has grown by
// more than 12, so O in tensor memory is rarely rescaled; P stays below 2^15,
// within fp16, which keeps fewer than eleven bits of weights below 2^-17 of 2^m
// and none of those below 2^-28; the sum counts them all.
//
// Tensor memory (512 columns): S of either tile (P over its middle) and O
// of either tile.  Each tile has an MMA warp that alternates P V of
// the previous keys with Q K^T of the next; one tile's softmax runs under the
// other's products.
//
// A prompt of 32768 tokens, 8 query heads on 2: 1495 us, 1.47 PFLOP/s (76 % of a
// bf16 library product); 2048 tokens over 67584, 16 heads on 2: 753 us.  The
// tensor pipe is busy 64 % of the time; the way from scores to weights is
// what the other tile's products do not hide completely.  Registers set the
// limit: 176 a softmax thread instead of 184 cost 3 %, 168 a third.
#include <cuda_fp16.h>

#include "gdn_dev.cuh"
#include "gdn_kv.cuh"

namespace gdn {
namespace {

constexpr int kRows = 256;
constexpr int kThreads = 512;  // two softmax warpgroups, one converting values, one of TMA and MMA warps
constexpr int kValuesWarp = 8, kTmaWarp = 12, kMmaWarp = 13;  // MMA warps 13 and 14
constexpr int kSoftRegs = 184, kOtherRegs = 72;  // 256 x 184 + 256 x 72 = 512 x 128, the registers at launch
constexpr int kTileBytes = kKvTile * kHeadDim;
constexpr int kKStages = 3, kVStages = 2, kHStages = 2, kScaleRing = 8;

constexpr uint32_t kOffQ = 0;                                  // tile, part (hi, lo): 16 KB each
constexpr uint32_t kOffK = kOffQ + 4 * kTileBytes;
constexpr uint32_t kOffV = kOffK + kKStages * kTileBytes;
constexpr uint32_t kOffH = kOffV + kVStages * kTileBytes;      // fp16 values: two panels of 64 columns
constexpr uint32_t kSmem = kOffH + kHStages * 2 * kTileBytes + 1024;

constexpr uint32_t kColS = 0, kColO = 256;  // + 128 for the second tile
constexpr uint32_t kColP = 32;              // P, two weights a column, within S

enum { kBarK = 1, kBarV, kBarKFree, kBarVFree, kBarQ, kBarS, kBarP, kBarO, kBarScale, kBarH, kBarHFree };

struct ManyCtl {
  uint64_t k_full[kKStages], k_free[kKStages], v_full[kVStages], v_free[kVStages], h_full[kHStages], h_free[kHStages];
  uint64_t q_full[2], s_full[2], p_full[2][2], o_full[2], scale_full[kScaleRing];
  alignas(16) float scale[kScaleRing][4];  // key scales of the tile's two pages, value scales
  uint32_t nan_keys[kHStages][4];   // keys of a masked tile whose values hold a NaN code
  KvRunScratch run;
  uint32_t tmem;
  int abort;
};

// What every role derives from an item.
struct ManyItem {
  int past;            // position of the first new token
  int all_lo, all_hi;  // keys that every live row attends to
  int q_tiles;         // 1 when the second tile has no rows
};
__device__ __forceinline__ ManyItem many_item(const KvAttnArgs& a, const KvCursor& c) {
  ManyItem m;
  const int r0 = c.rt * kRows, t0 = r0 / a.group, t1 = min(c.it.n - 1, (r0 + kRows - 1) / a.group);
  m.past = c.it.len - c.it.n;
  m.all_lo = kv_window_begin(m.past + t1, a.window);
  m.all_hi = a.causal ? min(m.past + t0 + 1, c.it.len) : c.it.len;
  m.q_tiles = c.it.n * a.group - r0 > 128 ? 2 : 1;
  return m;
}

// ---------------------------------------------------------------- TMA warp
__device__ __forceinline__ void many_load(const KvAttnArgs& a, ManyCtl* ctl, uint8_t* sm,
                                          const CUtensorMap* kmap, const CUtensorMap* vmap) {
  const int lane = threadIdx.x & 31;
  int i = 0;
  KvCursor cur;
#pragma unroll 1
  for (cur.start(a, ctl->run.run); cur.valid(); cur.next(a)) {
    const int tiles = cur.tiles();
    int page = -1, next_page = -1;
    float sk = 1.f, sv = 1.f, next_sk = 1.f, next_sv = 1.f;
    // 16 tiles' pages and scales at a time, one batch ahead: lane 2 i + j holds page j of tile i
    auto fetch = [&](int b) {
      const int slot = 2 * (cur.tile_begin() + 16 * b) + lane;
      next_page = -1;
      next_sk = next_sv = 1.f;
      if (16 * b + (lane >> 1) < tiles && slot * kPage < cur.it.len) {
        next_page = max(kv_page(a.c, cur.seq, slot), 0) * a.c.h_kv + cur.head;
        next_sk = a.c.k_scale[next_page];
        next_sv = a.c.v_scale[next_page];
      }
    };
    fetch(0);
#pragma unroll 1
    for (int b = 0; 16 * b < tiles; ++b) {
      page = next_page;
      sk = next_sk;
      sv = next_sv;
      fetch(b + 1);
      const int n = min(16, tiles - 16 * b);
#pragma unroll 1
      for (int j = 0; j < n; ++j, ++i) {
        const int ks = i % kKStages, vs = i % kVStages;
        const int p0 = __shfl_sync(0xffffffffu, page, 2 * j), p1 = __shfl_sync(0xffffffffu, page, 2 * j + 1);
        // a tile's second page may lie past the sequence: its rows keep what they hold and are masked
        const uint32_t bytes = p1 >= 0 ? kTileBytes : kTileBytes / 2;
        if (!kv_wait_warp([&] { return kv_wait(&ctl->k_free[ks], ((i / kKStages) & 1) ^ 1, &ctl->abort, 100 + kBarKFree); })) return;
        if ((lane >> 1) == j) {
          float* s = ctl->scale[i % kScaleRing];
          s[lane & 1] = sk;
          s[2 + (lane & 1)] = sv;
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&ctl->scale_full[i % kScaleRing]);
          uint8_t* dst = sm + kOffK + ks * kTileBytes;
          mbar_arrive_expect_tx(&ctl->k_full[ks], bytes);
          tma_load_3d(dst, kmap, &ctl->k_full[ks], 0, 0, p0);
          if (p1 >= 0) tma_load_3d(dst + kTileBytes / 2, kmap, &ctl->k_full[ks], 0, 0, p1);
        }
        if (!kv_wait_warp([&] { return kv_wait(&ctl->v_free[vs], ((i / kVStages) & 1) ^ 1, &ctl->abort, 100 + kBarVFree); })) return;
        if (lane == 0) {
          uint8_t* dst = sm + kOffV + vs * kTileBytes;
          mbar_arrive_expect_tx(&ctl->v_full[vs], bytes);
          tma_load_3d(dst, vmap, &ctl->v_full[vs], 0, 0, p0);
          if (p1 >= 0) tma_load_3d(dst + kTileBytes / 2, vmap, &ctl->v_full[vs], 0, 0, p1);
        }
      }
    }
  }
}

// ---------------------------------------------------------------- MMA warps, one a query tile
// One tile's waits run under the other tile's products.  The whole warp walks
// the loop, so addresses and descriptors stay in uniform registers, and one
// elected lane issues: a loop of one lane alone takes some 50 instructions an
// MMA, which the softmax warps' issue slots stretch from 64 to over 300
// cycles; this form takes about 20.
__device__ __forceinline__ void many_mma(const KvAttnArgs& a, ManyCtl* ctl, uint32_t sm, uint32_t tmem_any, int q) {
  constexpr uint32_t kIdS = idesc_e4m3(128, 128, false, false), kIdO = idesc_f16(128, 128, false, true);
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_any, 0);
  const uint32_t d_s = tmem + kColS + q * 128, d_o = tmem + kColO + q * 128;
  const uint64_t dq = sdesc_sw128(sm + kOffQ + q * 2 * kTileBytes, 0, 1024), dk = sdesc_sw128(sm + kOffK, 0, 1024);
  const uint64_t dh = sdesc_sw128(sm + kOffH, kTileBytes, 1024);
  const bool issue = elect_one();
  int ks = 0, hs = 1;                     // stages of the current key tile, and of the one before
  uint32_t k_par = 0, h_par = 1;          // and the parities of their barriers
  uint32_t p_par = 1, q_par = 0;          // weights of the tile before; queries
  KvCursor cur;
#pragma unroll 1
  for (cur.start(a, ctl->run.run); cur.valid(); cur.next(a)) {
    const int tiles = __shfl_sync(0xffffffffu, cur.tiles(), 0);
    if (tiles == 0) continue;
    const bool mine = __shfl_sync(0xffffffffu, (int)(q < many_item(a, cur).q_tiles), 0);
#pragma unroll 1
    for (int j = 0; j <= tiles; ++j) {
      // copies this step needs; long complete as a rule, and out of the way of the weights' wait
      if (j > 0 && !kv_wait_warp([&] { return kv_wait(&ctl->h_full[hs], h_par, &ctl->abort, 100 + kBarH); })) return;
      if (j < tiles && !kv_wait_warp([&] { return kv_wait(&ctl->k_full[ks], k_par, &ctl->abort, 100 + kBarK); })) return;
      if (mine) {
        if (j > 0) {  // O += P V as the weights of the key tile before come, the second page's first
          const uint64_t h = dh + hs * (2 * kTileBytes >> 4);
          if (!kv_wait_warp([&] { return kv_wait(&ctl->p_full[q][1], p_par, &ctl->abort, 100 + kBarP); })) return;
          tc_fence_after();
          if (issue) {
#pragma unroll
            for (int k = 4; k < 8; ++k)  // 16 keys a step
              mma_f16_ts(d_o, d_s + kColP + 8 * k, h + k * 128, kIdO, k > 4 || j > 1);
          }
          if (!kv_wait_warp([&] { return kv_wait(&ctl->p_full[q][0], p_par, &ctl->abort, 100 + kBarP); })) return;
          tc_fence_after();
          if (issue) {
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_f16_ts(d_o, d_s + kColP + 8 * k, h + k * 128, kIdO, 1);
            if (j == tiles) mma_commit(&ctl->o_full[q]);
          }
        } else {
          if (!kv_wait_warp([&] { return kv_wait(&ctl->q_full[q], q_par, &ctl->abort, 100 + kBarQ); })) return;
          tc_fence_after();
        }
        if (j < tiles && issue) {
          const uint64_t kk = dk + ks * (kTileBytes >> 4);
#pragma unroll
          for (int k = 0; k < 8; ++k)  // four steps with the high parts, four with the low ones
            mma_f8(d_s, dq + (k >> 2) * (kTileBytes >> 4) + (k & 3) * 2, kk + (k & 3) * 2, kIdS, k > 0);
          mma_commit(&ctl->s_full[q]);  // says too that the products with earlier values are done
        }
        if (j < tiles) p_par ^= 1;
      }
      // without products of its own in the item this only counts the stages on
      if (issue) {
        if (j < tiles) mma_commit(&ctl->k_free[ks]);
        if (j > 0) mma_commit(&ctl->h_free[hs]);
      }
      __syncwarp();
      if (j < tiles) {
        if (++ks == kKStages) {
          ks = 0;
          k_par ^= 1;
        }
        if (++hs == kHStages) {
          hs = 0;
          h_par ^= 1;
        }
      }
    }
    if (mine) q_par ^= 1;
  }
}

// ---------------------------------------------------------------- values to fp16
// Thread = key of the tile.  Four codes to four fp16 by the hardware's exact
// conversion; 16 codes are a 16-byte chunk of the e4m3 tile and two chunks of
// a panel of the fp16 tile, both in the swizzled image (conflict-free).
__device__ __forceinline__ void many_values(const KvAttnArgs& a, ManyCtl* ctl, uint8_t* sm) {
  const int tid = threadIdx.x & 127, lane = tid & 31, warp = tid >> 5;
  int i = 0;
  KvCursor cur;
#pragma unroll 1
  for (cur.start(a, ctl->run.run); cur.valid(); cur.next(a)) {
    const int tiles = cur.tiles();
    if (tiles == 0) continue;
    const ManyItem mi = many_item(a, cur);
#pragma unroll 1
    for (int j = 0; j < tiles; ++j, ++i) {
      const int vs = i % kVStages, hs = i % kHStages;
      const int key0 = (cur.tile_begin() + j) * kKvTile, key = key0 + tid;
      const bool masked = key0 < mi.all_lo || key0 + kKvTile > mi.all_hi;
      if (!kv_wait_warp([&] {
            return kv_wait(&ctl->v_full[vs], (i / kVStages) & 1, &ctl->abort, 100 + kBarV) &&
                   kv_wait(&ctl->h_free[hs], ((i / kHStages) & 1) ^ 1, &ctl->abort, 100 + kBarHFree);
          }))
        return;
      const uint8_t* v = sm + kOffV + vs * kTileBytes;
      uint8_t* h = sm + kOffH + hs * 2 * kTileBytes;
      uint32_t keep = 0xffffffffu;
      if (masked) {
        // Values no row may use must not meet a zero weight as NaN: a key past
        // the sequence, or one that holds a NaN code, becomes zeros; the rows
        // that do attend to the latter become NaN in the softmax.
        uint32_t carry = 0;
#pragma unroll 2
        for (int c = 0; c < 8; ++c) {  // b & 0x7f = 0x7f: adding 1 to the low seven bits carries into the eighth
          const uint4 w = *reinterpret_cast<const uint4*>(v + sw128_offset(tid, c));
          carry |= ((w.x & 0x7f7f7f7fu) + 0x01010101u) | ((w.y & 0x7f7f7f7fu) + 0x01010101u) |
                   ((w.z & 0x7f7f7f7fu) + 0x01010101u) | ((w.w & 0x7f7f7f7fu) + 0x01010101u);
        }
        const bool nan = (carry & 0x80808080u) != 0;
        const uint32_t word = __ballot_sync(0xffffffffu, nan && key < cur.it.len);
        if (lane == 0) ctl->nan_keys[hs][warp] = word;
        if (nan || key >= cur.it.len) keep = 0;
      }
#pragma unroll 2
      for (int c = 0; c < 8; ++c) {
        const uint4 w = *reinterpret_cast<const uint4*>(v + sw128_offset(tid, c));
        const uint32_t u[4] = {w.x & keep, w.y & keep, w.z & keep, w.w & keep};
        uint32_t f[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f[2 * e]) : "h"((uint16_t)u[e]));
          asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f[2 * e + 1]) : "h"((uint16_t)(u[e] >> 16)));
        }
        uint8_t* panel = h + (c >> 2) * kTileBytes;
        *reinterpret_cast<uint4*>(panel + sw128_offset(tid, 2 * (c & 3))) = make_uint4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<uint4*>(panel + sw128_offset(tid, 2 * (c & 3) + 1)) = make_uint4(f[4], f[5], f[6], f[7]);
      }
      kv_arrive_warp(&ctl->v_free[vs]);
      fence_proxy_async_smem();
      kv_arrive_warp(&ctl->h_full[hs]);
    }
  }
}

// ---------------------------------------------------------------- softmax warpgroups
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// Waits for this thread's tensor-memory loads; the fence on 32 registers keeps
// the compiler from using them before.
__device__ __forceinline__ void tmem_ld_done(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29])
               :
               : "memory");
  asm volatile("" : "+r"(r[30]), "+r"(r[31]));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// (a0, a1) * (b, b) + (c, c) and (a0, a1) + (b0, b1) in one instruction each.
__device__ __forceinline__ float2 fma2(float a0, float a1, float b, float c) {
  uint64_t x, y, z, d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a0), "f"(a1));
  asm("mov.b64 %0, {%1, %1};" : "=l"(y) : "f"(b));
  asm("mov.b64 %0, {%1, %1};" : "=l"(z) : "f"(c));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(x), "l"(y), "l"(z));
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(d));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float b0, float b1) {
  uint64_t x, y, d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b0), "f"(b1));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(d));
  return r;
}

constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLazy = 12.f, kLift = 3.f;
constexpr float kLeastFactor = 0x1p-126f;

// Under the masks: -inf for keys outside [lo, hi) of these 32, NaN for keys
// whose values hold one.
__device__ __forceinline__ void mask32(uint32_t (&s)[32], uint32_t nan, int lo, int hi) {
#pragma unroll
  for (int c = 0; c < 32; ++c) {
    if ((nan >> c) & 1) s[c] = 0x7fffffffu;
    if (c < lo || c >= hi) s[c] = 0xff800000u;
  }
}
__device__ __forceinline__ float max32(const uint32_t (&s)[32]) {
  float t[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) t[e] = fmaxf(__uint_as_float(s[e]), __uint_as_float(s[4 + e]));
#pragma unroll
  for (int c = 8; c < 32; c += 8)
#pragma unroll
    for (int e = 0; e < 4; ++e) t[e] = max3(t[e], __uint_as_float(s[c + e]), __uint_as_float(s[c + 4 + e]));
  return fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
}
// Weights 2^(s f + bias) of 32 keys to tensor memory as fp16 pairs; adds them to sum.
__device__ __forceinline__ void weights32(uint32_t t_p, const uint32_t (&s)[32], float f, float bias, float2& sum) {
  uint32_t w[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const float2 x = fma2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]), f, bias);
    const float p0 = ex2(x.x), p1 = ex2(x.y);
    sum = add2(sum, p0, p1);
    w[e] = pack_f16x2(p0, p1);
  }
  tmem_st16(t_p, w);
}

// This thread's query row (null: zeros) into its two e4m3 parts in shared
// memory; returns its score factor.
__device__ __forceinline__ float many_query(float scale_log2, const __nv_bfloat16* src, int row, uint8_t* hi_tile) {
  uint4 x[16];
#pragma unroll
  for (int c = 0; c < 16; ++c) x[c] = src ? __ldg(reinterpret_cast<const uint4*>(src) + c) : make_uint4(0, 0, 0, 0);
  // the largest magnitude: bf16 bits without the sign are ordered like integers
  uint32_t m2 = 0;
#pragma unroll
  for (int c = 0; c < 16; ++c)
    m2 = __vmaxu2(m2, __vmaxu2(__vmaxu2(x[c].x & 0x7fff7fffu, x[c].y & 0x7fff7fffu), __vmaxu2(x[c].z & 0x7fff7fffu, x[c].w & 0x7fff7fffu)));
  const uint32_t m = max(m2 << 16, m2 & 0xffff0000u);
  // below 2^-102 a row's scores are zero for any key the cache can hold
  const int ex = m < 0x7f800000u ? e4m3_scale_exp(m, -110) : 0;
  // The row's factor stays positive and finite.  A row that is not finite becomes
  // NaN codes: its scores are NaN, and those under a mask -inf like any other's.
  const float inv = m >= 0x7f800000u ? __int_as_float(0x7fffffff) : scale_log2 < 0.f ? -pow2f(-ex) : pow2f(-ex);
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const uint32_t w[8] = {x[2 * c].x, x[2 * c].y, x[2 * c].z, x[2 * c].w, x[2 * c + 1].x, x[2 * c + 1].y, x[2 * c + 1].z, x[2 * c + 1].w};
    uint32_t hi[8], lo[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) split_e4m3(__uint_as_float(w[e] << 16) * inv, __uint_as_float(w[e] & 0xffff0000u) * inv, hi[e], lo[e]);
    const uint32_t at = sw128_offset(row, c);
    *reinterpret_cast<uint4*>(hi_tile + at) = make_uint4(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16, hi[4] | hi[5] << 16, hi[6] | hi[7] << 16);
    *reinterpret_cast<uint4*>(hi_tile + kTileBytes + at) = make_uint4(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16, lo[4] | lo[5] << 16, lo[6] | lo[7] << 16);
  }
  return pow2f(ex) * fabsf(scale_log2);
}

// Where the epilogue keeps chunk c (16 bytes, of 16) of a warp's row: c < 8 in
// the row's high query part, the others in its low one.
__device__ __forceinline__ uint32_t stage_offset(int row, int c) {
  return (c >> 3) * kTileBytes + sw128_offset(row, c & 7);
}

// The warp's 32 rows of O out of tensor memory: divided by l in bf16, or, for
// a part of an item, as they are.  256 bytes of each row at a time go through
// shared memory, so that a store covers 512 contiguous bytes (a row a thread,
// it took 6000 cycles instead of 4000): through the bytes of the warp's own
// query rows, 128 a row in either part's tile, which no product reads any more.
// The other warps' next queries go to their own rows, so the warps need not
// wait for one another.  dst: this thread's row, or null.
__device__ __forceinline__ void many_output(uint32_t t_o, bool any, bool whole, float l, uint8_t* stage, uint8_t* dst) {
  const int lane = threadIdx.x & 31;
  const float inv = l == 0.f ? 0.f : 1.0f / l;
#pragma unroll 1
  for (int h = 0; h < (whole ? 1 : 2); ++h) {
#pragma unroll 1
    for (int c = 0; c < (whole ? 8 : 4); ++c) {
      uint32_t o[16];
      if (any) {
        tmem_ld16(t_o + 64 * h + 16 * c, o);
        tmem_ld_wait(o);
      }
      if (whole) {
        uint32_t w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          w[k] = !any || l == 0.f ? 0u : pack_bf16x2(__uint_as_float(o[2 * k]) * inv, __uint_as_float(o[2 * k + 1]) * inv);
#pragma unroll
        for (int k = 0; k < 2; ++k)
          *reinterpret_cast<uint4*>(stage + stage_offset(lane, 2 * c + k)) = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<uint4*>(stage + stage_offset(lane, 4 * c + k)) = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
      }
    }
    __syncwarp();
    const int c = lane & 15;
#pragma unroll 2
    for (int k = 0; k < 16; ++k) {
      const int row = 2 * k + (lane >> 4);
      uint8_t* to = reinterpret_cast<uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), row));
      const uint4 v = *reinterpret_cast<const uint4*>(stage + stage_offset(row, c));
      if (to) reinterpret_cast<uint4*>(to + 256 * h)[c] = v;
    }
    __syncwarp();
  }
}

__device__ __forceinline__ void many_softmax(const KvAttnArgs& a, ManyCtl* ctl, uint8_t* sm, uint32_t tmem) {
  const int q = threadIdx.x >> 7, row = threadIdx.x & 127, warp = row >> 5;
  const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
  const uint32_t t_s = tmem + lane_base + kColS + q * 128, t_o = tmem + lane_base + kColO + q * 128;
  int i = 0, n = 0, items = 0;  // key tiles of the run, those this query tile took part in, and its items with keys
  KvCursor cur;
#pragma unroll 1
  for (cur.start(a, ctl->run.run); cur.valid(); cur.next(a)) {
    const KvItem it = cur.it;
    const int tiles = cur.tiles(), first_key = cur.tile_begin() * kKvTile;
    const ManyItem mi = many_item(a, cur);
    if (q >= mi.q_tiles) {
      i += tiles;
      continue;
    }
    const int head0 = kv_first_q_head(a.c, cur.head);
    const int rr = cur.rt * kRows + q * 128 + row, t = rr / a.group, g = rr - t * a.group;
    const bool live = t < it.n && g < kv_first_q_head(a.c, cur.head + 1) - head0;
    float f = 0.f, m = kNegInf, l = 0.f;
    if (tiles > 0) {
      f = many_query(a.scale_log2, live ? reinterpret_cast<const __nv_bfloat16*>(a.q) + (int64_t)(it.tok0 + t) * a.q_stride + (head0 + g) * kHeadDim : nullptr,
                     row, sm + kOffQ + q * 2 * kTileBytes);
      fence_proxy_async_smem();
      kv_arrive_warp(&ctl->q_full[q]);
    }
#pragma unroll 1
    for (int j = 0; j < tiles; ++j, ++i, ++n) {
      const int key0 = first_key + j * kKvTile;
      const bool masked = key0 < mi.all_lo || key0 + kKvTile > mi.all_hi;
      const int stage = i % kHStages;
      if (!kv_wait_warp([&] {
            return kv_wait(&ctl->scale_full[i % kScaleRing], (i / kScaleRing) & 1, &ctl->abort, 100 + kBarScale) &&
                   kv_wait(&ctl->s_full[q], n & 1, &ctl->abort, 100 + kBarS) &&
                   (!masked || kv_wait(&ctl->h_full[stage], (i / kHStages) & 1, &ctl->abort, 100 + kBarH));
          }))
        return;
      tc_fence_after();
      // Four chunks of 32 keys, three of them in registers at a time: all are
      // read for the maximum, and the first once more for its weights.
      uint32_t s0[32], s1[32], s2[32];
      tmem_ld32(t_s, s0);
      tmem_ld32(t_s + 32, s1);
      tmem_ld32(t_s + 64, s2);
      const float4 sc = *reinterpret_cast<const float4*>(ctl->scale[i % kScaleRing]);
      int lo = 0, hi = 0;
      if (masked) {
        const int p = mi.past + t;
        lo = kv_window_begin(p, a.window) - key0;
        hi = (live ? (a.causal ? min(p + 1, it.len) : it.len) : 0) - key0;
      }
      if (masked) {
        // the masked scores back into tensor memory, by one copy of this code
        tmem_ld_done(s0);
        tmem_ld_done(s1);
        tmem_ld_done(s2);
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          tmem_ld32(t_s + 32 * c, s0);
          tmem_ld_done(s0);
          mask32(s0, ctl->nan_keys[stage][c], lo - 32 * c, hi - 32 * c);
          tmem_st32(t_s + 32 * c, s0);
        }
        tmem_st_wait();
        tmem_ld32(t_s, s0);
        tmem_ld32(t_s + 32, s1);
        tmem_ld32(t_s + 64, s2);
      }
      // log2 of the value scales, powers of two
      // The factors have to stay above zero: masked scores are -inf before they
      // meet them.  The product underflows for a tiny or zero query over a page
      // of tiny or zero keys (2^-113 2^-40); 2^-126 in its place keeps those
      // scores, at most 2^26 before it, below 2^-100.
      const float fk0 = fmaxf(f * sc.x, kLeastFactor), ev0 = (float)((int)(__float_as_uint(sc.z) >> 23) - 127);
      const float fk1 = fmaxf(f * sc.y, kLeastFactor), ev1 = (float)((int)(__float_as_uint(sc.w) >> 23) - 127);
      tmem_ld_done(s0);
      tmem_ld_done(s1);
      tmem_ld_done(s2);
      // s is -inf only under a mask, and the factors are positive
      float top0 = max32(s0);
      tmem_ld32(t_s + 96, s0);
      top0 = fmaxf(top0, max32(s1));
      float top1 = max32(s2);
      tmem_ld_done(s0);
      top1 = fmaxf(top1, max32(s0));
      const float top = fmaxf(fmaf(top0, fk0, ev0), fmaf(top1, fk1, ev1));
      const bool grow = top > m + kLazy;
      if (__any_sync(0xffffffffu, grow)) {
        const float alpha = grow ? ex2(m - top) : 1.f;
        if (j > 0) {  // O holds earlier tiles, whose products are done: the scores at hand came after them
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t o[16];
            tmem_ld16(t_o + 16 * c, o);
            tmem_ld_wait(o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st16(t_o + 16 * c, o);
          }
        }
        l *= alpha;
        if (grow) m = top;
      }
      const float ref = (m == kNegInf ? 0.f : m) - kLift;
      // The weights go over scores this thread has read: columns 32 to 95.
      float2 sum0 = make_float2(0.f, 0.f), sum1 = make_float2(0.f, 0.f);
      weights32(t_s + 64, s2, fk1, ev1 - ref, sum1);
      tmem_ld32(t_s, s2);
      weights32(t_s + 80, s0, fk1, ev1 - ref, sum1);
      tmem_st_wait();
      tc_fence_before();
      kv_arrive_warp(&ctl->p_full[q][1]);
      weights32(t_s + 48, s1, fk0, ev0 - ref, sum0);
      tmem_ld_done(s2);
      weights32(t_s + 32, s2, fk0, ev0 - ref, sum0);
      l = fmaf(sum0.x + sum0.y, __int_as_float((254 << 23) - __float_as_int(sc.z)), l);
      l = fmaf(sum1.x + sum1.y, __int_as_float((254 << 23) - __float_as_int(sc.w)), l);
      tmem_st_wait();
      tc_fence_before();
      kv_arrive_warp(&ctl->p_full[q][0]);
    }
    // ---- the row's output ----
    if (tiles > 0) {
      if (!kv_wait_warp([&] { return kv_wait(&ctl->o_full[q], items++ & 1, &ctl->abort, 100 + kBarO); })) return;
      tc_fence_after();
    }
    const int64_t tok = it.tok0 + t;
    const size_t part = (size_t)cur.slot() * kRows + q * 128 + row;
    const bool whole = cur.whole();
    uint8_t* dst = whole ? reinterpret_cast<uint8_t*>(reinterpret_cast<__nv_bfloat16*>(a.out) + tok * a.out_stride + (head0 + g) * kHeadDim)
                         : reinterpret_cast<uint8_t*>(a.o + part * kHeadDim);
    many_output(t_o, tiles > 0, whole, l, sm + kOffQ + q * 2 * kTileBytes + warp * 32 * kHeadDim, whole && !live ? nullptr : dst);
    tc_fence_before();
    if (whole) {
      if (live && a.lse) a.lse[tok * a.c.h_q + head0 + g] = kv_lse(m - kLift, l);
    } else {
      a.ml[part] = make_float2(m - kLift, l);
      if (threadIdx.x == 0 && cur.off == 0)
        kv_desc_put(a, ctl->run.run, cur);
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    attn_many_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                     const __grid_constant__ KvAttnArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ ManyCtl ctl;
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, warp = tid >> 5;
  if (tid == 0) {
    for (int s = 0; s < kKStages; ++s) {
      mbar_init(&ctl.k_full[s], 1);
      mbar_init(&ctl.k_free[s], 2);
    }
    for (int s = 0; s < kVStages; ++s) {
      mbar_init(&ctl.v_full[s], 1);
      mbar_init(&ctl.v_free[s], 4);
      mbar_init(&ctl.h_full[s], 4);
      mbar_init(&ctl.h_free[s], 2);
    }
    for (int q = 0; q < 2; ++q) {
      mbar_init(&ctl.q_full[q], 4);
      mbar_init(&ctl.s_full[q], 1);
      mbar_init(&ctl.p_full[q][0], 4);
      mbar_init(&ctl.p_full[q][1], 4);
      mbar_init(&ctl.o_full[q], 1);
    }
    for (int s = 0; s < kScaleRing; ++s) mbar_init(&ctl.scale_full[s], 1);
    fence_mbar_init();
    ctl.abort = 0;
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }
  if (warp == kTmaWarp) {
    tmem_alloc(&ctl.tmem, 512);
    tmem_relinquish();
  }
  grid_dependency_wait();
  if (tid == 0) kv_desc_none(a);
  kv_run<kThreads>(a, &ctl.run);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem;
  if (warp < kValuesWarp) {
    setmaxnreg_inc<kSoftRegs>();
    many_softmax(a, &ctl, sm, tmem);
  } else {
    setmaxnreg_dec<kOtherRegs>();
    if (warp < kTmaWarp) {
      many_values(a, &ctl, sm);
    } else if (warp == kTmaWarp) {
      many_load(a, &ctl, sm, &kmap, &vmap);
    } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
      many_mma(a, &ctl, smem_u32(sm), tmem, __shfl_sync(0xffffffffu, warp - kMmaWarp, 0));
    }
  }
  __syncwarp();
  grid_launch_dependents();
  tc_fence_before();
  __syncthreads();
  if (ctl.abort) {
    if (tid == 0) report(a.c.status, kDevTimeout, ctl.abort);
    // let copies and MMAs already in flight land before the memory is released
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 2000000ull) {
    }
  }
  __syncthreads();
  if (warp == kTmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

cudaError_t kv_many_setup() {
  return cudaFuncSetAttribute(attn_many_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
}

cudaError_t launch_kv_attn_many(const KvAttnArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap, unsigned grid,
                                cudaStream_t st) {
  return launch_kernel(attn_many_kernel, dim3(grid), dim3(kThreads), kSmem, st, true, kmap, vmap, a);
}

}  // namespace gdn
