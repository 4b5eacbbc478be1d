// Attention over the 8-bit key/value cache for few query rows (one generated
// token, or a few drafted ones, times the heads of a group): up to 32 rows
// meet a long axis, so the call is bound by reading the codes, 256 bytes a
// token and key/value head, from HBM.
//
// The codes go from HBM into the tensor cores as they are.  Keys and values
// are the 128-row operand of both products and the query rows the narrow one:
//   S^T [128 keys, rows]  = K [128 keys, 128 d] . Q^T
//   O^T [128 d, rows]     = V^T [128 d, 128 keys] . P^T
// with e4m3 on both sides (kind::f8f6f4).  A bf16 query row, scaled by a power
// of two so that its largest magnitude is in (224, 448], is the sum of two
// e4m3 rows hi + lo / 16: hi has its four leading bits, lo the remaining four,
// exactly where it is within 2^13 of the row's largest and to 2^-22 of that
// below.  Weights P = 2^(x - m + 8) enter as hi + lo / 16, eight bits (to 2^-8 of
// each weight, relative, down to 2^-14 of the step's largest and to 2^-22 of that
// below; a bf16 weight has 2^-9).  The two parts are columns of one product, so no
// key or value is converted or read twice.
//
// Softmax over the keys x_j = scale log2(e) q . k_j, by steps of one or two
// tiles of 128 keys: thread j of a warpgroup holds key j's column of S^T.  The
// values' page scale 2^e_v (a power of two) is folded into the exponent: with
// m_t the step's maximum of x + e_v, P_j = 2^(x_j + e_v - m_t + 8), so
// P . V-codes is the step's output in units of 2^(m_t - 8), and its sum is of
// P_j 2^-e_v, kept in fp32 from the unrounded P.  Weights count from their own
// step's maximum, so what e4m3 cannot hold is below 2^-22 of that, however many
// keys there are.  Steps are joined in fp32 registers, under the next step's
// second product: o <- o 2^(m - m') + O_t 2^(m_t - m'), m' the larger of m and
// m_t; the two factors of a row are found by one lane and shared.
//
// Roles: a warpgroup of four warps for every 8 rows, one TMA warp, one MMA warp.
// Up to 16 rows two CTAs an SM hide one another's latency.  More rows take one
// CTA with a deeper ring, whose warpgroups issue 40 % of all cycles: there a step of two
// tiles halves what a step costs a row whatever its keys (the maximum, the
// join, the waits).  32 sequences of 1000 to 8192 tokens, 8 heads, 20 rows:
// 56 us (209 MB, 3.8 TB/s), 82 with steps of one tile; with one row tile of 32
// instead of 24 it is 14 % more.  256 sequences of 32 to 32768 tokens, 2 heads, 4
// rows: 107 us (629 MB, 5.9 TB/s) with steps of one tile, some 8 more with two,
// whose second tile waits longer for HBM than it saves.
#include <cuda_fp16.h>

#include "gdn_dev.cuh"
#include "gdn_kv.cuh"

namespace gdn {
namespace {

constexpr int kTileBytes = kKvTile * kHeadDim;  // codes of a tile of keys or values
constexpr int kScaleRing = 8;                   // tiles whose page scales are in shared memory

// Details of the bounded waits (100 + barrier), as in the other kernels.
enum { kBarK = 1, kBarV, kBarKFree, kBarVFree, kBarQ, kBarS, kBarP, kBarO, kBarScale, kBarClean };

constexpr int kRowsWg = 8;                      // query rows of a warpgroup

template <int NR>
struct Few {
  static constexpr int kWgs = NR / kRowsWg;
  static constexpr int kSoft = kWgs * 128;               // softmax threads
  static constexpr int kThreads = kSoft + 64;
  static constexpr int kN = 2 * NR;                      // columns of the products
  static constexpr int kStages = NR > 16 ? 5 : 3;
  static constexpr int kTiles = NR > 16 ? 2 : 1;         // tiles a step takes together
  static constexpr int kCtasPerSm = NR > 16 ? 1 : 2;
  static constexpr uint32_t kColO = 2 * kTiles * kN;     // S of two steps, then O of two
  static constexpr uint32_t kTmemCols = kTiles == 1 ? (NR == 8 ? 64 : 128) : 512;  // a power of two
  static constexpr uint32_t kOffV = kStages * kTileBytes;
  static constexpr uint32_t kOffQ = 2 * kStages * kTileBytes;
  static constexpr uint32_t kOffP = kOffQ + kN * kHeadDim;
  static constexpr uint32_t kPBytes = kN * kKvTile;      // weights of a tile
  static constexpr uint32_t kSmem = kOffP + 2 * kTiles * kPBytes + 1024;  // + alignment
  static_assert(kStages > kTiles, "a step's first product runs ahead of the last step's second one");
};

template <int NR>
struct FewCtl {
  uint64_t k_full[5], k_free[5], v_full[5], v_free[5];
  uint64_t q_full, s_full[2], p_full[2], o_full[2], v_clean[4], scale_full[kScaleRing];
  float4 scale[kScaleRing][2]; // a page's key scale, log2 of its value scale, 1 / value scale
  uint32_t nan_keys[4][4];     // keys of a masked tile whose values hold a NaN code
  alignas(16) float f[NR];     // score factor of a row: its power of two times scale log2(e)
  int key_lo[NR], key_hi[NR];  // keys a row attends to
  alignas(16) float top[Few<NR>::kWgs][2][kRowsWg][4];  // tile maxima of the four warps
  alignas(16) float sum[Few<NR>::kWgs][kRowsWg][4];
  // a warp's copy, by row: what is added to its exponents; the factors of a join
  alignas(16) float ref[Few<NR>::kSoft / 32][kRowsWg];
  alignas(16) float alpha[Few<NR>::kSoft / 32][2][kRowsWg], beta[Few<NR>::kSoft / 32][2][kRowsWg];
  KvRunScratch run;
  uint32_t tmem;
  int abort;
};

// ---------------------------------------------------------------- TMA warp
template <int NR>
__device__ __forceinline__ void few_load(const KvAttnArgs& a, FewCtl<NR>* ctl, uint8_t* sm,
                                         const CUtensorMap* kmap, const CUtensorMap* vmap) {
  using F = Few<NR>;
  const int lane = threadIdx.x & 31;
  // 16 tiles' pages and scales are fetched at a time, one batch ahead: lane 2 i + j holds page j of tile i
  KvCursor ahead;
  int batch = 0;  // of `ahead`'s item
  int page = 0;
  float sk = 0.f, sv = 0.f;
  auto fetch = [&]() {
    const int slot = 2 * (ahead.tile_begin() + 16 * batch) + lane;
    page = -1;
    if (ahead.valid() && 16 * batch + (lane >> 1) < ahead.tiles() && slot * kPage < ahead.it.len) {
      page = max(kv_page(a.c, ahead.seq, slot), 0) * a.c.h_kv + ahead.head;
      sk = a.c.k_scale[page];
      sv = a.c.v_scale[page];
    }
  };
  ahead.start(a, ctl->run.run);
  while (ahead.valid() && ahead.tiles() == 0) ahead.next(a);
  fetch();
  int i = 0;  // tile of the run
  KvCursor cur;
#pragma unroll 1
  for (cur.start(a, ctl->run.run); cur.valid(); cur.next(a)) {
    const int tiles = cur.tiles();
#pragma unroll 1
    for (int b = 0; 16 * b < tiles; ++b) {
      const int my_page = page;
      const float my_sk = sk, my_sv = sv;
      if (16 * (++batch) >= ahead.tiles()) {
        batch = 0;
        do ahead.next(a);
        while (ahead.valid() && ahead.tiles() == 0);
      }
      fetch();
      const int n = min(16, tiles - 16 * b);
#pragma unroll 1
      for (int j = 0; j < n; ++j, ++i) {
        const int stage = i % F::kStages;
        const uint32_t parity = (i / F::kStages) & 1;
        const int p0 = __shfl_sync(0xffffffffu, my_page, 2 * j), p1 = __shfl_sync(0xffffffffu, my_page, 2 * j + 1);
        if (!kv_wait_warp([&] { return kv_wait(&ctl->k_free[stage], parity ^ 1, &ctl->abort, 100 + kBarKFree); })) return;
        // a tile's second page may lie past the sequence: its rows keep what they hold and are masked
        const uint32_t bytes = p1 >= 0 ? kTileBytes : kTileBytes / 2;
        if (lane == 0) {
          uint8_t* dst = sm + stage * kTileBytes;
          mbar_arrive_expect_tx(&ctl->k_full[stage], bytes);
          tma_load_3d(dst, kmap, &ctl->k_full[stage], 0, 0, p0);
          if (p1 >= 0) tma_load_3d(dst + kTileBytes / 2, kmap, &ctl->k_full[stage], 0, 0, p1);
        }
        if (!kv_wait_warp([&] { return kv_wait(&ctl->v_free[stage], parity ^ 1, &ctl->abort, 100 + kBarVFree); })) return;
        if (lane == 0) {
          uint8_t* dst = sm + F::kOffV + stage * kTileBytes;
          mbar_arrive_expect_tx(&ctl->v_full[stage], bytes);
          tma_load_3d(dst, vmap, &ctl->v_full[stage], 0, 0, p0);
          if (p1 >= 0) tma_load_3d(dst + kTileBytes / 2, vmap, &ctl->v_full[stage], 0, 0, p1);
        }
        // last, since the scales' loads follow the page's
        if ((lane >> 1) == j)  // a power of two: its log2 and reciprocal are its bits
          ctl->scale[i % kScaleRing][lane & 1] =
              my_page < 0 ? make_float4(1.f, 0.f, 1.f, 0.f)
                          : make_float4(my_sk, (float)((int)(__float_as_uint(my_sv) >> 23) - 127),
                                        __int_as_float((254 << 23) - __float_as_int(my_sv)), 0.f);
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->scale_full[i % kScaleRing]);
      }
    }
  }
}

// ---------------------------------------------------------------- MMA warp
// The whole warp walks the loop and one elected lane issues, so addresses and
// descriptors stay in uniform registers.
template <int NR>
__device__ __forceinline__ void few_mma(const KvAttnArgs& a, FewCtl<NR>* ctl, uint32_t sm, uint32_t tmem_any) {
  using F = Few<NR>;
  constexpr uint32_t kIdS = idesc_e4m3(128, F::kN, false, false), kIdO = idesc_e4m3(128, F::kN, true, true);
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_any, 0);
  const uint64_t dk = sdesc_sw128(sm, 0, 1024), dv = sdesc_sw128(sm + F::kOffV, 0, 1024);
  const uint64_t dq = sdesc_sw128(sm + F::kOffQ, 0, 1024);
  const uint64_t dp = sdesc_plain(sm + F::kOffP, 128, 16 * kKvTile);
  const bool issue = elect_one();
  int i = 0, ks = 0, vs = 0;  // step of the run; stages of its next keys and of the values of the step before
  uint32_t k_par = 0, v_par = 0, q_par = 0;
  // O^T of the step before step i, of n tiles, once its weights are in shared memory
  auto second = [&](int n) {
    const int buf = (i - 1) & 1;
    if (!kv_wait_warp([&] { return kv_wait(&ctl->p_full[buf], ((i - 1) >> 1) & 1, &ctl->abort, 100 + kBarP); })) return false;
#pragma unroll
    for (int h = 0; h < F::kTiles; ++h) {
      if (h >= n) break;
      if (!kv_wait_warp([&] { return kv_wait(&ctl->v_full[vs], v_par, &ctl->abort, 100 + kBarV); })) return false;
      tc_fence_after();
      if (issue) {
        const uint32_t d = tmem + F::kColO + buf * F::kN;
        const uint64_t v = dv + vs * (kTileBytes >> 4), p = dp + (buf * F::kTiles + h) * (F::kPBytes >> 4);
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_f8(d, v + k * 256, p + k * 32, kIdO, h + k > 0);
        mma_commit(&ctl->v_free[vs]);
        if (h == n - 1) mma_commit(&ctl->o_full[buf]);
      }
      __syncwarp();
      if (++vs == F::kStages) {
        vs = 0;
        v_par ^= 1;
      }
    }
    return true;
  };
  int last = 0;  // tiles of the step before
  KvCursor cur;
#pragma unroll 1
  for (cur.start(a, ctl->run.run); cur.valid(); cur.next(a)) {
    const int tiles = __shfl_sync(0xffffffffu, cur.tiles(), 0);
#pragma unroll 1
    for (int j = 0; j < tiles; j += F::kTiles) {
      // A new item's queries arrive only after the last step's softmax: finish that step first.
      if (j == 0) {
        if (i > 0 && !second(last)) return;
        if (!kv_wait_warp([&] { return kv_wait(&ctl->q_full, q_par, &ctl->abort, 100 + kBarQ); })) return;
        q_par ^= 1;
      }
      const int n = min(F::kTiles, tiles - j);
#pragma unroll
      for (int h = 0; h < F::kTiles; ++h) {
        if (h >= n) break;
        if (!kv_wait_warp([&] { return kv_wait(&ctl->k_full[ks], k_par, &ctl->abort, 100 + kBarK); })) return;
        tc_fence_after();
        if (issue) {
          const uint32_t d = tmem + ((i & 1) * F::kTiles + h) * F::kN;
          const uint64_t kk = dk + ks * (kTileBytes >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_f8(d, kk + k * 2, dq + k * 2, kIdS, k > 0);
          if (h == n - 1) mma_commit(&ctl->s_full[i & 1]);
          mma_commit(&ctl->k_free[ks]);
        }
        __syncwarp();
        if (++ks == F::kStages) {
          ks = 0;
          k_par ^= 1;
        }
      }
      if (j > 0 && !second(last)) return;
      last = n;
      ++i;
    }
  }
  if (i > 0) second(last);
}

// ---------------------------------------------------------------- softmax warpgroups
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float warp_max(float x) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
  return m;
}

// Two fp32 products and sums in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 bits2(const uint32_t* r) { return make_float2(__uint_as_float(r[0]), __uint_as_float(r[1])); }

constexpr float kNegInf = -__builtin_huge_valf();

template <int NR>
__device__ __forceinline__ void few_softmax(const KvAttnArgs& a, FewCtl<NR>* ctl, uint8_t* sm,
                                            uint32_t tmem) {
  using F = Few<NR>;
  constexpr int R = kRowsWg;
  const int wg = threadIdx.x >> 7, tid = threadIdx.x & 127, warp = tid >> 5, lane = tid & 31;
  const int row0 = wg * R;
  constexpr int T = F::kTiles;
  const uint32_t t_lane = tmem + ((uint32_t)(warp * 32) << 16) + wg * 2 * R;
  const int bar = 1 + wg;
  bool bad = false;
  int i = 0, tile = 0, cleaned = 0;  // steps and tiles of the run, and the masked tiles among them
  const int w = threadIdx.x >> 5;
  KvCursor cur;
#pragma unroll 1
  for (cur.start(a, ctl->run.run); cur.valid(); cur.next(a)) {
    const KvItem& it = cur.it;
    const int past = it.len - it.n, head0 = kv_first_q_head(a.c, cur.head);
    const int group = kv_first_q_head(a.c, cur.head + 1) - head0;
    const int tiles = cur.tiles();
    if (tiles > 0) {
      // ---- the item's query rows: every fourth one is this warp's, all loads in flight ----
      uint2 q4[R / 4];
#pragma unroll
      for (int k = 0; k < R / 4; ++k) {
        const int rr = cur.rt * NR + row0 + warp + 4 * k, t = rr / a.group, g = rr - t * a.group;
        q4[k] = make_uint2(0, 0);
        if (t < it.n && g < group)
          q4[k] = __ldg(reinterpret_cast<const uint2*>(reinterpret_cast<const __nv_bfloat16*>(a.q) +
                                                       (int64_t)(it.tok0 + t) * a.q_stride + (head0 + g) * kHeadDim + 4 * lane));
      }
#pragma unroll
      for (int k = 0; k < R / 4; ++k) {
        const int r = warp + 4 * k, rr = cur.rt * NR + row0 + r, t = rr / a.group, g = rr - t * a.group;
        const bool live = t < it.n && g < group;
        const uint2 w = q4[k];
        float x[4] = {__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                      __uint_as_float(w.y & 0xffff0000u)};
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) m = max(m, __float_as_uint(x[e]) & 0x7fffffffu);
        m = __reduce_max_sync(0xffffffffu, m);
        // below 2^-102 a row's scores are zero for any key the cache can hold
        const int ex = m < 0x7f800000u ? e4m3_scale_exp(m, -110) : 0;
        const float inv = pow2f(-ex);
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float y0 = x[2 * e] * inv, y1 = x[2 * e + 1] * inv;
          hi[e] = f32x2_to_e4m3x2(y0, y1);
          const float2 h = e4m3x2_to_f32x2(hi[e]);
          lo[e] = f32x2_to_e4m3x2((y0 - h.x) * 16.f, (y1 - h.y) * 16.f);
        }
        const int n = 2 * row0 + r;  // column of the products: hi; lo R columns on
        uint8_t* q = sm + F::kOffQ;
        *reinterpret_cast<uint32_t*>(q + sw128_offset(n, lane >> 2) + 4 * (lane & 3)) = hi[0] | hi[1] << 16;
        *reinterpret_cast<uint32_t*>(q + sw128_offset(n + R, lane >> 2) + 4 * (lane & 3)) = lo[0] | lo[1] << 16;
        if (lane == 0) {
          const int p = past + t;
          // a row that is not finite gives NaN
          ctl->f[row0 + r] = m < 0x7f800000u ? pow2f(ex) * a.scale_log2 : __int_as_float(0x7fffffff);
          ctl->key_lo[row0 + r] = kv_window_begin(p, a.window);
          ctl->key_hi[row0 + r] = live ? (a.causal ? min(max(p + 1, 0), it.len) : it.len) : 0;
        }
      }
      fence_proxy_async_smem();
      kv_arrive_warp(&ctl->q_full);
      named_bar_sync(bar, 128);
    }
    // tiles that lie within every live row's keys need no mask
    const int t0 = cur.rt * NR / a.group, t1 = min(it.n - 1, (cur.rt * NR + NR - 1) / a.group);
    const int all_lo = kv_window_begin(past + t1, a.window), all_hi = a.causal ? min(past + t0 + 1, it.len) : it.len;
    const bool dead = cur.rt * NR + row0 >= it.n * a.group;  // no row of this warpgroup: its columns may hold anything
    float m = kNegInf;  // running maximum of row lane % R
    // by pairs of rows: this key's part of the sums; column tid of the output, up to the step before last
    float2 l[R / 2], o[R / 2];
#pragma unroll
    for (int r = 0; r < R / 2; ++r) l[r] = o[r] = both(0.f);
    // O^T of step t, in units of 2^(its maximum - 8), joins the rest
    auto join = [&](int t) {
      bad |= !kv_wait_warp([&] { return kv_wait(&ctl->o_full[t & 1], (t >> 1) & 1, &ctl->abort, 100 + kBarO); });
      if (bad) return;
      tc_fence_after();
      uint32_t h[16];
      tmem_ld16(t_lane + F::kColO + (t & 1) * F::kN, h);
      tmem_ld_wait(h);
#pragma unroll
      for (int r = 0; r < R / 2; ++r) {
        const float2 alpha = *reinterpret_cast<const float2*>(&ctl->alpha[w][t & 1][2 * r]);
        const float2 beta = *reinterpret_cast<const float2*>(&ctl->beta[w][t & 1][2 * r]);
        const float2 now = fma2(bits2(h + R + 2 * r), both(0.0625f), bits2(h + 2 * r));
        o[r] = fma2(o[r], alpha, mul2(now, beta));
      }
    };
#pragma unroll 1
    for (int j = 0; j < tiles; j += T, ++i) {
      const int buf = i & 1, n = min(T, tiles - j), key0 = (cur.tile_begin() + j) * kKvTile;
      bool masked[T];
      int slot[T];
#pragma unroll
      for (int h = 0; h < T; ++h) {
        const int k0 = key0 + h * kKvTile, key = k0 + tid;
        masked[h] = h < n && (k0 < all_lo || k0 + kKvTile > all_hi);
        slot[h] = cleaned & 3;
        if (!masked[h]) continue;
        // Values no row may use must not meet a zero weight as NaN: the first
        // warpgroup makes zeros of a key row past the sequence, or with a NaN
        // code, before any product; in the second case the rows that do
        // attend to it become NaN.
        if (wg == 0) {
          const int at = tile + h, stage = at % F::kStages;
          bad |= !kv_wait_warp([&] { return kv_wait(&ctl->v_full[stage], (at / F::kStages) & 1, &ctl->abort, 100 + kBarV); });
          uint8_t* v = sm + F::kOffV + stage * kTileBytes + tid * kHeadDim;
          uint32_t carry = 0;
          if (!bad && key < it.len) {
            // each lane of eight from another chunk: no bank conflicts
#pragma unroll 2
            for (int e = 0; e < 8; ++e) {  // b & 0x7f = 0x7f: adding 1 to the low seven bits carries into the eighth
              const uint4 c = reinterpret_cast<const uint4*>(v)[(e + lane) & 7];
              carry |= ((c.x & 0x7f7f7f7fu) + 0x01010101u) | ((c.y & 0x7f7f7f7fu) + 0x01010101u) |
                       ((c.z & 0x7f7f7f7fu) + 0x01010101u) | ((c.w & 0x7f7f7f7fu) + 0x01010101u);
            }
          }
          const bool nan = (carry & 0x80808080u) != 0;
          const uint32_t word = __ballot_sync(0xffffffffu, nan);
          if (lane == 0) ctl->nan_keys[slot[h]][warp] = word;
          if (!bad && (nan || key >= it.len)) {
#pragma unroll 2
            for (int e = 0; e < 8; ++e) reinterpret_cast<uint4*>(v)[(e + lane) & 7] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          kv_arrive_warp(&ctl->v_clean[slot[h]]);
        }
        if (!dead) bad |= !kv_wait_warp([&] { return kv_wait(&ctl->v_clean[slot[h]], (cleaned >> 2) & 1, &ctl->abort, 100 + kBarClean); });
        ++cleaned;
      }
      bad |= !kv_wait_warp([&] {
        for (int h = 0; h < n; ++h)
          if (!kv_wait(&ctl->scale_full[(tile + h) % kScaleRing], ((tile + h) / kScaleRing) & 1, &ctl->abort, 100 + kBarScale))
            return false;
        return kv_wait(&ctl->s_full[buf], (i >> 1) & 1, &ctl->abort, 100 + kBarS);
      });
      if (dead) {
        if (bad) break;
        kv_arrive_warp(&ctl->p_full[buf]);
        tile += n;
        continue;
      }
      float x[T][R], inv_sv[T];
      if (!bad) {
        tc_fence_after();
        // a tile's columns of this warpgroup: R of hi, R of lo; of a tile that is not there, whatever they held
        uint32_t s[2][16];
        tmem_ld16(t_lane + buf * T * F::kN, s[0]);
        if (T == 2) {
          tmem_ld16(t_lane + buf * T * F::kN + F::kN, s[1]);
          tmem_ld_wait(s[0], s[1]);
        } else {
          tmem_ld_wait(s[0]);
        }
#pragma unroll
        for (int h = 0; h < T; ++h) {
          const float4 sc = ctl->scale[(tile + min(h, n - 1)) % kScaleRing][warp >> 1];  // key scale, log2 of the value scale, its inverse
          inv_sv[h] = sc.z;
#pragma unroll
          for (int r = 0; r < R; r += 2) {
            const float2 f = mul2(*reinterpret_cast<const float2*>(ctl->f + row0 + r), both(sc.x));
            const float2 y = fma2(bits2(s[h] + R + r), both(0.0625f), bits2(s[h] + r));
            const float2 z = fma2(y, f, both(sc.y));
            x[h][r] = z.x;
            x[h][r + 1] = z.y;
          }
          if (masked[h]) {
            const int key = key0 + h * kKvTile + tid;
            const bool nan = (ctl->nan_keys[slot[h]][warp] >> lane) & 1;
#pragma unroll
            for (int r = 0; r < R; ++r) {
              const bool in = key >= ctl->key_lo[row0 + r] && key < ctl->key_hi[row0 + r];
              x[h][r] = in ? (nan ? __int_as_float(0x7fffffff) : x[h][r]) : kNegInf;
            }
          }
          if (h >= n) {
            inv_sv[h] = 0.f;
#pragma unroll
            for (int r = 0; r < R; ++r) x[h][r] = kNegInf;
          }
        }
        float mine = kNegInf;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float c = warp_max(T == 2 ? fmaxf(x[0][r], x[T - 1][r]) : x[0][r]);
          if (lane == r) mine = c;
        }
        if (lane < R) ctl->top[wg][buf][lane][warp] = mine;
      }
      bad = named_bar_or(bar, 128, bad);
      if (bad) return;
      // lane: its row's factors for this step's join
      {
        const float4 c = *reinterpret_cast<const float4*>(ctl->top[wg][buf][lane % R]);
        const float top = fmaxf(fmaxf(c.x, c.y), fmaxf(c.z, c.w));
        const float both = fmaxf(m, top), at = both == kNegInf ? 0.f : both;
        if (lane < R) {
          ctl->ref[w][lane] = 8.f - (top == kNegInf ? 0.f : top);
          ctl->alpha[w][buf][lane] = ex2(m - at);
          ctl->beta[w][buf][lane] = ex2(top - at);
        }
        m = both;
        __syncwarp();
      }
#pragma unroll
      for (int r = 0; r < R; r += 2) {
        const float2 ref = *reinterpret_cast<const float2*>(&ctl->ref[w][r]);
#pragma unroll
        for (int h = 0; h < T; ++h) {
          const float2 z = add2(make_float2(x[h][r], x[h][r + 1]), ref);
          x[h][r] = ex2(z.x);
          x[h][r + 1] = ex2(z.y);
        }
      }
      // P^T, 16 columns of bytes a key: hi, then lo
#pragma unroll
      for (int h = 0; h < T; ++h) {
        if (h >= n) break;
        uint8_t* p = sm + F::kOffP + (buf * T + h) * F::kPBytes + wg * (16 * kKvTile) + tid * 16;
        uint32_t hi[R / 2], lo[R / 2];
#pragma unroll
        for (int r = 0; r < R / 2; ++r) split_e4m3<16>(x[h][2 * r], x[h][2 * r + 1], hi[r], lo[r]);
        *reinterpret_cast<uint4*>(p) = make_uint4(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16, lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      kv_arrive_warp(&ctl->p_full[buf]);
      // under this step's second product: the sums, and the output of the step before
#pragma unroll
      for (int r = 0; r < R; r += 2) {
        const float2 alpha = *reinterpret_cast<const float2*>(&ctl->alpha[w][buf][r]);
        const float2 beta = *reinterpret_cast<const float2*>(&ctl->beta[w][buf][r]);
        float2 sum = mul2(make_float2(x[0][r], x[0][r + 1]), both(inv_sv[0]));
        if (T == 2) sum = fma2(make_float2(x[T - 1][r], x[T - 1][r + 1]), both(inv_sv[T - 1]), sum);
        l[r / 2] = fma2(l[r / 2], alpha, mul2(sum, beta));
      }
      if (j > 0) join(i - 1);
      tile += n;
    }
    if (dead) {
      if (tiles > 0) bad = named_bar_or(bar, 128, bad);
      if (bad) return;
      continue;
    }
    if (tiles > 0) {
      join(i - 1);
      tc_fence_before();
      if (!bad) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float s = r & 1 ? l[r / 2].y : l[r / 2].x;
#pragma unroll
          for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
          if (lane == 0) ctl->sum[wg][r][warp] = s;
        }
      }
      bad = named_bar_or(bar, 128, bad);
      if (bad) return;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float4 c = *reinterpret_cast<const float4*>(ctl->sum[wg][r]);
        (r & 1 ? l[r / 2].y : l[r / 2].x) = (c.x + c.y) + (c.z + c.w);
      }
    }
    // ---- thread d writes column d of each row ----
    auto row = [](const float2* v, int r) { return r & 1 ? v[r / 2].y : v[r / 2].x; };
    if (cur.whole()) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int rr = cur.rt * NR + row0 + r, t = rr / a.group, g = rr % a.group;
        if (t < it.n && g < group) {
          const int64_t tok = it.tok0 + t;
          reinterpret_cast<__nv_bfloat16*>(a.out)[tok * a.out_stride + (head0 + g) * kHeadDim + tid] =
              __float2bfloat16_rn(row(l, r) == 0.f ? 0.f : row(o, r) / row(l, r));
          if (a.lse && tid == r) a.lse[tok * a.c.h_q + head0 + g] = kv_lse(m - 8.f, row(l, r));
        }
      }
    } else {
      const size_t at = (size_t)cur.slot() * NR + row0;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        a.o[(at + r) * kHeadDim + tid] = row(o, r);
        if (tid == r) a.ml[at + r] = make_float2(m - 8.f, row(l, r));
      }
      if (threadIdx.x == 0 && cur.off == 0)
        kv_desc_put(a, ctl->run.run, cur);
    }
    if (tiles > 0) named_bar_sync(bar, 128);  // the sums are read before the next item's are written
  }
}

template <int NR>
__global__ void __launch_bounds__(Few<NR>::kThreads, Few<NR>::kCtasPerSm)
    attn_few_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                    const __grid_constant__ KvAttnArgs a) {
  using F = Few<NR>;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ FewCtl<NR> ctl;
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, warp = tid >> 5;
  if (tid == 0) {
    for (int s = 0; s < F::kStages; ++s) {
      mbar_init(&ctl.k_full[s], 1);
      mbar_init(&ctl.k_free[s], 1);
      mbar_init(&ctl.v_full[s], 1);
      mbar_init(&ctl.v_free[s], 1);
    }
    mbar_init(&ctl.q_full, F::kSoft / 32);
    for (int b = 0; b < 4; ++b) mbar_init(&ctl.v_clean[b], 4);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ctl.s_full[b], 1);
      mbar_init(&ctl.p_full[b], F::kSoft / 32);
      mbar_init(&ctl.o_full[b], 1);
    }
    for (int s = 0; s < kScaleRing; ++s) mbar_init(&ctl.scale_full[s], 1);
    fence_mbar_init();
    ctl.abort = 0;
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }
  if (warp == F::kSoft / 32) {
    tmem_alloc(&ctl.tmem, F::kTmemCols);
    tmem_relinquish();
  }
  grid_dependency_wait();
  if (tid == 0) kv_desc_none(a);
  kv_run<F::kThreads>(a, &ctl.run);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem;
  if (warp < F::kSoft / 32) {
    few_softmax<NR>(a, &ctl, sm, tmem);
  } else if (warp == F::kSoft / 32) {
    few_load<NR>(a, &ctl, sm, &kmap, &vmap);
  } else {
    few_mma<NR>(a, &ctl, smem_u32(sm), tmem);
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
  if (warp == F::kSoft / 32) {
    tc_fence_after();
    tmem_dealloc(tmem, F::kTmemCols);
  }
}

template <int NR>
cudaError_t launch(const KvAttnArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap, unsigned grid,
                   cudaStream_t st) {
  return launch_kernel(attn_few_kernel<NR>, dim3(grid), dim3(Few<NR>::kThreads), Few<NR>::kSmem, st, true, kmap,
                       vmap, a);
}

}  // namespace

int kv_few_ctas_per_sm(int rows) { return rows > 16 ? Few<32>::kCtasPerSm : Few<16>::kCtasPerSm; }

cudaError_t kv_few_setup() {
  cudaError_t e;
  if ((e = cudaFuncSetAttribute(attn_few_kernel<8>, cudaFuncAttributeMaxDynamicSharedMemorySize, Few<8>::kSmem)) != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(attn_few_kernel<16>, cudaFuncAttributeMaxDynamicSharedMemorySize, Few<16>::kSmem)) != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(attn_few_kernel<24>, cudaFuncAttributeMaxDynamicSharedMemorySize, Few<24>::kSmem)) != cudaSuccess) return e;
  return cudaFuncSetAttribute(attn_few_kernel<32>, cudaFuncAttributeMaxDynamicSharedMemorySize, Few<32>::kSmem);
}

cudaError_t launch_kv_attn_few(const KvAttnArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap, unsigned grid,
                               cudaStream_t st) {
  switch (a.rows) {
    case 8: return launch<8>(a, kmap, vmap, grid, st);
    case 16: return launch<16>(a, kmap, vmap, grid, st);
    case 24: return launch<24>(a, kmap, vmap, grid, st);
    default: return launch<32>(a, kmap, vmap, grid, st);
  }
}

}  // namespace gdn
