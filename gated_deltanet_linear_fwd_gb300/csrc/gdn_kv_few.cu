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
// below.  Weights P = 2^(x - m + 8) enter as hi + lo, eight bits (to 2^-8 of
// each weight, relative; a bf16 weight has 2^-9).  The two parts are columns of
// one product, so no key or value is converted or read twice.
//
// Softmax over the keys x_j = scale log2(e) q . k_j, per tile of 128 keys (two
// pages): thread j of a warpgroup holds key j's column of S^T.  The values'
// page scale 2^e_v (a power of two) is folded into the exponent: with m_t the
// tile's maximum of x + e_v, P_j = 2^(x_j + e_v - m_t + 8), so P . V-codes is the
// tile's output in units of 2^(m_t - 8), and its sum is of P_j 2^-e_v, kept in
// fp32 from the unrounded P.  Weights count from their own tile's maximum, so
// what e4m3 cannot hold is below 2^-18 of that, however many keys there are.
// Tiles are joined in fp32 registers, under the next tile's second product:
// o <- o 2^(m - m') + O_t 2^(m_t - m'), m' the larger of m and m_t.
//
// Roles: warpgroups of four warps with 8 rows each (one with 16 for 16 rows),
// one TMA warp, one MMA warp.  Two CTAs an SM hide one another's tile latency;
// 32 rows take one CTA of four warpgroups (two of 16 rows took 2600 cycles a
// tile, four of 8 rows 1500, against 1400 for the tile's bytes from HBM).
#include <cuda_fp16.h>

#include "gdn_dev.cuh"
#include "gdn_kv.cuh"

namespace gdn {
namespace {

constexpr int kTileBytes = kKvTile * kHeadDim;  // codes of a tile of keys or values
constexpr int kScaleRing = 8;                   // tiles whose page scales are in shared memory

// Details of the bounded waits (100 + barrier), as in the other kernels.
enum { kBarK = 1, kBarV, kBarKFree, kBarVFree, kBarQ, kBarS, kBarP, kBarO, kBarScale, kBarClean };

template <int NR>
struct Few {
  static constexpr int kRowsWg = NR == 16 ? 16 : 8;      // rows of a warpgroup
  static constexpr int kWgs = NR / kRowsWg;
  static constexpr int kSoft = kWgs * 128;               // softmax threads
  static constexpr int kThreads = kSoft + 64;
  static constexpr int kN = 2 * NR;                      // columns of the products
  static constexpr int kStages = NR == 32 ? 5 : 3;
  static constexpr int kCtasPerSm = NR == 32 ? 1 : 2;
  static constexpr uint32_t kTmemCols = 4 * kN;          // S and O, two of each
  static constexpr uint32_t kOffV = kStages * kTileBytes;
  static constexpr uint32_t kOffQ = 2 * kStages * kTileBytes;
  static constexpr uint32_t kOffP = kOffQ + kN * kHeadDim;
  static constexpr uint32_t kSmem = kOffP + 2 * kN * kKvTile + 1024;  // + alignment
};

template <int NR>
struct FewCtl {
  uint64_t k_full[5], k_free[5], v_full[5], v_free[5];
  uint64_t q_full, s_full[2], p_full[2], o_full[2], v_clean[2], scale_full[kScaleRing];
  float scale[kScaleRing][4];  // key scales of the tile's two pages, value scales
  uint32_t nan_keys[2][4];     // keys of a masked tile whose values hold a NaN code
  alignas(16) float f[NR];     // score factor of a row: its power of two times scale log2(e)
  int key_lo[NR], key_hi[NR];  // keys a row attends to
  alignas(16) float top[Few<NR>::kWgs][2][Few<NR>::kRowsWg][4];  // tile maxima of the four warps
  alignas(16) float sum[Few<NR>::kWgs][Few<NR>::kRowsWg][4];
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
        if ((lane >> 1) == j) {
          float* s = ctl->scale[i % kScaleRing];
          s[lane & 1] = my_page >= 0 ? my_sk : 1.f;
          s[2 + (lane & 1)] = my_page >= 0 ? my_sv : 1.f;
        }
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
  int i = 0, ks = 0, vs = 0;  // tile of the run; stages of this tile's keys and of the values of the one before
  uint32_t k_par = 0, v_par = 0, q_par = 0;
  // O^T of the tile before tile i, once its weights are in shared memory
  auto second = [&]() {
    const int buf = (i - 1) & 1;
    if (!kv_wait_warp([&] {
          return kv_wait(&ctl->v_full[vs], v_par, &ctl->abort, 100 + kBarV) &&
                 kv_wait(&ctl->p_full[buf], ((i - 1) >> 1) & 1, &ctl->abort, 100 + kBarP);
        }))
      return false;
    tc_fence_after();
    if (issue) {
      const uint32_t d = tmem + (2 + buf) * F::kN;
      const uint64_t v = dv + vs * (kTileBytes >> 4), p = dp + buf * (F::kN * kKvTile >> 4);
#pragma unroll
      for (int k = 0; k < 4; ++k) mma_f8(d, v + k * 256, p + k * 32, kIdO, k > 0);
      mma_commit(&ctl->o_full[buf]);
      mma_commit(&ctl->v_free[vs]);
    }
    __syncwarp();
    if (++vs == F::kStages) {
      vs = 0;
      v_par ^= 1;
    }
    return true;
  };
  KvCursor cur;
#pragma unroll 1
  for (cur.start(a, ctl->run.run); cur.valid(); cur.next(a)) {
    const int tiles = __shfl_sync(0xffffffffu, cur.tiles(), 0);
#pragma unroll 1
    for (int j = 0; j < tiles; ++j) {
      // A new item's queries arrive only after the last tile's softmax: finish that tile first.
      if (j == 0) {
        if (i > 0 && !second()) return;
        if (!kv_wait_warp([&] { return kv_wait(&ctl->q_full, q_par, &ctl->abort, 100 + kBarQ); })) return;
        q_par ^= 1;
      }
      if (!kv_wait_warp([&] { return kv_wait(&ctl->k_full[ks], k_par, &ctl->abort, 100 + kBarK); })) return;
      tc_fence_after();
      if (issue) {
        const uint32_t d = tmem + (i & 1) * F::kN;
        const uint64_t kk = dk + ks * (kTileBytes >> 4);
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_f8(d, kk + k * 2, dq + k * 2, kIdS, k > 0);
        mma_commit(&ctl->s_full[i & 1]);
        mma_commit(&ctl->k_free[ks]);
      }
      __syncwarp();
      if (++ks == F::kStages) {
        ks = 0;
        k_par ^= 1;
      }
      if (j > 0 && !second()) return;
      ++i;
    }
  }
  if (i > 0) second();
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

constexpr float kNegInf = -__builtin_huge_valf();

template <int NR>
__device__ __forceinline__ void few_softmax(const KvAttnArgs& a, FewCtl<NR>* ctl, uint8_t* sm,
                                            uint32_t tmem) {
  using F = Few<NR>;
  constexpr int R = F::kRowsWg;
  const int wg = threadIdx.x >> 7, tid = threadIdx.x & 127, warp = tid >> 5, lane = tid & 31;
  const int row0 = wg * R;
  const uint32_t t_lane = tmem + ((uint32_t)(warp * 32) << 16) + wg * 2 * R;
  const int bar = 1 + wg;
  bool bad = false;
  int i = 0, cleaned = 0;  // tiles of the run, and the masked ones among them
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
          ctl->key_lo[row0 + r] = a.window > 0 ? max(0, p - a.window + 1) : 0;
          ctl->key_hi[row0 + r] = live ? (a.causal ? min(max(p + 1, 0), it.len) : it.len) : 0;
        }
      }
      fence_proxy_async_smem();
      kv_arrive_warp(&ctl->q_full);
      named_bar_sync(bar, 128);
    }
    // tiles that lie within every live row's keys need no mask
    const int t0 = cur.rt * NR / a.group, t1 = min(it.n - 1, (cur.rt * NR + NR - 1) / a.group);
    const int all_lo = a.window > 0 ? past + t1 - a.window + 1 : 0, all_hi = a.causal ? min(past + t0 + 1, it.len) : it.len;
    const bool dead = cur.rt * NR + row0 >= it.n * a.group;  // no row of this warpgroup: its columns may hold anything
    float m[R], l[R], o[R];        // up to the tile before last
    float top[R], sum[R];          // the last tile's maximum and this key's part of its sum
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r] = top[r] = kNegInf;
      l[r] = o[r] = sum[r] = 0.f;
    }
    // O^T of the last tile, in units of 2^(its maximum - 8), joins the rest
    auto join = [&](int t) {
      bad |= !kv_wait_warp([&] { return kv_wait(&ctl->o_full[t & 1], (t >> 1) & 1, &ctl->abort, 100 + kBarO); });
      if (bad) return;
      tc_fence_after();
      uint32_t h[16], q[16];
      tmem_ld16(t_lane + (2 + (t & 1)) * F::kN, h);
      if (R == 16) {
        tmem_ld16(t_lane + (2 + (t & 1)) * F::kN + 16, q);
        tmem_ld_wait(h, q);
      } else {
        tmem_ld_wait(h);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float w = fmaxf(m[r], top[r]), ref = w == kNegInf ? 0.f : w;
        const float alpha = ex2(m[r] - ref), beta = ex2(top[r] - ref);
        m[r] = w;
        l[r] = fmaf(l[r], alpha, sum[r] * beta);
        o[r] = fmaf(o[r], alpha, (__uint_as_float(h[r]) + __uint_as_float(R == 16 ? q[r] : h[8 + r])) * beta);
      }
    };
#pragma unroll 1
    for (int j = 0; j < tiles; ++j, ++i) {
      const int buf = i & 1, key0 = (cur.tile_begin() + j) * kKvTile, key = key0 + tid;
      const int stage = i % F::kStages;
      const bool masked = key0 < all_lo || key0 + kKvTile > all_hi;
      if (masked) {
        // Values no row may use must not meet a zero weight as NaN: the first
        // warpgroup makes zeros of a key row past the sequence, or with a NaN
        // code, before any product; in the second case the rows that do
        // attend to it become NaN.
        if (wg == 0) {
          bad |= !kv_wait_warp([&] { return kv_wait(&ctl->v_full[stage], (i / F::kStages) & 1, &ctl->abort, 100 + kBarV); });
          uint8_t* v = sm + F::kOffV + stage * kTileBytes + tid * kHeadDim;
          uint32_t carry = 0;
          if (!bad && key < it.len) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {  // b & 0x7f = 0x7f: adding 1 to the low seven bits carries into the eighth
              const uint4 w = reinterpret_cast<const uint4*>(v)[e];
              carry |= ((w.x & 0x7f7f7f7fu) + 0x01010101u) | ((w.y & 0x7f7f7f7fu) + 0x01010101u) |
                       ((w.z & 0x7f7f7f7fu) + 0x01010101u) | ((w.w & 0x7f7f7f7fu) + 0x01010101u);
            }
          }
          const bool nan = (carry & 0x80808080u) != 0;
          const uint32_t word = __ballot_sync(0xffffffffu, nan);
          if (lane == 0) ctl->nan_keys[cleaned & 1][warp] = word;
          if (!bad && (nan || key >= it.len)) {
#pragma unroll
            for (int e = 0; e < 8; ++e) reinterpret_cast<uint4*>(v)[e] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          kv_arrive_warp(&ctl->v_clean[cleaned & 1]);
        }
        if (!dead) bad |= !kv_wait_warp([&] { return kv_wait(&ctl->v_clean[cleaned & 1], (cleaned >> 1) & 1, &ctl->abort, 100 + kBarClean); });
        ++cleaned;
      }
      float x[R];
      float inv_sv = 1.f;
      bad |= !kv_wait_warp([&] {
        return kv_wait(&ctl->scale_full[i % kScaleRing], (i / kScaleRing) & 1, &ctl->abort, 100 + kBarScale) &&
               kv_wait(&ctl->s_full[buf], (i >> 1) & 1, &ctl->abort, 100 + kBarS);
      });
      if (dead) {
        if (bad) return;
        kv_arrive_warp(&ctl->p_full[buf]);
        continue;
      }
      if (!bad) {
        tc_fence_after();
        uint32_t hi[16], lo[16];
        tmem_ld16(t_lane + buf * F::kN, hi);
        if (R == 16) tmem_ld16(t_lane + buf * F::kN + 16, lo);
        const float* sc = ctl->scale[i % kScaleRing];
        const float sk = sc[warp >> 1], sv = sc[2 + (warp >> 1)];
        const float ev = (float)((int)(__float_as_uint(sv) >> 23) - 127);  // log2 of a power of two
        inv_sv = __int_as_float((254 << 23) - __float_as_int(sv));
        if (R == 16)
          tmem_ld_wait(hi, lo);
        else
          tmem_ld_wait(hi);
#pragma unroll
        for (int r = 0; r < R; r += 4) {
          const float4 f4 = *reinterpret_cast<const float4*>(ctl->f + row0 + r);
          const float f[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float s = fmaf(__uint_as_float(R == 16 ? lo[r + e] : hi[(8 + r + e) & 15]), 0.0625f, __uint_as_float(hi[r + e]));
            x[r + e] = fmaf(s, f[e] * sk, ev);
          }
        }
        if (masked) {
          const bool nan = (ctl->nan_keys[(cleaned - 1) & 1][warp] >> lane) & 1;
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const bool in = key >= ctl->key_lo[row0 + r] && key < ctl->key_hi[row0 + r];
            x[r] = in ? (nan ? __int_as_float(0x7fffffff) : x[r]) : kNegInf;
          }
        }
        float mine = kNegInf;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float w = warp_max(x[r]);
          if (lane == r) mine = w;
        }
        if (lane < R) ctl->top[wg][buf][lane][warp] = mine;
      }
      bad = named_bar_or(bar, 128, bad);
      if (bad) return;
      float now[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float4 w = *reinterpret_cast<const float4*>(ctl->top[wg][buf][r]);
        now[r] = fmaxf(fmaxf(w.x, w.y), fmaxf(w.z, w.w));
        x[r] = ex2(x[r] - (now[r] == kNegInf ? 0.f : now[r]) + 8.f);
      }
      // P^T, 16 columns of bytes a key: hi, then lo
      uint8_t* p = sm + F::kOffP + buf * (F::kN * kKvTile) + (wg * (2 * R / 16)) * (16 * kKvTile) + tid * 16;
      uint32_t hi[R / 2], lo[R / 2];
#pragma unroll
      for (int r = 0; r < R / 2; ++r) split_e4m3(x[2 * r], x[2 * r + 1], hi[r], lo[r]);
      if (R == 8) {
        *reinterpret_cast<uint4*>(p) = make_uint4(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16, lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
      } else {
        *reinterpret_cast<uint4*>(p) = make_uint4(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16, hi[R / 2 - 4] | hi[R / 2 - 3] << 16,
                                                  hi[R / 2 - 2] | hi[R / 2 - 1] << 16);
        *reinterpret_cast<uint4*>(p + 16 * kKvTile) = make_uint4(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16,
                                                                 lo[R / 2 - 4] | lo[R / 2 - 3] << 16,
                                                                 lo[R / 2 - 2] | lo[R / 2 - 1] << 16);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      kv_arrive_warp(&ctl->p_full[buf]);
      // under this tile's second product, the tile before
      if (j > 0) join(i - 1);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        top[r] = now[r];
        sum[r] = x[r] * inv_sv;
      }
    }
    if (dead) continue;
    if (tiles > 0) {
      join(i - 1);
      tc_fence_before();
      if (!bad) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float s = l[r];
#pragma unroll
          for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
          if (lane == 0) ctl->sum[wg][r][warp] = s;
        }
      }
      bad = named_bar_or(bar, 128, bad);
      if (bad) return;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float4 w = *reinterpret_cast<const float4*>(ctl->sum[wg][r]);
        l[r] = (w.x + w.y) + (w.z + w.w);
      }
    }
    // ---- thread d writes column d of each row ----
    if (cur.whole()) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int rr = cur.rt * NR + row0 + r, t = rr / a.group, g = rr % a.group;
        if (t < it.n && g < group) {
          const int64_t tok = it.tok0 + t;
          reinterpret_cast<__nv_bfloat16*>(a.out)[tok * a.out_stride + (head0 + g) * kHeadDim + tid] =
              __float2bfloat16_rn(l[r] == 0.f ? 0.f : o[r] / l[r]);
          if (a.lse && tid == r) a.lse[tok * a.c.h_q + head0 + g] = kv_lse(m[r] - 8.f, l[r]);
        }
      }
    } else {
      const size_t row = (size_t)cur.slot() * NR + row0;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        a.o[(row + r) * kHeadDim + tid] = o[r];
        if (tid == r) a.ml[row + r] = make_float2(m[r] - 8.f, l[r]);
      }
      if (threadIdx.x == 0 && cur.off == 0)
        a.desc[blockIdx.x] = make_int4(cur.seq, cur.rt, cur.head, kv_last_cta(a, ctl->run.run, cur));
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
    mbar_init(&ctl.v_clean[0], 4);
    mbar_init(&ctl.v_clean[1], 4);
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
  if (tid == 0 && a.n_ctas) a.desc[blockIdx.x] = make_int4(-1, 0, 0, 0);
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

int kv_few_ctas_per_sm(int rows) { return rows == 32 ? Few<32>::kCtasPerSm : Few<16>::kCtasPerSm; }

cudaError_t kv_few_setup() {
  cudaError_t e;
  if ((e = cudaFuncSetAttribute(attn_few_kernel<8>, cudaFuncAttributeMaxDynamicSharedMemorySize, Few<8>::kSmem)) != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(attn_few_kernel<16>, cudaFuncAttributeMaxDynamicSharedMemorySize, Few<16>::kSmem)) != cudaSuccess) return e;
  return cudaFuncSetAttribute(attn_few_kernel<32>, cudaFuncAttributeMaxDynamicSharedMemorySize, Few<32>::kSmem);
}

cudaError_t launch_kv_attn_few(const KvAttnArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap, unsigned grid,
                               cudaStream_t st) {
  switch (a.rows) {
    case 8: return launch<8>(a, kmap, vmap, grid, st);
    case 16: return launch<16>(a, kmap, vmap, grid, st);
    default: return launch<32>(a, kmap, vmap, grid, st);
  }
}

}  // namespace gdn
