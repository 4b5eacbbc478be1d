// Shared definitions of the 8-bit key/value cache: its arguments, e4m3
// conversions, and how the key tiles of an attention call are shared out to
// CTAs.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gdn_internal.cuh"
#include "sm103_ptx.cuh"

namespace gdn {

constexpr int kPage = 64;      // tokens of a page and of a scale
constexpr int kKvTile = 128;   // keys of an attention tile: two pages
constexpr int kHeadDim = 128;
constexpr int kPageBytes = kPage * kHeadDim;  // codes of one (page, head)

constexpr int kDetKvLengths = 7;  // offsets or a length outside their bounds
constexpr int kDetKvPage = 8;     // a page outside the pool

// The cache and the batch.
struct KvArgs {
  const int32_t* lens;   // [n_seqs]
  const int32_t* table;  // [n_seqs, max_pages]
  const int32_t* cu;     // [n_seqs + 1] or null
  uint8_t* k;            // [n_pages, h_kv, 64, 128]
  uint8_t* v;
  float* k_scale;        // [n_pages, h_kv]
  float* v_scale;
  int* status;
  int n_seqs, T, n_each; // n_each: tokens of every sequence when cu is null
  int h_q, h_kv, max_pages, n_pages;
};

struct KvAppendArgs {
  KvArgs c;
  void* k;  // append: const inputs; read: outputs
  void* v;
  int64_t k_stride, v_stride;
  int pages_each;  // cu null: page slots per sequence
};

struct KvAttnArgs {
  KvArgs c;
  const void* q;
  void* out;
  float* lse;
  int64_t q_stride, out_stride;
  int causal, window;
  float scale_log2;        // score scale times log2(e)
  int group;               // query heads per key/value head, rounded up
  int rows, max_row_tiles; // rows of a row tile; row tiles per (sequence, head), at most
  int slots;               // entries of the call when they are found by search (kv_entry), or 0
  int max_rows;            // rows of the longest sequence the plan allows
  int n_ctas;              // 0: CTA i takes item i whole
  int item_cost;           // what beginning and ending an item costs, in key tiles
  int4* desc;              // [2 n_ctas] item whose first part this CTA made, in two: {last CTA or -1, row tile, head}, {first token, tokens}
  float2* ml;              // [2 n_ctas, rows] running maximum (log2) and sum of a part
  float* o;                // [2 n_ctas, rows, 128] unnormalised output of a part
};

// First packed token, number of new tokens and length of sequence s.  What
// does not fit the call's bounds is reported and counts as empty.
struct KvSeq {
  int tok0, n, len;
};
__device__ __forceinline__ KvSeq kv_seq(const KvArgs& a, int s) {
  KvSeq r;
  int b, e;
  if (a.cu) {
    b = a.cu[s];
    e = a.cu[s + 1];
  } else {
    b = s * a.n_each;
    e = b + a.n_each;
  }
  r.tok0 = b;
  r.n = e - b;
  r.len = a.lens[s];
  if (b < 0 || e < b || e > a.T || r.len < 0 || r.len > (int64_t)a.max_pages * kPage) {
    report(a.status, kDevCheck, kDetKvLengths);
    r.tok0 = 0;
    r.n = r.len = 0;
  }
  return r;
}

// Pool page of page slot `slot` of sequence s, or -1 (reported) for one
// outside the pool.
__device__ __forceinline__ int kv_page(const KvArgs& a, int s, int slot) {
  const int p = a.table[(int64_t)s * a.max_pages + slot];
  if ((unsigned)p < (unsigned)a.n_pages) return p;
  report(a.status, kDevCheck, kDetKvPage);
  return -1;
}

// The first key that a window leaves a token at position p; p may be negative
// and the window any positive number.
__device__ __forceinline__ int kv_window_begin(int p, int window) { return window > 0 && p >= window ? p - window + 1 : 0; }

// Query heads of key/value head h: those j with floor(j h_kv / h_q) = h.
__device__ __forceinline__ int kv_first_q_head(const KvArgs& a, int h) {
  return (int)(((unsigned)h * (unsigned)a.h_q + (unsigned)a.h_kv - 1u) / (unsigned)a.h_kv);  // heads are at most 65535
}

// ---- e4m3 ----
// Two codes (low byte first) to fp32; exact.
__device__ __forceinline__ float2 e4m3x2_to_f32x2(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
  float lo, hi;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
  return make_float2(lo, hi);
}
// Two fp32 to codes: nearest even, saturating at 448, NaN to NaN.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
  return c;
}

// Two fp32 (below 2^9) as e4m3 parts, x = hi + lo / kLoScale: four leading bits
// and the next four, to 2^-10 / kLoScale at least; through fp16, whose 11 bits
// the parts do not reach.
template <int kLoScale = 1>
__device__ __forceinline__ void split_e4m3(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  uint32_t x16, h16;
  uint16_t h, l;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(x16) : "f"(x1), "f"(x0));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(h) : "r"(x16));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h16) : "h"(h));
  __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&x16), *reinterpret_cast<const __half2*>(&h16));
  if (kLoScale != 1) r = __hmul2(r, __float2half2_rn((float)kLoScale));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(l) : "r"(*reinterpret_cast<const uint32_t*>(&r)));
  hi = h;
  lo = l;
}

// ---- sharing out an attention call ----
// An item is (sequence, row tile, key/value head); its units are its key
// tiles, at least one (an item without keys still writes zeros), after
// item_cost units that stand for its beginning and end.  All units, in the
// order sequence, row tile, head, tile, are cut into n_ctas equal runs, one a
// CTA, so the SMs get the same amount of work whatever the lengths are.  A run
// covers whole items and at most one part of an item at each end (a cut among
// the item_cost units leaves the item whole to the later run); parts go to
// the workspace and the combine kernel joins them.
struct KvItem {
  int tok0, n, len;       // the sequence
  int first_tile, tiles;  // key tiles its masks touch; tiles < 0: no such item
};
__device__ __forceinline__ KvItem kv_item(const KvAttnArgs& a, int seq, int rt) {
  KvItem it;
  const KvSeq s = kv_seq(a.c, seq);
  it.tok0 = s.tok0;
  it.n = s.n;
  it.len = s.len;
  it.first_tile = 0;
  const int r0 = rt * a.rows, rows = s.n * a.group;
  if (rows > a.max_rows) report(a.c.status, kDevCheck, kDetKvLengths);
  if (r0 >= rows) {
    it.tiles = -1;
    return it;
  }
  int t0 = 0, t1 = s.n - 1;
  if (a.max_row_tiles > 1) {
    t0 = r0 / a.group;
    t1 = min(t1, (r0 + a.rows - 1) / a.group);
  }
  const int past = s.len - s.n;  // position of the first new token; negative for idle slots
  const int hi = a.causal ? min(max(past + t1 + 1, 0), s.len) : s.len;
  const int lo = kv_window_begin(past + t0, a.window);
  it.first_tile = lo / kKvTile;
  it.tiles = hi > lo ? (hi + kKvTile - 1) / kKvTile - it.first_tile : 0;
  return it;
}
// Entries enumerate the (sequence, row tile) pairs of a call in this order.
// Without slots entry e is row tile e % max_row_tiles of sequence e / max_row_tiles.
// When a sequence may bring most of the call's tokens those are up to n_seqs
// times as many as there are row tiles.  With slots, sequence s has the entries
// from b(s) = floor(cu[s] group / rows) + s on, as many as it has row tiles: they
// end before b(s + 1), since floor(x) + ceil(y) <= floor(x + y) + 1, and
// floor(T group / rows) + n_seqs entries are enough whatever the lengths.
__device__ __forceinline__ int kv_first_slot(const KvAttnArgs& a, int s) {
  const int tok = min(max(a.c.cu[s], 0), a.c.T);  // T * group is below 2^31
  return (int)((uint32_t)(tok * a.group) / (uint32_t)a.rows) + s;
}
template <bool kSlots>
__device__ __forceinline__ KvItem kv_entry(const KvAttnArgs& a, int e, int& seq, int& rt) {
  seq = e;
  rt = 0;
  if (kSlots) {  // the last sequence whose slots begin at e or before
    int lo = 0, hi = a.c.n_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (kv_first_slot(a, mid) <= e) lo = mid;
      else hi = mid - 1;
    }
    seq = lo;
    rt = e - kv_first_slot(a, lo);
    if (rt < 0 || rt >= a.max_row_tiles) return {0, 0, 0, 0, -1};
  } else if (a.max_row_tiles > 1) {
    seq = e / a.max_row_tiles;
    rt = e - seq * a.max_row_tiles;
  }
  return kv_item(a, seq, rt);
}
// Offsets that go back hide sequences from the search: every one is checked
// all the same.
__device__ __forceinline__ void kv_check_all(const KvAttnArgs& a) {
  if (blockIdx.x == 0)
    for (int s = threadIdx.x; s < a.c.n_seqs; s += blockDim.x) kv_seq(a.c, s);
}
__device__ __forceinline__ int kv_units(const KvItem& it) { return it.tiles < 0 ? 0 : max(1, it.tiles); }
__device__ __forceinline__ int kv_cost(const KvAttnArgs& a, const KvItem& it) {
  return it.tiles < 0 ? 0 : a.item_cost + max(1, it.tiles);
}

struct KvRun {
  int seq, rt, head, off;  // first item of the run and the unit of it (of item_cost + tiles) that the run starts with
  KvItem item;             // that item
  uint32_t begin, end;     // units
  uint32_t total;          // units of the call; the host refuses calls that could have 2^31
  int ctas;                // CTAs that have a run: no more than there are units
};

// A CTA's run, found by all its threads (NT of them, a multiple of 32) from
// the lengths and left in shared memory.
struct KvRunScratch {
  uint32_t part[32];
  KvRun run;
};
// Inclusive sum over the block's threads; total: the block's sum.
template <int NT>
__device__ __forceinline__ uint32_t block_inclusive_scan(uint32_t v, KvRunScratch* sc, uint32_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += u;
  }
  __syncthreads();
  if (lane == 31) sc->part[warp] = v;
  __syncthreads();
  const uint32_t p = lane < NT / 32 ? sc->part[lane] : 0;
  total = __reduce_add_sync(0xffffffffu, p);
  return v + __reduce_add_sync(0xffffffffu, lane < warp ? p : 0);
}
// All of it is on the way to a CTA's first load, mostly as instructions not
// yet in the cache: one scan when the threads have an entry each (any decode
// batch of up to NT sequences), no 64-bit division.
template <int NT, bool kSlots>
__device__ __noinline__ void kv_run_of(const KvAttnArgs& a, KvRunScratch* sc) {
  const int tid = threadIdx.x;
  if (kSlots) kv_check_all(a);
  if (a.n_ctas == 0) {  // one whole item a CTA
    if (tid == 0) {
      KvRun& r = sc->run;
      const int e = blockIdx.x / a.c.h_kv;  // the longest row tiles, under a causal mask the last ones, first
      r.head = blockIdx.x - e * a.c.h_kv;
      if (kSlots) {
        r.item = kv_entry<true>(a, a.slots - 1 - e, r.seq, r.rt);
      } else {
        r.rt = a.max_row_tiles - 1 - e / a.c.n_seqs;
        r.seq = e % a.c.n_seqs;
        r.item = kv_item(a, r.seq, r.rt);
      }
      r.off = 0;
      r.begin = 0;
      r.end = r.total = kv_cost(a, r.item);
      r.ctas = 0;
    }
    __syncthreads();
    return;
  }
  const int entries = kSlots ? a.slots : a.c.n_seqs * a.max_row_tiles;
  KvItem it;
  int seq = 0, rt = 0;
  uint32_t total = 0, base = 0, incl = 0, u = 0;
  auto entry = [&](int e) {
    u = 0;
    if (e < entries) {
      it = kv_entry<kSlots>(a, e, seq, rt);
      u = kv_cost(a, it) * a.c.h_kv;
    }
  };
#pragma unroll 1
  for (int e0 = 0; e0 < entries; e0 += NT) {
    entry(e0 + tid);
    uint32_t sub;
    incl = block_inclusive_scan<NT>(u, sc, sub);
    total += sub;
  }
  // run c is [total c / ctas, total (c + 1) / ctas), rounded down
  const uint32_t ctas = min((uint32_t)a.n_ctas, total), cta = blockIdx.x;
  uint32_t begin = 0, end = 0;
  if (cta < ctas) {
    const uint32_t each = total / ctas, rest = total - each * ctas;
    begin = each * cta + rest * cta / ctas;
    end = each * (cta + 1) + rest * (cta + 1) / ctas;
  }
  if (tid == 0) {
    sc->run.begin = begin;
    sc->run.end = end;
    sc->run.total = total;
    sc->run.ctas = (int)ctas;
  }
#pragma unroll 1
  for (int e0 = 0; e0 < entries && base <= begin && begin < end; e0 += NT) {
    uint32_t sub = total;
    if (entries > NT) {
      entry(e0 + tid);
      incl = base + block_inclusive_scan<NT>(u, sc, sub);
    }
    if (incl - u <= begin && begin < incl) {
      const uint32_t in = begin - (incl - u), cost = kv_cost(a, it), head = in / cost;
      sc->run.seq = seq;
      sc->run.rt = rt;
      sc->run.head = (int)head;
      sc->run.off = (int)(in - head * cost);
      sc->run.item = it;
    }
    base += sub;
  }
  __syncthreads();
}

template <int NT>
__device__ __forceinline__ void kv_run(const KvAttnArgs& a, KvRunScratch* sc) {
  if (a.slots) kv_run_of<NT, true>(a, sc);
  else kv_run_of<NT, false>(a, sc);
}

// Walks the items of a run; every warp that needs it walks its own.
struct KvCursor {
  KvItem it;
  int seq, rt, head;
  int off, len;       // tiles [off, off + len) of the item belong to the run; len = 0: the run is over
  int base, end;      // unit the item starts with, and the run's end, from the run's first unit
  __device__ __forceinline__ void clip(const KvAttnArgs& a) {
    len = max(0, min(kv_units(it), end - base - a.item_cost) - off);
  }
  __device__ __forceinline__ void start(const KvAttnArgs& a, const KvRun& r) {
    seq = r.seq;
    rt = r.rt;
    head = r.head;
    end = (int)(r.end - r.begin);
    len = 0;
    if (end > 0) {
      base = -r.off;
      off = max(0, r.off - a.item_cost);
      it = r.item;
      clip(a);
    }
  }
  __device__ __forceinline__ bool valid() const { return len > 0; }
  __device__ __forceinline__ void next(const KvAttnArgs& a) {
    base += kv_cost(a, it);
    off = len = 0;
    if (base >= end) return;
    if (++head == a.c.h_kv) {
      head = 0;
      ++rt;
      while (true) {  // a run ends before the items do, so there is a next one
        if (rt < a.max_row_tiles) {
          it = kv_item(a, seq, rt);
          if (it.tiles >= 0) break;
        }
        rt = 0;
        if (++seq >= a.c.n_seqs) return;
      }
    }
    clip(a);
  }
  // key tiles [tile_begin, tile_begin + tiles) of the run's part of the item
  __device__ __forceinline__ int tiles() const { return it.tiles == 0 ? 0 : len; }
  __device__ __forceinline__ int tile_begin() const { return it.first_tile + off; }
  __device__ __forceinline__ bool whole() const { return off == 0 && len == kv_units(it); }
  __device__ __forceinline__ int slot() const { return 2 * blockIdx.x + (off > 0 ? 0 : 1); }
};

// The last CTA that has a part of the item whose first part this cursor
// stands on: the one whose run has the item's last unit u, the largest c with
// total c / ctas <= u, so floor(((u + 1) ctas - 1) / total).  Offsets that go
// back can put an item past the end.
__device__ __forceinline__ int kv_last_cta(const KvAttnArgs& a, const KvRun& r, const KvCursor& c) {
  const int64_t item_end = (int64_t)r.begin + c.base + kv_cost(a, c.it);
  return (int)min((item_end * r.ctas - 1) / r.total, (int64_t)r.ctas - 1);
}

// What the second kernel needs of the item this CTA began and did not end, or
// that there is none (said by every CTA before its run).
__device__ __forceinline__ void kv_desc_none(const KvAttnArgs& a) {
  if (a.n_ctas) a.desc[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);
}
__device__ __forceinline__ void kv_desc_put(const KvAttnArgs& a, const KvRun& r, const KvCursor& c) {
  a.desc[2 * blockIdx.x] = make_int4(kv_last_cta(a, r, c), c.rt, c.head, 0);
  a.desc[2 * blockIdx.x + 1] = make_int4(c.it.tok0, c.it.n, 0, 0);
}

// Bounded wait on an mbarrier phase: gives up (false) after kWaitTries tries,
// recording `code` in *abort, or when another role has.  A try that fails
// suspends the thread for about 4 us (measured), so the limit is about a
// second.  Counting tries keeps the loop a few instructions: with the
// nanosecond clock in it the waits of the many-rows kernel, all of them
// complete or nearly so, took 700 cycles each, twice the kernel's time.
constexpr int kWaitTries = 1 << 18;
__device__ __forceinline__ bool kv_wait(uint64_t* bar, uint32_t parity, int* abort, int code) {
#pragma unroll 1
  for (int i = 0; i < kWaitTries; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*reinterpret_cast<volatile int*>(abort)) return false;
  }
  *reinterpret_cast<volatile int*>(abort) = code;
  return false;
}
// The same by all lanes of a converged warp, which then agree.
template <typename W>
__device__ __forceinline__ bool kv_wait_warp(W wait) {
  return __all_sync(0xffffffffu, wait());
}
// One arrival for a converged warp's work before it.
__device__ __forceinline__ void kv_arrive_warp(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// log sum exp from a running maximum (log2) and sum.
__device__ __forceinline__ float kv_lse(float m, float l) {
  return l == 0.f ? -__int_as_float(0x7f800000) : (m + log2f(l)) * 0.693147180559945309f;
}

__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }

// The exponent of the smallest power of two s with a / s <= 448, from a's
// fp32 bits (a finite, >= 0): a = m 2^x with 1 <= m < 2 and 448 = 1.75 2^8,
// so it is x - 8, or x - 7 when m > 1.75; not below `least`.
__device__ __forceinline__ int e4m3_scale_exp(uint32_t a_bits, int least) {
  const int x = (int)(a_bits >> 23) - 127;
  return max(x - 8 + ((a_bits & 0x7fffffu) > 0x600000u ? 1 : 0), least);
}

// ---- launchers ----
cudaError_t launch_kv_append(const KvAppendArgs& a, bool f32, unsigned entries, cudaStream_t st);
cudaError_t launch_kv_read(const KvAppendArgs& a, bool f32, unsigned entries, cudaStream_t st);
cudaError_t launch_kv_attn_f32(const KvAttnArgs& a, unsigned grid, cudaStream_t st);  // fp32 q and out
cudaError_t launch_kv_combine(const KvAttnArgs& a, bool f32, cudaStream_t st);
cudaError_t kv_f32_setup();
// rows: 8, 16, 24 or 32 (KvAttnArgs::rows); kmap, vmap: the pools as [page and head][64][128 bytes]
cudaError_t launch_kv_attn_few(const KvAttnArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap, unsigned grid,
                               cudaStream_t st);
cudaError_t kv_few_setup();
int kv_few_ctas_per_sm(int rows);
cudaError_t launch_kv_attn_many(const KvAttnArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap, unsigned grid,
                                cudaStream_t st);
cudaError_t kv_many_setup();

}  // namespace gdn
