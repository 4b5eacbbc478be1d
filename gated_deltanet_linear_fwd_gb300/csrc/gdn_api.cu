// Host side of the C ABI declared in include/gdn.h: planning, argument
// checks, TMA tensor maps, and the launch sequence of the forward.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <climits>
#include <cstring>
#include <initializer_list>
#include <mutex>
#include <vector>

#include "gdn.h"
#include "gdn_internal.cuh"
#include "gdn_conv.cuh"
#include "gdn_kv.cuh"
#include "gdn_kv_page.cuh"
#include "gdn_rope.cuh"

using namespace gdn;

namespace {

thread_local int g_last_cuda_error = 0;
std::atomic<uint32_t> g_debug_stall_ns{0};  // test hook of the timeout path (gdn_debug_stall_ns)

// ---- tracing: caller-provided events recorded around each launch ----
// Kernel i of a call is bracketed by events 2i and 2i + 1, recorded on the
// stream it is launched on.
constexpr int kMaxTrace = 32;
thread_local cudaEvent_t g_trace_ev[kMaxTrace];
thread_local int g_trace_n = 0;
thread_local const char* g_last_names[kMaxTrace / 2];
thread_local int g_last_count = 0;

struct LaunchLog {
  // keep: continue the list of the call's kernels (the backward after its forward)
  explicit LaunchLog(bool keep = false) {
    if (!keep) g_last_count = 0;
  }
  // Records the start event of the next kernel on st.
  cudaError_t before(cudaStream_t st) {
    const int k = 2 * g_last_count;
    return k < g_trace_n ? cudaEventRecord(g_trace_ev[k], st) : cudaSuccess;
  }
  // Names the kernel just launched on st and records its end event.
  cudaError_t after(const char* name, cudaStream_t st) {
    const int k = 2 * g_last_count + 1;
    if (g_last_count < kMaxTrace / 2) g_last_names[g_last_count++] = name;
    return k < g_trace_n ? cudaEventRecord(g_trace_ev[k], st) : cudaSuccess;
  }
};

gdn_status cuda_fail(cudaError_t e) {
  g_last_cuda_error = (int)e;
  return GDN_ERR_CUDA;
}

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// ---- one-time, per-device set-up ----
constexpr int kMaxDevices = 64;
std::mutex g_setup_mu;
bool g_setup_done[kMaxDevices] = {};
int g_sm_count[kMaxDevices] = {};
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn g_encode = nullptr;

gdn_status device_setup(int* dev_out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev < 0 || dev >= kMaxDevices) return GDN_ERR_UNSUPPORTED;
  *dev_out = dev;
  std::lock_guard<std::mutex> lk(g_setup_mu);
  if (g_setup_done[dev]) return GDN_OK;
  if (!g_encode) {
    cudaDriverEntryPointQueryResult q;
    void* fn = nullptr;
    e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !fn) return cuda_fail(e == cudaSuccess ? cudaErrorUnknown : e);
    g_encode = reinterpret_cast<EncodeTiledFn>(fn);
  }
  if ((e = scan_kernel_setup()) != cudaSuccess) return cuda_fail(e);
  if ((e = wy_kernel_setup()) != cudaSuccess) return cuda_fail(e);
  if ((e = combine_kernel_setup()) != cudaSuccess) return cuda_fail(e);
  if ((e = f32_kernel_setup()) != cudaSuccess) return cuda_fail(e);
  if ((e = bwd_kernel_setup()) != cudaSuccess) return cuda_fail(e);
  if ((e = kv_f32_setup()) != cudaSuccess) return cuda_fail(e);
  if ((e = kv_few_setup()) != cudaSuccess) return cuda_fail(e);
  if ((e = kv_many_setup()) != cudaSuccess) return cuda_fail(e);
  if ((e = rope_bwd_setup()) != cudaSuccess) return cuda_fail(e);
  int sms = 0;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return cuda_fail(e);
  g_sm_count[dev] = sms;
  g_setup_done[dev] = true;
  return GDN_OK;
}

// AutoCP's choice of lambda (FlashQLA pages, section "AutoCP": the degree
// of parallelism follows L = lambda sqrt(N)).  The scan kernel runs one CTA
// per (segment, value head), one CTA per SM; a CTA takes about (segment
// chunks + 3) chunk-times (start-up, pipeline fill and warmup chunks).  The
// block scheduler hands CTAs out in launch order (the segments of sequence
// 0, 1, ..., then the next value head) to whichever SM frees first, so the
// planner replays that list schedule.  The combine then walks each
// sequence's segments in order, about a chunk-time per segment.  Among
// lambda = k/8 the planner takes the smallest (schedule finish + the largest
// segment count of a sequence); ties go to fewer segments.
namespace {

constexpr int kCtaOverheadChunks = 3;

// The model's constants per path.  The bf16 scan: a CTA costs its chunks + 3
// (start-up, pipeline fill, warmup) and a combine step about a chunk.
// The fp32 path: a chunk is ~40x a combine step and the start-up is small
// against a chunk, so both count zero; its chains run two CTAs per SM.
struct PlanModel {
  int overhead;     // chunk-times a CTA costs beyond its chunks
  bool combine;     // count the combine's serial steps
};

struct SegStats {
  int64_t segs = 0;
  int longest = 0, most_segs = 0;
  int64_t work = 0;  // sum of (chunks + overhead) over one head's segments
};

SegStats seg_stats(const gdn_dims* d, const int32_t* cu, int q8, const PlanModel& m) {
  SegStats r;
  for (int n = 0; n < d->n_seqs; ++n) {
    const int64_t len = cu ? (int64_t)cu[n + 1] - cu[n] : d->T;
    const int N = chunks_of(len);
    const int ns = seg_count(N, q8, false);
    r.segs += ns;
    r.work += N + (int64_t)ns * m.overhead;
    r.longest = std::max(r.longest, (N + ns - 1) / ns);  // balanced split: ceil(N / ns) at most
    r.most_segs = std::max(r.most_segs, ns);
  }
  return r;
}

// Finish time of the list schedule of the scan's CTAs on sm_count SMs.  The
// earliest free time never decreases along the schedule, so SM free times
// are kept as counts per time step and the earliest is found by a forward
// scan; the finish is at most total / sm_count + the longest CTA (the list
// scheduling bound), which sizes the count array.
int64_t list_schedule(const gdn_dims* d, const int32_t* cu, int q8, int sm_count, const SegStats& st,
                      const PlanModel& m, std::vector<int32_t>& free_at) {
  const int64_t horizon = st.work * d->h_v / sm_count + st.longest + m.overhead + 2;
  free_at.assign((size_t)horizon, 0);
  free_at[0] = sm_count;
  int64_t t = 0, finish = 0;
  for (int j = 0; j < d->h_v; ++j)
    for (int n = 0; n < d->n_seqs; ++n) {
      const int64_t len = cu ? (int64_t)cu[n + 1] - cu[n] : d->T;
      const int N = chunks_of(len);
      const int ns = seg_count(N, q8, false);
      for (int s = 0; s < ns; ++s) {
        while (free_at[(size_t)t] == 0) ++t;
        --free_at[(size_t)t];
        const int64_t end = t + seg_first(s + 1, N, ns) - seg_first(s, N, ns) + m.overhead;
        ++free_at[(size_t)end];
        finish = std::max(finish, end);
      }
    }
  return finish;
}

}  // namespace

int pick_lambda_q8_uncached(const gdn_dims* d, const int32_t* cu, int slots, const PlanModel& m) {
  int best_q8 = 256;
  int64_t best_cost = INT64_MAX, best_segs = INT64_MAX;
  std::vector<int32_t> free_at;
  for (int q8 = 32; q8 <= 4096; q8 += 32) {
    const SegStats st = seg_stats(d, cu, q8, m);
    const int64_t comb = m.combine ? 2 * st.most_segs : 0;
    // in half chunk-times; no schedule ends before its longest CTA or the average slot load
    const int64_t total = st.work * d->h_v;
    const int64_t lower = 2 * std::max<int64_t>(st.longest + m.overhead, (total + slots - 1) / slots) + comb;
    if (lower > best_cost || (lower == best_cost && st.segs >= best_segs)) continue;
    const int64_t cost = 2 * list_schedule(d, cu, q8, slots, st, m, free_at) + comb;
    if (cost < best_cost || (cost == best_cost && st.segs < best_segs)) {
      best_cost = cost;
      best_segs = st.segs;
      best_q8 = q8;
    }
  }
  return best_q8;
}

// The choice depends only on the sequence lengths, h_v, the SM count and the
// path; a model plans the same lengths once per layer, so recent choices are
// kept.
int pick_lambda_q8(const gdn_dims* d, const int32_t* cu, int sm_count) {
  struct Entry {
    int h_v, sm_count, dtype;
    std::vector<int64_t> lens;
    int q8;
  };
  static std::mutex mu;
  static std::vector<Entry> recent;  // most recent last
  std::vector<int64_t> lens((size_t)d->n_seqs);
  for (int n = 0; n < d->n_seqs; ++n) lens[(size_t)n] = cu ? (int64_t)cu[n + 1] - cu[n] : d->T;
  {
    std::lock_guard<std::mutex> lk(mu);
    for (const Entry& e : recent)
      if (e.h_v == d->h_v && e.sm_count == sm_count && e.dtype == d->dtype && e.lens == lens) return e.q8;
  }
  const bool f32 = d->dtype == GDN_F32;
  const PlanModel m = f32 ? PlanModel{0, false} : PlanModel{kCtaOverheadChunks, true};
  const int q8 = pick_lambda_q8_uncached(d, cu, f32 ? 2 * sm_count : sm_count, m);
  std::lock_guard<std::mutex> lk(mu);
  if (recent.size() >= 8) recent.erase(recent.begin());
  recent.push_back(Entry{d->h_v, sm_count, d->dtype, std::move(lens), q8});
  return q8;
}

gdn_status check_dims(const gdn_dims* d) {
  if (!d) return GDN_ERR_INVALID_ARG;
  if (d->d_k != kDim || d->d_v != kDim) return GDN_ERR_UNSUPPORTED;
  if (d->dtype != GDN_BF16 && d->dtype != GDN_F32) return GDN_ERR_UNSUPPORTED;
  if (d->B < 1 || d->T < 0 || d->h_qk < 1 || d->h_v < 1 || d->n_seqs < 1) return GDN_ERR_INVALID_ARG;
  if ((int64_t)d->B * d->T > (int64_t)0x7fffffff - kChunk) return GDN_ERR_INVALID_ARG;
  if (d->h_qk > 65535 || d->h_v > 65535) return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}

// ---- tensor maps: [tokens, heads, 128] -> 3-D (d, head, token), 64x1x64 boxes, 128B swizzle ----
gdn_status encode_map(CUtensorMap* m, const void* base, int heads, int64_t tokens, bool f32) {
  const cuuint64_t esz = f32 ? 4 : 2;
  cuuint64_t dims[3] = {(cuuint64_t)kDim, (cuuint64_t)heads, (cuuint64_t)(tokens > 0 ? tokens : 1)};
  cuuint64_t strides[2] = {(cuuint64_t)kDim * esz, (cuuint64_t)heads * kDim * esz};
  cuuint32_t box[3] = {(cuuint32_t)(f32 ? 32 : 64), 1, (cuuint32_t)kChunk};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = g_encode(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                        const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    g_last_cuda_error = (int)r;
    return GDN_ERR_CUDA;
  }
  return GDN_OK;
}

// o: [tokens, h_v, 128] bf16 -> 3-D (d, head, token), whole 128 x 1 x 64 boxes, no swizzle
// (the scan stores each chunk's o from a plain [64][128] shared-memory tile).
gdn_status encode_out_map(CUtensorMap* m, void* base, int heads, int64_t tokens) {
  cuuint64_t dims[3] = {(cuuint64_t)kDim, (cuuint64_t)heads, (cuuint64_t)(tokens > 0 ? tokens : 1)};
  cuuint64_t strides[2] = {(cuuint64_t)kDim * 2, (cuuint64_t)heads * kDim * 2};
  cuuint32_t box[3] = {(cuuint32_t)kDim, 1, (cuuint32_t)kChunk};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    g_last_cuda_error = (int)r;
    return GDN_ERR_CUDA;
  }
  return GDN_OK;
}

// ---- fixed device workspace for callers that cannot allocate ----
// 8 MiB: small problems only (the chunk records take 41472 bytes per
// (chunk, value head); context parallelism adds three 64 KB states per
// (segment, value head)).
constexpr size_t kStaticWorkspaceBytes = size_t(8) << 20;
static __device__ __align__(256) uint8_t g_static_workspace[kStaticWorkspaceBytes];
void* g_static_ws_dev[kMaxDevices] = {};

// Device address of g_static_workspace on the current device, looked up once
// per device (the host-side name is not a device address).
gdn_status static_workspace(void** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev < 0 || dev >= kMaxDevices) return GDN_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lk(g_setup_mu);
  if (!g_static_ws_dev[dev]) {
    void* ptr = nullptr;
    e = cudaGetSymbolAddress(&ptr, g_static_workspace);
    if (e != cudaSuccess || !ptr) return cuda_fail(e == cudaSuccess ? cudaErrorInvalidSymbol : e);
    g_static_ws_dev[dev] = ptr;
  }
  *out = g_static_ws_dev[dev];
  return GDN_OK;
}

// ---- the 8-bit key/value cache ----
// Checks shared by its entry points; es: bytes of an element.
gdn_status check_kv(const gdn_kv_dims* d, const gdn_kv_cache* c, const int32_t* lens, const int32_t* table,
                    const int32_t* cu) {
  if (!d || !c) return GDN_ERR_INVALID_ARG;
  if (c->d != kHeadDim) return GDN_ERR_UNSUPPORTED;
  if (d->dtype != GDN_BF16 && d->dtype != GDN_F32) return GDN_ERR_UNSUPPORTED;
  if (!c->k || !c->v || !c->k_scale || !c->v_scale || !c->status || !lens || !table) return GDN_ERR_INVALID_ARG;
  if (!aligned16(c->k) || !aligned16(c->v)) return GDN_ERR_MISALIGNED;
  if ((reinterpret_cast<uintptr_t>(c->k_scale) | reinterpret_cast<uintptr_t>(c->v_scale) |
       reinterpret_cast<uintptr_t>(c->status) | reinterpret_cast<uintptr_t>(lens) |
       reinterpret_cast<uintptr_t>(table) | reinterpret_cast<uintptr_t>(cu)) & 3u)
    return GDN_ERR_MISALIGNED;
  if (d->n_seqs < 1 || d->T < 0 || d->max_pages < 1 || c->n_pages < 1 || c->h_kv < 1 || c->h_kv > 65535)
    return GDN_ERR_INVALID_ARG;
  if ((int64_t)c->n_pages * c->h_kv > 0x7fffffff || d->max_pages > 0x7fffffff / kPage) return GDN_ERR_INVALID_ARG;
  if (!cu && d->T % d->n_seqs) return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}

// A token stride in elements: 0 selects packed rows of `heads` heads.
gdn_status kv_stride(int64_t given, int heads, int dtype, int64_t* out) {
  const int64_t packed = (int64_t)heads * kHeadDim;
  *out = given ? given : packed;
  if (*out < packed || *out > ((int64_t)1 << 40)) return GDN_ERR_INVALID_ARG;
  return *out % (dtype == GDN_F32 ? 4 : 8) ? GDN_ERR_MISALIGNED : GDN_OK;
}

KvArgs kv_args(const gdn_kv_dims* d, const gdn_kv_cache* c, const int32_t* lens, const int32_t* table,
               const int32_t* cu) {
  KvArgs a;
  a.lens = lens;
  a.table = table;
  a.cu = cu;
  a.k = static_cast<uint8_t*>(c->k);
  a.v = static_cast<uint8_t*>(c->v);
  a.k_scale = c->k_scale;
  a.v_scale = c->v_scale;
  a.status = c->status;
  a.n_seqs = d->n_seqs;
  a.T = d->T;
  a.n_each = cu ? 0 : d->T / d->n_seqs;
  a.h_q = d->h_q;
  a.h_kv = c->h_kv;
  a.max_pages = d->max_pages;
  a.n_pages = c->n_pages;
  return a;
}

// What moving keys and values in or out takes beside the tensors, and the
// number of page slots of the call.
gdn_status kv_moves(const gdn_kv_dims* d, const gdn_kv_cache* cache, const int32_t* lens, const int32_t* table,
                    const int32_t* cu, KvAppendArgs* a, unsigned* n_entries) {
  gdn_status st;
  if ((st = kv_stride(d->k_stride, cache->h_kv, d->dtype, &a->k_stride)) != GDN_OK) return st;
  if ((st = kv_stride(d->v_stride, cache->h_kv, d->dtype, &a->v_stride)) != GDN_OK) return st;
  a->c = kv_args(d, cache, lens, table, cu);
  // n tokens from any position lie in at most (n + 62) / 64 + 1 pages
  a->pages_each = cu ? 0 : (a->c.n_each + 62) / kPage + 1;
  const int64_t entries = cu ? (int64_t)d->T / kPage + 2 * (int64_t)std::min(d->n_seqs, d->T)
                             : (int64_t)d->n_seqs * a->pages_each;
  if (entries > 0x7fffffff) return GDN_ERR_INVALID_ARG;
  *n_entries = (unsigned)entries;
  return GDN_OK;
}

gdn_status kv_move(bool read, void* k, void* v, const int32_t* lens, const int32_t* table, const int32_t* cu,
                   const gdn_kv_cache* cache, const gdn_kv_dims* d, void* stream) {
  gdn_status st = check_kv(d, cache, lens, table, cu);
  if (st != GDN_OK) return st;
  KvAppendArgs a;
  unsigned entries = 0;
  if ((st = kv_moves(d, cache, lens, table, cu, &a, &entries)) != GDN_OK) return st;
  if (d->T == 0) return GDN_OK;
  if (!k || !v) return GDN_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v)) return GDN_ERR_MISALIGNED;
  a.k = k;
  a.v = v;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const bool f32 = d->dtype == GDN_F32;
  LaunchLog log;
  cudaError_t e = log.before(cs);
  if (e == cudaSuccess) e = read ? launch_kv_read(a, f32, entries, cs) : launch_kv_append(a, f32, entries, cs);
  if (e == cudaSuccess) e = log.after(read ? "kv_read" : "kv_append", cs);
  return e == cudaSuccess ? GDN_OK : cuda_fail(e);
}

// ---- between the projections and the mixers ----
bool misaligned16(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!aligned16(p)) return true;
  return false;
}

// eps of a norm: 0 selects the default.  From 1e-20 on, squares that fp32 drops
// (below 1e-38 each, 128 of them) are nothing beside it; up to 1e20 it is nothing
// beside a sum of squares past 3e38 (its mean past 2e36), which the kernels take
// of scaled elements and without it.
gdn_status norm_eps(float given, float* out) {
  *out = given == 0.f ? 1e-6f : given;
  return *out >= 1e-20f && *out <= 1e20f ? GDN_OK : GDN_ERR_INVALID_ARG;
}

gdn_status rope_args(const gdn_rope* rope, int norm, float eps, RopeArgs* r) {
  if (norm < GDN_NORM_NONE || norm > GDN_NORM_UNIT) return GDN_ERR_UNSUPPORTED;
  r->turns = nullptr;
  r->rot = r->interleaved = 0;
  r->magnitude = 1.f;
  r->norm = norm;
  r->inv_n = norm == GDN_NORM_RMS ? 1.0f / kRopeD : 1.0f;
  if (rope) {
    if (rope->rot < 0 || rope->rot > kRopeD || rope->rot % 8) return GDN_ERR_UNSUPPORTED;
    if (rope->layout != GDN_ROPE_HALF && rope->layout != GDN_ROPE_INTERLEAVED) return GDN_ERR_UNSUPPORTED;
    if (!std::isfinite(rope->magnitude) || rope->magnitude < 0.f) return GDN_ERR_INVALID_ARG;
    if (rope->rot && !rope->turns) return GDN_ERR_INVALID_ARG;
    if (rope->rot && !aligned16(rope->turns)) return GDN_ERR_MISALIGNED;
    r->turns = rope->turns;
    r->rot = rope->rot;
    r->interleaved = rope->layout;
    if (rope->magnitude != 0.f) r->magnitude = rope->magnitude;
  }
  return norm_eps(eps, &r->eps);
}

// An output in place of its input has its token stride: with another it would
// write rows that are yet to be read.
bool other_rows(const void* in, int64_t in_stride, const void* out, int64_t out_stride, int T) {
  return in && in == out && in_stride != out_stride && T > 1;
}

// CTAs whose warps share the heads of a call: `most`, but a head of two tokens
// for a warp at least.  A warp's heads are counted in 32 bits.
gdn_status rope_ctas(int64_t most, QkRopeArgs* a) {
  const int64_t units = ((int64_t)a->pos.T + 1) / 2 * (a->side[0].heads + a->side[1].heads);
  a->ctas = (int)std::max<int64_t>(1, std::min((units + kRopeWarps - 1) / kRopeWarps, most));
  return units / a->ctas / kRopeWarps >= INT_MAX - 1 ? GDN_ERR_INVALID_ARG : GDN_OK;
}
constexpr int kRopeCtas = 4 * 152;  // what is resident of the forward

// Checks of gdn_qk_rope and its gradient that do not need the tensors.
gdn_status qk_rope_args(const gdn_rope_dims* d, const gdn_rope* rope, const float* q_weight, const float* k_weight,
                        const int32_t* positions, const int32_t* cu, QkRopeArgs* a) {
  if (!d) return GDN_ERR_INVALID_ARG;
  if (d->dtype != GDN_BF16 && d->dtype != GDN_F32) return GDN_ERR_UNSUPPORTED;
  if (d->n_seqs < 1 || d->T < 0 || d->h_q < 0 || d->h_k < 0 || d->h_q > 65535 || d->h_k > 65535 || d->h_q + d->h_k < 1)
    return GDN_ERR_INVALID_ARG;
  if (!positions && !cu && d->T % d->n_seqs) return GDN_ERR_INVALID_ARG;
  std::memset(a, 0, sizeof(*a));
  gdn_status st = rope_args(rope, d->norm, d->eps, &a->r);
  if (st != GDN_OK) return st;
  if (d->norm == GDN_NORM_NONE && (q_weight || k_weight)) return GDN_ERR_INVALID_ARG;
  if (misaligned16({q_weight, k_weight}) || (reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(cu)) & 3u)
    return GDN_ERR_MISALIGNED;
  RopeSide &q = a->side[0], &k = a->side[1];
  if ((st = kv_stride(d->q_stride, d->h_q, d->dtype, &q.in_stride)) != GDN_OK) return st;
  if ((st = kv_stride(d->k_stride, d->h_k, d->dtype, &k.in_stride)) != GDN_OK) return st;
  if ((st = kv_stride(d->q_out_stride, d->h_q, d->dtype, &q.out_stride)) != GDN_OK) return st;
  if ((st = kv_stride(d->k_out_stride, d->h_k, d->dtype, &k.out_stride)) != GDN_OK) return st;
  if ((st = kv_stride(d->dq_stride, d->h_q, d->dtype, &q.dx_stride)) != GDN_OK) return st;
  if ((st = kv_stride(d->dk_stride, d->h_k, d->dtype, &k.dx_stride)) != GDN_OK) return st;
  a->pos = {positions, cu, nullptr, d->n_seqs, d->T, positions || cu ? 0 : d->T / d->n_seqs};
  q.weight = q_weight;
  k.weight = k_weight;
  q.heads = d->h_q;
  k.heads = d->h_k;
  return GDN_OK;
}

// Tokens a warp (backward: each of a CTA's) takes in a row, of heads whose norm is
// taken and of the others, so that the warps (CTAs) are `fill`, what is resident or
// twice that, or a multiple, and all end together: the former cost `cost` times the
// others.  More tokens read less twice, the W - 1 before each run; past 192 that
// is nothing.  Multiples of `group`, the tokens of straight code.
void conv_runs(int64_t T, int64_t others, int64_t fill, double cost, int64_t group, int64_t warps, ConvArgs* a) {
  constexpr int64_t kLeast = 8, kMost = 192;
  const double width = a->n_unit * cost + others;
  const double waves = std::max(1.0, std::ceil((double)T / warps * width / (double)(fill * kMost)));
  for (int i = 0; i < 2; ++i) {
    const int64_t runs = std::max<int64_t>(1, (int64_t)(waves * fill / width * (i ? 1.0 : cost)));
    const int64_t run = std::min(std::max((T + runs * warps - 1) / (runs * warps), kLeast), kMost);
    a->run[i] = (int)((run + group - 1) / group * group);
    a->runs[i] = (int)((T + a->run[i] * warps - 1) / (a->run[i] * warps));
  }
}
constexpr int64_t kConvFill = 152 * 48;    // warps: twice what is resident
constexpr int64_t kConvBwdFill = 152 * 2;  // CTAs
// Measured on 2 + 2 + 8 heads: a token of a head whose norm is taken against one of the others.
constexpr double kConvUnitCost = 1.1, kConvBwdUnitCost = 1.5;

gdn_status conv_args(const gdn_conv_dims* d, const float* weight, const float* bias, const int32_t* cu, ConvArgs* a) {
  if (!d) return GDN_ERR_INVALID_ARG;
  if (d->dtype != GDN_BF16 && d->dtype != GDN_F32) return GDN_ERR_UNSUPPORTED;
  if (d->width < 2 || d->width > kConvMaxTaps) return GDN_ERR_UNSUPPORTED;
  if (d->activation != GDN_ACT_NONE && d->activation != GDN_ACT_SILU) return GDN_ERR_UNSUPPORTED;
  if (d->norm != 0 && d->norm != 1) return GDN_ERR_UNSUPPORTED;
  if (d->n_seqs < 1 || d->T < 0 || d->h_qk < 1 || d->h_v < 1 || d->h_qk > 16384 || d->h_v > 32768) return GDN_ERR_INVALID_ARG;
  if (!cu && d->T % d->n_seqs) return GDN_ERR_INVALID_ARG;
  std::memset(a, 0, sizeof(*a));
  gdn_status st = norm_eps(d->eps, &a->eps);
  if (st != GDN_OK) return st;
  const int heads = 2 * d->h_qk + d->h_v;
  if ((st = kv_stride(d->x_stride, heads, d->dtype, &a->x_stride)) != GDN_OK) return st;
  if ((st = kv_stride(d->dx_stride, heads, d->dtype, &a->dx_stride)) != GDN_OK) return st;
  // what is indexed by 32-bit block numbers
  if ((int64_t)d->T * heads >= (int64_t)1 << 33 || (int64_t)d->n_seqs * heads >= (int64_t)1 << 30) return GDN_ERR_INVALID_ARG;
  if (misaligned16({weight, bias}) || reinterpret_cast<uintptr_t>(cu) & 3u) return GDN_ERR_MISALIGNED;
  a->weight = weight;
  a->bias = bias;
  a->cu = cu;
  a->n_seqs = d->n_seqs;
  a->T = d->T;
  a->n_each = cu ? 0 : d->T / d->n_seqs;
  a->h_qk = d->h_qk;
  a->h_v = d->h_v;
  a->width = d->width;
  a->silu = d->activation == GDN_ACT_SILU;
  a->norm = d->norm;
  a->n_unit = d->norm ? 2 * d->h_qk : 0;
  return GDN_OK;
}

bool overlap(const void* a, const void* b, size_t bytes) {
  if (!a || !b) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + bytes && y < x + bytes;
}
size_t conv_state_bytes(const gdn_conv_dims* d) {
  return (size_t)d->n_seqs * (d->width - 1) * (2 * d->h_qk + d->h_v) * kConvD * (d->dtype == GDN_F32 ? 4 : 2);
}
constexpr int kConvBwdWarps = 8;  // runs of a CTA of the gradient
// Sets the runs of the gradient; returns its workspace, which is enough with and
// without the norm.
size_t conv_bwd_plan(const gdn_conv_dims* d, ConvArgs* a) {
  const int heads = 2 * d->h_qk + d->h_v;
  size_t most = 0;
  for (int n_unit : {2 * d->h_qk - a->n_unit, a->n_unit}) {  // the call's own last
    a->n_unit = n_unit;
    conv_runs(d->T, heads - n_unit, kConvBwdFill, kConvBwdUnitCost, 4, kConvBwdWarps, a);
    const size_t rows = (size_t)a->runs[0] * n_unit + (size_t)a->runs[1] * (heads - n_unit);
    most = std::max(most, rows * (d->width + 1) * kConvD * sizeof(float));
  }
  return most;
}

// A pool of codes as [page and head][64 tokens][128 bytes]: boxes of one page's
// codes of one head, in the swizzled image the MMAs read.
gdn_status encode_kv_map(CUtensorMap* m, void* base, const gdn_kv_cache* c) {
  cuuint64_t dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)kPage, (cuuint64_t)c->n_pages * c->h_kv};
  cuuint64_t strides[2] = {(cuuint64_t)kHeadDim, (cuuint64_t)kPageBytes};
  cuuint32_t box[3] = {(cuuint32_t)kHeadDim, (cuuint32_t)kPage, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, base, dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    g_last_cuda_error = (int)r;
    return GDN_ERR_CUDA;
  }
  return GDN_OK;
}

// Kernels of gdn_kv_attn.
constexpr int kKvPathF32 = 0;   // fp32
constexpr int kKvPathFew = 1;   // bf16, row tiles of up to 32: few rows (tokens times heads of a group), small calls
constexpr int kKvPathMany = 2;  // bf16, row tiles of 256
// What parts and the second kernel cost, in key tiles, against whole items:
// for few rows 6 us at 0.7 us a tile; in fp32 6 us at 2 us a tile; for many rows,
// at 1.5 us a tile, 18 us and more the longer a run is (`tiles`), since it then
// begins and ends more items, up to some 42 us.  Items of one tile are never
// cut: that leaves some 3 us of the second kernel's launch.
int64_t kv_join_tiles(int path, int64_t tiles, bool one_tile) {
  if (one_tile) return path == kKvPathMany ? 2 : path == kKvPathFew ? 4 : 1;
  return path == kKvPathMany ? std::min<int64_t>(28, 12 + tiles / 4) : path == kKvPathFew ? 8 : 3;
}
// Row tiles of a call: no sequence has more than max_row_tiles, and all of them
// no more than their tokens fill with one started tile each.
int64_t kv_most_row_tiles(int n_seqs, int T, int group, int rows, int max_row_tiles) {
  return std::min<int64_t>((int64_t)n_seqs * max_row_tiles, (int64_t)T * group / rows + n_seqs);
}
// Row tiles whose units the kernels can count in 32 bits, whatever the lengths on the device turn out to be.
int64_t kv_row_tiles_counted(const gdn_kv_dims* d, int h_kv, const gdn_kv_plan_t& p) {
  return 0x7fffffff / ((int64_t)d->max_pages * kPage / kKvTile + 1 + p.item_cost) / h_kv;
}
// The attention kernels round lengths up to a tile of keys in 32 bits.
constexpr int kKvMostPages = (0x7fffffff - kKvTile) / kPage;
constexpr int kKvMaxParts = 32;  // of an item on the path for many rows: a warp of the second kernel takes a row's in turn

}  // namespace

extern "C" {

const char* gdn_status_string(gdn_status s) {
  switch (s) {
    case GDN_OK: return "ok";
    case GDN_ERR_INVALID_ARG: return "invalid argument";
    case GDN_ERR_UNSUPPORTED: return "unsupported (d_k/d_v must be 128; dtype bf16 or f32)";
    case GDN_ERR_MISALIGNED: return "misaligned pointer (16 bytes; workspace 256 bytes)";
    case GDN_ERR_CUDA: return "CUDA call failed";
    case GDN_ERR_DEVICE_TIMEOUT: return "a bounded on-device wait timed out";
    case GDN_ERR_WORKSPACE: return "workspace missing or too small";
    case GDN_ERR_DEVICE_CHECK: return "a kernel's consistency check failed";
  }
  return "unknown status";
}

int gdn_last_cuda_error(void) { return g_last_cuda_error; }

gdn_status gdn_cp_plan(const gdn_dims* dims, const int32_t* cu, const gdn_cp_opts* opts, gdn_cp_plan_t* out) {
  if (!out) return GDN_ERR_INVALID_ARG;
  gdn_status st = check_dims(dims);
  if (st != GDN_OK) return st;
  const int64_t T_total = (int64_t)dims->B * dims->T;
  if (cu) {
    if (dims->B != 1) return GDN_ERR_INVALID_ARG;
    if (cu[0] != 0 || cu[dims->n_seqs] != dims->T) return GDN_ERR_INVALID_ARG;
    for (int n = 0; n < dims->n_seqs; ++n)
      if (cu[n + 1] < cu[n]) return GDN_ERR_INVALID_ARG;
  } else if (dims->n_seqs != dims->B) {
    return GDN_ERR_INVALID_ARG;
  }
  gdn_cp_opts o = {GDN_CP_AUTO, 0.0f, 8, 1e-4f, 0, GDN_TOL_NOISE};  // NULL opts: the planner picks lambda
  if (opts) o = *opts;
  if (o.mode < GDN_CP_OFF || o.mode > GDN_CP_AUTO) return GDN_ERR_UNSUPPORTED;
  if (o.tol_rule != GDN_TOL_FIXED && o.tol_rule != GDN_TOL_NOISE) return GDN_ERR_UNSUPPORTED;
  const bool auto_lambda = !(o.lambda > 0.f);
  if (o.lambda > 1000.f) return GDN_ERR_INVALID_ARG;
  if (o.warmup_chunks <= 0) o.warmup_chunks = 8;
  if (!(o.warmup_tol > 0.f)) o.warmup_tol = 1e-4f;
  if (o.sm_count <= 0) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_fail(e);
    o.sm_count = sms;
  }
  int mode = o.mode;
  if (mode == GDN_CP_AUTO) mode = ((int64_t)dims->n_seqs * dims->h_v < o.sm_count) ? GDN_CP_WARMUP : GDN_CP_OFF;

  gdn_cp_plan_t p;
  std::memset(&p, 0, sizeof(p));
  p.mode = mode;
  p.n_seqs = dims->n_seqs;
  p.T_total = (int)T_total;
  p.h_v = dims->h_v;
  p.h_qk = dims->h_qk;
  p.dtype = dims->dtype;
  if (auto_lambda) {
    p.lambda_q8 = mode == GDN_CP_OFF ? 256 : pick_lambda_q8(dims, cu, o.sm_count);
  } else {
    p.lambda_q8 = (int)std::lround(o.lambda * 256.0);
    if (p.lambda_q8 < 1) p.lambda_q8 = 1;
  }
  p.warmup_chunks = o.warmup_chunks;
  p.warmup_tol = o.warmup_tol;
  p.sm_count = o.sm_count;
  p.tol_rule = o.tol_rule;
  int64_t n_seg_total = 0, n_chunks_total = 0;
  for (int n = 0; n < dims->n_seqs; ++n) {
    const int64_t len = cu ? (int64_t)cu[n + 1] - cu[n] : dims->T;
    const int N = chunks_of(len);
    n_chunks_total += N;
    const int ns = seg_count(N, p.lambda_q8, mode == GDN_CP_OFF);
    n_seg_total += ns;
    if (N > p.max_chunks) p.max_chunks = N;
    for (int s = 0; s < ns; ++s) {
      const int w = seg_first(s + 1, N, ns) - seg_first(s, N, ns);
      if (w > p.max_seg_chunks) p.max_seg_chunks = w;
    }
  }
  if (n_seg_total > 0x7fffffff) return GDN_ERR_INVALID_ARG;
  if (n_chunks_total * std::max(dims->h_v, dims->h_qk) > 0x7fffffff) return GDN_ERR_INVALID_ARG;
  p.n_seg_total = (int)n_seg_total;
  p.n_chunks_total = (int)n_chunks_total;
  // workspace: status | head modes + bounds | segment bounds | R | S_loc | S_start |
  //            chunk index | chunk records (the last two: bf16 path only)
  const size_t heads = (size_t)dims->n_seqs * dims->h_v;
  const size_t segheads = (size_t)n_seg_total * dims->h_v;
  size_t off = 256;
  p.off_head = off;
  off = align_up(off + heads * 8, 256);
  p.off_seg_bound = off;  // seg_bound (fp32) then seg_w (int32)
  off = align_up(off + segheads * 8, 256);
  if (mode != GDN_CP_OFF) {
    const size_t mat = (size_t)kDim * kDim * 4;
    p.off_R = off;
    off += segheads * mat;
    p.off_Sloc = off;
    off += segheads * mat;
    p.off_Sstart = off;
    off += segheads * mat;
  }
  if (dims->dtype == GDN_BF16) {
    p.off_chunk_map = off;  // chunk index (sequence bases, then 16-byte chunk records), then the chunk
                            // warmup exponents
    off = align_up(off + ((size_t)dims->n_seqs + 1) * 4, 16) + (size_t)n_chunks_total * 16;
    off = align_up(off, 256);
    off = align_up(off + (size_t)n_chunks_total * dims->h_v * 4, 1024);
    p.off_wy = off;
    off += (size_t)n_chunks_total * dims->h_v * kRecBytes;
  }
  p.workspace_bytes = off;
  *out = p;
  return GDN_OK;
}

// The forward.  For the backward (hchunk != null) the WY and output-scan
// kernels also write A^T (wyA) and every output chunk's start state (hchunk),
// in the plan's own mode; *p_out receives the
// problem the kernels run with.  launch = false: only that problem (the
// backward of a forward that already ran with the same arguments).
static gdn_status forward_impl(const void* q, const void* k, const void* v, const float* g, const float* beta,
                               const float* initial_state, const int32_t* cu_dev, void* out, float* final_state,
                               const gdn_dims* dims, const gdn_cp_plan_t* plan, void* workspace,
                               size_t workspace_bytes, void* stream, uint8_t* wyA, uint8_t* hchunk,
                               Problem* p_out, bool launch = true) {
  gdn_status st = check_dims(dims);
  if (st != GDN_OK) return st;
  if (!plan) return GDN_ERR_INVALID_ARG;
  const int64_t T_total = (int64_t)dims->B * dims->T;
  if (plan->n_seqs != dims->n_seqs || plan->T_total != T_total || plan->h_v != dims->h_v ||
      plan->h_qk != dims->h_qk || plan->dtype != dims->dtype)
    return GDN_ERR_INVALID_ARG;
  if (cu_dev && dims->B != 1) return GDN_ERR_INVALID_ARG;
  if (!cu_dev && dims->n_seqs != dims->B) return GDN_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < plan->workspace_bytes) return GDN_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return GDN_ERR_MISALIGNED;
  if (T_total > 0) {
    if (!q || !k || !v || !g || !beta || !out) return GDN_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(g) || !aligned16(beta))
      return GDN_ERR_MISALIGNED;
  }
  if ((initial_state && !aligned16(initial_state)) || (final_state && !aligned16(final_state)) ||
      (cu_dev && (reinterpret_cast<uintptr_t>(cu_dev) & 3u)))
    return GDN_ERR_MISALIGNED;

  int dev = 0;
  st = device_setup(&dev);
  if (st != GDN_OK) return st;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);

  Problem p;
  std::memset(&p, 0, sizeof(p));
  p.q = q;
  p.k = k;
  p.v = v;
  p.g = g;
  p.beta = beta;
  p.h0 = initial_state;
  p.cu = cu_dev;
  p.out = out;
  p.hT = final_state;
  p.T_row = dims->T;
  p.n_seqs = dims->n_seqs;
  p.h_qk = dims->h_qk;
  p.h_v = dims->h_v;
  p.scale = dims->scale != 0.f ? dims->scale : 1.0f / std::sqrt((float)dims->d_k);
  p.elem_f32 = dims->dtype == GDN_F32;
  p.plan_mode = plan->mode == GDN_CP_OFF ? kModeOff : (plan->mode == GDN_CP_EXACT ? kModeExact : kModeWarmup);
  // a plan in which every sequence is one segment has nothing to combine: it
  // runs without the preprocessing and the combine
  const bool cp = plan->mode != GDN_CP_OFF && plan->n_seg_total > plan->n_seqs;
  if (!cp) p.plan_mode = kModeOff;
  p.wyA = wyA;
  p.hchunk = hchunk;
  p.lambda_q8 = plan->lambda_q8;
  p.warmup_chunks = plan->warmup_chunks;
  p.log_tol = std::log(plan->warmup_tol);
  p.tol_noise = plan->tol_rule == GDN_TOL_NOISE;
  p.n_seg_total = plan->n_seg_total;
  p.status = reinterpret_cast<int*>(ws);
  p.head_mode = reinterpret_cast<int*>(ws + plan->off_head);
  p.head_bound = reinterpret_cast<float*>(ws + plan->off_head + (size_t)dims->n_seqs * dims->h_v * 4);
  p.seg_bound = reinterpret_cast<float*>(ws + plan->off_seg_bound);
  p.seg_w = reinterpret_cast<int*>(ws + plan->off_seg_bound + (size_t)plan->n_seg_total * dims->h_v * 4);
  if (plan->mode != GDN_CP_OFF) {
    p.R = reinterpret_cast<float*>(ws + plan->off_R);
    p.Sloc = reinterpret_cast<float*>(ws + plan->off_Sloc);
    p.Sstart = reinterpret_cast<float*>(ws + plan->off_Sstart);
  }
  p.n_chunks_total = plan->n_chunks_total;
  if (dims->dtype == GDN_BF16) {
    const size_t info_off = align_up(plan->off_chunk_map + ((size_t)dims->n_seqs + 1) * 4, 16);
    p.seq_chunk_base = reinterpret_cast<int32_t*>(ws + plan->off_chunk_map);
    p.chunk_info = reinterpret_cast<int4*>(ws + info_off);
    p.chunk_exp = reinterpret_cast<float*>(ws + align_up(info_off + (size_t)plan->n_chunks_total * 16, 256));
    p.wy = ws + plan->off_wy;
  }
  p.stall_ns = g_debug_stall_ns.load(std::memory_order_relaxed);
  if (!launch) {
    if (p_out) *p_out = p;
    return GDN_OK;
  }

  cudaError_t e = cudaMemsetAsync(ws, 0, 256, cs);
  if (e != cudaSuccess) return cuda_fail(e);
  if (T_total == 0) {
    // No tokens: the final state is the initial state.
    if (final_state) {
      const size_t bytes = (size_t)dims->n_seqs * dims->h_v * kDim * kDim * 4;
      e = initial_state ? cudaMemcpyAsync(final_state, initial_state, bytes, cudaMemcpyDeviceToDevice, cs)
                        : cudaMemsetAsync(final_state, 0, bytes, cs);
      if (e != cudaSuccess) return cuda_fail(e);
    }
    return GDN_OK;
  }
  if (dims->dtype == GDN_F32) {
    // fp32 inputs: the recurrence on the CUDA cores, in fp32; a context-parallel
    // plan always combines its segments exactly (no warmup restarts)
    LaunchLog log;
    if (cp) {
      p.plan_mode = kModeExact;
      if ((e = log.before(cs)) != cudaSuccess || (e = launch_f32_prep(p, cs)) != cudaSuccess ||
          (e = log.after("recurrence_f32_prep", cs)) != cudaSuccess)
        return cuda_fail(e);
      if ((e = log.before(cs)) != cudaSuccess || (e = launch_combine(p, g_sm_count[dev], cs)) != cudaSuccess ||
          (e = log.after("combine", cs)) != cudaSuccess)
        return cuda_fail(e);
    }
    if ((e = log.before(cs)) != cudaSuccess ||
        (e = launch_recurrence_f32(p, cs, cp)) != cudaSuccess ||
        (e = log.after("recurrence_f32", cs)) != cudaSuccess)
      return cuda_fail(e);
    return GDN_OK;
  }
  CUtensorMap mq, mk, mv, mo;
  const bool f32 = false;
  if ((st = encode_map(&mq, q, dims->h_qk, T_total, f32)) != GDN_OK) return st;
  if ((st = encode_map(&mk, k, dims->h_qk, T_total, f32)) != GDN_OK) return st;
  if ((st = encode_map(&mv, v, dims->h_v, T_total, f32)) != GDN_OK) return st;
  if ((st = encode_out_map(&mo, out, dims->h_v, T_total)) != GDN_OK) return st;

  // chunk index (varlen) -> WY -> [context parallel: preprocessing -> combine]
  // -> output scan
  LaunchLog log;
  if (cu_dev) {  // varlen chunk index (fixed-length rows compute it)
    if ((e = log.before(cs)) != cudaSuccess || (e = launch_chunk_map(p, cs)) != cudaSuccess ||
        (e = log.after("chunk_map", cs)) != cudaSuccess)
      return cuda_fail(e);
  }
  if ((e = log.before(cs)) != cudaSuccess || (e = launch_wy(p, mq, mk, mv, cs, cu_dev != nullptr)) != cudaSuccess ||
      (e = log.after("wy", cs)) != cudaSuccess)
    return cuda_fail(e);
  if (cp) {
    if ((e = log.before(cs)) != cudaSuccess || (e = launch_scan_prep(p, mq, mk, cs)) != cudaSuccess ||
        (e = log.after("scan_prep", cs)) != cudaSuccess)
      return cuda_fail(e);
    if ((e = log.before(cs)) != cudaSuccess || (e = launch_combine(p, g_sm_count[dev], cs)) != cudaSuccess ||
        (e = log.after("combine", cs)) != cudaSuccess)
      return cuda_fail(e);
  }
  if ((e = log.before(cs)) != cudaSuccess || (e = launch_scan_out(p, mq, mk, mo, plan->n_seg_total, cs)) != cudaSuccess ||
      (e = log.after("scan_out", cs)) != cudaSuccess)
    return cuda_fail(e);
  if (p_out) *p_out = p;
  return GDN_OK;
}

gdn_status gdn_chunk_fwd(const void* q, const void* k, const void* v, const float* g, const float* beta,
                         const float* initial_state, const int32_t* cu_dev, void* out, float* final_state,
                         const gdn_dims* dims, const gdn_cp_plan_t* plan, void* workspace,
                         size_t workspace_bytes, void* stream) {
  return forward_impl(q, k, v, g, beta, initial_state, cu_dev, out, final_state, dims, plan, workspace,
                      workspace_bytes, stream, nullptr, nullptr, nullptr);
}

// ---- backward ----
// Sections after the forward's workspace, per (chunk, value head): A^T (8 KB),
// the chunk-start state, T', E and D (32 KB each); then a bf16 o the recompute
// writes and nobody reads.
struct BwdLayout {
  size_t wyA, hchunk, tmat, emat, dstate, out, end;
};
static BwdLayout bwd_layout(const gdn_cp_plan_t* plan) {
  BwdLayout L;
  const size_t ch = (size_t)plan->n_chunks_total * plan->h_v;
  size_t off = align_up(plan->workspace_bytes, 1024);
  L.wyA = off;
  off += ch * 8192;
  L.hchunk = off;
  off += ch * 32768;
  L.tmat = off;
  off += ch * 32768;
  L.emat = off;
  off += ch * 32768;
  L.dstate = off;
  off += ch * 32768;
  L.out = off;
  off = align_up(off + (size_t)plan->T_total * plan->h_v * kDim * 2, 256);
  L.end = off;
  return L;
}

gdn_status gdn_chunk_fwd_train(const void* q, const void* k, const void* v, const float* g, const float* beta,
                               const float* initial_state, const int32_t* cu_dev, void* out, float* final_state,
                               const gdn_dims* dims, const gdn_cp_plan_t* plan, void* workspace,
                               size_t workspace_bytes, void* stream) {
  if (!plan || !dims) return GDN_ERR_INVALID_ARG;
  if (dims->dtype != GDN_BF16 || plan->dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
  const BwdLayout L = bwd_layout(plan);
  if (!workspace || workspace_bytes < L.end) return GDN_ERR_WORKSPACE;
  uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);
  return forward_impl(q, k, v, g, beta, initial_state, cu_dev, out, final_state, dims, plan, workspace,
                      workspace_bytes, stream, ws + L.wyA, ws + L.hchunk, nullptr);
}

gdn_status gdn_bwd_workspace_bytes(const gdn_cp_plan_t* plan, size_t* bytes) {
  if (!plan || !bytes) return GDN_ERR_INVALID_ARG;
  if (plan->dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
  *bytes = bwd_layout(plan).end;
  return GDN_OK;
}

gdn_status gdn_chunk_bwd(const void* q, const void* k, const void* v, const float* g, const float* beta,
                         const float* initial_state, const int32_t* cu_dev, const void* d_out,
                         const float* d_final_state, void* dq, void* dk, void* dv, float* dg, float* dbeta,
                         float* d_initial_state, const gdn_dims* dims, const gdn_cp_plan_t* plan, void* workspace,
                         size_t workspace_bytes, int reuse_forward, void* stream) {
  gdn_status st = check_dims(dims);
  if (st != GDN_OK) return st;
  if (!plan) return GDN_ERR_INVALID_ARG;
  if (dims->dtype != GDN_BF16 || plan->dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
  const BwdLayout L = bwd_layout(plan);
  if (!workspace || workspace_bytes < L.end) return GDN_ERR_WORKSPACE;
  const int64_t T_total = (int64_t)dims->B * dims->T;
  if (T_total > 0) {
    if (!d_out || !dq || !dk || !dv || !dg || !dbeta) return GDN_ERR_INVALID_ARG;
    if (!aligned16(d_out) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv) || !aligned16(dg) ||
        !aligned16(dbeta))
      return GDN_ERR_MISALIGNED;
  }
  if ((d_final_state && !aligned16(d_final_state)) || (d_initial_state && !aligned16(d_initial_state)))
    return GDN_ERR_MISALIGNED;
  uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (T_total == 0) {
    // no tokens: h_T = h0, so the gradient of h0 is that of h_T
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return GDN_ERR_MISALIGNED;
    int dev = 0;
    if ((st = device_setup(&dev)) != GDN_OK) return st;
    cudaError_t e = cudaMemsetAsync(ws, 0, 256, cs);
    if (e == cudaSuccess && d_initial_state) {
      const size_t bytes = (size_t)dims->n_seqs * dims->h_v * kDim * kDim * 4;
      e = d_final_state ? cudaMemcpyAsync(d_initial_state, d_final_state, bytes, cudaMemcpyDeviceToDevice, cs)
                        : cudaMemsetAsync(d_initial_state, 0, bytes, cs);
    }
    return e == cudaSuccess ? GDN_OK : cuda_fail(e);
  }
  Problem p;
  st = forward_impl(q, k, v, g, beta, initial_state, cu_dev, ws + L.out, nullptr, dims, plan, workspace,
                    workspace_bytes, stream, ws + L.wyA, ws + L.hchunk, &p, reuse_forward == 0);
  if (st != GDN_OK) return st;
  int dev = 0;
  if ((st = device_setup(&dev)) != GDN_OK) return st;
  // The forward above kept the chunk states of the plan's own mode (a warmup
  // restart only where its acceptance rule allows one); the state gradient's
  // chain is always combined exactly.
  if (p.plan_mode != kModeOff) p.plan_mode = kModeExact;
  BwdArgs b;
  b.dout = d_out;
  b.dhT = d_final_state;
  b.dq = dq;
  b.dk = dk;
  b.dv = dv;
  b.dg = dg;
  b.dbeta = dbeta;
  b.dh0 = d_initial_state;
  b.tmat = ws + L.tmat;
  b.emat = ws + L.emat;
  b.dstate = ws + L.dstate;
  LaunchLog log(true);
  cudaError_t e;
  if ((e = log.before(cs)) != cudaSuccess || (e = launch_bwd_pre_tc(p, b, cs)) != cudaSuccess ||
      (e = log.after("bwd_pre", cs)) != cudaSuccess)
    return cuda_fail(e);
  if (p.plan_mode != kModeOff) {
    // context parallel: per segment the transition and the local offset, then
    // the segments' end-state gradients by the combine run backwards
    if ((e = log.before(cs)) != cudaSuccess || (e = launch_bwd_chain_tc(p, b, true, cs)) != cudaSuccess ||
        (e = log.after("bwd_chain_prep", cs)) != cudaSuccess)
      return cuda_fail(e);
    Problem pc = p;
    pc.h0 = d_final_state;
    if ((e = log.before(cs)) != cudaSuccess || (e = launch_combine_bwd(pc, g_sm_count[dev], cs)) != cudaSuccess ||
        (e = log.after("bwd_combine", cs)) != cudaSuccess)
      return cuda_fail(e);
  }
  if ((e = log.before(cs)) != cudaSuccess || (e = launch_bwd_chain_tc(p, b, false, cs)) != cudaSuccess ||
      (e = log.after("bwd_chain", cs)) != cudaSuccess)
    return cuda_fail(e);
  if ((e = log.before(cs)) != cudaSuccess || (e = launch_bwd_local_tc(p, b, cs)) != cudaSuccess ||
      (e = log.after("bwd_local", cs)) != cudaSuccess)
    return cuda_fail(e);
  return GDN_OK;
}

gdn_status gdn_decode_step(const void* q, const void* k, const void* v, const float* g, const float* beta,
                           float* state, void* out, const gdn_dims* dims, void* stream) {
  gdn_status st = check_dims(dims);
  if (st != GDN_OK) return st;
  if (dims->T != 1 || dims->n_seqs != dims->B) return GDN_ERR_INVALID_ARG;
  if (!q || !k || !v || !g || !beta || !state || !out) return GDN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(g) || !aligned16(beta) || !aligned16(state) ||
      !aligned16(out))
    return GDN_ERR_MISALIGNED;
  if (dims->B > 65535 * 32768) return GDN_ERR_INVALID_ARG;
  DecodeArgs a;
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.beta = beta;
  a.state = state;
  a.out = out;
  a.n_seqs = dims->B;
  a.h_qk = dims->h_qk;
  a.h_v = dims->h_v;
  a.scale = dims->scale != 0.f ? dims->scale : 1.0f / std::sqrt((float)dims->d_k);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  LaunchLog log;
  cudaError_t e = log.before(cs);
  if (e == cudaSuccess) e = launch_decode(a, dims->dtype == GDN_F32, cs);
  if (e == cudaSuccess) e = log.after("decode", cs);
  return e == cudaSuccess ? GDN_OK : cuda_fail(e);
}

gdn_status gdn_kv_append(const void* k, const void* v, const int32_t* lens, const int32_t* table, const int32_t* cu,
                         const gdn_kv_cache* cache, const gdn_kv_dims* dims, void* stream) {
  return kv_move(false, const_cast<void*>(k), const_cast<void*>(v), lens, table, cu, cache, dims, stream);
}

gdn_status gdn_kv_read(void* k_out, void* v_out, const int32_t* lens, const int32_t* table, const int32_t* cu,
                       const gdn_kv_cache* cache, const gdn_kv_dims* dims, void* stream) {
  return kv_move(true, k_out, v_out, lens, table, cu, cache, dims, stream);
}

gdn_status gdn_kv_attn_plan(const gdn_kv_dims* d, int h_kv, int max_q_len, int max_kv_len, int sm_count,
                            gdn_kv_plan_t* out) {
  if (!d || !out) return GDN_ERR_INVALID_ARG;
  if (d->dtype != GDN_BF16 && d->dtype != GDN_F32) return GDN_ERR_UNSUPPORTED;
  if (d->causal != 0 && d->causal != 1) return GDN_ERR_UNSUPPORTED;
  if (d->n_seqs < 1 || d->T < 0 || d->h_q < 1 || h_kv < 1 || h_kv > d->h_q || d->h_q > 65535 || d->max_pages < 1 ||
      d->window < 0 || d->max_pages > kKvMostPages || !(std::isfinite(d->scale)))
    return GDN_ERR_INVALID_ARG;
  // With no bound a sequence may bring all the tokens; what follows then
  // supposes equally many each, and only speed depends on that.
  const bool bound = max_q_len > 0 && max_q_len <= d->T;
  if (!bound) max_q_len = d->T;
  const int q_len = bound ? max_q_len : (int)(((int64_t)d->T + d->n_seqs - 1) / d->n_seqs);
  const int64_t longest = (int64_t)d->max_pages * kPage;
  if (max_kv_len <= 0 || max_kv_len > longest) max_kv_len = (int)std::min<int64_t>(longest, 0x7fffffff);
  if (sm_count <= 0) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sm_count, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_fail(e);
  }
  gdn_kv_plan_t p;
  std::memset(&p, 0, sizeof(p));
  const int group = (d->h_q + h_kv - 1) / h_kv;
  if ((int64_t)d->T * group > 0x7fffffff - 4096) return GDN_ERR_INVALID_ARG;
  const int64_t rows = (int64_t)q_len * group;
  // Key tiles, every sequence taken at its longest and with q tokens, with item_cost for each item.
  struct Units {
    int64_t total, longest_item, shortest;
    int row_tiles;
  };
  auto units_of = [&](int q, int tile_rows, int item_cost) {
    Units u = {0, 0, INT64_MAX, (int)std::max<int64_t>(1, ((int64_t)q * group + tile_rows - 1) / tile_rows)};
    const int64_t past = std::max(0, max_kv_len - q);
    for (int rt = 0; rt < u.row_tiles; ++rt) {
      const int64_t t0 = (int64_t)rt * tile_rows / group;
      const int64_t t1 = std::min<int64_t>(q - 1, ((int64_t)(rt + 1) * tile_rows - 1) / group);
      const int64_t hi = d->causal ? std::min<int64_t>(past + t1 + 1, max_kv_len) : max_kv_len;
      const int64_t lo = d->window ? std::max<int64_t>(0, past + t0 - d->window + 1) : 0;
      const int64_t cost = item_cost + std::max<int64_t>(1, (hi + kKvTile - 1) / kKvTile - lo / kKvTile);
      u.total += cost;
      u.longest_item = std::max(u.longest_item, cost);
      u.shortest = std::min(u.shortest, cost);
    }
    u.total *= (int64_t)d->n_seqs * h_kv;
    return u;
  };
  p.path = kKvPathF32;
  p.rows = 128;
  p.item_cost = 2;
  int per_sm = 1;
  Units u;
  if (d->dtype == GDN_BF16) {
    // Kernel and row tile by the rows that share a key, and by how much there is
    // to do: small calls are sooner done in tiles of 32 rows, which there are more
    // of and which begin sooner, up to 8 units an SM.  Measured, tiles of 256 rows
    // and of 32 or fewer, in us: 64 sequences to 32768 tokens, 4 key/value heads, 32
    // rows 324 and 216, 48 rows 326 and 399; 8 query heads on 2, 64 tokens over 64
    // keys 14.6 and 11.0 (1 unit an SM), over 8192 keys 26.6 and 18.9 (8), over 65536
    // 54.1 and 58.7 (55), prompts of 512 tokens 20.9 and 18.2, or 13.4 as whole items
    // (9), 1024 tokens 28.2 and 31.9, or 26.9 as whole items (21).
    p.path = kKvPathFew;
    p.rows = (int)std::min<int64_t>(32, std::max<int64_t>(8, (rows + 7) / 8 * 8));  // at least 8: a call may bring no tokens
    // measured: 64 sequences to 65536 tokens, 16 rows, 62.7 us at 3 and 58.5 at 8; 256 to 32768, 8 rows, 116 at 3,
    // 111 at 4 and 113 at 12
    p.item_cost = p.rows <= 8 ? 4 : 8;
    per_sm = kv_few_ctas_per_sm(p.rows);
    // Past 32 rows without a bound, one sequence may bring most of them, which
    // small tiles would read all its keys for: it is taken to bring them all.
    if (rows > 32 && (rows >= 32 * (int64_t)sm_count || units_of(max_q_len, 32, p.item_cost).total > 8 * (int64_t)sm_count)) {
      p.path = kKvPathMany;
      p.rows = 256;
      p.item_cost = 6;
    }
  }
  u = units_of(q_len, p.rows, p.item_cost);
  p.max_row_tiles = (int)std::max<int64_t>(1, ((int64_t)max_q_len * group + p.rows - 1) / p.rows);
  if (kv_most_row_tiles(d->n_seqs, d->T, group, p.rows, p.max_row_tiles) > kv_row_tiles_counted(d, h_kv, p))
    return GDN_ERR_INVALID_ARG;
  const int64_t items = (int64_t)d->n_seqs * u.row_tiles * h_kv;
  const int64_t slots = (int64_t)per_sm * sm_count;
  // Two ways to share out the items: each whole to one CTA, the longest first
  // (n_ctas = 0), or all key tiles in equal runs, whose cut items are joined
  // by a second kernel.  Whole items end with the longest one, or with the last
  // round of equal ones; runs end together, plus the parts' way through
  // memory and the second kernel.  Measured, whole and runs, in us: 16 tokens
  // over 1024 keys of 8 heads 12.6 and 14.0, 40 over 2048 keys 46.5 and 37.9, 147
  // over 28 keys of 16 heads 55.1 and 41.2;
  // with 8 query heads on 2, 1024 tokens over 4096 keys 69 and 40, prompts of
  // 1024 tokens 28.9 and 28.8, 4096 tokens 67 and 66, 8192 tokens 119 and 149,
  // 4096 tokens over 65536 keys 794 and 694; fp32 prompts of 2048 tokens 66 and
  // 53, 4096 tokens 120 and 131 (the estimate takes runs there).
  const int64_t rounds = (items + slots - 1) / slots;  // a CTA's start in each but the first counts a unit
  const int64_t whole = rounds - 1 + (u.longest_item == u.shortest
                                          ? rounds * u.longest_item
                                          : std::max(u.longest_item, (u.total + slots - 1) / slots + u.shortest));
  const bool one_tile = u.longest_item == p.item_cost + 1;  // then runs are of whole items too
  const int64_t run = one_tile ? rounds * u.longest_item : (u.total + slots - 1) / slots;
  const int64_t runs = run + kv_join_tiles(p.path, run, one_tile);
  int64_t ctas = std::min(slots, u.total);
  if (p.path == kKvPathMany) ctas = std::min(ctas, kKvMaxParts * items);  // of 2 items, 70 parts each 32.6 us, 35 26.9
  p.n_ctas = whole <= runs ? 0 : (int)ctas;
  p.n_seqs = d->n_seqs;
  p.T = d->T;
  p.h_q = d->h_q;
  p.h_kv = h_kv;
  p.dtype = d->dtype;
  p.max_q_len = max_q_len;
  p.off_desc = 0;
  p.off_ml = align_up((size_t)2 * p.n_ctas * sizeof(int4), 256);
  p.off_o = align_up(p.off_ml + (size_t)2 * p.n_ctas * p.rows * sizeof(float2), 256);
  p.workspace_bytes = p.off_o + (size_t)2 * p.n_ctas * p.rows * kHeadDim * sizeof(float);
  *out = p;
  return GDN_OK;
}

gdn_status gdn_kv_attn(const void* q, const int32_t* lens, const int32_t* table, const int32_t* cu,
                       const gdn_kv_cache* cache, void* out, float* lse, const gdn_kv_dims* d,
                       const gdn_kv_plan_t* plan, void* workspace, size_t workspace_bytes, void* stream) {
  gdn_status st = check_kv(d, cache, lens, table, cu);
  if (st != GDN_OK) return st;
  if (!plan || plan->path < kKvPathF32 || plan->path > kKvPathMany || plan->n_seqs != d->n_seqs || plan->T != d->T || plan->h_q != d->h_q || plan->h_kv != cache->h_kv ||
      plan->dtype != d->dtype)
    return GDN_ERR_INVALID_ARG;
  if (d->causal != 0 && d->causal != 1) return GDN_ERR_UNSUPPORTED;
  if (d->window < 0 || d->max_pages > kKvMostPages || !std::isfinite(d->scale)) return GDN_ERR_INVALID_ARG;
  KvAttnArgs a;
  if ((st = kv_stride(d->q_stride, d->h_q, d->dtype, &a.q_stride)) != GDN_OK) return st;
  if ((st = kv_stride(d->out_stride, d->h_q, d->dtype, &a.out_stride)) != GDN_OK) return st;
  if (d->T == 0) return GDN_OK;
  if (!q || !out) return GDN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out) || (reinterpret_cast<uintptr_t>(lse) & 3u)) return GDN_ERR_MISALIGNED;
  if (!cu && d->T / d->n_seqs > plan->max_q_len) return GDN_ERR_INVALID_ARG;
  const int group = (d->h_q + cache->h_kv - 1) / cache->h_kv;
  const int64_t most = kv_most_row_tiles(d->n_seqs, d->T, group, plan->rows, plan->max_row_tiles);
  const int64_t counted = kv_row_tiles_counted(d, cache->h_kv, *plan);  // the page table may be wider than the one planned for
  if (most > counted) return GDN_ERR_INVALID_ARG;
  if (plan->n_ctas > 0) {
    if (!workspace || workspace_bytes < plan->workspace_bytes) return GDN_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return GDN_ERR_MISALIGNED;
  }
  int dev = 0;
  if ((st = device_setup(&dev)) != GDN_OK) return st;
  a.c = kv_args(d, cache, lens, table, cu);
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.causal = d->causal;
  a.window = d->window;
  a.scale_log2 = (d->scale != 0.f ? d->scale : 1.0f / std::sqrt((float)kHeadDim)) * 1.44269504088896341f;
  a.group = group;
  a.rows = plan->rows;
  a.max_rows = plan->max_q_len * a.group;
  a.max_row_tiles = plan->max_row_tiles;
  a.slots = 0;
  int64_t entries = (int64_t)d->n_seqs * a.max_row_tiles;
  if (!cu) {  // equally many tokens each, however many the plan allows
    a.max_row_tiles = std::max(1, std::min(a.max_row_tiles, (int)(((int64_t)a.c.n_each * a.group + a.rows - 1) / a.rows)));
    entries = (int64_t)d->n_seqs * a.max_row_tiles;
  } else {
    // The search costs a few loads in turn: worth it from half as many entries,
    // when these are more than the threads of a block take at once.  Offsets that
    // go back may give every entry a row tile, which then have to be countable.
    if ((entries > 256 && 2 * most <= entries) || entries > counted)
      entries = a.slots = (int)((int64_t)d->T * group / a.rows + d->n_seqs);
  }
  a.n_ctas = plan->n_ctas;
  a.item_cost = plan->item_cost;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.desc = reinterpret_cast<int4*>(ws + plan->off_desc);
  a.ml = reinterpret_cast<float2*>(ws + plan->off_ml);
  a.o = reinterpret_cast<float*>(ws + plan->off_o);
  const unsigned grid = a.n_ctas ? (unsigned)a.n_ctas : (unsigned)(entries * cache->h_kv);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const bool f32 = d->dtype == GDN_F32;
  LaunchLog log;
  cudaError_t e = log.before(cs);
  if (e == cudaSuccess) {
    if (plan->path != kKvPathF32) {
      CUtensorMap km, vm;
      if ((st = encode_kv_map(&km, cache->k, cache)) != GDN_OK) return st;
      if ((st = encode_kv_map(&vm, cache->v, cache)) != GDN_OK) return st;
      e = plan->path == kKvPathFew ? launch_kv_attn_few(a, km, vm, grid, cs) : launch_kv_attn_many(a, km, vm, grid, cs);
    } else {
      e = launch_kv_attn_f32(a, grid, cs);
    }
  }
  if (e == cudaSuccess) e = log.after("kv_attn", cs);
  if (a.n_ctas) {
    if (e == cudaSuccess) e = log.before(cs);
    if (e == cudaSuccess) e = launch_kv_combine(a, f32, cs);
    if (e == cudaSuccess) e = log.after("kv_combine", cs);
  }
  return e == cudaSuccess ? GDN_OK : cuda_fail(e);
}

gdn_status gdn_rope_table(const gdn_rope_opts* o, uint64_t* turns) {
  if (!o || !turns) return GDN_ERR_INVALID_ARG;
  if (o->rot < 8 || o->rot > kRopeD || o->rot % 8 || o->scaling < GDN_ROPE_PLAIN || o->scaling > GDN_ROPE_PARTS)
    return GDN_ERR_UNSUPPORTED;
  const double factor = o->scaling == GDN_ROPE_PLAIN ? 1.0 : o->factor;
  if (!std::isfinite(o->base) || !(o->base > 1.0) || !std::isfinite(factor) || !(factor >= 1.0)) return GDN_ERR_INVALID_ARG;
  if (o->scaling == GDN_ROPE_PARTS &&
      (!std::isfinite(o->original_len) || !(o->original_len > 0.0) || !std::isfinite(o->low) || !std::isfinite(o->high) ||
       !(o->low < o->high)))
    return GDN_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925286766559;
  double base = o->base;
  if (o->scaling == GDN_ROPE_NTK) base *= std::pow(factor, (double)o->rot / (o->rot - 2));
  for (int i = 0; i < o->rot / 2; ++i) {
    double f = std::pow(base, -2.0 * i / o->rot);
    if (o->scaling == GDN_ROPE_LINEAR) f /= factor;
    if (o->scaling == GDN_ROPE_PARTS) {
      const double r = o->original_len * f / two_pi;
      const double keep = std::min(1.0, std::max(0.0, (r - o->low) / (o->high - o->low)));
      f = f * keep + f / factor * (1.0 - keep);
    }
    turns[i] = (uint64_t)std::nearbyint(std::ldexp(f / two_pi, 64));  // f <= 1: below 2^62
  }
  return GDN_OK;
}

gdn_status gdn_qk_rope(const void* q, const void* k, const float* q_weight, const float* k_weight,
                       const int32_t* positions, const int32_t* cu, const gdn_rope* rope, void* q_out, void* k_out,
                       const gdn_rope_dims* d, void* stream) {
  QkRopeArgs a;
  gdn_status st = qk_rope_args(d, rope, q_weight, k_weight, positions, cu, &a);
  if (st != GDN_OK) return st;
  if (d->T == 0) return GDN_OK;
  if ((d->h_q && (!q || !q_out)) || (d->h_k && (!k || !k_out))) return GDN_ERR_INVALID_ARG;
  if (misaligned16({q, k, q_out, k_out})) return GDN_ERR_MISALIGNED;
  if (other_rows(q, a.side[0].in_stride, q_out, a.side[0].out_stride, d->T) ||
      other_rows(k, a.side[1].in_stride, k_out, a.side[1].out_stride, d->T))
    return GDN_ERR_INVALID_ARG;
  a.side[0].in = q;
  a.side[1].in = k;
  a.side[0].out = q_out;
  a.side[1].out = k_out;
  if ((st = rope_ctas(kRopeCtas, &a)) != GDN_OK) return st;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  LaunchLog log;
  cudaError_t e = log.before(cs);
  if (e == cudaSuccess) e = launch_qk_rope(a, d->dtype == GDN_F32, cs);
  if (e == cudaSuccess) e = log.after("qk_rope", cs);
  return e == cudaSuccess ? GDN_OK : cuda_fail(e);
}

gdn_status gdn_qk_rope_bwd_workspace_bytes(size_t* bytes) {
  if (!bytes) return GDN_ERR_INVALID_ARG;
  *bytes = (size_t)kRopeBwdCtas * 2 * kRopeD * sizeof(float);
  return GDN_OK;
}

gdn_status gdn_qk_rope_bwd(const void* q, const void* k, const float* q_weight, const float* k_weight,
                           const int32_t* positions, const int32_t* cu, const gdn_rope* rope, const void* d_q_out,
                           const void* d_k_out, void* dq, void* dk, float* dq_weight, float* dk_weight,
                           const gdn_rope_dims* d, void* workspace, size_t workspace_bytes, void* stream) {
  QkRopeArgs a;
  gdn_status st = qk_rope_args(d, rope, q_weight, k_weight, positions, cu, &a);
  if (st != GDN_OK) return st;
  if ((dq_weight && !q_weight) || (dk_weight && !k_weight)) return GDN_ERR_INVALID_ARG;
  if (misaligned16({dq_weight, dk_weight, workspace})) return GDN_ERR_MISALIGNED;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  const bool sums = dq_weight || dk_weight;
  if (d->T == 0) {
    if (dq_weight) e = cudaMemsetAsync(dq_weight, 0, kRopeD * sizeof(float), cs);
    if (e == cudaSuccess && dk_weight) e = cudaMemsetAsync(dk_weight, 0, kRopeD * sizeof(float), cs);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e);
  }
  const bool read = d->norm != GDN_NORM_NONE;
  if ((d->h_q && ((read && !q) || !d_q_out || !dq)) || (d->h_k && ((read && !k) || !d_k_out || !dk))) return GDN_ERR_INVALID_ARG;
  if (misaligned16({q, k, d_q_out, d_k_out, dq, dk})) return GDN_ERR_MISALIGNED;
  if (other_rows(d_q_out, a.side[0].out_stride, dq, a.side[0].dx_stride, d->T) ||
      other_rows(d_k_out, a.side[1].out_stride, dk, a.side[1].dx_stride, d->T))
    return GDN_ERR_INVALID_ARG;
  size_t need = 0;
  gdn_qk_rope_bwd_workspace_bytes(&need);
  if (sums && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
  a.side[0].in = q;
  a.side[1].in = k;
  a.side[0].out = const_cast<void*>(d_q_out);
  a.side[1].out = const_cast<void*>(d_k_out);
  a.side[0].dx = dq;
  a.side[1].dx = dk;
  a.side[0].d_weight = dq_weight;
  a.side[1].d_weight = dk_weight;
  a.part = sums ? static_cast<float*>(workspace) : nullptr;
  if ((st = rope_ctas(kRopeBwdCtas, &a)) != GDN_OK) return st;
  const int64_t units = ((int64_t)d->T + 1) / 2 * (d->h_q + d->h_k);
  a.fold = sums && units > (int64_t)kRopeFold * a.ctas * kRopeWarps;
  int dev = 0;
  if (a.fold && (st = device_setup(&dev)) != GDN_OK) return st;
  LaunchLog log;
  e = log.before(cs);
  if (e == cudaSuccess) e = launch_qk_rope_bwd(a, d->dtype == GDN_F32, cs);
  if (e == cudaSuccess) e = log.after("qk_rope_bwd", cs);
  if (sums) {
    if (e == cudaSuccess) e = log.before(cs);
    if (e == cudaSuccess) e = launch_qk_rope_weights(a, cs);
    if (e == cudaSuccess) e = log.after("qk_rope_weights", cs);
  }
  return e == cudaSuccess ? GDN_OK : cuda_fail(e);
}

gdn_status gdn_kv_append_rope(const void* k, const void* v, const float* k_weight, const void* q,
                              const float* q_weight, void* q_out, const int32_t* lens, const int32_t* table,
                              const int32_t* cu, const gdn_kv_cache* cache, const gdn_kv_dims* d, const gdn_rope* rope,
                              int norm, float eps, void* stream) {
  gdn_status st = check_kv(d, cache, lens, table, cu);
  if (st != GDN_OK) return st;
  KvRopeArgs a;
  std::memset(&a, 0, sizeof(a));
  if ((st = rope_args(rope, norm, eps, &a.q.r)) != GDN_OK) return st;
  if (norm == GDN_NORM_NONE && (q_weight || k_weight)) return GDN_ERR_INVALID_ARG;
  if ((q == nullptr) != (q_out == nullptr) || (!q && q_weight)) return GDN_ERR_INVALID_ARG;
  if (q && (d->h_q < 1 || d->h_q > 65535)) return GDN_ERR_INVALID_ARG;
  if (misaligned16({q_weight, k_weight, q, q_out})) return GDN_ERR_MISALIGNED;
  if ((st = kv_moves(d, cache, lens, table, cu, &a.p, &a.entries)) != GDN_OK) return st;
  if (q) {
    RopeSide& s = a.q.side[0];
    if ((st = kv_stride(d->q_stride, d->h_q, d->dtype, &s.in_stride)) != GDN_OK) return st;
    if ((st = kv_stride(d->out_stride, d->h_q, d->dtype, &s.out_stride)) != GDN_OK) return st;
    if (other_rows(q, s.in_stride, q_out, s.out_stride, d->T)) return GDN_ERR_INVALID_ARG;
    a.q.pos = {nullptr, cu, lens, d->n_seqs, d->T, a.p.c.n_each};
    s.in = q;
    s.out = q_out;
    s.weight = q_weight;
    s.heads = d->h_q;
    // of the resident CTAs as many as their share of the bytes, read and written
    const bool f32 = d->dtype == GDN_F32;
    const int64_t es = f32 ? 4 : 2, bytes_q = 2 * es * d->h_q, bytes_kv = 2 * (es + 1) * cache->h_kv;
    const int64_t ctas = 152 * (f32 ? kAppendRopeCtas<float> : kAppendRopeCtas<__nv_bfloat16>);
    if ((st = rope_ctas(ctas * bytes_q / (bytes_q + bytes_kv), &a.q)) != GDN_OK) return st;
  }
  if (d->T == 0) return GDN_OK;
  if (!k || !v) return GDN_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v)) return GDN_ERR_MISALIGNED;
  a.p.k = const_cast<void*>(k);
  a.p.v = const_cast<void*>(v);
  a.k_weight = k_weight;
  if (append_tasks(a) + a.q.ctas > 0x7fffffff) return GDN_ERR_INVALID_ARG;  // blocks, or warps of them
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  LaunchLog log;
  cudaError_t e = log.before(cs);
  if (e == cudaSuccess) e = launch_kv_append_rope(a, d->dtype == GDN_F32, cs);
  if (e == cudaSuccess) e = log.after("kv_append_rope", cs);
  return e == cudaSuccess ? GDN_OK : cuda_fail(e);
}

gdn_status gdn_conv_fwd(const void* x, const float* weight, const float* bias, const void* initial_state,
                        const int32_t* cu, void* q, void* k, void* v, void* final_state, const gdn_conv_dims* d,
                        void* stream) {
  ConvArgs a;
  gdn_status st = conv_args(d, weight, bias, cu, &a);
  if (st != GDN_OK) return st;
  if (!weight || (d->T && (!x || !q || !k || !v))) return GDN_ERR_INVALID_ARG;
  if (misaligned16({x, initial_state, q, k, v, final_state})) return GDN_ERR_MISALIGNED;
  if (overlap(initial_state, final_state, conv_state_bytes(d))) return GDN_ERR_INVALID_ARG;
  a.x = x;
  a.state = initial_state;
  a.q = q;
  a.k = k;
  a.v = v;
  a.final_state = final_state;
  conv_runs(d->T, 2 * d->h_qk + d->h_v - a.n_unit, kConvFill, kConvUnitCost, 4, 1, &a);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  LaunchLog log;
  if (d->T == 0 && !final_state) return GDN_OK;
  cudaError_t e = log.before(cs);
  if (e == cudaSuccess) e = launch_conv(a, d->dtype == GDN_F32, cs);
  if (e == cudaSuccess) e = log.after("conv", cs);
  return e == cudaSuccess ? GDN_OK : cuda_fail(e);
}

gdn_status gdn_conv_bwd_workspace_bytes(const gdn_conv_dims* d, size_t* bytes) {
  if (!d || !bytes) return GDN_ERR_INVALID_ARG;
  static const int32_t offsets[1] = {0};  // not read: lengths do not matter here
  ConvArgs a;
  gdn_status st = conv_args(d, nullptr, nullptr, offsets, &a);
  if (st != GDN_OK) return st;
  *bytes = conv_bwd_plan(d, &a);
  return GDN_OK;
}

gdn_status gdn_conv_bwd(const void* x, const float* weight, const float* bias, const void* initial_state,
                        const int32_t* cu, const void* d_q, const void* d_k, const void* d_v, const void* d_final_state,
                        void* dx, float* d_weight, float* d_bias, void* d_initial_state, const gdn_conv_dims* d,
                        void* workspace, size_t workspace_bytes, void* stream) {
  ConvArgs a;
  gdn_status st = conv_args(d, weight, bias, cu, &a);
  if (st != GDN_OK) return st;
  if (!weight || (d->T && (!x || !d_q || !d_k || !d_v || !dx))) return GDN_ERR_INVALID_ARG;
  if (misaligned16({x, initial_state, d_q, d_k, d_v, d_final_state, dx, d_weight, d_bias, d_initial_state, workspace}))
    return GDN_ERR_MISALIGNED;
  if (dx && dx == x) return GDN_ERR_INVALID_ARG;  // the inputs of a run are read by the one after it
  if (overlap(initial_state, d_initial_state, conv_state_bytes(d)) || overlap(d_final_state, d_initial_state, conv_state_bytes(d)))
    return GDN_ERR_INVALID_ARG;
  const size_t need = conv_bwd_plan(d, &a);
  a.sums = d_weight || d_bias;
  if (a.sums && need && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
  a.x = x;
  a.state = initial_state;
  a.q = const_cast<void*>(d_q);
  a.k = const_cast<void*>(d_k);
  a.v = const_cast<void*>(d_v);
  a.d_final = d_final_state;
  a.dx = dx;
  a.d_weight = d_weight;
  a.d_bias = d_bias;
  a.d_state = d_initial_state;
  a.part = static_cast<float*>(workspace);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  LaunchLog log;
  cudaError_t e = cudaSuccess;
  if (d->T) {
    e = log.before(cs);
    if (e == cudaSuccess) e = launch_conv_bwd(a, d->dtype == GDN_F32, cs);
    if (e == cudaSuccess) e = log.after("conv_bwd", cs);
  }
  if (a.sums || d_initial_state) {
    if (e == cudaSuccess) e = log.before(cs);
    if (e == cudaSuccess) e = launch_conv_bwd_sums(a, d->dtype == GDN_F32, cs);
    if (e == cudaSuccess) e = log.after("conv_bwd_sums", cs);
  }
  return e == cudaSuccess ? GDN_OK : cuda_fail(e);
}

gdn_status gdn_conv_step(const void* x, const float* weight, const float* bias, void* state, void* q, void* k,
                         void* v, const gdn_conv_dims* d, void* stream) {
  ConvArgs a;
  gdn_status st = conv_args(d, weight, bias, nullptr, &a);
  if (st != GDN_OK) return st;
  if (d->T != d->n_seqs || !x || !weight || !state || !q || !k || !v) return GDN_ERR_INVALID_ARG;
  if (misaligned16({x, state, q, k, v})) return GDN_ERR_MISALIGNED;
  a.x = x;
  a.q = q;
  a.k = k;
  a.v = v;
  a.final_state = state;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  LaunchLog log;
  cudaError_t e = log.before(cs);
  if (e == cudaSuccess) e = launch_conv_step(a, d->dtype == GDN_F32, cs);
  if (e == cudaSuccess) e = log.after("conv_step", cs);
  return e == cudaSuccess ? GDN_OK : cuda_fail(e);
}

gdn_status gdn_debug_stall_ns(uint32_t ns) {
  g_debug_stall_ns.store(ns, std::memory_order_relaxed);
  return GDN_OK;
}

gdn_status gdn_set_trace_events(void* const* events, int n_events) {
  if (n_events < 0 || n_events > kMaxTrace) return GDN_ERR_INVALID_ARG;
  if (!events) n_events = 0;
  for (int i = 0; i < n_events; ++i) {
    if (!events[i]) return GDN_ERR_INVALID_ARG;
    g_trace_ev[i] = reinterpret_cast<cudaEvent_t>(events[i]);
  }
  g_trace_n = n_events;
  return GDN_OK;
}

int gdn_trace_last(const char** names, int max_names) {
  if (names)
    for (int i = 0; i < g_last_count && i < max_names; ++i) names[i] = g_last_names[i];
  return g_last_count;
}

gdn_status gdn_get_device_status(const void* workspace, void* stream, int* code, int* detail) {
  if (!workspace || !code) return GDN_ERR_INVALID_ARG;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  int h[2] = {0, 0};
  cudaError_t e = cudaMemcpyAsync(h, workspace, sizeof(h), cudaMemcpyDeviceToHost, cs);
  if (e == cudaSuccess) e = cudaStreamSynchronize(cs);
  if (e != cudaSuccess) return cuda_fail(e);
  *code = h[0];
  if (detail) *detail = h[1];
  return GDN_OK;
}

gdn_status gdn_cp_head_modes(const void* workspace, const gdn_cp_plan_t* plan, int32_t* modes, float* bounds,
                             void* stream) {
  if (!workspace || !plan) return GDN_ERR_INVALID_ARG;
  const size_t heads = (size_t)plan->n_seqs * plan->h_v;
  if (plan->mode == GDN_CP_OFF || plan->dtype == GDN_F32 || plan->n_seg_total <= plan->n_seqs) {
    // no warmup decision taken: no context parallelism, the fp32 path (always
    // exact), or one segment per sequence (nothing to combine or restart)
    for (size_t i = 0; i < heads; ++i) {
      if (modes) modes[i] = plan->mode == GDN_CP_OFF ? GDN_CP_OFF : plan->dtype == GDN_F32 ? GDN_CP_EXACT : plan->mode;
      if (bounds) bounds[i] = -INFINITY;
    }
    return GDN_OK;
  }
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const uint8_t* ws = reinterpret_cast<const uint8_t*>(workspace);
  cudaError_t e = cudaSuccess;
  if (modes) e = cudaMemcpyAsync(modes, ws + plan->off_head, heads * 4, cudaMemcpyDeviceToHost, cs);
  if (e == cudaSuccess && bounds)
    e = cudaMemcpyAsync(bounds, ws + plan->off_head + heads * 4, heads * 4, cudaMemcpyDeviceToHost, cs);
  if (e == cudaSuccess) e = cudaStreamSynchronize(cs);
  if (e != cudaSuccess) return cuda_fail(e);
  return GDN_OK;
}

}  // extern "C"

extern "C" gdn_status gdn_chunk_fwd_static(const void* q, const void* k, const void* v, const float* g,
                                          const float* beta, const float* initial_state,
                                          const int32_t* cu_seqlens_dev, void* out, float* final_state,
                                          const gdn_dims* dims, const gdn_cp_plan_t* plan, void* stream) {
  if (!plan) return GDN_ERR_INVALID_ARG;
  if (plan->workspace_bytes > kStaticWorkspaceBytes) return GDN_ERR_WORKSPACE;
  void* ws = nullptr;
  gdn_status st = static_workspace(&ws);
  if (st != GDN_OK) return st;
  return gdn_chunk_fwd(q, k, v, g, beta, initial_state, cu_seqlens_dev, out, final_state, dims, plan, ws,
                       kStaticWorkspaceBytes, stream);
}

extern "C" gdn_status gdn_get_static_device_status(void* stream, int* code, int* detail) {
  if (!code) return GDN_ERR_INVALID_ARG;
  void* ws = nullptr;
  gdn_status st = static_workspace(&ws);
  if (st != GDN_OK) return st;
  return gdn_get_device_status(ws, stream, code, detail);
}
