/*
 * gdn.h -- C ABI of the GB300 (sm_103a) Gated Delta Network chunked-prefill
 * forward.
 *
 * Sources cited below:
 *   [FlashQLA] the FlashQLA blog pages, "FlashQLA: fused linear-attention
 *     kernels for CP/backward (GDN)" (Traditional Chinese and Korean
 *     editions), sections "Optimising GDN chunked prefill", "AutoCP",
 *     "TileLang warp-specialised kernels", "Benchmarks", "Implementation and
 *     requirements"; and the Telegram post on FlashQLA (Russian) on the
 *     fast-decaying heads and the 6-8 chunk warmup.
 *   [GDN] Yang, Kautz, Hatamizadeh, "Gated Delta Networks: Improving Mamba2
 *     with Delta Rule", ICLR 2025, section "Gated delta rule" (the recurrence).
 *
 * The layer (per sequence, per value head j, tokens t in order):
 *   S_t = exp(g_t) * S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T
 *   o_t = scale * S_t q_t
 * with S_t a d_v x d_k fp32 matrix, q/k taken from query/key head
 * floor(j * h_qk / h_v) (grouped heads) [GDN; FlashQLA, "Benchmarks" table
 * columns h_qk, h_v].  It is evaluated over 64-token chunks, aligned to each
 * sequence's own start, through the chunk-local WY form [FlashQLA,
 * "Optimising GDN chunked prefill"], optionally split into context-parallel
 * segments on one GPU [FlashQLA, "AutoCP"].
 *
 * Conventions for every entry point:
 *   - Device pointers are CUDA device addresses on the current device; host
 *     pointers are ordinary host memory.  The caller owns all memory,
 *     including the workspace; the library allocates nothing and keeps no
 *     per-call state.  The only global state is a per-device cache of the
 *     SM count and of the kernel attribute set-up.
 *   - `stream` is a cudaStream_t (NULL = legacy default stream).  Device
 *     work is enqueued asynchronously; nothing synchronises except
 *     gdn_get_device_status.
 *   - Every entry point returns a gdn_status.  No exception crosses the ABI.
 *     Kernels never trap: a kernel that fails its own bounds/consistency
 *     check, or whose bounded wait runs out, records a code in the
 *     workspace's status word (read it with gdn_get_device_status) and
 *     returns.
 */
#ifndef GDN_H_
#define GDN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum gdn_status {
  GDN_OK = 0,
  GDN_ERR_INVALID_ARG = 1,    /* null pointer, bad size, inconsistent dims/plan */
  GDN_ERR_UNSUPPORTED = 2,    /* d_k or d_v != 128, unknown dtype or mode */
  GDN_ERR_MISALIGNED = 3,     /* a device pointer not 16-byte (workspace: 256-byte) aligned */
  GDN_ERR_CUDA = 4,           /* a CUDA runtime/driver call failed; see gdn_last_cuda_error() */
  GDN_ERR_DEVICE_TIMEOUT = 5, /* (from gdn_get_device_status) a bounded on-device wait ran out */
  GDN_ERR_WORKSPACE = 6,      /* workspace missing or smaller than plan->workspace_bytes */
  GDN_ERR_DEVICE_CHECK = 7    /* (from gdn_get_device_status) a kernel's own check failed */
} gdn_status;

/* Element types of q, k, v and out.  g, beta, states are always fp32.
 *   GDN_BF16: the chunked tcgen05 path (fp16 MMA operands, fp32 accumulation),
 *             with the plan's context parallelism.
 *   GDN_F32:  fp32 throughout, on the CUDA cores: the recurrence itself,
 *             one state row per thread pair, with the plan's segments always
 *             combined exactly (a WARMUP plan runs as EXACT).  For results
 *             within 1e-4 of exact. */
enum { GDN_BF16 = 0, GDN_F32 = 1 };

/* Intra-card context parallelism [FlashQLA, "AutoCP"]. */
enum {
  GDN_CP_OFF = 0,    /* one CTA-level scan per (sequence, value head) */
  GDN_CP_EXACT = 1,  /* segments; start states combined exactly through M */
  GDN_CP_WARMUP = 2, /* segments; a (sequence, head) whose gate bound is under
                        its tolerance (see tol_rule) restarts each segment
                        from zero up to warmup_chunks chunks early and skips
                        M; the others run exactly */
  GDN_CP_AUTO = 3    /* WARMUP when n_seqs * h_v < sm_count, else OFF */
};

/* How a warmup restart's tolerance is set [FlashQLA, "AutoCP": a restart is
 * good once the state error it leaves is under the noise floor].
 *   GDN_TOL_FIXED: warmup_tol, the same for every head and segment.
 *   GDN_TOL_NOISE: per (sequence, value head) and segment, the larger of
 *     warmup_tol and the noise floor of the exact bf16 path at the segment
 *     start: the fp16 rounding of the state operand in every chunk (relative
 *     2^-11) carried to the start, 2^-11 * (1 + sum over m = 1..w of
 *     min(1, the bound of the last m chunks before the start)), w =
 *     min(warmup_chunks, 8, chunks before the start); so at most 9 * 2^-11.  A head whose gates decay slowly carries more
 *     of that rounding, so its floor, and the depth error it tolerates, is
 *     higher; the warmup error stays below the error the exact path makes
 *     anyway.  The fp32 path always combines exactly. */
enum { GDN_TOL_FIXED = 0, GDN_TOL_NOISE = 1 };

typedef struct gdn_dims {
  int B;      /* batch; must be 1 when cu_seqlens is used */
  int T;      /* tokens per batch row (varlen: total packed tokens) */
  int h_qk;   /* query/key heads */
  int h_v;    /* value heads (one recurrent state each) */
  int d_k;    /* key dim; must be 128 */
  int d_v;    /* value dim; must be 128 */
  int n_seqs; /* varlen: number of sequences (len(cu_seqlens) - 1); fixed length: B */
  float scale; /* output scale; 0 selects 1/sqrt(d_k) */
  int dtype;   /* GDN_BF16 or GDN_F32 */
} gdn_dims;

typedef struct gdn_cp_opts {
  int mode;          /* GDN_CP_* */
  float lambda;      /* segment length L = round(lambda * sqrt(N)) chunks, lambda used in
                        steps of 1/256; <= 0 lets the planner choose it: the lambda (a
                        multiple of 1/8) minimising 2 x (finish of the list schedule of
                        the scan's CTAs in launch order on sm_count SMs, each taking its
                        segment's chunks + 3) + 2 x (most segments of one sequence: a
                        combine step costs about a chunk-time); ties go
                        to fewer segments.  For GDN_F32, whose chains run two CTAs per
                        SM and whose chunks dwarf a combine step, the schedule has 2 x
                        sm_count slots, a CTA takes its chunks alone, and the score is
                        2 x the finish */
  int warmup_chunks; /* warmup restart depth w in chunks; <= 0 selects 8 */
  float warmup_tol;  /* accept warmup for a (sequence, head) when, for every segment,
                        some depth w <= warmup_chunks has its bound exp(sum over the w
                        chunks before the segment of g + log max(1, |1 - beta ||k||^2|))
                        <= the segment's tolerance (see tol_rule); <= 0 selects 1e-4 */
  int sm_count;      /* SMs to plan for; <= 0 queries the current device */
  int tol_rule;      /* GDN_TOL_FIXED or GDN_TOL_NOISE (NULL opts: GDN_TOL_NOISE) */
} gdn_cp_opts;

/* Plain-data plan; fill with gdn_cp_plan, do not edit. */
typedef struct gdn_cp_plan_t {
  int mode;             /* resolved mode: GDN_CP_OFF, GDN_CP_EXACT or GDN_CP_WARMUP */
  int n_seqs;           /* sequences the plan was made for */
  int T_total;          /* B * T */
  int h_v, h_qk, dtype; /* copied from dims, checked by gdn_chunk_fwd */
  int lambda_q8;        /* lambda * 256, rounded */
  int warmup_chunks;
  float warmup_tol;
  int sm_count;
  int tol_rule;         /* GDN_TOL_FIXED or GDN_TOL_NOISE */
  int n_seg_total;      /* segments summed over sequences */
  int max_seg_chunks;   /* longest segment, in chunks */
  int max_chunks;       /* longest sequence, in chunks */
  size_t workspace_bytes;
  size_t off_head;      /* byte offsets of the workspace sections */
  size_t off_seg_bound;
  size_t off_R, off_Sloc, off_Sstart;
  int n_chunks_total;   /* 64-token chunks summed over sequences */
  size_t off_chunk_map; /* chunk index: first chunk of each sequence, sequence of each chunk */
  size_t off_wy;        /* chunk-local records (-W, U, P, gates), 41472 bytes per (chunk, value head) */
} gdn_cp_plan_t;

/*
 * gdn_cp_plan -- host-only planning [FlashQLA, "AutoCP": L = lambda * sqrt(N),
 * N = chunks, L = chunks per segment].  No device work.
 *   dims              : problem sizes (see gdn_dims).
 *   cu_seqlens_host   : n_seqs+1 non-decreasing token offsets starting at 0
 *                       and ending at T, or NULL for B fixed-length rows of T.
 *   opts              : may be NULL (all defaults: mode AUTO, lambda chosen by
 *                       the planner, warmup up to 8 chunks at 1e-4 or the noise
 *                       floor (GDN_TOL_NOISE), SMs of the device).  A tol_rule
 *                       other than GDN_TOL_FIXED or GDN_TOL_NOISE is refused
 *                       with GDN_ERR_UNSUPPORTED.
 *   out_plan          : written on success.
 * Segmentation of a sequence with N = ceil(len/64) chunks: L = max(1,
 * floor((isqrt(lambda_q8^2 * N) + 128) / 256)), n_seg = max(1, ceil(N / L)),
 * segment s = chunks [floor(s N / n_seg), floor((s+1) N / n_seg)).  Mode OFF
 * uses one segment per sequence.  An empty sequence has one empty segment.
 * Errors: INVALID_ARG, UNSUPPORTED, CUDA (only when opts->sm_count <= 0 and
 * the device query fails).
 */
gdn_status gdn_cp_plan(const gdn_dims* dims, const int32_t* cu_seqlens_host,
                       const gdn_cp_opts* opts, gdn_cp_plan_t* out_plan);

/*
 * gdn_chunk_fwd -- the chunked-prefill forward [FlashQLA, "Optimising GDN
 * chunked prefill", "AutoCP", "TileLang warp-specialised kernels" (forward
 * pass: V', S and O)].  Asynchronous on `stream`.
 *   q, k          : device, [B*T, h_qk, d_k] (token-major, heads interleaved), dims->dtype.
 *   v             : device, [B*T, h_v, d_v], dims->dtype.
 *   g             : device, [B*T, h_v] fp32, log of the decay gate (alpha = exp(g)).
 *   beta          : device, [B*T, h_v] fp32, write strength.
 *   initial_state : device, [n_seqs, h_v, d_k, d_v] fp32 (H = S^T), or NULL for zeros.
 *   cu_seqlens_dev: device int32 [n_seqs+1], the same offsets given to gdn_cp_plan,
 *                   or NULL for fixed-length rows.  The kernels check them before
 *                   following them: offsets outside [0, T], going back, not ending
 *                   at T, or giving other chunk or segment counts than the plan's
 *                   are reported as GDN_ERR_DEVICE_CHECK with detail 3 in the status
 *                   word, and no access follows them outside the buffers (o and
 *                   final_state are then incomplete).  Other boundaries with the
 *                   same counts go undetected.
 *   out           : device, [B*T, h_v, d_v], dims->dtype (bf16 rounded to nearest even).
 *   final_state   : device, [n_seqs, h_v, d_k, d_v] fp32, or NULL (not written).
 *   dims, plan    : host; plan must come from gdn_cp_plan with these dims.
 *   workspace     : device, 256-byte aligned; its contents on entry do not
 *                   matter.  Must not be shared by calls that may run
 *                   concurrently.
 *   workspace_bytes: size of `workspace`; must be >= plan->workspace_bytes.
 * All device pointers must be 16-byte aligned.  q/k/v/out may not overlap.
 * Errors: INVALID_ARG, UNSUPPORTED, MISALIGNED, WORKSPACE, CUDA (launch failure).
 */
gdn_status gdn_chunk_fwd(const void* q, const void* k, const void* v, const float* g,
                         const float* beta, const float* initial_state,
                         const int32_t* cu_seqlens_dev, void* out, float* final_state,
                         const gdn_dims* dims, const gdn_cp_plan_t* plan, void* workspace,
                         size_t workspace_bytes, void* stream);

/* Human-readable name of a status code (static storage). */
const char* gdn_status_string(gdn_status status);

/* The cudaError_t of the most recent GDN_ERR_CUDA on this thread (0 if none). */
int gdn_last_cuda_error(void);

/*
 * gdn_get_device_status -- synchronises `stream`, then reads the status word
 * the kernels of the last gdn_chunk_fwd on this workspace wrote.
 *   workspace : device workspace passed to gdn_chunk_fwd.
 *   code      : host; receives GDN_OK, GDN_ERR_DEVICE_TIMEOUT or GDN_ERR_DEVICE_CHECK.
 *   detail    : host, may be NULL; receives a kernel-specific detail word.
 * Returns CUDA on a failed copy/sync, INVALID_ARG on null pointers.
 */
gdn_status gdn_get_device_status(const void* workspace, void* stream, int* code, int* detail);

/*
 * gdn_cp_head_modes -- diagnostics: synchronises `stream` and copies, per
 * (sequence, value head), the mode the last gdn_chunk_fwd on this workspace
 * took (GDN_CP_EXACT or GDN_CP_WARMUP; GDN_CP_OFF for plans without CP; always
 * GDN_CP_EXACT on the fp32 path with CP; the plan's mode when every sequence
 * is a single segment, where nothing is combined or restarted) and
 * the natural log of its warmup error bound (-inf when no segment needs one).
 *   modes_host    : host int32 [n_seqs * h_v], or NULL.
 *   log_bound_host: host fp32 [n_seqs * h_v], or NULL.
 */
gdn_status gdn_cp_head_modes(const void* workspace, const gdn_cp_plan_t* plan, int32_t* modes_host,
                             float* log_bound_host, void* stream);

/*
 * gdn_chunk_fwd_static -- gdn_chunk_fwd for callers that cannot allocate
 * device memory.  The FlashQLA pages have no counterpart: this is a library
 * convenience.  Some callers can't call cudaMalloc or hand out scratch: code
 * running under a runtime that owns all device memory (an inference
 * server's arena, a plugin interface that passes only its inputs and
 * outputs), or code that must not allocate after start-up.  This entry point
 * takes the same arguments as gdn_chunk_fwd minus the workspace and uses a
 * fixed 8 MiB device array built into the library instead; every GPU that
 * loads the library holds that array until the process exits.
 *   - Fits plans whose plan->workspace_bytes is at most 8 MiB: the chunk
 *     records take 41472 bytes per (chunk, value head), so about 200
 *     chunk-heads (e.g. 1000 tokens with 12 value heads, context parallelism
 *     off; with it, each segment adds 192 KB per value head of segment
 *     states); larger plans are rejected with GDN_ERR_WORKSPACE before any
 *     device work.
 *   - Allocates nothing.  Its first call on a device looks up the array's
 *     device address (cudaGetSymbolAddress) with that device current; make
 *     that first call before any stream capture.
 *   - All calls share the one array and it keeps the last call's contents;
 *     every part the forward reads is written or cleared within the call.
 *     Calls that may overlap on the GPU (other streams, other host threads)
 *     race on the array: serialise them.
 *   - The device status word of these calls lives in the shared array;
 *     read it with gdn_get_static_device_status.
 * Errors: as gdn_chunk_fwd, plus WORKSPACE for plans above the limit.
 */
gdn_status gdn_chunk_fwd_static(const void* q, const void* k, const void* v, const float* g,
                                const float* beta, const float* initial_state,
                                const int32_t* cu_seqlens_dev, void* out, float* final_state,
                                const gdn_dims* dims, const gdn_cp_plan_t* plan, void* stream);

/*
 * gdn_get_static_device_status -- gdn_get_device_status for the calls of
 * gdn_chunk_fwd_static on the current device: synchronises `stream`, then
 * reads the status word the kernels of the last such call wrote into the
 * library's built-in array (no counterpart on the FlashQLA pages).  The
 * first use on a device looks up the array's address like
 * gdn_chunk_fwd_static does.
 *   code   : host; receives GDN_OK, GDN_ERR_DEVICE_TIMEOUT or GDN_ERR_DEVICE_CHECK.
 *   detail : host, may be NULL; receives the kernel-specific detail word.
 * Errors: INVALID_ARG (code NULL), CUDA (address lookup, copy or sync failed).
 */
gdn_status gdn_get_static_device_status(void* stream, int* code, int* detail);

/*
 * gdn_decode_step -- one new token for each of a batch of sequences: the
 * recurrence step itself [GDN, "Gated delta rule"], the generation-time
 * counterpart of gdn_chunk_fwd.  Per sequence n and value head j (q/k head
 * floor(j * h_qk / h_v)):
 *   S <- exp(g) S (I - beta k k^T) + beta v k^T,   o = scale * S q,
 * with the state stored as H = S^T like initial_state/final_state, so the
 * final_state of a prefill continues here directly.  fp32 arithmetic on the
 * CUDA cores; asynchronous on `stream`.
 *   q, k  : device, [B, h_qk, d_k], dims->dtype.
 *   v     : device, [B, h_v, d_v], dims->dtype.
 *   g, beta: device, [B, h_v] fp32.
 *   state : device, [B, h_v, d_k, d_v] fp32; read, then overwritten with the
 *           new state.
 *   out   : device, [B, h_v, d_v], dims->dtype (bf16 rounded to nearest even).
 *   dims  : B sequences, T must be 1, n_seqs must equal B; d_k = d_v = 128.
 * No workspace.  out may not overlap the inputs or the state.
 * Errors: INVALID_ARG (null pointer, T != 1, n_seqs != B), UNSUPPORTED,
 * MISALIGNED (16 bytes), CUDA (launch failure).
 */
gdn_status gdn_decode_step(const void* q, const void* k, const void* v, const float* g, const float* beta,
                           float* state, void* out, const gdn_dims* dims, void* stream);

/*
 * gdn_bwd_workspace_bytes -- device workspace gdn_chunk_bwd needs for `plan`:
 * the forward's plan->workspace_bytes, then, per (chunk, value head), 136 KB
 * (A^T, the chunk-start state and three 32 KB backward tiles), then a bf16
 * copy of o.  Host only.  Errors: INVALID_ARG (NULL), UNSUPPORTED (fp32 plan).
 */
gdn_status gdn_bwd_workspace_bytes(const gdn_cp_plan_t* plan, size_t* bytes);

/*
 * gdn_chunk_bwd -- gradients of the chunked-prefill forward [FlashQLA,
 * "TileLang warp-specialised kernels" (backward pass: the dv, state-gradient,
 * dq/dk/dw/dg and WY gradient steps); the pages give no formulas: these are
 * the exact gradients of gdn_chunk_fwd's function].  For the scalar
 *   sum(o * d_out) + sum(final_state * d_final_state),
 * writes its gradient with respect to q, k, v, g, beta and initial_state.
 * Asynchronous on `stream`.  The forward is recomputed inside the call unless
 * reuse_forward = 1, in which case `workspace` must hold the state a
 * gdn_chunk_fwd_train with the same inputs and plan left there.  The chunk
 * states the gradients use are the forward's in the plan's mode (with
 * GDN_CP_AUTO, a warmup restart where the forward's acceptance rule allows
 * one, so they agree with the exact states within its tolerance; GDN_CP_EXACT
 * gives the exact forward's gradients); the state gradient's own chain is
 * always combined exactly.  bf16 only.
 *   q, k, v, g, beta, initial_state, cu_seqlens_dev, dims, plan: as gdn_chunk_fwd.
 *   d_out         : device, [B*T, h_v, d_v] bf16.
 *   d_final_state : device, [n_seqs, h_v, d_k, d_v] fp32, or NULL (zero).
 *   dq, dk        : device, [B*T, h_qk, d_k] bf16 (summed over each q/k head's value heads).
 *   dv            : device, [B*T, h_v, d_v] bf16.
 *   dg, dbeta     : device, [B*T, h_v] fp32.
 *   d_initial_state: device, [n_seqs, h_v, d_k, d_v] fp32, or NULL (not written);
 *                   written also when initial_state is NULL (the gradient at zero).
 *   workspace     : device, 256-byte aligned, at least gdn_bwd_workspace_bytes(plan).
 * All device pointers 16-byte aligned; outputs may not overlap inputs.
 * Kernels report through the workspace status word like the forward's
 * (gdn_get_device_status), including GDN_ERR_DEVICE_CHECK when an fp16
 * operand of the backward left the fp16 range.
 * Errors: INVALID_ARG, UNSUPPORTED (fp32 dtype), MISALIGNED, WORKSPACE, CUDA.
 */
gdn_status gdn_chunk_bwd(const void* q, const void* k, const void* v, const float* g, const float* beta,
                         const float* initial_state, const int32_t* cu_seqlens_dev, const void* d_out,
                         const float* d_final_state, void* dq, void* dk, void* dv, float* dg, float* dbeta,
                         float* d_initial_state, const gdn_dims* dims, const gdn_cp_plan_t* plan,
                         void* workspace, size_t workspace_bytes, int reuse_forward, void* stream);

/*
 * gdn_chunk_fwd_train -- gdn_chunk_fwd that also keeps, in `workspace`, what
 * gdn_chunk_bwd needs (no counterpart on the FlashQLA pages: the training
 * pattern of forward then backward).  Same arguments and outputs as
 * gdn_chunk_fwd; the workspace must hold gdn_bwd_workspace_bytes(plan).  It
 * runs in the plan's mode like gdn_chunk_fwd (o and final_state are the same);
 * besides them the call writes A^T and every chunk's start state into the
 * workspace.  A later
 * gdn_chunk_bwd with the same inputs, plan and workspace and reuse_forward = 1
 * then skips its own recompute; nothing checks that the inputs are the same.
 * bf16 only.  Errors: as gdn_chunk_fwd, UNSUPPORTED for fp32.
 */
gdn_status gdn_chunk_fwd_train(const void* q, const void* k, const void* v, const float* g, const float* beta,
                               const float* initial_state, const int32_t* cu_seqlens_dev, void* out,
                               float* final_state, const gdn_dims* dims, const gdn_cp_plan_t* plan,
                               void* workspace, size_t workspace_bytes, void* stream);

/*
 * ---- 8-bit key/value cache and attention over it ----
 * What a model that mixes gated-delta-rule layers with softmax-attention
 * layers keeps for the latter while it generates (no counterpart on the
 * FlashQLA pages).
 *
 * The cache holds keys and values of d = 128 elements in pages of 64 tokens
 * (GDN_KV_PAGE), as e4m3 codes c with one fp32 scale s per (page, key/value
 * head) for the keys and one for the values: x = c s.  Scales are powers of
 * two from 2^-40 to 2^40, so c s is exact in bf16 and fp32, and a scale that
 * grows re-encodes earlier codes exactly unless they fall into e4m3's
 * subnormal range.
 *
 * A batch: sequence i brings n_i tokens, packed over the batch by
 * cu_seqlens_dev (int32 [n_seqs + 1]; NULL: T / n_seqs tokens each).  They
 * are the last n_i of its kv_lens_dev[i] tokens: packed token t of sequence i
 * has position p = kv_lens[i] - n_i + t.  Position p lives in row p % 64 of
 * pool page page_table_dev[i * max_pages + p / 64].  kv_lens[i] < n_i is
 * allowed (an idle slot of a captured decode batch has kv_lens[i] = 0):
 * tokens at p < 0 are not stored, read as zeros, and attend to nothing under
 * the causal mask.
 *
 * The lengths and the table are device data, so a captured call may be
 * replayed as the caller advances them between calls; they, and a call's
 * workspace, must not change while it runs.  The kernels check lengths and
 * table before following them: offsets that leave [0, T] or go back, a length
 * outside [0, 64 max_pages], or a page outside [0, n_pages) is recorded as
 * GDN_ERR_DEVICE_CHECK with detail 7 (offsets, length) or 8 (page) in
 * cache->status and no access follows it outside the buffers; the outputs of
 * that sequence (with such offsets, of any) are then undefined.  cache->status keeps the first failure
 * until the caller zeroes it; read it with gdn_get_device_status(cache->status, ...).
 */
#define GDN_KV_PAGE 64

typedef struct gdn_kv_cache {
  void* k;          /* device, [n_pages, h_kv, 64, 128] e4m3 codes */
  void* v;          /* device, the same */
  float* k_scale;   /* device, [n_pages, h_kv] */
  float* v_scale;   /* device, [n_pages, h_kv] */
  int32_t* status;  /* device, int32[2] {code, detail}; zeroed by the caller at the start */
  int n_pages;
  int h_kv;
  int d;            /* must be 128 */
} gdn_kv_cache;

typedef struct gdn_kv_dims {
  int n_seqs;
  int T;          /* tokens of the call, over all sequences */
  int h_q;        /* query heads; query head j reads key/value head floor(j h_kv / h_q) */
  int max_pages;  /* row length of page_table */
  int causal;     /* attention: 1: keys at positions <= p; 0: all kv_lens keys */
  int window;     /* attention: > 0: only keys at positions > p - window; 0: no bound */
  float scale;    /* attention: score scale; 0 selects 1/sqrt(128) */
  int dtype;      /* GDN_BF16 or GDN_F32: type of k, v, q and out */
  int64_t q_stride;   /* elements from one token to the next in q, k, v and out; 0: */
  int64_t k_stride;   /* heads * 128 (packed).  A multiple of 16 bytes and at least */
  int64_t v_stride;   /* heads * 128, so k and v may be parts of one fused projection. */
  int64_t out_stride;
} gdn_kv_dims;

/*
 * gdn_kv_append -- quantises n_i new tokens of each sequence into the cache.
 * Per (page, key/value head) that receives tokens, with r tokens of the
 * sequence already in the page (positions before the new ones), a the largest
 * finite |x| of the new ones, and s(a) the smallest power of two with
 * a / s <= 448, held within [2^-40, 2^40] (s(0) = 2^-40):
 *   s = s(a) if r = 0, else max(old scale, s(a));
 *   earlier codes c <- e4m3(c s_old / s) if s > s_old; new codes e4m3(x / s),
 * rounded to nearest even, saturating at 448.  Infinities and NaN are stored
 * as e4m3's NaN and do not enter a.  Rows of a page after the last token are
 * left as they are.  Asynchronous on `stream`; no workspace.
 *   k, v : device, [T, h_kv, 128] with token strides dims->k_stride, v_stride.
 * A page may receive tokens of one sequence only.
 * Errors: INVALID_ARG, UNSUPPORTED, MISALIGNED (16 bytes), CUDA.
 */
gdn_status gdn_kv_append(const void* k, const void* v, const int32_t* kv_lens_dev, const int32_t* page_table_dev,
                         const int32_t* cu_seqlens_dev, const gdn_kv_cache* cache, const gdn_kv_dims* dims,
                         void* stream);

/*
 * gdn_kv_read -- the cache's values of the last n_i tokens of each sequence
 * (n_i = kv_lens[i]: all of it), as bf16 or fp32: x = c s, exact.
 *   k_out, v_out : device, [T, h_kv, 128], packed; dims->k_stride and
 *                  v_stride apply to them.
 * Errors: as gdn_kv_append.
 */
gdn_status gdn_kv_read(void* k_out, void* v_out, const int32_t* kv_lens_dev, const int32_t* page_table_dev,
                       const int32_t* cu_seqlens_dev, const gdn_kv_cache* cache, const gdn_kv_dims* dims,
                       void* stream);

/* How gdn_kv_attn runs; plain data, fill with gdn_kv_attn_plan, do not edit. */
typedef struct gdn_kv_plan_t {
  int path;          /* which kernel: see gdn_kv_attn_plan */
  int rows;          /* query rows (token, query head of one group) per row tile */
  int max_row_tiles; /* row tiles of one sequence and key/value head, at most */
  int n_ctas;        /* CTAs the key tiles of all row tiles are shared out to; 0: a CTA each row tile */
  int item_cost;     /* what a row tile costs beyond its key tiles, in key tiles */
  int n_seqs, T, h_q, h_kv, dtype; /* copied, checked by gdn_kv_attn */
  int max_q_len;
  size_t off_desc, off_ml, off_o;  /* workspace sections */
  size_t workspace_bytes;
} gdn_kv_plan_t;

/*
 * gdn_kv_attn_plan -- host-only planning of gdn_kv_attn.
 *   max_q_len  : no sequence brings more tokens than this (<= 0: unknown; any
 *                number up to T, and the choice of kernel supposes T / n_seqs).
 *   max_kv_len : the longest sequence expected (<= 0: 64 max_pages); sizes the
 *                split only, so replays of a captured call may pass it.
 *   sm_count   : SMs to plan for; <= 0 queries the current device.
 * Errors: INVALID_ARG (also for calls past 2^31 units: row tiles times key
 * tiles of 128), UNSUPPORTED, CUDA (device query).
 */
gdn_status gdn_kv_attn_plan(const gdn_kv_dims* dims, int h_kv, int max_q_len, int max_kv_len, int sm_count,
                            gdn_kv_plan_t* out_plan);

/*
 * gdn_kv_attn -- attention of each new token over its sequence's cached keys
 * and values (the new tokens' own included: append them first).  For the
 * token at position p and query head j, over the keys the masks leave:
 *   w = softmax(scale q . k),  out = sum w v,  lse = log sum exp(scale q . k).
 * A token whose masks leave no key has out = 0 and lse = -inf.  Keys outside
 * the masks do not enter, whatever their codes.  A NaN code in an attended key,
 * or a q that is not finite, makes the whole row and its lse NaN; one in an
 * attended value the element it is in, and the whole row and its lse where the
 * masks cut the key's tile of 128.
 *   q    : device, [T, h_q, 128], dims->dtype, token stride dims->q_stride.
 *   out  : device, [T, h_q, 128], dims->dtype, token stride dims->out_stride.
 *   lse  : device, [T, h_q] fp32, or NULL.
 *   dims, plan : host; the plan must come from gdn_kv_attn_plan with these dims.
 *   workspace  : device, 256-byte aligned, >= plan->workspace_bytes; its
 *                contents on entry do not matter.  Not to be shared by calls
 *                that may run concurrently.
 * Both types run on the tensor cores; keys and values enter the products
 * exactly, and the softmax, the sum of the weights and all sums are fp32.
 * Queries and weights are rounded as they enter the products.  Below, a query
 * element stands against its row's largest, and a weight, times its value's
 * page scale, against the row's largest such product:
 *   GDN_BF16, plan->rows <= 32: a weight to 2^-8 of itself down to 2^-14 of the
 *     largest, below that to 2^-22 of the largest; a query element in full down
 *     to 2^-13 of the largest, below that to 2^-22 of it.
 *   GDN_BF16, plan->rows = 256: a weight to 2^-11 of itself down to 2^-17 of the
 *     largest, below that to 2^-28 of it; a query element to 2^-17.8 of the
 *     largest, so in full down to 2^-10 of it only.
 *   GDN_F32: a weight to 2^-22 of itself down to 2^-17 of the largest, below
 *     that to 2^-39 of it; a query element to 2^-24 of itself, or 2^-39 of the
 *     largest.
 * So an output whose heavy keys all have a value of zero there is coarser than
 * the others of its row.  Results repeat bit for bit under the same plan.
 * Asynchronous on `stream`; one or two kernels.
 * A sequence that brings more tokens than the plan's max_q_len is recorded as
 * the same device check (detail 7).
 * Errors: INVALID_ARG (also, as in planning, for calls past 2^31 units under
 * this call's max_pages), UNSUPPORTED, MISALIGNED, WORKSPACE, CUDA.
 */
gdn_status gdn_kv_attn(const void* q, const int32_t* kv_lens_dev, const int32_t* page_table_dev,
                       const int32_t* cu_seqlens_dev, const gdn_kv_cache* cache, void* out, float* lse,
                       const gdn_kv_dims* dims, const gdn_kv_plan_t* plan, void* workspace, size_t workspace_bytes,
                       void* stream);

/*
 * ---- Between the projections and the mixers ----
 * What the layers do with a projection's output before gdn_chunk_fwd,
 * gdn_decode_step, gdn_kv_append and gdn_kv_attn take it (no counterpart on
 * the FlashQLA pages).  Heads have 128 elements.  fp32 arithmetic; results are
 * rounded once, to dims->dtype, to nearest even.  All asynchronous on `stream`.
 */

/* Rotary positions: the pairs of a head's first `rot` elements turn by the
 * angle p f_i at position p, f_i = base^(-2i / rot) radians a token, i < rot/2. */
enum { GDN_ROPE_HALF = 0,         /* pairs (i, i + rot/2) */
       GDN_ROPE_INTERLEAVED = 1 }; /* pairs (2i, 2i + 1) */
/* Frequencies for contexts `factor` times longer than the model was trained on: */
enum { GDN_ROPE_PLAIN = 0,
       GDN_ROPE_LINEAR = 1,  /* f / factor */
       GDN_ROPE_NTK = 2,     /* base factor^(rot / (rot - 2)) instead of base: the slowest pair is slowed by factor, the fastest not */
       GDN_ROPE_PARTS = 3 }; /* with r = original_len f / 2 pi turns over the trained length and
                                keep = (r - low) / (high - low) held within [0, 1]: f keep + f / factor (1 - keep) */

typedef struct gdn_rope_opts {
  int rot;              /* elements of a head that turn: a multiple of 8, 8 to 128 */
  int scaling;          /* GDN_ROPE_PLAIN, LINEAR, NTK or PARTS */
  double base;          /* > 1 */
  double factor;        /* >= 1 (PLAIN: not read) */
  double original_len;  /* PARTS: > 0 tokens, and low < high turns */
  double low, high;
} gdn_rope_opts;

/*
 * gdn_rope_table -- host only: the frequencies as turns a token times 2^64,
 * to nearest: uint64 [rot / 2].  Copied to the device once, they give the
 * angle of any 32-bit position as the low 64 bits of a product, which is exact;
 * the table itself is off by half a unit (2^-65 turns a token) and by a few
 * roundings of fp64 in the frequency.
 * Errors: INVALID_ARG, UNSUPPORTED (rot, scaling).
 */
gdn_status gdn_rope_table(const gdn_rope_opts* opts, uint64_t* turns_host);

typedef struct gdn_rope {
  const uint64_t* turns;  /* device, [rot / 2], from gdn_rope_table */
  int rot;                /* 0: nothing turns, turns is not read */
  int layout;             /* GDN_ROPE_HALF or GDN_ROPE_INTERLEAVED */
  float magnitude;        /* turned elements are multiplied by it; 0 selects 1 */
} gdn_rope;

/* Norms of a head x, with weight w (or 1): x r w, */
enum { GDN_NORM_NONE = 0,
       GDN_NORM_RMS = 1,   /* r = 1 / sqrt(sum x^2 / 128 + eps) */
       GDN_NORM_UNIT = 2 }; /* r = 1 / sqrt(sum x^2 + eps) */

typedef struct gdn_rope_dims {
  int n_seqs;   /* sequences; without offsets and positions T / n_seqs tokens each */
  int T;        /* tokens of the call */
  int h_q, h_k; /* heads of q and of k; one of them may be 0, with its pointers null */
  int norm;     /* GDN_NORM_* */
  float eps;    /* 0 selects 1e-6; otherwise 1e-20 to 1e20 */
  int dtype;    /* GDN_BF16 or GDN_F32 */
  /* Elements from one token to the next, 0: heads * 128 (packed); a multiple of
   * 16 bytes and at least heads * 128, so the tensors may be parts of one fused
   * projection. */
  int64_t q_stride, k_stride, q_out_stride, k_out_stride;
  int64_t dq_stride, dk_stride; /* gdn_qk_rope_bwd; there q_out and k_out are d_q_out and d_k_out */
} gdn_rope_dims;

/*
 * gdn_qk_rope -- queries and keys, each head normalised, then rotated by its
 * token's position: y = m R_p (x r w), m the magnitude.
 *   q, k              : device, [T, h_q, 128] and [T, h_k, 128], dims->dtype.
 *   q_weight, k_weight: device fp32 [128], or NULL (1).  Not with GDN_NORM_NONE.
 *   positions         : device int32 [T], any values; or NULL: token t of the packed
 *                       batch is at t - cu_seqlens_dev[i] of its sequence i, or
 *                       with both NULL at t % (T / n_seqs).
 *   cu_seqlens_dev    : device int32 [n_seqs + 1], not read when positions are given.
 *                       Tokens outside every sequence (behind the last offset, say)
 *                       are left as they were.  Offsets that go back leave undefined
 *                       which tokens are done, with which positions; no access
 *                       leaves the buffers.
 *   rope              : host, or NULL (nothing turns).
 *   q_out, k_out      : device, like q and k.  Each may be its input itself (same
 *                       address and stride; the same address with another stride is
 *                       refused); otherwise outputs overlap nothing.
 * Where a head's sum of squares passes fp32's range it is taken of scaled
 * elements, so finite heads of any size are normalised.  Under a norm a NaN makes
 * NaN of its whole head, and an infinity NaN of itself and zeros of the others (r = 0).
 * A NaN that is turned makes NaN of its pair; an infinity makes infinities or NaN of
 * its pair, as its products with cosine and sine are.
 * Errors: INVALID_ARG, UNSUPPORTED (dtype, norm, rot, layout), MISALIGNED (16 bytes), CUDA.
 */
gdn_status gdn_qk_rope(const void* q, const void* k, const float* q_weight, const float* k_weight,
                       const int32_t* positions, const int32_t* cu_seqlens_dev, const gdn_rope* rope, void* q_out,
                       void* k_out, const gdn_rope_dims* dims, void* stream);

/* Device workspace of gdn_qk_rope_bwd, whatever its sizes.  Errors: INVALID_ARG (NULL). */
gdn_status gdn_qk_rope_bwd_workspace_bytes(size_t* bytes);

/*
 * gdn_qk_rope_bwd -- gradients of sum(q_out d_q_out) + sum(k_out d_k_out).  With
 * du = m R_p^T dy and n = x r:
 *   dw = sum over tokens and heads of du n,   dn = du w,
 *   dx = r (dn - n sum(dn n) / 128)  (GDN_NORM_UNIT: without the 128).
 * Inputs as gdn_qk_rope's; q and k are not read with GDN_NORM_NONE (may be NULL).
 *   d_q_out, d_k_out      : device, [T, h, 128], dims->dtype.
 *   dq, dk                : device, the same; each may be its d_q_out or d_k_out itself, as
 *                           gdn_qk_rope's outputs their inputs.
 *                           Tokens outside every sequence are left as they were, and
 *                           do not count in the weights' gradients.
 *   dq_weight, dk_weight  : device fp32 [128], or NULL (not wanted); need the weight.
 *   workspace             : device, 16-byte aligned, of gdn_qk_rope_bwd_workspace_bytes;
 *                           NULL without dq_weight and dk_weight.  Its contents on entry do
 *                           not matter; not to be shared by calls that may run concurrently.
 * The weights' gradients are summed in a fixed order: results repeat bit for bit.
 * Errors: as gdn_qk_rope, WORKSPACE.
 */
gdn_status gdn_qk_rope_bwd(const void* q, const void* k, const float* q_weight, const float* k_weight,
                           const int32_t* positions, const int32_t* cu_seqlens_dev, const gdn_rope* rope,
                           const void* d_q_out, const void* d_k_out, void* dq, void* dk, float* dq_weight,
                           float* dk_weight, const gdn_rope_dims* dims, void* workspace, size_t workspace_bytes,
                           void* stream);

/*
 * gdn_kv_append_rope -- gdn_kv_append of keys that are normalised and rotated on
 * the way, each by its position p in the cache (see there), and the queries
 * of the same tokens normalised and rotated beside them, in one launch.  The
 * keys' fp32 results are quantised without a rounding in between: page
 * scales, codes and what is not finite follow gdn_kv_append with them as x.
 *   k, v, kv_lens_dev, page_table_dev, cu_seqlens_dev, cache, dims: as gdn_kv_append.
 *   q      : device, [T, dims->h_q, 128], token stride dims->q_stride; or NULL.
 *   q_out  : device, like q, token stride dims->out_stride; may be q itself.  A
 *            token at p < 0 is rotated by that position; one outside every
 *            sequence is left as it was.
 *   k_weight, q_weight, rope, norm, eps: as gdn_qk_rope.
 * Errors: as gdn_kv_append and gdn_qk_rope.
 */
gdn_status gdn_kv_append_rope(const void* k, const void* v, const float* k_weight, const void* q,
                              const float* q_weight, void* q_out, const int32_t* kv_lens_dev,
                              const int32_t* page_table_dev, const int32_t* cu_seqlens_dev, const gdn_kv_cache* cache,
                              const gdn_kv_dims* dims, const gdn_rope* rope, int norm, float eps, void* stream);

/*
 * The short causal convolution before the gated delta rule [GDN, the layer's
 * block design]: C = (2 h_qk + h_v) 128 channels of a projection, heads of q,
 * then of k, then of v.  Per channel, with W taps w_0 .. w_{W-1}, a bias b and
 * the W - 1 inputs kept from before the sequence (or zeros) as x_{-W+1} .. x_{-1}:
 *   u_t = b + sum_j w_j x_{t - W + 1 + j},   y = u sigmoid(u)  or  y = u,
 * then q's and k's heads scaled to unit length: y / sqrt(sum y^2 + eps).
 */
enum { GDN_ACT_NONE = 0, GDN_ACT_SILU = 1 };

typedef struct gdn_conv_dims {
  int n_seqs;     /* sequences; without offsets T / n_seqs tokens each */
  int T;          /* tokens of the call; gdn_conv_step: n_seqs */
  int h_qk, h_v;
  int width;      /* taps W: 2, 3 or 4 */
  int activation; /* GDN_ACT_* */
  int norm;       /* 1: q's and k's heads to unit length; 0: not */
  float eps;      /* 0 selects 1e-6; otherwise 1e-20 to 1e20 */
  int dtype;      /* GDN_BF16 or GDN_F32: type of x, q, k, v and the states */
  int64_t x_stride;  /* elements from one token to the next in x, 0: C.  A multiple of */
  int64_t dx_stride; /* 16 bytes and at least C.  dx_stride: gdn_conv_bwd's dx. */
} gdn_conv_dims;

/*
 * gdn_conv_fwd -- the convolution of packed sequences.
 *   x              : device, [T, C], row stride dims->x_stride.
 *   weight         : device fp32 [C, W], w_{W-1} the tap of the token itself.
 *   bias           : device fp32 [C], or NULL.
 *   initial_state  : device, [n_seqs, W - 1, C] inputs before each sequence, oldest
 *                    first, or NULL (zeros).
 *   cu_seqlens_dev : device int32 [n_seqs + 1], or NULL.  Tokens outside every sequence
 *                    (behind the last offset, say) are left as they were.  With
 *                    offsets that leave [0, T] or go back the outputs are
 *                    undefined; no access leaves the buffers.
 *   q, k, v        : device, [T, h_qk, 128], [T, h_qk, 128], [T, h_v, 128], packed, as
 *                    gdn_chunk_fwd takes them.
 *   final_state    : device, like initial_state: each sequence's last W - 1 inputs, the
 *                    state's own among them where it is shorter; or NULL.  May not
 *                    overlap initial_state.
 * Outputs may not overlap inputs.
 * Errors: INVALID_ARG, UNSUPPORTED (dtype, width, activation), MISALIGNED (16 bytes), CUDA.
 */
gdn_status gdn_conv_fwd(const void* x, const float* weight, const float* bias, const void* initial_state,
                        const int32_t* cu_seqlens_dev, void* q, void* k, void* v, void* final_state,
                        const gdn_conv_dims* dims, void* stream);

/* Device workspace of gdn_conv_bwd for these dims.  Host only.  Errors: INVALID_ARG, UNSUPPORTED. */
gdn_status gdn_conv_bwd_workspace_bytes(const gdn_conv_dims* dims, size_t* bytes);

/*
 * gdn_conv_bwd -- gradients of sum(q d_q) + sum(k d_k) + sum(v d_v) +
 * sum(final_state d_final_state), gdn_conv_fwd's outputs, which are computed
 * again.  With g the gradient of a head's output, r = 1 / sqrt(sum y^2 + eps) and
 * n = y r:  dy = r (g - n sum(g n)) for q and k,  du = dy (s + u s (1 - s)), s =
 * sigmoid(u),  dx_t = sum_j w_j du_{t + W - 1 - j},  dw_j = sum_t du_t x_{t - W + 1 + j},
 * db = sum_t du_t; the gradient at the kept inputs is the initial state's.
 *   x, weight, bias, initial_state, cu_seqlens_dev, dims: as gdn_conv_fwd.
 *   d_q, d_k, d_v   : device, like q, k, v.
 *   d_final_state   : device, [n_seqs, W - 1, C], or NULL (zero).
 *   dx              : device, [T, C], row stride dims->dx_stride; tokens outside every
 *                     sequence are left as they were.
 *   d_weight, d_bias: device fp32 [C, W] and [C], or NULL (not wanted).
 *   d_initial_state : device, [n_seqs, W - 1, C], or NULL; written also when
 *                     initial_state is NULL (the gradient at zero).
 *   workspace       : device, 16-byte aligned, of gdn_conv_bwd_workspace_bytes; NULL without
 *                     d_weight and d_bias.  Its contents on entry do not matter; not to be
 *                     shared by calls that may run concurrently.
 * Sums over tokens are taken in a fixed order: results repeat bit for bit.
 * Outputs may not overlap inputs.  Errors: as gdn_conv_fwd, WORKSPACE.
 */
gdn_status gdn_conv_bwd(const void* x, const float* weight, const float* bias, const void* initial_state,
                        const int32_t* cu_seqlens_dev, const void* d_q, const void* d_k, const void* d_v,
                        const void* d_final_state, void* dx, float* d_weight, float* d_bias, void* d_initial_state,
                        const gdn_conv_dims* dims, void* workspace, size_t workspace_bytes, void* stream);

/*
 * gdn_conv_step -- one new token for each of n_seqs sequences, the
 * generation-time form of gdn_conv_fwd beside gdn_decode_step.
 *   x       : device, [n_seqs, C], row stride dims->x_stride; dims->T = n_seqs.
 *   state   : device, [n_seqs, W - 1, C], read, then overwritten with the last W - 1
 *             inputs, x's row among them.
 *   q, k, v : device, [n_seqs, h, 128], as gdn_decode_step takes them.
 * Errors: as gdn_conv_fwd.
 */
gdn_status gdn_conv_step(const void* x, const float* weight, const float* bias, void* state, void* q, void* k,
                         void* v, const gdn_conv_dims* dims, void* stream);

/*
 * gdn_debug_stall_ns -- test hook of the failure path (no counterpart on the
 * FlashQLA pages).  While ns > 0, each later gdn_chunk_fwd of this process on
 * the bf16 path makes the blocks of its chunk-local kernel first wait ns
 * nanoseconds on an mbarrier that nothing arrives on.  That bounded wait
 * runs out: the blocks record GDN_ERR_DEVICE_TIMEOUT with detail 6 in the
 * workspace's status word, free their tensor memory and return, and every
 * kernel after them sees the recorded failure and does no work, so o and
 * final_state are left unwritten.  ns = 0 (the default) turns it off.  A
 * process-wide setting for tests; not for production calls.
 * Errors: none.
 */
gdn_status gdn_debug_stall_ns(uint32_t ns);

/*
 * gdn_set_trace_events -- optional per-kernel timing (tracing).  Registers,
 * for the calling host thread, up to 32 caller-created cudaEvent_t handles.
 * While registered, each gdn_chunk_fwd (gdn_chunk_bwd, gdn_decode_step) on this thread
 * brackets its i-th kernel launch with events[2i] (recorded right before the
 * launch) and events[2i + 1] (right after it), both on the stream the kernel
 * is launched on, so cudaEventElapsedTime(events[2i], events[2i + 1]) is the
 * device time of kernel i.  n_events = 0 (or events = NULL) turns tracing
 * off.  The caller keeps ownership of the events.
 * Errors: INVALID_ARG for n_events outside 0..32 or a NULL event.
 */
gdn_status gdn_set_trace_events(void* const* events, int n_events);

/*
 * gdn_trace_last -- names of the kernels the last gdn_chunk_fwd (gdn_chunk_bwd,
 * gdn_decode_step) on this thread launched, in launch order (static
 * strings), and their count (at most 16).
 *   names : host array of at least max_names pointers, or NULL.
 * Returns the number of kernels launched (0 before any call).
 */
int gdn_trace_last(const char** names, int max_names);

#ifdef __cplusplus
}
#endif
#endif /* GDN_H_ */
