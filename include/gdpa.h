/*
 * gdpa.h -- C ABI of libgdpa: forward and backward passes of jagged
 * Generalized Dot-Product Attention (GDPA) on NVIDIA GB300 (sm_103a).
 *
 * The operation (techfeed summary of "GEM Training", sections "JFA" and
 * "GDPA"; remio.ai commentary, section on model/system co-design): attention
 * over a batch of variable-length, unpadded sequences, where the activation
 * applied to the scores is either a softmax or a GELU (tanh form), and where
 * the self-attention variant may be restricted to 64-token block-aligned
 * windows (techfeed summary, section "BlockAttention"; aigeeknews translation,
 * co-design section).  For sequence b, head h and query row i < Lq_b:
 *
 *   s_ij = scale * <q_i, k_j>                                  j in K(i)
 *   softmax : o_i = sum_j exp(s_ij - max s) v_j / sum_j exp(s_ij - max s)
 *   GELU    : o_i = (1/Lkv_b) * sum_j gelu_tanh(s_ij) v_j
 *   SiLU    : o_i = (1/Lkv_b) * sum_j silu(s_ij) v_j        (GDPA_ACT_SILU)
 *
 *   K(i) = all keys j < Lkv_b of sequence b            (window_blocks == 0)
 *        = keys j <= i with floor(i/64) - floor(j/64) <= window_blocks - 1
 *                                                      (window_blocks  > 0)
 *        = keys i - W < j <= i   (gdpa_fwd_sliding / gdpa_bwd_sliding, W tokens)
 *
 * The training entry points keep the softmax row logsumexp in the forward
 * (gdpa_fwd_lse, gdpa_fwd_sliding) and return dq, dk, dv in the backward
 * (gdpa_bwd, gdpa_bwd_sliding).  gdpa_fwd_mx takes q and k in MXFP8,
 * gdpa_fwd_mxfp8 q, k and v.
 *
 * For serving, keys and values of earlier calls stay in a paged cache of e4m3
 * codes (gdpa_cache_t): gdpa_cache_append stores new tokens, rotating them by
 * their position on the way, and gdpa_cache_fwd attends from new tokens to
 * everything that is stored.  For long histories gdpa_rope rotates jagged rows by
 * any positions (and returns the gradient of that), gdpa_cache_weights adds up
 * the attention weight that stored keys receive, and gdpa_cache_evict cuts
 * sequences to the tokens that received most.
 *
 * An empty key set gives o_i = 0.  The GELU's tanh is rewritten as a
 * logistic function, gelu(x) = x sigma(2u), whose sigma takes one of two
 * routes (gdpa_act_route_t): the special-function unit's exp2 and reciprocal
 * (the default), or the ALU-only form of the GDPA section ("ALU-only
 * activation", valid because QK-norm bounds the scores): a range-reduced
 * 6th-order Taylor polynomial of exp and a Newton reciprocal.  Either is
 * within 1e-3 of the exact tanh-GELU for |s| <= 17 and saturates correctly
 * beyond.
 *
 * Data layout (all pointers are device pointers unless named h_*):
 *   q    bf16 [Tq,  H, D]   row-major, contiguous, Tq  = q_offsets[B]
 *   k, v bf16 [Tkv, H, D]   row-major, contiguous, Tkv = kv_offsets[B]
 *   out  bf16 [Tq,  H, D]   every row is written (zeros for empty key sets)
 *   q_offsets, kv_offsets  int32 [B+1], offsets[0] = 0, non-decreasing
 * q, k, v and out must be 16-byte aligned.  D must be 64 or 128 (128 for
 * gdpa_fwd_mx, whose q and k are e4m3 codes with E8M0 scales).  Tq and Tkv
 * must be below 2^31.  Windows (block or sliding) require q_offsets ==
 * kv_offsets and act == GDPA_ACT_SOFTMAX.
 *
 * Ownership: the caller owns every buffer it passes; the library never frees
 * them and keeps no reference after the call returns (the GPU may still be
 * reading them until the stream reaches the end of the launched work).  The
 * library owns its plans and internal per-device work-list buffers (two,
 * used in turn).
 *
 * Streams: `stream` is a cudaStream_t passed as void* (NULL = legacy default
 * stream).  All kernels are enqueued on it; the entry points that plan on
 * every call (gdpa_fwd, gdpa_fwd_async, gdpa_fwd_lse, gdpa_fwd_sliding,
 * gdpa_fwd_mx, gdpa_fwd_mxfp8) copy their work list up on a library-owned
 * stream that `stream` then waits for (on a stream being captured, the copy
 * stays on that stream).  The pair
 * kernels take their work items at run time from a device counter; each
 * launch uses its own counter from a fixed pool of 1024, so launches in
 * flight at the same time on different streams are independent unless more
 * than 1024 are.
 *
 * Errors: every entry point returns a gdpa_status_t and never throws or
 * aborts.  Kernel-side failures (a bounded wait that ran out) are recorded in
 * a device status word; gdpa_device_status() reads and clears it.
 */
#ifndef GDPA_H_
#define GDPA_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  GDPA_ACT_SOFTMAX = 0,    /* online softmax */
  GDPA_ACT_GELU_TANH = 1,  /* (1/Lkv) * sum gelu_tanh(s) v (sigma route: gdpa_act_route_t) */
  GDPA_ACT_SILU = 2        /* (1/Lkv) * sum silu(s) v, silu(x) = x sigma(x), the same sigma
                              (an alternative activation of GDPA: remio.ai commentary,
                              model/system co-design section); no windows */
} gdpa_act_t;

/*
 * How the GELU and SiLU activations evaluate their sigma (process-wide, see
 * gdpa_set_act_route).  Both compute the same function to fp32 level:
 *   GDPA_ROUTE_SFU: sigma(z) = 1 / (1 + 2^(-z log2 e)) with the
 *     special-function unit's ex2.approx and rcp.approx (the default: on
 *     sm_103a it measured faster than the polynomial in every forward kernel);
 *   GDPA_ROUTE_ALU: the ALU-only form of the GDPA section of the techfeed
 *     summary of "GEM Training" (a 6th-order Taylor polynomial of exp after
 *     range reduction, Newton reciprocal), FMA and integer instructions only.
 * The backward follows the same route (value and derivative).
 */
typedef enum {
  GDPA_ROUTE_SFU = 0,
  GDPA_ROUTE_ALU = 1
} gdpa_act_route_t;

typedef enum {
  GDPA_OK = 0,
  GDPA_ERR_INVALID_ARG = 1,    /* bad pointer, size, offsets or combination */
  GDPA_ERR_UNSUPPORTED = 2,    /* valid request the library does not implement */
  GDPA_ERR_CUDA = 3,           /* a CUDA runtime/driver call failed */
  GDPA_ERR_DEVICE_TIMEOUT = 4, /* a kernel wait ran out of time (device status word) */
  GDPA_ERR_NO_MEMORY = 5       /* host or device allocation failed, or capacity too small */
} gdpa_status_t;

/* One unit of GPU work: query rows [q0, q0+R) of sequence `seq`, head
 * `head` (R = 128, or 256 for full attention over sequences averaging more
 * than 128 queries), against keys from `kv0` (sequence-local) to the end of
 * its key range.  Produced by the host tile planner (GDPA section: valid tiles are
 * precomputed on the CPU, empty ones skipped, and spread over the SMs). */
typedef struct {
  int32_t seq;
  int32_t head;
  int32_t q0;
  int32_t kv0;
} gdpa_work_item_t;

typedef struct gdpa_plan gdpa_plan_t;

/*
 * gdpa_fwd -- the whole forward pass in one call.
 * q_offsets / kv_offsets are DEVICE pointers: the call copies them to the host
 * (this synchronises `stream` once), plans the work list, uploads it to a
 * library-owned device buffer and launches the kernel on `stream`.  `scale`
 * multiplies every score.  Returns GDPA_OK once the kernel is enqueued.
 */
gdpa_status_t gdpa_fwd(const void* q, const void* k, const void* v, const int32_t* q_offsets,
                       const int32_t* kv_offsets, int B, int H, int D, int act, int window_blocks,
                       float scale, void* out, void* stream);

/*
 * gdpa_fwd_async -- the whole forward pass, fully asynchronous: the caller
 * passes the offsets twice, as HOST arrays (h_*, read during the call to plan
 * the work list; the caller may reuse them once the call returns) and as
 * DEVICE arrays (read by the kernel, same values).  Planning runs on the
 * calling thread while earlier work on `stream` is still executing; the work
 * list goes up through a library-owned pinned buffer.  No synchronisation.
 */
gdpa_status_t gdpa_fwd_async(const void* q, const void* k, const void* v, const int32_t* h_q_offsets,
                             const int32_t* h_kv_offsets, const int32_t* q_offsets, const int32_t* kv_offsets,
                             int B, int H, int D, int act, int window_blocks, float scale, void* out,
                             void* stream);

/*
 * gdpa_fwd_lse -- gdpa_fwd_async that also keeps, for the backward pass, the
 * row logsumexp of every softmax query row: lse[t * H + h] =
 * ln sum_j exp(scale <q_t, k_j>) over the row's key set (natural log; -inf
 * for a row whose sequence has no keys).  lse: device fp32 [Tq, H], 4-byte
 * aligned, written in full for softmax and not touched for GELU (may be
 * NULL then).  Every other argument, layout and result as gdpa_fwd_async.
 * The row logsumexp is the quantity the backward needs to rebuild the
 * softmax weights tile by tile (techfeed summary of "GEM Training", JFA
 * section: the forward of a training step feeds its backward).
 */
gdpa_status_t gdpa_fwd_lse(const void* q, const void* k, const void* v, const int32_t* h_q_offsets,
                           const int32_t* h_kv_offsets, const int32_t* q_offsets, const int32_t* kv_offsets, int B,
                           int H, int D, int act, int window_blocks, float scale, void* out, float* lse,
                           void* stream);

/*
 * gdpa_fwd_sliding -- the forward with a causal sliding window of
 * window_tokens tokens instead of block windows: query i of a sequence sees
 * the keys i - window_tokens < j <= i of its own sequence (the token-granular
 * window the BlockAttention section of the techfeed summary of "GEM
 * Training" names as the step before block-aligned attention).  Softmax only
 * (GDPA_ERR_UNSUPPORTED for GELU), self attention (q and kv offsets equal),
 * window_tokens >= 1.  lse: optional (may be NULL) device fp32 [Tq, H], as
 * gdpa_fwd_lse.  Offsets twice (host and device) and everything else as
 * gdpa_fwd_async; asynchronous on `stream`.
 */
gdpa_status_t gdpa_fwd_sliding(const void* q, const void* k, const void* v, const int32_t* h_q_offsets,
                               const int32_t* h_kv_offsets, const int32_t* q_offsets, const int32_t* kv_offsets,
                               int B, int H, int D, int act, int window_tokens, float scale, void* out, float* lse,
                               void* stream);

/*
 * gdpa_fwd_mx -- the forward (full attention) with q and k in MXFP8, the
 * microscaling FP8 format the techfeed summary of "GEM Training" (section on
 * MXFP8 ultra-low-precision training) and the aigeeknews translation
 * (compute-efficiency section, "MXFP8 attention") apply to attention:
 *
 *   q8, k8  uint8 [T, H, D]     OCP e4m3 element codes ("E4M3FN": no
 *                               infinities, S.1111.111 NaN)
 *   q_sf, k_sf uint8 [T, H, D/32]  OCP E8M0 scale codes, 2^(e - 127): code b
 *                               of a (token, head) row scales its elements
 *                               [32 b, 32 b + 32)
 *   q_id = e4m3(q8_id) * 2^(q_sf_i,floor(d/32) - 127), k likewise
 *
 * The score product runs on the block-scaled e4m3 tensor-core MMA with fp32
 * accumulation; v and out stay bf16, and everything after the scores is
 * gdpa_fwd_lse's (softmax, GELU or SiLU; lse optional, may be NULL).  D must
 * be 128 (GDPA_ERR_UNSUPPORTED otherwise), no windows.  q8, k8, v and out
 * 16-byte aligned, q_sf and k_sf 4-byte aligned (each row's four codes are
 * read as one 32-bit word).  Offsets twice (host and device) as
 * gdpa_fwd_async; asynchronous on `stream`.  The buffers stay the caller's.
 */
gdpa_status_t gdpa_fwd_mx(const void* q8, const void* q_sf, const void* k8, const void* k_sf, const void* v,
                          const int32_t* h_q_offsets, const int32_t* h_kv_offsets, const int32_t* q_offsets,
                          const int32_t* kv_offsets, int B, int H, int D, int act, float scale, void* out, float* lse,
                          void* stream);

/*
 * gdpa_fwd_mxfp8 -- the forward (full attention, softmax) with q, k and v
 * all in MXFP8, both products on the block-scaled e4m3 tensor-core MMA (same
 * sources as gdpa_fwd_mx).  q8, q_sf, k8, k_sf as gdpa_fwd_mx; v is
 * quantised along the contraction of the P V product, the keys, so it
 * arrives key-major:
 *
 *   vt8    uint8 [H*D, VT]      e4m3 codes; row h*D + d holds coordinate d
 *                               of head h for every key: sequence b's keys
 *                               at columns [P_b, P_b + Lkv_b),
 *                               P_b = 32 * sum_{b' < b} ceil(Lkv_b' / 32),
 *                               VT = P_B; the columns [P_b + Lkv_b, P_{b+1})
 *                               must hold finite codes (zero)
 *   vt_sf  uint8 [VT/32, H*D]   E8M0 scales: byte [c, h*D + d] scales
 *                               columns [32 c, 32 c + 32) of row h*D + d
 *   v_jd = e4m3(vt8[h*D + d, P_b + j]) * 2^(vt_sf[(P_b + j) / 32, h*D + d] - 127)
 *
 * The weights P_ij (exp2 of the scaled scores less the row's running
 * maximum) are rounded on chip to e4m3 with one E8M0 scale per 32 keys of a
 * row -- the scale puts the block's largest weight just under 448, so no
 * code saturates -- and the row sum takes the unrounded weights.  D must be
 * 128 and act GDPA_ACT_SOFTMAX (GDPA_ERR_UNSUPPORTED otherwise).  q8, k8,
 * vt8 and out 16-byte aligned; q_sf, k_sf 4-byte aligned; vt_sf any.  lse
 * optional (may be NULL).  Offsets twice (host and device) as
 * gdpa_fwd_async; the host copy also fixes VT.  Asynchronous on `stream`;
 * the buffers stay the caller's.
 */
gdpa_status_t gdpa_fwd_mxfp8(const void* q8, const void* q_sf, const void* k8, const void* k_sf, const void* vt8,
                             const void* vt_sf, const int32_t* h_q_offsets, const int32_t* h_kv_offsets,
                             const int32_t* q_offsets, const int32_t* kv_offsets, int B, int H, int D, int act,
                             float scale, void* out, float* lse, void* stream);

/*
 * gdpa_bwd -- gradients of the forward for an upstream gradient dout:
 *   dq = dL/dq, dk = dL/dk, dv = dL/dv for L = sum(dout * out), computed by
 * the chain rule of the forward's definition (techfeed summary of "GEM
 * Training", JFA section: a backward over batch x heads without atomics):
 *   softmax: P_ij = exp(scale <q_i,k_j> - lse_i), dS_ij = P_ij (<dO_i,v_j> - <dO_i,o_i>)
 *   GELU:    P_ij = gelu(scale <q_i,k_j>) / Lkv,  dS_ij = gelu'(...) <dO_i,v_j> / Lkv
 *   dv_j = sum_i P_ij dO_i,  dq_i = scale sum_j dS_ij k_j,  dk_j = scale sum_i dS_ij q_i
 * q, k, v, out, dout: device bf16 [tokens, H, D] (out and lse from
 * gdpa_fwd_lse on the same inputs); lse: device fp32 [Tq, H] (softmax only;
 * may be NULL for GELU); offsets twice, host (h_*, read during the call) and
 * device, as gdpa_fwd_async; dq: device bf16 [Tq, H, D]; dk, dv: device bf16
 * [Tkv, H, D]; all written in full (keys no query sees get zero gradients).
 * Tensors 16-byte aligned.  window_blocks > 0 (block windows, softmax, self
 * attention) as in the forward: each query row's gradient runs over its
 * window only.  Asynchronous on `stream`; the library keeps a
 * grow-only device buffer for the work lists and 8 Tq H bytes of scratch.
 * Errors as gdpa_fwd (a wait that runs out shows in gdpa_device_status).
 */
gdpa_status_t gdpa_bwd(const void* q, const void* k, const void* v, const void* out, const void* dout,
                       const float* lse, const int32_t* h_q_offsets, const int32_t* h_kv_offsets,
                       const int32_t* q_offsets, const int32_t* kv_offsets, int B, int H, int D, int act,
                       int window_blocks, float scale, void* dq, void* dk, void* dv, void* stream);

/*
 * gdpa_bwd_sliding -- gdpa_bwd for the causal sliding window of
 * window_tokens tokens (the forward of gdpa_fwd_sliding, whose out and lse
 * it takes).  Softmax only, self attention, window_tokens >= 1; everything
 * else as gdpa_bwd.
 */
gdpa_status_t gdpa_bwd_sliding(const void* q, const void* k, const void* v, const void* out, const void* dout,
                               const float* lse, const int32_t* h_q_offsets, const int32_t* h_kv_offsets,
                               const int32_t* q_offsets, const int32_t* kv_offsets, int B, int H, int D, int act,
                               int window_tokens, float scale, void* dq, void* dk, void* dv, void* stream);

/*
 * gdpa_fwd_noalloc -- gdpa_fwd for callers that must not allocate memory.
 * The pages describe no such entry point; it exists for users of this
 * library.  Some callers cannot allocate where they run attention: a serving
 * process that splits all device memory into a fixed arena at start-up and
 * forbids allocation on its request path, or a framework hook that must not
 * go around its own caching allocator.  This call allocates nothing -- no
 * cudaMalloc, cudaFree, cudaMallocHost or other allocating routine -- on the
 * device or the host: the work list lives in a file-scope device array of
 * 4 MiB and is planned in fixed host arrays by the same planner gdpa_fwd
 * uses.
 * Arguments, layout and results are those of gdpa_fwd (device offsets; every
 * call copies them to the host and synchronises `stream`).  Limits: B <= 65536
 * sequences and at most 261632 work items (query tiles x heads, about 33M
 * query rows x heads); larger requests return GDPA_ERR_NO_MEMORY before any
 * GPU work.
 * First call on a device: it looks up the array's device address (with that
 * device current); make it before any stream capture.  With CUDA's lazy
 * module loading (the default), the driver loads the array and the kernels
 * onto a device the first time they are used there, and that load reserves
 * device memory (the 4 MiB array and the kernels' code); a device holds them
 * from then until the process exits.  A caller that carves device memory
 * into an arena should therefore make one small call per device at start-up,
 * before carving it (or load modules eagerly, CUDA_MODULE_LOADING=EAGER).
 * Every call shares the array and the host arrays: calls are serialised on
 * the host, but two calls whose kernels overlap on the GPU (different
 * streams) race on the work list -- order them on one stream or synchronise
 * between them.  Each call rewrites the whole part of the array its launch
 * reads.
 */
gdpa_status_t gdpa_fwd_noalloc(const void* q, const void* k, const void* v, const int32_t* q_offsets,
                               const int32_t* kv_offsets, int B, int H, int D, int act, int window_blocks,
                               float scale, void* out, void* stream);

/*
 * gdpa_plan_create -- build a reusable plan from HOST offsets (the same
 * arrays the caller will later pass on the device).  Allocates the plan and
 * its device work list; *plan is NULL on failure.  Planning is host work:
 * tile enumeration plus longest-processing-time-first balancing over the SMs
 * of the current device.
 */
gdpa_status_t gdpa_plan_create(const int32_t* h_q_offsets, const int32_t* h_kv_offsets, int B, int H,
                               int D, int act, int window_blocks, gdpa_plan_t** plan);

/*
 * gdpa_plan_create_sliding -- the plan of gdpa_fwd_sliding (causal sliding
 * window of window_tokens >= 1 tokens; self attention: h_q_offsets and
 * h_kv_offsets equal; softmax).  Launch it with gdpa_fwd_planned.
 * GDPA_ERR_INVALID_ARG for window_tokens < 1, unequal offsets or another act.
 */
gdpa_status_t gdpa_plan_create_sliding(const int32_t* h_q_offsets, const int32_t* h_kv_offsets, int B, int H,
                                       int D, int act, int window_tokens, gdpa_plan_t** plan);

/*
 * gdpa_fwd_planned -- launch the forward pass with a plan; fully asynchronous
 * on `stream`.  The device offsets must hold the values the plan was built
 * from.  The kernels clip every work item to the rows of the tensors the plan
 * was built for, so offsets that reach past them never make the launch read
 * or write outside q, k, v or out; such a launch is flagged and
 * gdpa_device_status() then returns GDPA_ERR_INVALID_ARG (its output is
 * undefined).  Offsets that differ from the plan's but stay inside the
 * tensors are not detected: the output is then undefined.
 */
gdpa_status_t gdpa_fwd_planned(const gdpa_plan_t* plan, const void* q, const void* k, const void* v,
                               const int32_t* q_offsets, const int32_t* kv_offsets, float scale,
                               void* out, void* stream);

/* Frees the plan (synchronises the device if its buffers may be in use). */
void gdpa_plan_destroy(gdpa_plan_t* plan);

/* Number of work items / CTAs of a plan (for reporting); -1 on NULL. */
int64_t gdpa_plan_num_items(const gdpa_plan_t* plan);
int gdpa_plan_num_ctas(const gdpa_plan_t* plan);

/*
 * gdpa_fwd_host -- end-to-end call with HOST buffers: copies q, k, v and the
 * offsets to library-owned device buffers on `stream`, runs the forward pass
 * and copies `h_out` back, then synchronises `stream`.  Host buffers should be
 * pinned (page-locked) for full copy bandwidth.
 */
gdpa_status_t gdpa_fwd_host(const void* h_q, const void* h_k, const void* h_v, const int32_t* h_q_offsets,
                            const int32_t* h_kv_offsets, int B, int H, int D, int act, int window_blocks,
                            float scale, void* h_out, void* stream);

/*
 * gdpa_plan_enumerate -- the host planner alone, no GPU needed.  Fills
 * `items` (capacity `capacity`) grouped by CTA and `cta_begin` [num_ctas+1]
 * (items of CTA c are items[cta_begin[c] .. cta_begin[c+1])); `cost` (may be
 * NULL) receives each item's estimated cost; `rows_per_item` (may be NULL)
 * receives R; `kv_tile` (may be NULL) receives the keys per K/V tile the
 * kernel stages (64 for block windows and short key ranges on 256-row
 * items, else 128).  *n_items always receives the required count;
 * GDPA_ERR_NO_MEMORY if it exceeds `capacity`.
 */
gdpa_status_t gdpa_plan_enumerate(const int32_t* h_q_offsets, const int32_t* h_kv_offsets, int B, int H,
                                  int D, int act, int window_blocks, int num_ctas,
                                  gdpa_work_item_t* items, int64_t capacity, int32_t* cta_begin,
                                  int64_t* cost, int64_t* n_items, int32_t* rows_per_item, int32_t* kv_tile);

/*
 * gdpa_act_eval -- evaluates the kernel's device activation elementwise:
 * y[i] = gelu(x[i]) (act = GDPA_ACT_GELU_TANH) or y[i] = silu(x[i])
 * (act = GDPA_ACT_SILU) through the current route (gdpa_set_act_route),
 * or y[i] = 2^x[i] with the exponential the softmax path uses
 * (act = GDPA_ACT_SOFTMAX).  x, y: device fp32 [n].  For accuracy tests;
 * GDPA_ERR_INVALID_ARG for any other act.
 */
gdpa_status_t gdpa_act_eval(int act, const float* x, float* y, int64_t n, void* stream);

/*
 * gdpa_set_act_route -- selects the route (gdpa_act_route_t) every later
 * forward launch and gdpa_act_eval call of this process uses for the GELU and
 * SiLU sigma; launches already enqueued keep theirs.  Thread-safe (an atomic
 * word).  GDPA_ERR_INVALID_ARG for any other value (the route is unchanged).
 * gdpa_get_act_route returns the current one.
 */
gdpa_status_t gdpa_set_act_route(int route);
int gdpa_get_act_route(void);

/*
 * gdpa_device_status -- synchronises `stream`, then reads and clears the
 * device status word of the current device.  Returns GDPA_OK,
 * GDPA_ERR_DEVICE_TIMEOUT (a kernel gave up on a wait; its output is
 * undefined), GDPA_ERR_INVALID_ARG (a forward launch met device offsets past
 * its tensors, see gdpa_fwd_planned; its output is undefined) or
 * GDPA_ERR_CUDA.
 */
gdpa_status_t gdpa_device_status(void* stream);

/*
 * gdpa_wait_selftest -- launches one thread that waits, with the same
 * bounded mbarrier wait every role of the forward kernel uses, on a barrier
 * nothing ever arrives on.  After `timeout_ms` (1..10000) the wait gives up
 * and sets the device status word; gdpa_device_status() then returns
 * GDPA_ERR_DEVICE_TIMEOUT and the context stays usable.  For tests of the
 * failure path: no fault, trap or hang is involved.
 */
gdpa_status_t gdpa_wait_selftest(int timeout_ms, void* stream);

/* How gdpa_cache_append pairs the coordinates it rotates (rot_dim of a head's D). */
typedef enum {
  GDPA_ROPE_HALF = 0,        /* pairs (i, i + rot_dim / 2) */
  GDPA_ROPE_INTERLEAVED = 1  /* pairs (2 i, 2 i + 1) */
} gdpa_rope_style_t;

/*
 * A paged key/value cache in 8 bits.  The struct and every buffer it names
 * are the caller's; the calls below read the struct only while they run.
 *
 *   k_codes, v_codes  device uint8 [num_pages, H, page_tokens, D]  OCP e4m3
 *   k_sf, v_sf        device uint8 [num_pages, H, page_tokens/16]  OCP E8M0
 *   value = e4m3(code) * 2^(sf - 127), one scale for 16 tokens of one head; a
 *   scale is at most 254 (gdpa_cache_append never writes more than 247)
 *
 * Token t of sequence b lies in page page_table[b, t / page_tokens] at slot
 * t % page_tokens.  H is the number of key/value heads, D 64 or 128,
 * page_tokens a power of two from 16 to 1024.  Codes must be 16-byte aligned,
 * scales 4-byte.  A new page needs no clearing: a block's scale and codes are not read before
 * they were written.
 *
 * inv_freq: HOST double [rot_dim / 2], radians per position of each rotated
 * pair (NULL with rot_dim 0: no rotation); rot_dim: how many leading
 * coordinates of a head turn, a multiple of 16 up to D.
 */
typedef struct {
  void* k_codes;
  void* v_codes;
  void* k_sf;
  void* v_sf;
  int32_t num_pages;
  int32_t page_tokens;
  int32_t H;
  int32_t D;
  const double* inv_freq;
  int32_t rot_dim;
  int32_t rope_style; /* gdpa_rope_style_t */
} gdpa_cache_t;

/*
 * gdpa_cache_append -- stores the keys and values of new tokens, and rotates
 * keys and (optionally) queries by their positions.
 *
 *   k, v   device bf16, row t at k + t * k_stride (elements): [H, D]
 *   q      device bf16, row t at q + t * q_stride: [Hq, D]; may be NULL
 *          (Hq, q_stride and q_out are ignored then)
 *   q_out  device bf16 [T, Hq, D] contiguous: the rotated queries (may be q
 *          itself if q is contiguous)
 *   offsets     device int32 [B+1], offsets[0] = 0, non-decreasing: rows
 *               [offsets[b], offsets[b+1]) are the new tokens of sequence b
 *   kv_lens     device int32 [B]: tokens of each sequence AFTER this call, so
 *               new row i of sequence b has position
 *               kv_lens[b] - (offsets[b+1] - offsets[b]) + i
 *   page_table  device int32 [B, max_pages]; entries behind a sequence's last
 *               page are not read
 *   T           rows of q, k and v; rows from offsets[B] on are padding, not
 *               read, and q_out keeps what it held there
 *
 * A pair (x, y) at position p turns by p * inv_freq: (x cos - y sin, y cos + x
 * sin).  The angle is right to 2^-32 turns at every position (a 64-bit fraction
 * of a turn, times p, modulo 1) and then rounded to fp32 (2^-26 turns at most);
 * sine, cosine and the rotated pair are fp32.
 *
 * Quantisation: for the tokens that this call adds to a block of 16 and one
 * head, A = the largest finite magnitude; e = the smallest integer >= -127
 * with A <= 448 * 2^e.  If the block holds earlier tokens, e is at least its
 * present exponent, and where it grows the earlier codes are rounded again to
 * e4m3(code * 2^(e_old - e)).  Codes are rounded to nearest even; what is not
 * finite becomes the NaN code.
 *
 * Strides are in elements, multiples of 8, and at least H * D (Hq * D); q, k,
 * v and q_out 16-byte aligned.  T is below 2^31 - 256, B below 2^31 - 4097,
 * max_pages * page_tokens below 2^31.  Two sequences may share pages that both only
 * read; a block into which both append has undefined contents.
 *
 * Asynchronous on `stream`, one kernel, no allocation, no host read of device
 * data: it may be captured into a graph, which then reads offsets, lengths and
 * table anew at each replay.  Offsets, lengths or page numbers out of range
 * never make it write outside the buffers: the tokens concerned are skipped
 * and gdpa_device_status() returns GDPA_ERR_INVALID_ARG.
 */
gdpa_status_t gdpa_cache_append(const gdpa_cache_t* cache, const void* q, int64_t q_stride, const void* k,
                                int64_t k_stride, const void* v, int64_t v_stride, const int32_t* offsets,
                                const int32_t* kv_lens, const int32_t* page_table, int64_t T, int B, int Hq,
                                int max_pages, void* q_out, void* stream);

/*
 * gdpa_cache_fwd -- softmax attention of new tokens over the cache:
 *   o = sum_j exp(scale <q, k_j> - m) v_j / sum_j exp(scale <q, k_j> - m)
 * Query head h reads key/value head h / (Hq / H); Hq must be a multiple of H.
 * Row i of sequence b (n rows, kv_lens[b] = L tokens in the cache) sees
 *   causal = 1: the keys j <= L - n + i (its own position: the rows are the
 *               last n tokens); with window_tokens W > 0 only those with
 *               j > L - n + i - W as well
 *   causal = 0: all L keys (window_tokens must be 0)
 * A row that sees no key gives 0, and -inf in lse.  Keys that a row does not
 * see never influence it, whatever they hold (NaN codes included; beside hidden
 * values above 2^100 a row's own below 2^-80 may lose bits).
 *
 * Scores, softmax statistics, sums and lse are fp32; a score that fp32 does not
 * hold may make its row NaN.  Rounded to fewer bits are
 *   q        to fp16 after a division by the row's largest power of two:
 *            elements down to 2^-17 of the largest are exact, smaller ones are
 *            off by 2^-25 of it
 *   weights  exp(s - m) to fp16: 2^-11 of themselves down to 2^-15 of the row's
 *            largest, fewer bits below, and zero below 2^-25
 *   out      to bf16
 * Blocks of V that a row sees should have scales less than 2^100 apart: what
 * smaller ones add may be lost.
 *
 *   q      device bf16, row t at q + t * q_stride (elements): [Hq, D]
 *   out    device bf16 [T, Hq, D] contiguous; rows from offsets[B] on keep
 *          what they held
 *   lse    optional (may be NULL) device fp32 [T, Hq]: ln sum_j exp(scale <q, k_j>)
 *   offsets, kv_lens, page_table, max_pages, T, B  as gdpa_cache_append; the
 *          cache must already hold the kv_lens[b] tokens
 *   max_q  the most rows any sequence has, as far as the caller knows: it
 *          picks the kernel, one for the whole batch; sequences with more rows
 *          are still computed.  max_pages is taken for the longest sequence in
 *          that choice: a table much wider than the sequences costs short ones
 *          a second kernel (about 7 us)
 *   workspace  device memory, 16-byte aligned, of at least
 *          gdpa_cache_workspace_size() bytes, the caller's.  It holds nothing
 *          between calls; calls (or captured graphs) that may run at the same
 *          time need one each
 *
 * T * Hq / H must be below 2^31 - 256.
 *
 * Asynchronous on `stream`, no allocation, no host read of device data (may
 * be captured).  Offsets, lengths or page numbers out of range are handled as
 * in gdpa_cache_append: keys on a page out of range are not seen.  A workspace
 * that is too small returns GDPA_ERR_NO_MEMORY.
 *
 * With many rows (max_q * Hq / H above 48, and few keys aside 96) a sequence and
 * head whose blocks of V have scales 2^16 or more apart, zeros aside, or a NaN
 * value that some rows see and others do not, is computed row by row: right, but
 * about 1400 times as slow.
 */
gdpa_status_t gdpa_cache_fwd(const gdpa_cache_t* cache, const void* q, int64_t q_stride, const int32_t* offsets,
                             const int32_t* kv_lens, const int32_t* page_table, int64_t T, int B, int Hq,
                             int max_pages, int max_q, int causal, int window_tokens, float scale, void* out,
                             float* lse, void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace gdpa_cache_fwd needs on the current device for Hq query
 * heads and max_q rows a sequence. */
gdpa_status_t gdpa_cache_workspace_size(const gdpa_cache_t* cache, int Hq, int max_q, int64_t* bytes);

/* How gdpa_rope_freqs stretches the positions of a context longer than the trained one. */
typedef enum {
  GDPA_ROPE_SCALE_NONE = 0,   /* f_i = base^(-2 i / rot_dim) */
  GDPA_ROPE_SCALE_LINEAR = 1, /* f_i / factor */
  GDPA_ROPE_SCALE_BASE = 2,   /* base * factor^(rot_dim / (rot_dim - 2)) in place of base: the first pair
                                 keeps its frequency, the last one's is divided by factor (a base that 64
                                 bits do not hold is refused) */
  GDPA_ROPE_SCALE_RAMP = 3    /* by wave length: f_i where a pair turns `fast` times or more over the trained
                                 context, f_i / factor where it turns `slow` times or less, a linear ramp of
                                 the pair's index between; magnitude 0.1 ln(factor) + 1 */
} gdpa_rope_scaling_t;

/*
 * gdpa_rope_freqs -- fills inv_freq (HOST double [rot_dim / 2], radians per
 * position of each rotated pair) and *magnitude, for gdpa_rope and, as
 * gdpa_cache_t's inv_freq, for gdpa_cache_append (which has no magnitude:
 * multiply the attention's scale by its square instead where whole heads turn).
 * rot_dim: a multiple of 16 up to 128; base > 1; factor >= 1 (ignored without
 * scaling); trained, fast, slow: the ramp's only, trained > 0, fast > slow > 0.
 * The ramp begins at the pair of index floor(i(fast)) and ends at that of index
 * ceil(i(slow)), i(turns) = rot_dim ln(trained / (2 pi turns)) / (2 ln base),
 * limited to [0, rot_dim - 1].  All in 64 bits, on the host; needs no GPU.
 */
gdpa_status_t gdpa_rope_freqs(int rot_dim, double base, int scaling, double factor, int64_t trained, double fast,
                              double slow, double* inv_freq, float* magnitude);

/*
 * gdpa_rope -- rotates rows of a jagged batch by their positions, or (inverse =
 * 1) returns the gradient of that: the same magnitude, the opposite turn.
 *
 *   x   device bf16, row t at x + t * x_stride (elements): [H, D]
 *   y   device bf16, row t at y + t * y_stride: [H, D]; may be x itself with
 *       the same stride; otherwise no row of y may overlap one of x (which is
 *       refused; rows of both may lie between one another)
 *   offsets    device int32 [B+1], offsets[0] = 0, non-decreasing: rows
 *              [offsets[b], offsets[b+1]) are those of sequence b
 *   first      device int32 [B]: the position of each sequence's first row (NULL:
 *              0); row i of sequence b has position first[b] + i.  (After an
 *              eviction a new token's position is no longer its cache's length:
 *              rotate it here and append it to a cache without rotation.)
 *   T          rows of x and y; rows from offsets[B] on are padding: not read,
 *              and y keeps what it held there
 *   inv_freq   HOST double [rot_dim / 2], radians per position, read during the
 *              call; may be NULL with rot_dim 0
 *   rot_dim    how many leading coordinates of a head turn, a multiple of 16 up to
 *              D; the others are copied
 *   magnitude  what the turned coordinates are multiplied by
 *
 * A pair (x, y) at position p turns by a = p * inv_freq:
 *   inverse = 0:  magnitude (x cos a - y sin a, y cos a + x sin a)
 *   inverse = 1:  magnitude (x cos a + y sin a, y cos a - x sin a)
 * rope_style (gdpa_rope_style_t) says which coordinates are a pair.  Queries and
 * keys that lie side by side in a fused projection's rows are turned by one call
 * (H: the heads of both).  The angle is as exact as gdpa_cache_append's; sine,
 * cosine and the rotated pair are fp32, rounded once to bf16.
 *
 * D is 64 or 128.  Strides are multiples of 8 and at least H * D; x and y
 * 16-byte aligned.  T is below 2^31 - 256, B below 2^31 - 4097.  Asynchronous
 * on `stream`, one kernel, no allocation, no host read of device data (may be
 * captured; a replay reads offsets and first anew).  Offsets out of range never make
 * it read or write outside the buffers: the rows of a sequence that begins
 * below 0 or ends behind T are skipped and gdpa_device_status() returns
 * GDPA_ERR_INVALID_ARG (where offsets decrease, which sequence a row counts to is
 * undefined).
 */
gdpa_status_t gdpa_rope(const void* x, int64_t x_stride, const int32_t* offsets, const int32_t* first, int64_t T, int B,
                        int H, int D, const double* inv_freq, int rot_dim, int rope_style, float magnitude, int inverse,
                        void* y, int64_t y_stride, void* stream);

/*
 * gdpa_cache_weights -- how much attention weight each stored key has received:
 * adds what the rows of this call give it, for gdpa_cache_evict to choose by.
 *
 *   weights[j] = (j < L - n ? decay * weights_in[j] : 0) + sum p_ij
 *   p_ij = exp(scale <q_i, k_j> - lse_i)
 *
 * for every key j < L of a sequence with n > 0 rows and L = kv_lens[b] tokens, over
 * the rows i of the sequence that see key j (as in gdpa_cache_fwd: causal,
 * window_tokens) and the query heads that read its key head.  The last n keys, the
 * rows' own, begin at 0, so a new page needs no clearing.  Sequences without rows
 * keep their weights.
 *
 *   weights     device fp32 [num_pages, H, page_tokens], in the cache's pages;
 *               16-byte aligned
 *   weights_in  the same layout, or NULL (all zero: what this call gives alone); may
 *               be weights itself, and must not overlap it otherwise
 *   decay       finite, >= 0; 1 sums over all calls, less lets old weight fade
 *   lse         device fp32 [T, Hq] from gdpa_cache_fwd on the same rows.  A row of
 *               -inf saw no key and gives nothing.  (The last rows of a prompt may
 *               stand for all of it; the keys in front of them count as earlier ones
 *               then, so weights_in is NULL, or holds something for them)
 *   q, q_stride, offsets, kv_lens, page_table, T, B, Hq, max_pages, max_q, causal,
 *   window_tokens, scale  as gdpa_cache_fwd
 *
 * Scores, weights and their sums are fp32, summed in an order that does not depend
 * on timing.  Keys that a row does not see take nothing from it, whatever it
 * holds; a NaN in a row or its lse goes to the keys that it sees, one in a key to that key.
 * With few rows (max_q * Hq / H up to 64, up to 112 with D = 64) queries are
 * rounded as in gdpa_cache_fwd; with more they are taken as they are.
 *
 * A page that two sequences of the call share has undefined weights.
 * Asynchronous on `stream`, no allocation, no workspace, no host read of device data (may
 * be captured).  Offsets, lengths or page numbers out of range are handled as in
 * gdpa_cache_fwd: nothing is written outside the buffers, and
 * gdpa_device_status() returns GDPA_ERR_INVALID_ARG.
 */
gdpa_status_t gdpa_cache_weights(const gdpa_cache_t* cache, const void* q, int64_t q_stride, const float* lse,
                                 const int32_t* offsets, const int32_t* kv_lens, const int32_t* page_table, int64_t T,
                                 int B, int Hq, int max_pages, int max_q, int causal, int window_tokens, float scale,
                                 float decay, const float* weights_in, float* weights, void* stream);

/*
 * gdpa_cache_evict -- cuts each sequence to its `budget` most attended tokens,
 * every head by its own weights, and stores what is kept in other pages.
 *
 * Of a sequence of L = kv_lens[b] tokens each head keeps K = min(L, budget): the
 * first `sink` and the last `recent` ones always, and of the others those with
 * the largest weights, equal ones by the lower place (a NaN counts as less than
 * any number).  They keep their order: the i-th kept token goes to page
 * new_table[b, i / page_tokens], slot i % page_tokens, with its codes of K and
 * V and its weight.  16 tokens of a new block take the largest of their scales,
 * and codes from smaller ones are rounded to it: e4m3(code * 2^(e - e_new)), to
 * nearest even.
 *
 * In a sequence that was cut a token's place is no longer its position, and the same
 * place holds another token in every head.  gdpa_cache_fwd and gdpa_cache_weights go by places:
 * causal = 1 still hides later tokens from earlier ones, but window_tokens > 0 counts the
 * kept tokens of a head, however far apart their positions are.
 *
 *   weights    device fp32 [num_pages, H, page_tokens] (gdpa_cache_weights), read
 *              in the old pages and written in the new ones; 16-byte aligned
 *   kv_lens    device int32 [B];  page_table  device int32 [B, max_pages]
 *   budget     >= 1;  sink, recent  >= 0, sink + recent <= budget
 *   new_table  device int32 [B, new_max_pages]: new_max_pages * page_tokens at
 *              least budget or max_pages * page_tokens, whichever is less.  No page
 *              in it may appear in page_table or twice (pages of page_table may be shared:
 *              they are only read, and the caller frees them afterwards)
 *   kept       device int32 [B, H, budget]: the old place of each kept token,
 *              ascending; entries from K on keep what they held
 *   new_lens   device int32 [B]: K; must not overlap kv_lens
 *
 * The cache's codes and scales are read in the old pages and written in the new
 * ones.  max_pages * page_tokens is below 2^31; a table wider than the sequences costs up
 * to a fourth more (64 histories cut to 2048 tokens 112 us, with a table of twice the longest
 * one's width 138).  Asynchronous on `stream`, no allocation, no workspace, no host
 * read of device data (may be captured).  A sequence whose
 * length does not fit the table is skipped, with new_lens 0; tokens on an old page
 * out of range count as NaN and leave the new slot as it was, as does a new page
 * out of range; gdpa_device_status() then returns GDPA_ERR_INVALID_ARG.
 */
gdpa_status_t gdpa_cache_evict(const gdpa_cache_t* cache, float* weights, const int32_t* kv_lens,
                               const int32_t* page_table, int B, int max_pages, int budget, int sink, int recent,
                               const int32_t* new_table, int new_max_pages, int32_t* kept, int32_t* new_lens,
                               void* stream);

/* Human-readable name of a status code (static string). */
const char* gdpa_status_string(int status);

/* Library version, e.g. "gdpa 0.1 sm_103a". */
const char* gdpa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GDPA_H_ */
