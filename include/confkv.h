/*
 * confkv.h — C ABI of the B200 CONF-KV decode-step library (libconfkv.so).
 *
 * CONF-KV ("Conf-KV: confidence-aware KV-cache eviction with mixed ..."
 * rcap.io post, and the chatpaper.ai abstract "CONF-KV: Confidence-Aware KV
 * Cache Eviction with Mixed-Precision Storage for Long-Horizon LLMs") is a
 * KV-cache manager: every decode step it turns the next-token distribution
 * into a confidence score, picks a token budget from it, keeps the tokens with
 * the highest blend of attention-mass EMA and recency inside that budget
 * (never the most recent P), stores older tokens in INT8 and the recent window
 * in FP16, and keeps the cache contiguous. The same select also runs the
 * fixed-budget B = s + w + k mode of the KVpop summary (gist.science,
 * sections 2.1 and 2.4): sinks + protected window + top-k static priorities.
 *
 * One decode step, in the order of the CONF-KV post's decode-loop pseudo-code:
 *   confkv_decode_attn   (append the new token, attention, attention-mass EMA)
 *   confkv_confidence    (confidence of the step's logits -> budget per layer)
 *   confkv_evict_compact (select victims, compact, convert the token leaving
 *                         the FP16 window to INT8)
 *
 * Conventions shared by every entry point:
 *  - Pointers named *_host are host memory; every other array pointer is
 *    device memory of the current CUDA device, owned by the caller, never
 *    freed or retained by the library after the call's work completes.
 *  - fp16 arrays are IEEE binary16 passed as `const void*`; fp32 as float.
 *    K/V/q/out arrays must start on a 16-byte boundary (ERR_ARG otherwise).
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *    stream). Every call is asynchronous on that stream unless documented as
 *    synchronising. One handle must not be used from two streams at once: the
 *    cache and the scratch belong to the handle. The library's kernels are
 *    launched with programmatic stream serialisation: each starts by waiting
 *    for the work before it on the stream to complete, so the next one's
 *    launch overlaps its end; work of the caller in between is ordered as
 *    usual.
 *  - Errors the host can detect (bad arguments, capacity, wrong state) are
 *    returned before anything is launched, and the call has no effect.
 *    Conditions only the device can see (non-finite logits, a failed device
 *    check) set a sticky device error word read by confkv_last_error.
 *  - No call traps, asserts on the device, or throws across the ABI.
 */
#ifndef CONFKV_H
#define CONFKV_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define CONFKV_API __attribute__((visibility("default")))
#else
#define CONFKV_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef struct confkv_handle confkv_handle;

typedef enum {
  CONFKV_OK = 0,
  CONFKV_ERR_ARG = 1,        /* invalid argument (null pointer, out of range, inconsistent) */
  CONFKV_ERR_CAPACITY = 2,   /* the call could exceed the cache capacity sized at create */
  CONFKV_ERR_STATE = 3,      /* wrong call order (e.g. decode before prefill) or destroyed handle */
  CONFKV_ERR_NONFINITE = 4,  /* device word: a logit row held NaN/Inf (that row used the larger budget) */
  CONFKV_ERR_CUDA = 5,       /* a CUDA runtime call failed */
  CONFKV_ERR_OOM = 6,        /* device allocation failed at create */
  CONFKV_ERR_DEVICE = 7      /* device word: a kernel's own bounds check fired (work skipped) */
} confkv_status;

enum { CONFKV_MODE_CONF = 0, CONFKV_MODE_FIXED = 1 };
/* Budget gate polarity. PROSE (default): confident (c >= tau) -> n_low, else
 * n_high, as the CONF-KV abstract and post describe. LITERAL: the
 * pseudo-code line's polarity, n_high when c >= tau. */
enum { CONFKV_GATE_PROSE = 0, CONFKV_GATE_LITERAL = 1 };
/* Compaction variant and window layout; all give the same logical cache
 * content (the tokens, their precision, payload, scales and EMA):
 *   HOLEFILL  survivors above the new end of the INT8 region move into the
 *             holes below it (bytes in proportion to the victims); the FP16
 *             window is a ring, slot = position mod W;
 *   STABLE    order-preserving compaction of the INT8 region (every survivor
 *             after the first hole moves down); the window is a ring;
 *   LINEAR    no ring: the INT8 region is compacted in order and the FP16
 *             window occupies slots [0, n) in position order, so the whole
 *             cache is position-ordered; every conversion or window eviction
 *             moves the window's later slots down. Confidence mode with INT8
 *             on only. */
enum { CONFKV_COMPACT_HOLEFILL = 0, CONFKV_COMPACT_STABLE = 1, CONFKV_COMPACT_LINEAR = 2 };
/* Score source of the confidence mode's ranking (score = alpha*source +
 * (1-alpha)*recency):
 *   EMA    ema <- beta*ema + (1-beta)*a (the CONF-KV post's EMA; the default);
 *   ACCUM  acc <- acc + a, the attention mass accumulated over the steps (the
 *          heavy-hitter score the CONF-KV post's related work, H2O, uses);
 *   RANDOM a static per-token draw u in [0, 1), from SplitMix64 (Steele, Lea
 *          and Flood, 2014) at counter pos | h << 32 | b << 40 | l << 52
 *          (position, KV head, sequence, layer): state seed + (counter + 1) *
 *          0x9E3779B97F4A7C15, mixed, u = (mix >> 40) * 2^-24.
 * a is the token's attention probability this step, averaged over the G query
 * heads. These are the ranker variants of the matched-rate ablation. */
enum { CONFKV_SCORE_EMA = 0, CONFKV_SCORE_ACCUM = 1, CONFKV_SCORE_RANDOM = 2 };

#define CONFKV_ALL_LAYERS (-1)

typedef struct {
  int32_t mode;          /* CONFKV_MODE_CONF or CONFKV_MODE_FIXED */
  int32_t n_low;         /* tight budget (tokens per KV head), >= 1 */
  int32_t n_high;        /* loose budget, >= 1 */
  float tau;             /* confidence threshold, compared with >= */
  float alpha;           /* score = alpha*EMA + (1-alpha)*recency, in [0, 1] */
  float ema_decay;       /* beta in ema <- beta*ema + (1-beta)*a, in [0, 1] */
  int32_t protect_last;  /* P: tokens with age t-pos < P are never evicted (fixed mode: w) */
  int32_t fp16_window;   /* W: tokens with age < W are FP16 while attention runs; >= 1 when int8_enable */
  int32_t n_sink;        /* s: positions < s are never evicted */
  int32_t fixed_budget;  /* B = s + w + k (fixed mode only), >= s + w */
  int32_t pyramidal;     /* nonzero: layer l gets floor(N(4(L-1)-3l)/(2(L-1))) */
  int32_t gate;          /* CONFKV_GATE_PROSE or CONFKV_GATE_LITERAL */
  int32_t int8_enable;   /* nonzero: tokens older than the window are stored INT8 */
  int32_t compact;       /* CONFKV_COMPACT_HOLEFILL or CONFKV_COMPACT_STABLE */
  int32_t max_batch;     /* sequences the cache is sized for */
  int32_t max_prefill;   /* longest prompt confkv_prefill accepts (tokens) */
  int32_t score_source;  /* CONFKV_SCORE_EMA, CONFKV_SCORE_ACCUM or CONFKV_SCORE_RANDOM (confidence mode) */
  uint32_t seed;         /* CONFKV_SCORE_RANDOM: seed of the per-token draws */
  int32_t single_stream; /* nonzero: every kernel of a call runs inside that call, on the caller's
                            stream (the EMA pass runs in confkv_decode_attn instead of being deferred
                            to the next eviction, and no event joins calls), so that a caller can
                            capture a whole decode step in a CUDA graph. Launch configurations are
                            then fixed at capture time, and the handle's host-side length bounds are
                            not advanced by replays */
} confkv_params;

typedef struct {
  int64_t tokens_int8;        /* tokens stored INT8, all segments */
  int64_t tokens_fp16;        /* tokens stored FP16, all segments */
  int64_t bytes_payload;      /* K/V payload bytes + INT8 scales resident (all segments) */
  int64_t bytes_meta;         /* position + EMA/priority bytes resident */
  int64_t bytes_capacity;     /* device bytes the handle allocated */
  int32_t min_len, max_len;   /* over the active segments */
  int64_t attn_tokens_int8;   /* cumulative INT8 token-rows read by decode attention (per KV head) */
  int64_t attn_tokens_fp16;   /* cumulative FP16 token-rows read by decode attention (per KV head) */
  int64_t evict_tokens;       /* cumulative tokens scanned by eviction */
  int64_t moved_rows;         /* cumulative rows moved by compaction */
  int64_t requant_rows;       /* cumulative tokens converted FP16 -> INT8 */
  int64_t kernel_launches;    /* cumulative kernels launched by this handle */
  int64_t evict_block_segments; /* cumulative segments evicted by the whole-CTA path (many victims) */
  int64_t moved_window_rows;  /* cumulative FP16 window rows moved (the linear layout's window shifts) */
} confkv_stats;

/* Fill *p with the defaults: CONF mode, N_low 256, N_high 512, tau 0.6,
 * alpha 0.5, beta 0.9, P 64, W 128, s 0, prose gate, INT8 on, hole-fill
 * compaction, max_batch 1, max_prefill 4096. Returns CONFKV_ERR_ARG if p is
 * NULL. */
CONFKV_API confkv_status confkv_default_params(confkv_params* p);

/* Allocate a cache for `layers` layers of `kv_heads` KV heads of head_dim
 * (64 or 128) each, for up to params->max_batch sequences, with q_heads query
 * heads (a multiple of kv_heads, at most 8 per KV head). All device memory is
 * allocated here, on the current device; nothing allocates later. *out
 * receives the handle. Errors: ARG (invalid shape or parameter), OOM, CUDA. */
CONFKV_API confkv_status confkv_create(int32_t layers, int32_t kv_heads, int32_t q_heads, int32_t head_dim,
                            const confkv_params* params, confkv_handle** out);

/* Free everything the handle owns (synchronises the device first). A NULL
 * handle is a no-op returning OK. The handle must not be used afterwards. */
CONFKV_API confkv_status confkv_destroy(confkv_handle* h);

/* Ingest prompts and reset the cache of `layer` (or every layer with
 * CONFKV_ALL_LAYERS) for `batch` sequences (1..max_batch).
 *   lens_host[batch]  prompt length per sequence, 0..max_prefill (host)
 *   k, v   fp16 [batch][kv_heads][t_stride][head_dim] for one layer, or with a
 *          leading [layers] dimension for CONFKV_ALL_LAYERS; rows >= len unused
 *   priority  fp32 [batch][kv_heads][t_stride] (leading [layers] likewise);
 *          required in fixed mode, must be NULL otherwise
 * Confidence mode evicts nothing here. Fixed mode keeps the s sinks, the last
 * w and the top k by (priority, position) as it ingests (KVpop summary 2.1).
 * With INT8 on, positions <= len - W are quantised (per token, per KV head,
 * K and V separately, round-half-even). Positions restart at 0. The batch
 * size given here is the active batch of later calls. */
CONFKV_API confkv_status confkv_prefill(confkv_handle* h, int32_t layer, int32_t batch, const int32_t* lens_host,
                             int32_t t_stride, const void* k, const void* v, const float* priority,
                             void* stream);

/* Confidence of each sequence's next-token distribution and its budget
 * (CONF-KV post, pseudo-code and method paragraphs):
 *   c = 0.4(1 - H(p)/ln V) + 0.3 sigmoid(l_(1) - l_(2)) + 0.3 max p,
 *   p = softmax(logits), H in nats, l_(1) >= l_(2) the two largest logits
 *   counted with multiplicity.
 * logits fp32 [batch][vocab] (batch = the active batch, vocab >= 2). The
 * budget N per sequence follows the gate polarity, then the pyramid; the
 * handle keeps budget[batch][layers] for confkv_evict_compact. c_out fp32
 * [batch] and budget_out int32 [batch][layers] are optional (NULL skips). A
 * row with a NaN/Inf logit gets c = NaN and the larger budget, and sets the
 * device word CONFKV_ERR_NONFINITE. Not used in fixed mode (returns STATE). */
CONFKV_API confkv_status confkv_confidence(confkv_handle* h, const float* logits, int32_t batch, int32_t vocab,
                                float* c_out, int32_t* budget_out, void* stream);

/* One decode step's attention for `layer` (or CONFKV_ALL_LAYERS):
 * append the new token at the next position of every segment (FP16), then
 * softmax attention of the G = q_heads/kv_heads query heads of each KV head
 * over its whole cache (scale 1/sqrt(head_dim), INT8 rows dequantised
 * in-kernel), then, in confidence mode, the attention-mass EMA update of every
 * cached token: ema <- beta*ema + (1-beta)*mean over the G heads of its
 * normalised attention probability (new tokens start at 0).
 *   q      fp16 [batch][q_heads][head_dim]   (leading [layers] for ALL)
 *   k_new, v_new  fp16 [batch][kv_heads][head_dim]  (likewise)
 *   prio_new  fp32 [batch][kv_heads] (likewise); fixed mode only, else NULL
 *   out    fp32 [batch][q_heads][head_dim]   (likewise)
 *   lse_out  fp32 [batch][q_heads] (likewise) natural-log log-sum-exp of the
 *          scaled scores; optional
 * Query head h reads KV head h / G. Errors: STATE before prefill, CAPACITY if
 * the cache could overflow (calls without eviction grow it).
 * Unless single_stream is set, the EMA update is deferred: the next
 * confkv_evict_compact over the same layers runs it inside the eviction kernel
 * (one launch for both). Whatever reads the cache first -- another decode call
 * over those layers, confkv_query, confkv_export_segment -- sees it applied;
 * a prefill of those layers discards it. */
CONFKV_API confkv_status confkv_decode_attn(confkv_handle* h, int32_t layer, const void* q, const void* k_new,
                                 const void* v_new, const float* prio_new, float* out, float* lse_out,
                                 void* stream);

/* Attention of several drafted tokens per sequence, the nodes of a tree, over
 * the cache and over one another: the step that checks a draft. The cache is
 * read only; confkv_append adds the nodes that were accepted.
 *   nodes  rows of the draft buffers per sequence, 1..CONFKV_MAX_NODES
 *   q      fp16 [batch][nodes][q_heads][head_dim]   (leading [layers] for ALL)
 *   k, v   fp16 [batch][nodes][kv_heads][head_dim]  (likewise)
 *   mask   uint64 [batch][nodes], one for all layers and heads: bit j of node
 *          i's word set means that node i attends to node j (usually its
 *          ancestors and itself). Every node attends to the whole cache. Bits
 *          of nodes past the sequence's count are ignored
 *   counts int32 [batch], device, optional: nodes of each sequence, 0..nodes
 *          (NULL: nodes). Rows past a count are not read as keys or values,
 *          and their outputs are left as they were. A count out of range is
 *          taken as 0 and sets the device word (ERR_DEVICE)
 *   out    fp16 [batch][nodes][q_heads][head_dim]   (likewise)
 *   lse_out  fp32 [batch][nodes][q_heads] (likewise), optional, as in
 *          confkv_decode_attn
 *   track  nonzero: the attention of node 0 (the root, which is always
 *          accepted) updates the attention mass of the cached tokens as
 *          confkv_decode_attn does with its token's; a sequence without nodes
 *          gives mass 0. Confidence mode only (ARG in fixed mode)
 * A node that attends to nothing (an empty cache and an empty mask) gets out 0
 * and lse -inf. Scores and sums are fp32. The weights of the second product
 * (relative to the largest, and times the V scale for INT8 rows) keep 22 bits, down
 * to steps of 2^-31 max(1, the largest V scale of the cache): beside a V row 2^20
 * times the others, at a scale of 1, those keep 11 bits. The output's rounding to
 * fp16 is the only other one below fp32. Keys and values of a node reach only the
 * nodes that attend to it, whatever they are (NaN, inf).
 * Errors: STATE before prefill or with another device current. */
enum { CONFKV_MAX_NODES = 64 };
CONFKV_API confkv_status confkv_tree_attn(confkv_handle* h, int32_t layer, int32_t nodes, const void* q, const void* k,
                                          const void* v, const uint64_t* mask, const int32_t* counts, void* out,
                                          float* lse_out, int32_t track, void* stream);

/* Append several tokens to every sequence of `layer` (or CONFKV_ALL_LAYERS)
 * without attention: the accepted path of a tree. They take the next
 * positions, FP16, with score source 0 (or their draw, or their priority);
 * tokens that leave the FP16 window are converted to INT8 as in
 * confkv_decode_attn. The following confkv_evict_compact brings the cache back
 * to its budget.
 *   tokens most tokens per sequence, at least 1
 *   rows   rows of k and v per sequence
 *   k, v   fp16 [batch][rows][kv_heads][head_dim]  (leading [layers] for ALL)
 *   prio   fp32 [batch][rows][kv_heads] (likewise); fixed mode only, else NULL
 *   index  int32 [batch][tokens], device, optional: the row of each token
 *          (NULL: 0, 1, ...; then tokens must not exceed rows)
 *   counts int32 [batch], device, optional: tokens of each sequence, 0..tokens
 *          (NULL: tokens)
 * A count or row out of range, or a list that a full cache has no room for (in
 * replays of a captured call), sets the device word (ERR_DEVICE) and that
 * sequence gets none of its tokens. CAPACITY if `tokens` more could overflow
 * the cache: in confidence mode size max_prefill for the longest draft beyond
 * the budget; a fixed-budget cache has room for CONFKV_MAX_NODES beyond its own. */
CONFKV_API confkv_status confkv_append(confkv_handle* h, int32_t layer, int32_t tokens, int32_t rows, const void* k,
                                       const void* v, const float* prio, const int32_t* index, const int32_t* counts,
                                       void* stream);

/* Evict and compact `layer` (or CONFKV_ALL_LAYERS): for every segment over its
 * effective budget max(budget_l, P + s) (fixed mode: B), evict the
 * lowest-ranked unprotected tokens by the key (score, position), score =
 * fp32(fp32(alpha*ema) + fp32((1-alpha)*recency)), recency =
 * (pos+1)/(t+1) (fixed mode: the priority), equal scores keeping the newer
 * token; tokens with age < P and positions < s are never evicted. Survivors
 * are compacted so the INT8 region stays a hole-free prefix, and the token
 * the next append would push out of the FP16 window is quantised to INT8
 * (CONF-KV post, pseudo-code). Called on the stream of the handle's last
 * confkv_confidence, right after it, the deferred EMA pass runs beside that
 * confidence reduction and only the eviction waits for its budgets. */
CONFKV_API confkv_status confkv_evict_compact(confkv_handle* h, int32_t layer, void* stream);

/* Synchronising: counts of the active segments and cumulative counters. */
CONFKV_API confkv_status confkv_query(confkv_handle* h, confkv_stats* out);

/* Synchronising: copy the raw state of one segment (layer, seq, kv_head) to
 * host memory. With host_buf NULL, *bytes receives the size needed. Layout
 * (all little-endian, packed in this order):
 *   int32 header[8] = { n_cold, ring_slots, next_pos, cold_int8, head_dim,
 *                       mode, 0, 0 }
 *   cold region, n_cold rows in physical order:
 *     int32 pos[n_cold]; float score_src[n_cold]; float ks[n_cold]; float vs[n_cold];
 *     K rows [n_cold][head_dim] (int8 if cold_int8 else fp16); V rows likewise
 *   ring, ring_slots rows (slot order; pos < 0 marks an empty slot):
 *     int32 pos[W]; float score_src[W]; fp16 K[W][head_dim]; fp16 V[W][head_dim]
 * score_src is the EMA (confidence mode) or the priority (fixed mode). */
CONFKV_API confkv_status confkv_export_segment(confkv_handle* h, int32_t layer, int32_t seq, int32_t kv_head,
                                    void* host_buf, size_t* bytes);

/* Synchronising: the sticky device error word (CONFKV_OK if none); with
 * clear nonzero it is reset. */
CONFKV_API confkv_status confkv_last_error(confkv_handle* h, int32_t clear);

/* Synchronising: like confkv_last_error (not clearing), and when a device-side
 * check failed, detail[3] receives (check site, segment id, offending value)
 * of the first failure. Sites: 1xx append, 2xx attention, 3xx EMA, 4xx
 * eviction, 5xx prefill, 6xx combine; the work guarded by a failed check is
 * skipped, never performed out of bounds. */
CONFKV_API confkv_status confkv_last_error_detail(confkv_handle* h, int32_t* detail);

/* Per-kernel timing. While enabled, every kernel launch of the handle is
 * bracketed by CUDA events on its stream (a few microseconds of host work per
 * launch, nothing on the device). confkv_profile_read synchronises on the
 * recorded events and returns, per kernel kind, the launches and the summed
 * milliseconds since the last reset. */
enum {
  CONFKV_K_CONFIDENCE = 0, CONFKV_K_APPEND = 1, CONFKV_K_ATTENTION = 2, CONFKV_K_COMBINE = 3,
  CONFKV_K_EMA = 4, CONFKV_K_EVICT = 5, CONFKV_K_PREFILL = 6,
  CONFKV_K_EMA_EVICT = 7,   /* the eviction kernel with the step's EMA pass fused in */
  CONFKV_K_KINDS = 8
};
typedef struct {
  int64_t launches[CONFKV_K_KINDS];
  double ms[CONFKV_K_KINDS];
} confkv_profile;
CONFKV_API confkv_status confkv_profile_enable(confkv_handle* h, int32_t enable);
CONFKV_API confkv_status confkv_profile_read(confkv_handle* h, confkv_profile* out, int32_t reset);

/* Confidence and per-layer budgets without a handle and without allocating.
 * The pages describe no counterpart: this entry point exists for callers that
 * cannot allocate device memory, such as code running under an allocator
 * that owns the whole device or a runtime that hands the library a fixed
 * memory budget. It computes what confkv_confidence computes, for the gate,
 * threshold, budgets and pyramid in *params (its other fields are ignored),
 * for `layers` layers:
 *   logits fp32 [batch][vocab], c_out fp32 [batch], budget_out int32
 *   [batch][layers], all device memory owned by the caller (required).
 * Its scratch is a fixed array inside the library (about 197 KB per device,
 * held by every GPU that loads the library until the process exits), so:
 *  - batch may be at most 256 and vocab at most 262144; larger sizes return
 *    CONFKV_ERR_CAPACITY before anything runs;
 *  - the first call on a device looks up the array's device address (a
 *    host-side step, no allocation) and keeps it for the life of the process;
 *    make that first call before any stream capture. A device reset
 *    (cudaDeviceReset, or a reset of the primary context) reloads the library
 *    on that device and leaves the kept address stale: do not call this entry
 *    point on a device after resetting it;
 *  - every call shares the one array: calls that overlap on the GPU (on two
 *    streams, or from two threads) race and give wrong results. Serialise them.
 * It calls no cudaMalloc, cudaFree or allocating routine. A row with a NaN or
 * Inf logit gets c = NaN and the larger budget; no error word is kept. */
CONFKV_API confkv_status confkv_confidence_noalloc(const confkv_params* params, int32_t layers, const float* logits,
                                                   int32_t batch, int32_t vocab, float* c_out, int32_t* budget_out,
                                                   void* stream);

/* Element types of the entry points that take more than one. */
enum { CONFKV_F32 = 0, CONFKV_F16 = 1, CONFKV_BF16 = 2 };

/* ---------------------------------------------------------------------------
 * Rotary positions of queries and keys, optionally after a norm of each head:
 * what stands between a model's projections and confkv_prefill,
 * confkv_decode_attn or confkv_tree_attn. No handle and no device allocation.
 *
 *   y = R(w * x / sqrt(mean(x^2) + eps)),
 *
 * where R turns pair i of the first rotary_dim dimensions by the angle
 * position * f_i and copies the other dimensions; without a weight the norm is
 * left out. Pairs are (i, i + rotary_dim/2) in the HALF layout, (2i, 2i+1) in
 * the INTERLEAVED one. f_i = theta^(-2i/rotary_dim), scaled for contexts
 * longer than the trained one by
 *   LINEAR  f_i / factor;
 *   NTK     theta * factor^(rotary_dim / (rotary_dim - 2)) in theta's place;
 *   BANDED  by the turns n_i = original_length f_i / 2 pi: f_i from high_band
 *           turns on, f_i / factor up to low_band, and between them the blend
 *           linear in n_i;
 *   YARN    (Peng et al., 2023) the blend linear in i between the pairs that
 *           make beta_fast and beta_slow turns within original_length (rounded
 *           outwards, kept in [0, rotary_dim - 1]); the rotated dimensions are
 *           multiplied by 0.1 ln(factor) + 1, or by `magnitude` where it is
 *           above 0 (which holds for every scaling).
 * ------------------------------------------------------------------------- */
enum { CONFKV_ROPE_HALF = 0, CONFKV_ROPE_INTERLEAVED = 1 };
enum { CONFKV_ROPE_PLAIN = 0, CONFKV_ROPE_LINEAR = 1, CONFKV_ROPE_NTK = 2, CONFKV_ROPE_BANDED = 3,
       CONFKV_ROPE_YARN = 4 };
enum { CONFKV_ROPE_MAX_PAIRS = 128 };

typedef struct {
  int32_t head_dim;         /* even, 2..256 */
  int32_t rotary_dim;       /* even, 0..head_dim */
  int32_t layout;           /* CONFKV_ROPE_HALF or CONFKV_ROPE_INTERLEAVED */
  int32_t scaling;          /* CONFKV_ROPE_PLAIN .. CONFKV_ROPE_YARN */
  double theta;             /* above 1 */
  double factor;            /* every scaling but PLAIN; at least 1 */
  double low_band, high_band;    /* BANDED */
  double beta_fast, beta_slow;   /* YARN */
  double magnitude;         /* 0: the scaling's own */
  int32_t original_length;  /* BANDED and YARN */
} confkv_rope_params;

/* The prepared frequencies: plain host data that the caller keeps (one per
 * model) and may copy. turns[i] is the fraction of a turn that pair i makes a
 * position, in units of 2^-64. */
typedef struct {
  int32_t head_dim, rotary_dim, layout;
  float magnitude;
  uint64_t turns[CONFKV_ROPE_MAX_PAIRS];
} confkv_rope_table;

/* The rows of one side (queries, or keys): [batch][tokens][heads][head_dim]
 * with the last dimension contiguous and the other strides given in elements
 * (not negative; that of a dimension of size 1 is not looked at; a column block of
 * a packed projection, or a [batch][heads][tokens][head_dim] buffer, are such rows). Rows of y lie apart:
 * in the order of their strides, each dimension steps over all that the ones
 * before it span (ARG otherwise). y may be x itself with the same type and
 * strides; any other overlap, of the two sides' y among them, is not allowed. */
typedef struct {
  const void* x;
  void* y;
  const float* weight;      /* fp32 [head_dim], or NULL: no norm */
  int32_t heads;
  int64_t x_batch, x_token, x_head;
  int64_t y_batch, y_token, y_head;
} confkv_rope_rows;

/* Defaults: head_dim and rotary_dim 128, half layout, PLAIN, theta 10000,
 * factor 1, bands 1 and 4, betas 32 and 1, original_length 8192. */
CONFKV_API confkv_status confkv_default_rope_params(confkv_rope_params* p);

/* Host only: turn parameters into a table. ARG for values out of range. */
CONFKV_API confkv_status confkv_rope_prepare(const confkv_rope_params* params, confkv_rope_table* out);

/* Norm and rotate q and (unless NULL) k.
 *   positions  int32 [batch][tokens], device; any value (a negative position
 *              turns backwards)
 *   x_type, y_type  CONFKV_F32, CONFKV_F16 or CONFKV_BF16, the same for q and k
 * Arithmetic is fp32. Angles are right to 2^-26 of a turn, and |position| * 2^-55
 * of one for the frequencies, which are prepared in fp64. The output type's
 * rounding is the only one below fp32. batch or tokens of 0 does nothing. */
CONFKV_API confkv_status confkv_rope(const confkv_rope_table* table, int32_t batch, int32_t tokens,
                                     const int32_t* positions, int32_t x_type, int32_t y_type, float eps,
                                     const confkv_rope_rows* q, const confkv_rope_rows* k, void* stream);

/* ---------------------------------------------------------------------------
 * Sampling of the next token from the logits that confkv_confidence reads, with
 * the random numbers given by the caller. No handle and no device allocation.
 * ------------------------------------------------------------------------- */

/* Draw one token per row. With w_i = exp((x_i - max x) / T) and the tokens of a
 * row ordered by descending logit (equal logits: the lower index first), the
 * tokens kept are those
 *   - among the first top_k,
 *   - before which, among those, less than top_p of their weight lies,
 *   - with x_i >= max x + T ln(min_p);
 * token_out is the first of them, by index, at which the running sum of their
 * weights exceeds u times the total, prob_out its share of the total.
 *   logits  [rows] rows of `vocab` values of `type`, row_stride elements apart
 *           (at least vocab); -inf marks a token that is never drawn
 *   u       fp32 [rows], in [0, 1)
 *   temperature  fp32 [rows] (NULL: 1); below 2^-60, 0 among them: the largest logit,
 *           the lowest index among equals
 *   top_k   int32 [rows] (NULL: off); 0 or less, or at least the tokens there are: off
 *   top_p   fp32 [rows] (NULL: off); 1 or more: off; 0 or less: the first token only
 *   min_p   fp32 [rows] (NULL: off); 0 or less: off; above 1: taken as 1
 *   token_out  int32 [rows];  prob_out  fp32 [rows], optional
 * A row with a NaN or +inf logit, without a logit above -inf, or with a NaN
 * parameter, a negative or infinite temperature, or u outside [0, 1), gets
 * token -1 and probability 0. Weights are fp32: off by about 2^-22 of their value, and by
 * 2^-24 |x_i - max x| / T of it where that difference of two fp32 logits is not exact. Their sums
 * are fp64 over fours added in fp32, or integers: for the top_p cut of 2^-30 of each weight's own
 * magnitude and 2^-32 of the largest weight over the whole row, over up to 2048 gathered tokens
 * of 2^-40 of the largest. None depends on timing: a call repeated gives the same bits.
 * CAPACITY: vocab above 1048576, or rows above 2^27. rows of 0 does nothing. */
CONFKV_API confkv_status confkv_sample(int32_t type, const void* logits, int64_t row_stride, int32_t rows,
                                       int32_t vocab, const float* u, const float* temperature, const int32_t* top_k,
                                       const float* top_p, const float* min_p, int32_t* token_out, float* prob_out,
                                       void* stream);

/* Static description of a status code. */
CONFKV_API const char* confkv_status_string(confkv_status s);

/* Library version as MAJOR*10000 + MINOR*100 + PATCH. */
CONFKV_API int32_t confkv_version(void);

#ifdef __cplusplus
}
#endif
#endif /* CONFKV_H */
