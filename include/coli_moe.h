/*
 * coli_moe.h -- C ABI of the routed-expert MoE layer on NVIDIA B200 (sm_100a).
 *
 * The layer (colibri-strix README, "What's implemented"): a sigmoid router in the DeepSeek-V3
 * manner, whose noaux_tc bias steers the selection and whose weights are renormalised and scaled
 * by routed_scaling_factor; batch-union grouping, in which every expert that some token of the
 * batch selects is fetched one time and serves all of those tokens; SwiGLU experts stored as
 * packed int4 (also int8 / packed int2) with per-row scales, dequantised on use; a shared
 * expert; and the weighted combine.  The JustVugg/colibri README ("Never wait for the disk
 * twice") keeps an expert's gate, up and down matrices together in one record.
 *
 * Conventions shared by every call
 *   - All tensor pointers are DEVICE pointers owned by the caller.  The library allocates no
 *     device memory; scratch comes from a caller-provided workspace (coli_moe_workspace_size).
 *   - Every compute call is asynchronous on `stream` (a cudaStream_t passed as void*; NULL is
 *     the legacy default stream).  Host-side validation happens before any launch; a non-OK
 *     status means nothing was launched.
 *   - Device-side anomalies (an expert id out of range, inconsistent grouping arrays) never
 *     trap: the kernel skips the bad item and records a code in the workspace's error word,
 *     which coli_moe_error_word() reads back.
 *   - There is no CPU fallback: every step runs in this library's CUDA kernels.
 *
 * Record format (one per expert; the same for the shared expert with its own inter size)
 *   Wg codes [I][H] | Wu codes [I][H] | Wd codes [H][I] | sg | su | sd (float32 scales),
 *   rows packed to whole bytes: int4 element 2j in the low nibble of byte j and 2j+1 in the
 *   high nibble (two's complement, [-8,7]); int2 element 4j+k in bits [2k,2k+1] of byte j
 *   ([-2,1]); int8 one signed byte.  Per-row container (group_size 0): sg[I], su[I], sd[H], the
 *   weight is code * scale of its output row.  Group-scaled container (group_size 64, int4 only;
 *   the JustVugg/colibri README, "Get started -> 2. Get the model", recommends this GLM-5.2
 *   build): sg[I][H/64], su[I][H/64], sd[H][I/64], the weight is code * scale of its group of 64
 *   consecutive columns of the row.  Records sit `expert_stride` bytes apart (a multiple of
 *   256) and the record base must be 256-byte aligned.
 *
 *   Microscaled 4-bit containers (COLI_W_NVFP4, COLI_W_MXFP4; group_size 0): W1 codes [2 I][H] | Wd
 *   codes [H][I] | scale tiles of W1 | scale tiles of Wd | with COLI_W_NVFP4 the float32 row scales
 *   of W1 [2 I] and of Wd [H].  W1 holds 16 gate rows, the same 16 up rows, the next 16 gate rows and so on
 *   (row 32 j + i is gate row 16 j + i, row 32 j + 16 + i up row 16 j + i, i < 16).  Codes, scales and tiles
 *   as the microscaled 4-bit section below has them; coli_moe_fp4_pack_record writes a record.  With
 *   these containers the layer quantises its activations too: x of every token, and h = SiLU(g) * u
 *   rounded to bf16, as coli_moe_fp4_quantize does; y is rounded to bf16 before the combine, whose
 *   order is fixed.  coli_moe_layer routes by coli_moe_route_scores (sigmoid, groups by two, renormalised).
 *
 * Tensor layouts (row-major):
 *   x        [T][H]   float32 (act = COLI_ACT_F32) or bfloat16 bits (COLI_ACT_BF16), 16-B aligned
 *   logits   [T][E]   float32
 *   topk_ids [T][K]   int32, slot order = descending biased score (ties: lower expert id)
 *   topk_w   [T][K]   float32
 *   out      [T][H]   float32, 16-B aligned
 */
#ifndef COLI_MOE_H
#define COLI_MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    COLI_OK = 0,
    COLI_ERR_INVALID_ARG = 1,  /* NULL pointer, negative size, bad enum value */
    COLI_ERR_SHAPE = 2,        /* sizes inconsistent with each other or with the formats */
    COLI_ERR_ALIGN = 3,        /* a pointer or stride misses its required alignment */
    COLI_ERR_UNSUPPORTED = 4,  /* a valid configuration that this library does not implement */
    COLI_ERR_CUDA = 5,         /* a CUDA runtime call failed (launch, attribute, copy) */
    COLI_ERR_DEVICE = 6,       /* the device error word was set by a kernel */
    COLI_ERR_WORKSPACE = 7     /* workspace NULL, misaligned or smaller than required */
} coli_status;

typedef enum {
    COLI_W_INT2 = 2,
    COLI_W_INT4 = 4,
    COLI_W_INT8 = 8,
    COLI_W_NVFP4 = 20,  /* e2m1, an e4m3 scale per 16 (COLI_FP4_NV below) */
    COLI_W_MXFP4 = 36   /* e2m1, a power-of-two scale per 32 (COLI_FP4_MX below) */
} coli_wfmt;
typedef enum { COLI_ACT_F32 = 0, COLI_ACT_BF16 = 1 } coli_act;

/* Device error word codes (bit flags, OR-ed together by the kernels). */
#define COLI_DEVERR_EXPERT_ID 0x1   /* an expert id or unique-list entry outside [0, E) */
#define COLI_DEVERR_GROUPING 0x2    /* offsets/perm inconsistent (slot outside [0, T*K)) */
#define COLI_DEVERR_TIMEOUT 0x4     /* a bounded device-side wait ran out (the call's output is invalid) */

typedef struct {
    int hidden;             /* H */
    int inter;              /* I, routed expert intermediate size */
    int n_experts;          /* E (<= 1024) */
    int top_k;              /* K (<= 32) */
    int n_group;            /* G; E % G == 0 */
    int topk_group;         /* TG, 1 <= TG <= G */
    int n_shared;           /* 0 or 1 */
    int shared_inter;       /* I_s; must equal inter when n_shared == 1 */
    double routed_scaling;  /* rsf */
    int wfmt;               /* coli_wfmt */
    int act;                /* coli_act */
    int group_size;         /* 0: one scale per weight row; 64: one per 64 columns (int4 only) */
} coli_moe_config;

typedef struct {
    const float *router_w;     /* [E][H] float32 */
    const float *router_bias;  /* [E] float32, the noaux_tc selection bias */
    const uint8_t *experts;    /* E records, expert_stride bytes apart, 256-B aligned */
    size_t expert_stride;      /* bytes; multiple of 256 and >= the record size */
    const uint8_t *shared;     /* the shared expert's record (NULL when n_shared == 0) */
} coli_moe_weights;

/* Text for a status code (static storage). */
const char *coli_moe_status_str(coli_status s);

/* Name and text of the CUDA error behind the calling thread's last COLI_ERR_CUDA ("" if none). */
const char *coli_moe_last_cuda_error(void);

/* Bytes of one record for (hidden, inter, wfmt, group_size), before padding to 256.  Host only. */
coli_status coli_moe_record_bytes(int hidden, int inter, int wfmt, int group_size, size_t *bytes);

/* Validates a configuration (the same checks every call makes).  Host only. */
coli_status coli_moe_check_config(const coli_moe_config *cfg);

/* Workspace bytes that coli_moe_layer / coli_moe_ffn / coli_moe_group need for up to
 * max_tokens tokens.  The workspace must be 256-byte aligned and is owned by the caller; calls
 * that share one workspace must be ordered on the GPU (same stream or events).  Its first 512
 * bytes (error word and the counters of the fused decode path) must be zero before its first
 * use: call coli_moe_clear_error once after allocating it (and after a call that reported
 * COLI_DEVERR_TIMEOUT).  Complete calls leave the header ready for the next call.  Host only. */
coli_status coli_moe_workspace_size(const coli_moe_config *cfg, int max_tokens, size_t *bytes);

/* Number of kernels coli_moe_layer launches for T tokens with this configuration (1 on the fused
 * decode path: one persistent kernel for the whole layer; 7 on the tensor-core path; 8 over records
 * in 4-bit containers; 5 otherwise).  Host only. */
coli_status coli_moe_layer_kernels(const coli_moe_config *cfg, int T, int *n_kernels);

/* Zeroes the workspace header: the device error word and the counters (asynchronous). */
coli_status coli_moe_clear_error(void *ws, void *stream);

/* Synchronises `stream` and returns the workspace's device error word in *code (0 = clean). */
coli_status coli_moe_error_word(void *ws, void *stream, int *code);

/* a1, router gate projection (colibri-strix README, "What's implemented": sigmoid router).
 * logits[t][e] = float32( sum_h x[t][h] * router_w[e][h] ), the products and the sum taken in
 * double precision, rounded once to float32.  T = 0 is a no-op; more than 65535 * 64 tokens are
 * COLI_ERR_UNSUPPORTED, here and in the layer. */
coli_status coli_moe_gate(const coli_moe_config *cfg, const float *router_w, const void *x,
                          int T, float *logits, void *stream);

/* a2, noaux_tc routing (colibri-strix README, "What's implemented": the DeepSeek-V3 sigmoid
 * router, its noaux_tc bias and routed_scaling_factor).  Per token, in double: s = 1/(1+exp(-logit)),
 * c = s + bias; if G > 1 each group scores the sum of its two largest c and the TG best groups
 * are kept (ties: lower group); the K largest c among kept experts are selected (ties: lower
 * id), written in descending c order; topk_w[k] = float32(s_k / sum_k s_k * routed_scaling).
 * The bias steers selection only.  T = 0 is a no-op. */
coli_status coli_moe_route(const coli_moe_config *cfg, const float *logits, const float *bias,
                           int T, int32_t *topk_ids, float *topk_w, void *stream);

/* a3, batch-union grouping (colibri-strix README, "What's implemented": batch-union MoE).
 * A stable counting sort of the T*K slots s = t*K + k by expert id: counts[E], offsets[E+1]
 * (exclusive scan, offsets[E] = T*K), perm[T*K] (slot indices grouped by expert, ascending
 * slot index inside each expert), unique_ids[E] (ids with counts > 0, ascending, the rest -1),
 * n_unique[1].  Ids outside [0,E) are skipped and flagged in the error word of `ws`. */
coli_status coli_moe_group(const coli_moe_config *cfg, const int32_t *topk_ids, int T,
                           int32_t *counts, int32_t *offsets, int32_t *perm,
                           int32_t *unique_ids, int32_t *n_unique, void *ws, size_t ws_bytes,
                           void *stream);

/* a4..a7 for a given routing (JustVugg/colibri README, "Never wait for the disk twice":
 * the experts a batch needs are fetched once for all of its positions; colibri-strix README,
 * "What's implemented":
 * dequant-on-use, shared expert).  For every unique expert e and every slot routed to it:
 * y = sd .* (Qd (SiLU(sg .* (Qg x)) .* (su .* (Qu x)))) with the codes Q dequantised in
 * registers; out[t] = sum over t's experts of topk_w * y + y_shared (weight 1).  The grouping
 * arrays are those coli_moe_group writes.  `out` is fully overwritten.  Each expert's weights
 * are streamed from HBM once per call. */
coli_status coli_moe_ffn(const coli_moe_config *cfg, const coli_moe_weights *w, const void *x,
                         int T, const float *topk_w, const int32_t *offsets,
                         const int32_t *perm, const int32_t *unique_ids,
                         const int32_t *n_unique, float *out, void *ws, size_t ws_bytes,
                         void *stream);

/* The whole layer: gate, route, group, ffn (all of the above, in that order, on `stream`).
 * topk_ids_out / topk_w_out may be NULL; when given they receive the routing.
 * The call issues no host-blocking operation and reads no device data on the host, so it may be
 * captured into a CUDA graph and replayed: the fused decode kernel keeps its counters in the
 * workspace header, and consecutive calls (or replays) on one workspace must be ordered on the
 * GPU, as calls on one stream are.  Replays read the pointers captured with the call. */
coli_status coli_moe_layer(const coli_moe_config *cfg, const coli_moe_weights *w,
                           const void *x, int T, float *out, int32_t *topk_ids_out,
                           float *topk_w_out, void *ws, size_t ws_bytes, void *stream);

/* Residual update between chained layers (JustVugg/colibri README, "Never wait for the disk
 * twice": the GPU-resident pipeline keeps the residual stream on the device across layers).
 * x_next[t][h] = x[t][h] + out[t][h] for t < T, h < hidden: one float32 addition (round to
 * nearest even); with bf16 activations (cfg->act) x and x_next are bf16 and the sum is rounded
 * to bf16 (round to nearest even, NaN kept), with float32 activations they are float32.
 *   x, x_next  [T][hidden] device, row-major, the activation type of cfg; x_next may be x (in
 *              place) but must not overlap out.
 *   out        [T][hidden] float32 device, a layer's output.
 * Pointers 16-byte aligned (COLI_ERR_ALIGN otherwise); T < 0 is COLI_ERR_SHAPE, T = 0 a no-op.
 * Asynchronous on `stream`; allocates nothing. */
coli_status coli_moe_residual(const coli_moe_config *cfg, const void *x, const float *out, int T,
                              void *x_next, void *stream);

/* a5' per-expert dispatch on the grouped tensor-core path (batches above 4 tokens): within a call,
 * work experts with at most max_tokens routed tokens are computed by the CUDA-core GEMV kernels
 * (streaming their codes once at HBM speed) and the others by the grouped GEMM; the GEMV kernels'
 * down projection adds into out alongside the GEMM's combine.  0 puts every expert on the tensor
 * cores.  Process-wide, read at each call; coli_moe_layer_kernels then reports 9 kernels on that
 * path instead of 7.  Host only; COLI_ERR_INVALID_ARG outside [0, 65536]. */
coli_status coli_moe_set_dispatch_threshold(int max_tokens);
int coli_moe_dispatch_threshold(void);

/* Testing aid for the bounded device-side waits of the fused decode kernel (the one-launch
 * path that coli_moe_layer_kernels reports as 1 kernel).  wait_cycles > 0 replaces the default
 * bound (about 2 s of SM clock) of every wait in that kernel's later launches made by the
 * calling thread; unreachable != 0 raises its grid-barrier targets beyond reach, so that every
 * such wait runs out: the call still completes, each wait ends within its bound, nothing traps,
 * the workspace's error word gets COLI_DEVERR_TIMEOUT and the outputs are invalid.  (0, 0)
 * restores the defaults.  Host only; COLI_ERR_INVALID_ARG for a negative bound. */
coli_status coli_moe_debug_set_wait(long long wait_cycles, int unreachable);

/* Size of the static scratch array behind coli_moe_layer_noalloc (8 MiB per GPU). */
#define COLI_MOE_STATIC_SCRATCH_BYTES (8u << 20)

/* The whole layer, like coli_moe_layer, for callers that cannot allocate device memory: a
 * plugin inside a serving engine whose GPU memory pool is fixed when the engine starts, or a
 * real-time loop that must never pay for cudaMalloc's device-wide synchronisation.  The pages
 * have no counterpart of this call; it exists for such callers only.
 *   - Allocates nothing.  The caller passes x, out and the optional routing outputs as for
 *     coli_moe_layer; every other byte the layer needs lives in one static device array of
 *     COLI_MOE_STATIC_SCRATCH_BYTES that every GPU loading this library holds until exit.
 *   - The first call on each device looks up that array's device address (cudaGetSymbolAddress
 *     with the device current) and caches it; make that first call before any stream capture.
 *   - Returns COLI_ERR_WORKSPACE when the call needs more scratch than the array holds
 *     (coli_moe_workspace_size(cfg, T) > COLI_MOE_STATIC_SCRATCH_BYTES), before any launch.
 *   - All calls on a device share the one array and it keeps the last call's contents; each call
 *     clears the part that must start at zero.  Calls that overlap on the GPU (different streams
 *     without ordering between them) race on the array and give wrong results: order them.
 *   - The device error word lives inside the array: coli_moe_noalloc_error_word reads it.
 *     Device anomalies never trap. */
coli_status coli_moe_layer_noalloc(const coli_moe_config *cfg, const coli_moe_weights *w,
                                   const void *x, int T, float *out, int32_t *topk_ids_out,
                                   float *topk_w_out, void *stream);

/* Synchronises `stream` and returns in *code the device error word of the current device's
 * static scratch array (the one coli_moe_layer_noalloc uses): 0 = clean, else COLI_DEVERR_*
 * bits of the last coli_moe_layer_noalloc call on this device (each call clears it first).
 * code NULL: COLI_ERR_INVALID_ARG; COLI_ERR_CUDA if the array cannot be reached.  Like the first
 * coli_moe_layer_noalloc call, the first call on a device looks the array up (before any
 * stream capture). */
coli_status coli_moe_noalloc_error_word(void *stream, int *code);

/* ---------------------------------------------------------------- router scores ------------
 * a2 in its general form: softmax or sigmoid scores, with or without a selection bias, with
 * masked experts, for routers other than the noaux_tc one of coli_moe_route. */
typedef enum { COLI_SCORE_SIGMOID = 0, COLI_SCORE_SOFTMAX = 1 } coli_score;
typedef enum { COLI_GROUP_TOP2 = 0, COLI_GROUP_MAX = 1 } coli_group_score;

typedef struct {
    int n_experts;      /* E (<= 1024) */
    int top_k;          /* K (<= 32), at most topk_group * E / n_group */
    int n_group;        /* G (<= 32); E % G == 0 */
    int topk_group;     /* TG, 1 <= TG <= G */
    int score;          /* coli_score */
    int group_score;    /* coli_group_score: what ranks the groups when TG < G */
    int renorm;         /* 1: the chosen scores are divided by their sum; 0: taken as they are */
    int logits;         /* coli_act: type of the logits */
    double scaling;     /* factor of the weights, > 0 */
} coli_moe_router;

/* Validates a router description (the checks of coli_moe_route_scores).  Host only. */
coli_status coli_moe_check_router(const coli_moe_router *r);

/* Routing of T tokens from their logits (row t at logits + t * ld elements, ld >= n_experts; 0:
 * n_experts), an optional selection bias[E] (NULL: none) to topk_ids[T][K] and topk_w[T][K].
 *   s = 1/(1+exp(-l)), or the softmax of the row; c = s + bias.  Without a bias the experts are
 *   ranked by l itself (s grows with it).
 *   An expert can be chosen when l and c are neither NaN nor -inf: a logit of -inf (or NaN)
 *   masks an expert of a token, a bias of -inf masks it for all tokens.  NaN logits and logits
 *   of -inf take no part in the softmax; logits of +inf share it equally.
 *   TG < G: each group is ranked by the largest c (l without a bias) of the experts that can be
 *   chosen (COLI_GROUP_MAX), or the sum of the two largest c, s without a bias, or of the only
 *   one (COLI_GROUP_TOP2); the TG best are kept, ties going to the lower group, groups without an
 *   expert that can be chosen last.
 *   The K best of the kept groups in descending order, ties to the lower id, with weights
 *   s / sum(chosen s) * scaling (renorm; 0 where that sum is 0) or s * scaling.  Where fewer than
 *   K can be chosen the row is filled up with the lowest other ids, in ascending order, with
 *   weight 0: every row holds K different ids, so it can be grouped and multiplied as it is.
 * Biased scores are compared in double, logits exactly; weights carry float32 sums.
 * T = 0 is a no-op.  Asynchronous on `stream`; one kernel; may be captured. */
coli_status coli_moe_route_scores(const coli_moe_router *r, const void *logits, size_t ld,
                                  const float *bias, int T, int32_t *topk_ids, float *topk_w,
                                  void *stream);

/* ---------------------------------------------------------------- microscaled 4-bit --------
 * Rows of e2m1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives; element 2j in the low
 * nibble of byte j) with one scale per block of consecutive elements of a row.
 *   COLI_FP4_MX  blocks of 32, scale 2^(byte - 127) (e8m0)
 *   COLI_FP4_NV  blocks of 16, scale e4m3 (not negative)
 * A value is code * block scale * row scale, the row scale a float32 per row (NULL: 1).
 * k is a multiple of 32.  A row's block scales take coli_moe_fp4_scale_pitch bytes: whole runs of
 * 256 elements, the bytes behind the last block zero.  Two layouts of the scales:
 *   COLI_FP4_ROWS   [rows][pitch], for activations
 *   COLI_FP4_TILES  for weight matrices: tiles of 128 rows x 4 scales, 512 bytes each, the tiles
 *                   of 128 rows one after another: scale j of row r at byte
 *                   (r / 128) * 128 * pitch + (j / 4) * 512 + (r % 32) * 16 + (r % 128) / 32 * 4 + j % 4;
 *                   rows behind the last one zero. */
typedef enum { COLI_FP4_MX = 0, COLI_FP4_NV = 1 } coli_fp4;
typedef enum { COLI_FP4_ROWS = 0, COLI_FP4_TILES = 1 } coli_fp4_layout;

/* Bytes of one row of block scales, and of a whole array of them.  Host only. */
coli_status coli_moe_fp4_scale_pitch(int fmt, int k, size_t *bytes);
coli_status coli_moe_fp4_scale_bytes(int fmt, int layout, int rows, int k, size_t *bytes);

/* Quantises `rows` rows of k values.  Row r is read from source row r (row_index NULL; rows ==
 * src_rows) or row_index[r] / row_div (device int32; a slot's token with row_div = top_k), source
 * row i at x + i * ldx elements (act: coli_act).
 *   NV: row scale 2^(floor(log2(largest |x| of the row)) - 10), at least 2^-126 (1 for a row of
 *       zeros), block scale the e4m3 nearest to (largest |x| of the block) / (6 * row scale); where
 *       that is 0 the codes are 0;
 *   MX: block scale 2^(floor(log2(largest |x| of the block)) - 2), at least 2^-127; row scale 1;
 *   code: the e2m1 nearest to x / (block scale * row scale), ties to the even code, at most 6.
 * Both are exact: the quotients are those of the real numbers.  A block that holds a NaN or an
 * infinity gets the scale NaN (0x7F, 0xFF) and codes 0, and does not count for the row scale.
 * codes [rows][k/2] (8-byte aligned), scales in `layout` (4-byte aligned), row_scale [rows].  An
 * index outside [0, src_rows) writes a row of zeros and sets COLI_DEVERR_GROUPING in the error
 * word of `ws` (256-byte aligned, its header cleared once, as for the layer).
 * x 16-byte aligned, ldx a multiple of 16 bytes.  rows = 0 is a no-op.  One kernel. */
coli_status coli_moe_fp4_quantize(int fmt, int layout, int act, const void *x, int src_rows,
                                  size_t ldx, const int32_t *row_index, int row_div, int rows,
                                  int k, uint8_t *codes, uint8_t *scales, float *row_scale,
                                  void *ws, void *stream);

/* The values that codes and scales stand for, code * block scale * row scale rounded to float32 and
 * that to `act` (a row scale that is a power of two takes part in no rounding but that of results
 * below 2^-126): out row r at out + r * ldo elements (16-byte aligned, ldo a multiple of 16 bytes).
 * row_scale NULL: 1.  One kernel. */
coli_status coli_moe_fp4_dequantize(int fmt, int layout, const uint8_t *codes,
                                    const uint8_t *scales, const float *row_scale, int rows,
                                    int k, int act, void *out, size_t ldo, void *stream);

typedef struct {
    const uint8_t *codes;    /* [rows][k/2], 16-byte aligned */
    const uint8_t *scales;   /* COLI_FP4_ROWS, 16-byte aligned */
    const float *row_scale;  /* [rows], or NULL */
    int rows;
} coli_fp4_rows;

typedef struct {
    const uint8_t *codes;    /* `count` matrices [n][k/2], 16-byte aligned */
    const uint8_t *scales;   /* `count` arrays in COLI_FP4_TILES, 16-byte aligned */
    const float *row_scale;  /* `count` arrays [n], or NULL */
    int count, n;            /* count <= 1024 */
    size_t codes_stride;     /* bytes between matrices; a multiple of 16 */
    size_t scales_stride;    /* bytes; a multiple of 16 */
    size_t row_scale_stride; /* elements */
} coli_fp4_mats;

/* out[i][j] = sum_k a[i][k] * w[j][k] for every row i of `a`, w the matrix of the row's group:
 * rows offsets[e] .. offsets[e+1] - 1 belong to matrix e (device int32 [count + 1], ascending, as
 * coli_moe_group writes them); offsets NULL: one matrix (count == 1) for all rows.  Rows outside
 * every group keep what `out` held.  A group whose own two offsets are not ascending within
 * [0, rows] is left out and sets COLI_DEVERR_GROUPING in the error word of `ws`; where such offsets
 * make two groups overlap, the rows they share hold one's results or the other's.
 * Products on the tensor cores, block scales applied there, float32 sums.  A sum is multiplied with
 * the product of its two row scales, both rounded to float32 (exact for powers of two), and the
 * result rounded to out_type (coli_act); any finite scales will do, their product may leave
 * float32's range where the result does not.  No atomics: the same call gives the same bits.
 * Tiles are counted in 32 bits: COLI_ERR_UNSUPPORTED where (rows / 16 + 1) * ceil(n / 128) *
 * (count + 1) does not fit.
 * out: row i at out + i * ldo elements, ldo >= n, aligned to its elements.  rows = 0 is a no-op.
 * One kernel; allocates nothing; may be captured. */
coli_status coli_moe_fp4_product(int fmt, const coli_fp4_rows *a, const coli_fp4_mats *w, int k,
                                 const int32_t *offsets, int out_type, void *out, size_t ldo,
                                 void *ws, void *stream);

/* Quantises one expert's matrices (device, act: coli_act; gate and up [I][H], down [H][I], rows without
 * padding, 16-byte aligned) into a record of cfg's 4-bit container (256-byte aligned,
 * coli_moe_record_bytes bytes).  COLI_ERR_UNSUPPORTED for the integer containers.  Two kernels. */
coli_status coli_moe_fp4_pack_record(const coli_moe_config *cfg, int act, const void *wg,
                                     const void *wu, const void *wd, uint8_t *record, void *ws,
                                     void *stream);

/* ---------------------------------------------------------------- rows to the experts and back ----
 * For batches whose expert products run one by one (coli_moe_fp4_product, coli_moe_i8_product, a caller's own), in
 * training too.  hidden may be any number up to 2^20, top_k up to 32, T * top_k up to 2^30 (COLI_ERR_UNSUPPORTED
 * above); rows may lie any number of elements apart, at any address of their type.  Rows, pointers and strides that
 * are multiples of 16 bytes go in 16-byte pieces, others element by element.  `ws`: 256-byte aligned, its
 * header cleared once (coli_moe_clear_error), as for the layer. */

/* a3 with positions and rows: a stable counting sort of the slots s = t * top_k + k by expert id.
 *   offsets [n_experts + 1]  rows offsets[e] .. offsets[e+1] - 1 belong to expert e (n_experts <= 1024)
 *   perm    [T * top_k]      slot of each row in that order; -1 from offsets[n_experts] on
 *   place   [T * top_k]      row of each slot, or -1
 *   rows                     row place[s] (at rows + place[s] * ldr elements) = row s / top_k of x (at x + t * ldx); rows from
 *                            offsets[n_experts] on are left as they are.  x and rows both NULL: the sort alone.
 * An id of -1 leaves its slot out (an expert of another device, a padded token); other ids outside [0,
 * n_experts) do too and set COLI_DEVERR_EXPERT_ID in the error word of `ws`.  A token may name an expert twice.
 * The gradient in x is coli_moe_combine of the rows' gradients without weights.  T = 0 writes offsets alone.
 * One kernel, or two for many slots; may be captured. */
coli_status coli_moe_sort_rows(int n_experts, int top_k, int act, const void *x, int T, int hidden,
                               size_t ldx, const int32_t *topk_ids, int32_t *offsets, int32_t *perm,
                               int32_t *place, void *rows, size_t ldr, void *ws, void *stream);

/* a7 for any rows: out[t] = add[t] + sum_k topk_w[t][k] * y[place[t][k]], float32 sums in the order add, k = 0, 1, ..,
 * rounded once to out_type (coli_act; y has type act).  topk_w NULL: weights of 1 (the gradient of
 * coli_moe_sort_rows); add NULL: 0; add may be out with the same stride, else out overlaps nothing.  A place of
 * -1 adds nothing; another one outside [0, rows) neither, and sets COLI_DEVERR_GROUPING in the error word of
 * `ws`.  A token without rows gives add[t].  T = 0 is a no-op.  One kernel, no atomics; may be captured. */
coli_status coli_moe_combine(int act, const void *y, int rows, size_t ldy, const int32_t *place,
                             const float *topk_w, int T, int top_k, int hidden, int out_type,
                             const void *add, size_t ld_add, void *out, size_t ldo, void *ws,
                             void *stream);

/* The gradient of coli_moe_combine (that in add is dout itself):
 *   dy[place[t][k]] = topk_w[t][k] * dout[t], rounded to act; rows that no place names are left as they are
 *   dw[t][k] = sum_h dout[t][h] * y[place[t][k]][h], a float32 sum; 0 where the slot has no row
 * dout has type out_type.  dy or dw may be NULL (not both); y is read for dw alone.  dy overlaps nothing.  Places as
 * in coli_moe_combine, but different ones for all slots that have a row.  T = 0 is a no-op.  One kernel, no
 * atomics; may be captured. */
coli_status coli_moe_combine_grad(int act, const void *y, int rows, size_t ldy, const int32_t *place,
                                  const float *topk_w, int T, int top_k, int hidden, int out_type,
                                  const void *dout, size_t ld_dout, void *dy, size_t ld_dy, float *dw,
                                  void *ws, void *stream);

/* ---------------------------------------------------------------- 8-bit rows and products ----
 * Rows of signed 8-bit codes with one float32 scale each: activations with a scale per token, weight matrices [n][k]
 * with one per output channel.  k is any number up to 131071; rows lie `ld` bytes apart, a multiple of 16.
 * An int8 record is such a pair of matrices: gate and up rows together n = 2 * inter, k = hidden, scales sg and su
 * one after the other; down n = hidden, k = inter (codes_stride the record stride, scale_stride a quarter of it). */

/* Quantises src_rows rows of k values: scale = m / 127 with m the row's largest |x|, at least 127 * 2^-126, rounded to
 * float32; code = the whole number nearest to x * 127 / m of the real numbers, ties to even, so within [-127, 127].
 * A row that holds a NaN or an infinity gets the scale NaN and codes 0.
 *   swiglu = 0: row i is x + i * ldx (act: coli_act), k values.
 *   swiglu = 1: row i holds k gate and then k up values; what is quantised is gate / (1 + exp(-gate)) * up in float32
 *               (within 2^-20 of the real value for every finite gate; a gate of -infinity gives NaN).
 * Row i goes to the rows place[i * copies + c], c < copies, of the result (device int32; a place of -1 is left out, another
 * one outside [0, rows) too and sets COLI_DEVERR_GROUPING in the error word of `ws`; the places differ), as
 * coli_moe_sort_rows gives them with copies = top_k.  place NULL: row i to row i, copies == 1, rows == src_rows.
 * Rows of the result that nothing names are left as they are.  codes overlap nothing, 16-byte aligned, ldc bytes from row to row, a
 * multiple of 16; bytes from k to the next multiple of 16 become 0.  COLI_ERR_UNSUPPORTED where rows, src_rows or src_rows *
 * copies is above 2^30, or k above 131071.  src_rows = 0 is a no-op.  One kernel. */
coli_status coli_moe_i8_quantize(int act, int swiglu, const void *x, int src_rows, size_t ldx, int k,
                                 const int32_t *place, int copies, int rows, int8_t *codes, size_t ldc,
                                 float *scale, void *ws, void *stream);

typedef struct {
    const int8_t *codes;   /* [rows], ld bytes apart, 16-byte aligned */
    const float *scale;    /* [rows], or NULL: 1 */
    int rows;              /* <= 2^30 */
    size_t ld;             /* bytes; a multiple of 16, < 2^30 */
} coli_i8_rows;

typedef struct {
    const int8_t *codes;   /* `count` matrices of n rows, ld bytes apart, 16-byte aligned */
    const float *scale;    /* `count` arrays [n], or NULL: 1 */
    int count, n;          /* count <= 1024 */
    size_t ld;             /* bytes; a multiple of 16, < 2^30; n * ld < 2^40 */
    size_t codes_stride;   /* bytes between matrices; a multiple of 16, < 2^40 */
    size_t scale_stride;   /* elements */
} coli_i8_mats;

/* out[i][j] = a.scale[i] * w.scale[j] * sum_k a[i][k] * w[j][k] for every row i of `a`, w the matrix of the row's
 * group; offsets, groups, rows outside every group, bad offsets, out_type, out and ldo as in coli_moe_fp4_product.
 * Sums are exact (32-bit integers; any codes, -128 too), rounded to float32 and multiplied with the product of the two
 * scales, itself rounded to float32; any finite scales will do, their product may leave float32's range where the
 * result does not.  The same call gives the same bits.  COLI_ERR_UNSUPPORTED for k above 131071, rows, counts and strides beyond
 * the bounds above (codes_stride and scale_stride are not looked at where count == 1), and, as tiles are counted in 32 bits, where
 * (rows / 16 + 1) * ceil(n / 128) * (count + 1) does not fit.  rows = 0 is a no-op.  One kernel; allocates nothing; may be
 * captured. */
coli_status coli_moe_i8_product(const coli_i8_rows *a, const coli_i8_mats *w, int k,
                                const int32_t *offsets, int out_type, void *out, size_t ldo, void *ws,
                                void *stream);

#ifdef __cplusplus
}
#endif
#endif /* COLI_MOE_H */
