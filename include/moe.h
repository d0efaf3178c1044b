/*
 * moe.h -- C ABI of the GB300 (sm_103a) routed-expert MoE FFN layer, inference hot path, of the
 * attention over a paged cache that stands before it in a decoder layer (moe_attn_*), and of matrices
 * in MXFP4 and their product, for the projections around the attention (moe_mx_*).
 *
 * The layer, as the pages state it:
 *   router     -- score every routed expert for each token, keep the top-k
 *                 ("DeepSeek-V4-Pro on NVIDIA H200", section 0.2.2, step D4);
 *   permute    -- reorder the token rows by expert ("第 6 章 超節點", section 6.2.6: the receiver
 *                 reorders rows by expert, multiplies, then restores token order);
 *   expert FFN -- per expert Y = [SiLU(X W_g) (.) (X W_u)] W_d ("第 6 章 超節點", section 6.2.2),
 *                 three GEMMs per expert ("DeepSeek V3/R1 Inference Efficiency (1)", Parameters);
 *   combine    -- routing-weighted sum of the experts' outputs, a1*y1 + a6*y6, plus the
 *                 always-on shared expert ("第 6 章 超節點", sections 6.2.6 and 6.4.1;
 *                 "DeepSeek-V4-Pro on NVIDIA H200", section 0.1.2 and step D7).
 * On one GPU the dispatch and combine exchanges become in-HBM gathers.
 *
 * One GPU. The library has no multi-GPU path: every call works on buffers of the current
 * device only, and no kernel loads from another GPU's memory or multicasts a load. Its prefill
 * tiles run on CTA pairs (tcgen05 cta_group::2): each CTA of a 2-CTA cluster loads its own
 * weight rows and half of the token tile, and one MMA of the pair reads both CTAs' operands.
 *
 * Conventions shared by every entry point
 *   - Pointers named x, wg, bias, topk_*, expert_offsets, perm_token, inv_slot, w13, s13, w2,
 *     s2, y_perm, y and ws are DEVICE pointers, allocated and owned by the caller. The library
 *     never allocates, frees or synchronises in these calls; work is enqueued on `stream`
 *     (a cudaStream_t, NULL = legacy default stream) and the call returns immediately
 *     (moe_expert_ffn may also use one library-owned stream per device; see there).
 *   - `shape` is a host pointer read during the call only.
 *   - Arguments are validated on the host first: a negative status is returned before any
 *     launch and nothing is written (no side effects).
 *   - Device-side checks (an index out of range, a duplicated expert in a token's top-k row, a
 *     bounded wait that gave up) never fault: the kernel skips the bad access and records the
 *     first error code in the workspace; moe_check_device_status() reports it.
 *   - Tensors are dense row-major; "bf16" is IEEE-style bfloat16, "E4M3" is OCP FP8 E4M3;
 *     "MXFP4" is the OCP Microscaling (MX) v1.0 FP4 format: E2M1 elements with one E8M0 scale
 *     per 32 consecutive elements of a row.
 *   - Every pointer must be 16-byte aligned (256-byte for ws; 32-byte for MXFP4 w13 and w2).
 *   - Shapes: 1 <= E <= 1024, 1 <= k <= min(E, 32), n_shared in {0, 1}, d and f multiples of
 *     128 with 128 <= d <= 16384 and 128 <= f <= 16384, 0 <= T and T*(k+1) <= 2^30.
 *   - What a call writes (outputs, ws) overlaps no other array of the call, unless its description
 *     says so; blocks read and write in any order. moe_mx_* check this and refuse arrays that do.
 *   - Not thread-safe per workspace: calls that share a workspace must be ordered on one stream.
 */
#ifndef MOE_GB300_H
#define MOE_GB300_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define MOE_API __attribute__((visibility("default")))
#else
#define MOE_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = -1,     /* bad pointer, shape or alignment (host check)             */
  MOE_ERR_UNSUPPORTED = -2,     /* valid request this build does not serve (e.g. no GPU)    */
  MOE_ERR_WORKSPACE = -3,       /* ws_bytes < moe_workspace_size(shape)                     */
  MOE_ERR_CUDA = -4,            /* a CUDA runtime/driver call or a launch failed            */
  MOE_ERR_DEVICE_TIMEOUT = -5,  /* a bounded device wait gave up (reported by the check)    */
  MOE_ERR_DEVICE_BOUNDS = -6    /* a device-side index check failed (reported by the check) */
} moe_status;

typedef enum {
  MOE_W_BF16 = 0,            /* expert weights bf16                                          */
  MOE_W_FP8_E4M3_B128 = 1,   /* expert weights E4M3 with one fp32 scale per 128x128 block    */
  MOE_W_MXFP4_E8M0_B32 = 2   /* expert weights MXFP4: E2M1 codes, one E8M0 scale per 32      */
} moe_wdtype;

typedef struct {
  int32_t T;         /* tokens in the batch                                                   */
  int32_t d;         /* hidden size                                                           */
  int32_t E;         /* routed experts                                                        */
  int32_t k;         /* routed experts chosen per token                                       */
  int32_t f;         /* expert intermediate size                                              */
  int32_t n_shared;  /* shared (always-on) experts, 0 or 1; the shared expert is index E      */
  int32_t wdtype;    /* moe_wdtype of w13/w2                                                  */
} moe_shape;

/* Bytes of scratch (`ws`) the four calls need for this shape; 0 for an invalid shape. One
 * workspace serves all four calls of a layer. Its first 4 bytes are the device status word:
 * moe_route clears it (a layer starts there); a caller that skips moe_route must zero those
 * 4 bytes once before its first call. Nothing else in it needs initialisation. */
MOE_API size_t moe_workspace_size(const moe_shape* shape);

/* Router ("DeepSeek-V4-Pro on NVIDIA H200", 0.2.2 D4; "CANN DeepSeek-V4推理优化", MoE
 * 专家模型规格, soft routing).
 *   x        [T, d] bf16 tokens.        wg [E, d] bf16 router weight (one row per expert).
 *   bias     [E] fp32 added to the logits, or NULL.
 *   topk_idx [T, k] int32 out: the k experts with the largest logits, by descending logit,
 *            ties to the lower expert index.
 *   topk_w   [T, k] fp32 out: softmax over all E logits, renormalised over the k chosen
 *            (= softmax over the k chosen logits).
 * The logit l[t,e] = x[t].wg[e] (+ bias[e]) is formed in fp32 in one fixed order, so the
 * choice is reproducible bit for bit: d is cut into 8-element chunks, lane j of 32 accumulates
 * chunks j, j+32, ... element by element with fused multiply-add from +0, the 32 lane sums
 * are combined by an xor butterfly (offsets 16, 8, 4, 2, 1), then the bias is added.
 * Batches of 1024 tokens or more, with E a multiple of 128 and d a multiple of 64, first form
 * approximate logits on the tensor cores; each is taken to lie within 2^-12 |x[t]| |wg[e]| of
 * the defined logit (a bound checked on every logit recomputed), so only the experts that can
 * still reach the top k (the candidates) get their logits recomputed in the order above, and the
 * choice and the gate weights are the same bits. Words
 * 1 and 2 of the workspace (bytes 4..11) then hold the number of tokens whose logits were all
 * recomputed because a recomputed logit missed its bound (0 on every test input), and the largest
 * share of the bound a candidate used (fp32 bits). Inputs must be finite. */
MOE_API moe_status moe_route(const moe_shape* shape, const void* x, const void* wg, const float* bias,
                     int32_t* topk_idx, float* topk_w, void* ws, size_t ws_bytes, void* stream);

/* The router of moe_route without a workspace, for callers that cannot allocate device memory
 * themselves -- for instance a plugin whose host process owns every device allocation through
 * its own pool and lends it no scratch, or a deployment that fixes its device memory budget at
 * start-up and forbids allocations afterwards. The pages have no counterpart of this entry point.
 * Same arguments, results and validation as moe_route, minus ws/ws_bytes; it allocates nothing
 * and calls no allocating routine. Its logits scratch is a fixed 4 MiB device array inside the
 * library (one copy per GPU that loads the library, kept until the process exits), so it serves
 * shapes with T*E <= 1,048,576 (e.g. T <= 4096 at E = 256) and rejects larger ones with
 * MOE_ERR_INVALID_ARG. Each call looks up that array's device address in the current context
 * (cudaGetSymbolAddress, which allocates nothing), so the address stays right after a
 * cudaDeviceReset; a device's first call also loads the library's device code there, so make
 * that first call before any stream capture. Every call shares the one array, so calls
 * that overlap on the GPU (different streams, or different host threads on the same device)
 * race on it; order them on one stream. Nothing in the array needs to start at zero: each call
 * overwrites the logits it reads. It records no device status. */
MOE_API moe_status moe_route_noalloc(const moe_shape* shape, const void* x, const void* wg,
                                     const float* bias, int32_t* topk_idx, float* topk_w,
                                     void* stream);

/* Hash routing ("CANN DeepSeek-V4推理优化", MoE 专家模型规格: V4's first layers pick experts by
 * hash routing, the others by learned soft routing). The page gives no hash function; here the
 * choice is a table supplied with the model, and the gate weights are the soft router's:
 *   token_ids      [T] int32 token ids in [0, vocab).
 *   tid2eid        [vocab, k] int32: row v holds the k distinct experts (in [0, E)) of token
 *                  id v.
 *   topk_idx       [T, k] int32 out: tid2eid[token_ids[t]], in the table's order.
 *   topk_w         [T, k] fp32 out: softmax over the token's E router logits, kept at those k
 *                  experts and renormalised -- equal to exp(l_j - max) / sum over the k, in
 *                  fp32, so only the k hashed logits are formed (each in moe_route's order).
 * x, wg, bias, ws as in moe_route (the status word is cleared: a layer starts here). A token id or table entry out of range is recorded as MOE_ERR_DEVICE_BOUNDS
 * (the entry is replaced by 0). Returns MOE_ERR_INVALID_ARG for vocab < 1. */
MOE_API moe_status moe_route_hash(const moe_shape* shape, const void* x, const void* wg,
                                  const float* bias, const int32_t* token_ids,
                                  const int32_t* tid2eid, int32_t vocab, int32_t* topk_idx,
                                  float* topk_w, void* ws, size_t ws_bytes, void* stream);

/* Scored routing: softmax or sigmoid scores, a bias that balances the experts' load and only
 * chooses, groups of experts of which some are kept, weights renormalised and scaled.
 *   l  the token's E logits;  s = softmax(l) or 1 / (1 + exp(-l));  c = s + sel_bias (or s).
 *   n_group > 1: the experts lie in n_group groups of E / n_group in a row; a group's value is the
 *   sum of its group_top largest c; the topk_group groups of the largest values are kept.
 *   topk_idx: the k largest c of the kept groups, by descending c, ties (of groups and of experts)
 *   to the lower index.  topk_w = scale * s, or with renorm scale * s / (sum of the k s). */
typedef enum {
  MOE_SCORE_SOFTMAX = 0,
  MOE_SCORE_SIGMOID = 1
} moe_score;

typedef struct {
  int32_t score;       /* moe_score                                                           */
  int32_t n_group;     /* groups of experts, 1 .. 32; E a multiple                            */
  int32_t topk_group;  /* groups kept, 1 .. n_group; k <= topk_group * E / n_group            */
  int32_t group_top;   /* experts whose c make a group's value: 1 or 2, <= E / n_group        */
  int32_t renorm;      /* nonzero: the k weights are divided by their sum                     */
  float scale;         /* of the weights; finite                                              */
} moe_gate;

/* The selection alone, from logits that the caller has.
 *   logits   [T, E] fp32.   sel_bias [E] fp32, or NULL.
 *   topk_idx [T, k] int32 out, topk_w [T, k] fp32 out (fp32 arithmetic).
 * The choice is that of the formulas in 64-bit arithmetic: fp32 values nearer to each other than
 * their error bounds are computed again in 64 bits. Without sel_bias the experts rank by their logits
 * (the same order). A NaN c ranks below every number. Sigmoid weights of logits that are all
 * -infinity are 0. Only T, E and k of `shape` are used (it must be valid); no workspace. */
MOE_API moe_status moe_route_select(const moe_shape* shape, const moe_gate* gate,
                                    const float* logits, const float* sel_bias,
                                    int32_t* topk_idx, float* topk_w, void* stream);

/* The router from the tokens: moe_route's logits (each in its fixed order, bias added to the logit),
 * then the selection of moe_route_select. x, wg, bias, topk_idx, topk_w, ws as in moe_route (the
 * status word is cleared: a layer starts here). The experts are those that all logits in that order
 * give; large batches form only the logits that the choice depends on (the others by tensor cores, in
 * the workspace), unless softmax scores need them all: with sel_bias, without renorm, or in sums of two.
 * A caller with logits of its own uses moe_route_select. */
MOE_API moe_status moe_route_gate(const moe_shape* shape, const moe_gate* gate, const void* x,
                                  const void* wg, const float* bias, const float* sel_bias,
                                  int32_t* topk_idx, float* topk_w, void* ws, size_t ws_bytes,
                                  void* stream);

/* Token -> expert permutation ("第 6 章 超節點", 6.2.6).
 *   topk_idx       [T, k] int32, each row k distinct experts in [0, E).
 *   expert_offsets [E+2] int32 out: expert e (< E) owns slots [offsets[e], offsets[e+1]);
 *                  offsets[E] = T*k starts the shared expert's segment and
 *                  offsets[E+1] = T*k + n_shared*T ends it.
 *   perm_token     [T*k] int32 out: token of each routed slot; slots are expert-major and,
 *                  within an expert, in ascending token order (a stable counting sort).
 *   inv_slot       [T*k] int32 out: inv_slot[t*k + j] = slot of token t's j-th choice.
 * The shared segment is implicit: slot T*k + t belongs to token t. Deterministic (no atomics
 * decide any order). */
MOE_API moe_status moe_permute(const moe_shape* shape, const int32_t* topk_idx, int32_t* expert_offsets,
                       int32_t* perm_token, int32_t* inv_slot, void* ws, size_t ws_bytes,
                       void* stream);

/* Per-expert SwiGLU FFN over every slot ("第 6 章 超節點", 6.2.2: Y = [SiLU(X W_g) (.) (X W_u)] W_d).
 *   x              [T, d] bf16 tokens; perm_token and expert_offsets as made by moe_permute.
 *   w13            [E+n_shared, 2f, d]: rows 0..f-1 of expert e are its gate projection, rows
 *                  f..2f-1 its up projection (one row per output feature, d contiguous).
 *   w2             [E+n_shared, d, f]: the down projection (one row per output feature).
 *                  bf16; E4M3 codes (one byte each) for MOE_W_FP8_E4M3_B128; or, for
 *                  MOE_W_MXFP4_E8M0_B32, E2M1 codes two per byte ([E+n_shared, 2f, d/2] and
 *                  [E+n_shared, d, f/2] bytes; element 2j of a row in the low nibble of byte j,
 *                  element 2j+1 in the high nibble), 32-byte aligned.
 *   s13, s2        E4M3 weights: fp32 block scales [E+n_shared, 2f/128, d/128] and
 *                  [E+n_shared, d/128, f/128] (weight = code value * scale of its 128x128
 *                  block). MXFP4 weights: E8M0 bytes [E+n_shared, 2f, d/32] and
 *                  [E+n_shared, d, f/32], one per 32 consecutive elements of a row (weight =
 *                  element value * 2^(scale - 127); "DeepSeek-V4-Pro on NVIDIA H200", 0.1.3:
 *                  FP4 expert weights; "CANN DeepSeek-V4推理优化", 量化策略: MXFP4). NULL for
 *                  bf16.
 *   y_perm         [T*k + n_shared*T, d] fp32 out: row s = expert output for slot s, i.e.
 *                  W_d^T (SiLU(W_g^T x) * (W_u^T x)) for the slot's token and expert.
 * The intermediate h = SiLU(G) * U is kept in bf16; accumulation is fp32. With MXFP4 weights
 * the tensor cores multiply the E2M1 codes as stored, so the activations (x, then h) enter the
 * products as two E4M3 terms with their own E8M0 scales per 32 elements, within 2^-8 of each
 * 32-element block's largest magnitude (about one bf16 rounding of that element).
 * Prefill-sized batches with bf16 weights (more than 32 routed tokens per expert on average)
 * run the experts with few tokens and those with many on two streams at once: `stream` and a
 * second stream the library creates on its first such call on each device (a host-side object;
 * no device memory is allocated), ordered against `stream` with events inside the call, so the
 * call still behaves as work enqueued on `stream` (also under CUDA-graph capture). */
MOE_API moe_status moe_expert_ffn(const moe_shape* shape, const void* x, const int32_t* perm_token,
                          const int32_t* expert_offsets, const void* w13, const void* s13,
                          const void* w2, const void* s2, float* y_perm, void* ws,
                          size_t ws_bytes, void* stream);

/* Combine ("第 6 章 超節點", 6.2.6 and 6.4.1: send back, restore token order, sum with the
 * routing weights).
 *   y[t] = y_perm[T*k + t] (if n_shared) + sum_j topk_w[t, j] * y_perm[inv_slot[t*k + j]],
 *   accumulated in fp32 in that order and rounded once to bf16 (nearest even).
 *   y [T, d] bf16 out. ws is used only to record device-side index errors. */
MOE_API moe_status moe_combine(const moe_shape* shape, const float* y_perm, const int32_t* inv_slot,
                       const float* topk_w, void* y, void* ws, size_t ws_bytes, void* stream);

/* The whole layer in one call: moe_route, moe_permute, moe_expert_ffn and moe_combine with the
 * same arguments and results (every output buffer above is filled), with one difference in
 * scheduling: the shared expert does not depend on the routing, so its FFN runs on a second,
 * library-owned stream (one per device, created on the first such call; no device memory is
 * allocated) while the router, the permutation and the row gather run on `stream` ("CANN
 * DeepSeek-V4推理优化", 多流并行优化: the shared and the routed experts on parallel streams). The
 * call joins both before the combine, so it behaves as work enqueued on `stream`. Calls that
 * overlap on the GPU (different streams, same device) order their shared-expert work through
 * that one second stream. The overlap is used for prefill-sized batches (more than 32 routed
 * tokens per expert on average) with n_shared = 1; otherwise the four steps run in order on
 * `stream`. y_perm [T*k + n_shared*T, d] fp32 and y [T, d] bf16 as in moe_expert_ffn and
 * moe_combine. The status word is cleared as the call starts (batches of at most 8 tokens: by
 * the call's first kernel, so that a CUDA graph of consecutive calls holds no memset node). */
MOE_API moe_status moe_forward(const moe_shape* shape, const void* x, const void* wg,
                               const float* bias, const void* w13, const void* s13,
                               const void* w2, const void* s2, int32_t* topk_idx, float* topk_w,
                               int32_t* expert_offsets, int32_t* perm_token, int32_t* inv_slot,
                               float* y_perm, void* y, void* ws, size_t ws_bytes, void* stream);

/* ---- attention over a paged key-value cache -------------------------------------------------
 * The other half of a decoder layer, between the qkv projection and the output projection:
 * moe_attn_append norms and rotates a step's queries and keys and writes keys and values into
 * the cache; moe_attn_decode (one new token per sequence) and moe_attn_prefill (any number)
 * attend over it. Hq = G * Hkv query heads, G per key head; head h * G + g reads key head h.
 *
 * Sequence b holds kv_len[b] cached tokens, this step's included, in the pages
 * block_table[b, 0 ..]: cache place j lies in page block_table[b, j / page_size] at row
 * j % page_size. Its new tokens are rows q_start[b] .. q_start[b+1]-1 of q, k, v and o; the i-th
 * of n has place kv_len[b] - n + i (a negative place is padding: nothing is cached for it and
 * its output is zero). Place p sees place j if j <= p and (window = 0 or p - j < window or
 * j < n_sink). block_table entries of pages that hold no visible place are not read; what the
 * cache holds beyond kv_len never reaches a result, nor what it holds outside the window but for
 * moe_attn_prefill's tiles (see there).
 *
 * q_start, kv_len, block_table and positions are DEVICE int32 arrays and are checked there: a
 * page outside [0, num_pages), a length beyond the table or a rotary position outside
 * [0, max_pos) is recorded as MOE_ERR_DEVICE_BOUNDS and the access is skipped. Two sequences
 * must not append to the same place. */
typedef enum {
  MOE_KV_BF16 = 0,          /* cache of bf16 keys and values                                  */
  MOE_KV_FP8_E4M3 = 1       /* cache of E4M3 codes, one fp32 scale per key head               */
} moe_kv_dtype;

typedef struct {
  int32_t T;          /* new tokens in the step, all sequences together (decode: T = B)       */
  int32_t B;          /* sequences                                                            */
  int32_t Hq, Hkv;    /* query heads and key heads; Hq a multiple of Hkv, Hq / Hkv <= 128     */
  int32_t D;          /* head width: 64 or 128                                                */
  int32_t kv_dtype;   /* moe_kv_dtype of the cache                                            */
  int32_t page_size;  /* tokens of a page, >= 1                                               */
  int32_t max_pages;  /* columns of block_table                                               */
  int32_t num_pages;  /* pages of the cache                                                   */
  int32_t window;     /* 0: every earlier place is visible; else the last `window` places     */
  int32_t n_sink;     /* with a window: the first n_sink places stay visible                  */
  int32_t rot_dim;    /* leading elements of a head that are rotated: a multiple of 16, <= D  */
  int32_t rot_pairs;  /* 0: element i turns with i + rot_dim/2; 1: element 2i with 2i + 1     */
  int32_t max_pos;    /* rows of cos_sin                                                      */
  float scale;        /* softmax scale; 0 means 1 / sqrt(D)                                   */
  float eps;          /* of the norms                                                         */
  /* Strides in elements; 0 means packed. Every stride is a multiple of 16 bytes.             */
  int64_t q_stride, k_stride, v_stride;   /* append's inputs, between tokens (Hq*D, Hkv*D)    */
  int64_t qr_stride;                      /* append's q_out, the attentions' q (Hq*D)         */
  int64_t o_stride;                       /* the attentions' o (Hq*D)                         */
  /* both caches: between pages, between key heads, between tokens of a page. Packed is
   * [num_pages, Hkv, page_size, D]; [num_pages, page_size, Hkv, D] is head_stride = D,
   * token_stride = Hkv * D, page_stride = page_size * Hkv * D. */
  int64_t page_stride, head_stride, token_stride;
} moe_attn_shape;

/* Bytes of scratch for moe_attn_append and moe_attn_decode, or (prefill != 0) for
 * moe_attn_prefill as well; 0 for an invalid shape. The first moe_attn_workspace_zero_bytes()
 * bytes (the device status word) must be zero before the first call; nothing else needs
 * initialisation, and one workspace may serve several shapes. moe_check_device_status reads its
 * status word. */
MOE_API size_t moe_attn_workspace_size(const moe_attn_shape* shape, int prefill);
MOE_API size_t moe_attn_workspace_zero_bytes(void);

/* Norms, rotation and cache append in one pass over a step's projections.
 *   q [T, Hq, D], k [T, Hkv, D], v [T, Hkv, D] bf16 (token strides q_stride, k_stride, v_stride:
 *     they may be parts of one projection's rows).
 *   q_norm, k_norm [D] bf16, or NULL for no norm: y = x / sqrt(mean(x^2) + eps) * norm, per head.
 *   cos_sin [max_pos, rot_dim] fp32: the cosines of the rot_dim/2 angles, then the sines; (a, b)
 *     becomes (a cos - b sin, b cos + a sin). NULL if rot_dim = 0.
 *   positions [T] int32 rotary positions, or NULL for the tokens' places in the cache.
 *   q_start [B+1], or NULL with T = B for one new token per sequence. Rows from q_start[B] on
 *     are padding.
 *   k_scale, v_scale [Hkv] fp32 (E4M3 caches; NULL for 1, and for bf16 caches): the cache holds
 *     e4m3(value / scale), rounded to nearest even and saturating at +-448.
 *   q_out [T, Hq, D] bf16 out (may be q itself if the strides agree); k_cache, v_cache updated.
 * The arithmetic is fp32 with one rounding at the end. */
MOE_API moe_status moe_attn_append(const moe_attn_shape* shape, const void* q, const void* k,
                                   const void* v, const void* q_norm, const void* k_norm,
                                   const float* cos_sin, const int32_t* positions,
                                   const int32_t* block_table, const int32_t* kv_len,
                                   const int32_t* q_start, const float* k_scale,
                                   const float* v_scale, void* q_out, void* k_cache,
                                   void* v_cache, void* ws, size_t ws_bytes, void* stream);

/* Attention of one new token per sequence (T = B) over the cache.
 *   s_j = scale * q . k_j over the visible places, o = sum_j softmax(s)_j v_j, lse = ln sum_j e^s_j
 *   q [B, Hq, D] bf16, o [B, Hq, D] bf16 out, lse [B, Hq] fp32 out or NULL.
 * A sequence with kv_len = 0 gives o = 0 and lse = -inf. Scores, the softmax's maximum and sum
 * and the output are held in fp32; the probabilities enter the product with v as f16 (E4M3 cache)
 * or as the sum of two bf16 (bf16 cache). A NaN among the scores that a row sees makes the row NaN.
 * The result does not depend on the order in which blocks run. */
MOE_API moe_status moe_attn_decode(const moe_attn_shape* shape, const void* q,
                                   const void* k_cache, const void* v_cache,
                                   const float* k_scale, const float* v_scale,
                                   const int32_t* block_table, const int32_t* kv_len, void* o,
                                   float* lse, void* ws, size_t ws_bytes, void* stream);

/* Attention of any number of new tokens per sequence over the cache, which holds them already:
 * prompts, chunks of prompts over what is cached, in one ragged step.
 *   q [T, Hq, D] bf16, o [T, Hq, D] bf16 out, lse [T, Hq] fp32 out or NULL; rows of o and lse from
 *   q_start[B] on are not written. A token that sees no place gives o = 0 and lse = -inf.
 * Scores, the softmax's maximum and sum and the output are held in fp32; the probabilities enter
 * the product with v as bf16. What the cache holds at the places of a sequence must be finite:
 * 0 times a NaN or an infinity of v is a NaN, so one spreads to the tokens of its tile (128 / G
 * or more tokens, 64 places) that do not see it. Beyond kv_len, and in pages that no token of
 * the step sees anything of, it does not. E4M3 caches, and bf16 caches whose pages are not a
 * multiple of 16 tokens, are first unpacked into the workspace
 * (4 B Hkv max_pages page_size D bytes, max_pages page_size rounded up to 128, at most 2^40): the
 * tables' width counts, not the lengths. */
MOE_API moe_status moe_attn_prefill(const moe_attn_shape* shape, const void* q,
                                    const void* k_cache, const void* v_cache,
                                    const float* k_scale, const float* v_scale,
                                    const int32_t* block_table, const int32_t* kv_len,
                                    const int32_t* q_start, void* o, float* lse, void* ws,
                                    size_t ws_bytes, void* stream);

/* ---- matrices in MXFP4 and their product ------------------------------------------------------
 * The format of the MXFP4 expert weights: E2M1 codes, two a byte (element 2j of a row in the low
 * nibble of byte j), one E8M0 scale 2^(e - 127) for every 32 consecutive elements of a row. Rows are
 * packed: K / 2 bytes of codes each. The scales lie in one of two layouts:
 *   rows   [rows, K/32] bytes, as the experts' s13 and s2;
 *   tiles  as the tensor cores take them: for every 128 rows and every 128 elements of K a block of
 *          512 bytes, blocks of the same rows in a row; the scale of row r, element 32 j lies in block
 *          (r / 128, j / 4) at byte 16 (r % 32) + 4 (r % 128 / 32) + j % 4. Padding of K in the last
 *          block of a row holds 127; padding rows hold anything. */
typedef enum {
  MOE_T_BF16 = 0,
  MOE_T_F32 = 1,
  MOE_T_MXFP4 = 2
} moe_mx_dtype;

typedef struct {
  int32_t rows;      /* 0 .. 2^24                                                             */
  int32_t K;         /* elements of a row: a multiple of 32, 32 .. 2^17                       */
  int32_t dtype;     /* of the wide side: MOE_T_BF16 or MOE_T_F32                             */
  int32_t tiles;     /* scales in tiles (nonzero) or in rows (0)                              */
  int64_t stride;    /* elements between the rows of the wide side; 0: K. Multiple of 16 bytes */
} moe_mx_rows;

/* Bytes of the scale array of these rows; 0 for invalid ones. */
MOE_API size_t moe_mx_scale_bytes(const moe_mx_rows* rows);

/* x [rows, K] to MXFP4: for each 32 elements 2^(floor(log2 max|x|) - 2) as the scale (at least 2^-127;
 * 1 if all are 0), elements divided by it and rounded to the nearest E2M1 value, ties to the even
 * code, magnitudes above 6 to 6. A NaN or an infinity among the 32 makes the scale NaN (0xFF).
 *   codes [rows, K/2] out, scales out (moe_mx_scale_bytes). */
MOE_API moe_status moe_mx_quantize(const moe_mx_rows* rows, const void* x, void* codes,
                                   void* scales, void* stream);

/* The values back: y [rows, K] = code value * scale, exact in fp32 and, below 2^128, in bf16. A NaN
 * scale gives NaNs. */
MOE_API moe_status moe_mx_dequantize(const moe_mx_rows* rows, const void* codes,
                                     const void* scales, void* y, void* stream);

/* Scales in rows to scales in tiles (rows->rows and rows->K are used): once for a weight matrix that
 * was stored with scales in rows. */
MOE_API moe_status moe_mx_tile_scales(const moe_mx_rows* rows, const void* scales, void* tiles,
                                      void* stream);

typedef struct {
  int32_t T;         /* rows of x and y, 0 .. 2^24                                            */
  int32_t N;         /* rows of w: columns of y, 1 .. 2^20                                    */
  int32_t K;         /* elements of a row of x and of w: a multiple of 32, 32 .. 2^17         */
  int32_t x_dtype;   /* MOE_T_BF16: quantised by the call; MOE_T_MXFP4: codes and tiled scales */
  int64_t x_stride;  /* elements between rows of a bf16 x; 0: K. A multiple of 8              */
  int64_t y_stride;  /* elements between rows of y; 0: N                                      */
  int64_t r_stride;  /* elements between rows of the residual; 0: N                           */
} moe_mx_shape;

/* Bytes of scratch for moe_mx_linear; 0 for an invalid shape. Its first 4 bytes are a device status
 * word (moe_check_device_status reads it): zero before the first call. Nothing else needs
 * initialisation, and one workspace may serve several shapes. */
MOE_API size_t moe_mx_linear_workspace_size(const moe_mx_shape* shape);

/* y = x w^T + bias + residual, both matrices in MXFP4, on block-scaled tensor-core products: the
 * projections before and after the attention.
 *   x        [T, K] bf16 (x_scales NULL; quantised as by moe_mx_quantize), or codes [T, K/2] with
 *            x_scales in tiles.
 *   w        codes [N, K/2], w_scales in tiles.
 *   bias     [N] fp32, or NULL.   residual [T, N] bf16, or NULL; it may be y itself (same stride).
 *            Columns of one buffer (x, residual and y with the buffer's stride) do not overlap.
 *   y        [T, N] bf16 out.
 * Products are exact, sums are fp32, with one rounding to bf16 at the end. The result does not depend on the
 * order in which blocks run. */
MOE_API moe_status moe_mx_linear(const moe_mx_shape* shape, const void* x, const void* x_scales,
                                 const void* w, const void* w_scales, const float* bias,
                                 const void* residual, void* y, void* ws, size_t ws_bytes,
                                 void* stream);

/* Reads (and clears) the first device-side error recorded in `ws` since the last check.
 * Synchronises `stream`. Returns MOE_OK, MOE_ERR_DEVICE_BOUNDS or MOE_ERR_DEVICE_TIMEOUT (or
 * MOE_ERR_CUDA if the read itself fails). */
MOE_API moe_status moe_check_device_status(void* ws, void* stream);

/* Failure-path self-test (no counterpart on the pages). Launches one kernel whose single thread
 * waits on a shared-memory mbarrier that nothing ever completes, using the same bounded-wait
 * pattern as the tensor-core pipelines but with a limit of `limit_us` microseconds
 * (1 .. 2,000,000; MOE_ERR_INVALID_ARG otherwise). When the limit passes the kernel records
 * MOE_ERR_DEVICE_TIMEOUT in the status word of `ws` (first error wins) and returns, so the
 * context stays usable; moe_check_device_status() then reports and clears it. `ws` is a
 * workspace of any shape (only its status word is touched). Asynchronous like the other calls. */
MOE_API moe_status moe_selftest_bounded_wait(void* ws, uint32_t limit_us, void* stream);

/* Phase timing for benchmarks and profilers (no counterpart on the pages).
 * moe_profile_enable(1) starts a session (and clears the previous one): from then on every
 * moe_expert_ffn call records three CUDA events on its stream -- before its gate/up kernels,
 * between them and its down kernels, and after -- and every call counts the kernels it
 * launches. Events are created by the library while a session is on (host-side objects; no
 * device memory is allocated). moe_profile_enable(0) stops recording.
 * The events are recorded as external events, so a moe_expert_ffn call captured into a CUDA
 * graph records them on every replay (moe_profile_read then reports the latest replay).
 * moe_profile_read waits for the recorded events and returns the summed device milliseconds of
 * the gate/up and down phases over the session, the number of moe_expert_ffn calls timed, and
 * the number of kernels launched by all four calls; any output pointer may be NULL. */
MOE_API moe_status moe_profile_enable(int on);
MOE_API moe_status moe_profile_read(double* ms_gate_up, double* ms_down, int64_t* ffn_calls,
                                    int64_t* kernel_launches);

/* Message for the last non-OK status returned on the calling thread (thread-local storage;
 * valid until the next call on that thread). */
MOE_API const char* moe_last_error_string(void);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GB300_H */
