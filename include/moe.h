/*
 * moe.h -- C ABI of the top-k gated Mixture-of-Experts FFN layer for one NVIDIA
 * GB300 GPU (sm_103a): its forward pass, the gradients of its steps, and an
 * AdamW step.
 *
 * The layer (sources: "Qwen2-MoE代码解析：MoE架构原理、工程实现与部署避坑指南",
 * jsqmd.com, sections 3.1, 3.3, 3.4; the Qwen2-MoE module article, mlqm.cn,
 * sections 2.2 and 3.2; the MoE sparse-activation article, wmrh.cn, section 2.2):
 *
 *   l      = x Wg^T (+ gate_bias)                      router scores      [T, E]
 *   p      = softmax(l)                                                   [T, E]
 *   ids    = top-k of l, largest first, ties to the lower expert index    [T, K]
 *   w      = p[ids] / sum_j p[ids_j]                   renormalised       [T, K]
 *   group slots s = t*K + j by expert, stable in s; keep the first
 *   `capacity` slots of each expert (capacity <= 0: keep all)
 *   y_s    = W2[e] GELU(W1[e] x_t (+ b1[e])) (+ b2[e]) for kept slot s of expert e
 *   out[t] = sum_j w[t,j] * y_{t*K+j}   (dropped slots add nothing)
 *   aux    = E * sum_i (count_i / (T*K)) * (sum_t p[t,i] / T)
 *
 * Conventions for every call:
 *   - Tensor arguments are DEVICE pointers owned by the caller, dense and
 *     row-major, 16-byte aligned, unless a call says otherwise.  Weights are
 *     read-only.  The library keeps no pointer after a call returns.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Calls are
 *     asynchronous on it: they enqueue kernels and return.  They never
 *     allocate device memory and never synchronise, except moe_get_device_error.
 *   - `ws` is a caller-owned device workspace of at least moe_workspace_size()
 *     bytes, 256-byte aligned.  Calls that overlap on the GPU must not share one.
 *   - Return value: MOE_OK (0) or a negative moe_status.  Arguments are checked
 *     on the host before any launch; on error nothing is enqueued, except for
 *     MOE_ERR_CUDA (a launch failed; outputs are undefined).
 *   - Element types follow desc->dtype: MOE_BF16 -> x, Wg, W1, W2, x_perm,
 *     h_perm, y_perm and out are bf16; MOE_F32 -> all of them are fp32.
 *     Router logits, routing weights, biases and the loss are always fp32;
 *     indices and counts are int32.
 */
#ifndef MOE_GB300_H
#define MOE_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum moe_status {
  MOE_OK = 0,
  MOE_ERR_INVALID = -1,      /* bad argument: null pointer, shape, alignment */
  MOE_ERR_UNSUPPORTED = -2,  /* valid layer the library does not implement   */
  MOE_ERR_WORKSPACE = -3,    /* ws is NULL or smaller than moe_workspace_size */
  MOE_ERR_CUDA = -4,         /* a CUDA runtime / driver call failed          */
  MOE_ERR_TIMEOUT = -5,      /* a kernel gave up a bounded wait (device flag) */
  MOE_ERR_DEVICE = -6        /* a kernel's own bounds check fired (device flag) */
} moe_status;

typedef enum moe_dtype { MOE_F32 = 0, MOE_BF16 = 1 } moe_dtype;

/* desc->flags bits */
#define MOE_FLAG_HOST_IO    (1u << 0) /* moe_layer_forward: x and out are host pointers */
#define MOE_FLAG_SIMT_FFN   (1u << 1) /* bf16: CUDA-core expert FFN instead of tensor cores (testing) */
#define MOE_FLAG_NO_DECODE  (1u << 2) /* never take the small-batch weight-streaming FFN */
#define MOE_FLAG_SIMT_ROUTER (1u << 3) /* bf16: CUDA-core router instead of tensor cores (testing) */
#define MOE_FLAG_GEMM_SINGLE (1u << 4) /* bf16: 128x256 single-SM expert GEMM tiles */
#define MOE_FLAG_GEMM_PAIR   (1u << 5) /* bf16: 256x256 tiles on SM pairs (cta_group::2) */
#define MOE_FLAG_SWIGLU      (1u << 6) /* experts are W2 (SiLU(W1 x) * W3 x); see moe_expert_ffn */
/* Testing only: with MOE_FLAG_GEMM_SINGLE, every CTA of the first expert
 * product withholds its first operand load, so the MMA's bounded wait runs
 * out (about 2 s): the kernel records MOE_ERR_TIMEOUT in the workspace error
 * word, drains the loads it issued, frees its tensor memory and returns;
 * outputs are undefined.  It exercises the timeout path without a fault.
 * moe_expert_ffn_backward and moe_router_backward on the tensor cores do the
 * same: the barrier of each kernel's first stage waits for an arrival that
 * nobody makes (about 4 s a kernel, the drain's own wait running out too). */
#define MOE_FLAG_TEST_WAIT_TIMEOUT (1u << 7)
/* bf16 with SM pairs: every block of an expert's token rows runs with the
 * rows on the MMA's M side (padded to 256), instead of the default where an
 * expert's last, short block runs swapped (rows on the N side, padded to
 * 16).  Same results; for comparing the two (testing). */
#define MOE_FLAG_GEMM_ROWS   (1u << 8)
/* Run the two expert products as two launches.  By default one persistent
 * launch runs both.  On SM pairs a tile of the second product starts as
 * soon as the first product has written every hidden column of its 256-row
 * block, so the second product's tiles fill the first one's tail; in the
 * weight-streaming kernel of decode-sized batches the second product's
 * weights stream right behind the first's through the same ring, and its
 * activation rows load once every CTA of the expert has stored its share.
 * Same results; for comparing the two (testing). */
#define MOE_FLAG_FFN_SPLIT   (1u << 9)
/* drop_tokens = False (the Qwen2-MoE walkthrough, jsqmd.com, section 3.4:
 * tokens over an expert's capacity go to the next-best expert instead of
 * being dropped).  With a capacity, moe_layer_forward keeps the slots the
 * capacity keeps and moves each other slot, in slot order, to the
 * best-scored expert its token does not use yet that still has room (see
 * moe_reroute); a moved slot keeps its routing weight.  `count` and the loss
 * stay those of the routing's own choices; `dropped` counts the slots left
 * without an expert.  No effect without a capacity. */
#define MOE_FLAG_REROUTE     (1u << 10)
/* bf16, K <= 2, SM-pair expert GEMMs: moe_layer_forward folds the weighted
 * combine into the second expert product's epilogue (each output row adds
 * w * y, with y rounded to bf16 as stored, to an fp32 copy of out in the
 * workspace with vector reductions; two additions onto zero give the same
 * sum in either order, so the result is deterministic), then converts it to
 * out.  y_perm is not written.  Ignored where it does not apply.  For
 * comparing the two (the MoE sparse-activation article, wmrh.cn, section
 * 4.3, on the dispatcher's memory traffic). */
#define MOE_FLAG_FUSED_COMBINE (1u << 11)
/* bf16 batches of at most 16 tokens: moe_layer_forward runs the layer as
 * its separate steps (router, dispatch, weight-streaming expert products,
 * combine: four launches) instead of the default one-launch decode layer,
 * in which one grid with every CTA resident computes the gate scores,
 * routes and places every token in each CTA, spreads the used experts'
 * weight rows evenly over the CTAs and combines, with counters in the
 * workspace between the steps.  Same results, bit for bit; for comparing
 * the two (testing). */
#define MOE_FLAG_DECODE_SPLIT  (1u << 12)
/* bf16 layers on the SM-pair expert GEMMs, without MOE_FLAG_REROUTE:
 * moe_layer_forward runs no gather of x rows; the first expert product
 * copies each kept row's token row from x itself (slot s = src[r] of kept
 * row r is token s / K; Qwen2-MoE walkthrough, jsqmd.com, section 3.1 item
 * 3, grouping without a host-side sort), so x_perm is never written.  Same
 * results, bit for bit.  Ignored where it does not apply. */
#define MOE_FLAG_GATHER_GEMM   (1u << 13)

/*
 * Layer description.  Field names follow the Qwen2MoEConfig fields of the
 * Qwen2-MoE module article (mlqm.cn), section 2.2: E = num_experts,
 * K = num_experts_per_tok, capacity = expert_capacity.
 * Limits: T >= 0; 1 <= K <= 8; K <= E <= 256; H, F >= 8 and multiples of 8;
 * T * K < 2^31.
 * temperature: the router softmax is taken of l / temperature (the MoE
 * sparse-activation article, wmrh.cn, section 5.2: 1.0 by default, 2.0
 * flattens, 0.5 sharpens).  It changes the routing weights and the
 * load-balancing probabilities, not which experts are chosen.  <= 0 means 1;
 * NaN or infinity is MOE_ERR_INVALID.
 */
typedef struct moe_desc {
  int64_t T;         /* tokens (batch * sequence, flattened)                 */
  int32_t H;         /* hidden size                                          */
  int32_t E;         /* number of experts                                    */
  int32_t K;         /* experts chosen per token (top-k)                     */
  int32_t F;         /* expert FFN width                                     */
  int32_t capacity;  /* slots kept per expert; <= 0 means no limit           */
  int32_t dtype;     /* moe_dtype                                            */
  uint32_t flags;    /* MOE_FLAG_*                                           */
  float temperature; /* router softmax temperature; <= 0 means 1             */
} moe_desc;

/* Human-readable name of a status code (static storage). */
const char* moe_status_string(int status);

/* ceil(T / E) * K, the expert_capacity of the Qwen2-MoE module article
 * (mlqm.cn), section 2.2.  Returns -1 if E <= 0 or K <= 0. */
int64_t moe_capacity_default(int64_t T, int32_t E, int32_t K);

/* Rows of the permuted buffers (x_perm, h_perm, y_perm) needed for `desc`:
 * min(T*K, E*capacity) with a capacity, else T*K.  -1 if desc is invalid. */
int64_t moe_max_rows(const moe_desc* desc);

/* Bytes of device workspace every call below needs for `desc` (the same value
 * for all of them).  It holds routing results, dispatch tables, the permuted
 * activations and a device error word.  Returns MOE_ERR_INVALID for a bad desc. */
int moe_workspace_size(const moe_desc* desc, size_t* bytes);

/*
 * Router: gate linear, softmax, top-k, renormalisation (jsqmd.com section 3.1:
 * `gate` is nn.Linear(hidden, num_experts, bias=False), then F.softmax,
 * torch.topk and the division by the sum of the k weights; mlqm.cn section 3.2
 * steps 1-2).
 *   x         [T, H]  dtype
 *   Wg        [E, H]  dtype (nn.Linear [out, in] layout)
 *   gate_bias [E] fp32 or NULL (added to the scores; the pages' gate has none)
 *   logits    [T, E] fp32 out, or NULL: the scores l, fp32-accumulated (before
 *             the temperature is applied)
 *   ids       [T, K] int32 out: chosen experts, largest score first, equal
 *             scores ordered by ascending expert index
 *   w         [T, K] fp32 out: p[ids] / sum_j p[ids_j]  (sum to 1), with
 *             p = softmax(l / temperature)
 *   psum      [E] fp32 out, or NULL: sum over tokens of p[t, e], summed in a
 *             fixed order (deterministic)
 */
int moe_router_topk(const moe_desc* desc, const void* x, const void* Wg,
                    const float* gate_bias, float* logits, int32_t* ids,
                    float* w, float* psum, void* ws, size_t ws_bytes,
                    void* stream);

/*
 * Dispatch: group the T*K slots by expert (jsqmd.com section 3.1 item 3:
 * scatter + argsort by expert id) with the capacity rule of jsqmd.com section
 * 3.4 (tokens over an expert's capacity are dropped).  Slot s = t*K + j.
 * Within an expert, slots keep ascending s order, so with a capacity the
 * earliest tokens are kept.
 *   ids     [T, K] int32 in (each value in [0, E), or -1 for a slot with no
 *           expert, which is dropped; a token's other ids distinct)
 *   x       [T, H] dtype in, or NULL to skip the gather
 *   count   [E]    int32 out: slots routed to each expert, before dropping
 *   offs    [E+1]  int32 out: first permuted row of each expert; offs[E] = rows
 *   src     [moe_max_rows] int32 out: slot held by permuted row r (r < offs[E])
 *   pos     [T*K]  int32 out: permuted row of slot s, or -1 if dropped
 *   x_perm  [moe_max_rows, H] dtype out (if x != NULL): x_perm[r] = x[src[r] / K]
 *   dropped [1]    int32 out, or NULL: number of dropped slots
 * Out-of-range ids make the kernel set MOE_ERR_DEVICE in the workspace error
 * word (read it with moe_get_device_error); such slots are dropped.
 */
int moe_dispatch(const moe_desc* desc, const int32_t* ids, const void* x,
                 int32_t* count, int32_t* offs, int32_t* src, int32_t* pos,
                 void* x_perm, int32_t* dropped, void* ws, size_t ws_bytes,
                 void* stream);

/*
 * moe_dispatch without a workspace, for callers that cannot allocate device
 * memory where they route tokens: code running inside an allocator or memory-
 * pool callback, runtimes that reserve all device memory up front, plugin hosts
 * that forbid allocation on their execution path.  The pages have no
 * counterpart; this is a library convenience.
 *   Same arguments and results as moe_dispatch, minus ws/ws_bytes, plus
 *   device_error [1] int32 (device, or NULL): cleared by the call, then set to
 *   a nonzero code if an id is out of range (such slots are dropped).
 * The per-block histograms live in a 64 KiB array in device memory owned by
 * the library (held by every GPU that loads it until the process exits).  The
 * layer must fit it: E * blocks <= 8192, where for S = T*K slots
 * blocks = ceil(S / b), b = max(2048, ceil(S / 64)) rounded up to a multiple
 * of 256 (so at most 64 blocks: E <= 128 always fits, E = 256 up to
 * S = 65536); larger layers get MOE_ERR_UNSUPPORTED.  The call allocates
 * nothing.  Each call outside stream capture looks up the array's address on
 * the current device; a call during capture reuses the last one, so make the
 * first call on each device before any stream capture (and one more after a
 * device reset).  All calls on a device share the array: calls that overlap
 * on the GPU race and must be serialised by the caller.
 */
int moe_dispatch_noalloc(const moe_desc* desc, const int32_t* ids, const void* x,
                         int32_t* count, int32_t* offs, int32_t* src, int32_t* pos,
                         void* x_perm, int32_t* dropped, int32_t* device_error,
                         void* stream);

/*
 * Move the slots a capacity-limited dispatch dropped (drop_tokens = False;
 * the Qwen2-MoE walkthrough, jsqmd.com, section 3.4: tokens over capacity are
 * routed to the next-best expert instead of being dropped).  The slots the
 * capacity kept stay.  The others are taken one at a time in slot order
 * s = t*K + j; each goes to the expert with the highest score logits[t, e]
 * (equal scores: the lower index) that token t uses neither among its K
 * choices nor as the target of an earlier move, and that still has room
 * (capacity minus the slots it holds so far); if none has, the slot is
 * dropped.  The result equals that one-at-a-time walk exactly.
 *   logits  [T, E] fp32 in: the router's scores (moe_router_topk's logits)
 *   ids     [T, K] int32 in: the routing
 *   pos     [T*K]  int32 in: moe_dispatch's pos for ids with desc->capacity
 *                  (pos < 0: over capacity)
 *   offs    [E+1]  int32 in: moe_dispatch's offs for the same call
 *   ids_out [T, K] int32 out: each slot's expert after the moves, -1 if dropped
 *   dropped [1]    int32 out, or NULL: slots left without an expert
 * Dispatching ids_out again (moe_dispatch accepts -1 as "no expert") groups
 * the moved routing; no expert exceeds the capacity any more.  One block does
 * the walk: meant for capacities that drop a minority of the slots.
 */
int moe_reroute(const moe_desc* desc, const float* logits, const int32_t* ids, const int32_t* pos,
                const int32_t* offs, int32_t* ids_out, int32_t* dropped, void* ws, size_t ws_bytes,
                void* stream);

/*
 * Expert FFN over the permuted rows: for each expert e and each row r in
 * [offs[e], offs[e+1]):
 *   h_perm[r] = GELU(W1[e] x_perm[r] + b1[e])       (GELU erf form)
 *   y_perm[r] = W2[e] h_perm[r] + b2[e]
 * (mlqm.cn section 2.2: every expert is Linear - GELU - Linear).  On the bf16
 * path the products are accumulated in fp32 and h and y are rounded to bf16.
 *   x_perm [rows, H] dtype in; offs [E+1] int32 in (device; read on device only)
 *   W1 [E, F, H] dtype; W2 [E, H, F] dtype (nn.Linear [out, in] layout)
 *   b1 [E, F] fp32 or NULL; b2 [E, H] fp32 or NULL
 * With MOE_FLAG_SWIGLU the experts have three matrices W1, W2, W3 (the
 * Qwen2-MoE walkthrough, jsqmd.com, section 4.6), read as
 *   h_perm[r] = SiLU(W1[e] x + b1[e][:F]) * (W3[e] x + b1[e][F:])
 * and the W1 argument holds W1 and W3 stacked per expert: [E, 2F, H] (rows
 * 0..F-1 = W1, rows F..2F-1 = W3); b1 is then [E, 2F].
 *   h_perm [moe_max_rows, F] dtype out (intermediate, kept for inspection)
 *   y_perm [moe_max_rows, H] dtype out
 * bf16 with K-major operands runs on the tcgen05 tensor cores, either as
 * 128x256 tiles per SM or as 256x256 tiles per SM pair (chosen from the shape
 * unless a MOE_FLAG_GEMM_* flag forces one); fp32 runs on CUDA cores; T <= 16
 * runs a weight-streaming kernel (unless MOE_FLAG_NO_DECODE).
 */
int moe_expert_ffn(const moe_desc* desc, const void* x_perm, const int32_t* offs,
                   const void* W1, const float* b1, const void* W2, const float* b2,
                   void* h_perm, void* y_perm, void* ws, size_t ws_bytes,
                   void* stream);

/*
 * Combine: out[t] = sum_{j=0..K-1} w[t,j] * y_perm[pos[t*K+j]], summed in fp32
 * in the order j = 0..K-1, then stored in dtype; slots with pos < 0 add
 * nothing (jsqmd.com section 3.1 item 2; wmrh.cn section 2.2).  No residual.
 *   y_perm [rows, H] dtype; pos [T*K] int32; w [T, K] fp32; out [T, H] dtype
 */
int moe_combine(const moe_desc* desc, const void* y_perm, const int32_t* pos,
                const float* w, void* out, void* stream);

/*
 * Load-balancing loss (jsqmd.com section 3.3):
 *   loss = E * sum_i f_i * P_i,  P_i = psum[i] / T,  f_i = count[i] / (T*K).
 * The raw value is returned; the caller scales it by router_aux_loss_coef.
 *   psum [E] fp32; count [E] int32; loss [1] fp32 out (device)
 */
int moe_aux_loss(const moe_desc* desc, const float* psum, const int32_t* count,
                 float* loss, void* stream);

/*
 * The whole layer: router -> dispatch -> expert FFN -> combine (+ aux loss),
 * enqueued on one stream with no host synchronisation (mlqm.cn section 3.2).
 *   x [T, H], out [T, H] dtype: device pointers, or host pointers if
 *     desc->flags has MOE_FLAG_HOST_IO (then the call copies x in and out
 *     through the workspace; pinned host memory is fastest, and `out` is
 *     valid once `stream` has been synchronised).  With host pointers, no
 *     capacity and T >= 2048, the batch runs as two halves of tokens whose
 *     copies overlap the other half's layer (the second half's output is
 *     combined and copied back in two parts, the copy of the first part
 *     overlapping the combine of the second): the copies go on two internal
 *     streams (created on the first such call of each host thread on each
 *     device, kept until the process exits) joined to `stream` by events,
 *     the outputs are the same bits, and count and the loss are the whole
 *     batch's.
 *   aux [1] fp32 out or NULL; count [E] int32 out or NULL; dropped [1] int32
 *     out or NULL (device pointers)
 */
int moe_layer_forward(const moe_desc* desc, const void* x, const void* Wg,
                      const float* gate_bias, const void* W1, const float* b1,
                      const void* W2, const float* b2, void* out, float* aux,
                      int32_t* count, int32_t* dropped, void* ws, size_t ws_bytes,
                      void* stream);

/*
 * Training.  The gradient of the layer in its steps, for a program that ran
 * the forward pass with the separate calls above and kept what they wrote:
 *   moe_combine_backward -> moe_expert_ffn_backward -> moe_dispatch_backward
 * and the optimiser's step, moe_adamw_step.  The pages describe inference and
 * name training only in passing; these are the calculus of the formulas above.
 * Results must not overlap inputs, unless a call says otherwise.
 */

/*
 * Gradient of moe_combine: from dout, the gradient of out,
 *   dy_perm[pos[s]] = w[s] * dout[t]            for each kept slot s = t*K + j
 *   dw[s]           = <dout[t], y_perm[pos[s]]> in fp32; 0 for a dropped slot
 *   dout [T, H] dtype; y_perm [moe_max_rows, H] dtype (the forward pass's; not
 *   read if dw is NULL, may be NULL then); pos [T*K] int32; w [T, K] fp32
 *   dy_perm [moe_max_rows, H] dtype out or NULL: rows that no slot holds are
 *   left as they are
 *   dw [T, K] fp32 out or NULL
 * Deterministic.
 */
int moe_combine_backward(const moe_desc* desc, const void* dout, const void* y_perm, const int32_t* pos,
                         const float* w, void* dy_perm, float* dw, void* stream);

/*
 * Gradient of moe_dispatch's copy x_perm[pos[s]] = x[t]:
 *   dx[t] = sum_j dx_perm[pos[t*K + j]] (+ dx_add[t])
 * summed in fp32 over the kept slots in the order j = 0..K-1, then dx_add.
 *   dx_perm [moe_max_rows, H] dtype; pos [T*K] int32
 *   dx_add [T, H] dtype or NULL: what other paths of the same x have (the
 *   residual's, the gate's); may be dx itself
 *   dx [T, H] dtype out; a token without a kept slot gets dx_add, or zeros
 */
int moe_dispatch_backward(const moe_desc* desc, const void* dx_perm, const int32_t* pos, const void* dx_add,
                          void* dx, void* stream);

/* Bytes of device workspace moe_expert_ffn_backward needs for `desc`: the
 * error word (moe_get_device_error reads it; clear its 256 bytes once) and the
 * hidden gradients, which a call writes before it reads them.  Returns
 * MOE_ERR_INVALID for a bad desc. */
int moe_backward_workspace_size(const moe_desc* desc, size_t* bytes);

/*
 * Gradient of moe_expert_ffn.  For each expert e and its rows r in
 * [offs[e], offs[e+1]), with a = W1[e] x_perm[r] + b1[e] computed again:
 *   dh  = W2[e]^T dy_perm[r],  da = dh * GELU'(a)
 *   dx_perm[r] = W1[e]^T da
 *   dW1[e] = sum_r da x_perm[r]^T,     db1[e] = sum_r da
 *   dW2[e] = sum_r dy_perm[r] h_perm[r]^T,  db2[e] = sum_r dy_perm[r]
 * (zeros for an expert without a row).  With MOE_FLAG_SWIGLU a holds the
 * gate's and the up projection's columns, W1, b1, dW1 and db1 are stacked as
 * in moe_expert_ffn, and h = SiLU(gate) * up is what is differentiated.
 *   x_perm [moe_max_rows, H], h_perm [moe_max_rows, F] (as moe_expert_ffn wrote
 *   it; NULL if dW2 is), dy_perm [moe_max_rows, H] dtype; rows from offs[E] on
 *   may hold anything
 *   W1, b1 (nullable), W2: the forward pass's
 *   dx_perm [moe_max_rows, H] dtype out or NULL; rows from offs[E] on are left
 *   as they are
 *   dW1, dW2 dtype out, shaped as W1 and W2, or NULL; db1, db2 fp32 out
 *   ([E, F] or [E, 2F], and [E, H]) or NULL.  Results are written, not added.
 * On the bf16 path products are accumulated in fp32; da is rounded to bf16 as
 * an operand of the products after it (on CUDA cores it stays in fp32), the
 * bias gradients sum it before that.  The tensor cores' fp32 sums round
 * towards zero: db1, which is not rounded to bf16 after them, is about 1e-6
 * small.
 * Deterministic.  bf16 runs on the tensor cores, fp32 (and MOE_FLAG_SIMT_FFN)
 * on CUDA cores.  moe_max_rows + 256 (on CUDA cores + 64) has to stay below
 * 2^31: MOE_ERR_UNSUPPORTED.
 */
int moe_expert_ffn_backward(const moe_desc* desc, const void* x_perm, const void* h_perm, const void* dy_perm,
                            const int32_t* offs, const void* W1, const float* b1, const void* W2, void* dx_perm,
                            void* dW1, float* db1, void* dW2, float* db2, void* ws, size_t ws_bytes, void* stream);

/* Elements that share a scale in 8-bit moments. */
#define MOE_ADAMW_BLOCK 256

/*
 * One parameter tensor of moe_adamw_step: device pointers, n elements each,
 * aligned to their element (vector accesses are used where p, p_bf16, grad, m
 * and v are all 16-byte aligned).  Tensors of one call must not overlap.
 *   p [n] fp32; p_bf16 [n] bf16 or NULL: receives p rounded to bf16
 *   grad [n]: fp32 or bf16 (grad_dtype of the call)
 *   state_bits 32: m, v [n] fp32; m_scale, v_scale NULL
 *   state_bits 8: m, v [n] e4m3 codes of m and of sqrt(v); m_scale, v_scale
 *     [ceil(n / MOE_ADAMW_BLOCK)] fp32: a value is its code times the scale of
 *     its block of MOE_ADAMW_BLOCK elements, which is the block's largest
 *     magnitude / 448.  Zeroed buffers are the start.
 *   weight_decay: decoupled, for this tensor
 */
typedef struct moe_adamw_tensor {
  float* p;
  void* p_bf16;
  const void* grad;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  int64_t n;
  float weight_decay;
  int32_t reserved;      /* 0 */
} moe_adamw_tensor;

/* lr >= 0, 0 <= beta1, beta2 < 1, eps >= 0 (below 1e-30: taken as 0), all
 * finite; step = 1 for the first. */
typedef struct moe_adamw_params {
  double lr;
  double beta1;
  double beta2;
  double eps;
  int64_t step;
} moe_adamw_params;

/*
 * One AdamW step over `count` tensors, in place, in one launch for up to 400
 * of them:
 *   g = grad * (grad_scale ? *grad_scale : 1)
 *   m = beta1 m + (1 - beta1) g;  v = beta2 v + (1 - beta2) g^2
 *   p = p (1 - lr weight_decay)
 *       - lr / (1 - beta1^step) * m / (sqrt(v / (1 - beta2^step)) + eps)
 * in fp32, the moments of this step before they are rounded to 8 bits.
 *   tensors: host array, read during the call only
 *   grad_dtype: moe_dtype of every grad; state_bits: 32 or 8, for every tensor
 *   grad_scale [1] fp32 device or NULL (a clipping or loss-scale factor)
 *   skip [1] int32 device or NULL: nothing is changed if it is not 0
 * p's quotient is within 2 units of its last place.
 * 8-bit moments are rounded to nearest, code = e4m3(x * (1 / largest) * 448); a
 * block of moments with a NaN or an infinity reads back as NaN throughout
 * (guard it with skip).  A code moves only where one step changes its value,
 * as a share of its block's largest, by half a code (3 to 6 %).  For sqrt(v)
 * that takes a gradient of 8 to 11 times sqrt(v) with beta2 = 0.999, of 1.5 to
 * 1.9 times with 0.95, and it decays only as fast as its block's largest does:
 * 8 bits go with a beta2 of about 0.95 or below.
 */
int moe_adamw_step(const moe_adamw_tensor* tensors, int32_t count, int32_t grad_dtype, int32_t state_bits,
                   const moe_adamw_params* params, const float* grad_scale, const int32_t* skip, void* stream);

/*
 * Load-balancing loss over the tokens that count, and the statistics that its
 * gradient needs: with p = softmax(logits / temperature),
 *   tokens = the number n of tokens with mask[t] != 0 (T without a mask)
 *   count[e] = their slots with ids = e;  psum[e] = the sum of their p[t, e]
 *   loss = E * sum_e count[e] / (n K) * psum[e] / n       (0 if n = 0)
 * moe_aux_loss of a whole batch is the same number.  A token with mask[t] = 0
 * (the padding of a batch of sequences) takes no part, whatever its scores
 * and ids hold.
 *   logits [T, E] fp32; ids [T, K] int32: moe_router_topk's (an id of -1 counts
 *   for no expert)
 *   mask [T] bytes or NULL
 *   psum [E] fp32 out, count [E] int32 out, tokens [1] int32 out, loss [1] fp32
 *   out, or NULL each.  Ranks of a data-parallel batch add up the first three
 *   before they take the loss (moe_aux_loss) or its gradient.
 *   ws: of moe_router_backward_workspace_size() bytes
 * psum is summed in a fixed order, in fp32 over at most 2^13 tokens and with
 * twice its bits beyond.  An id outside [-1, E) of a token that counts sets MOE_ERR_DEVICE in
 * the workspace error word and counts for no expert.  Deterministic.
 */
int moe_balance_loss(const moe_desc* desc, const float* logits, const int32_t* ids, const uint8_t* mask,
                     float* psum, int32_t* count, int32_t* tokens, float* loss, void* ws, size_t ws_bytes,
                     void* stream);

/* Bytes of device workspace moe_balance_loss and moe_router_backward need for
 * `desc`; its first 256 bytes (the error word among them) have to be zeros
 * before the first call.  Returns MOE_ERR_INVALID for a bad desc. */
int moe_router_backward_workspace_size(const moe_desc* desc, size_t* bytes);

/*
 * Gradient of moe_router_topk's weights w and of moe_balance_loss, through the
 * softmax to the scores and through the gate's product to its matrix and x:
 *   dlogits[t, e] = 1 / temperature * (
 *       sum over j with ids[t, j] = e of w_j (dw[t, j] - sum_i w_i dw[t, i])
 *       + p_e (c_e - sum_i p_i c_i) ),   c_e = dloss E count[e] / (n^2 K)
 *   dWg = dlogits^T x,  dgate_bias = sum_t dlogits[t],  dx = dlogits Wg
 * with w computed again as the softmax over the scores of the token's ids.
 * Tokens with mask[t] = 0 have dlogits and dx of zeros and add nothing to dWg
 * and dgate_bias, whatever x, logits, ids and dw hold for them.
 *   x [T, H] dtype (not read if dWg is NULL, may be NULL then)
 *   Wg [E, H] dtype (not read if dx is NULL, may be NULL then)
 *   logits [T, E] fp32, ids [T, K] int32: the forward pass's; an id of -1 has
 *   no weight, an id outside [-1, E) the same, with MOE_ERR_DEVICE in the
 *   workspace error word
 *   dw [T, K] fp32 or NULL (no gradient of the weights): moe_combine_backward's
 *   dloss [1] fp32 device or NULL (no gradient of the loss): the loss' factor
 *   in what is minimised; then count [E] and tokens [1] (device): those of the
 *   loss, over every rank's tokens if the loss is; they may be NULL without it
 *   dlogits [T, E] fp32 out, dWg [E, H] fp32 out, dgate_bias [E] fp32 out,
 *   dx [T, H] dtype out, or NULL each, not all.  Results are written, not added:
 *   dx goes to moe_dispatch_backward as dx_add.
 * bf16: the products run on the tensor cores, dlogits split in three bf16 parts
 * for dWg (24 bits) and two for dx (2^-18 of each left out, less than what dx'
 * own rounding loses), fp32 sums.
 * fp32 and MOE_FLAG_SIMT_ROUTER: CUDA cores.  Deterministic.
 */
int moe_router_backward(const moe_desc* desc, const void* x, const void* Wg, const float* logits,
                        const int32_t* ids, const float* dw, const float* dloss, const int32_t* count,
                        const int32_t* tokens, const uint8_t* mask, float* dlogits, float* dWg, float* dgate_bias,
                        void* dx, void* ws, size_t ws_bytes, void* stream);

/*
 * Orthogonalised updates.  A matrix u [rows, cols] is made nearly orthogonal by
 * Newton-Schulz products: with X = u / |u| (Frobenius norm; zeros for a zero
 * matrix), transposed if rows > cols so that its rows are the short side,
 *   `iterations` times: A = X X^T;  X = (a I + b A + c A A) X
 *   (a, b, c) = (3.4445, -4.7750, 2.0315)
 * which takes every singular value that is not tiny into about [0.7, 1.2] (five
 * iterations: those above 1/500 of |u|).  X and the products are held in fp16
 * times 2^12, their sums in fp32.  That is as if each element of u were off by
 * up to 2^-12 of itself (a bf16 gradient is off by 2^-8): 1e-3 to 3e-3 of the
 * result in the 2-norm for gradients with strong directions over noise; what
 * lies far below the elements it is part of is off by more (2e-2 for a matrix
 * of rank one over noise 100 times smaller).  Matrices with a short side of up
 * to 16 and a long one of up to 4096 are held in fp32.  For large batches of
 * longer matrices (more columns than 5/4 of the rows) two iterations are taken
 * at a time, (B2 B1) X, and for batches of 2^23 elements X is held times the
 * norm over a power of two: bits then depend on the batch.  A matrix with a NaN
 * or an infinity becomes NaN throughout; the others of its batch do not.
 */
#define MOE_ORTHOGONALIZE_MAX_SIDE 32768       /* rows, cols <= this */
#define MOE_ORTHOGONALIZE_MAX_ITERATIONS 16
/* Testing, added to `iterations`: the first barrier of each kernel that waits
 * for its tensor cores waits for an arrival that nobody makes (2 s); the call
 * then ends as after any expired wait, with MOE_ERR_TIMEOUT in the workspace
 * error word.  Each element of out, or of p and its bf16 copy, has its old value
 * or its new one then, m the new one.  The next call in that workspace is not
 * affected. */
#define MOE_ORTHOGONALIZE_TEST_WAIT_TIMEOUT (1 << 30)

/* Bytes of device workspace moe_orthogonalize needs for `batch` matrices (a
 * large batch runs in parts of 4 GiB; matrices of up to 128 x 4096 stay on
 * chip and need 256 bytes); its first 256 bytes have to be zeros before the
 * first call. */
int moe_orthogonalize_workspace_size(int64_t batch, int32_t rows, int32_t cols, size_t* bytes);

/*
 * out[i] = x[i] made nearly orthogonal, for each of `batch` matrices.
 *   x, out [batch, rows, cols], of dtype x_dtype and out_dtype (moe_dtype),
 *   aligned to their element; out may be x if the dtypes are the same
 */
int moe_orthogonalize(const void* x, int32_t x_dtype, int64_t batch, int32_t rows, int32_t cols, int32_t iterations,
                      void* out, int32_t out_dtype, void* ws, size_t ws_bytes, void* stream);

/*
 * One parameter tensor of moe_muon_step: `batch` matrices [rows, cols] one
 * after the other (an expert's W1 each, say; SwiGLU's stacked W1 is 2 E
 * matrices [F, H]), each orthogonalised by itself.  Device pointers, aligned to
 * their element.  Tensors of one call must not overlap.
 */
typedef struct moe_muon_tensor {
  float* p;            /* [batch, rows, cols] fp32                             */
  void* p_bf16;        /* the same in bf16, or NULL: receives p rounded        */
  const void* grad;    /* fp32 or bf16 (grad_dtype of the call)                */
  float* m;            /* fp32 momentum; zeros are the start                   */
  int64_t batch;
  int32_t rows, cols;
  float weight_decay;  /* decoupled, for this tensor                           */
  float scale;         /* of its orthogonalised update, e.g. 0.2 sqrt(max(rows, cols)) */
} moe_muon_tensor;

/* lr >= 0, 0 <= momentum < 1, finite; nesterov 0 or 1; 1 <= iterations <=
 * MOE_ORTHOGONALIZE_MAX_ITERATIONS. */
typedef struct moe_muon_params {
  double lr;
  double momentum;
  int32_t nesterov;
  int32_t iterations;
} moe_muon_params;

/* Bytes of device workspace moe_muon_step needs for these tensors; its first
 * 256 bytes have to be zeros before the first call. */
int moe_muon_workspace_size(const moe_muon_tensor* tensors, int32_t count, size_t* bytes);

/*
 * One Muon step over `count` tensors, in place:
 *   g = grad * (grad_scale ? *grad_scale : 1)
 *   m = momentum m + g;   u = nesterov ? g + momentum m : m
 *   p = p (1 - lr weight_decay) - lr scale orthogonalize(u)
 * in fp32 but for the orthogonalisation (see above).  Matrices of one size,
 * whichever way round they lie, run together.
 *   tensors: host array, read during the call only
 *   grad_dtype: moe_dtype of every grad
 *   grad_scale [1] fp32 device or NULL; skip [1] int32 device or NULL: nothing
 *   is changed if it is not 0
 * Deterministic.
 */
int moe_muon_step(const moe_muon_tensor* tensors, int32_t count, int32_t grad_dtype, const moe_muon_params* params,
                  const float* grad_scale, const int32_t* skip, void* ws, size_t ws_bytes, void* stream);

/*
 * How many kernels one moe_layer_forward with this description launches
 * (no counterpart on the pages; it lets a caller or a benchmark account for
 * the launches it issues).  Depends on the shape only: the path taken
 * (one-block or multi-block dispatch, router variant) is chosen from it.
 * Returns the count (>= 1), or a negative MOE_ERR_* for an invalid desc.
 */
int moe_layer_launches(const moe_desc* desc);

/*
 * Which expert-FFN kernel moe_expert_ffn and moe_layer_forward run for this
 * description (no counterpart on the pages; it lets a caller or a benchmark
 * account for the launches and attribute time).  Depends on the shape and
 * flags only.  Returns one of MOE_FFN_*, or a negative MOE_ERR_* for an
 * invalid desc.
 */
#define MOE_FFN_STREAM    0 /* weight streaming for decode-sized batches, both products in 1 launch */
#define MOE_FFN_SIMT      1 /* CUDA cores (f32, or forced): 2 launches */
#define MOE_FFN_TC_SINGLE 2 /* tensor cores, 128x256 tiles per SM: 2 launches */
#define MOE_FFN_TC_PAIRS  3 /* tensor cores on SM pairs, one launch per product: 2 launches */
#define MOE_FFN_TC_FUSED  4 /* tensor cores on SM pairs, both products in 1 launch */
#define MOE_FFN_STREAM_SPLIT 5 /* weight streaming, one launch per product: 2 launches */
int moe_ffn_kernel(const moe_desc* desc);

/*
 * Whether moe_layer_forward runs this description as the one-launch decode
 * layer (see MOE_FLAG_DECODE_SPLIT): 1 if it does (two launches: its
 * counters zeroed, then the layer), 0 if it runs the separate steps, or a
 * negative MOE_ERR_* for an invalid desc.  No counterpart on the pages; it
 * lets a benchmark attribute the time.  Depends on the shape and flags only.
 */
int moe_layer_decode_fused(const moe_desc* desc);

/*
 * Stage timing for moe_layer_forward on the calling host thread (no
 * counterpart on the pages; a tracing aid in the spirit of the profiler runs
 * they describe).  `events` holds 6 cudaEvent_t created by the caller; each
 * later moe_layer_forward on this thread records them on its stream at the
 * stage boundaries: [0] start, [1] router done, [2] dispatch done, [3] first
 * expert product done, [4] second product done, [5] combine done.
 * events = NULL or n = 0 switches it off.  MOE_ERR_INVALID if n < 6 or an
 * event is NULL.
 */
int moe_profile_events(void* const* events, int n);

/*
 * Read and clear the workspace's device error word.  Synchronises `stream`.
 * *code receives MOE_OK, MOE_ERR_TIMEOUT (a tensor-core kernel gave up a
 * bounded wait) or MOE_ERR_DEVICE (an index check fired).  Returns MOE_OK or
 * MOE_ERR_CUDA.
 */
int moe_get_device_error(void* ws, int32_t* code, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GB300_H */
