/*
 * rdt.h -- C ABI of librdt.so: one training step of a Qwen3-style decoder
 * block stack on one GB300 (sm_103a).
 *
 * Operations follow the aprender-train ("entrenar") pages:
 *   cuda_block.rs   (0.32.0): CudaTransformerBlock::forward, ::backward,
 *                   compute_attention_cuda, optimizer_step;
 *   cuda_trainer.rs (0.34.0): train_step_inner (fused cross-entropy),
 *                   gpu_forward / gpu_backward (final norm + LM head),
 *                   compute_workspace_clip_scale_gpu and
 *                   fused_clip_workspace_gradients (squared-sum clip),
 *                   run_nonblock_optimizer_step (AdamW).
 *
 * Conventions shared by every call:
 *  - Pointers are DEVICE pointers unless marked "host". The caller owns and
 *    allocates every buffer; the library never allocates, frees or
 *    synchronises (except rdt_device_error, which says so).
 *  - `stream` is a cudaStream_t passed as void*. Work is enqueued on it and
 *    the call returns before the GPU finishes.
 *  - Outputs are overwritten, never accumulated into.
 *  - Matrices are row-major. Weights are [out, in]; a projection computes
 *    y = x W^T. Activations are token-major [T, width] with T = batch*seq and
 *    token t = b*seq + s at position s of sequence b.
 *  - rdt_bf16 is the bit pattern of a bfloat16. Dense contractions take bf16
 *    operands (round-to-nearest-even copies of the fp32 masters) and
 *    accumulate in fp32; norms, softmax, loss and optimizer math are fp32.
 *  - Every call returns an rdt_status. Host-detectable problems (null
 *    pointers, unsupported shapes, misaligned pointers, buffers too small)
 *    return RDT_EINVAL before anything is enqueued; a failed launch returns
 *    RDT_ECUDA. rdt_last_error() gives a thread-local message for the last
 *    failure. Device-side waits in the kernels are bounded: one that gives up
 *    records RDT_ETIMEOUT in the device error word read by
 *    rdt_device_error().
 */
#ifndef RDT_H_
#define RDT_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef uint16_t rdt_bf16;

typedef enum rdt_status {
  RDT_OK = 0,
  RDT_EINVAL = 1,      /* bad argument, shape, alignment or buffer size */
  RDT_ECUDA = 2,       /* a CUDA runtime call or kernel launch failed */
  RDT_ETIMEOUT = 3,    /* a bounded device wait gave up (rdt_device_error) */
  RDT_ENONFINITE = 4,  /* reserved for callers: non-finite gradient norm */
  RDT_EINDEX = 5,      /* a token id outside [0, vocab) met on the device
                          (rdt_device_error; its row was zeroed / skipped) */
} rdt_status;

/* Model shape. hidden, head_dim and intermediate must be multiples of 16,
 * head_dim one of 16, 32, 64, 128; n_heads a multiple of n_kv_heads;
 * hidden <= 4096. rms_eps is used by every RMSNorm, forward and backward.
 * RoPE-neox rotates pairs (i, i + head_dim/2) by pos * rope_theta^(-2i/head_dim). */
typedef struct rdt_config {
  int32_t hidden;
  int32_t n_heads;
  int32_t n_kv_heads;
  int32_t head_dim;
  int32_t intermediate;
  int32_t vocab;
  float rms_eps;
  float rope_theta;
} rdt_config;

/* ---------------------------------------------------------------------------
 * Parameter layout of one block. A block's trainable tensors live in ONE flat
 * fp32 array (the masters) in this order, each starting at the offset
 * rdt_block_param_offsets() reports (multiples of 16 elements):
 *   WQ [nh*d, H], WK [nkv*d, H], WV [nkv*d, H], WO [H, nh*d],
 *   WG [I, H], WU [I, H], WD [H, I], G_ATTN [H], G_FFN [H], G_Q [d], G_K [d].
 * WQ/WK/WV are adjacent, so together they form the stacked [nh*d+2*nkv*d, H]
 * matrix; WG/WU likewise form [2I, H]. The matching bf16 shadow and the
 * gradient array use the same layout.
 * ------------------------------------------------------------------------- */
enum {
  RDT_WQ = 0, RDT_WK, RDT_WV, RDT_WO, RDT_WG, RDT_WU, RDT_WD,
  RDT_G_ATTN, RDT_G_FFN, RDT_G_Q, RDT_G_K, RDT_BLOCK_NTENSORS
};

/* Validates cfg (RDT_EINVAL on an unsupported shape). */
rdt_status rdt_check_config(const rdt_config* cfg);

/* Element count of one block's flat parameter array (fp32 or bf16), or -1. */
int64_t rdt_block_param_count(const rdt_config* cfg);

/* Host arrays of RDT_BLOCK_NTENSORS entries: element offset and element
 * count of each tensor inside the block's flat array. */
rdt_status rdt_block_param_offsets(const rdt_config* cfg, int64_t* offsets, int64_t* counts);

/* Bytes of the activations rdt_block_forward saves for rdt_block_backward
 * (opaque layout, caller-allocated, 256-byte aligned). */
size_t rdt_block_saved_bytes(const rdt_config* cfg, int32_t batch, int32_t seq);
/* Scratch bytes of rdt_block_forward / rdt_block_backward (256-byte aligned). */
size_t rdt_block_workspace_bytes(const rdt_config* cfg, int32_t batch, int32_t seq);
/* Scratch bytes of rdt_fused_cross_entropy for `tokens` tokens: O(tokens *
 * H) plus one vocabulary chunk of at most 256 MB; it does not grow with
 * tokens * V (the logits are never stored whole). */
size_t rdt_head_workspace_bytes(const rdt_config* cfg, int32_t tokens);
/* Scratch bytes of rdt_sq_sum. */
size_t rdt_sq_sum_workspace_bytes(void);

/* ---------------------------------------------------------------------------
 * Block forward (CudaTransformerBlock::forward with compute_attention_cuda;
 * the fused residual + RMSNorm of the NF4 block's forward):
 *   xn = RMSNorm(x, G_ATTN); q,k,v = xn Wq^T, xn Wk^T, xn Wv^T;
 *   per head: RMSNorm over head_dim (G_Q / G_K), then RoPE-neox at the
 *   token's position in its own sequence;
 *   o = causal softmax(q k^T / sqrt(d)) v, query head h reading kv head
 *       h / (nh/nkv); r1 = x + o Wo^T; xn2 = RMSNorm(r1, G_FFN);
 *   y = r1 + (silu(xn2 Wg^T) * (xn2 Wu^T)) Wd^T.
 * w      fp32 masters of this block (flat layout; the gains are read here)
 * w_bf16 bf16 shadow of the same layout (matrices are read here)
 * x, y   fp32 [batch*seq, hidden]; y must not alias x
 * saved  rdt_block_saved_bytes() bytes, written; keep for the backward
 * ws     rdt_block_workspace_bytes() bytes of scratch
 * ------------------------------------------------------------------------- */
rdt_status rdt_block_forward(const rdt_config* cfg, int32_t batch, int32_t seq,
                             const float* w, const rdt_bf16* w_bf16,
                             const float* x, float* y,
                             void* saved, size_t saved_bytes,
                             void* ws, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Block backward (CudaTransformerBlock::backward: backward_ffn,
 * backward_post_attn_norm, backward_attention with the GQA reduction and the
 * inverse RoPE, backward_residual_and_input_norm; the per-head QK-norm
 * backward and its gain gradients, which that path leaves out, are included).
 * x      the block's forward input, fp32 [T, H]
 * saved  what rdt_block_forward wrote for the same x and w
 * dy     upstream gradient fp32 [T, H]
 * dx     gradient w.r.t. x, fp32 [T, H] (overwritten; may alias dy)
 * grads  fp32 flat array in the block layout: every tensor overwritten
 *        (accumulate == 0) or added to (accumulate == 1: gradient
 *        accumulation over micro-batches, GpuGradientAccumulator in
 *        cuda_trainer.rs, here done in place by the gradient producers)
 * grad_sq  optional (may be null) fp64 device scalar: *grad_sq += the sum of
 *          the squares of every gradient this call leaves in grads (after
 *          the accumulation, so pass it on a step's last micro-batch only;
 *          the global-norm clip's squared sum, accumulated by the
 *          weight-gradient GEMMs' epilogues and the gain reductions as they
 *          produce the values; fixed summation order, so the same inputs give
 *          the same bits)
 * ------------------------------------------------------------------------- */
rdt_status rdt_block_backward(const rdt_config* cfg, int32_t batch, int32_t seq,
                              const float* w, const rdt_bf16* w_bf16,
                              const float* x, const void* saved, size_t saved_bytes,
                              const float* dy, float* dx, float* grads, int32_t accumulate,
                              double* grad_sq, void* ws, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Final RMSNorm + LM head + cross-entropy, forward and backward in one call
 * (train_step_inner's fused cross-entropy; gpu_forward's final norm and LM
 * head; gpu_backward's LM-head and final-norm backward; KAIZEN-050/052's
 * fused CE). The logits are never stored whole, on the device or the host:
 * the vocabulary is walked in chunks of at most 256 MB of bf16 dz; each chunk's
 * logits are formed in the GEMMs' fp32 tensor-memory accumulators, once for
 * the log-sum-exp and the target's logit (forward) and once more for dz,
 * computed in fp32 from the saved log-sum-exp (backward). Nothing but the
 * caller's copy of loss_partials reaches the host.
 *   hn = RMSNorm(h, gamma_f); z = hn W_lm^T;
 *   loss_partials[t] = logsumexp(z_t) - z_t[targets[t]]   (unscaled NLL);
 *   dz = (softmax(z_t) - onehot(targets[t])) * loss_scale;
 *   dh, dgamma_f, dw_lm = gradients of sum_t loss_scale * loss_partials[t].
 * h        fp32 [tokens, H], the last block's output
 * gamma_f  fp32 [H]; w_lm bf16 [V, H]
 * targets  int32 [tokens], device; each must lie in [0, V) (not checked on
 *          the device: the caller validates ids before upload)
 * loss_scale  normally 1/tokens (loss = mean NLL); 1/(tokens * n) for each of
 *          n accumulated micro-batches (train_step_inner divides by
 *          accumulation_steps)
 * dh fp32 [tokens, H] (overwritten); dgamma_f fp32 [H] and dw_lm fp32 [V, H]
 *          overwritten (accumulate == 0) or added to (accumulate == 1)
 * grad_sq  optional (may be null) fp64 device scalar: *grad_sq = the sum of
 *          the squares of dgamma_f and dw_lm as this call leaves them (a
 *          step's backward starts here, so this call starts the clip's
 *          squared sum that each rdt_block_backward then adds to; pass it on
 *          the last micro-batch only when accumulating)
 * ------------------------------------------------------------------------- */
rdt_status rdt_fused_cross_entropy(const rdt_config* cfg, int32_t tokens,
                                   const float* h, const float* gamma_f,
                                   const rdt_bf16* w_lm, const int32_t* targets,
                                   float loss_scale, float* loss_partials,
                                   float* dh, float* dgamma_f, float* dw_lm, int32_t accumulate,
                                   double* grad_sq, void* ws, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Squared-sum gradient clip (compute_workspace_clip_scale_gpu,
 * fused_clip_workspace_gradients; contract C-CLIP-001).
 * rdt_sq_sum: *sumsq = sum over the nbuf buffers of sum(g^2), accumulated in
 *   fp64 (fp32 within a thread's short run). bufs and lens are HOST arrays of
 *   device pointers / element counts; each buffer 16-byte aligned.
 * rdt_clip_scale: norm = sqrt(*sumsq) (the squared sums are not squared
 *   again); *scale = max_norm / norm if norm > max_norm else 1;
 *   *nonfinite = 1 if norm is not finite (then *scale = 1), else 0.
 * ------------------------------------------------------------------------- */
rdt_status rdt_sq_sum(const float* const* bufs, const int64_t* lens, int32_t nbuf,
                      double* sumsq, void* ws, size_t ws_bytes, void* stream);
rdt_status rdt_clip_scale(const double* sumsq, float max_norm, float* scale,
                          int32_t* nonfinite, void* stream);

/* rdt_sq_sum for callers that cannot allocate device memory (code inside an
 * allocator or pool callback, a runtime whose footprint is fixed once it
 * starts, a plugin whose host gives it no scratch buffer). The pages have no
 * counterpart of this call: it exists for those callers only. Same result as
 * rdt_sq_sum; no workspace argument and no allocation of any kind. Its
 * scratch is a fixed 32 KiB array (4096 fp64 partial sums) inside librdt.so
 * that every GPU loading the library keeps until the process exits; any total
 * length fits in it, and more than 64 buffers per call is rejected with
 * RDT_EINVAL. The first call on a device looks up the array's device address
 * (make that first call before any stream capture). Every call shares the one
 * array, so calls that may overlap on the GPU (different streams, or
 * different host threads on one device) race and must be serialised by the
 * caller; each call rewrites every partial it reads, so nothing needs
 * clearing in between. */
rdt_status rdt_sq_sum_noalloc(const float* const* bufs, const int64_t* lens, int32_t nbuf,
                              double* sumsq, void* stream);

/* ---------------------------------------------------------------------------
 * AdamW over n contiguous fp32 elements (optimizer_step's adamw_step_cuda;
 * step counted from 1 as run_nonblock_optimizer_step does):
 *   g' = scale * g; m = b1 m + (1-b1) g'; v = b2 v + (1-b2) g'^2;
 *   w = w - lr * ( (m/(1-b1^step)) / (sqrt(v/(1-b2^step)) + eps) + wd * w ).
 * scale     device fp32 scalar from rdt_clip_scale, or NULL for 1
 * skip_flag device int32, or NULL; when *skip_flag != 0 nothing is written
 * w_bf16    if not NULL, receives the bf16 (RNE) copy of the updated w
 * step_dev  if not NULL, a device int32 holding the step (>= 1) that the
 *           kernel reads instead of `step` (which is then ignored): a step
 *           count that lives on the device, so a captured CUDA graph of the
 *           training step can be replayed unchanged (see rdt_step_advance)
 * w, g, m, v, w_bf16 16-byte aligned. step >= 1 unless step_dev is given.
 * rdt_step_advance: *step += 1 on the device, in stream order.
 * ------------------------------------------------------------------------- */
rdt_status rdt_adamw_step(float* w, const float* g, float* m, float* v, int64_t n,
                          const float* scale, const int32_t* skip_flag, int32_t step,
                          const int32_t* step_dev, float lr, float beta1, float beta2,
                          float eps, float weight_decay, rdt_bf16* w_bf16, void* stream);
rdt_status rdt_step_advance(int32_t* step, void* stream);

/* The tensor-core GEMM every projection of the path runs on, exposed so it
 * can be tested on its own: C[M, N] (fp32, row stride ldc) = A' B'^T over K,
 * with A' = A ([M, K], row stride lda) when a_mn == 0, or the transpose of A
 * given as [K, M] when a_mn == 1; likewise B' = B ([N, K]) or B^T with B
 * given as [K, N]. A, B bf16; lda, ldb multiples of 8; ldc a multiple of 4.
 * split_ws (optional, 16-byte aligned, split_ws_floats fp32 elements): scratch
 * that lets a problem with too few 128 x 256 output tiles to fill the GPU run
 * as K-slices whose partials are then summed in slice order (the NF4 block's
 * adapter GEMMs take this path); null: one pass over K. */
rdt_status rdt_gemm(const rdt_bf16* A, int32_t a_mn, int64_t lda, const rdt_bf16* B,
                    int32_t b_mn, int64_t ldb, int32_t M, int32_t N, int32_t K, float* C,
                    int64_t ldc, float* split_ws, int64_t split_ws_floats, void* stream);

/* The NF4 GEMM of the NF4-frozen block (CudaNf4TransformerBlock in
 * cuda_block.rs: frozen projection weights stored as packed 4-bit NormalFloat
 * codes with one fp32 scale per 64-element block), exposed for tests:
 * C[M, N] (fp32, row stride ldc) = A [M, K1] (bf16, lda) times B^T, plus an
 * optional tail A2 [M, K2] times B2^T (K2 <= 64; the LoRA term folded in as
 * extra K). W is [w_rows, w_cols] row-major: codes uint8 [w_rows, w_cols/2]
 * (element 2j in the low nibble of byte j), scales fp32 [w_rows, w_cols/64];
 * W = level[code] * scale, levels the 16 NormalFloat-4 values of QLoRA.
 * b_mn == 0: B = W (N = w_rows, K1 = w_cols; y = x W^T), B2 [N, K2] (ldb2);
 * b_mn == 1: B = W^T (N = w_cols, K1 = w_rows; dX = dY W), B2 [K2, N].
 * w_cols % 256 == 0 and w_rows % 64 == 0; leading dimensions in elements,
 * bf16 ones multiples of 8, ldc a multiple of 4; 16-byte aligned pointers.
 * split_ws (optional, as in rdt_gemm): scratch for running the problem as
 * K-slices when its tiles would leave most of the GPU idle. */
rdt_status rdt_gemm_nf4(const rdt_bf16* A, int64_t lda, const uint8_t* codes,
                        const float* scales, int64_t w_rows, int64_t w_cols, int32_t b_mn,
                        const rdt_bf16* A2, int64_t lda2, const rdt_bf16* B2, int64_t ldb2,
                        int32_t K2, int32_t M, float* C, int64_t ldc, float* split_ws,
                        int64_t split_ws_floats, void* stream);

/* dst[i] = bf16(src[i]) with round-to-nearest-even; n elements, 16-byte aligned. */
rdt_status rdt_cast_bf16(const float* src, rdt_bf16* dst, int64_t n, void* stream);

/* ---------------------------------------------------------------------------
 * NF4-frozen block with LoRA adapters (CudaNf4TransformerBlock in
 * cuda_block.rs: the seven projection weights frozen as packed 4-bit
 * NormalFloat codes, one fp32 scale per block of 64 consecutive elements of
 * the row-major [out, in] weight; lora_scale = alpha / rank as in
 * cuda_trainer.rs; lora_forward in wgpu_trainer.rs: y = x W^T +
 * (alpha/rank) (x A^T) B^T with A [rank, in], B [out, rank]). The block is
 * the block above with every projection replaced by that LoRA projection on
 * the dequantized W = level[code] * scale (levels: the 16 NormalFloat-4
 * values of QLoRA); the norm gains are frozen and only the adapters get
 * gradients.
 *
 * Constraints (rdt_nf4_check): rdt_check_config's, hidden, n_heads*head_dim
 * and intermediate multiples of 256, n_kv_heads*head_dim a multiple of 64,
 * rank 8 or 16 (the stacked Q/K/V adapters, 3*rank columns, fit one 64-deep
 * GEMM step).
 *
 * codes   uint8, the seven projections' packed codes back to back in the
 *         order q, k, v, o, gate, up, down, each [out, in/2] row-major with
 *         element 2j in the low nibble of byte j (rdt_nf4_offsets: byte offsets)
 * scales  fp32, the seven projections' block scales in the same order, each
 *         [out, in/64] (rdt_nf4_offsets: element offsets)
 * gains   fp32 [hidden | hidden | head_dim | head_dim]: input-norm,
 *         post-attention-norm, q-norm and k-norm gains (frozen)
 * lora    fp32 adapters, tensors RDT_LORA_* back to back (rdt_lora_param_offsets);
 *         A's are [rank, in], B's [out, rank]
 * shadow  bf16 operand copy of the adapters the GEMMs read, rdt_lora_shadow_count
 *         elements, written by rdt_lora_shadow from lora (call it after every
 *         update of lora)
 * ------------------------------------------------------------------------- */
enum {
  RDT_LORA_A_Q, RDT_LORA_A_K, RDT_LORA_A_V, RDT_LORA_A_O, RDT_LORA_A_G, RDT_LORA_A_U,
  RDT_LORA_A_D, RDT_LORA_B_Q, RDT_LORA_B_K, RDT_LORA_B_V, RDT_LORA_B_O, RDT_LORA_B_G,
  RDT_LORA_B_U, RDT_LORA_B_D, RDT_LORA_NTENSORS
};

/* RDT_OK when cfg and rank meet the constraints above, else RDT_EINVAL. */
rdt_status rdt_nf4_check(const rdt_config* cfg, int32_t rank);
/* Total code bytes / scale elements of the seven projections (-1 if invalid). */
int64_t rdt_nf4_code_bytes(const rdt_config* cfg);
int64_t rdt_nf4_scale_count(const rdt_config* cfg);
/* Host arrays of 7 entries (q, k, v, o, gate, up, down): byte offsets into
 * codes and element offsets into scales. */
rdt_status rdt_nf4_offsets(const rdt_config* cfg, int64_t* code_offsets, int64_t* scale_offsets);
/* Adapter layout: element count; host arrays of RDT_LORA_NTENSORS offsets and counts. */
int64_t rdt_lora_param_count(const rdt_config* cfg, int32_t rank);
rdt_status rdt_lora_param_offsets(const rdt_config* cfg, int32_t rank, int64_t* offsets,
                                  int64_t* counts);
/* bf16 elements of the adapters' operand copy; rdt_lora_shadow writes it. */
int64_t rdt_lora_shadow_count(const rdt_config* cfg, int32_t rank);
rdt_status rdt_lora_shadow(const rdt_config* cfg, int32_t rank, const float* lora,
                           rdt_bf16* shadow, void* stream);
/* Saved-activation and scratch bytes of the NF4 block calls (256-byte aligned). */
size_t rdt_nf4_saved_bytes(const rdt_config* cfg, int32_t rank, int32_t batch, int32_t seq);
size_t rdt_nf4_workspace_bytes(const rdt_config* cfg, int32_t rank, int32_t batch, int32_t seq);

/* Forward of the NF4 + LoRA block: x, y fp32 [batch*seq, hidden] (y must not
 * alias x); saved written for rdt_nf4_block_backward. */
rdt_status rdt_nf4_block_forward(const rdt_config* cfg, int32_t rank, float alpha, int32_t batch,
                                 int32_t seq, const uint8_t* codes, const float* scales,
                                 const float* gains, const rdt_bf16* shadow, const float* x,
                                 float* y, void* saved, size_t saved_bytes, void* ws,
                                 size_t ws_bytes, void* stream);
/* Backward of the NF4 + LoRA block: dx fp32 [batch*seq, hidden] (may alias
 * dy); lora_grads fp32 in the adapter layout, every tensor overwritten;
 * grad_sq optional (may be null): *grad_sq += the sum of the squares of the
 * adapter gradients (fixed summation order). The frozen weights and gains get
 * no gradient. */
rdt_status rdt_nf4_block_backward(const rdt_config* cfg, int32_t rank, float alpha,
                                  int32_t batch, int32_t seq, const uint8_t* codes,
                                  const float* scales, const float* gains,
                                  const rdt_bf16* shadow, const float* x, const void* saved,
                                  size_t saved_bytes, const float* dy, float* dx,
                                  float* lora_grads, double* grad_sq, void* ws, size_t ws_bytes,
                                  void* stream);

/* ---------------------------------------------------------------------------
 * Measurement hooks (host-side bookkeeping only; no device memory).
 * rdt_gemm_timing_arm: while armed, the i-th tensor-core GEMM launch (any
 *   entry point) records the caller-created cudaEvent_t events[2i] on its
 *   stream just before the launch and events[2i+1] just after it, and stores
 *   its algorithmic FLOP count 2*M*N*K in flops[i] and, when kinds is not
 *   null, its kernel in kinds[i] (0: bf16 single-CTA tiles, 1: bf16 CTA-pair
 *   tiles, 2: NF4-decoding kernel; host arrays), for i < capacity. rdt_gemm_timing_disarm stops it and returns the number of
 *   launches seen (which may exceed capacity; only the first capacity are
 *   recorded).
 * rdt_launch_count: kernels this process has launched through the library
 *   so far (all entry points, all devices). */
rdt_status rdt_gemm_timing_arm(void* const* events, double* flops, int32_t* kinds,
                               int32_t capacity);
int64_t rdt_gemm_timing_disarm(void);
int64_t rdt_launch_count(void);

/* ---------------------------------------------------------------------------
 * Token embedding on the device (cuda_trainer.rs: gpu_forward's embedding
 * lookup and embed_backward's scatter-add, C-EMBED-GRAD-001, both of which
 * the pages run on the host).
 * rdt_embedding_forward: x[t, :] = table[ids[t], :]; table fp32 [vocab,
 *   hidden] (hidden % 4 == 0), ids int32 [tokens] on the device, x fp32
 *   [tokens, hidden]. An id outside [0, vocab) gives a zero row and records
 *   RDT_EINDEX in the device error word.
 * rdt_embedding_backward: dtable[id, :] = (accumulate == 0: every row first
 *   zeroed) or += scale * sum over the tokens t with ids[t] == id of
 *   dx[t, :], the sum taken in token order (deterministic, no atomics);
 *   scale an optional device fp32 scalar (null: 1), normally the activation
 *   gradient's own clip scale from rdt_sq_sum + rdt_clip_scale
 *   (C-EMBED-GRAD-001); ids outside [0, vocab) are skipped. ws: device
 *   scratch of rdt_embedding_workspace_bytes(tokens) bytes, 256-byte aligned.
 * ------------------------------------------------------------------------- */
size_t rdt_embedding_workspace_bytes(int32_t tokens);
rdt_status rdt_embedding_forward(const float* table, int64_t vocab, int32_t hidden,
                                 const int32_t* ids, int32_t tokens, float* x, void* stream);
rdt_status rdt_embedding_backward(const int32_t* ids, int32_t tokens, const float* dx,
                                  int32_t hidden, const float* scale, float* dtable,
                                  int64_t vocab, int32_t accumulate, void* ws, size_t ws_bytes,
                                  void* stream);

/* ---------------------------------------------------------------------------
 * Log probabilities of given tokens from logits, with entropy, log-sum-exp and
 * the most likely alternatives, and their gradient. The fused cross-entropy
 * above returns a target's NLL together with the gradient of its mean; these
 * calls are for what needs the values themselves or another loss: scoring,
 * distillation, policy training, sampling reports.
 *
 * A row z of `vocab` logits stands for the distribution p = softmax(logit_scale
 * z); logit_scale is 1 / temperature, in [1e-6, 1e6]. Logits are fp32, bf16 or
 * fp16, [rows, vocab] with row stride ld elements (ld >= vocab, any alignment
 * an element has), vocab in [1, 2^30]; all arithmetic is fp32.
 *
 * rdt_token_logprobs, for each row t:
 *   logp[t]     = ln p[targets[t]]
 *   entropy[t]  = -sum_j p_j ln p_j
 *   lse[t]      = ln sum_j exp(logit_scale z_j)
 *   stats[2t]   = max_j z_j, stats[2t + 1] = lse[t] - logit_scale max_j z_j:
 *                 what the gradient needs (lse alone loses digits when the
 *                 logits are large)
 *   top_ids / top_logp [t * top + i]: id and ln p of the i-th largest logit,
 *                 equal logits in order of id; `top` in [0, RDT_MAX_TOP]
 * Each output may be null (logp needs targets; top_ids and top_logp go
 * together, with top >= 1); at least one is given.
 *  - targets int32 [rows], or null: no logp, every row is computed. A row with
 *    targets[t] < 0 is not scored, whatever its logits (where rows are many
 *    they are not even read): its outputs are 0 and its ids -1. targets[t] >= vocab gives logp NaN.
 *  - A logit of -inf is a masked token: p = 0, never an alternative; a masked
 *    target has logp -inf. Where fewer than `top` tokens are left, the rest
 *    has id -1 and ln p -inf. A row with every token masked has lse, logp,
 *    stats[2t] and top_logp -inf, entropy and stats[2t + 1] 0, ids -1.
 *  - A row that holds a NaN or +inf has NaN outputs and ids -1.
 * rows may be 0. logits and outputs must not overlap.
 *
 * rdt_token_logprobs_backward: the gradient of sum_t (d_logp[t] logp[t] +
 * d_entropy[t] entropy[t] + d_lse[t] lse[t]) with respect to the logits,
 *   d_logits[t, j] = logit_scale ( [j = targets[t]] d_logp[t]
 *        + p_j (d_lse[t] - d_logp[t] - d_entropy[t] (ln p_j + entropy[t])) ),
 * rounded once to d_dtype. logits, logit_scale and targets as in the forward,
 * stats and entropy as it wrote them. d_logp, d_entropy, d_lse fp32 [rows],
 * each may be null for 0 but not all; d_logp needs targets, d_entropy needs
 * entropy. d_logits [rows, vocab] with row stride ld_d; it may be the logits
 * themselves (same pointer, type and stride), else they must not overlap.
 * Rows not scored (targets[t] < 0) or with every token masked get zeros;
 * targets[t] >= vocab and rows with NaN stats get NaN.
 * ------------------------------------------------------------------------- */
typedef enum rdt_dtype { RDT_F32 = 0, RDT_BF16 = 1, RDT_F16 = 2 } rdt_dtype;
#define RDT_MAX_TOP 32

rdt_status rdt_token_logprobs(const void* logits, int32_t dtype, int64_t ld, int32_t rows,
                              int32_t vocab, float logit_scale, const int32_t* targets,
                              float* logp, float* entropy, float* lse, float* stats, int32_t top,
                              int32_t* top_ids, float* top_logp, void* stream);
rdt_status rdt_token_logprobs_backward(const void* logits, int32_t dtype, int64_t ld,
                                       int32_t rows, int32_t vocab, float logit_scale,
                                       const int32_t* targets, const float* stats,
                                       const float* entropy, const float* d_logp,
                                       const float* d_entropy, const float* d_lse, void* d_logits,
                                       int32_t d_dtype, int64_t ld_d, void* stream);

/* Final RMSNorm + LM head + rdt_token_logprobs: scores hidden states with the
 * head of rdt_fused_cross_entropy, without its gradients.
 *   hn = bf16(RMSNorm(h, gamma_f)); z = hn W_lm^T in fp32, a chunk of rows at
 *   a time (at most 1 GiB of logits, and at least 128 rows).
 * h fp32 [tokens, H], gamma_f fp32 [H], w_lm bf16 [V, H]; the other arguments
 * as in rdt_token_logprobs. ws: rdt_head_logprobs_workspace_bytes(cfg, tokens)
 * bytes of scratch, 256-byte aligned (0 for an unsupported cfg). */
size_t rdt_head_logprobs_workspace_bytes(const rdt_config* cfg, int32_t tokens);
rdt_status rdt_head_logprobs(const rdt_config* cfg, int32_t tokens, const float* h,
                             const float* gamma_f, const rdt_bf16* w_lm, float logit_scale,
                             const int32_t* targets, float* logp, float* entropy, float* lse,
                             int32_t top, int32_t* top_ids, float* top_logp, void* ws,
                             size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * One clip and AdamW update of many tensors at once (rdt_sq_sum and
 * rdt_adamw_step take 64 buffers and one flat buffer): parameters that live in
 * allocations of their own, with a learning rate and weight decay each, fp32
 * or bf16 gradients, and moments in 32 bits or in 8.
 *
 * tensors is a HOST array of `count` entries (0 to 1,000,000), read before the
 * call returns. An entry with n == 0 is skipped. Device pointers 16-byte
 * aligned, scales 4-byte aligned; no two entries may share memory that the
 * call writes (entries whose w overlap are rejected).
 *
 * rdt_tensors_sq_sum: *sumsq = sum over all g of g^2, relative error
 *   below 1e-12, for any number of values, where each square is 0 or at least
 *   1e-30 and the sum at most 1e38 (it is formed in fp32 with the rounding
 *   errors kept; a larger one may come out as not finite); order of summation
 *   fixed by the sizes. Only g and n of each entry are read, so entries may
 *   share memory here. For rdt_clip_scale. ws:
 *   rdt_tensors_sq_sum_workspace_bytes(tensors, count) bytes, 8-byte aligned.
 *
 * rdt_tensors_adamw, step t (>= 1, or *step_dev), each operation rounded to
 * fp32 in this order (the quotient by a reciprocal, relative error below
 * 2^-22):
 *   g' = g scale;  m = b1 m + (1 - b1) g';  v = b2 v + ((1 - b2) g') g'
 *   w = w (1 - lr weight_decay) - (m / (sqrt(v) / sqrt(1 - b2^t) + eps)) (lr / (1 - b1^t))
 * with b1 and b2 in [0, 1) and eps in [1e-30, 1e30]
 * (1 - b1, 1 - b2, 1 / (1 - b1^t) and 1 / sqrt(1 - b2^t) are formed in double
 * and rounded once; sqrt(v) is multiplied by the last.) w_bf16, where not
 * null, receives the bf16 copy of w. scale, skip_flag and step_dev as in
 * rdt_adamw_step; with *skip_flag != 0 nothing is written.
 *
 * state_bits 32: m and v are fp32 [n]; m_scale and v_scale are not read.
 * state_bits 8: m and v are e4m3 codes, one byte per element; each run of 256
 *   elements of a tensor (the last may be shorter) has one scale in m_scale
 *   and v_scale, fp32 [ceil(n / 256)]. m = code m_scale. v's codes hold its
 *   square root: sqrt(v) = code v_scale, whose range of exponents is half of
 *   v's. A scale is the run's largest magnitude / 448, and a code is rounded
 *   from value (1 / largest) 448; a run whose largest is below 2^-100 is
 *   stored as zeros. The update uses the new m and v before they are rounded.
 *   A sqrt(v) > 0 never becomes code 0, so no later step divides by eps alone.
 *   Zeroed codes and scales are the initial state.
 *   seed < 0: codes are rounded to nearest even. seed in [0, 2^32): rounded up
 *   or down with the probability of the distance, from 16 bits that are a
 *   function of (seed, step, index of the entry, index of the element): on
 *   average the state is the value itself, to 2^-16 of a code's step, so that
 *   changes smaller than half a code (a decay of v by 1 - b2) are not lost. A
 *   sqrt(v) below the smallest code (2^-9) is stored as that code each time.
 *   Ignored for 32 bits.
 *   A NaN in g makes its element NaN; an infinite g makes its run of 256 NaN
 *   (rdt_clip_scale's nonfinite flag, passed as skip_flag, prevents both).
 * ------------------------------------------------------------------------- */
typedef struct rdt_opt_tensor {
  float* w;
  const void* g;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  rdt_bf16* w_bf16;
  int64_t n;
  float lr;
  float weight_decay;
} rdt_opt_tensor;

size_t rdt_tensors_sq_sum_workspace_bytes(const rdt_opt_tensor* tensors, int32_t count);
rdt_status rdt_tensors_sq_sum(const rdt_opt_tensor* tensors, int32_t count, int32_t g_dtype,
                              double* sumsq, void* ws, size_t ws_bytes, void* stream);
rdt_status rdt_tensors_adamw(const rdt_opt_tensor* tensors, int32_t count, int32_t g_dtype,
                             int32_t state_bits, int64_t seed, const float* scale,
                             const int32_t* skip_flag, int32_t step, const int32_t* step_dev,
                             float beta1, float beta2, float eps, void* stream);

/* ---------------------------------------------------------------------------
 * Attention for packed documents, prompts, windows and single tokens, and the
 * per-head norm with rotation that feeds it. The block calls above do both for
 * a dense batch of causal sequences of equal length, at positions 0, 1, ...;
 * here every token has positions of its own and every query a span of keys.
 *
 * A tensor of heads is [tokens, heads, head_dim] with the head_dim values
 * contiguous: element (t, h, i) at data + t token_stride + h head_stride + i,
 * strides in elements, at least head_dim, multiples of 16 bytes, data 16-byte
 * aligned. So q, k and v may lie together as a projection wrote them, or head
 * by head. The stride of an axis with one element is not looked at.
 * ------------------------------------------------------------------------- */
typedef struct rdt_heads {
  void* data;
  int64_t token_stride;
  int64_t head_stride;
} rdt_heads;

/* rdt_qk_norm_rope: for every head of q and k, with x its head_dim values,
 *   n = x / sqrt(mean(x^2) + eps) gain                 (gain null: n = x)
 *   out_i = n_i cos a - n_{i+d/2} sin a,  out_{i+d/2} = n_{i+d/2} cos a + n_i sin a,
 *   a = positions[axis(i)][t] theta^(-2i / head_dim)    (positions null: out = n)
 * in fp32, rounded once to out_dtype. positions int32 [axes, tokens], any
 * value; axes in [1, 4]. sections is a HOST array of `axes` counts that add up
 * to head_dim / 2: the first sections[0] pairs turn by axis 0, the next
 * sections[1] by axis 1, and so on; null with one axis. An angle is that of the
 * pair's rate theta^(-2i / head_dim) as rounded in 64 bits (2^-51 of the rate),
 * and exact to 2^-31 of a half turn beside that, however far the position.
 * head_dim a multiple of 16 in [16, 256]; n_heads and n_kv_heads in [0, 4096],
 * not both 0 (a tensor without heads is not looked at and may be null);
 * gain_q, gain_k fp32 [head_dim]; eps >= 0; theta > 0. tokens may be 0.
 * An output may be its input itself (same address, type and strides), else
 * outputs overlap neither inputs nor each other.
 *
 * rdt_qk_norm_rope_backward: gradients with respect to q, k and the gains from
 * d_q_out and d_k_out (of type d_dtype); q and k are the forward's inputs. dq
 * and dk of type out_dtype; they may be q and k, or d_q_out and d_k_out,
 * themselves. d_gain_q and d_gain_k fp32 [head_dim], each may be null, = or
 * (accumulate != 0) += the sum over tokens and heads, its order fixed by the
 * sizes. ws: rdt_qk_norm_rope_backward_workspace_bytes() bytes, 256-byte
 * aligned; not looked at when neither gain gradient is wanted. */
rdt_status rdt_qk_norm_rope(int32_t tokens, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                            const rdt_heads* q, const rdt_heads* k, int32_t dtype,
                            const float* gain_q, const float* gain_k, float eps,
                            const int32_t* positions, int32_t axes, const int32_t* sections,
                            float theta, const rdt_heads* q_out, const rdt_heads* k_out,
                            int32_t out_dtype, void* stream);
size_t rdt_qk_norm_rope_backward_workspace_bytes(int32_t tokens, int32_t n_heads,
                                                 int32_t n_kv_heads, int32_t head_dim);
rdt_status rdt_qk_norm_rope_backward(int32_t tokens, int32_t n_heads, int32_t n_kv_heads,
                                     int32_t head_dim, const rdt_heads* q, const rdt_heads* k,
                                     int32_t dtype, const float* gain_q, const float* gain_k,
                                     float eps, const int32_t* positions, int32_t axes,
                                     const int32_t* sections, float theta,
                                     const rdt_heads* d_q_out, const rdt_heads* d_k_out,
                                     int32_t d_dtype, const rdt_heads* dq, const rdt_heads* dk,
                                     int32_t out_dtype, float* d_gain_q, float* d_gain_k,
                                     int32_t accumulate, void* ws, size_t ws_bytes, void* stream);

/* rdt_attention: query t sees the keys j with lo[t] <= j < hi[t] (and
 * 0 <= j < keys). For every query head h, which reads kv head h / (n_heads /
 * n_kv_heads),
 *   s_j = scale q_t . k_j,  and with softcap > 0  s_j = softcap tanh(s_j / softcap)
 *   o_t = sum_j p_j v_j,  p = softmax of the s_j it sees,  lse_t = ln sum_j exp(s_j).
 * A query that sees nothing has o = 0 and lse = -inf. Spans give a causal
 * batch, packed documents, a prompt that is seen whole, a sliding window, or
 * new tokens against a cache: any mask in which a query sees a run of keys.
 * lo and hi int32 [queries], device memory; lo null: 0, hi null: keys.
 * What a query does not see does not reach its results, whatever it holds
 * (nor a key's gradients what does not see it, unless a query that does is not
 * finite itself); where an infinity that it sees makes a result not finite, that
 * may be NaN. NaN or infinities in memory that no query sees make a call a few
 * times as long; in keys (queries) that some queries (keys) of a neighbourhood see
 * and others do not, the others' rows are computed one by one, by one warp each:
 * some 16 us for 32 keys seen, 30 us for 32 queries and heads.
 * The cost goes by the keys between the least lo and the largest hi of
 * neighbouring queries, so queries of one document belong together.
 *
 * q, k, v, o bf16, head_dim a multiple of 16 in [16, 128]; n_heads a multiple
 * of n_kv_heads, at most 128 times it, at most 4096; queries and keys in
 * [0, 2^30]. n_kv_heads times the groups of floor(128 / (n_heads / n_kv_heads))
 * queries, and times the groups of 128 keys, at most 2^29. scale in
 * [1e-6, 1e6]; softcap 0 (none) or scale times [1e-5, 1e5]. Scores, softmax and
 * sums are fp32, p is rounded to bf16 for its product with v. lse fp32 [queries,
 * n_heads], natural logarithm; may be null. Outputs overlap nothing else. ws:
 * rdt_attention_workspace_bytes(..., 0) bytes, 256-byte aligned (may be 0
 * bytes). Results do not depend on scheduling.
 *
 * rdt_attention_backward: gradients of sum(d_o o) + sum(d_lse lse) with
 * respect to q, k and v, those of k and v summed over the query heads that
 * share them, each rounded once to bf16; p and the scores' gradients are rounded
 * to bf16 for their products. o and lse as rdt_attention wrote
 * them; d_o bf16, d_lse fp32 [queries, n_heads] or null. Rows that nothing
 * sees or that see nothing get zeros. ws:
 * rdt_attention_workspace_bytes(..., 1) bytes, 256-byte aligned. */
size_t rdt_attention_workspace_bytes(int32_t queries, int32_t keys, int32_t n_heads,
                                     int32_t n_kv_heads, int32_t head_dim, int32_t backward);
rdt_status rdt_attention(int32_t queries, int32_t keys, int32_t n_heads, int32_t n_kv_heads,
                         int32_t head_dim, const rdt_heads* q, const rdt_heads* k,
                         const rdt_heads* v, const int32_t* lo, const int32_t* hi, float scale,
                         float softcap, const rdt_heads* o, float* lse, void* ws, size_t ws_bytes,
                         void* stream);
rdt_status rdt_attention_backward(int32_t queries, int32_t keys, int32_t n_heads,
                                  int32_t n_kv_heads, int32_t head_dim, const rdt_heads* q,
                                  const rdt_heads* k, const rdt_heads* v, const rdt_heads* o,
                                  const float* lse, const rdt_heads* d_o, const float* d_lse,
                                  const int32_t* lo, const int32_t* hi, float scale, float softcap,
                                  const rdt_heads* dq, const rdt_heads* dk, const rdt_heads* dv,
                                  void* ws, size_t ws_bytes, void* stream);

/* Thread-local description of the last failure on this thread ("" if none). */
const char* rdt_last_error(void);

/* Test hook for the bounded device waits (the error path the tensor-core
 * kernels take when a wait gives up; cuda_trainer.rs train_step_inner
 * reports a poisoned CUDA context after a device failure, which these bounds
 * avoid). Launches one warp on `stream` that holds 32 tensor-memory columns,
 * waits on an mbarrier with a limit of limit_ns nanoseconds (in [1e3, 1e10]),
 * then frees the columns and returns whatever the outcome. arrive != 0: the
 * warp arrives on the barrier first, so the wait completes at once;
 * arrive == 0: nothing arrives, the wait gives up after limit_ns and records
 * RDT_ETIMEOUT in the device error word (read it with rdt_device_error).
 * waited_ns: optional device uint64 that receives the wait's duration.
 * RDT_EINVAL for an out-of-range limit or a misaligned waited_ns. */
rdt_status rdt_wait_probe(int64_t limit_ns, int32_t arrive, uint64_t* waited_ns, void* stream);

/* Synchronises the current device, then reads and clears the device error
 * word of the current device (0 = none, else an rdt_status such as
 * RDT_ETIMEOUT). Writes it to *code (host). */
rdt_status rdt_device_error(int32_t* code);

#ifdef __cplusplus
}
#endif
#endif /* RDT_H_ */
