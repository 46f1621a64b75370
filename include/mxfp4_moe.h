/*
 * mxfp4_moe.h -- the mixture-of-experts serving calls of libmxfp4 (GB300,
 * sm_103a): residual sum + RMSNorm with an MXFP8 output, routing of tokens to
 * experts, and the experts' products of MXFP8 activations with MXFP4 weights.
 *
 * The conventions of mxfp4.h hold for every call here (device pointers, caller
 * owned memory, no allocation and no synchronization, work enqueued on
 * `stream`, arguments checked on the host before anything is enqueued, bounded
 * waits reported through mxfp4_get_device_error), except that a call may be
 * given zero tokens, which enqueues nothing and returns MXFP4_OK.
 *
 * MXFP8 matrix [R, K]: E4M3 values, one byte each, row-major, and one E8M0
 * scale byte b (2^(b-127)) per 32 elements along K, in the 128x4 blocked
 * layout of mxfp4.h, mxfp4_sf_bytes(R, K, 32) bytes. Quantization here takes
 * the smallest power of two 2^e, e >= -127, with amax <= 448 * 2^e over the 32
 * values (so that nothing saturates; amax = 0 gives byte 0) and rounds x * 2^-e
 * to E4M3, ties to even. A block that holds a NaN or an infinity gets the scale
 * byte 0xFF (NaN), so that whatever is computed from it is NaN.
 *
 * Overlap of consecutive calls: every launch uses programmatic dependent
 * launch, but none reads or writes anything before the kernels that were in the
 * stream before the call have completed (the later launches of one call may
 * read weights while an earlier one of it runs), so all inputs, weights too, are
 * read in stream order.
 */
#ifndef MXFP4_MOE_GB300_H
#define MXFP4_MOE_GB300_H

#include "mxfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of bf16 / fp16 / fp32 inputs. */
#define MXFP4_DTYPE_BF16 0
#define MXFP4_DTYPE_FP16 1
#define MXFP4_DTYPE_FP32 2

/* Residual sum, RMSNorm and MXFP8 quantization of rows X [M, K] (bf16 or fp16):
 *   h   = X + residual, in fp32, rounded to the element type (residual NULL: h = X)
 *   r   = 1 / sqrt(mean_k(h_k^2) + eps), good to 2^-42, for rows of any finite size; r = 0
 *         where every h_k^2 is below fp32 (2^-149) and K eps too; an infinite h gives NaN in
 *         its place and zeros in the rest of its row
 *   y_k = h_k * r * weight_k (Y: in fp32, then rounded)
 *   Aq, A_sf = MXFP8 of y (see above), the codes and scales of 64-bit arithmetic (values
 *         of y below 2^-126: of fp32); pad cells of A_sf are written with 0x7F.
 *   X, residual, weight, H, Y : element type `dtype` (MXFP4_DTYPE_BF16 / _FP16).
 *   weight : [K], 16-byte aligned.
 *   H   : out, [M, K], h (NULL: not stored). May be X or residual itself (same
 *         pointer and stride): a row is read whole before it is written.
 *   Y   : out, [M, K], y rounded to the element type (NULL: not stored).
 *   Aq  : out, uint8 [M, K] E4M3, row stride ldq bytes.
 * M >= 0; K a positive multiple of 32. Strides ldx, ldr, ldh, ldy in elements,
 * multiples of 8; ldq a multiple of 8; X, residual, H, Y 16-byte aligned, Aq 8,
 * A_sf 4. eps finite and >= 0. Outputs must not overlap anything else. */
MXFP4_API mxfp4_status_t mxfp8_add_rmsnorm_quantize(const void *X, int64_t ldx, const void *residual, int64_t ldr,
                                                    const void *weight, int dtype, float eps, int64_t M, int64_t K,
                                                    void *H, int64_t ldh, void *Y, int64_t ldy, void *Aq,
                                                    int64_t ldq, void *A_sf, void *stream);

#define MOE_SCORE_SOFTMAX 0
#define MOE_SCORE_SIGMOID 1
#define MOE_MAX_EXPERTS 512
#define MOE_MAX_TOPK 32

/* Routing: for every token t, from logits z [T, E],
 *   s_e = softmax(z)_e or 1 / (1 + exp(-z_e));   c_e = s_e + bias_e (bias NULL: s_e)
 *   with groups > 1: experts e * groups / E form the groups; a group's score is
 *     the sum of its group_top (1 or 2) largest c; only the experts of the
 *     topk_groups best groups stay
 *   ids [t, :]     = the k experts with the largest c, largest first
 *   weights [t, :] = s of those, divided by (their sum + 1e-20) if renormalize,
 *                    times scale
 * Equal scores go to the lower index, in groups and in experts. The choice is
 * that of 64-bit arithmetic: it is taken in 32 bits with an error bound, and
 * again in 64 bits for rows in which that bound leaves it open. Without a bias
 * and without groups the experts are ranked by their logits, which rank them as
 * their scores do, but also where scores saturate. A NaN score ranks first.
 * The weights are computed in fp32 from the chosen logits: good to 2^-17 of
 * themselves at worst, 2^-24 on average; a score below 2^-126 may count as 0.
 * An expert whose logit is -inf is not chosen: a slot for which no expert is
 * left gets id -1 and weight 0 (a row of -inf: all of them).
 *   logits : [T, E] of type dtype (bf16, fp16, fp32), row stride ldl elements, aligned to its type.
 *   bias   : fp32 [E] or NULL.   ids : out, int32 [T, k].   weights : out, fp32 [T, k].
 * T >= 0; 1 <= E <= MOE_MAX_EXPERTS; groups divides E; 1 <= topk_groups <= groups;
 * 1 <= k <= min(MOE_MAX_TOPK, topk_groups * E / groups); scale finite. */
MXFP4_API mxfp4_status_t moe_route(const void *logits, int dtype, int64_t ldl, int64_t T, int E, const float *bias,
                                   int score, int groups, int topk_groups, int group_top, int k, int renormalize,
                                   float scale, int32_t *ids, float *weights, void *stream);

/* Workspace bytes of mxfp4_moe_experts for T tokens of k choices among E
 * experts, hidden size H, intermediate size I (0 for sizes that it refuses). It
 * grows with T: one made for the largest T serves smaller ones too. */
MXFP4_API size_t mxfp4_moe_experts_workspace_bytes(int64_t T, int k, int E, int64_t H, int64_t I);

/* The experts' products of a mixture-of-experts layer: for every token t
 *   out[t] = bf16_rne( sum_j weights[t, j] * ( act_j . W2[e]^T ) ),  e = ids[t, j],
 *   act_j  = MXFP8( silu(x_t . G[e]^T) * (x_t . U[e]^T) ),   silu(g) = g / (1 + exp(-g)),
 * summed in the order of j in fp32; all products accumulate in fp32 on the
 * tensor cores (tcgen05.mma kind::mxf8f6f4); silu is good to (5 + 1.2 |g|) 2^-23
 * of its value, and 0 for g < -87.3. A choice whose id is outside
 * [0, E) is left out (experts of other devices, slots without one); a token
 * with no choice left gets zeros.
 *   Xq, X_sf : MXFP8 activations [T, H], row stride ldx bytes.
 *   ids      : int32 [T, k].     weights : fp32 [T, k].
 *   W13q     : packed E2M1 [E, 2I, H/2], contiguous: the I rows of G, then those of U.
 *   W13_sf   : E blocked E8M0 buffers of mxfp4_sf_bytes(2I, H, 32) bytes, one after another.
 *   W2q      : packed E2M1 [E, H, I/2], contiguous;  W2_sf : E buffers of mxfp4_sf_bytes(H, I, 32).
 *   out      : bf16 [T, H], row stride ldo elements.
 * T >= 0; H and I positive multiples of 128 up to 2^20; 1 <= k <= MOE_MAX_TOPK;
 * 1 <= E <= MOE_MAX_EXPERTS; T * k < 2^30; 2 I E, H E, (T k / 32 + E) (I / 64) and
 * (T k / 32 + E) (H / 128) < 2^31 (the workspace query refuses the same sizes). Xq 16-byte aligned with ldx a multiple of 16;
 * W13q and W2q 32-byte aligned; scales 16; out 16 with ldo a multiple of 8;
 * workspace 256. The workspace needs no initialisation and keeps nothing from
 * one call for the next; calls that share one must not overlap. */
MXFP4_API mxfp4_status_t mxfp4_moe_experts(const void *Xq, int64_t ldx, const void *X_sf, const int32_t *ids,
                                           const float *weights, const void *W13q, const void *W13_sf,
                                           const void *W2q, const void *W2_sf, void *out, int64_t ldo, int64_t T,
                                           int k, int E, int64_t H, int64_t I, void *workspace, size_t ws_bytes,
                                           void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MXFP4_MOE_GB300_H */
