/*
 * mxfp4_layer.h -- the calls of libmxfp4 (GB300, sm_103a) around a decoder
 * layer's attention when many requests are served at once: low-rank adapters
 * beside a shared projection, the norm and rotation of queries and keys, and the
 * whole mixture-of-experts half of a layer for a few tokens.
 *
 * The conventions of mxfp4_moe.h hold for every call here (device pointers,
 * caller-owned memory, no allocation and no synchronization, work enqueued on
 * `stream`, arguments checked on the host before anything is enqueued, zero
 * tokens enqueue nothing and give MXFP4_OK, and every input is read in stream
 * order). Element types are the MXFP4_DTYPE_ constants of that header.
 */
#ifndef MXFP4_LAYER_GB300_H
#define MXFP4_LAYER_GB300_H

#include "mxfp4_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LORA_MAX_ADAPTERS 4096
#define LORA_MAX_RANK 256

/* Workspace bytes of lora_add for T tokens of width K and L adapters of rank up
 * to R (0 for sizes that it refuses). It grows with each of the four: one made
 * for the largest serves smaller ones too. */
MXFP4_API size_t lora_workspace_bytes(int64_t T, int64_t K, int R, int L);

/* Low-rank adapters of many requests beside a projection they share: for every
 * token t whose adapter is a = ids[t],
 *   C[t, n] = round( base[t, n] + scales[a] * sum_{r < ranks[a]} u[r] * B[a, n, r] ),
 *   u[r]    = sum_k X[t, k] * A[a, r, k],
 * both sums in fp32 and one rounding, to C's type; between the products scales[a] * u[r]
 * is held to 2^-17 of itself or 2^-134 (as two bf16; infinite beyond bf16's largest, and an infinity
 * in B may come out as NaN). A token whose id is outside [0, L) has no adapter: its row of C is that
 * of base. Elements of A and B at or beyond an adapter's rank are not used, whatever they hold.
 *   X      : bf16 [T, K], row stride ldx.     base, C : [T, N] of type dtype (bf16 or fp16),
 *            row strides ldb and ldc; C may be base itself (same pointer and stride).
 *   A      : bf16 [L, R, K], contiguous.      B : bf16 [L, N, R], contiguous.
 *   ids    : int32 [T], in any order.         scales : fp32 [L] or NULL (1).
 *   ranks  : int32 [L] or NULL (all R); taken as 0 below 0 and as R above R.
 * T >= 0; 1 <= L <= LORA_MAX_ADAPTERS; R a multiple of 8 up to LORA_MAX_RANK; K and N
 * positive multiples of 8 up to 2^30; T up to 2^30. C must not overlap anything but
 * base in its own place. Strides in elements, multiples of 8;
 * X, base, C, A, B 16-byte aligned; ids, scales, ranks 4; workspace 256. The
 * workspace needs no initialisation and keeps nothing from one call for the next;
 * calls that share one must not overlap. */
MXFP4_API mxfp4_status_t lora_add(const void *X, int64_t ldx, const void *A, const void *B, const int32_t *ids,
                                  const float *scales, const int32_t *ranks, const void *base, int64_t ldb, int dtype,
                                  void *C, int64_t ldc, int64_t T, int64_t K, int64_t N, int R, int L, void *workspace,
                                  size_t ws_bytes, void *stream);

/* Norm and rotation of queries and keys, one pass: for every token t and head x of
 * q [T, Hq, D] and k [T, Hk, D],
 *   y   = x / sqrt(mean(x^2) + eps) * weight     (weight NULL: y = x)
 *   out = y with the pairs (y_i, y_j) of its first `rot` elements turned by the token's angle i:
 *         (y_i cos - y_j sin, y_j cos + y_i sin),  j = i + rot / 2, or with `interleaved`
 *         the pair i is (2i, 2i + 1),
 * in fp32 with one rounding. Rows of any finite size are normalized; where mean + eps is 0 the
 * result is 0; an infinite x gives NaN in its place, and its pair's if it turns, and zeros in the rest of its
 * head. Without a weight an infinity or NaN reaches no element but those two, and elements that
 * nothing turns keep their bits (a NaN stays some NaN).
 *   table     : fp32 [P, rot], row p: the rot / 2 cosines, then the rot / 2 sines of position p.
 *   positions : int32 [T] (pos64 0) or int64 [T] (pos64 1). A position outside [0, P) gives
 *               NaN in all of its token's outputs.
 *   q, k, q_out, k_out : type dtype (bf16 or fp16), rows of D; strides in elements between
 *               tokens (st) and heads (sh), any multiples of 8, so that views of a joint
 *               projection need no copy; an output's such that no two of its heads share elements
 *               (refused otherwise). An output may be its own input (same pointer and strides) and
 *               overlaps nothing else.
 *   q_weight, k_weight : type dtype [D], or NULL; elements 0 or 2^-40 to 2^40 in size.
 * T, Hq, Hk >= 0 (zero heads: that tensor is not touched); D a positive multiple of 8 up to 256;
 * 0 <= rot <= D, a multiple of 16, with `interleaved` of 8 (rot 0: no table and no positions);
 * T * (Hq + Hk) < 2^31; eps finite and >= 0. Tensors, weights and table 16-byte aligned. */
MXFP4_API mxfp4_status_t qk_norm_rope(const void *q, int64_t q_st, int64_t q_sh, const void *k, int64_t k_st,
                                      int64_t k_sh, const void *q_weight, const void *k_weight, const float *table,
                                      const void *positions, int pos64, int dtype, float eps, int64_t T, int Hq, int Hk,
                                      int D, int rot, int interleaved, int64_t P, void *q_out, int64_t qo_st,
                                      int64_t qo_sh, void *k_out, int64_t ko_st, int64_t ko_sh, void *stream);

#define MOE_LAYER_MAX_TOKENS 16

/* Workspace bytes of mxfp4_moe_layer (0 for sizes that it refuses). It grows with
 * T: one made for the largest T serves smaller ones too. */
MXFP4_API size_t mxfp4_moe_layer_workspace_bytes(int64_t T, int k, int E, int64_t H, int64_t I);

/* The feed-forward half of a mixture-of-experts layer for up to MOE_LAYER_MAX_TOKENS
 * tokens, in four launches (for more tokens: mxfp8_add_rmsnorm_quantize, the router's
 * product, moe_route and mxfp4_moe_experts):
 *   h       = X + residual, in fp32, rounded to bf16 (residual NULL: h = X)
 *   y       = h / sqrt(mean(h^2) + eps) * weight, in fp32 (0 where mean + eps is 0)
 *   logits  = y . router^T, of y unrounded, good to 2^-20 of the sum of their terms' sizes
 *   ids, weights = moe_route of those logits (see there for score .. scale), but decided by
 *             scores in fp32, good to 2^-20 beside what the logits' error makes of them: of two
 *             choices that lie closer than these errors either may come first
 *   out[t]  = bf16_rne( sum_j weights[t, j] * ( act_j . W2[e]^T ) ),  e = ids[t, j],
 *   act_j   = MXFP8( silu(q . G[e]^T) * (q . U[e]^T) ),  q = MXFP8(y),
 * with sums, silu and the order of the weighted sum as in mxfp4_moe_experts; the codes of y
 * and act are those of fp32 arithmetic, and enter the products exactly, but for blocks of 32 whose
 * largest is below 2^-111: those values to 2^-127 each. Rows of h of any finite size are normalized; an infinite h gives
 * NaN in its token. Infinities and NaN stay in their tokens.
 *   X, residual, H : bf16 [T, Hd], row strides ldx, ldr, ldh. H (out, NULL: not stored)
 *                    may be X or residual itself (same pointer and stride).
 *   weight : bf16 [Hd], elements 0 or 2^-40 to 2^40 in size.    bias : fp32 [E] or NULL.
 *   router : bf16 [E, Hd], contiguous, elements up to 2^20 in size.
 *   W13q, W13_sf, W2q, W2_sf : as in mxfp4_moe_experts, Hd and I its H and I.
 *   out    : bf16 [T, Hd], row stride ldo; may be X or residual where H is not.
 *   ids, out_weights : out, int32 and fp32 [T, k], or NULL.
 * 0 <= T <= MOE_LAYER_MAX_TOKENS; the other sizes as in moe_route and mxfp4_moe_experts.
 * Strides in elements, multiples of 8; X, residual, H, out, weight, router and scales 16-byte
 * aligned; W13q and W2q 32; workspace 256. eps finite and >= 0. The workspace needs
 * no initialisation and keeps nothing from one call for the next; calls that
 * share one must not overlap. */
MXFP4_API mxfp4_status_t mxfp4_moe_layer(const void *X, int64_t ldx, const void *residual, int64_t ldr,
                                         const void *weight, float eps, const void *router, const float *bias, int score,
                                         int groups, int topk_groups, int group_top, int k, int renormalize, float scale,
                                         const void *W13q, const void *W13_sf, const void *W2q, const void *W2_sf,
                                         void *H, int64_t ldh, void *out, int64_t ldo, int32_t *ids, float *out_weights,
                                         int64_t T, int E, int64_t Hd, int64_t I, void *workspace, size_t ws_bytes,
                                         void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MXFP4_LAYER_GB300_H */
