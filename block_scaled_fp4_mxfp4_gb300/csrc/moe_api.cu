// extern "C" entry points of include/mxfp4_moe.h: argument validation, tensor
// maps and workspace layout. Nothing here allocates device memory or
// synchronizes.
#include <cmath>
#include <cstring>

#include "internal.h"
#include "moe.h"
#include "mxfp4_moe.h"

using namespace mxfp4;

namespace {

inline bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline mxfp4_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MXFP4_OK : MXFP4_ERR_CUDA; }

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;

mxfp4_status_t check_moe_sizes(int64_t T, int k, int E, int64_t H, int64_t I)
{
    if (T < 0 || k < 1 || E < 1 || H < 1 || I < 1) return MXFP4_ERR_INVALID_ARG;
    if (k > MOE_MAX_TOPK || E > MOE_MAX_EXPERTS || H % 128 != 0 || I % 128 != 0) return MXFP4_ERR_UNSUPPORTED_SHAPE;
    // sorted rows and weight rows are 32-bit coordinates
    if (T > (int64_t(1) << 30) || T * k >= (int64_t(1) << 30)) return MXFP4_ERR_UNSUPPORTED_SHAPE;
    if (H > (int64_t(1) << 20) || I > (int64_t(1) << 20) || 2 * I * E > kMaxDim || H * E > kMaxDim)
        return MXFP4_ERR_UNSUPPORTED_SHAPE;
    // units of work: token tiles x weight tiles
    const int64_t tiles = T * k / 32 + E;
    if (tiles * (I / 64) > kMaxDim || tiles * (H / 128) > kMaxDim) return MXFP4_ERR_UNSUPPORTED_SHAPE;
    return MXFP4_OK;
}

// Tensor map of contiguous 8-bit rows [rows, K], box 128 bytes x half a large token tile.
bool token_map(CUtensorMap *out, const void *base, int64_t K, int64_t rows)
{
    return encode_map_2d(out, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, static_cast<uint64_t>(K), static_cast<uint64_t>(rows),
                         static_cast<uint64_t>(K), 128u, kMoeLargeTile / 2, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

// Tensor map of blocks of 512 scale bytes, box two blocks.
bool block_map(CUtensorMap *out, const void *base, int64_t blocks)
{
    return encode_map_2d(out, CU_TENSOR_MAP_DATA_TYPE_UINT32, base, 128u, static_cast<uint64_t>(blocks), 512u, 128u, 2u,
                         CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

}  // namespace

extern "C" {

mxfp4_status_t mxfp8_add_rmsnorm_quantize(const void *X, int64_t ldx, const void *residual, int64_t ldr,
                                          const void *weight, int dtype, float eps, int64_t M, int64_t K, void *H,
                                          int64_t ldh, void *Y, int64_t ldy, void *Aq, int64_t ldq, void *A_sf,
                                          void *stream)
{
    if (dtype != MXFP4_DTYPE_BF16 && dtype != MXFP4_DTYPE_FP16) return MXFP4_ERR_INVALID_ARG;
    if (M < 0 || K < 1 || M > kMaxDim || K > kMaxDim || !(eps >= 0.0f) || std::isinf(eps)) return MXFP4_ERR_INVALID_ARG;
    if (K % 32 != 0) return MXFP4_ERR_UNSUPPORTED_SHAPE;
    if (M == 0) return MXFP4_OK;
    if (!X || !weight || !Aq || !A_sf) return MXFP4_ERR_INVALID_ARG;
    if (ldx < K || ldq < K || (residual && ldr < K) || (H && ldh < K) || (Y && ldy < K)) return MXFP4_ERR_INVALID_ARG;
    if (ldx % 8 || ldq % 8 || (residual && ldr % 8) || (H && ldh % 8) || (Y && ldy % 8)) return MXFP4_ERR_MISALIGNED;
    if (!aligned(X, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(H, 16) || !aligned(Y, 16) ||
        !aligned(Aq, 8) || !aligned(A_sf, 4))
        return MXFP4_ERR_MISALIGNED;
    int sms = 0;
    if (!current_device_sms(&sms)) return MXFP4_ERR_NO_DEVICE;
    return cuda_status(launch_add_rmsnorm_mxfp8(X, ldx, residual, ldr, weight, dtype == MXFP4_DTYPE_FP16, eps, M, K, H,
                                                ldh, Y, ldy, Aq, ldq, A_sf, sms, static_cast<cudaStream_t>(stream)));
}

mxfp4_status_t moe_route(const void *logits, int dtype, int64_t ldl, int64_t T, int E, const float *bias, int score,
                         int groups, int topk_groups, int group_top, int k, int renormalize, float scale, int32_t *ids,
                         float *weights, void *stream)
{
    if (dtype < MXFP4_DTYPE_BF16 || dtype > MXFP4_DTYPE_FP32) return MXFP4_ERR_INVALID_ARG;
    if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) return MXFP4_ERR_INVALID_ARG;
    if (T < 0 || T > kMaxDim || E < 1 || ldl < E || groups < 1 || topk_groups < 1 || topk_groups > groups ||
        (group_top != 1 && group_top != 2) || k < 1 || !std::isfinite(scale))
        return MXFP4_ERR_INVALID_ARG;
    if (E > MOE_MAX_EXPERTS || E % groups != 0 || k > MOE_MAX_TOPK || k > topk_groups * (E / groups))
        return MXFP4_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MXFP4_OK;
    if (!logits || !ids || !weights) return MXFP4_ERR_INVALID_ARG;
    if (!aligned(logits, dtype == MXFP4_DTYPE_FP32 ? 4 : 2) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4))
        return MXFP4_ERR_MISALIGNED;
    int sms = 0;
    if (!current_device_sms(&sms)) return MXFP4_ERR_NO_DEVICE;
    RouteParams p;
    p.logits = logits;
    p.bias = bias;
    p.ids = ids;
    p.weights = weights;
    p.ldl = ldl;
    p.T = T;
    p.E = E;
    p.k = k;
    p.groups = groups;
    p.topk_groups = topk_groups;
    p.group_top = group_top;
    p.sigmoid = score == MOE_SCORE_SIGMOID;
    p.renorm = renormalize != 0;
    p.scale = scale;
    return cuda_status(launch_moe_route(p, dtype, sms, static_cast<cudaStream_t>(stream)));
}

size_t mxfp4_moe_experts_workspace_bytes(int64_t T, int k, int E, int64_t H, int64_t I)
{
    if (check_moe_sizes(T, k, E, H, I) != MXFP4_OK || T == 0) return 0;
    return moe_layout(T, k, E, H, I).total;
}

mxfp4_status_t mxfp4_moe_experts(const void *Xq, int64_t ldx, const void *X_sf, const int32_t *ids, const float *weights,
                                 const void *W13q, const void *W13_sf, const void *W2q, const void *W2_sf, void *out,
                                 int64_t ldo, int64_t T, int k, int E, int64_t H, int64_t I, void *workspace,
                                 size_t ws_bytes, void *stream)
{
    mxfp4_status_t st = check_moe_sizes(T, k, E, H, I);
    if (st != MXFP4_OK) return st;
    if (T == 0) return MXFP4_OK;
    if (!Xq || !X_sf || !ids || !weights || !W13q || !W13_sf || !W2q || !W2_sf || !out || !workspace)
        return MXFP4_ERR_INVALID_ARG;
    if (ldx < H || ldo < H) return MXFP4_ERR_INVALID_ARG;
    if (ldx % 16 || ldo % 8 || !aligned(Xq, 16) || !aligned(X_sf, 16) || !aligned(ids, 4) || !aligned(weights, 4) ||
        !aligned(W13q, 32) || !aligned(W2q, 32) || !aligned(W13_sf, 16) || !aligned(W2_sf, 16) || !aligned(out, 16) ||
        !aligned(workspace, 256))
        return MXFP4_ERR_MISALIGNED;
    const MoeLayout l = moe_layout(T, k, E, H, I);
    if (ws_bytes < l.total) return MXFP4_ERR_WORKSPACE_TOO_SMALL;
    int sms = 0;
    if (!current_device_sms(&sms)) return MXFP4_ERR_NO_DEVICE;
    MoeArgs a;
    memset(&a, 0, sizeof(a));
    a.xq = static_cast<const uint8_t *>(Xq);
    a.ldx = ldx;
    a.x_sf = static_cast<const uint8_t *>(X_sf);
    a.ids = ids;
    a.weights = weights;
    a.w13_sf = static_cast<const uint8_t *>(W13_sf);
    a.w2_sf = static_cast<const uint8_t *>(W2_sf);
    a.out = static_cast<uint16_t *>(out);
    a.ldo = ldo;
    a.T = T;
    a.k = k;
    a.E = E;
    a.H = static_cast<int>(H);
    a.I = static_cast<int>(I);
    a.ws = static_cast<uint8_t *>(workspace);
    bool maps = encode_packed_map(W13q, H / 2, 2 * I * E, H / 2, 64, &a.tm_w13) &&
                encode_packed_map(W2q, I / 2, H * E, I / 2, 64, &a.tm_w2);
    if (l.nt == kMoeLargeTile)
        maps = maps && token_map(&a.tm_xs, a.ws + l.xs, H, T * k) && token_map(&a.tm_act, a.ws + l.act, I, T * k) &&
               block_map(&a.tm_xs_sf, a.ws + l.xs_sf, int64_t(l.max_tiles) * (H / 128) * 2) &&
               block_map(&a.tm_act_sf, a.ws + l.act_sf, int64_t(l.max_tiles) * (I / 128) * 2);
    if (!maps) return MXFP4_ERR_CUDA;
    return cuda_status(launch_moe_experts(a, l, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
