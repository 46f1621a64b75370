// extern "C" entry points of include/mxfp4_layer.h: argument validation and
// workspace layout. Nothing here allocates device memory or synchronizes.
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <utility>

#include "internal.h"
#include "layer.h"
#include "mxfp4_layer.h"

using namespace mxfp4;

namespace {

inline bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline mxfp4_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MXFP4_OK : MXFP4_ERR_CUDA; }

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
// of adapters: the end of a group's last tile, or of the last chunk of channels, is a 32-bit index
constexpr int64_t kMaxWidth = int64_t(1) << 30;

mxfp4_status_t check_lora_sizes(int64_t T, int64_t K, int R, int L)
{
    if (T < 0 || K < 1 || R < 1 || L < 1) return MXFP4_ERR_INVALID_ARG;
    if (T > kMaxWidth || K > kMaxWidth || K % 8 || R % 8 || R > LORA_MAX_RANK || L > LORA_MAX_ADAPTERS)
        return MXFP4_ERR_UNSUPPORTED_SHAPE;
    return MXFP4_OK;
}

// Do heads of D elements at t * st + h * sh (t < T, h < heads) share elements? They do if some |t * st + h * sh| < D
// for a difference (t, h) other than none, |t| < T, |h| < heads.
bool heads_overlap(int64_t T, int64_t heads, int64_t D, int64_t st, int64_t sh)
{
    // sizes alone matter: of h there are both signs. Beyond 2^62 a stride is no distance in memory
    const int64_t most = int64_t(1) << 62;
    st = st <= -most || st >= most ? most : std::abs(st);
    sh = sh <= -most || sh >= most ? most : std::abs(sh);
    if (T > 1 && st < D) return true;
    if (heads > 1 && sh < D) return true;
    if (T == 1 || heads == 1) return false;
    // the usual layouts: all heads of a token, or all tokens of a head, before the next one
    if (st >= sh && (st - D) / sh >= heads - 1) return false;
    if (sh >= st && (sh - D) / st >= T - 1) return false;
    // otherwise the dimension with fewer steps (46340 at most), against the next places of the other
    if (T < heads) {
        std::swap(T, heads);
        std::swap(st, sh);
    }
    for (int64_t h = 1; h < heads; ++h) {
        if (h > most / sh) return false;                 // from here on nothing in memory is that far
        const int64_t at = h * sh, t = at / st, after = at - t * st;
        if ((t < T && after < D) || (t + 1 < T && st - after < D)) return true;
    }
    return false;
}

}  // namespace

extern "C" {

size_t lora_workspace_bytes(int64_t T, int64_t K, int R, int L)
{
    if (check_lora_sizes(T, K, R, L) != MXFP4_OK || T == 0) return 0;
    return lora_layout(T, K, R, L).total;
}

mxfp4_status_t lora_add(const void *X, int64_t ldx, const void *A, const void *B, const int32_t *ids, const float *scales,
                        const int32_t *ranks, const void *base, int64_t ldb, int dtype, void *C, int64_t ldc, int64_t T,
                        int64_t K, int64_t N, int R, int L, void *workspace, size_t ws_bytes, void *stream)
{
    if (dtype != MXFP4_DTYPE_BF16 && dtype != MXFP4_DTYPE_FP16) return MXFP4_ERR_INVALID_ARG;
    if (N < 1) return MXFP4_ERR_INVALID_ARG;
    if (N > kMaxWidth || N % 8) return MXFP4_ERR_UNSUPPORTED_SHAPE;
    const mxfp4_status_t st = check_lora_sizes(T, K, R, L);
    if (st != MXFP4_OK) return st;
    if (T == 0) return MXFP4_OK;
    if (!X || !A || !B || !ids || !base || !C || !workspace) return MXFP4_ERR_INVALID_ARG;
    if (ldx < K || ldb < N || ldc < N || (C == base && ldc != ldb)) return MXFP4_ERR_INVALID_ARG;
    if (ldx % 8 || ldb % 8 || ldc % 8 || !aligned(X, 16) || !aligned(A, 16) || !aligned(B, 16) || !aligned(base, 16) ||
        !aligned(C, 16) || !aligned(ids, 4) || !aligned(scales, 4) || !aligned(ranks, 4) || !aligned(workspace, 256))
        return MXFP4_ERR_MISALIGNED;
    const LoraLayout l = lora_layout(T, K, R, L);
    if (ws_bytes < l.total) return MXFP4_ERR_WORKSPACE_TOO_SMALL;
    int sms = 0;
    if (!current_device_sms(&sms)) return MXFP4_ERR_NO_DEVICE;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    LoraParams p;
    memset(&p, 0, sizeof(p));
    p.x = static_cast<const uint16_t *>(X);
    p.a = static_cast<const uint16_t *>(A);
    p.b = static_cast<const uint16_t *>(B);
    p.ids = ids;
    p.scales = scales;
    p.ranks = ranks;
    p.base = static_cast<const uint16_t *>(base);
    p.c = static_cast<uint16_t *>(C);
    p.ldx = ldx;
    p.ldb = ldb;
    p.ldc = ldc;
    p.T = static_cast<int>(T);
    p.K = static_cast<int>(K);
    p.N = static_cast<int>(N);
    p.R = R;
    p.L = L;
    p.copy = C != base;
    p.u = reinterpret_cast<float *>(ws + l.u);
    p.order = reinterpret_cast<int *>(ws + l.order);
    p.tiles = reinterpret_cast<int4 *>(ws + l.tiles);
    return cuda_status(launch_lora(p, l, dtype == MXFP4_DTYPE_FP16, static_cast<cudaStream_t>(stream)));
}

mxfp4_status_t qk_norm_rope(const void *q, int64_t q_st, int64_t q_sh, const void *k, int64_t k_st, int64_t k_sh,
                            const void *q_weight, const void *k_weight, const float *table, const void *positions,
                            int pos64, int dtype, float eps, int64_t T, int Hq, int Hk, int D, int rot, int interleaved,
                            int64_t P, void *q_out, int64_t qo_st, int64_t qo_sh, void *k_out, int64_t ko_st,
                            int64_t ko_sh, void *stream)
{
    if (dtype != MXFP4_DTYPE_BF16 && dtype != MXFP4_DTYPE_FP16) return MXFP4_ERR_INVALID_ARG;
    if (T < 0 || Hq < 0 || Hk < 0 || D < 1 || rot < 0 || rot > D || !(eps >= 0.0f) || std::isinf(eps))
        return MXFP4_ERR_INVALID_ARG;
    if (D % 8 || D > 256 || rot % (interleaved ? 8 : 16)) return MXFP4_ERR_UNSUPPORTED_SHAPE;
    if (T > kMaxDim || T * (static_cast<int64_t>(Hq) + Hk) > kMaxDim) return MXFP4_ERR_UNSUPPORTED_SHAPE;
    if (T == 0 || (Hq == 0 && Hk == 0)) return MXFP4_OK;
    if ((Hq && (!q || !q_out)) || (Hk && (!k || !k_out))) return MXFP4_ERR_INVALID_ARG;
    if (rot && (!table || !positions || P < 1)) return MXFP4_ERR_INVALID_ARG;
    const int64_t strides[8] = {q_st, q_sh, qo_st, qo_sh, k_st, k_sh, ko_st, ko_sh};
    for (int i = Hq ? 0 : 4; i < (Hk ? 8 : 4); ++i)
        if (strides[i] % 8) return MXFP4_ERR_MISALIGNED;
    // heads of an output do not share elements
    const int64_t ost[2] = {qo_st, ko_st}, osh[2] = {qo_sh, ko_sh};
    const int heads[2] = {Hq, Hk};
    for (int i = 0; i < 2; ++i)
        if (heads[i] && heads_overlap(T, heads[i], D, ost[i], osh[i])) return MXFP4_ERR_INVALID_ARG;
    if ((Hq && q == q_out && (q_st != qo_st || q_sh != qo_sh)) || (Hk && k == k_out && (k_st != ko_st || k_sh != ko_sh)))
        return MXFP4_ERR_INVALID_ARG;
    if ((Hq && (!aligned(q, 16) || !aligned(q_out, 16))) || (Hk && (!aligned(k, 16) || !aligned(k_out, 16))) ||
        !aligned(q_weight, 16) || !aligned(k_weight, 16) ||
        (rot && (!aligned(table, 16) || !aligned(positions, pos64 ? 8 : 4))))
        return MXFP4_ERR_MISALIGNED;
    int sms = 0;
    if (!current_device_sms(&sms)) return MXFP4_ERR_NO_DEVICE;
    QkParams p;
    memset(&p, 0, sizeof(p));
    const void *x[2] = {q, k}, *w[2] = {q_weight, k_weight};
    void *o[2] = {q_out, k_out};
    for (int i = 0; i < 2; ++i) {
        p.x[i] = static_cast<const uint16_t *>(x[i]);
        p.out[i] = static_cast<uint16_t *>(o[i]);
        p.w[i] = static_cast<const uint16_t *>(w[i]);
        p.st[i] = strides[4 * i];
        p.sh[i] = strides[4 * i + 1];
        p.ost[i] = strides[4 * i + 2];
        p.osh[i] = strides[4 * i + 3];
        p.heads[i] = heads[i];
    }
    p.table = table;
    p.positions = positions;
    p.T = T;
    p.P = P;
    p.D = D;
    p.rot = rot;
    p.pos64 = pos64 != 0;
    p.eps = eps;
    return cuda_status(launch_qk_norm_rope(p, dtype == MXFP4_DTYPE_FP16, interleaved != 0, sms,
                                           static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
