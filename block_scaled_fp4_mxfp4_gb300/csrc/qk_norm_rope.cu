// Norm and rotation of queries and keys (qk_norm_rope).
//
// Mathematics, per head x of D elements at position p: y = x r w with
// r = (mean x^2 + eps)^-1/2, and pairs (y_i, y_j) turned by the angle i of p. Both
// are linear in x once r is known, so an element is
//   out_i = r (x_i a_i + x_j b_i),  a_i = w_i cos, b_i = -+ w_j sin,
// (a = w, b = 0 where nothing turns), and a, b are the same for all heads of a token.
//
// Bound: HBM (2 bytes read, 2 written an element). A head is one 16-byte vector for
// each of LPH lanes, read once and kept in registers between the sum of squares and
// the rotation; the partner's vector in the layout of halves comes by shuffles of
// packed registers. A group of LPH lanes takes U heads of one token, all loads
// ahead, and forms a, b once for them.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "layer.h"
#include "ptx.cuh"

namespace mxfp4 {

namespace {

constexpr int kThreads = 256;

template <bool F16>
__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8])
{
    const uint32_t r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (F16) {
            const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&r[i]));
            f[2 * i] = t.x;
            f[2 * i + 1] = t.y;
        } else {
            f[2 * i] = __uint_as_float(r[i] << 16);
            f[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
        }
    }
}

template <bool F16>
__device__ __forceinline__ uint4 pack8(const float (&f)[8])
{
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (F16) {
            const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            r[i] = *reinterpret_cast<const uint32_t *>(&h);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            r[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

template <int LPH>
__device__ __forceinline__ float group_sum(float v)
{
#pragma unroll
    for (int o = LPH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// r for a head whose squares leave fp32, or whose sum is so small that it lost bits
// and eps does not hide it: the values are brought to about 1 by a power of two
// first (exact), and x and its partner are left scaled by it.
template <int LPH>
__device__ __noinline__ float rescaled_r(float (&x)[8], float (&xp)[8], bool odd, float eps, int D)
{
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[i]));
#pragma unroll
    for (int o = LPH / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float s = 1.0f;
    if (odd && top > 0.0f && !isinf(top)) s = exp2f(static_cast<float>(max(-126, min(126, -ilogbf(top)))));
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] *= s;
        xp[i] *= s;
        ss = fmaf(x[i], x[i], ss);
    }
    ss = group_sum<LPH>(ss);
    const double m = static_cast<double>(ss) / D + static_cast<double>(eps) * s * s;
    return m == 0.0 ? 0.0f : static_cast<float>(1.0 / sqrt(m));
}

template <bool F16, bool INTER, int LPH, int U>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const QkParams p)
{
    const int j = threadIdx.x & (LPH - 1);              // this lane's vector of a head
    const int per_token = p.units[0] + p.units[1];
    const int64_t total = p.T * per_token;
    int64_t unit = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / LPH;
    const bool live = unit < total;
    if (!live) unit = total - 1;                        // a whole warp stays for the shuffles
    const int64_t t = unit / per_token;
    int c = static_cast<int>(unit - t * per_token);
    const int is_k = c >= p.units[0];
    if (is_k) c -= p.units[0];
    const int h0 = c * U, heads = min(U, p.heads[is_k] - h0);
    const bool mine = live && 8 * j < p.D;
    const int half = p.rot >> 1;

    grid_dependency_wait();
    grid_launch_dependents();
    const uint16_t *src = p.x[is_k] + t * p.st[is_k] + h0 * p.sh[is_k] + 8 * j;
    uint4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        raw[u] = make_uint4(0, 0, 0, 0);
        if (mine && u < heads) raw[u] = *reinterpret_cast<const uint4 *>(src + u * p.sh[is_k]);
    }

    // partner lane of the layout of halves; lanes beyond the rotated part keep their own
    const int hv = p.rot >> 4;                          // vectors of a half
    const bool turned = 8 * j < p.rot;
    const int group = (threadIdx.x & 31) & ~(LPH - 1);
    const int partner = INTER || !turned ? j : (j < hv ? j + hv : j - hv);

    float a[8], b[8];
    float bad = 0.0f;                                   // NaN for a position outside the table
    {
        const uint16_t *w = p.w[is_k];
        float own[8], other[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) own[i] = other[i] = 1.0f;
        if (w && mine) {
            unpack8<F16>(*reinterpret_cast<const uint4 *>(w + 8 * j), own);
            if constexpr (!INTER) unpack8<F16>(*reinterpret_cast<const uint4 *>(w + 8 * partner), other);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            a[i] = own[i];
            b[i] = 0.0f;
        }
        if (p.rot) {
            const int64_t pos = p.pos64 ? static_cast<const int64_t *>(p.positions)[t]
                                        : static_cast<const int32_t *>(p.positions)[t];
            const bool inside = pos >= 0 && pos < p.P;
            if (!inside) bad = __int_as_float(0x7FC00000);
            if (turned && inside) {
                const float *row = p.table + pos * p.rot;
                if constexpr (INTER) {
                    const float4 cs = *reinterpret_cast<const float4 *>(row + 4 * j);
                    const float4 sn = *reinterpret_cast<const float4 *>(row + half + 4 * j);
                    const float cv[4] = {cs.x, cs.y, cs.z, cs.w}, sv[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        a[2 * i] = own[2 * i] * cv[i];
                        b[2 * i] = -own[2 * i + 1] * sv[i];
                        a[2 * i + 1] = own[2 * i + 1] * cv[i];
                        b[2 * i + 1] = own[2 * i] * sv[i];
                    }
                } else {
                    const int at = 8 * (j < hv ? j : j - hv);
                    const float sign = j < hv ? -1.0f : 1.0f;
#pragma unroll
                    for (int i = 0; i < 8; i += 4) {
                        const float4 cs = *reinterpret_cast<const float4 *>(row + at + i);
                        const float4 sn = *reinterpret_cast<const float4 *>(row + half + at + i);
                        const float cv[4] = {cs.x, cs.y, cs.z, cs.w}, sv[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
                        for (int l = 0; l < 4; ++l) {
                            a[i + l] = own[i + l] * cv[l];
                            b[i + l] = sign * other[i + l] * sv[l];
                        }
                    }
                }
            }
        }
    }

    uint16_t *dst = p.out[is_k] + t * p.ost[is_k] + h0 * p.osh[is_k] + 8 * j;
    const bool norm = p.w[is_k] != nullptr;
    const float inv_d = 1.0f / static_cast<float>(p.D);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float x[8], xp[8];
        unpack8<F16>(raw[u], x);
        if constexpr (INTER) {
#pragma unroll
            for (int i = 0; i < 8; ++i) xp[i] = x[i ^ 1];
        } else {
            uint4 q;
            q.x = __shfl_sync(0xffffffffu, raw[u].x, group + partner);
            q.y = __shfl_sync(0xffffffffu, raw[u].y, group + partner);
            q.z = __shfl_sync(0xffffffffu, raw[u].z, group + partner);
            q.w = __shfl_sync(0xffffffffu, raw[u].w, group + partner);
            unpack8<F16>(q, xp);
        }
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
        ss = group_sum<LPH>(ss);
        float r = 1.0f;
        // 1e36: the sum has not overflowed; 1e-24: squares below 2^-126 are less than 2^-24 of it
        const bool odd = norm && u < heads && (!(ss < 1e36f) || (ss < 1e-24f && p.eps < 1e-20f));
        if (norm) r = rsqrtf(fmaf(ss, inv_d, p.eps));
        if (__any_sync(0xffffffffu, odd)) {
            const float rr = rescaled_r<LPH>(x, xp, odd, p.eps, p.D);
            if (odd) r = rr;
        }
        r += bad;
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = r * fmaf(xp[i], b[i], x[i] * a[i]);
        if (mine && u < heads) *reinterpret_cast<uint4 *>(dst + u * p.osh[is_k]) = pack8<F16>(o);
    }
}

template <bool F16, bool INTER, int LPH>
cudaError_t launch_lph(QkParams p, int num_sms, cudaStream_t stream)
{
    // four heads a lane group as soon as that still gives every SM a full set of threads
    const int64_t vectors = p.T * (p.heads[0] + p.heads[1]) * LPH;
    const bool many = vectors >= int64_t(4) * num_sms * 1024;
    const int U = many ? 4 : 1;
    for (int i = 0; i < 2; ++i) p.units[i] = (p.heads[i] + U - 1) / U;
    const int64_t threads = p.T * (p.units[0] + p.units[1]) * LPH;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((threads + kThreads - 1) / kThreads));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (many) return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<F16, INTER, LPH, 4>, p);
    return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<F16, INTER, LPH, 1>, p);
}

template <bool F16, bool INTER>
cudaError_t launch_type(const QkParams &p, int num_sms, cudaStream_t stream)
{
    if (p.D <= 64) return launch_lph<F16, INTER, 8>(p, num_sms, stream);
    if (p.D <= 128) return launch_lph<F16, INTER, 16>(p, num_sms, stream);
    return launch_lph<F16, INTER, 32>(p, num_sms, stream);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkParams &p, bool f16, bool interleaved, int num_sms, cudaStream_t stream)
{
    if (f16) return interleaved ? launch_type<true, true>(p, num_sms, stream) : launch_type<true, false>(p, num_sms, stream);
    return interleaved ? launch_type<false, true>(p, num_sms, stream) : launch_type<false, false>(p, num_sms, stream);
}

}  // namespace mxfp4
