// Residual sum + RMSNorm + MXFP8 quantization (mxfp8_add_rmsnorm_quantize).
//
// Mathematics, per row: h = x + res; r = (sum h^2 / K + eps)^-1/2; y = (h r) w;
// per 32 values the smallest power of two that leaves |y| <= 448, and E4M3 of
// the quotients. h is rounded to the element type before it is squared: the
// norm is that of the values the next layer reads.
//
// Bound: HBM (2 or 4 bytes read, 1 to 5 written an element; ~6 operations). So
// each row is read once: a block keeps its row in registers between the sum of
// squares and the quantization, eight elements (one 16-byte vector) a lane, and
// four neighbouring lanes hold one block of 32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstring>

#include "internal.h"
#include "moe.h"
#include "mxfp8_math.cuh"
#include "ptx.cuh"

namespace mxfp4 {

namespace {

struct NormParams {
    const uint16_t *x, *res, *w;
    uint16_t *h, *y;
    uint8_t *q;
    uint8_t *sf;
    int64_t ldx, ldr, ldh, ldy, ldq;
    int64_t M;
    int K;
    float eps;
};

template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t v)
{
    if constexpr (F16) return __half22float2(*reinterpret_cast<const __half2 *>(&v));
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}

template <bool F16>
__device__ __forceinline__ uint32_t round2(float a, float b)
{
    if constexpr (F16) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

template <bool F16>
__device__ __forceinline__ uint4 add8(const uint4 &a, const uint4 &b)
{
    uint4 o;
    const uint32_t *pa = &a.x, *pb = &b.x;
    uint32_t *po = &o.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 u = unpack2<F16>(pa[i]), v = unpack2<F16>(pb[i]);
        po[i] = round2<F16>(u.x + v.x, u.y + v.y);
    }
    return o;
}

template <bool F16>
__device__ __forceinline__ float sumsq8(const uint4 &a)
{
    const uint32_t *p = &a.x;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 u = unpack2<F16>(p[i]);
        s = fmaf(u.x, u.x, s);
        s = fmaf(u.y, u.y, s);
    }
    return s;
}

// Normalizes, stores and quantizes the vector of eight values of row `row` at
// column 8 * vec; `live`: vec lies within the row (all lanes of the warp call).
template <bool F16>
__device__ __forceinline__ void finish8(const NormParams &p, int64_t row, int vec, bool live, const uint4 &hv, float r)
{
    float y[8];
    uint32_t amax = 0;
    if (live) {
        const uint4 wv = __ldg(reinterpret_cast<const uint4 *>(p.w) + vec);
        const uint32_t *ph = &hv.x, *pw = &wv.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 a = unpack2<F16>(ph[i]), b = unpack2<F16>(pw[i]);
            y[2 * i] = __fmul_rn(a.x * r, b.x);
            y[2 * i + 1] = __fmul_rn(a.y * r, b.y);
        }
        if (p.y) {
            uint4 o;
            uint32_t *po = &o.x;
#pragma unroll
            for (int i = 0; i < 4; ++i) po[i] = round2<F16>(y[2 * i], y[2 * i + 1]);
            *reinterpret_cast<uint4 *>(p.y + row * p.ldy + 8 * vec) = o;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(y[i]) & 0x7FFFFFFFu);
    }
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const uint32_t b = live ? mxfp8_scale_byte(amax) : 0x7Fu;
    if (live) {
        const float inv = mxfp8_scale_inverse(b);
        uint2 c;
        c.x = e4m3x4_rn(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
        c.y = e4m3x4_rn(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv);
        *reinterpret_cast<uint2 *>(p.q + row * p.ldq + 8 * vec) = c;
    }
    // the four scale bytes of 128 columns are one word of the blocked layout
    const uint32_t b01 = b | (__shfl_down_sync(0xffffffffu, b, 4) << 8);
    const uint32_t word = b01 | (__shfl_down_sync(0xffffffffu, b01, 8) << 16);
    if ((threadIdx.x & 15) == 0 && 8 * vec < (p.K + 127) / 128 * 128)
        *reinterpret_cast<uint32_t *>(p.sf + ((row >> 7) * ((p.K + 127) / 128) + (vec >> 4)) * 512 + (row & 31) * 16 +
                                      ((row & 127) >> 5) * 4) = word;
}

// Sum of v over the block, the same in every thread.
__device__ __forceinline__ float block_sum(float v, float *buf)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int nw = blockDim.x >> 5;
    if (nw == 1) return v;
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = static_cast<int>(threadIdx.x & 31) < nw ? buf[threadIdx.x & 31] : 0.0f;
#pragma unroll
    for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    return t;
}

// One row a block; VPT vectors a thread stay in registers (VPT = 0: rows of any
// length, read a second time for the quantization).
template <bool F16, int VPT>
__global__ void __launch_bounds__(1024) add_rmsnorm_mxfp8_kernel(const NormParams p)
{
    __shared__ float buf[32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t row = blockIdx.x;
    const int nvec = p.K >> 3, nt = blockDim.x;
    const int64_t xo = row * p.ldx, ro = row * p.ldr, ho = row * p.ldh;
    auto load_h = [&](int v) {
        uint4 a = *reinterpret_cast<const uint4 *>(p.x + xo + 8 * v);
        if (p.res) a = add8<F16>(a, *reinterpret_cast<const uint4 *>(p.res + ro + 8 * v));
        return a;
    };
    float ss = 0.0f;
    if constexpr (VPT > 0) {
        uint4 hv[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = threadIdx.x + i * nt;
            if (v < nvec) hv[i] = load_h(v);
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = threadIdx.x + i * nt;
            if (v < nvec) {
                ss += sumsq8<F16>(hv[i]);
                if (p.h) *reinterpret_cast<uint4 *>(p.h + ho + 8 * v) = hv[i];
            }
        }
        const float m = block_sum(ss, buf) / static_cast<float>(p.K) + p.eps;
        const float r = m == 0.0f ? 0.0f : rsqrtf(m);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = threadIdx.x + i * nt;
            if (v - static_cast<int>(threadIdx.x & 31) < (nvec + 15) / 16 * 16) finish8<F16>(p, row, v, v < nvec, hv[i], r);
        }
    } else {
        for (int v = threadIdx.x; v < nvec; v += nt) ss += sumsq8<F16>(load_h(v));
        const float m = block_sum(ss, buf) / static_cast<float>(p.K) + p.eps;
        const float r = m == 0.0f ? 0.0f : rsqrtf(m);
        for (int v0 = threadIdx.x & ~31; v0 < nvec; v0 += nt) {
            const int v = v0 + (threadIdx.x & 31);
            uint4 hv = make_uint4(0, 0, 0, 0);
            if (v < nvec) {
                hv = load_h(v);
                if (p.h) *reinterpret_cast<uint4 *>(p.h + ho + 8 * v) = hv;
            }
            finish8<F16>(p, row, v, v < nvec, hv, r);
        }
    }
    // pad rows of the last 128-row block of scales, shared out over the blocks
    const int64_t rows_pad = (p.M + 127) / 128 * 128;
    const int kc = (p.K + 127) / 128;
    for (int64_t pr = p.M + blockIdx.x; pr < rows_pad; pr += gridDim.x)
        for (int c = threadIdx.x; c < kc; c += nt)
            *reinterpret_cast<uint32_t *>(p.sf + ((pr >> 7) * kc + c) * 512 + (pr & 31) * 16 + ((pr & 127) >> 5) * 4) =
                0x7F7F7F7Fu;
}

template <bool F16>
cudaError_t launch_norm(const NormParams &p, cudaStream_t stream)
{
    const int nvec = p.K / 8;
    int threads = (nvec + 31) / 32 * 32, vpt = 1;
    while (threads > 256 && vpt < 4) {
        vpt *= 2;
        threads = ((nvec + vpt - 1) / vpt + 31) / 32 * 32;
    }
    if (threads > 1024) {
        vpt = 0;
        threads = 1024;
    }
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(static_cast<unsigned>(p.M), 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    switch (vpt) {
    case 1: return cudaLaunchKernelEx(&cfg, add_rmsnorm_mxfp8_kernel<F16, 1>, p);
    case 2: return cudaLaunchKernelEx(&cfg, add_rmsnorm_mxfp8_kernel<F16, 2>, p);
    case 4: return cudaLaunchKernelEx(&cfg, add_rmsnorm_mxfp8_kernel<F16, 4>, p);
    default: return cudaLaunchKernelEx(&cfg, add_rmsnorm_mxfp8_kernel<F16, 0>, p);
    }
}

}  // namespace

cudaError_t launch_add_rmsnorm_mxfp8(const void *X, int64_t ldx, const void *res, int64_t ldr, const void *w, bool f16,
                                     float eps, int64_t M, int64_t K, void *H, int64_t ldh, void *Y, int64_t ldy,
                                     void *Aq, int64_t ldq, void *sf, cudaStream_t stream)
{
    NormParams p;
    p.x = static_cast<const uint16_t *>(X);
    p.res = static_cast<const uint16_t *>(res);
    p.w = static_cast<const uint16_t *>(w);
    p.h = static_cast<uint16_t *>(H);
    p.y = static_cast<uint16_t *>(Y);
    p.q = static_cast<uint8_t *>(Aq);
    p.sf = static_cast<uint8_t *>(sf);
    p.ldx = ldx;
    p.ldr = ldr;
    p.ldh = ldh;
    p.ldy = ldy;
    p.ldq = ldq;
    p.M = M;
    p.K = static_cast<int>(K);
    p.eps = eps;
    return f16 ? launch_norm<true>(p, stream) : launch_norm<false>(p, stream);
}

}  // namespace mxfp4
