// Residual sum + RMSNorm + MXFP8 quantization (mxfp8_add_rmsnorm_quantize).
//
// Mathematics, per row: h = x + res; r = (sum h^2 / K + eps)^-1/2; y = (h r) w;
// per 32 values the smallest power of two that leaves |y| <= 448, and E4M3 of
// the quotients. h is rounded to the element type before it is squared: the
// norm is that of the values the next layer reads.
//
// Bound: instructions and their latency (45 an element, with the exactness below, in
// 68 % of the cycles), not far above HBM (2 or 4 bytes read, 1 to 5 written an
// element). Each row is read once: a block keeps its row in registers between the sum
// of squares and the quantization, eight elements (one 16-byte vector) a lane, and
// four neighbouring lanes hold one block of 32. The variant of four vectors a lane has
// 40 registers, so that six blocks fit an SM, and spills a few. Measured: 4096 x 7168 bf16 with
// residual, h and y (265 MB) 54 us, 4.9 TB/s; one row 4.2 us.
//
// Exactness: an E4M3 rounding turns an fp32 error of 2^-23 into a step of 2^-3 where
// a value lies next to a midpoint, about one element in a million. So the sum of
// squares is carried in two floats, by error-free additions from the first square on
// (a row is often dominated by a few channels: with the eight squares of a vector
// summed in fp32, its r was off by up to 2^-24; 4096 x 7168 53.4 us so, 54.4 us now),
// and r is two floats good to 2^-42: the low parts add up in fp32, 2^-48 of the sum an
// addition, about forty in a row. A value within the fp32 error (3 units) of a
// midpoint, or a block's maximum within it of the border between two scales, is
// decided again in 64 bits; what those find within 2^-40 of either counts as on it.
// The rule costs four instructions an element. Lanes that hold a subnormal code, whose
// midpoints are others, look a second time (no difference at 4096 x 7168; with the
// 64-bit part entered for every such lane, 59.5 us).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
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
    float keps_hi, keps_lo;     // K * eps
    float rootk_hi, rootk_lo;   // sqrt(K)
};

// An unevaluated sum of two floats.
struct Two {
    float hi, lo;
};

// Knuth's TwoSum of the high parts; the low ones are added in fp32.
__device__ __forceinline__ Two two_add(const Two &a, const Two &b)
{
    const float s = __fadd_rn(a.hi, b.hi), z = __fsub_rn(s, a.hi);
    const float e = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, z)), __fsub_rn(b.hi, z));
    return Two{s, __fadd_rn(e, __fadd_rn(a.lo, b.lo))};
}

// sqrt(K / m) of an ordinary sum, or 0 or NaN: rsqrt and one Newton step on its exact
// residual.
__device__ __forceinline__ Two reciprocal_rms(const Two &m, const NormParams &p)
{
    if (!(m.hi > 0.0f)) return Two{m.hi, 0.0f};
    const float q = rsqrtf(m.hi);
    const float s = q * q, se = fmaf(q, q, -s);
    const float t = fmaf(-m.hi, s, 1.0f) - fmaf(m.hi, se, m.lo * s);
    const float hi = q * p.rootk_hi;
    const float lo = fmaf(q, p.rootk_hi, -hi) + fmaf(q, p.rootk_lo, 0.5f * t * hi);
    const float r = hi + lo;
    return Two{r, lo - (r - hi)};
}

// Sums whose squares, reciprocal or its residual may leave fp32 (bf16 values above 10^13
// or below 10^-15, or an eps as far out) take the way of finish_far_row.
__device__ __forceinline__ bool is_far(const Two &m) { return m.hi >= 1e30f || (m.hi > 0.0f && m.hi <= 1e-30f); }

// 16 bytes that this kernel reads once. Not through the read-only path: the sum may
// be written over them.
__device__ __forceinline__ uint4 ld_row(const void *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

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

// Two such sums side by side: the lanes of 64-bit registers of packed fp32
// arithmetic, half the instructions of two.
struct TwoPair {
    uint64_t hi, lo;
};

__device__ __forceinline__ uint64_t pack(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack(uint64_t v)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t sub_pair(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t square_pair(uint64_t a)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %1;" : "=l"(r) : "l"(a));
    return r;
}

// Adds the squares of eight values to s. The square of a bf16 or fp16 value is exact
// in fp32 (16 or 22 bits), and so is each addition to hi with its error to lo.
template <bool F16>
__device__ __forceinline__ void add_squares8(TwoPair &s, const uint4 &a)
{
    const uint32_t *p = &a.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 u = unpack2<F16>(p[i]);
        const uint64_t q = square_pair(pack(u.x, u.y));
        const uint64_t t = add_pair(s.hi, q), z = sub_pair(t, s.hi);
        s.lo = add_pair(s.lo, add_pair(sub_pair(s.hi, sub_pair(t, z)), sub_pair(q, z)));
        s.hi = t;
    }
}

__device__ __forceinline__ Two total(const TwoPair &s)
{
    const float2 hi = unpack(s.hi), lo = unpack(s.lo);
    return two_add(Two{hi.x, lo.x}, Two{hi.y, lo.y});
}

// What 64 bits find closer than this (relative) to a midpoint or a border is on it:
// beyond the error of r, and a tie to the definition where its r has few bits.
constexpr double kTie = 0x1p-40;

// Normalizes, stores and quantizes the vector of eight values of row `row` at
// column 8 * vec; `live`: vec lies within the row (all lanes of the warp call).
// HUGE_ROW: r is 2^64 of the reciprocal, for values taken as 2^-64 of theirs.
template <bool F16, bool HUGE_ROW = false>
__device__ __forceinline__ void finish8(const NormParams &p, int64_t row, int vec, bool live, const uint4 &hv, const Two &r)
{
    constexpr float kPre = HUGE_ROW ? 0x1p-64f : 1.0f;
    float y[8];
    // element i from 64-bit arithmetic
    auto exact = [&](int i) {
        const uint32_t *ph = &hv.x;
        const uint32_t wv = __ldg(reinterpret_cast<const uint32_t *>(p.w) + 4 * vec + (i >> 1));
        const float2 a = unpack2<F16>(ph[i >> 1]), b = unpack2<F16>(wv);
        return static_cast<double>((i & 1 ? a.y : a.x) * kPre) * (static_cast<double>(r.hi) + static_cast<double>(r.lo)) *
               static_cast<double>(i & 1 ? b.y : b.x);
    };
    uint32_t amax = 0;
    if (live) {
        const uint4 wv = __ldg(reinterpret_cast<const uint4 *>(p.w) + vec);
        const uint32_t *ph = &hv.x, *pw = &wv.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 a = unpack2<F16>(ph[i]), b = unpack2<F16>(pw[i]);
            y[2 * i] = __fmul_rn(__fmul_rn(a.x * kPre, r.hi), b.x);
            y[2 * i + 1] = __fmul_rn(__fmul_rn(a.y * kPre, r.hi), b.y);
        }
        if (p.y) {
            uint4 o;
            uint32_t *po = &o.x;
#pragma unroll
            for (int i = 0; i < 4; ++i) po[i] = round2<F16>(y[2 * i], y[2 * i + 1]);
            *reinterpret_cast<uint4 *>(p.y + row * p.ldy + 8 * vec) = o;
        }
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(y[i])));
        amax = __float_as_uint(m);
    }
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    uint32_t b = live ? mxfp8_scale_byte(amax) : 0x7Fu;
    // a maximum within 3 units of 1.75 * 2^n takes its scale from its exact value
    const bool border = live && (amax & 0x7FFFFFu) - 0x5FFFFDu <= 6u && amax < 0x7F800000u;
    if (__any_sync(0xffffffffu, border)) {
        double top = 0.0;
        if (border)
            for (int i = 0; i < 8; ++i) top = fmax(top, fabs(exact(i)));
        top = fmax(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmax(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const double at = static_cast<double>(__uint_as_float((amax & 0x7F800000u) | 0x600000u));
        if (border && amax >= 0x04800000u) b = (amax >> 23) - 8 + (top > at * (1.0 + kTie) ? 1u : 0u);
    }
    if (live) {
        const float inv = mxfp8_scale_inverse(b);
        // E4M3 keeps three bits of the mantissa: its midpoints have 0x80000 in the other 20.
        // Below 2^-6 it keeps steps of 2^-9: there those bits are looked at in |v| + 2^-6.
        auto is_near = [](float v) { return (__float_as_uint(v) & 0xFFFFFu) - 0x7FFFDu <= 6u; };
        bool near = false, small = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            y[i] *= inv;
            near |= is_near(y[i]);
            small |= fabsf(y[i]) < 0x1p-6f;
        }
        if (small) {
#pragma unroll
            for (int i = 0; i < 8; ++i) near |= fabsf(y[i]) < 0x1p-6f && is_near(fabsf(y[i]) + 0x1p-6f);
        }
        if (near) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float v = fabsf(y[i]), up = v < 0x1p-6f ? 0x1p-6f : 0.0f;
                if (is_near(v + up)) {
                    const float mid = __uint_as_float((__float_as_uint(v + up) & 0x7FF00000u) | 0x80000u) - up;
                    const double d = fabs(exact(i)) * static_cast<double>(inv), md = static_cast<double>(mid);
                    const int to = d > md * (1.0 + kTie) ? 1 : d < md * (1.0 - kTie) ? -1 : 0;
                    y[i] = copysignf(__int_as_float(__float_as_int(mid) + to), y[i]);
                }
            }
        }
        uint2 c;
        c.x = e4m3x4_rn(y[0], y[1], y[2], y[3]);
        c.y = e4m3x4_rn(y[4], y[5], y[6], y[7]);
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
__device__ __forceinline__ Two block_sum(Two v, Two *buf)
{
    auto warp_sum = [](Two x) {
#pragma unroll
        for (int o = 16; o; o >>= 1)
            x = two_add(x, Two{__shfl_xor_sync(0xffffffffu, x.hi, o), __shfl_xor_sync(0xffffffffu, x.lo, o)});
        return x;
    };
    v = warp_sum(v);
    const int nw = blockDim.x >> 5, lane = threadIdx.x & 31;
    if (nw == 1) return v;
    if (lane == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    // up to 8 warps: three rounds; more: all five
    v = buf[nw <= 8 ? lane & 7 : lane];
    if ((nw <= 8 ? lane & 7 : lane) >= nw) v = Two{0.0f, 0.0f};
    for (int o = nw <= 8 ? 4 : 16; o; o >>= 1)
        v = two_add(v, Two{__shfl_xor_sync(0xffffffffu, v.hi, o), __shfl_xor_sync(0xffffffffu, v.lo, o)});
    return v;
}

// h of vector v of a row, from X and the residual.
template <bool F16>
__device__ __forceinline__ uint4 load_h(const NormParams &p, int64_t row, int v)
{
    uint4 a = ld_row(p.x + row * p.ldx + 8 * v);
    if (p.res) a = add8<F16>(a, ld_row(p.res + row * p.ldr + 8 * v));
    return a;
}

// The rest of a row whose sum of squares is_far, with that sum taken again in 64 bits.
// `stored`: h is in H already (each thread's own vectors). An infinite value makes
// r = 0, so it becomes NaN and the finite ones 0. Seldom, so kept out of line.
template <bool F16>
__device__ __noinline__ void finish_far_row(const NormParams &p, int64_t row, bool stored, double *buf)
{
    const int nvec = p.K >> 3, nt = blockDim.x, nw = nt >> 5, lane = threadIdx.x & 31;
    auto load = [&](int v) { return stored ? ld_row(p.h + row * p.ldh + 8 * v) : load_h<F16>(p, row, v); };
    double ss = 0.0;
    for (int v = threadIdx.x; v < nvec; v += nt) {
        const uint4 hv = load(v);
        const uint32_t *w = &hv.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 u = unpack2<F16>(w[i]);
            ss += static_cast<double>(u.x) * u.x + static_cast<double>(u.y) * u.y;
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (lane == 0) buf[threadIdx.x >> 5] = ss;
    __syncthreads();
    ss = 0.0;
    for (int i = 0; i < nw; ++i) ss += buf[i];
    const double m = ss + static_cast<double>(p.eps) * p.K;
    const bool huge = m > 1.0;      // the same in all threads
    const double r64 = (huge ? 0x1p64 : 1.0) * sqrt(p.K / m);
    const float hi = static_cast<float>(r64);
    const Two r{hi, static_cast<float>(r64 - hi)};
    for (int v0 = threadIdx.x & ~31; v0 < nvec; v0 += nt) {
        const int v = v0 + lane;
        uint4 hv = make_uint4(0, 0, 0, 0);
        if (v < nvec) {
            hv = load(v);
            if (p.h && !stored) *reinterpret_cast<uint4 *>(p.h + row * p.ldh + 8 * v) = hv;
        }
        if (huge)
            finish8<F16, true>(p, row, v, v < nvec, hv, r);
        else
            finish8<F16>(p, row, v, v < nvec, hv, r);
    }
}

// One row a block; VPT vectors a thread stay in registers (VPT = 0: rows of any
// length, read a second time for the quantization).
template <bool F16, int VPT, int MAX_THREADS>
__global__ void __launch_bounds__(MAX_THREADS, MAX_THREADS == 256 ? 6 : 1) add_rmsnorm_mxfp8_kernel(const __grid_constant__ NormParams p)
{
    __shared__ Two buf[32];
    __shared__ double buf64[32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t row = blockIdx.x;
    const int nvec = p.K >> 3, nt = blockDim.x;
    const int64_t ho = row * p.ldh;
    TwoPair ss{0, 0};
    const Two keps{p.keps_hi, p.keps_lo};
    if constexpr (VPT > 0) {
        uint4 hv[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = threadIdx.x + i * nt;
            if (v < nvec) hv[i] = load_h<F16>(p, row, v);
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = threadIdx.x + i * nt;
            if (v < nvec) {
                add_squares8<F16>(ss, hv[i]);
                if (p.h) *reinterpret_cast<uint4 *>(p.h + ho + 8 * v) = hv[i];
            }
        }
        const Two m = two_add(block_sum(total(ss), buf), keps);
        if (is_far(m)) {
            finish_far_row<F16>(p, row, p.h != nullptr, buf64);
        } else {
            const Two r = reciprocal_rms(m, p);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int v = threadIdx.x + i * nt;
                if (v - static_cast<int>(threadIdx.x & 31) < nvec) finish8<F16>(p, row, v, v < nvec, hv[i], r);
            }
        }
    } else {
        for (int v = threadIdx.x; v < nvec; v += nt) add_squares8<F16>(ss, load_h<F16>(p, row, v));
        const Two m = two_add(block_sum(total(ss), buf), keps);
        if (is_far(m)) {
            finish_far_row<F16>(p, row, false, buf64);
        } else {
            const Two r = reciprocal_rms(m, p);
            for (int v0 = threadIdx.x & ~31; v0 < nvec; v0 += nt) {
                const int v = v0 + (threadIdx.x & 31);
                uint4 hv = make_uint4(0, 0, 0, 0);
                if (v < nvec) {
                    hv = load_h<F16>(p, row, v);
                    if (p.h) *reinterpret_cast<uint4 *>(p.h + ho + 8 * v) = hv;
                }
                finish8<F16>(p, row, v, v < nvec, hv, r);
            }
        }
    }
    // pad rows of the last 128-row block of scales, shared out over all threads in the
    // order of memory: word w of a 512-byte block is row w / 4 + 32 (w % 4)
    const int last = static_cast<int>(p.M & 127), words = (p.K + 127) / 128 * 128;
    if (last == 0) return;
    uint32_t *sf = reinterpret_cast<uint32_t *>(p.sf + (p.M >> 7) * (static_cast<int64_t>(words) * 4));
    for (int64_t i = row * nt + threadIdx.x; i < words; i += static_cast<int64_t>(gridDim.x) * nt) {
        const int w = static_cast<int>(i) & 127;
        if ((w >> 2) + 32 * (w & 3) >= last) sf[i] = 0x7F7F7F7Fu;
    }
}

template <bool F16>
cudaError_t launch_norm(const NormParams &p, int num_sms, cudaStream_t stream)
{
    // Many rows: blocks of up to 256 threads, several on an SM, whose phases (load,
    // sum, store) overlap. Few rows: a row's latency counts, so a vector a thread.
    const int nvec = p.K / 8, most = p.M <= 2 * num_sms ? 1024 : 256;
    int vpt = 1;
    while ((nvec + vpt - 1) / vpt > most && vpt < 4) vpt *= 2;
    int threads = ((nvec + vpt - 1) / vpt + 31) / 32 * 32;
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
    if (vpt == 0) return cudaLaunchKernelEx(&cfg, add_rmsnorm_mxfp8_kernel<F16, 0, 1024>, p);
    if (threads <= 256) {
        if (vpt == 1) return cudaLaunchKernelEx(&cfg, add_rmsnorm_mxfp8_kernel<F16, 1, 256>, p);
        if (vpt == 2) return cudaLaunchKernelEx(&cfg, add_rmsnorm_mxfp8_kernel<F16, 2, 256>, p);
        return cudaLaunchKernelEx(&cfg, add_rmsnorm_mxfp8_kernel<F16, 4, 256>, p);
    }
    if (vpt == 1) return cudaLaunchKernelEx(&cfg, add_rmsnorm_mxfp8_kernel<F16, 1, 1024>, p);
    if (vpt == 2) return cudaLaunchKernelEx(&cfg, add_rmsnorm_mxfp8_kernel<F16, 2, 1024>, p);
    return cudaLaunchKernelEx(&cfg, add_rmsnorm_mxfp8_kernel<F16, 4, 1024>, p);
}

}  // namespace

cudaError_t launch_add_rmsnorm_mxfp8(const void *X, int64_t ldx, const void *res, int64_t ldr, const void *w, bool f16,
                                     float eps, int64_t M, int64_t K, void *H, int64_t ldh, void *Y, int64_t ldy,
                                     void *Aq, int64_t ldq, void *sf, int num_sms, cudaStream_t stream)
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
    // constants of the row's reciprocal, each as the sum of two floats
    const double keps = static_cast<double>(eps) * static_cast<double>(K), rootk = std::sqrt(static_cast<double>(K));
    p.keps_hi = static_cast<float>(keps);
    p.keps_lo = std::isinf(p.keps_hi) ? 0.0f : static_cast<float>(keps - p.keps_hi);
    p.rootk_hi = static_cast<float>(rootk);
    p.rootk_lo = static_cast<float>(rootk - p.rootk_hi);
    return f16 ? launch_norm<true>(p, num_sms, stream) : launch_norm<false>(p, num_sms, stream);
}

}  // namespace mxfp4
