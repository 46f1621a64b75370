// Norm and rotation of queries and keys (qk_norm_rope).
//
// Mathematics, per head x of D elements at position p: y = x r w with
// r = (mean x^2 + eps)^-1/2, and pairs (y_i, y_j) turned by the angle i of p. Both
// are linear in x once r is known, so an element is
//   out_i = r (x_i a_i + x_j b_i),  a_i = w_i cos, b_i = -+ w_j sin,
// (r x_i w_i where nothing turns), and a, b are the same for all heads of a token.
//
// Bound: HBM (2 bytes read, 2 written an element). A lane has two 16-byte vectors of a
// head: in the layout of halves the two whose elements turn with each other, so that
// nothing but the sum of squares crosses lanes. A group of LPH lanes has a head, a warp
// heads of one token, which share a and b; four of a group's heads are on their way at a
// time, by cp.async, so that they hold no registers. Arithmetic in pairs of floats (mul
// and fma of f32x2: one issue for two). Measured: 8192 tokens of 64 + 8 heads of 128 51 us (302 MB,
// 45 us at the copy bandwidth), 53 us interleaved, 16 tokens of 32 + 8 2.2 us; one vector a lane with its
// partner by shuffles was 105 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "internal.h"
#include "layer.h"
#include "ptx.cuh"

namespace mxfp4 {

namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;        // heads of a lane group on their way

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

// Two floats in a register pair, and operations on both at once.
struct Pair {
    uint64_t v;
};
__device__ __forceinline__ Pair pair(float x, float y)
{
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p.v) : "f"(x), "f"(y));
    return p;
}
__device__ __forceinline__ float2 floats(Pair p)
{
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p.v));
    return f;
}
__device__ __forceinline__ Pair mul(Pair a, Pair b)
{
    Pair d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}
__device__ __forceinline__ Pair fma(Pair a, Pair b, Pair c)
{
    Pair d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return d;
}

// A vector of eight as four pairs.
struct Vec {
    Pair p[4];
};
// c += a b where `on`.
__device__ __forceinline__ void fma_if(bool on, const Vec &a, const Vec &b, Vec &c)
{
    asm("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %12, 0;\n\t"
        "@p fma.rn.f32x2 %0, %4, %8, %0;\n\t@p fma.rn.f32x2 %1, %5, %9, %1;\n\t"
        "@p fma.rn.f32x2 %2, %6, %10, %2;\n\t@p fma.rn.f32x2 %3, %7, %11, %3;\n\t}"
        : "+l"(c.p[0].v), "+l"(c.p[1].v), "+l"(c.p[2].v), "+l"(c.p[3].v)
        : "l"(a.p[0].v), "l"(a.p[1].v), "l"(a.p[2].v), "l"(a.p[3].v), "l"(b.p[0].v), "l"(b.p[1].v), "l"(b.p[2].v),
          "l"(b.p[3].v), "r"(static_cast<int>(on)));
}
template <bool F16>
__device__ __forceinline__ Vec unpack(const uint4 &v)
{
    float f[8];
    unpack8<F16>(v, f);
    Vec o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.p[i] = pair(f[2 * i], f[2 * i + 1]);
    return o;
}
template <bool F16>
__device__ __forceinline__ uint4 pack(const Vec &v)
{
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = floats(v.p[i]);
        f[2 * i] = t.x;
        f[2 * i + 1] = t.y;
    }
    return pack8<F16>(f);
}

template <int LPH>
__device__ __forceinline__ float group_sum(float v)
{
#pragma unroll
    for (int o = LPH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// For heads whose squares leave fp32, or whose sum is so small that it lost bits and eps
// does not hide it (`odd`): a power of two s that brings the values to about 1, and r for
// the values times s. (By value: with references the vectors of every head went through
// local memory, 70 us instead of 51 at 8192 tokens of 72 heads.)
template <bool F16, int LPH>
__device__ __noinline__ float2 rescaled(uint4 raw0, uint4 raw1, bool odd, float eps, int D)
{
    float x[16];
    unpack8<F16>(raw0, *reinterpret_cast<float(*)[8]>(x));
    unpack8<F16>(raw1, *reinterpret_cast<float(*)[8]>(x + 8));
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(x[i]));
#pragma unroll
    for (int o = LPH / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float s = 1.0f;
    if (odd && top > 0.0f && !isinf(top)) s = exp2f(static_cast<float>(max(-126, min(126, -ilogbf(top)))));
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) ss = fmaf(x[i] * s, x[i] * s, ss);
    ss = group_sum<LPH>(ss);
    const double m = static_cast<double>(ss) / D + static_cast<double>(eps) * s * s;
    return make_float2(s, m == 0.0 ? 0.0f : static_cast<float>(1.0 / sqrt(m)));
}

// Vectors of a head that turn: none, all, or some of them. 8192 tokens of 72 heads of 128: 48.3, 50.8 and 54.6 us (half
// of the head); the code for some took 50.3 and 54.1 for none and all. (With every product taken, those of
// vectors that do not turn by zero, half a head was 52.4 us, but an infinity came out at its neighbour as NaN.)
enum Turning { kNone, kAll, kSome };

// Heads h0 .. h1 - 1 of one token's queries or keys (which: 0, 1).
template <bool F16, bool INTER, int LPH, bool FULL, Turning TURN>
__device__ __forceinline__ void heads_of(const QkParams &p, int which, int64_t t, int64_t pos, int h0, int h1, int j, int hv,
                                         int v0, int v1, bool in0, bool in1, uint4 *slots)
{
    constexpr int G = 32 / LPH;                         // heads a warp has side by side
    const int group = (threadIdx.x & 31) / LPH;
    const int64_t in_step = 2 * G * p.sh[which], out_step = 2 * G * p.osh[which];      // bytes to a group's next head
    const char *src0 = reinterpret_cast<const char *>(p.x[which] + t * p.st[which] + (h0 + group) * p.sh[which] + 8 * v0);
    char *dst0 = reinterpret_cast<char *>(p.out[which] + t * p.ost[which] + (h0 + group) * p.osh[which] + 8 * v0);
    const int far = 16 * (v1 - v0);                      // bytes to the second vector
    // kAhead heads of a lane group are on their way to shared memory; a thread reads what it
    // copied itself, so that nothing but its own copies is waited for
    const uint32_t ring = smem_u32(slots) + threadIdx.x * 16;
    constexpr uint32_t kSecond = kAhead * kThreads * 16;
    auto request = [&](int h, int slot) {
        if (h + group < h1) {
            if (in0) cp_async<16>(ring + slot * (kThreads * 16), src0);
            if (in1) cp_async<16>(ring + slot * (kThreads * 16) + kSecond, src0 + far);
        }
        src0 += in_step;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kAhead - 1; ++i) request(h0 + G * i, i);

    // What an element is multiplied with (a), and what its partner is (b): of vectors that turn only. (A product with
    // zero would take a partner's infinity or NaN to an element that it has nothing to do with.)
    const bool turns0 = TURN == kAll || (TURN == kSome && (INTER ? 8 * v0 < p.rot : j < hv));
    const bool turns1 = TURN == kAll || (TURN == kSome && (INTER ? 8 * v1 < p.rot : j < hv));
    Vec a0, a1, b0, b1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a0.p[i] = a1.p[i] = pair(1.0f, 1.0f);
        b0.p[i] = b1.p[i] = pair(0.0f, 0.0f);
    }
    float bad = 0.0f;                                   // NaN for a position outside the table
    if (p.rot) {
        const float *row = p.table + pos * p.rot, *sines = row + (p.rot >> 1);
        auto turn_pairs = [&](int v, Vec &a, Vec &b) {
            const float4 cs = *reinterpret_cast<const float4 *>(row + 4 * v), sn = *reinterpret_cast<const float4 *>(sines + 4 * v);
            a.p[0] = pair(cs.x, cs.x);
            a.p[1] = pair(cs.y, cs.y);
            a.p[2] = pair(cs.z, cs.z);
            a.p[3] = pair(cs.w, cs.w);
            b.p[0] = pair(-sn.x, sn.x);
            b.p[1] = pair(-sn.y, sn.y);
            b.p[2] = pair(-sn.z, sn.z);
            b.p[3] = pair(-sn.w, sn.w);
        };
        if (pos < 0 || pos >= p.P) {
            bad = __int_as_float(0x7FC00000);
        } else if constexpr (INTER) {
            if (in0 && turns0) turn_pairs(v0, a0, b0);
            if (in1 && turns1) turn_pairs(v1, a1, b1);
        } else if (j < hv) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 cs = *reinterpret_cast<const float4 *>(row + 8 * j + 4 * i);
                const float4 sn = *reinterpret_cast<const float4 *>(sines + 8 * j + 4 * i);
                a0.p[2 * i] = a1.p[2 * i] = pair(cs.x, cs.y);
                a0.p[2 * i + 1] = a1.p[2 * i + 1] = pair(cs.z, cs.w);
                b0.p[2 * i] = pair(-sn.x, -sn.y);
                b0.p[2 * i + 1] = pair(-sn.z, -sn.w);
                b1.p[2 * i] = pair(sn.x, sn.y);
                b1.p[2 * i + 1] = pair(sn.z, sn.w);
            }
        }
    }
    const float least = p.eps < 1e-20f ? 1e-24f : 0.0f;
    const uint16_t *w = p.w[which];
    if (w) {
        const Vec w0 = unpack<F16>(in0 ? *reinterpret_cast<const uint4 *>(w + 8 * v0) : make_uint4(0, 0, 0, 0));
        const Vec w1 = unpack<F16>(in1 ? *reinterpret_cast<const uint4 *>(w + 8 * v1) : make_uint4(0, 0, 0, 0));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a0.p[i] = mul(a0.p[i], w0.p[i]);
            a1.p[i] = mul(a1.p[i], w1.p[i]);
            if constexpr (INTER) {
                const float2 f0 = floats(w0.p[i]), f1 = floats(w1.p[i]);
                b0.p[i] = mul(b0.p[i], pair(f0.y, f0.x));
                b1.p[i] = mul(b1.p[i], pair(f1.y, f1.x));
            } else {
                b0.p[i] = mul(b0.p[i], w1.p[i]);
                b1.p[i] = mul(b1.p[i], w0.p[i]);
            }
        }
    }
    const float inv_d = 1.0f / static_cast<float>(p.D);
    // one head, in the registers of its lane group
    auto turn = [&](const uint4 &raw0, const uint4 &raw1, bool live, uint4 &out0, uint4 &out1) {
        Vec x0 = unpack<F16>(raw0), x1 = unpack<F16>(raw1);
        float r = 1.0f;
        if (w) {
            Pair q = mul(x0.p[0], x0.p[0]), q1 = mul(x1.p[0], x1.p[0]);
#pragma unroll
            for (int i = 1; i < 4; ++i) {
                q = fma(x0.p[i], x0.p[i], q);
                q1 = fma(x1.p[i], x1.p[i], q1);
            }
            const float2 f = floats(q), f1 = floats(q1);
            const float ss = group_sum<LPH>((f.x + f.y) + (f1.x + f1.y));
            r = rsqrtf(fmaf(ss, inv_d, p.eps));
            // 1e36: the sum has not overflowed; 1e-24: squares below 2^-126 are less than 2^-24 of it
            const bool odd = live && !(ss < 1e36f && ss >= least);
            if (__any_sync(0xffffffffu, odd)) {
                const float2 sr = rescaled<F16, LPH>(raw0, raw1, odd, p.eps, p.D);
                if (odd) {
                    r = sr.y;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x0.p[i] = mul(x0.p[i], pair(sr.x, sr.x));
                        x1.p[i] = mul(x1.p[i], pair(sr.x, sr.x));
                    }
                }
            }
        }
        r += bad;
        const Pair r2 = pair(r, r);
        Vec o0, o1, y0 = x1, y1 = x0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o0.p[i] = mul(x0.p[i], a0.p[i]);
            o1.p[i] = mul(x1.p[i], a1.p[i]);
            if constexpr (INTER) {
                const float2 f0 = floats(x0.p[i]), f1 = floats(x1.p[i]);
                y0.p[i] = pair(f0.y, f0.x);
                y1.p[i] = pair(f1.y, f1.x);
            }
            if constexpr (TURN == kAll) {
                o0.p[i] = fma(y0.p[i], b0.p[i], o0.p[i]);
                o1.p[i] = fma(y1.p[i], b1.p[i], o1.p[i]);
            }
        }
        if constexpr (TURN == kSome) {
            fma_if(turns0, y0, b0, o0);
            fma_if(turns1, y1, b1, o1);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o0.p[i] = mul(o0.p[i], r2);
            o1.p[i] = mul(o1.p[i], r2);
        }
        out0 = pack<F16>(o0);
        out1 = pack<F16>(o1);
    };
    int slot = 0;
    for (int h = h0; h < h1; h += G) {
        request(h + G * (kAhead - 1), (slot + kAhead - 1) % kAhead);
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
        const bool live = h + group < h1;
        uint4 raw0 = make_uint4(0, 0, 0, 0), raw1 = raw0, o0, o1;
        if (FULL || in0) raw0 = slots[slot * kThreads + threadIdx.x];
        if (FULL || in1) raw1 = slots[(kAhead + slot) * kThreads + threadIdx.x];
        turn(raw0, raw1, live, o0, o1);
        if (live && in0) *reinterpret_cast<uint4 *>(dst0) = o0;
        if (live && in1) *reinterpret_cast<uint4 *>(dst0 + far) = o1;
        dst0 += out_step;
        slot = (slot + 1) % kAhead;
    }
}

template <bool F16, bool INTER, int LPH, bool FULL, Turning TURN>
__global__ void __launch_bounds__(kThreads, 3) qk_norm_rope_kernel(const QkParams p)
{
    __shared__ uint4 slots[2 * kAhead * kThreads];
    const int j = threadIdx.x & (LPH - 1);
    const uint32_t item = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const uint32_t t = item / p.units, unit = item - t * p.units;
    if (t >= p.T) return;                               // whole warps
    // heads of this warp, queries before keys
    const int h0 = unit * p.unit_heads, h1 = min(p.heads[0] + p.heads[1], h0 + p.unit_heads);

    // Vectors of this lane. Halves: those that turn with each other, and two of the rest for
    // the lanes behind; pairs: any two.
    const int nv = p.D >> 3, hv = INTER ? 0 : p.rot >> 4, half_rest = (nv - 2 * hv + 1) >> 1;
    const bool in0 = j < hv + half_rest;
    const int v0 = j < hv ? j : j + hv, v1 = v0 + (j < hv ? hv : half_rest);
    const bool in1 = in0 && v1 < nv;

    grid_dependency_wait();
    grid_launch_dependents();
    int64_t pos = 0;
    if (p.rot) pos = p.pos64 ? static_cast<const int64_t *>(p.positions)[t] : static_cast<const int32_t *>(p.positions)[t];
    const int hq = p.heads[0];
    if (h0 < hq) heads_of<F16, INTER, LPH, FULL, TURN>(p, 0, t, pos, h0, min(h1, hq), j, hv, v0, v1, in0, in1, slots);
    if (h1 > hq) heads_of<F16, INTER, LPH, FULL, TURN>(p, 1, t, pos, max(h0, hq) - hq, h1 - hq, j, hv, v0, v1, in0, in1, slots);
}

template <bool F16, bool INTER, int LPH>
cudaError_t launch_lph(QkParams p, int num_sms, cudaStream_t stream)
{
    // A warp takes as many of a token's heads, as still leave
    // three rounds of 24 warps an SM; below that one head a lane group.
    constexpr int G = 32 / LPH;
    const int heads = p.heads[0] + p.heads[1], all = (heads + G - 1) / G;
    p.unit_heads = G * static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(all, p.T * all / (int64_t(num_sms) * 24 * 3))));
    p.units = (heads + p.unit_heads - 1) / p.unit_heads;
    const int64_t items = p.T * p.units;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((items + kThreads / 32 - 1) / (kThreads / 32)));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // every lane has two vectors of a head of 64, 128 or 256
    const bool full = p.D == 16 * LPH;
    if (p.rot == p.D)
        return full ? cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<F16, INTER, LPH, true, kAll>, p)
                    : cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<F16, INTER, LPH, false, kAll>, p);
    if (p.rot)
        return full ? cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<F16, INTER, LPH, true, kSome>, p)
                    : cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<F16, INTER, LPH, false, kSome>, p);
    return full ? cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<F16, false, LPH, true, kNone>, p)
                : cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<F16, false, LPH, false, kNone>, p);
}

template <bool F16, bool INTER>
cudaError_t launch_type(const QkParams &p, int num_sms, cudaStream_t stream)
{
    if (p.D <= 64) return launch_lph<F16, INTER, 4>(p, num_sms, stream);
    if (p.D <= 128) return launch_lph<F16, INTER, 8>(p, num_sms, stream);
    return launch_lph<F16, INTER, 16>(p, num_sms, stream);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkParams &p, bool f16, bool interleaved, int num_sms, cudaStream_t stream)
{
    if (f16) return interleaved ? launch_type<true, true>(p, num_sms, stream) : launch_type<true, false>(p, num_sms, stream);
    return interleaved ? launch_type<false, true>(p, num_sms, stream) : launch_type<false, false>(p, num_sms, stream);
}

}  // namespace mxfp4
