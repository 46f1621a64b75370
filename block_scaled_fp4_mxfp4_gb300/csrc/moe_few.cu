// The feed-forward half of a mixture-of-experts layer for a few tokens
// (mxfp4_moe_layer).
//
// Mathematics, for token t: h = x + residual, r = (mean h^2 + eps)^-1/2, y = h r w,
// logits z_e = r sum_k h_k w_k Wr[e, k], the k best experts and their weights, then
//   act = MXFP8(silu(G_e q) * (U_e q)),  q = MXFP8(y),  out_t = sum_j w_tj (W2_e act).
//
// Four launches, each one starting while the last drains:
//   router   blocks take 64 channels each: h, sums of squares and of the router's
//            products over them, for all tokens
//   tokens   a block or two a token: adds those sums in two floats, y in MXFP8, routing
//   experts  both products. Weights are what there is to read, so the
//            kernel is a stream of them into a ring of shared memory, by TMA, as they
//            lie in memory, and tcgen05.mma kind::mxf4 of them with the activations'
//            digits (below). (mxfp4_moe_experts multiplies with kind::mxf8f6f4, which
//            takes E2M1 in 8-bit containers: widening them in shared memory holds a decoding
//            batch at half of HBM's rate. Widening in registers for mma.sync was measured
//            too: 90 instructions for 512 weights, 114 us where the stream takes 28.)
//   sum      the weighted sum of a token's rows, in the order of its choices
//
// Units of work: 32 channels of an expert in product 1 (their rows of G and of U: a block of
// the activations' MXFP8), 128 in product 2, each for up to four of its tokens: more than
// four take another unit, whose weights come from L2. Blocks claim them from one counter,
// product 1 first, so that a unit that waits for activations only waits for units that
// somebody already works on: no assumption on which blocks run at the same time. While it
// waits, its weights fill the ring. (Units of 64 channels were as many as the blocks for one
// token, all ended at once, and product 2 stood still for 6 us until their results were
// published: 45.5 us, 44.8 with 32.)
//
// Bound: HBM, the weights of the experts that some token chose: they stream at 6 to 6.5 TB/s in product 1, 60 to 65 % of
// HBM's rate over the experts' kernel. Routing before them takes 7 us and the last unit and the sum
// 4. Measured on the device, inputs changing: 1 token x 8 of 32 experts (7168 x 2048, 187 MB, 28 us
// at the copy bandwidth) 43.8 us, 16 x 8 of 128 (2048 x 768, 207 MB, 31 us) 42.4 us, 5 x 6 of 40 (2560 x
// 1408, 128 MB, 19 us) 34.4 us; the four calls for any number of tokens 63, 61 and 50 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <cstddef>
#include <cstring>

#include "internal.h"
#include "moe.h"
#include "mxfp8_math.cuh"
#include "ptx.cuh"

namespace mxfp4 {

__device__ int g_moe_few_error;

namespace {

constexpr int kMaxTokens = kMoeFewTokens;
constexpr int kMaxExperts = 512;
constexpr int kMaxChoices = kMaxTokens * 32;

// ------------------------------------------------------------------ digits
//
// The products run in kind::mxf4, whose operands are both E2M1: weights as they lie in
// memory. An MXFP8 activation goes in as six E2M1 columns: the magnitude of an E4M3
// value is a whole number n < 2^18 of 2^-9, and n = sum_i d_i 8^i with d_i in -3 .. 4 for
// i < 5; what is left for i = 5 is 0 .. 7, and 5 and 7 become 6 with d_4 less or more by 8
// (n has four significant bits: d_4 is then a multiple of 4 from 0 to 4). All of 0, 1, 2, 3, 4, 6, 8
// are twice an E2M1 value, so digit i enters with the scale 2^(e - 8 + 3 i), e the
// exponent of the activation's own scale, and the six columns' sums add up to the product
// of the activation itself: every term is exact.

// E8M0 byte of digit i where the activations' byte is b (255: NaN).
__device__ __forceinline__ uint32_t digit_scale(uint32_t b, int i)
{
    return b == 255 ? 255 : max(static_cast<int>(b) - 8 + 3 * i, 0);
}

// The six digits of the magnitudes of all E4M3 codes, four bits each as E2M1, d_0 lowest.
struct DigitTable {
    uint32_t of[128];
};
constexpr DigitTable digit_table()
{
    DigitTable t{};
    for (int c = 0; c < 128; ++c) {
        const int ex = c >> 3, m = c & 7;
        int n = c == 127 ? 0 : (ex ? (8 + m) << (ex - 1) : m);      // 127: NaN, its scale says so
        int d[6] = {};
        for (int i = 0; i < 5; ++i) {
            d[i] = ((n + 3) & 7) - 3;
            n = (n - d[i]) / 8;
        }
        d[5] = n;
        if (n == 5 || n == 7) {
            d[5] = 6;
            d[4] += n == 5 ? -8 : 8;
        }
        for (int i = 0; i < 6; ++i) {
            const int a = d[i] < 0 ? -d[i] : d[i];
            t.of[c] |= static_cast<uint32_t>((a <= 4 ? a : a / 2 + 2) | (d[i] < 0 ? 8 : 0)) << (4 * i);
        }
    }
    return t;
}
__constant__ DigitTable kDigits = digit_table();

// A copy of it in shared memory, where lanes may look up different codes at once; of
// the block's first 128 threads.
__device__ __forceinline__ void copy_digits(uint32_t (&table)[128])
{
    if (threadIdx.x < 128) table[threadIdx.x] = kDigits.of[threadIdx.x];
}

// The six digits of an E4M3 code in a block whose scale byte is b, four bits each. Those
// whose scale lies below 2^-127 are left out.
__device__ __forceinline__ uint32_t digits_of(const uint32_t (&table)[128], uint32_t c, uint32_t b)
{
    uint32_t d = table[c & 0x7Fu] ^ (c & 0x80u ? 0x888888u : 0u);
#pragma unroll
    for (int i = 0; i < 3; ++i)
        if (b + 3 * i < 8) d &= ~(0xFu << (4 * i));
    return d;
}

// Eight E2M1 codes a digit of y (four bits each, the first lowest), y of a block whose
// MXFP8 scale byte is b.
__device__ __forceinline__ void digits_of(const uint32_t (&table)[128], const float (&y)[8], uint32_t b, uint32_t (&out)[6])
{
    const float inv = mxfp8_scale_inverse(b);
    uint32_t codes[2];
    codes[0] = e4m3x4_rn(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
    codes[1] = e4m3x4_rn(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv);
#pragma unroll
    for (int i = 0; i < 6; ++i) out[i] = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t c = (codes[j >> 2] >> (8 * (j & 3))) & 0xFFu;
        const uint32_t d = digits_of(table, c, b);
#pragma unroll
        for (int i = 0; i < 6; ++i) out[i] |= ((d >> (4 * i)) & 0xFu) << (4 * j);
    }
}

// ------------------------------------------------------------------ router

constexpr int kSlice = 64;              // channels of a block
constexpr int kRouterThreads = 256;
constexpr int kSub = 20;                // floats from one 16 channels to the next, spread over the banks

struct RouterParams {
    const uint16_t *x, *res, *w, *router;
    int64_t ldx, ldr;
    uint16_t *h;                        // [T, H]
    float *part;                        // [slices][T][E]
    float *part_ss;                     // [slices][T]
    int *counters;                      // of the experts' kernel, set to zero here
    int num_counters;
    int T, H, E;
};

__device__ __forceinline__ float2 bf16x2(uint32_t v)
{
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}

__global__ void __launch_bounds__(kRouterThreads) moe_few_router_kernel(const RouterParams p)
{
    __shared__ __align__(16) float hw[kMaxTokens][4 * kSub];
    const int tid = threadIdx.x, k0 = blockIdx.x * kSlice;
    grid_dependency_wait();
    grid_launch_dependents();
    if (blockIdx.y == 0)
        for (int i = blockIdx.x * kRouterThreads + tid; i < p.num_counters; i += gridDim.x * kRouterThreads) p.counters[i] = 0;
    // four neighbouring lanes take 16 channels each of one expert, a block 64 experts
    const int sub = tid & 3;
    const int e = blockIdx.y * (kRouterThreads / 4) + (tid >> 2);
    float wr[16];
    {
        uint4 a = make_uint4(0, 0, 0, 0), b = a;
        if (e < p.E) {
            const uint4 *src = reinterpret_cast<const uint4 *>(p.router + static_cast<int64_t>(e) * p.H + k0 + 16 * sub);
            a = __ldg(src);
            b = __ldg(src + 1);
        }
        const uint32_t r[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 f = bf16x2(r[i]);
            wr[2 * i] = f.x;
            wr[2 * i + 1] = f.y;
        }
    }
    // eight neighbouring threads have the 64 channels of a token; whole warps go on for the shuffles
    const int t = tid >> 3, v = tid & 7, c = k0 + 8 * v;
    if ((t & ~3) < p.T) {
        float ss = 0.0f;
        if (t < p.T) {
            const uint4 xv = *reinterpret_cast<const uint4 *>(p.x + t * p.ldx + c);
            uint32_t hv[4] = {xv.x, xv.y, xv.z, xv.w};
            if (p.res) {
                const uint4 rv = *reinterpret_cast<const uint4 *>(p.res + t * p.ldr + c);
                const uint32_t r[4] = {rv.x, rv.y, rv.z, rv.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 a = bf16x2(hv[i]), b = bf16x2(r[i]);
                    const __nv_bfloat162 s = __floats2bfloat162_rn(a.x + b.x, a.y + b.y);
                    hv[i] = *reinterpret_cast<const uint32_t *>(&s);
                }
            }
            const uint4 h4 = make_uint4(hv[0], hv[1], hv[2], hv[3]);
            if (blockIdx.y == 0) *reinterpret_cast<uint4 *>(p.h + static_cast<int64_t>(t) * p.H + c) = h4;
            const uint4 wv = *reinterpret_cast<const uint4 *>(p.w + c);
            const uint32_t w[4] = {wv.x, wv.y, wv.z, wv.w};
            float *o = &hw[t][(v >> 1) * kSub + (v & 1) * 8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 a = bf16x2(hv[i]), b = bf16x2(w[i]);
                ss = fmaf(a.x, a.x, fmaf(a.y, a.y, ss));
                o[2 * i] = a.x * b.x;      // exact: 8 bits by 8
                o[2 * i + 1] = a.y * b.y;
            }
        }
        ss += __shfl_xor_sync(0xffffffffu, ss, 1);
        ss += __shfl_xor_sync(0xffffffffu, ss, 2);
        ss += __shfl_xor_sync(0xffffffffu, ss, 4);
        if (t < p.T && v == 0 && blockIdx.y == 0) p.part_ss[blockIdx.x * p.T + t] = ss;
    }
    __syncthreads();
    if ((e & ~7) < p.E) {
        for (int tk = 0; tk < p.T; ++tk) {
            const float4 *q = reinterpret_cast<const float4 *>(&hw[tk][sub * kSub]);
            // four chains of four: a product (exact: 16 bits by 8) passes three additions there, two that join
            // the chains and two that join the lanes. One chain lost small terms behind a large one in 15.
            float4 s4;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 f = q[i];
                s4.x = i ? fmaf(f.x, wr[4 * i], s4.x) : f.x * wr[0];
                s4.y = i ? fmaf(f.y, wr[4 * i + 1], s4.y) : f.y * wr[1];
                s4.z = i ? fmaf(f.z, wr[4 * i + 2], s4.z) : f.z * wr[2];
                s4.w = i ? fmaf(f.w, wr[4 * i + 3], s4.w) : f.w * wr[3];
            }
            float s = (s4.x + s4.y) + (s4.z + s4.w);
            s += __shfl_xor_sync(0xffffffffu, s, 1);
            s += __shfl_xor_sync(0xffffffffu, s, 2);
            if (sub == 0 && e < p.E) p.part[(static_cast<int64_t>(blockIdx.x) * p.T + tk) * p.E + e] = s;
        }
    }
}

// ------------------------------------------------------------------ tokens

constexpr int kTokenThreads = 512;

struct TokenParams {
    const uint16_t *h, *w, *router;
    const float *part, *part_ss;
    const float *bias;                  // [E] or null
    uint8_t *xd;                        // [T][6][H / 2] digits of y
    uint32_t *xsf;                      // [T][H / 128][8] their scales, four blocks of 32 a word, six words used
    uint16_t *h_out;                    // the caller's, or null
    int64_t ldh;
    int *ids;                           // [T, k], of the workspace
    float *weights;
    int *ids_out;                       // the caller's, or null
    float *weights_out;
    int T, H, E, k, slices, groups, topk_groups, group_top, sigmoid, renorm;
    float eps, heps, root_h, scale;     // H eps, sqrt(H)
};

// A key that orders as the values do, NaN above all; 0 stands for "none".
__device__ __forceinline__ uint32_t order_key(float v)
{
    const uint32_t b = __float_as_uint(v);
    if (isnan(v)) return 0xFFFFFFFFu;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
constexpr uint32_t kKeyNone = 0x007FFFFFu;      // of -infinity: neither it nor what lies below is chosen

__device__ __forceinline__ float key_value(uint32_t key)
{
    return __uint_as_float(key == 0xFFFFFFFFu ? 0x7FC00000u : (key & 0x80000000u ? key & 0x7FFFFFFFu : ~key));
}

// An unevaluated sum of two floats, and what is added to it: by error-free additions of
// the high parts, the low ones in fp32.
struct Two {
    float hi, lo;
};
__device__ __forceinline__ void add(Two &a, float hi, float lo)
{
    const float s = a.hi + hi, b = s - a.hi;
    a.lo += ((a.hi - (s - b)) + (hi - b)) + lo;
    a.hi = s;
}

// Rows are taken as they are while the sum of their squares and H eps lie in these bounds: squares and products with
// weights (up to 2^40) and the router's elements (up to 2^20) then stay in fp32.
constexpr float kLeastSum = 0x1p-80f, kMostSum = 0x1p100f;

// Other rows, by a whole block: a power of two s that brings the largest value to 1 or 2, and r for the values times s.
// Rows of zeros, and such that are not finite, keep what they have (s = 0). (A pass over the row, and over the router's matrix
// for its logits: 31 us more for a token of 7168 channels and 32 experts.)
__device__ __noinline__ float2 rescaled(const TokenParams &p, int t, uint32_t *top, float2 *part)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint4 *row = reinterpret_cast<const uint4 *>(p.h + static_cast<int64_t>(t) * p.H);
    uint32_t most = 0;
    for (int v = tid; v < p.H / 8; v += kTokenThreads) {
        const uint4 h = row[v];
        const uint32_t a[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) most = max(most, max(a[i] & 0x7FFFu, a[i] >> 16 & 0x7FFFu));
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) top[warp] = most;
    __syncthreads();
    most = __reduce_max_sync(0xffffffffu, top[lane % (kTokenThreads / 32)]);
    if (most == 0 || most >= 0x7F80u) return make_float2(0.0f, 0.0f);
    const int e = max(-126, min(126, ilogbf(__uint_as_float(most << 16))));
    const float s = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    Two ss{0.0f, 0.0f};
    for (int v = tid; v < p.H / 8; v += kTokenThreads) {
        const uint4 h = row[v];
        const uint32_t a[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = bf16x2(a[i]);
            add(ss, f.x * s * (f.x * s), 0.0f);
            add(ss, f.y * s * (f.y * s), 0.0f);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) add(ss, __shfl_xor_sync(0xffffffffu, ss.hi, o), __shfl_xor_sync(0xffffffffu, ss.lo, o));
    if (lane == 0) part[warp] = make_float2(ss.hi, ss.lo);
    __syncthreads();
    double m = 0.0;
    for (int i = 0; i < kTokenThreads / 32; ++i) m += static_cast<double>(part[i].x) + part[i].y;
    m = m / p.H + static_cast<double>(p.eps) * s * s;
    return make_float2(s, static_cast<float>(1.0 / sqrt(m)));
}

// Their logits: a warp an expert.
__device__ __noinline__ void rescaled_logits(const TokenParams &p, int t, float2 sr, float *logit)
{
    const int lane = threadIdx.x & 31;
    const uint4 *row = reinterpret_cast<const uint4 *>(p.h + static_cast<int64_t>(t) * p.H);
    for (int e = threadIdx.x >> 5; e < p.E; e += kTokenThreads / 32) {
        const uint4 *weights = reinterpret_cast<const uint4 *>(p.router + static_cast<int64_t>(e) * p.H);
        Two z{0.0f, 0.0f};
        for (int v = lane; v < p.H / 8; v += 32) {
            const uint4 h = row[v], w = reinterpret_cast<const uint4 *>(p.w)[v], q = weights[v];
            const uint32_t a[4] = {h.x, h.y, h.z, h.w}, b[4] = {w.x, w.y, w.z, w.w}, c[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = bf16x2(a[i]), g = bf16x2(b[i]), k = bf16x2(c[i]);
                add(z, f.x * sr.x * g.x * k.x, 0.0f);
                add(z, f.y * sr.x * g.y * k.y, 0.0f);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) add(z, __shfl_xor_sync(0xffffffffu, z.hi, o), __shfl_xor_sync(0xffffffffu, z.lo, o));
        if (lane == 0) logit[e] = (z.hi + z.lo) * sr.y;
    }
}

// Grid: tokens x parts of their channels; the first part of a token routes it too.
__global__ void __launch_bounds__(kTokenThreads) moe_few_token_kernel(const __grid_constant__ TokenParams p)
{
    __shared__ float2 sums[kTokenThreads];
    __shared__ float logit[kMaxExperts], chosen_score[32];
    __shared__ uint32_t keys[kMaxExperts], group_key[kMaxExperts];
    __shared__ int rank[kMaxExperts], chosen[32];
    __shared__ float r_shared;
    __shared__ int odd;                  // a row that is taken times a power of two
    __shared__ uint32_t table[128];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, t = blockIdx.x;
    const int v = blockIdx.y * kTokenThreads + tid;          // this thread's eight channels
    const bool in = v < p.H / 8;                             // H / 8 is a multiple of 16: whole groups of four
    copy_digits(table);
    // the launch before let this one start when all of its inputs were there
    const uint4 wv = in ? *reinterpret_cast<const uint4 *>(p.w + 8 * v) : make_uint4(0, 0, 0, 0);
    grid_dependency_wait();
    grid_launch_dependents();
    const uint4 hv = in ? *reinterpret_cast<const uint4 *>(p.h + static_cast<int64_t>(t) * p.H + 8 * v) : make_uint4(0, 0, 0, 0);

    // r, by one warp
    if (warp == 0) {
        Two ss{0.0f, 0.0f};
        for (int s0 = 0; s0 < p.slices; s0 += 128) {
            float f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = s0 + 32 * i + lane < p.slices ? p.part_ss[(s0 + 32 * i + lane) * p.T + t] : 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) add(ss, f[i], 0.0f);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) add(ss, __shfl_xor_sync(0xffffffffu, ss.hi, o), __shfl_xor_sync(0xffffffffu, ss.lo, o));
        if (lane == 0) {
            // a root of fp32 and one step of Newton's method: m r^2 - 1 to 2^-40. (Below 2^-125 r^2 may leave fp32; a
            // row of zeros keeps the 0, any other is taken again.)
            add(ss, p.heps, 0.0f);
            const float r0 = rsqrtf(ss.hi);
            const float q = r0 * r0, qe = fmaf(r0, r0, -q);
            const float e = fmaf(ss.hi, q, -1.0f) + (fmaf(ss.hi, qe, ss.lo * q));
            r_shared = ss.hi < 0x1p-125f || isinf(ss.hi) ? 0.0f : fmaf(r0 * p.root_h, -0.5f * e, r0 * p.root_h);
            odd = !(ss.hi >= kLeastSum && ss.hi <= kMostSum);
        }
    }
    // logits: `parts` threads an expert over interleaved slices, added in a fixed order
    const int parts = kTokenThreads / p.E;           // E <= 512
    if (blockIdx.y == 0) {
        Two z{0.0f, 0.0f};
        const int e = tid % p.E, part = tid / p.E;
        if (part < parts) {
            const float *src = p.part + static_cast<int64_t>(t) * p.E + e;
            const int64_t step = static_cast<int64_t>(p.T) * p.E;
            for (int s0 = part; s0 < p.slices; s0 += 8 * parts) {
                float f[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = s0 + i * parts < p.slices ? src[(s0 + i * parts) * step] : 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) add(z, f[i], 0.0f);
            }
        }
        sums[tid] = make_float2(z.hi, z.lo);
    }
    __syncthreads();
    float rf = r_shared, hs = 1.0f;
    bool again = false;
    if (odd) {
        const float2 sr = rescaled(p, t, keys, sums);
        again = sr.x != 0.0f;
        if (again) {
            hs = sr.x;
            rf = sr.y;
        }
    }
    {
        // y in MXFP8, four lanes a block of 32
        // only now: H may be X or residual, which the launch before read
        if (in && p.h_out) *reinterpret_cast<uint4 *>(p.h_out + t * p.ldh + 8 * v) = hv;
        const uint32_t ha[4] = {hv.x, hv.y, hv.z, hv.w}, wa[4] = {wv.x, wv.y, wv.z, wv.w};
        float y[8];
        uint32_t amax = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 a = bf16x2(ha[i]), b = bf16x2(wa[i]);
            y[2 * i] = a.x * hs * b.x * rf;
            y[2 * i + 1] = a.y * hs * b.y * rf;
            amax = max(amax, max(__float_as_uint(y[2 * i]) & 0x7FFFFFFFu, __float_as_uint(y[2 * i + 1]) & 0x7FFFFFFFu));
        }
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        if (in) {
            const uint32_t b = mxfp8_scale_byte(amax);
            uint32_t dg[6];
            digits_of(table, y, b, dg);
            uint8_t *o = p.xd + static_cast<size_t>(t) * 6 * (p.H >> 1) + 4 * v;
#pragma unroll
            for (int d = 0; d < 6; ++d) *reinterpret_cast<uint32_t *>(o + static_cast<size_t>(d) * (p.H >> 1)) = dg[d];
            if ((v & 3) == 0) {
                uint8_t *f = reinterpret_cast<uint8_t *>(p.xsf + (static_cast<size_t>(t) * (p.H >> 7) + (v >> 4)) * 8) + ((v >> 2) & 3);
#pragma unroll
                for (int d = 0; d < 6; ++d) f[4 * d] = static_cast<uint8_t>(digit_scale(b, d));
            }
        }
    }
    if (blockIdx.y > 0) return;
    if (again) {
        rescaled_logits(p, t, make_float2(hs, rf), logit);
    } else if (tid < p.E) {
        Two z{sums[tid].x, sums[tid].y};
        for (int i = 1; i < parts; ++i) add(z, sums[i * p.E + tid].x, sums[i * p.E + tid].y);
        logit[tid] = (z.hi + z.lo) * rf;
    }
    __syncthreads();
    // scores: every warp finds the largest logit and the sum by itself
    float largest = -INFINITY, sum = 0.0f;
    if (!p.sigmoid) {
        bool nan = false;
        for (int e = lane; e < p.E; e += 32) {
            largest = fmaxf(largest, logit[e]);
            nan |= isnan(logit[e]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) largest = fmaxf(largest, __shfl_xor_sync(0xffffffffu, largest, o));
        for (int e = lane; e < p.E; e += 32) sum += logit[e] > -INFINITY ? expf(logit[e] - largest) : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (__any_sync(0xffffffffu, nan)) sum = __int_as_float(0x7FC00000);
    }
    float s = 0.0f;
    uint32_t key = 0;                        // of this thread's expert; 0 where there is none
    if (tid < p.E) {
        const float z = logit[tid];
        if (p.sigmoid)
            s = 1.0f / (1.0f + expf(-z));
        else if (isnan(sum))
            s = sum;
        else
            s = sum > 0.0f && z > -INFINITY ? expf(z - largest) / sum : 0.0f;
        // without a bias and groups the logits rank the experts as the scores do, also where those saturate
        float c = p.bias || p.groups > 1 ? s + (p.bias ? p.bias[tid] : 0.0f) : (isnan(s) ? s : z);
        if (z == -INFINITY) c = -INFINITY;
        key = order_key(c);
        keys[tid] = key;
        rank[tid] = 0;
    }
    __syncthreads();
    const int n = p.E / p.groups;
    if (p.groups > 1) {
        // a group's score: the sum of its best, or two best
        for (int g = warp; g < p.groups; g += kTokenThreads / 32) {
            uint32_t k1 = 0, k2 = 0;
            for (int i = lane; i < n; i += 32) {
                const uint32_t k = keys[g * n + i];
                if (k > k1) {
                    k2 = k1;
                    k1 = k;
                } else if (k > k2) {
                    k2 = k;
                }
            }
            const uint32_t top = __reduce_max_sync(0xffffffffu, k1);
            const unsigned who = __ballot_sync(0xffffffffu, k1 == top);
            if (lane == __ffs(who) - 1) k1 = k2;
            const uint32_t second = __reduce_max_sync(0xffffffffu, k1);
            // half of a sum of two, which cannot overflow
            if (lane == 0)
                group_key[g] = order_key(p.group_top == 2 && n > 1 ? 0.5f * key_value(top) + 0.5f * key_value(second) : key_value(top));
        }
        __syncthreads();
        if (tid < p.E) {
            const int own = tid / n;
            int before = 0;
            for (int g = 0; g < p.groups; ++g) before += group_key[g] > group_key[own] || (group_key[g] == group_key[own] && g < own);
            if (before >= p.topk_groups) keys[tid] = key = 0;
        }
        __syncthreads();
    }
    // An expert's place is the number of those before it: larger keys, and equal ones with a
    // lower index. `parts` threads count for one expert.
    {
        const int e = tid % p.E, part = tid / p.E;
        if (part < parts) {
            const uint32_t own = keys[e];
            const int per = (p.E + parts - 1) / parts, end = min(p.E, (part + 1) * per);
            int before = 0;
            for (int i = part * per; i < end; ++i) before += keys[i] > own || (keys[i] == own && i < e);
            if (before) atomicAdd(&rank[e], before);
        }
    }
    if (tid < 32) chosen[tid] = -1;
    __syncthreads();
    if (tid < p.E && key > kKeyNone && rank[tid] < p.k) {
        chosen[rank[tid]] = tid;
        chosen_score[rank[tid]] = s;
    }
    __syncthreads();
    if (warp == 0) {
        const int id = lane < p.k ? chosen[lane] : -1;
        float w = id >= 0 ? chosen_score[lane] : 0.0f;
        if (p.renorm) {
            float all = w;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
            w = w / (all + 1e-20f);
        }
        w *= p.scale;
        if (lane < p.k) {
            p.ids[t * p.k + lane] = id;
            p.weights[t * p.k + lane] = w;
            if (p.ids_out) p.ids_out[t * p.k + lane] = id;
            if (p.weights_out) p.weights_out[t * p.k + lane] = w;
        }
    }
}

// ----------------------------------------------------------------- experts

constexpr int kExpertThreads = 352;
constexpr int kRoom = 4;                                 // tokens of a unit at most
constexpr int kMaxEntries = kMaxChoices;
constexpr int kMaxStages = 4;
constexpr int kMadeAt = 32;                              // counters of the entries behind the queue's
// A stage holds 16 KB of weights: in product 1 64 rows x 512 elements, as two tiles of 256
// elements one after another, in product 2 one tile of 128 rows x 256. (An MMA takes 128
// rows: of a tile of 64 the other 64 are whatever follows it, and so are their sums.)
constexpr uint32_t kStageWeights = 128 * 128;
constexpr uint32_t kStageScales = 2048;                  // four blocks of 512 bytes: of the weights, then of the tokens
constexpr uint32_t kTokenTile = 1024;                    // of a token: eight rows (six used) x 256 elements
constexpr uint32_t kTokenBytes = 2 * kTokenTile;
constexpr uint32_t kAccColumns = 8 * kRoom;
constexpr uint32_t kSfColumns = 32;                      // of a stage: four blocks of weights, four of tokens
constexpr uint32_t kTmemColumns = 256;
static_assert(2 * kAccColumns + kMaxStages * kSfColumns <= kTmemColumns, "TMEM budget: half of it, two blocks an SM");

struct ExpertsParams {
    CUtensorMap tm_w13;                 // packed weights [E * 2I, H / 2] u8, box 128 bytes x 32 rows
    CUtensorMap tm_w2;                  // the same of [E * H, I / 2], box 64 rows
    const uint8_t *w13_sf, *w2_sf;
    const uint8_t *xd;                  // [T][6][H / 2] digits of the tokens
    const uint32_t *xsf;                // [T][H / 128][8] their scales
    const int *ids;
    uint8_t *ad;                        // [T * k][6][I / 2] of the activations
    uint32_t *asf;                      // [T * k][I / 128][8]
    float *y;                           // [T * k, H]
    int *queue;                         // units claimed
    int *made;                          // [entries] rows of units of an entry's product 1 that are complete
    int T, k, E, H, I;
    int stages, room;                   // stages of the ring, tokens that one has room for
    uint64_t wait_ns;
};

// A unit of work: weight tile c of expert e for up to four of its choices.
struct Unit {
    int first;                          // product 1; -1: there are no more units
    int e, c;
    int entry, slots, rows;             // in the list of entries; its first choice in `slot`, and how many
};

struct ExpertsShared {
    float epi[kRoom][64];               // G, then U of 32 channels
    uint64_t w_full[kMaxStages];        // weights have landed
    uint64_t t_full[kMaxStages];        // tokens and scales have landed
    uint64_t empty[kMaxStages];         // the stage's MMAs have completed
    uint64_t unit_full[4], unit_empty[4];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t written[4];                // a unit's results are written
    uint64_t mma_done;
    uint32_t tmem;
    int abort, entries, go[2];
    Unit unit[4];                       // in the order they were claimed
    uint32_t digits[128];
    uint16_t entry_expert[kMaxEntries], entry_slots[kMaxEntries];
    uint16_t slot[kMaxChoices];         // choices t * k + j by expert
    uint16_t start[kMaxExperts];        // the first of an expert's choices there
    uint8_t entry_rows[kMaxEntries];
    uint8_t token[kMaxChoices];         // tokens of the choices in slot
    alignas(16) uint32_t tokens[kMaxExperts];   // a bit for each token that chose the expert
};
static_assert(offsetof(ExpertsShared, w_full) % 8 == 0 && kMaxTokens <= 32, "aligned and sized as it is used");

__device__ __forceinline__ void epilogue_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

__device__ __forceinline__ int load_acquire(const int *p)
{
    int v;
    asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// A position in the ring of stages.
struct Place {
    int slot;
    uint32_t parity;
    __device__ __forceinline__ void step(int n)
    {
        if (++slot == n) {
            slot = 0;
            parity ^= 1u;
        }
    }
};

// Warps:
//   0-3  epilogue of a finished tile while the next one's products run
//   4-7  copy tokens' digits and all scales into the ring by cp.async
//   8    lane 0 claims units and loads their weights by TMA
//   9    issues scale copies and MMAs (an elected lane); owns TMEM
//   10   publishes the activations that the epilogue wrote: a fence for the whole GPU takes
//        two microseconds here, in which the epilogue goes on
// Two blocks share an SM: what a unit costs beside its bytes (a microsecond or two of
// latencies at its start and end) passes while the other block's weights stream.
// Waits name a round of a barrier by its parity. Nobody can be a round behind: the next
// round of a stage needs the TMA thread and every copying thread, the next of a unit's
// entry or of an accumulator everyone who waits for this one.
__global__ void __launch_bounds__(kExpertThreads, 2) moe_few_experts_kernel(const __grid_constant__ ExpertsParams p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int S = p.stages;
    const uint32_t stage_bytes = kStageWeights + 2 * kStageScales + p.room * kTokenBytes;
    ExpertsShared &sh = *reinterpret_cast<ExpertsShared *>(smem + S * stage_bytes);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&sh.w_full[i], 1);
            mbar_init(&sh.t_full[i], 128);
            mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&sh.unit_full[i], 1);
            mbar_init(&sh.unit_empty[i], 7);     // four copying warps, the issuer, the epilogue, the publisher
            mbar_init(&sh.written[i], 4);        // the epilogue's warps
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.acc_full[i], 1);
            mbar_init(&sh.acc_empty[i], 128);
        }
        mbar_init(&sh.mma_done, 1);
        sh.abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&p.tm_w13);
        tma_prefetch_desc(&p.tm_w2);
    }
    copy_digits(sh.digits);
    for (int i = tid; i < kMaxExperts; i += kExpertThreads) sh.tokens[i] = 0;
    if (warp == 9) {
        tmem_alloc(&sh.tmem, kTmemColumns);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, sh.tmem, 0);
    grid_dependency_wait();
    grid_launch_dependents();        // the sum's blocks have room beside this kernel's, and wait
    int claimed = 0;
    if (tid == 256) claimed = atomicAdd(p.queue, 1);     // on its way while the lists are made
    // Choices by expert, and an expert's by token. Every block makes the same list, whatever
    // the order its threads come in: an entry has to be the same tokens for all of them.
    int expert[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int c = tid + i * kExpertThreads;
        expert[i] = c < p.T * p.k ? __ldcg(p.ids + c) : -1;
        if (expert[i] >= 0) atomicOr(&sh.tokens[expert[i]], 1u << (c / p.k));
    }
    __syncthreads();
    if (warp == 0) {
        // a lane takes neighbouring experts
        const int per = (p.E + 31) >> 5, e0 = lane * per, e1 = min(p.E, e0 + per);
        int own = 0;                         // entries << 16 | choices
        for (int e = e0; e < e1; ++e) {
            const int r = __popc(sh.tokens[e]);
            own += ((r + kRoom - 1) / kRoom) << 16 | r;
        }
        int sums = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, sums, o);
            if (lane >= o) sums += x;
        }
        if (lane == 31) sh.entries = sums >> 16;
        int at = (sums - own) >> 16, c0 = (sums - own) & 0xFFFF;
        for (int e = e0; e < e1; ++e) {
            const int r = __popc(sh.tokens[e]);
            sh.start[e] = static_cast<uint16_t>(c0);
            for (int i = 0; i < r; i += kRoom) {
                sh.entry_expert[at] = static_cast<uint16_t>(e);
                sh.entry_slots[at] = static_cast<uint16_t>(c0 + i);
                sh.entry_rows[at++] = static_cast<uint8_t>(min(kRoom, r - i));
            }
            c0 += r;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (expert[i] >= 0) {
            const int c = tid + i * kExpertThreads, t = c / p.k;
            const int at = sh.start[expert[i]] + __popc(sh.tokens[expert[i]] & ((1u << t) - 1));
            sh.slot[at] = static_cast<uint16_t>(c);
            sh.token[at] = static_cast<uint8_t>(t);
        }
    __syncthreads();
    const int tiles1 = p.I >> 5, tiles2 = p.H >> 7, n1 = sh.entries * tiles1, n2 = sh.entries * tiles2;

    if (warp == 8) {
        if (lane == 0) {
            // ---------------------------------------------- weights, by TMA
            const uint64_t pol = policy_evict_first();
            Place at{0, 0};
            int issued = 0;
            bool ok = true;
            // Unit u: product 1 first, entry by entry in both products, so that the first experts'
            // activations are there when product 2 begins.
            auto unit_at = [&](int u) {
                Unit w;
                w.first = u < n1 + n2 ? u < n1 : -1;
                if (w.first < 0) return w;
                const int i = w.first ? u : u - n1, tiles = w.first ? tiles1 : tiles2;
                w.entry = i / tiles;
                w.c = i - w.entry * tiles;
                w.e = sh.entry_expert[w.entry];
                w.slots = sh.entry_slots[w.entry];
                w.rows = sh.entry_rows[w.entry];
                return w;
            };
            // the weight scales of a unit go to L2 ahead of their copies
            auto ask_scales = [&](const Unit &w) {
                if (w.first < 0) return;
                if (w.first) {
                    const uint32_t run = (p.H >> 7) * 512;
                    const size_t blk = static_cast<size_t>(2 * p.I >> 7) * w.e + (w.c >> 2);
                    prefetch_l2_bulk(p.w13_sf + blk * run, run);
                    prefetch_l2_bulk(p.w13_sf + (blk + (p.I >> 7)) * run, run);
                } else {
                    const uint32_t run = (p.I >> 7) * 512;
                    prefetch_l2_bulk(p.w2_sf + (static_cast<size_t>(p.H >> 7) * w.e + w.c) * run, run);
                }
            };
            Unit w = unit_at(claimed);
            ask_scales(w);
            for (int i = 0;; ++i) {
                if (!(ok = mbar_wait(&sh.unit_empty[i & 3], ((i >> 2) & 1) ^ 1u, &g_moe_few_error, kErrWaitEmpty, p.wait_ns)))
                    break;
                sh.unit[i & 3] = w;
                mbar_arrive(&sh.unit_full[i & 3]);
                if (w.first < 0) break;
                const int next = atomicAdd(p.queue, 1);    // on its way while this unit loads
                const int kc = (w.first ? p.H : p.I) >> 7, stages = w.first ? (kc + 3) >> 2 : (kc + 1) >> 1;
                // 32 rows of G and the same of U, or 128 rows
                const int r0 = w.first ? w.e * 2 * p.I + 32 * w.c : w.e * p.H + 128 * w.c;
                for (int ks = 0; ks < stages; ++ks) {
                    if (!(ok = mbar_wait(&sh.empty[at.slot], at.parity ^ 1u, &g_moe_few_error, kErrWaitEmpty, p.wait_ns))) break;
                    uint8_t *st = smem + at.slot * stage_bytes;
                    uint64_t *full = &sh.w_full[at.slot];
                    if (w.first) {
                        const bool two = 4 * ks + 2 < kc;
                        mbar_arrive_expect_tx(full, two ? kStageWeights : kStageWeights / 2);
                        tma_load_2d(st, &p.tm_w13, ks * 256, r0, full, pol);
                        tma_load_2d(st + 4096, &p.tm_w13, ks * 256, r0 + p.I, full, pol);
                        if (two) {
                            tma_load_2d(st + 8192, &p.tm_w13, ks * 256 + 128, r0, full, pol);
                            tma_load_2d(st + 12288, &p.tm_w13, ks * 256 + 128, r0 + p.I, full, pol);
                        }
                    } else {
                        mbar_arrive_expect_tx(full, kStageWeights);
                        tma_load_2d(st, &p.tm_w2, ks * 128, r0, full, pol);
                        tma_load_2d(st + 8192, &p.tm_w2, ks * 128, r0 + 64, full, pol);
                    }
                    ++issued;
                    at.step(S);
                }
                if (!ok) break;
                w = unit_at(next);
                ask_scales(w);
            }
            if (!ok) *reinterpret_cast<volatile int *>(&sh.abort) = 1;
            // copies in flight land before the block leaves
            for (int i = max(0, issued - S); i < issued; ++i)
                mbar_wait(&sh.w_full[i % S], (i / S) & 1, &g_moe_few_error, kErrWaitDrain);
        }
    } else if (warp == 9) {
        // ------------------------------------------------ scales and products
        Place at{0, 0};
        bool ok = true;
        for (int i = 0; ok; ++i) {
            ok = mbar_wait_warp(&sh.unit_full[i & 3], (i >> 2) & 1, &g_moe_few_error, kErrWaitFull, p.wait_ns);
            if (!ok) break;
            const Unit w = sh.unit[i & 3];
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.unit_empty[i & 3]);
            if (w.first < 0) break;
            const int kc = (w.first ? p.H : p.I) >> 7, stages = w.first ? (kc + 3) >> 2 : (kc + 1) >> 1, buf = i & 1;
            ok = mbar_wait_warp(&sh.acc_empty[buf], ((i >> 1) & 1) ^ 1u, &g_moe_few_error, kErrWaitAccum, p.wait_ns);
            if (!ok) break;
            tc_fence_after();
            const uint32_t idesc = __shfl_sync(0xffffffffu, idesc_block_scaled((8 * w.rows + 15) & ~15, true), 0);
            const uint32_t d = tmem + buf * kAccColumns;
            for (int ks = 0; ks < stages; ++ks) {
                ok = mbar_wait_warp(&sh.w_full[at.slot], at.parity, &g_moe_few_error, kErrWaitFull, p.wait_ns) &&
                     mbar_wait_warp(&sh.t_full[at.slot], at.parity, &g_moe_few_error, kErrWaitOperand, p.wait_ns);
                if (!ok) break;
                // cp.async wrote through the generic proxy; scale copies and MMAs read through the async one
                fence_proxy_async_smem();
                tc_fence_after();
                const uint32_t st = smem_u32(smem) + at.slot * stage_bytes;
                const uint64_t ad = sdesc_sw128(st), bd = sdesc_sw128(st + kStageWeights + 2 * kStageScales);
                const uint64_t sd = sdesc_scale(st + kStageWeights);
                const uint32_t tsf = tmem + 2 * kAccColumns + at.slot * kSfColumns;
                if (elect_one()) {
                    // block b of 128 elements: two MMAs of 64
                    auto block = [&](int b, uint32_t accumulate) {
                        const uint64_t a = ad + (b >> 1) * 512 + (b & 1) * 4;
                        const uint64_t x = bd + (b >> 1) * (p.room * (kTokenTile >> 4)) + (b & 1) * 4;
                        const uint32_t sa = tsf + 4 * b, sx = tsf + 16 + 4 * b;
                        tc_cp_scale_block(sa, sd + 32 * b);
                        tc_cp_scale_block(sx, sd + 128 + 32 * b);
                        mma_mxf4(d, a, x, idesc_with_sf_ids(idesc, 0, 0), sa, sx, accumulate);
                        mma_mxf4(d, a + 2, x + 2, idesc_with_sf_ids(idesc, 2, 2), sa, sx, 1u);
                    };
                    const int left = w.first ? kc - 4 * ks : min(2, kc - 2 * ks);
                    block(0, ks > 0 ? 1u : 0u);
                    if (left > 1) block(1, 1u);
                    if (left > 2) block(2, 1u);
                    if (left > 3) block(3, 1u);
                    tc_commit(&sh.empty[at.slot]);
                }
                __syncwarp();
                at.step(S);
            }
            if (!ok) break;
            if (elect_one()) tc_commit(&sh.acc_full[buf]);
            __syncwarp();
        }
        if (!ok) *reinterpret_cast<volatile int *>(&sh.abort) = 1;
        // no MMA may be running when TMEM is released
        if (elect_one()) tc_commit(&sh.mma_done);
        __syncwarp();
        mbar_wait_warp(&sh.mma_done, 0, &g_moe_few_error, kErrWaitDrain);
    } else if (warp == 10) {
        if (lane == 0) {
            // ----------------------------------------------------- publishing
            // It gives up its entry of the ring of units last, so the epilogue is at most four units ahead.
            for (int i = 0;; ++i) {
                if (!mbar_wait(&sh.unit_full[i & 3], (i >> 2) & 1, &g_moe_few_error, kErrWaitFull, p.wait_ns)) break;
                const Unit w = sh.unit[i & 3];
                if (w.first < 0 || !mbar_wait(&sh.written[i & 3], (i >> 2) & 1, &g_moe_few_error, kErrWaitAccum, p.wait_ns)) break;
                if (w.first)
                    // what the epilogue's warps wrote is there before the count says so
                    asm volatile("red.release.gpu.global.add.s32 [%0], %1;" ::"l"(p.made + w.entry), "r"(w.rows) : "memory");
                mbar_arrive(&sh.unit_empty[i & 3]);
            }
        }
    } else if (warp >= 4) {
        // -------------------------------------------------- tokens and scales
        const int t = tid - 128;
        Place at{0, 0};
        int count = 0;
        int ready = -1;                  // entries up to this one have all their activations
        bool ok = true;
        for (int i = 0; ok; ++i) {
            ok = mbar_wait_warp(&sh.unit_full[i & 3], (i >> 2) & 1, &g_moe_few_error, kErrWaitFull, p.wait_ns);
            if (!ok) break;
            const Unit w = sh.unit[i & 3];
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.unit_empty[i & 3]);
            if (w.first < 0) break;
            // row of a choice among the tokens or the activations
            auto row_of = [&](int r) { return static_cast<size_t>(w.first ? sh.token[w.slots + r] : sh.slot[w.slots + r]); };
            const int K = w.first ? p.H : p.I, kc = K >> 7, stages = w.first ? (kc + 3) >> 2 : (kc + 1) >> 1;
            // a row of digits is K / 2 bytes, six of them a token; pieces of 16 bytes, column c of row n at c ^ (n % 8)
            const uint8_t *digits = w.first ? p.xd : p.ad;
            const uint32_t *scales = w.first ? p.xsf : p.asf;
            const uint8_t *src[2] = {nullptr, nullptr};
            uint32_t dst[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int piece = t + 128 * j, r = piece / 48, dc = piece - 48 * r, c = dc & 7, dg = dc >> 3;
                dst[j] = kStageWeights + 2 * kStageScales + (8 * r + dg) * 128 + ((c ^ dg) << 4);
                if (r < w.rows) src[j] = digits + (row_of(r) * 6 + dg) * (K >> 1) + 16 * c;
            }
            const bool low = (t & 7) < 4;                    // columns of a tile's first 128 elements (piece 128 j + t: column t % 8)
            // scale words: thread t < 64 those of blocks t % 2 (and that + 2), digit t / 2 % 8, token t / 16
            const int sr = t >> 4, sdg = (t >> 1) & 7, sblk = t & 1;
            const uint32_t sdst = kStageWeights + kStageScales + sblk * 512 + (8 * sr + sdg) * 16;
            const uint32_t *ssrc = sr < w.rows && sdg < 6 ? scales + (row_of(sr) * kc + sblk) * 8 + sdg : nullptr;
            // scales of the weights, lane l line l of a block: in product 1 the word of each line that
            // is of the 32 rows of G (threads 64 to 95) and of U, in product 2 the whole line
            const uint8_t *wsf = nullptr;
            uint32_t wdst = kStageWeights + lane * 16;
            if (w.first && t >= 64) {
                const size_t blk = static_cast<size_t>(2 * p.I >> 7) * w.e + (w.c >> 2) + (t >= 96 ? p.I >> 7 : 0);
                wsf = p.w13_sf + blk * kc * 512 + lane * 16 + (w.c & 3) * 4;
                wdst += t >= 96 ? 4 : 0;
            } else if (!w.first && t >= 64 && t < 96) {
                wsf = p.w2_sf + (static_cast<size_t>(p.H >> 7) * w.e + w.c) * kc * 512 + lane * 16;
            }
            if (!w.first && w.entry > ready) {
                // this entry's activations have to be there
                int v = 1;
                if (lane == 0) {
                    const uint64_t t0 = global_timer_ns();
                    while (load_acquire(p.made + w.entry) < w.rows * tiles1) {
                        if (global_timer_ns() - t0 > p.wait_ns) {
                            atomicCAS(&g_moe_few_error, 0, kErrWaitOperand);
                            v = 0;
                            break;
                        }
                    }
                }
                ok = __shfl_sync(0xffffffffu, v, 0) != 0;
                __syncwarp();
                if (!ok) break;
                ready = w.entry;
            }
            for (int ks = 0; ks < stages; ++ks) {
                ok = mbar_wait_warp(&sh.empty[at.slot], at.parity ^ 1u, &g_moe_few_error, kErrWaitEmpty, p.wait_ns);
                if (!ok) break;
                const uint32_t st = smem_u32(smem) + at.slot * stage_bytes;
                if (w.first) {
                    const int left = kc - 4 * ks;            // blocks of 128 elements
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        if (src[j] && (left > 1 || low)) cp_async<16>(st + dst[j], src[j] + ks * 256);
                        if (src[j] && (left > 3 || (left > 2 && low)))
                            cp_async<16>(st + dst[j] + p.room * kTokenTile, src[j] + ks * 256 + 128);
                    }
                    if (ssrc && sblk < left) cp_async<4>(st + sdst, ssrc + ks * 32);
                    if (ssrc && sblk + 2 < left) cp_async<4>(st + sdst + 1024, ssrc + ks * 32 + 16);
                    if (wsf)
#pragma unroll
                        for (int b = 0; b < 4; ++b)
                            if (b < left) cp_async<4>(st + wdst + b * 512, wsf + ks * 2048 + b * 512);
                } else {
                    const bool whole = 2 * ks + 1 < kc;
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        if (src[j] && (whole || low)) cp_async<16>(st + dst[j], src[j] + ks * 128);
                    if (ssrc && (whole || sblk == 0)) cp_async<4>(st + sdst, ssrc + ks * 16);
                    if (wsf) {
                        cp_async<16>(st + wdst, wsf + ks * 1024);
                        if (whole) cp_async<16>(st + wdst + 512, wsf + ks * 1024 + 512);
                    }
                }
                cp_async_arrive(&sh.t_full[at.slot]);
                ++count;
                at.step(S);
            }
        }
        if (!ok) *reinterpret_cast<volatile int *>(&sh.abort) = 1;
        cp_async_wait_all();   // also after an abort: nothing of this thread is in flight when the block leaves
        // nor are the arrivals of the last MMAs, which nobody else waits for
        for (int i = max(0, count - S); i < count && ok; ++i)
            ok = mbar_wait_warp(&sh.empty[i % S], (i / S) & 1, &g_moe_few_error, kErrWaitDrain);
    } else {
        // ------------------------------------------------------------ epilogue
        for (int i = 0;; ++i) {
            const int buf = i & 1;
            // one thread waits for all, so that all four warps leave after the same unit
            if (tid == 0) {
                bool ok = mbar_wait(&sh.unit_full[i & 3], (i >> 2) & 1, &g_moe_few_error, kErrWaitFull, p.wait_ns);
                const bool more = ok && sh.unit[i & 3].first >= 0;
                if (more) ok = mbar_wait(&sh.acc_full[buf], (i >> 1) & 1, &g_moe_few_error, kErrWaitAccum, p.wait_ns);
                if (!ok) *reinterpret_cast<volatile int *>(&sh.abort) = 1;
                sh.go[buf] = more && ok && !*reinterpret_cast<volatile int *>(&sh.abort);
            }
            epilogue_sync();
            if (!sh.go[buf]) break;
            tc_fence_after();
            const Unit w = sh.unit[i & 3];
            uint32_t v[32];
            tmem_ld32(tmem + buf * kAccColumns + (static_cast<uint32_t>(warp * 32) << 16), v);
            tmem_ld_wait();
            tc_fence_before();
            mbar_arrive(&sh.acc_empty[buf]);
#pragma unroll
            for (int r = 0; r < kRoom; ++r) {
                if (r >= w.rows) break;
                // the digits' sums, smallest first
                float s = __uint_as_float(v[8 * r]);
#pragma unroll
                for (int d = 1; d < 6; ++d) s += __uint_as_float(v[8 * r + d]);
                if (w.first && tid < 64)
                    sh.epi[r][tid] = s;
                else if (!w.first)
                    p.y[static_cast<size_t>(sh.slot[w.slots + r]) * p.H + 128 * w.c + tid] = s;
            }
            epilogue_sync();
            if (tid == 0) mbar_arrive(&sh.unit_empty[i & 3]);
            if (!w.first) {
                if (lane == 0) mbar_arrive(&sh.written[i & 3]);
                continue;
            }
            // a warp has a token, a lane one of its 32 channels: a block of MXFP8
            const int r = warp;
            if (r < w.rows) {
                // silu as in moe_experts.cu: off by up to (5 + 1.2 |g|) 2^-23 of itself, 0 below -87.3
                const float g = sh.epi[r][lane], a = __fdividef(g, 1.0f + __expf(-g)) * sh.epi[r][32 + lane];
                const uint32_t b = mxfp8_scale_byte(__reduce_max_sync(0xffffffffu, __float_as_uint(a) & 0x7FFFFFFFu));
                const uint32_t code = e4m3x4_rn(a * mxfp8_scale_inverse(b), 0.0f, 0.0f, 0.0f) & 0xFFu;
                const uint32_t d0 = digits_of(sh.digits, code, b), d1 = __shfl_down_sync(0xffffffffu, d0, 1);
                const size_t row = sh.slot[w.slots + r];
                if (!(lane & 1)) {
                    uint8_t *o = p.ad + row * 6 * (p.I >> 1) + 16 * w.c + (lane >> 1);
#pragma unroll
                    for (int d = 0; d < 6; ++d)
                        o[static_cast<size_t>(d) * (p.I >> 1)] =
                            static_cast<uint8_t>(((d0 >> (4 * d)) & 0xFu) | (((d1 >> (4 * d)) & 0xFu) << 4));
                }
                if (lane < 6)
                    reinterpret_cast<uint8_t *>(p.asf + (row * (p.I >> 7) + (w.c >> 2)) * 8)[4 * lane + (w.c & 3)] =
                        static_cast<uint8_t>(digit_scale(b, lane));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.written[i & 3]);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemColumns);
    }
}

// --------------------------------------------------------------------- sum

struct SumParams {
    const float *y;                     // [T * k, H]
    const int *ids;
    const float *weights;
    uint16_t *out;
    int64_t ldo;
    int T, k, H;
};

// out_t = sum_j w_tj y[t, j], in the order of j. Grid: blocks of 512 channels x tokens, four
// channels a thread.
__global__ void __launch_bounds__(128) moe_few_sum_kernel(const SumParams p)
{
    __shared__ float weight[32];
    __shared__ int id[32];
    const int t = blockIdx.y, ch = (blockIdx.x * 128 + threadIdx.x) * 4;
    // what the launches before the last one wrote is there already
    if (threadIdx.x < p.k) {
        id[threadIdx.x] = __ldcg(p.ids + t * p.k + threadIdx.x);
        weight[threadIdx.x] = __ldcg(p.weights + t * p.k + threadIdx.x);
    }
    __syncthreads();
    grid_dependency_wait();
    grid_launch_dependents();
    if (ch >= p.H) return;
    const float *y = p.y + static_cast<size_t>(t) * p.k * p.H + ch;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int j0 = 0; j0 < p.k; j0 += 8) {
        float4 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = j0 + j < p.k && id[j0 + j] >= 0 ? __ldcg(reinterpret_cast<const float4 *>(y + static_cast<size_t>(j0 + j) * p.H))
                                                   : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j0 + j >= p.k || id[j0 + j] < 0) continue;
            const float w = weight[j0 + j];
            s.x = fmaf(w, v[j].x, s.x);
            s.y = fmaf(w, v[j].y, s.y);
            s.z = fmaf(w, v[j].z, s.z);
            s.w = fmaf(w, v[j].w, s.w);
        }
    }
    const __nv_bfloat162 a = __floats2bfloat162_rn(s.x, s.y), b = __floats2bfloat162_rn(s.z, s.w);
    *reinterpret_cast<uint2 *>(p.out + t * p.ldo + ch) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

constexpr uint32_t kExpertsSmem = 113664;   // two blocks an SM, and room for some of the sum's

template <typename Kern, typename P>
cudaError_t launch_pdl(Kern kern, dim3 grid, unsigned block, size_t smem, cudaStream_t stream, const P &params)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, params);
}

}  // namespace

MoeFewLayout moe_few_layout(int64_t T, int k, int E, int64_t H, int64_t I)
{
    MoeFewLayout l;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t was = at;
        at += (bytes + 255) / 256 * 256;
        return was;
    };
    const size_t slices = H / kSlice, R = static_cast<size_t>(T) * k;
    l.counters = take(sizeof(int) * (kMadeAt + kMaxEntries));
    l.h = take(2 * T * H);
    l.part = take(4 * slices * T * E);
    l.part_ss = take(4 * slices * T);
    l.xd = take(3 * T * H);
    l.xsf = take(32 * T * (H / 128));
    l.ids = take(4 * R);
    l.weights = take(4 * R);
    l.ad = take(3 * R * I);
    l.asf = take(32 * R * (I / 128));
    l.y = take(4 * R * H);
    l.total = at;
    return l;
}

cudaError_t launch_moe_few(const MoeFewArgs &a, const MoeFewLayout &l, cudaStream_t stream)
{
    static KernelOnce once;
    int sms = 0;
    cudaError_t e = prepare_kernel(moe_few_experts_kernel, kExpertsSmem, once, &sms);
    if (e != cudaSuccess) return e;
    RouterParams r;
    memset(&r, 0, sizeof(r));
    r.x = a.x;
    r.res = a.res;
    r.w = a.w;
    r.router = a.router;
    r.ldx = a.ldx;
    r.ldr = a.ldr;
    r.h = reinterpret_cast<uint16_t *>(a.ws + l.h);
    r.part = reinterpret_cast<float *>(a.ws + l.part);
    r.part_ss = reinterpret_cast<float *>(a.ws + l.part_ss);
    r.counters = reinterpret_cast<int *>(a.ws + l.counters);
    r.num_counters = kMadeAt + kMaxEntries;
    r.T = a.T;
    r.H = a.H;
    r.E = a.route.E;
    e = launch_pdl(moe_few_router_kernel, dim3(a.H / kSlice, (a.route.E + 63) / 64), kRouterThreads, 0, stream, r);
    if (e != cudaSuccess) return e;

    TokenParams t;
    memset(&t, 0, sizeof(t));
    t.h = r.h;
    t.w = a.w;
    t.router = a.router;
    t.part = r.part;
    t.part_ss = r.part_ss;
    t.bias = a.route.bias;
    t.xd = a.ws + l.xd;
    t.xsf = reinterpret_cast<uint32_t *>(a.ws + l.xsf);
    t.h_out = a.h_out;
    t.ldh = a.ldh;
    t.ids = reinterpret_cast<int *>(a.ws + l.ids);
    t.weights = reinterpret_cast<float *>(a.ws + l.weights);
    t.ids_out = a.route.ids;
    t.weights_out = a.route.weights;
    t.T = a.T;
    t.H = a.H;
    t.E = a.route.E;
    t.k = a.route.k;
    t.slices = a.H / kSlice;
    t.groups = a.route.groups;
    t.topk_groups = a.route.topk_groups;
    t.group_top = a.route.group_top;
    t.sigmoid = a.route.sigmoid;
    t.renorm = a.route.renorm;
    t.eps = a.eps;
    t.heps = static_cast<float>(static_cast<double>(a.H) * a.eps);
    t.root_h = static_cast<float>(std::sqrt(static_cast<double>(a.H)));
    t.scale = a.route.scale;
    e = launch_pdl(moe_few_token_kernel, dim3(a.T, (a.H / 8 + kTokenThreads - 1) / kTokenThreads), kTokenThreads, 0, stream, t);
    if (e != cudaSuccess) return e;

    ExpertsParams p;
    memset(&p, 0, sizeof(p));
    p.tm_w13 = a.tm_w13;
    p.tm_w2 = a.tm_w2;
    p.w13_sf = a.w13_sf;
    p.w2_sf = a.w2_sf;
    p.xd = t.xd;
    p.xsf = t.xsf;
    p.ids = t.ids;
    p.ad = a.ws + l.ad;
    p.asf = reinterpret_cast<uint32_t *>(a.ws + l.asf);
    p.y = reinterpret_cast<float *>(a.ws + l.y);
    p.queue = r.counters;
    p.made = r.counters + kMadeAt;
    p.T = a.T;
    p.k = a.route.k;
    p.E = a.route.E;
    p.H = a.H;
    p.I = a.I;
    p.wait_ns = wait_limit_ns();
    // a stage has room for the tokens of a unit, and for the 16 columns of the smallest MMA
    p.room = p.T <= 2 ? 2 : kRoom;
    const uint32_t stage = kStageWeights + 2 * kStageScales + p.room * kTokenBytes;
    p.stages = std::min<int>(kMaxStages, (kExpertsSmem - 1024 - sizeof(ExpertsShared)) / stage);
    // no more blocks than there can be units
    const int64_t entries = std::min<int64_t>(p.E + p.T * p.k / kRoom, int64_t(p.T) * p.k);
    const int64_t units = entries * (p.I / 32 + p.H / 128);
    e = launch_pdl(moe_few_experts_kernel, static_cast<unsigned>(std::min<int64_t>(2 * sms, units)), kExpertThreads,
                   kExpertsSmem, stream, p);
    if (e != cudaSuccess) return e;

    SumParams c;
    memset(&c, 0, sizeof(c));
    c.y = p.y;
    c.ids = t.ids;
    c.weights = t.weights;
    c.out = a.out;
    c.ldo = a.ldo;
    c.T = a.T;
    c.k = a.route.k;
    c.H = a.H;
    return launch_pdl(moe_few_sum_kernel, dim3((a.H + 511) / 512, a.T), 128, 0, stream, c);
}

int read_and_clear_moe_few_error()
{
    int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_moe_few_error, sizeof(int)) != cudaSuccess) return -1;
    cudaMemcpyToSymbol(g_moe_few_error, &zero, sizeof(int));
    return v;
}

}  // namespace mxfp4
