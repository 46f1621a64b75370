// The feed-forward half of a mixture-of-experts layer for a few tokens
// (mxfp4_moe_layer).
//
// Mathematics, for token t: h = x + residual, r = (mean h^2 + eps)^-1/2, y = h r w,
// logits z_e = r sum_k h_k w_k Wr[e, k], the k best experts and their weights, then
//   act = MXFP8(silu(G_e q) * (U_e q)),  q = MXFP8(y),  out_t = sum_j w_tj (W2_e act).
//
// Three launches, each one starting while the last drains:
//   router   blocks take 64 channels each: h, sums of squares and of the router's
//            products over them, for all tokens
//   tokens   a block a token: adds those sums in 64 bits, y in MXFP8, routing
//   experts  both products and the sum. Weights are what there is to read, so the
//            kernel is a stream of them: a ring of shared memory that one thread fills by TMA,
//            and warps that widen packed codes in registers (one conversion gives
//            two fp16) and multiply with mma.sync, 16 weight rows x 8 tokens x 16. An
//            E4M3 or E2M1 value is exact in fp16 and so is each product in fp32; the
//            sums of one block of 32 take the two scales in fp32, whatever their size.
//
// Why not tcgen05, which mxfp4_moe_experts uses for the same products: its weights have
// to lie in shared memory in 8-bit containers, and writing them there (690 wavefronts
// a stage of 16 KB) holds a decoding batch at half of HBM's rate. Here a packed word is read
// from shared memory once, and the tensor work is small: 8 columns.
//
// Units of work: 32 channels of an expert in product 1 (its rows of G and U: one block of
// the activations' MXFP8, quantized where it is made), 64 channels in product 2. Blocks
// claim them from one counter, product 1 first, so that a unit that waits for
// activations only waits for units that somebody already works on: no assumption on
// which blocks run at the same time. While it waits, its weights fill the ring.
//
// Bound: HBM, the weights of the experts that some token chose.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
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

// ------------------------------------------------------------------ router

constexpr int kSlice = 64;              // channels of a block
constexpr int kRouterThreads = 256;
constexpr int kSub = 20;                // floats from one 16 channels to the next, spread over the banks

struct RouterParams {
    const uint16_t *x, *res, *w, *router;
    uint16_t *h_out;                    // the caller's, or null
    int64_t ldx, ldr, ldh;
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
    for (int i = blockIdx.x * kRouterThreads + tid; i < p.num_counters; i += gridDim.x * kRouterThreads) p.counters[i] = 0;
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
            *reinterpret_cast<uint4 *>(p.h + static_cast<int64_t>(t) * p.H + c) = h4;
            if (p.h_out) *reinterpret_cast<uint4 *>(p.h_out + t * p.ldh + c) = h4;
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
        if (t < p.T && v == 0) p.part_ss[blockIdx.x * p.T + t] = ss;
    }
    __syncthreads();
    // four neighbouring lanes take 16 channels each of one expert
    const int sub = tid & 3;
    for (int e0 = (tid >> 5) * 8; e0 < p.E; e0 += kRouterThreads / 4) {
        const int e = e0 + ((tid & 31) >> 2);
        float wr[16];
        if (e < p.E) {
            const uint4 *src = reinterpret_cast<const uint4 *>(p.router + static_cast<int64_t>(e) * p.H + k0 + 16 * sub);
            const uint4 a = __ldg(src), b = __ldg(src + 1);
            const uint32_t r[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 f = bf16x2(r[i]);
                wr[2 * i] = f.x;
                wr[2 * i + 1] = f.y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) wr[i] = 0.0f;
        }
        for (int tk = 0; tk < p.T; ++tk) {
            const float4 *q = reinterpret_cast<const float4 *>(&hw[tk][sub * kSub]);
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 f = q[i];
                s = fmaf(f.x, wr[4 * i], s);
                s = fmaf(f.y, wr[4 * i + 1], s);
                s = fmaf(f.z, wr[4 * i + 2], s);
                s = fmaf(f.w, wr[4 * i + 3], s);
            }
            s += __shfl_xor_sync(0xffffffffu, s, 1);
            s += __shfl_xor_sync(0xffffffffu, s, 2);
            if (sub == 0 && e < p.E) p.part[(static_cast<int64_t>(blockIdx.x) * p.T + tk) * p.E + e] = s;
        }
    }
}

// ------------------------------------------------------------------ tokens

constexpr int kTokenThreads = 512;

struct TokenParams {
    const uint16_t *h, *w;
    const float *part, *part_ss;
    const float *bias;                  // [E] or null
    uint16_t *xh;                       // [T, H] the E4M3 values of y as fp16
    float *sx;                          // [T, H / 32] their scales
    int *ids;                           // [T, k], of the workspace
    float *weights;
    int *ids_out;                       // the caller's, or null
    float *weights_out;
    int T, H, E, k, slices, groups, topk_groups, group_top, sigmoid, renorm;
    float eps, scale;
};

// 2^(b - 127) of a scale byte, NaN for 255.
__device__ __forceinline__ float scale_value(uint32_t b)
{
    return __uint_as_float(b == 255 ? 0x7FC00000u : (b == 0 ? 0x00400000u : b << 23));
}

// A key that orders as the values do, NaN above all; 0 stands for "none".
__device__ __forceinline__ uint32_t order_key(float v)
{
    const uint32_t b = __float_as_uint(v);
    if (isnan(v)) return 0xFFFFFFFFu;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
constexpr uint32_t kKeyNone = 0x007FFFFFu;      // of -infinity: nothing below it is chosen

// Position of the largest of `n` <= 512 keys, the first of equals; all lanes of one warp,
// lane l holding keys l, l + 32, ...; takes it out (0). -1 if none is above `floor`.
__device__ __forceinline__ int take_best(uint32_t (&key)[kMaxExperts / 32], int n, uint32_t floor)
{
    const int lane = threadIdx.x & 31;
    uint32_t best = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < kMaxExperts / 32; ++i) {
        if (32 * i >= n) break;
        if (key[i] > best) {
            best = key[i];
            at = i;
        }
    }
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    if (top <= floor) return -1;
    const uint32_t mine = best == top ? static_cast<uint32_t>(32 * at + lane) : 0xFFFFFFFFu;
    const uint32_t e = __reduce_min_sync(0xffffffffu, mine);
#pragma unroll
    for (int i = 0; i < kMaxExperts / 32; ++i)
        if (static_cast<uint32_t>(32 * i + lane) == e) key[i] = 0;
    return static_cast<int>(e);
}

__global__ void __launch_bounds__(kTokenThreads) moe_few_token_kernel(const TokenParams p)
{
    __shared__ double sums[kTokenThreads];
    __shared__ float choice[kMaxExperts], score[kMaxExperts], group_score[kMaxExperts];
    __shared__ double r_shared;
    __shared__ float red[kTokenThreads / 32];
    __shared__ uint32_t group_kept[kMaxExperts / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, t = blockIdx.x;
    grid_dependency_wait();
    grid_launch_dependents();

    // r, by one warp
    if (warp == 0) {
        double ss = 0.0;
        for (int s = lane; s < p.slices; s += 32) ss += static_cast<double>(p.part_ss[s * p.T + t]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (lane == 0) {
            const double m = ss / p.H + static_cast<double>(p.eps);
            r_shared = m == 0.0 ? 0.0 : 1.0 / sqrt(m);
        }
    }
    // logits: `parts` threads an expert over interleaved slices, added in a fixed order
    const int parts = kTokenThreads / p.E;           // E <= 512
    const int e = tid % p.E, part = tid / p.E;
    double z = 0.0;
    if (part < parts)
        for (int s = part; s < p.slices; s += parts)
            z += static_cast<double>(p.part[(static_cast<int64_t>(s) * p.T + t) * p.E + e]);
    sums[tid] = z;
    __syncthreads();
    const double r = r_shared;
    float zf = -INFINITY;
    if (tid < p.E) {
        for (int i = 1; i < parts; ++i) z += sums[i * p.E + tid];
        zf = static_cast<float>(z * r);
    }
    // scores
    float s = 0.0f;
    if (p.sigmoid) {
        s = 1.0f / (1.0f + expf(-zf));
    } else {
        float m = zf;
        bool nan = isnan(zf);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (lane == 0) red[warp] = m;
        nan = __syncthreads_or(nan);
        m = red[0];
#pragma unroll
        for (int i = 1; i < kTokenThreads / 32; ++i) m = fmaxf(m, red[i]);
        __syncthreads();
        const float ex = tid < p.E && zf > -INFINITY ? expf(zf - m) : 0.0f;
        float sum = ex;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) red[warp] = sum;
        __syncthreads();
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kTokenThreads / 32; ++i) sum += red[i];
        s = nan ? __int_as_float(0x7FC00000) : (sum > 0.0f ? ex / sum : 0.0f);
    }
    if (tid < p.E) {
        score[tid] = s;
        // without a bias and groups the logits rank the experts as the scores do, also where those saturate
        float c = p.bias || p.groups > 1 ? s + (p.bias ? p.bias[tid] : 0.0f) : (isnan(s) ? s : zf);
        if (zf == -INFINITY) c = -INFINITY;
        choice[tid] = c;
    }
    __syncthreads();
    const int n = p.E / p.groups;
    if (p.groups > 1) {
        for (int g = warp; g < p.groups; g += kTokenThreads / 32) {
            // the two best keys of the group
            uint32_t k1 = 0, k2 = 0;
            for (int i = lane; i < n; i += 32) {
                const uint32_t key = order_key(choice[g * n + i]);
                if (key > k1) {
                    k2 = k1;
                    k1 = key;
                } else if (key > k2) {
                    k2 = key;
                }
            }
            const uint32_t top = __reduce_max_sync(0xffffffffu, k1);
            const unsigned who = __ballot_sync(0xffffffffu, k1 == top);
            if (lane == __ffs(who) - 1) k1 = k2;
            const uint32_t second = __reduce_max_sync(0xffffffffu, k1);
            auto value = [](uint32_t key) {
                return __uint_as_float(key == 0xFFFFFFFFu ? 0x7FC00000u : (key & 0x80000000u ? key & 0x7FFFFFFFu : ~key));
            };
            if (lane == 0) group_score[g] = value(top) + (p.group_top == 2 && n > 1 ? value(second) : 0.0f);
        }
        __syncthreads();
    }
    if (warp == 0) {
        uint32_t key[kMaxExperts / 32];
        if (p.groups > 1) {
#pragma unroll
            for (int i = 0; i < kMaxExperts / 32; ++i) {
                key[i] = 32 * i + lane < p.groups ? order_key(group_score[32 * i + lane]) : 0;
                if (lane == 0) group_kept[i] = 0;
            }
            __syncwarp();
            for (int i = 0; i < p.topk_groups; ++i) {
                const int g = take_best(key, p.groups, 0);
                if (g >= 0 && lane == 0) group_kept[g >> 5] |= 1u << (g & 31);
            }
            __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < kMaxExperts / 32; ++i) {
            const int x = 32 * i + lane;
            key[i] = 0;
            if (x < p.E && (p.groups == 1 || (group_kept[(x / n) >> 5] >> ((x / n) & 31) & 1))) key[i] = order_key(choice[x]);
        }
        int id = -1;
        for (int i = 0; i < p.k; ++i) {
            const int x = take_best(key, p.E, kKeyNone);
            if (lane == i) id = x;
        }
        float w = id >= 0 ? score[id] : 0.0f;
        if (p.renorm) {
            float sum = w;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            w = w / (sum + 1e-20f);
        }
        w *= p.scale;
        if (lane < p.k) {
            p.ids[t * p.k + lane] = id;
            p.weights[t * p.k + lane] = w;
            if (p.ids_out) p.ids_out[t * p.k + lane] = id;
            if (p.weights_out) p.weights_out[t * p.k + lane] = w;
        }
    }
    // y in MXFP8, four lanes a block of 32
    const float rf = static_cast<float>(r);
    for (int v = tid; v < p.H / 8; v += kTokenThreads) {     // H / 8 is a multiple of 16: whole groups of four
        const uint4 hv = *reinterpret_cast<const uint4 *>(p.h + static_cast<int64_t>(t) * p.H + 8 * v);
        const uint4 wv = *reinterpret_cast<const uint4 *>(p.w + 8 * v);
        const uint32_t ha[4] = {hv.x, hv.y, hv.z, hv.w}, wa[4] = {wv.x, wv.y, wv.z, wv.w};
        float y[8];
        uint32_t amax = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 a = bf16x2(ha[i]), b = bf16x2(wa[i]);
            y[2 * i] = a.x * b.x * rf;
            y[2 * i + 1] = a.y * b.y * rf;
            amax = max(amax, max(__float_as_uint(y[2 * i]) & 0x7FFFFFFFu, __float_as_uint(y[2 * i + 1]) & 0x7FFFFFFFu));
        }
        const unsigned quad = 0xFu << (lane & ~3);
        amax = max(amax, __shfl_xor_sync(quad, amax, 1));
        amax = max(amax, __shfl_xor_sync(quad, amax, 2));
        const uint32_t b = mxfp8_scale_byte(amax);
        const float inv = mxfp8_scale_inverse(b);
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = f16x2_of_e4m3(y[2 * i] * inv, y[2 * i + 1] * inv);
        *reinterpret_cast<uint4 *>(p.xh + static_cast<int64_t>(t) * p.H + 8 * v) = make_uint4(o[0], o[1], o[2], o[3]);
        if ((v & 3) == 0) p.sx[static_cast<int64_t>(t) * (p.H >> 5) + (v >> 2)] = scale_value(b);
    }
}

// ----------------------------------------------------------------- experts

constexpr int kConsumers = 256;                  // eight warps: four groups of 16 rows x two halves of a stage's K
constexpr int kExpertThreads = kConsumers + 32;
constexpr int kStages = 8;
constexpr uint32_t kStageWeights = 64 * 128;     // 64 rows x 256 elements
constexpr uint32_t kStageBytes = kStageWeights + 2048;   // and up to four blocks of scales

struct ExpertsParams {
    CUtensorMap tm_w13;                 // packed weights [E * 2I, H / 2] u8, box 128 bytes x 32 rows
    CUtensorMap tm_w2;                  // the same of [E * H, I / 2], box 64 rows
    const uint8_t *w13_sf, *w2_sf;
    const uint16_t *xh;
    const float *sx;
    const int *ids;
    const float *weights;
    uint16_t *act;                      // [T * k, I] fp16 of E4M3 values
    float *act_sx;                      // [T * k, I / 32]
    float *y;                           // [T * k, H]
    uint16_t *out;
    int64_t ldo;
    int *queue;                         // units claimed
    int *made;                          // units of product 1 that are complete
    int *arrived;                       // [H / 64] experts whose product 2 of these channels is complete
    int T, k, E, H, I;
    uint64_t wait_ns;
};

struct ExpertsShared {
    uint64_t full[kStages], empty[kStages];
    int header[kStages];                // unit of a stage, -1: there are no more
    int abort[2];
    int last;
    int active;
    uint16_t expert[kMaxChoices];       // the experts that some token chose
    uint8_t rows[kMaxExperts];          // choices of an expert
    uint16_t slot[kMaxExperts * kMaxTokens];   // t * k + j of them
    float red[2][4][8][32];             // sums of the second half of K: [unit parity][rows][value][lane]
    float act[kMaxTokens][33];
};
constexpr uint32_t kExpertsSmem = kStages * kStageBytes + sizeof(ExpertsShared) + 1024;

__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ void first_half_sync() { asm volatile("bar.sync 2, 128;" ::: "memory"); }

__device__ __forceinline__ int load_acquire(const int *p)
{
    int v;
    asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// fp16 pairs of the eight E2M1 codes of a word.
__device__ __forceinline__ void widen(uint32_t w, uint32_t (&h)[4])
{
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Activations of this lane for 128 elements of K: of the token of its MMA column, and
// the scales of the two tokens whose sums it holds.
struct Tokens {
    uint4 x[4];
    float4 s[2];
};

__global__ void __launch_bounds__(kExpertThreads, 2) moe_few_experts_kernel(const __grid_constant__ ExpertsParams p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    ExpertsShared &sh = *reinterpret_cast<ExpertsShared *>(smem + kStages * kStageBytes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], kConsumers / 32);
        }
        sh.abort[0] = sh.abort[1] = 0;
        fence_mbar_init();
        tma_prefetch_desc(&p.tm_w13);
        tma_prefetch_desc(&p.tm_w2);
    }
    for (int i = tid; i < kMaxExperts / 4; i += kExpertThreads) reinterpret_cast<uint32_t *>(sh.rows)[i] = 0;
    __syncthreads();
    grid_dependency_wait();
    // which experts have which choices: their order in a list does not matter, columns of
    // an MMA do not mix
    for (int i = tid; i < p.T * p.k; i += kExpertThreads) {
        const int e = __ldcg(p.ids + i);
        if (e >= 0) {
            const uint32_t was = atomicAdd(reinterpret_cast<uint32_t *>(sh.rows) + (e >> 2), 1u << (8 * (e & 3)));
            sh.slot[e * kMaxTokens + ((was >> (8 * (e & 3))) & 0xFF)] = static_cast<uint16_t>(i);
        }
    }
    __syncthreads();
    if (warp == 0) {
        int n = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const bool has = e0 + lane < p.E && sh.rows[e0 + lane] > 0;
            const unsigned m = __ballot_sync(0xffffffffu, has);
            if (has) sh.expert[n + __popc(m & ((1u << lane) - 1))] = static_cast<uint16_t>(e0 + lane);
            n += __popc(m);
        }
        if (lane == 0) sh.active = n;
    }
    __syncthreads();
    const int active = sh.active;
    const int n1 = active * (p.I >> 5), n2 = active * (p.H >> 6);

    if (warp == kConsumers / 32) {
        if (lane == 0) {
            // ---------------------------------------------- weights, by TMA
            const uint64_t pol = policy_evict_first();
            int gs = 0;
            bool ok = true;
            auto slot_free = [&]() {
                return gs < kStages || mbar_wait(&sh.empty[gs % kStages], ((gs / kStages) & 1) ^ 1u, &g_moe_few_error,
                                                 kErrWaitEmpty, p.wait_ns);
            };
            int u = atomicAdd(p.queue, 1);
            while (u < n1 + n2) {
                const int next = atomicAdd(p.queue, 1);    // on its way while this unit loads
                const bool first = u < n1;
                const int K = first ? p.H : p.I, kc = K >> 7, stages = (kc + 1) >> 1;
                const int tiles = p.I >> 5;
                int e, r0;
                const uint8_t *sf0, *sf1 = nullptr;
                if (first) {
                    // 32 channels: their rows of G and of U
                    const int a = u / tiles, c = u - a * tiles;
                    e = sh.expert[a];
                    r0 = e * 2 * p.I + 32 * c;
                    sf0 = p.w13_sf + (static_cast<size_t>(e) * (2 * p.I >> 7) + (c >> 2)) * kc * 512;
                    sf1 = sf0 + static_cast<size_t>(p.I >> 7) * kc * 512;
                } else {
                    const int c = (u - n1) / active;
                    e = sh.expert[u - n1 - c * active];
                    r0 = e * p.H + 64 * c;
                    sf0 = p.w2_sf + (static_cast<size_t>(e) * (p.H >> 7) + (c >> 1)) * kc * 512;
                }
                for (int ks = 0; ks < stages; ++ks, ++gs) {
                    if (!(ok = slot_free())) break;
                    const int s = gs % kStages;
                    uint8_t *st = smem + s * kStageBytes;
                    const uint32_t sf_bytes = 512u * min(2, kc - 2 * ks);
                    sh.header[s] = u;
                    mbar_arrive_expect_tx(&sh.full[s], kStageWeights + sf_bytes * (first ? 2 : 1));
                    if (first) {
                        tma_load_2d(st, &p.tm_w13, ks * 128, r0, &sh.full[s], pol);
                        tma_load_2d(st + 4096, &p.tm_w13, ks * 128, r0 + p.I, &sh.full[s], pol);
                        bulk_load(st + kStageWeights + 1024, sf1 + ks * 1024, sf_bytes, &sh.full[s], pol);
                    } else {
                        tma_load_2d(st, &p.tm_w2, ks * 128, r0, &sh.full[s], pol);
                    }
                    bulk_load(st + kStageWeights, sf0 + ks * 1024, sf_bytes, &sh.full[s], pol);
                }
                if (!ok) break;
                u = next;
            }
            grid_launch_dependents();
            if (ok && (ok = slot_free())) {
                sh.header[gs % kStages] = -1;
                mbar_arrive(&sh.full[gs % kStages]);
                ++gs;
            }
            // copies in flight land before the block leaves
            for (int i = max(0, gs - kStages); i < gs; ++i)
                mbar_wait(&sh.full[i % kStages], (i / kStages) & 1, &g_moe_few_error, kErrWaitDrain);
        }
        return;
    }

    // ------------------------------------------------------------- products
    const int m = warp & 3, kh = warp >> 2, g = lane >> 2, q = lane & 3;
    int gs = 0;
    for (int it = 0;; ++it) {
        // Every consumer warp passes consumers_sync once a turn, whatever it met, and
        // they all leave after the same one: abort[it & 1] is written before it and read
        // after it, and not written again before the next.
        bool ok = mbar_wait_warp(&sh.full[gs % kStages], (gs / kStages) & 1, &g_moe_few_error, kErrWaitFull, p.wait_ns);
        const int u = ok ? *reinterpret_cast<volatile int *>(&sh.header[gs % kStages]) : -1;
        const bool first = u < n1;
        int a = 0, c = 0, rows = 0;
        float acc[2][4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[nt][i] = 0.0f;
        const uint16_t *slots = sh.slot;
        if (u >= 0) {
            const int tiles = p.I >> 5;
            if (first) {
                a = u / tiles;
                c = u - a * tiles;
            } else {
                c = (u - n1) / active;
                a = u - n1 - c * active;
            }
            const int e = sh.expert[a];
            rows = sh.rows[e];
            slots = sh.slot + e * kMaxTokens;
            const int K = first ? p.H : p.I, kc = K >> 7, stages = (kc + 1) >> 1;
            if (!first) {
                // all activations have to be there
                int v = 1;
                if (lane == 0 && load_acquire(p.made) < n1) {
                    const uint64_t t0 = global_timer_ns();
                    while (load_acquire(p.made) < n1) {
                        if (global_timer_ns() - t0 > p.wait_ns) {
                            atomicCAS(&g_moe_few_error, 0, kErrWaitOperand);
                            v = 0;
                            break;
                        }
                        __nanosleep(64);
                    }
                }
                ok = __shfl_sync(0xffffffffu, v, 0) != 0;
                __syncwarp();
            }
            const uint16_t *xsrc = first ? p.xh : p.act;
            const float *ssrc = first ? p.sx : p.act_sx;
            // row of a choice among the activations: its token in product 1
            auto row_of = [&](int i) { return static_cast<int64_t>(first ? slots[i] / p.k : slots[i]); };
            const uint16_t *xr[2];
            const float *sr[2][2];
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
                xr[nt] = 8 * nt + g < rows ? xsrc + row_of(8 * nt + g) * K + kh * 128 + 8 * q : nullptr;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int col = 8 * nt + 2 * q + i;
                    sr[nt][i] = col < rows ? ssrc + row_of(col) * (K >> 5) + kh * 4 : nullptr;
                }
            }
            // where this lane's rows and their scales lie in a stage
            const uint32_t w0 = (first ? 8 * m + g : 16 * m + g) * 128, w1 = w0 + (first ? 4096 : 1024);
            uint32_t f0, f1;
            if (first) {
                f0 = kStageWeights + (8 * m + g) * 16 + (c & 3) * 4;
                f1 = f0 + 1024;
            } else {
                f0 = kStageWeights + ((m & 1) * 16 + g) * 16 + ((c & 1) * 2 + (m >> 1)) * 4;
                f1 = f0 + 128;
            }
            const bool wide = rows > 8;
            for (int ks = 0; ks < stages && ok; ++ks, ++gs) {
                const bool mine = 2 * ks + kh < kc;            // the last stage may have one half only
                Tokens tk[2];
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    if (nt && !wide) break;
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        tk[nt].x[b] = xr[nt] && mine ? *reinterpret_cast<const uint4 *>(xr[nt] + ks * 256 + 32 * b)
                                                     : make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        tk[nt].s[i] = sr[nt][i] && mine ? *reinterpret_cast<const float4 *>(sr[nt][i] + ks * 8)
                                                        : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                }
                const int s = gs % kStages;
                if (ks && !(ok = mbar_wait_warp(&sh.full[s], (gs / kStages) & 1, &g_moe_few_error, kErrWaitFull, p.wait_ns)))
                    break;
                const uint8_t *st = smem + s * kStageBytes;
                if (mine) {
                    const uint32_t sf0 = *reinterpret_cast<const uint32_t *>(st + f0 + kh * 512);
                    const uint32_t sf1 = *reinterpret_cast<const uint32_t *>(st + f1 + kh * 512);
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const uint32_t at = ((4 * kh + b) ^ g) * 16 + 4 * q;
                        uint32_t h0[4], h1[4];
                        widen(*reinterpret_cast<const uint32_t *>(st + w0 + at), h0);
                        widen(*reinterpret_cast<const uint32_t *>(st + w1 + at), h1);
                        const float s0 = __uint_as_float(((sf0 >> (8 * b)) & 0xFFu) << 23);
                        const float s1 = __uint_as_float(((sf1 >> (8 * b)) & 0xFFu) << 23);
#pragma unroll
                        for (int nt = 0; nt < 2; ++nt) {
                            if (nt && !wide) break;
                            float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                            mma_f16(d, h0[0], h1[0], h0[1], h1[1], tk[nt].x[b].x, tk[nt].x[b].y);
                            mma_f16(d, h0[2], h1[2], h0[3], h1[3], tk[nt].x[b].z, tk[nt].x[b].w);
                            const float x0 = (&tk[nt].s[0].x)[b], x1 = (&tk[nt].s[1].x)[b];
                            acc[nt][0] = fmaf(d[0] * x0, s0, acc[nt][0]);
                            acc[nt][1] = fmaf(d[1] * x1, s0, acc[nt][1]);
                            acc[nt][2] = fmaf(d[2] * x0, s1, acc[nt][2]);
                            acc[nt][3] = fmaf(d[3] * x1, s1, acc[nt][3]);
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.empty[s]);
            }
            if (kh == 1) {
#pragma unroll
                for (int i = 0; i < 8; ++i) sh.red[it & 1][m][i][lane] = acc[i >> 2][i & 3];
            }
        }
        if (!ok) *reinterpret_cast<volatile int *>(&sh.abort[it & 1]) = 1;
        consumers_sync();
        if (*reinterpret_cast<volatile int *>(&sh.abort[it & 1]) || u < 0) break;
        if (kh == 1) continue;
        // ------------------------------------------ epilogue, by the first half
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i >> 2][i & 3] += sh.red[it & 1][m][i][lane];
        if (first) {
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int col = 8 * nt + 2 * q + i;
                    // silu as in moe_experts.cu: off by up to (5 + 1.2 |g|) 2^-23 of itself, 0 below -87.3
                    const float gv = acc[nt][i];
                    if (col < rows) sh.act[col][8 * m + g] = __fdividef(gv, 1.0f + __expf(-gv)) * acc[nt][2 + i];
                }
            first_half_sync();
            for (int r = m; r < rows; r += 4) {
                const float v = sh.act[r][lane];
                const uint32_t b = mxfp8_scale_byte(__reduce_max_sync(0xffffffffu, __float_as_uint(v) & 0x7FFFFFFFu));
                const int64_t row = slots[r];
                p.act[row * p.I + 32 * c + lane] =
                    static_cast<uint16_t>(f16x2_of_e4m3(v * mxfp8_scale_inverse(b), 0.0f) & 0xFFFFu);
                if (lane == 0) p.act_sx[row * (p.I >> 5) + c] = scale_value(b);
            }
            first_half_sync();
            if (tid == 0) {
                __threadfence();
                atomicAdd(p.made, 1);
            }
        } else {
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int col = 8 * nt + 2 * q + (i & 1);
                    if (col < rows)
                        p.y[static_cast<int64_t>(slots[col]) * p.H + 64 * c + 16 * m + g + 8 * (i >> 1)] = acc[nt][i];
                }
            first_half_sync();
            if (tid == 0) {
                __threadfence();
                sh.last = atomicAdd(p.arrived + c, 1) == active - 1;
                __threadfence();
            }
            first_half_sync();
            if (sh.last) {
                // all experts' rows of these channels are there: the weighted sum, in the order of a token's choices
                for (int i = tid; i < p.T * 64; i += 128) {
                    const int t = i >> 6, ch = 64 * c + (i & 63);
                    float s = 0.0f;
                    for (int j = 0; j < p.k; ++j)
                        if (p.ids[t * p.k + j] >= 0)
                            s = fmaf(p.weights[t * p.k + j], __ldcg(p.y + static_cast<int64_t>(t * p.k + j) * p.H + ch), s);
                    p.out[t * p.ldo + ch] = __bfloat16_as_ushort(__float2bfloat16_rn(s));
                }
            }
        }
    }
}

template <typename Kern, typename P>
cudaError_t launch_pdl(Kern kern, unsigned grid, unsigned block, size_t smem, cudaStream_t stream, const P &params)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
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
    l.counters = take(sizeof(int) * (64 + H / 64));
    l.h = take(2 * T * H);
    l.part = take(4 * slices * T * E);
    l.part_ss = take(4 * slices * T);
    l.xh = take(2 * T * H);
    l.sx = take(4 * T * (H / 32));
    l.ids = take(4 * R);
    l.weights = take(4 * R);
    l.act = take(2 * R * I);
    l.act_sx = take(4 * R * (I / 32));
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
    r.h_out = a.h_out;
    r.ldx = a.ldx;
    r.ldr = a.ldr;
    r.ldh = a.ldh;
    r.h = reinterpret_cast<uint16_t *>(a.ws + l.h);
    r.part = reinterpret_cast<float *>(a.ws + l.part);
    r.part_ss = reinterpret_cast<float *>(a.ws + l.part_ss);
    r.counters = reinterpret_cast<int *>(a.ws + l.counters);
    r.num_counters = 64 + a.H / 64;
    r.T = a.T;
    r.H = a.H;
    r.E = a.route.E;
    e = launch_pdl(moe_few_router_kernel, a.H / kSlice, kRouterThreads, 0, stream, r);
    if (e != cudaSuccess) return e;

    TokenParams t;
    memset(&t, 0, sizeof(t));
    t.h = r.h;
    t.w = a.w;
    t.part = r.part;
    t.part_ss = r.part_ss;
    t.bias = a.route.bias;
    t.xh = reinterpret_cast<uint16_t *>(a.ws + l.xh);
    t.sx = reinterpret_cast<float *>(a.ws + l.sx);
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
    t.scale = a.route.scale;
    e = launch_pdl(moe_few_token_kernel, a.T, kTokenThreads, 0, stream, t);
    if (e != cudaSuccess) return e;

    ExpertsParams p;
    memset(&p, 0, sizeof(p));
    p.tm_w13 = a.tm_w13;
    p.tm_w2 = a.tm_w2;
    p.w13_sf = a.w13_sf;
    p.w2_sf = a.w2_sf;
    p.xh = t.xh;
    p.sx = t.sx;
    p.ids = t.ids;
    p.weights = t.weights;
    p.act = reinterpret_cast<uint16_t *>(a.ws + l.act);
    p.act_sx = reinterpret_cast<float *>(a.ws + l.act_sx);
    p.y = reinterpret_cast<float *>(a.ws + l.y);
    p.out = a.out;
    p.ldo = a.ldo;
    p.queue = r.counters;
    p.made = r.counters + 32;
    p.arrived = r.counters + 64;
    p.T = a.T;
    p.k = a.route.k;
    p.E = a.route.E;
    p.H = a.H;
    p.I = a.I;
    p.wait_ns = wait_limit_ns();
    // no more blocks than there can be units
    const int64_t experts = std::min<int64_t>(p.E, int64_t(p.T) * p.k);
    const int64_t units = experts * (p.I / 32 + p.H / 64);
    return launch_pdl(moe_few_experts_kernel, static_cast<unsigned>(std::min<int64_t>(2 * sms, units)), kExpertThreads,
                      kExpertsSmem, stream, p);
}

int read_and_clear_moe_few_error()
{
    int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_moe_few_error, sizeof(int)) != cudaSuccess) return -1;
    cudaMemcpyToSymbol(g_moe_few_error, &zero, sizeof(int));
    return v;
}

}  // namespace mxfp4
