// Routing of tokens to experts (moe_route): scores, groups, top k, weights.
//
// One warp a token; lane l holds the V experts from V l on in registers. What a
// token costs is not its E logits (a few hundred bytes) but the instructions of the
// selection: k rounds of a warp-wide maximum (redux.sync) over order-preserving
// integer keys, of which the lowest lane that has it, and there the first expert, is
// the one of lowest index. A lane enters a round with its best key and keeps its
// second, so most rounds look at no other key of the lane; which expert a chosen key
// belongs to, and how close two choices came, is worked out for all k at once after
// the rounds (a lane a choice). A group of experts is a run of lanes where its size
// allows (a power of two of them); its score then takes a few shuffles, all groups
// at once.
//
// Exactness. With a bias or groups the choice compares sums s + bias that fp32
// holds to about 2^-22 only, and two experts of a large batch come closer than
// that. Every fp32 decision is therefore checked against a margin `tol` that
// bounds the error of both sides. In units of 2^-24 of max(s, |c|): expf 2, the
// sum 1 + e 1, its reciprocal 2 (rcp.approx), c itself 1, so 2^-21 for the sigmoid; the
// softmax adds 1 for x - max and up to V + 7 for the sum of the row, so 2^-19.
// Rows with a closer decision (one in a few hundred) are decided again from 64-bit
// scores of the few experts that fp32 leaves in question: those about the border
// between two groups, or about the last choice. FP64 instructions are slow here (a
// warp's takes 16 clocks or more): scoring whole rows in 64 bits took half of the
// kernel's time, though it was for so few. Without bias and groups the logits
// themselves are compared, which is exact. The weights are computed in fp32, with IEEE
// divisions, from the chosen logits: they only scale rows that go into an fp32 sum
// (off from 64 bits by 6e-8 of their size, where one rounding costs 3e-8).
//
// Measured: 16384 x 256 fp32, sigmoid, bias, 4 of 8 groups, 8 experts: 24 us (1130
// instructions a token, issued in 73 % of the cycles; the logits alone are 2.5 us of
// HBM time; 21 us without any 64-bit decision; 39 us when each round searched
// its lane's keys). 3001 x 60: 6.5 us. One token: 3.2 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstring>

#include "internal.h"
#include "moe.h"
#include "ptx.cuh"

namespace mxfp4 {

namespace {

constexpr unsigned kAll = 0xffffffffu;

// Monotone integer key of a float: larger value, larger key; NaN above all;
// -inf is 0x007FFFFF, and 0 stands for "taken".
__device__ __forceinline__ uint32_t key32(float v)
{
    if (v != v) return 0xFFFFFFFFu;
    if (v == 0.0f) v = 0.0f;   // -0 ranks as 0
    const uint32_t b = __float_as_uint(v);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;

__device__ __forceinline__ float load_logit(const void *p, int64_t i, int dtype)
{
    if (dtype == 0) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
    if (dtype == 1) return __half2float(static_cast<const __half *>(p)[i]);
    return static_cast<const float *>(p)[i];
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
__device__ __forceinline__ double warp_sum(double v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
}

// 64-bit ranking of a row: `a` before `b`; NaN first, then larger values, then lower indices.
__device__ __forceinline__ bool before64(double a, int ia, double b, int ib)
{
    const bool na = a != a, nb = b != b;
    if (na != nb) return na;
    if (!na && a != b) return a > b;
    return ia < ib;
}

// The best (value, index) of the warp.
__device__ __forceinline__ void warp_best64(double &v, int &i)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const double ov = __shfl_xor_sync(kAll, v, o);
        const int oi = __shfl_xor_sync(kAll, i, o);
        if (before64(ov, oi, v, i)) {
            v = ov;
            i = oi;
        }
    }
}

// A row decided in 64 bits: the ids of its k experts in lane order (lane j < k
// holds the j-th; -1 where nothing is left), for rows with values that have no order
// (NaN, infinities) or groups that are no runs of lanes. `c` is the warp's shared
// memory, [E] doubles and two a group.
__device__ __noinline__ int route_row64(const RouteParams &p, int dtype, int64_t t, double *c)
{
    const int lane = threadIdx.x & 31;
    const double kNegInf = -__longlong_as_double(0x7FF0000000000000ll);
    double m = kNegInf;
    double s = 0.0;
    if (!p.sigmoid) {
        for (int e = lane; e < p.E; e += 32) {
            const double z = load_logit(p.logits, t * p.ldl + e, dtype);
            m = z > m || z != z ? z : m;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const double om = __shfl_xor_sync(kAll, m, o);
            m = om > m || om != om ? om : m;
        }
        for (int e = lane; e < p.E; e += 32) {
            const double z = load_logit(p.logits, t * p.ldl + e, dtype);
            s += z == kNegInf ? 0.0 : exp(z - m);
        }
        s = warp_sum(s);
    }
    for (int e = lane; e < p.E; e += 32) {
        const double z = load_logit(p.logits, t * p.ldl + e, dtype);
        const double score = p.sigmoid ? 1.0 / (1.0 + exp(-z)) : exp(z - m) / s;
        c[e] = z == kNegInf ? kNegInf : p.bias ? score + static_cast<double>(p.bias[e]) : score;
    }
    __syncwarp();
    if (p.groups > 1) {
        const int n = p.E / p.groups;
        for (int g = lane; g < p.groups; g += 32) {
            double b1 = kNegInf, b2 = kNegInf;
            for (int i = 0; i < n; ++i) {
                const double v = c[g * n + i];
                if (before64(v, 0, b1, 0)) {
                    b2 = b1;
                    b1 = v;
                } else if (before64(v, 0, b2, 0)) {
                    b2 = v;
                }
            }
            c[p.E + g] = p.group_top == 2 && n > 1 ? b1 + b2 : b1;
            c[p.E + p.groups + g] = 0.0;   // 1: dropped
        }
        __syncwarp();
        for (int r = 0; r < p.groups - p.topk_groups; ++r) {
            // drop the worst group that is left
            double v = 0.0;
            int gi = -1;
            for (int g = lane; g < p.groups; g += 32)
                if (c[p.E + p.groups + g] == 0.0 && (gi < 0 || before64(v, gi, c[p.E + g], g))) {
                    v = c[p.E + g];
                    gi = g;
                }
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                const double ov = __shfl_xor_sync(kAll, v, o);
                const int og = __shfl_xor_sync(kAll, gi, o);
                if (og >= 0 && (gi < 0 || before64(v, gi, ov, og))) {
                    v = ov;
                    gi = og;
                }
            }
            for (int i = lane; i < n; i += 32) c[gi * n + i] = kNegInf;
            if (lane == 0) c[p.E + p.groups + gi] = 1.0;
            __syncwarp();
        }
    }
    int mine = -1;
    for (int j = 0; j < p.k; ++j) {
        double v = kNegInf;
        int i = p.E;
        for (int e = lane; e < p.E; e += 32)
            if (before64(c[e], e, v, i)) {
                v = c[e];
                i = e;
            }
        warp_best64(v, i);
        if (v == kNegInf) break;   // nothing is left
        if (lane == j) mine = i;
        if (lane == 0) c[i] = kNegInf;
        __syncwarp();
    }
    return mine;
}

// The 64-bit exponentials exp(z - max) of a softmax row, to `c` [E] (each lane its own V
// from e0 on), and their sum.
template <int V>
__device__ __noinline__ double softmax_terms64(const RouteParams &p, int dtype, int64_t t, int e0, double *c)
{
    const float kNegInf = -__int_as_float(0x7F800000);
    float m = kNegInf;
    for (int e = e0; e < e0 + V && e < p.E; ++e) m = fmaxf(m, load_logit(p.logits, t * p.ldl + e, dtype));
    m = warp_max(m);
    double s = 0.0;
    for (int e = e0; e < e0 + V && e < p.E; ++e) {
        const float z = load_logit(p.logits, t * p.ldl + e, dtype);
        const double x = z == kNegInf ? 0.0 : exp(static_cast<double>(z) - m);
        c[e] = x;
        s += x;
    }
    return warp_sum(s);
}

// Score + bias of expert e in 64 bits, as a monotone integer key (finite values).
// `terms`, `sum`: of a softmax row, from softmax_terms64.
__device__ __noinline__ unsigned long long exact_key64(const RouteParams &p, int dtype, int64_t t, int e, double sum,
                                                       const double *terms)
{
    double c;
    if (p.sigmoid)
        c = 1.0 / (1.0 + exp(-static_cast<double>(load_logit(p.logits, t * p.ldl + e, dtype))));
    else
        c = terms[e] / sum;
    if (p.bias) c += static_cast<double>(p.bias[e]);
    if (c == 0.0) c = 0.0;
    const unsigned long long u = __double_as_longlong(c);
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ double value64(unsigned long long k)
{
    return __longlong_as_double((k >> 63) ? (k & 0x7FFFFFFFFFFFFFFFull) : ~k);
}

// The largest key of the warp, and the lowest lane that has it.
__device__ __forceinline__ unsigned long long warp_max64(unsigned long long k, int &lane_of)
{
    const uint32_t hi = __reduce_max_sync(kAll, static_cast<uint32_t>(k >> 32));
    const bool in = static_cast<uint32_t>(k >> 32) == hi;
    const uint32_t lo = __reduce_max_sync(kAll, in ? static_cast<uint32_t>(k) : 0u);
    lane_of = __ffs(__ballot_sync(kAll, in && static_cast<uint32_t>(k) == lo)) - 1;
    return (static_cast<unsigned long long>(hi) << 32) | lo;
}

// 1 / x to one unit in the last place; results below 2^-126 become 0.
__device__ __forceinline__ float reciprocal_approx(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// key32 of what is neither NaN nor -0
__device__ __forceinline__ uint32_t key32_plain(float v)
{
    const uint32_t b = __float_as_uint(v);
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float value_of(uint32_t k)   // inverse of key32
{
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The two largest keys of a lane.
template <int V>
__device__ __forceinline__ void best_two(const uint32_t (&key)[V], uint32_t &k1, uint32_t &k2)
{
    k1 = key[0];
    k2 = 0u;
#pragma unroll
    for (int i = 1; i < V; ++i) {
        k2 = max(k2, min(k1, key[i]));
        k1 = max(k1, key[i]);
    }
}

// The V logits from element i on (E of them in the row from column e): by 16-byte
// vectors where `vec` says that rows allow them.
template <int V, int DTYPE>
__device__ __forceinline__ void load_row(const RouteParams &p, int64_t t, int e, float (&z)[V])
{
    constexpr int W = DTYPE == 2 ? 4 : 8;   // elements of a vector
    const float kNegInf = -__int_as_float(0x7F800000);
    const int64_t at = t * p.ldl + e;
    if (V % W == 0 && p.vec && e + V <= p.E) {
#pragma unroll
        for (int i = 0; i < V / W; ++i) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if constexpr (V % W == 0)
                v = *(reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p.logits) + at * (16 / W)) + i);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (DTYPE == 2) {
                    z[W * i + j] = __uint_as_float(w[j]);
                } else if constexpr (DTYPE == 0) {
                    z[W * i + 2 * j] = __uint_as_float(w[j] << 16);
                    z[W * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
                } else {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[j]));
                    z[W * i + 2 * j] = f.x;
                    z[W * i + 2 * j + 1] = f.y;
                }
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] = e + i < p.E ? load_logit(p.logits, at + i, DTYPE) : kNegInf;
    }
}

// V: experts a lane, E <= 32 V.
// Eight blocks an SM hold 64 registers a thread: 25.0 us against 26.6 us of five (16384 x 256).
template <int V, int DTYPE>
__global__ void __launch_bounds__(128, V <= 8 ? 8 : 5) moe_route_kernel(const RouteParams p)
{
    extern __shared__ double smem_route[];
    grid_dependency_wait();
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nwarps = blockDim.x >> 5;
    double *c64 = smem_route + static_cast<size_t>(warp) * (p.E + 2 * p.groups);
    const float kNegInf = -__int_as_float(0x7F800000);
    const int e0 = lane * V, n = p.E / p.groups;
    float bias[V];
#pragma unroll
    for (int i = 0; i < V; ++i) bias[i] = p.bias && e0 + i < p.E ? p.bias[e0 + i] : 0.0f;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * nwarps + warp; t < p.T;
         t += static_cast<int64_t>(gridDim.x) * nwarps) {
        float z[V];
        uint32_t key[V];
        load_row<V, DTYPE>(p, t, e0, z);
        float zmax = 0.0f, sum = 1.0f;
        if (!p.sigmoid) {
            zmax = kNegInf;
            bool nan = false;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                nan |= z[i] != z[i];
                zmax = fmaxf(zmax, z[i]);
            }
            zmax = warp_max(zmax);
            sum = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) sum += z[i] == kNegInf ? 0.0f : expf(z[i] - zmax);
            sum = warp_sum(sum);
            if (__any_sync(kAll, nan)) sum = zmax = __int_as_float(0x7FC00000);
        }
        auto score = [&](float x) {
            if (x == kNegInf) return 0.0f;
            return p.sigmoid ? 1.0f / (1.0f + expf(-x)) : expf(x - zmax) / sum;
        };
        const bool by_logit = !p.bias && p.groups == 1 && (p.sigmoid || sum == sum);
        bool open = false;         // a decision closer than fp32 can tell
        bool open_groups = false;  // such a one between groups that are no runs of lanes, or a value without order
        float tol = 0.0f;
        double sum64 = 1.0;
        bool have64 = false;
        if (by_logit) {
#pragma unroll
            for (int i = 0; i < V; ++i) key[i] = key32(z[i]);
        } else {
            auto set = [&](int i, float s) {
                const float c = z[i] == kNegInf ? kNegInf : s + bias[i];
                const float size = max_nan(s, fabsf(c));
                tol = max_nan(tol, c == kNegInf ? 0.0f : size);
                key[i] = key32_plain(c);   // a NaN shows in tol; s + bias is no -0
            };
            if (p.sigmoid) {
#pragma unroll
                for (int i = 0; i < V; ++i) set(i, reciprocal_approx(1.0f + expf(-z[i])));
            } else {
                const float rsum = 1.0f / sum;
#pragma unroll
                for (int i = 0; i < V; ++i) set(i, expf(z[i] - zmax) * rsum);
            }
            // tol >= 0 or the largest NaN, so its bits order as it does; 2^-125 stands for scores that became 0
            tol = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(tol))) * (p.sigmoid ? 0x1p-21f : 0x1p-19f) +
                  0x1p-125f;
            open_groups = !(tol < 1e20f);
        }
        // this lane's two best keys that are left; a second of 0 stands for "not known"
        uint32_t mine = 0u, next = 0u;
        bool in = true;        // this lane's experts may be chosen
        best_two<V>(key, mine, next);
        if (p.groups > 1 && !open_groups) {
            // A group's two best keys, in every lane of the group (`run` lanes of it, from
            // a multiple of run on), or group g's in lane g, g + 32, ...
            uint32_t kept = 0u;       // groups of this lane that stay: bit 0, or bit i for group lane + 32 i
            const int run = p.group_lanes;
            if (run > 0) {
                uint32_t k1 = mine, k2 = next;
                for (int o = 1; o < run; o <<= 1) {
                    const uint32_t a1 = __shfl_xor_sync(kAll, k1, o), a2 = __shfl_xor_sync(kAll, k2, o);
                    k2 = max(max(k2, a2), min(k1, a1));
                    k1 = max(k1, a1);
                }
                const float gs = value_of(k1) + (p.group_top == 2 && n > 1 ? value_of(k2) : 0.0f);
                const bool real = e0 < p.E;
                const uint32_t group = real ? key32(gs) : 0u;
                // groups before this one: each lane of a group compares it with every run-th
                // group, and the lanes add up
                const int sub = lane & (run - 1), base = lane - sub;
                int rank = 0;
                for (int g0 = 0; g0 < p.groups; g0 += run) {
                    const int from = (g0 + sub) * run;
                    const uint32_t other = __shfl_sync(kAll, group, from & 31);
                    rank += g0 + sub < p.groups && (other > group || (other == group && from < base));
                }
                for (int o = 1; o < run; o <<= 1) rank += __shfl_xor_sync(kAll, rank, o);
                kept = real && rank < p.topk_groups;
                // the worst that stays against the best that goes; sums of two carry twice the error
                const uint32_t low = __reduce_min_sync(kAll, kept ? group : 0xFFFFFFFFu);
                const uint32_t high = __reduce_max_sync(kAll, real && !kept ? group : 0u);
                if (high > kKeyNegInf && !(value_of(low) - value_of(high) > 4.0f * tol)) {
                    // In question: the groups that stay by less than the error over the best that
                    // goes, and those that go by less under the worst that stays. Their exact
                    // scores come from the experts that may be among their best.
                    if (!p.sigmoid && !have64) {
                        sum64 = softmax_terms64<V>(p, DTYPE, t, e0, c64);
                        have64 = true;
                    }
                    const bool asked = real && group > kKeyNegInf &&
                                       (kept ? gs <= value_of(high) + 4.0f * tol : gs >= value_of(low) - 4.0f * tol);
                    const float from = value_of(p.group_top == 2 && n > 1 ? k2 : k1) - 2.0f * tol;
                    unsigned long long d1 = 0, d2 = 0;
                    uint32_t todo = 0u;
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (asked && key[i] > kKeyNegInf && value_of(key[i]) >= from) todo |= 1u << i;
                    for (; todo; todo &= todo - 1) {
                        const unsigned long long x = exact_key64(p, DTYPE, t, e0 + __ffs(todo) - 1, sum64, c64);
                        d2 = max(d2, min(d1, x));
                        d1 = max(d1, x);
                    }
                    __syncwarp();
                    for (int o = 1; o < run; o <<= 1) {
                        const unsigned long long a1 = __shfl_xor_sync(kAll, d1, o), a2 = __shfl_xor_sync(kAll, d2, o);
                        d2 = max(max(d2, a2), min(d1, a1));
                        d1 = max(d1, a1);
                    }
                    // a group with one expert left has -inf beside it, and with that is not asked
                    double exact = asked ? value64(d1) : 0.0;
                    if (asked && p.group_top == 2 && n > 1) exact += value64(d2);
                    const int places = p.topk_groups - __popc(__ballot_sync(kAll, kept && !asked)) / run;
                    int before = 0;
                    for (int g = 0; g < p.groups; ++g) {
                        const double other = __shfl_sync(kAll, exact, g * run);
                        const bool is = __shfl_sync(kAll, asked, g * run);
                        before += is && (other > exact || (other == exact && g * run < base));
                    }
                    if (asked) kept = before < places;
                }
                in = kept;
                if (!in) mine = next = 0u;
            } else {
                // groups that are no runs of lanes: one lane a group, through shared memory
                float *cs = reinterpret_cast<float *>(c64);
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (e0 + i < p.E) cs[e0 + i] = value_of(key[i]);
                __syncwarp();
                constexpr int GV = V;      // groups a lane: at most as many as experts
                uint32_t best[GV];
#pragma unroll
                for (int i = 0; i < GV; ++i) {
                    const int g = lane + 32 * i;
                    best[i] = 0u;
                    if (g < p.groups) {
                        float b1 = kNegInf, b2 = kNegInf;
                        for (int j = 0; j < n; ++j) {
                            const float c = cs[g * n + j];
                            b2 = fmaxf(b2, fminf(b1, c));
                            b1 = fmaxf(b1, c);
                        }
                        best[i] = key32(p.group_top == 2 && n > 1 ? b1 + b2 : b1);
                    }
                }
                __syncwarp();
                uint32_t low = 0u;
                for (int r = 0; r <= p.topk_groups && r < p.groups; ++r) {
                    uint32_t b = 0u;
#pragma unroll
                    for (int i = 0; i < GV; ++i)
                        if (!(kept >> i & 1)) b = max(b, best[i]);
                    const uint32_t m = __reduce_max_sync(kAll, b);
                    if (r == p.topk_groups) {
                        if (m > kKeyNegInf && !(value_of(low) - value_of(m) > 4.0f * tol)) open_groups = true;
                        break;
                    }
                    int first = 1 << 20;
#pragma unroll
                    for (int i = GV - 1; i >= 0; --i)
                        if (!(kept >> i & 1) && best[i] == m && lane + 32 * i < p.groups) first = lane + 32 * i;
                    const int g = __reduce_min_sync(kAll, first);
                    if ((g & 31) == lane) kept |= 1u << (g >> 5);
                    low = m;
                }
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int g = e0 + i < p.E ? (e0 + i) / n : 0;
                    const uint32_t bits = __shfl_sync(kAll, kept, g & 31);
                    if (e0 + i < p.E && !(bits >> (g >> 5) & 1)) key[i] = kKeyNegInf;
                }
                best_two<V>(key, mine, next);
            }
        }
        int id = -1;               // lane j < k: the j-th choice
        float least = kNegInf;     // value of the last choice
        if (!open_groups) {
            // lane j notes the j-th choice: its key, its lane, and how many of that lane's
            // equal keys went before (equal keys of one lane go one after another)
            uint32_t chosen = 0u, prev = 0u;
            int from = 0, dup = 0, prev_lane = -1, nth = 0, j = 0;
            for (; j < p.k; ++j) {
                const uint32_t m = __reduce_max_sync(kAll, mine);
                if (m <= kKeyNegInf) break;    // nothing is left
                const int winner = __ffs(__ballot_sync(kAll, mine == m)) - 1;
                dup = m == prev && winner == prev_lane ? dup + 1 : 0;
                prev = m;
                prev_lane = winner;
                if (lane == j) {
                    chosen = m;
                    from = winner;
                    nth = dup;
                }
                if (lane == winner) {
                    mine = next;
                    next = 0u;
                    if (mine == 0u) {
                        int equal = 0;
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            equal += key[i] == m;
                            if (key[i] < m) mine = max(mine, key[i]);
                        }
                        if (equal > dup + 1) mine = m;
                    }
                }
                __syncwarp();
            }
            if (j > 0) least = value_of(prev);
            if (!by_logit) {
                // each choice against the one after it, the last against the best that is left
                uint32_t after = __shfl_down_sync(kAll, chosen, 1);
                const uint32_t rest = j == p.k ? __reduce_max_sync(kAll, mine) : 0u;
                if (lane == j - 1) after = rest;
                open = __any_sync(kAll, lane < j && after > kKeyNegInf &&
                                            !(value_of(chosen) - value_of(after) > 2.0f * tol));
            }
            int at = 0;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (__shfl_sync(kAll, key[i], from) == chosen && nth-- == 0) at = i;
            if (lane < j) id = from * V + at;
        }
        if (open && !open_groups) {
            // the candidates: what lies within the error of the last choice, or above
            if (!p.sigmoid && !have64) sum64 = softmax_terms64<V>(p, DTYPE, t, e0, c64);
            unsigned long long *k64 = reinterpret_cast<unsigned long long *>(c64) + e0;   // this lane's own
            uint32_t left = 0u;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (in && key[i] > kKeyNegInf && value_of(key[i]) >= least - 2.0f * tol) left |= 1u << i;
            for (uint32_t todo = left; todo; todo &= todo - 1) {
                const int i = __ffs(todo) - 1;
                k64[i] = exact_key64(p, DTYPE, t, e0 + i, sum64, c64);
            }
            __syncwarp();
            id = -1;
            for (int j = 0; j < p.k; ++j) {
                unsigned long long best = 0;
                int at = 0;
                for (uint32_t todo = left; todo; todo &= todo - 1) {
                    const int i = __ffs(todo) - 1;
                    if (k64[i] > best) {
                        best = k64[i];
                        at = i;
                    }
                }
                int winner;
                if (warp_max64(best, winner) == 0) break;     // nothing is left
                if (lane == winner) left &= ~(1u << at);
                const int e = __shfl_sync(kAll, e0 + at, winner);
                if (lane == j) id = e;
            }
        } else if (open_groups) {
            id = route_row64(p, DTYPE, t, c64);
            __syncwarp();
        }
        float w = 0.0f;
        if (id >= 0) w = score(load_logit(p.logits, t * p.ldl + id, DTYPE));
        if (p.renorm) {
            // in pairs: every lane that writes has the same sum
            float total = w;
            for (int o = 1; o < p.k; o <<= 1) total += __shfl_xor_sync(kAll, total, o);
            w = w / (total + 1e-20f);
        }
        if (lane < p.k) {
            p.ids[t * p.k + lane] = id;
            p.weights[t * p.k + lane] = w * p.scale;
        }
    }
}

template <int V, int DTYPE>
cudaError_t launch_v(RouteParams p, int num_sms, cudaStream_t stream)
{
    constexpr int kWarps = 4;
    const int n = p.E / p.groups, lanes = n / V;
    p.group_lanes = n % V == 0 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
    const int size = DTYPE == 2 ? 4 : 2;
    p.vec = (reinterpret_cast<uintptr_t>(p.logits) & 15u) == 0 && p.ldl * size % 16 == 0;
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    const int64_t blocks = (p.T + kWarps - 1) / kWarps;
    const int64_t most = static_cast<int64_t>(num_sms) * 16;
    cfg.gridDim = dim3(static_cast<unsigned>(blocks < most ? blocks : most), 1, 1);
    cfg.blockDim = dim3(32 * kWarps, 1, 1);
    cfg.dynamicSmemBytes = sizeof(double) * kWarps * (p.E + 2 * p.groups);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // 4 warps x (512 + 2 * 512) doubles is 48 KB, the limit without opting in
    return cudaLaunchKernelEx(&cfg, moe_route_kernel<V, DTYPE>, p);
}

template <int DTYPE>
cudaError_t launch_dtype(const RouteParams &p, int num_sms, cudaStream_t stream)
{
    if (p.E <= 32) return launch_v<1, DTYPE>(p, num_sms, stream);
    if (p.E <= 64) return launch_v<2, DTYPE>(p, num_sms, stream);
    if (p.E <= 128) return launch_v<4, DTYPE>(p, num_sms, stream);
    if (p.E <= 256) return launch_v<8, DTYPE>(p, num_sms, stream);
    return launch_v<16, DTYPE>(p, num_sms, stream);
}

}  // namespace

cudaError_t launch_moe_route(const RouteParams &p, int dtype, int num_sms, cudaStream_t stream)
{
    return dtype == 0 ? launch_dtype<0>(p, num_sms, stream)
                      : dtype == 1 ? launch_dtype<1>(p, num_sms, stream) : launch_dtype<2>(p, num_sms, stream);
}

}  // namespace mxfp4
