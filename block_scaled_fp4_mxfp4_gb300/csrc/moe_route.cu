// Routing of tokens to experts (moe_route): scores, groups, top k, weights.
//
// One warp a token; lane l holds experts l, l + 32, ... in registers. What a
// token costs is not its E logits (a few hundred bytes) but the selection: k
// rounds of a warp-wide maximum over order-preserving integer keys
// (redux.sync), each giving the lowest index among equals.
//
// Exactness. With a bias or groups the choice compares sums s + bias that fp32
// holds to about 2^-22 only, and two experts of a large batch come closer than
// that. Every fp32 decision is therefore checked against a margin `tol` that
// bounds the error of both sides. In units of 2^-24 of max(s, |c|): expf 2, the
// sum 1 + e or the division 1 each, c itself 1, so 2^-21 for the sigmoid; the
// softmax adds 1 for x - max and up to V + 7 for the sum of the row, so 2^-19.
// Rows with a closer decision (under one in a hundred) are decided again from
// 64-bit scores. Without bias and groups the logits themselves are compared,
// which is exact.
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
// holds the j-th; -1 where nothing is left). `c` is the warp's [E] doubles of
// shared memory.
__device__ __noinline__ int route_row64(const RouteParams &p, int dtype, int64_t t, double *c)
{
    const int lane = threadIdx.x & 31;
    const double kNegInf = -__longlong_as_double(0x7FF0000000000000ll);
    double m = kNegInf;
    for (int e = lane; e < p.E; e += 32) {
        const double z = load_logit(p.logits, t * p.ldl + e, dtype);
        c[e] = z;
        m = z > m || z != z ? z : m;
    }
    double s = 0.0;
    if (!p.sigmoid) {
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const double om = __shfl_xor_sync(kAll, m, o);
            m = om > m || om != om ? om : m;
        }
        for (int e = lane; e < p.E; e += 32) s += c[e] == kNegInf ? 0.0 : exp(c[e] - m);
        s = warp_sum(s);
    }
    for (int e = lane; e < p.E; e += 32) {
        const double z = c[e];
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

// V: experts a lane, E <= 32 V.
template <int V>
__global__ void __launch_bounds__(128) moe_route_kernel(const RouteParams p, int dtype)
{
    extern __shared__ double smem_route[];
    grid_dependency_wait();
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nwarps = blockDim.x >> 5;
    double *c64 = smem_route + static_cast<size_t>(warp) * (p.E + 2 * p.groups);
    const float kNegInf = -__int_as_float(0x7F800000);
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * nwarps + warp; t < p.T;
         t += static_cast<int64_t>(gridDim.x) * nwarps) {
        float z[V];
        uint32_t key[V];
        float zmax = kNegInf;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + 32 * i;
            z[i] = e < p.E ? load_logit(p.logits, t * p.ldl + e, dtype) : kNegInf;
            zmax = z[i] != z[i] || z[i] > zmax ? z[i] : zmax;
        }
        float sum = 1.0f;
        if (!p.sigmoid) {
            bool nan = zmax != zmax;
            zmax = warp_max(zmax);
            nan = __any_sync(kAll, nan);
            sum = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) sum += z[i] == kNegInf ? 0.0f : expf(z[i] - zmax);
            sum = warp_sum(sum);
            if (nan) sum = zmax = __int_as_float(0x7FC00000);
        }
        auto score = [&](float x) {
            if (x == kNegInf) return 0.0f;
            return p.sigmoid ? 1.0f / (1.0f + expf(-x)) : expf(x - zmax) / sum;
        };
        const bool by_logit = !p.bias && p.groups == 1 && (p.sigmoid || sum == sum);
        bool open = false;    // a decision closer than fp32 can tell
        float tol = 0.0f;
        if (by_logit) {
#pragma unroll
            for (int i = 0; i < V; ++i) key[i] = lane + 32 * i < p.E ? key32(z[i]) : 0u;
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = lane + 32 * i;
                key[i] = 0u;
                if (e < p.E) {
                    const float s = score(z[i]);
                    const float c = z[i] == kNegInf ? kNegInf : p.bias ? s + p.bias[e] : s;
                    if (c != kNegInf) tol = fmaxf(tol, fmaxf(s, fabsf(c)));
                    open |= c != c;
                    key[i] = key32(c);
                }
            }
            tol = warp_max(tol) * (p.sigmoid ? 0x1p-21f : 0x1p-19f);
            open = __any_sync(kAll, open) || !(tol < 1e30f);
        }
        auto value_of = [&](uint32_t k) {   // inverse of key32
            return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
        };
        if (p.groups > 1 && !open) {
            const int n = p.E / p.groups;
            // scores of the groups, lane g (and g + 32, ...) holding group g's;
            // at most 512 groups of one expert each
            uint32_t best[V];
#pragma unroll
            for (int i = 0; i < V; ++i) best[i] = 0u;
            for (int g = 0; g < p.groups; ++g) {
                uint32_t k1 = 0u, k2 = 0u;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int e = lane + 32 * i;
                    if (e >= g * n && e < (g + 1) * n) {
                        if (key[i] > k1) {
                            k2 = k1;
                            k1 = key[i];
                        } else if (key[i] > k2) {
                            k2 = key[i];
                        }
                    }
                }
                const uint32_t m1 = __reduce_max_sync(kAll, k1);
                float gs = value_of(m1);
                if (p.group_top == 2 && n > 1) {
                    const unsigned has = __ballot_sync(kAll, k1 == m1);
                    const uint32_t second = lane == __ffs(has) - 1 ? k2 : k1;
                    gs += value_of(__reduce_max_sync(kAll, second));
                }
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (lane + 32 * i == g) best[i] = key32(gs);
            }
            // the topk_groups best; a group that is not among them loses its experts
            float last = 0.0f;
            bool any_last = false;
            uint32_t keep_bits = 0u;   // bit i: this lane's group lane + 32 i is kept
            for (int r = 0; r <= p.topk_groups && r < p.groups; ++r) {
                uint32_t b = 0u;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (!(keep_bits >> i & 1)) b = max(b, best[i]);
                const uint32_t m = __reduce_max_sync(kAll, b);
                if (r == p.topk_groups) {
                    // against the best group left out; sums of two carry twice the error
                    if (any_last && !(last - value_of(m) > 4.0f * tol) && value_of(m) != kNegInf) open = true;
                    break;
                }
                int mine = 1 << 20;
#pragma unroll
                for (int i = V - 1; i >= 0; --i)
                    if (!(keep_bits >> i & 1) && best[i] == m && lane + 32 * i < p.groups) mine = lane + 32 * i;
                const int g = __reduce_min_sync(kAll, mine);
                if ((g & 31) == lane) keep_bits |= 1u << (g >> 5);
                last = value_of(m);
                any_last = true;
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = lane + 32 * i;
                const int g = e < p.E ? e / n : 0;
                const uint32_t bits = __shfl_sync(kAll, keep_bits, g & 31);
                if (e < p.E && !(bits >> (g >> 5) & 1)) key[i] = kKeyNegInf;
            }
        }
        int id = -1;          // lane j < k: the j-th choice
        if (!open) {
            float prev = 0.0f;
            for (int j = 0; j <= p.k; ++j) {
                uint32_t b = 0u;
#pragma unroll
                for (int i = 0; i < V; ++i) b = max(b, key[i]);
                const uint32_t m = __reduce_max_sync(kAll, b);
                if (m <= kKeyNegInf) break;    // nothing is left
                if (!by_logit) {
                    const float v = value_of(m);
                    if (j > 0 && !(prev - v > 2.0f * tol)) {
                        open = true;
                        break;
                    }
                    prev = v;
                }
                if (j == p.k) break;
                int mine = 1 << 20;
#pragma unroll
                for (int i = V - 1; i >= 0; --i)
                    if (key[i] == m) mine = lane + 32 * i;
                const int e = __reduce_min_sync(kAll, mine);
                if (lane == j) id = e;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (lane + 32 * i == e) key[i] = 0u;
            }
        }
        if (open) id = route_row64(p, dtype, t, c64);
        float w = 0.0f;
        if (id >= 0) w = score(load_logit(p.logits, t * p.ldl + id, dtype));
        if (p.renorm) {
            // the sum in the order of the choices
            float total = 0.0f;
            for (int j = 0; j < p.k; ++j) total += __shfl_sync(kAll, w, j);
            w = w / (total + 1e-20f);
        }
        if (lane < p.k) {
            p.ids[t * p.k + lane] = id;
            p.weights[t * p.k + lane] = w * p.scale;
        }
    }
}

template <int V>
cudaError_t launch_v(const RouteParams &p, int dtype, int num_sms, cudaStream_t stream)
{
    constexpr int kWarps = 4;
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
    return cudaLaunchKernelEx(&cfg, moe_route_kernel<V>, p, dtype);
}

}  // namespace

cudaError_t launch_moe_route(const RouteParams &p, int dtype, int num_sms, cudaStream_t stream)
{
    if (p.E <= 32) return launch_v<1>(p, dtype, num_sms, stream);
    if (p.E <= 64) return launch_v<2>(p, dtype, num_sms, stream);
    if (p.E <= 128) return launch_v<4>(p, dtype, num_sms, stream);
    if (p.E <= 256) return launch_v<8>(p, dtype, num_sms, stream);
    return launch_v<16>(p, dtype, num_sms, stream);
}

}  // namespace mxfp4
