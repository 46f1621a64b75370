// Low-rank adapters of many requests beside a shared projection (lora_add).
//
// Mathematics, for token t of adapter a: u = x_t A_a^T (R numbers), then
// C_t = base_t + s_a u B_a^T. Two launches, and one before them for long batches:
//   sort    tokens by adapter, in tiles of up to 64 tokens of one adapter. Up to
//           kInline tokens every block works the tiles out for itself, from the ids
//           in shared memory.
//   shrink  u. The 16 rows of an MMA are rows of A_a, its columns are tokens, so that a
//           tile of one token wastes columns only. K is split over blocks, and inside
//           a block over its warps: a warp holds all of the tile's u (up to 64 ranks x
//           64 tokens) in registers and reads each x and each a of its part of K
//           once, from global memory straight into the MMA's registers (which order
//           of K the operands take is free as long as it is the same for both: a lane
//           holds 8 neighbouring k, one 16-byte vector). Sums of a block go to
//           the workspace, those of the splits are added in order by the next launch.
//   expand  u B_a^T + base. Rows of the MMA are tokens, columns are channels, chosen so
//           that a lane ends with 8 neighbouring channels of a token: one 16-byte
//           load of base and one store. u, summed in fp32, enters as two bf16 (high
//           and low part, 2^-17 together): twice the MMAs of a product that is not
//           bound by them, where one bf16 would cost 2^-9 of the update.
//
// Bound: few tokens, latency of two dependent launches; many, HBM (x once, base and C).
// mma.sync and not tcgen05: tiles are as small as one token, and a tile of 128 rows of
// the latter would be filled by padding; the products take R operations a byte.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "internal.h"
#include "layer.h"
#include "ptx.cuh"

namespace mxfp4 {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 64;          // tokens of a tile
constexpr int kInline = 64;        // tokens up to which blocks work out the tiles themselves
constexpr int kRanks = 64;         // ranks of one block of the first product
constexpr int kMaxRank = 256;
constexpr int kSortThreads = 1024;

// ------------------------------------------------------------------ tiles

struct Tile {
    int adapter, first, count;     // adapter L: tokens without one
};

__device__ __forceinline__ int adapter_of(int id, int L) { return id >= 0 && id < L ? id : L; }

// Tokens by adapter, and the tiles of it. One block: counts in shared memory, prefix
// sums, ranks. In which order a tile's tokens stand does not matter to their results.
__global__ void __launch_bounds__(kSortThreads) lora_sort_kernel(const LoraParams p)
{
    extern __shared__ int bins[];            // [L + 1]: tokens, then the next free place
    __shared__ int scan[2][32];
    const int tid = threadIdx.x, groups = p.L + 1;
    for (int i = tid; i < groups; i += kSortThreads) bins[i] = 0;
    __syncthreads();
    grid_dependency_wait();
    grid_launch_dependents();
    // neighbours often share an adapter: one atomic for all of a warp's lanes that do
    for (int64_t base = 0; base < p.T; base += kSortThreads) {
        const int64_t i = base + tid;
        const int g = i < p.T ? adapter_of(p.ids[i], p.L) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, g);
        if (g >= 0 && (tid & 31) == __ffs(same) - 1) atomicAdd(&bins[g], __popc(same));
    }
    __syncthreads();
    int places = 0, tiles = 0;               // of the groups before this round's
    for (int g0 = 0; g0 < groups; g0 += kSortThreads) {
        const int g = g0 + tid;
        const int n = g < groups ? bins[g] : 0;
        const bool skip = g == p.L && !p.copy;
        const int nt = skip ? 0 : (n + kTile - 1) / kTile;
        int a = n, b = nt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
            if ((tid & 31) >= o) {
                a += x;
                b += y;
            }
        }
        if ((tid & 31) == 31) {
            scan[0][tid >> 5] = a;
            scan[1][tid >> 5] = b;
        }
        __syncthreads();
        int before_a = places, before_b = tiles;
        for (int w = 0; w < kSortThreads / 32; ++w) {
            if (w < (tid >> 5)) {
                before_a += scan[0][w];
                before_b += scan[1][w];
            }
            places += scan[0][w];
            tiles += scan[1][w];
        }
        if (g < groups) {
            const int first = before_a + a - n, tile = before_b + b - nt;
            bins[g] = first;
            for (int i = 0; i < nt; ++i)
                p.tiles[tile + i] = make_int4(g, first + i * kTile, min(kTile, n - i * kTile), 0);
        }
        __syncthreads();
    }
    if (tid == 0) *p.num_tiles = tiles;
    for (int64_t base = 0; base < p.T; base += kSortThreads) {
        const int64_t i = base + tid;
        const int g = i < p.T ? adapter_of(p.ids[i], p.L) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, g);
        const int leader = __ffs(same) - 1, lane = tid & 31;
        int at = 0;
        if (g >= 0 && lane == leader) at = atomicAdd(&bins[g], __popc(same));
        at = __shfl_sync(0xffffffffu, at, leader);
        if (g >= 0) p.order[at + __popc(same & ((1u << lane) - 1))] = static_cast<int>(i);
    }
}

// Tile `index` of the batch and its tokens in `tok` (shared memory). False if there is
// no such tile. Called by a whole block; inline tiles are worked out from the ids: a
// token is first of a tile if no token before it has its adapter, and tiles stand
// in the order of their first tokens.
template <bool INLINE>
__device__ __forceinline__ bool find_tile(const LoraParams &p, int index, Tile &tile, int *tok, int *ids, int *found)
{
    const int tid = threadIdx.x;
    if constexpr (INLINE) {
        if (tid < kInline) ids[tid] = tid < p.T ? adapter_of(p.ids[tid], p.L) : -1;
        if (tid == 0) found[0] = -1;
        __syncthreads();
        if (tid < 32) {
            int tiles = 0;
            for (int base = 0; base < p.T; base += 32) {
                const int i = base + tid, g = i < p.T ? ids[i] : -1;
                bool first = g >= 0 && !(g == p.L && !p.copy);
                for (int k = 0; k < i && first; ++k) first = ids[k] != g;
                const unsigned m = __ballot_sync(0xffffffffu, first);
                if (first && tiles + __popc(m & ((1u << tid) - 1)) == index) found[0] = g;
                tiles += __popc(m);
            }
        }
        __syncthreads();
        const int g = found[0];
        if (g < 0) return false;
        const bool in = tid < kInline && ids[tid] == g;
        int at = 0;
        if (in) {
            for (int k = 0; k < tid; ++k) at += ids[k] == g;
            tok[at] = tid;
        }
        const int n = __syncthreads_count(in);
        tile = Tile{g, 0, n};
        return true;
    } else {
        if (index >= *p.num_tiles) return false;
        const int4 r = p.tiles[index];
        tile = Tile{r.x, r.y, r.z};
        if (tid < r.z) tok[tid] = p.order[r.y + tid];
        __syncthreads();
        return true;
    }
}

__device__ __forceinline__ int rank_of(const LoraParams &p, int a)
{
    return p.ranks ? max(0, min(p.R, p.ranks[a])) : p.R;
}

// ------------------------------------------------------------------- MMA

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// ----------------------------------------------------------------- shrink

// u of MT * 16 ranks and NT * 8 tokens of one tile, over this warp's 32-element steps
// of K; d[m][n] are the MMA's accumulators: ranks 16m + g, + 8, tokens 8n + 2q, + 1 of
// lane 4g + q.
template <int MT, int NT>
__device__ __forceinline__ void shrink_steps(const LoraParams &p, const uint16_t *a, int rows, const int *tok, int count,
                                             int k_begin, int k_end, float *red)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    float d[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) d[m][n][i] = 0.0f;
    const uint16_t *xr[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) xr[n] = 8 * n + g < count ? p.x + static_cast<int64_t>(tok[8 * n + g]) * p.ldx : nullptr;
    // a warp takes 64 elements at a time: whole 128-byte lines of every row
    for (int k0 = k_begin + 64 * warp; k0 < k_end; k0 += 64 * kWarps) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int k = k0 + 32 * s + 8 * q;
            const bool in = k < k_end;
            uint4 x[NT], w[MT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n)
                x[n] = in && xr[n] ? __ldg(reinterpret_cast<const uint4 *>(xr[n] + k)) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = 16 * m + 8 * h + g;
                    w[m][h] = in && r < rows ? __ldg(reinterpret_cast<const uint4 *>(a + static_cast<int64_t>(r) * p.K + k))
                                             : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mma_bf16(d[m][n], w[m][0].x, w[m][1].x, w[m][0].y, w[m][1].y, x[n].x, x[n].y);
                    mma_bf16(d[m][n], w[m][0].z, w[m][1].z, w[m][0].w, w[m][1].w, x[n].z, x[n].w);
                }
        }
    }
    // red: [warp][token][rank], rows one float apart from a multiple of 32 so that
    // neither side conflicts much
    constexpr int LD = 16 * MT + 1;
    float *mine = red + warp * (8 * NT * LD);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) mine[(8 * n + 2 * q + (i & 1)) * LD + 16 * m + g + 8 * (i >> 1)] = d[m][n][i];
    __syncthreads();
    for (int i = threadIdx.x; i < count * 16 * MT; i += kThreads) {
        const int t = i / (16 * MT), r = i - t * (16 * MT);
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum += red[w * (8 * NT * LD) + t * LD + r];
        const int rank = blockIdx.z * kRanks + r;
        if (rank < p.R) p.u[(static_cast<int64_t>(blockIdx.y) * p.T + tok[t]) * p.R + rank] = sum;
    }
}

// Shared memory of the warps' sums, for the most tokens a tile of a batch can have.
constexpr size_t shrink_smem(int T)
{
    return sizeof(float) * kWarps * (T <= 8 ? 8 : (T <= 16 ? 16 : (T <= 32 ? 32 : kTile))) * (kRanks + 1);
}

template <int MT>
__device__ __forceinline__ void shrink_tile(const LoraParams &p, const uint16_t *a, int rows, const int *tok, int count,
                                            int kb, int ke, float *red)
{
    if (count <= 8)
        shrink_steps<MT, 1>(p, a, rows, tok, count, kb, ke, red);
    else if (count <= 16)
        shrink_steps<MT, 2>(p, a, rows, tok, count, kb, ke, red);
    else if (count <= 32)
        shrink_steps<MT, 4>(p, a, rows, tok, count, kb, ke, red);
    else
        shrink_steps<MT, 8>(p, a, rows, tok, count, kb, ke, red);
}

// Grid: tiles x splits of K x blocks of 64 ranks.
template <bool INLINE>
__global__ void __launch_bounds__(kThreads) lora_shrink_kernel(const LoraParams p)
{
    extern __shared__ float red[];
    __shared__ int tok[kTile], ids[kInline], found[1];
    grid_dependency_wait();
    grid_launch_dependents();
    Tile tile;
    if (!find_tile<INLINE>(p, blockIdx.x, tile, tok, ids, found) || tile.adapter == p.L) return;
    // the adapter's ranks of this block; those it lacks are zeros
    const int rows = rank_of(p, tile.adapter) - blockIdx.z * kRanks;
    if (rows <= 0) return;                       // nobody reads sums beyond the rank
    const uint16_t *a = p.a + (static_cast<int64_t>(tile.adapter) * p.R + blockIdx.z * kRanks) * p.K;
    const int per = (p.K + 64 * p.splits - 1) / (64 * p.splits) * 64;
    const int kb = static_cast<int>(min(static_cast<int64_t>(blockIdx.y) * per, static_cast<int64_t>(p.K)));
    const int ke = static_cast<int>(min(static_cast<int64_t>(kb) + per, static_cast<int64_t>(p.K)));
    if (rows <= 16)
        shrink_tile<1>(p, a, rows, tok, tile.count, kb, ke, red);
    else if (rows <= 32)
        shrink_tile<2>(p, a, rows, tok, tile.count, kb, ke, red);
    else
        shrink_tile<4>(p, a, rows, tok, tile.count, kb, ke, red);
}

// ----------------------------------------------------------------- expand

// 16-bit values of C's type
template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t v)
{
    if constexpr (F16) return __half22float2(*reinterpret_cast<const __half2 *>(&v));
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float x, float y)
{
    if constexpr (F16) {
        const __half2 h = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// The elements of a vector of 8 below `n`, zeros for the others.
__device__ __forceinline__ uint4 keep_first(uint4 v, int n)
{
    uint32_t r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (2 * i >= n)
            r[i] = 0;
        else if (2 * i + 1 >= n)
            r[i] &= 0xFFFFu;
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// Columns 32c .. 32c + 31 of C for the 16 tokens 16m ...: channel of column `col` of the
// n-tile j is 32c + 8 (col / 2) + 2j + (col & 1), so lane (g, q) ends with channels 8q .. 8q + 7 of
// tokens g and g + 8.
template <bool F16>
__device__ __forceinline__ void expand_block(const LoraParams &p, const uint16_t *b, int rank, const uint32_t *hi,
                                             const uint32_t *lo, int ldu, const int *tok, int count, int m, int c)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    float d[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) d[j][i] = 0.0f;
    const int n = 32 * c + 8 * q;            // this lane's channels of C
    const bool in = n < p.N;
    int64_t row[2];
    uint4 base[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int t = 16 * m + 8 * h + g;
        row[h] = t < count ? tok[t] : -1;
        base[h] = make_uint4(0, 0, 0, 0);
        if (in && row[h] >= 0) base[h] = *reinterpret_cast<const uint4 *>(p.base + row[h] * p.ldb + n);
    }
    for (int k0 = 0; k0 < rank; k0 += 32) {
        const int k = k0 + 8 * q;
        uint4 w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int ch = 32 * c + 8 * (g >> 1) + 2 * j + (g & 1);
            w[j] = make_uint4(0, 0, 0, 0);
            if (k < rank && ch < p.N)
                w[j] = keep_first(__ldg(reinterpret_cast<const uint4 *>(b + static_cast<int64_t>(ch) * p.R + k)), rank - k);
        }
        // two words of hi / lo hold four k of a token
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int at = (16 * m + g) * ldu + (k >> 1) + 2 * s;
            const uint2 h0 = *reinterpret_cast<const uint2 *>(hi + at), h1 = *reinterpret_cast<const uint2 *>(hi + at + 8 * ldu);
            const uint2 l0 = *reinterpret_cast<const uint2 *>(lo + at), l1 = *reinterpret_cast<const uint2 *>(lo + at + 8 * ldu);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t b0 = s ? w[j].z : w[j].x, b1 = s ? w[j].w : w[j].y;
                mma_bf16(d[j], l0.x, l1.x, l0.y, l1.y, b0, b1);
                mma_bf16(d[j], h0.x, h1.x, h0.y, h1.y, b0, b1);
            }
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (!in || row[h] < 0) continue;
        const uint32_t v[4] = {base[h].x, base[h].y, base[h].z, base[h].w};
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = unpack2<F16>(v[j]);
            o[j] = pack2<F16>(f.x + d[j][2 * h], f.y + d[j][2 * h + 1]);
        }
        *reinterpret_cast<uint4 *>(p.c + row[h] * p.ldc + n) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// Grid: tiles x blocks of channels. Shared memory: the tile's u as high and low bf16,
// [64 tokens][ranks rounded up to 32, and 8 more against conflicts].
template <bool INLINE, bool F16>
__global__ void __launch_bounds__(kThreads) lora_expand_kernel(const LoraParams p)
{
    extern __shared__ uint32_t ushared[];
    __shared__ int tok[kTile], ids[kInline], found[1];
    grid_dependency_wait();
    grid_launch_dependents();
    Tile tile;
    if (!find_tile<INLINE>(p, blockIdx.x, tile, tok, ids, found)) return;
    const int chunks = (p.N + 31) / 32;
    if (tile.adapter == p.L) {
        // no adapter: a copy of base, as it is
        const int vectors = p.N / 8, total = gridDim.y * kThreads;
        for (int t = 0; t < tile.count; ++t) {
            const uint4 *s = reinterpret_cast<const uint4 *>(p.base + tok[t] * p.ldb);
            uint4 *o = reinterpret_cast<uint4 *>(p.c + tok[t] * p.ldc);
            for (int64_t i = blockIdx.y * kThreads + threadIdx.x; i < vectors; i += total) o[i] = s[i];
        }
        return;
    }
    const int rank = rank_of(p, tile.adapter);
    const int rows = (tile.count + 15) / 16 * 16, cols = (rank + 31) / 32 * 32, ldu = ((p.R + 31) / 32 * 32 + 8) / 2;
    uint32_t *hi = ushared, *lo = ushared + kTile * ldu;
    const float scale = p.scales ? p.scales[tile.adapter] : 1.0f;
    for (int i = threadIdx.x; i < rows * (cols / 2); i += kThreads) {
        const int t = i / (cols / 2), r = 2 * (i - t * (cols / 2));
        float2 v = make_float2(0.0f, 0.0f);
        if (t < tile.count && r < rank) {
            const float *u = p.u + static_cast<int64_t>(tok[t]) * p.R + r;
            for (int s = 0; s < p.splits; ++s) {
                const float2 part = __ldcg(reinterpret_cast<const float2 *>(u + static_cast<int64_t>(s) * p.T * p.R));
                v.x += part.x;
                v.y += part.y;
            }
            v.x *= scale;
            v.y = r + 1 < rank ? v.y * scale : 0.0f;
        }
        const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
        const uint32_t hb = *reinterpret_cast<const uint32_t *>(&h);
        // what rounds to infinity has no low part
        const float hx = __uint_as_float(hb << 16), hy = __uint_as_float(hb & 0xFFFF0000u);
        const __nv_bfloat162 l = __floats2bfloat162_rn(isinf(hx) ? 0.0f : v.x - hx, isinf(hy) ? 0.0f : v.y - hy);
        hi[t * ldu + r / 2] = hb;
        lo[t * ldu + r / 2] = *reinterpret_cast<const uint32_t *>(&l);
    }
    __syncthreads();
    const uint16_t *b = p.b + static_cast<int64_t>(tile.adapter) * p.N * p.R;
    const int mt = rows / 16, step = gridDim.y * kWarps;
    for (int64_t i = blockIdx.y * kWarps + (threadIdx.x >> 5); i < static_cast<int64_t>(chunks) * mt; i += step)
        expand_block<F16>(p, b, rank, hi, lo, ldu, tok, tile.count, static_cast<int>(i % mt), static_cast<int>(i / mt));
}

template <typename Kern>
cudaError_t launch(Kern kern, dim3 grid, int threads, size_t smem, cudaStream_t stream, const LoraParams &p)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <bool INLINE, bool F16>
cudaError_t launch_products(const LoraParams &p, const LoraLayout &l, cudaStream_t stream)
{
    static KernelOnce shrink_once, expand_once;
    cudaError_t e = prepare_kernel(lora_shrink_kernel<INLINE>, shrink_smem(kTile), shrink_once, nullptr);
    if (e != cudaSuccess) return e;
    const size_t expand_smem = sizeof(uint32_t) * 2 * kTile * (((p.R + 31) / 32 * 32 + 8) / 2);
    constexpr size_t most = sizeof(uint32_t) * 2 * kTile * ((kMaxRank + 8) / 2);
    int sms = 0;
    e = prepare_kernel(lora_expand_kernel<INLINE, F16>, most, expand_once, &sms);
    if (e != cudaSuccess) return e;
    e = launch(lora_shrink_kernel<INLINE>, dim3(l.max_tiles, l.splits, (p.R + kRanks - 1) / kRanks), kThreads,
               shrink_smem(p.T), stream, p);
    if (e != cudaSuccess) return e;
    // blocks of channels: as many as give every SM two blocks, no more than one step a warp
    const int items = (p.N + 31) / 32 * ((std::min(p.T, kTile) + 15) / 16);
    const int blocks = std::max(1, std::min((items + kWarps - 1) / kWarps, (2 * sms + l.max_tiles - 1) / l.max_tiles));
    return launch(lora_expand_kernel<INLINE, F16>, dim3(l.max_tiles, blocks), kThreads, expand_smem, stream, p);
}

}  // namespace

LoraLayout lora_layout(int64_t T, int64_t K, int R, int L)
{
    LoraLayout l;
    const int64_t full = (T + kTile - 1) / kTile;
    // splits of K: two blocks an SM if all tokens shared one adapter, each with 512
    // elements at least (one step of every warp)
    l.splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({304 / full, 32, (K + 511) / 512})));
    // every group of tokens wastes less than one tile
    l.max_tiles = static_cast<int>(std::min<int64_t>(T, T / kTile + L + 1));
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    // splits * T is at most 32 T, and at most 304 / (T / 64) * T or T: a bound that grows with T
    const int64_t most = std::min<int64_t>(32 * T, std::max<int64_t>(304 * kTile, T));
    l.u = 0;
    l.order = l.u + up(sizeof(float) * static_cast<size_t>(most) * R);
    l.tiles = l.order + up(sizeof(int) * static_cast<size_t>(T));
    l.count = l.tiles + up(sizeof(int4) * static_cast<size_t>(l.max_tiles));
    l.total = l.count + 256;
    return l;
}

cudaError_t launch_lora(LoraParams p, const LoraLayout &l, bool f16, cudaStream_t stream)
{
    p.splits = l.splits;
    if (p.T <= kInline)
        return f16 ? launch_products<true, true>(p, l, stream) : launch_products<true, false>(p, l, stream);
    cudaError_t e = launch(lora_sort_kernel, dim3(1), kSortThreads, sizeof(int) * (p.L + 1), stream, p);
    if (e != cudaSuccess) return e;
    return f16 ? launch_products<false, true>(p, l, stream) : launch_products<false, false>(p, l, stream);
}

}  // namespace mxfp4
