// Low-rank adapters of many requests beside a shared projection (lora_add).
//
// Mathematics, for token t of adapter a: u = x_t A_a^T (R numbers), then
// C_t = base_t + s_a u B_a^T. Two launches, and one before them for long batches:
//   sort    tokens by adapter, in tiles of up to 128 tokens of one adapter. Up to
//           kInline tokens every block works the tiles out for itself, from the ids
//           in shared memory.
//   shrink  u, K split over blocks: sums go to the workspace, and those of the splits are added
//           in order by the next launch. Up to kInline tokens a block's warps split its
//           part of K once more; a warp holds all of the tile's u in registers
//           (mma.sync: 16 ranks x 8 tokens, so that a tile of one token wastes columns only)
//           and reads each x and each a once, from global memory straight into the
//           MMA's registers (which order of K the operands take is free as long as it
//           is the same for both: a lane holds 8 neighbouring k, one 16-byte vector).
//           Longer batches: tcgen05.mma kind::f16 with up to 128 tokens as rows and the
//           ranks as columns, token rows gathered by cp.async, a_a by TMA, which take a
//           ring of shared memory at the rate of HBM.
//   expand  u B_a^T + base, for up to 64 tokens a block. Rows of the MMA are tokens, columns
//           are channels, chosen so that a lane ends with 8 neighbouring channels of a
//           token: one 16-byte load of base and one store. u, summed in fp32, enters as two
//           bf16 (high and low part, 2^-17 together): twice the MMAs, where one bf16 would cost
//           2^-9 of the update.
// Batches whose tiles are filled to a half or more, of up to 64 ranks, take both products by tcgen05: the blocks
// that share a tile's K are a cluster, add their sums in shared memory and leave u as the two bf16 that the
// second product loads as an operand. (Sums of splits through global memory were read again by every block of
// channels, and mma.sync took half of the second product's time: 7168 -> 2112, rank 64, 16384 tokens 108 us, 87 now; 4096
// tokens 37.2 and 31.4. In a tile of few tokens the 128 rows are mostly empty: 333 tokens of 20 adapters up to
// rank 24, 2048 -> 7168, 23.3 us, 17.6 without.)
//
// Bound: few tokens, latency of two dependent launches; many, HBM (x once, base and C) and the
// latencies of three. Measured on the device, 7168 -> 2112: 1 token of rank 16 4.8 us, 16 tokens with
// adapters of rank 32 of their own 7.4 us (9.9 MB, 1.5 us at the copy bandwidth), 4096 tokens of 6
// adapters of rank 64 31.4 us (100 MB, 15 us), of rank 128 54.6, of rank 256 94.3; 16384 tokens of rank 64 87 us (381 MB, 56 us).
// Grids and splits go by the adapters that are held, which the host knows, not by those that a batch uses: 64 tokens
// of one adapter (rank 16, 4096 -> 4096) 9.4 us, 19.8 where 64 or 4096 are held; 4096 tokens 29.3, 79.8 of 4096.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "internal.h"
#include "layer.h"
#include "ptx.cuh"

namespace mxfp4 {

__device__ int g_lora_error;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 128;         // tokens of a tile
constexpr int kHalf = 64;          // tokens of a block of the second product
constexpr int kInline = 64;        // tokens up to which blocks work out the tiles themselves
constexpr int kRanks = 64;         // ranks of a block of the first product (up to kInline tokens), and of the
                                   // ring of the second
constexpr int kMaxRank = 256;

// ------------------------------------------------------------------ tiles

struct Tile {
    int adapter, first, count;     // adapter L: tokens without one
};

__device__ __forceinline__ int adapter_of(int id, int L) { return id >= 0 && id < L ? id : L; }

// Tokens by adapter, and the tiles of it. One block: counts in shared memory, prefix
// sums, ranks. In which order a tile's tokens stand does not matter to their results. A
// thread keeps its first kSortKeep ids in registers; more are read again for their places. LONG (more ids than
// the block keeps): a warp takes kSortKeep * 32 neighbouring ids at a time, in a prompt all of one
// adapter, for which one atomic is enough: the whole call of 32768 tokens of 6 adapters (7168 -> 2112, rank 64) 151.2 us,
// 155.8 with an atomic for every 32; of 16384 87.2 and 88.3. Up to 8192 the ids lie better spread over all warps.
constexpr int kSortKeep = 8;
template <int THREADS, bool LONG>
__global__ void __launch_bounds__(THREADS) lora_sort_kernel(const LoraParams p)
{
    extern __shared__ int bins[];            // [L + 1]: tokens, then the next free place
    __shared__ int2 scan[THREADS / 32];      // tokens and tiles of the groups before a warp's
    __shared__ int2 all;
    const int tid = threadIdx.x, lane = tid & 31, groups = p.L + 1;
    for (int i = tid; i < groups; i += THREADS) bins[i] = 0;
    __syncthreads();
    grid_dependency_wait();
    grid_launch_dependents();
    constexpr int kBatch = 32 * kSortKeep, kStep = LONG ? 32 : THREADS;     // from a lane's id to its next
    const int64_t own = (tid >> 5) * (LONG ? kBatch : 32);
    auto load = [&](int64_t at, int (&g)[kSortKeep]) {
#pragma unroll
        for (int i = 0; i < kSortKeep; ++i) {
            const int64_t t = at + kStep * i + lane;
            g[i] = t < p.T ? adapter_of(p.ids[t], p.L) : -1;
        }
    };
    auto alike = [&](const int (&g)[kSortKeep]) {
        if (!LONG) return false;
        const int first = __shfl_sync(0xffffffffu, g[0], 0);
        bool same = first >= 0;
#pragma unroll
        for (int i = 0; i < kSortKeep; ++i) same &= g[i] == first;
        return __all_sync(0xffffffffu, same) != 0;
    };
    // neighbours often share an adapter: one atomic for all of a warp's lanes that do
    auto count = [&](int64_t at, const int (&g)[kSortKeep]) {
        if (alike(g)) {
            if (lane == 0) atomicAdd(&bins[g[0]], kBatch);
            return;
        }
#pragma unroll
        for (int i = 0; i < kSortKeep; ++i) {
            if (at + kStep * i >= p.T) break;
            const unsigned same = __match_any_sync(0xffffffffu, g[i]);
            if (g[i] >= 0 && lane == __ffs(same) - 1) atomicAdd(&bins[g[i]], __popc(same));
        }
    };
    int kept[kSortKeep], more[kSortKeep];
    load(own, kept);
    if (own < p.T) count(own, kept);
    for (int64_t at = own + kSortKeep * THREADS; at < p.T; at += kSortKeep * THREADS) {
        load(at, more);
        count(at, more);
    }
    __syncthreads();
    int2 before = make_int2(0, 0);           // tokens and tiles of the groups before this pass's
    for (int g0 = 0; g0 < groups; g0 += THREADS) {
        const int g = g0 + tid;
        const int n = g < groups ? bins[g] : 0;
        const int nt = g == p.L && !p.copy ? 0 : (n + kTile - 1) / kTile;
        int a = n, b = nt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
            if (lane >= o) {
                a += x;
                b += y;
            }
        }
        if (lane == 31) scan[tid >> 5] = make_int2(a, b);
        __syncthreads();
        if (tid < 32) {
            const int2 own = lane < THREADS / 32 ? scan[lane] : make_int2(0, 0);
            int2 sum = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, sum.x, o), y = __shfl_up_sync(0xffffffffu, sum.y, o);
                if (lane >= o) {
                    sum.x += x;
                    sum.y += y;
                }
            }
            if (lane < THREADS / 32) scan[lane] = make_int2(sum.x - own.x, sum.y - own.y);
            if (lane == 31) all = sum;
        }
        __syncthreads();
        if (g < groups) {
            const int first = before.x + scan[tid >> 5].x + a - n, tile = before.y + scan[tid >> 5].y + b - nt;
            bins[g] = first;
            for (int i = 0; i < nt; ++i)
                p.tiles[tile + i] = make_int4(g, first + i * kTile, min(kTile, n - i * kTile), 0);
        }
        before.x += all.x;
        before.y += all.y;
        __syncthreads();
    }
    // the others of the grid's tiles are empty
    for (int i = before.y + tid; i < p.max_tiles; i += THREADS) p.tiles[i] = make_int4(p.L, 0, 0, 0);
    auto place = [&](int64_t at, const int (&g)[kSortKeep]) {
        const int here = static_cast<int>(at) + lane;
        if (alike(g)) {
            int first = 0;
            if (lane == 0) first = atomicAdd(&bins[g[0]], kBatch);
            first = __shfl_sync(0xffffffffu, first, 0) + lane;
#pragma unroll
            for (int i = 0; i < kSortKeep; ++i) p.order[first + 32 * i] = here + 32 * i;
            return;
        }
#pragma unroll
        for (int i = 0; i < kSortKeep; ++i) {
            if (at + kStep * i >= p.T) break;
            const unsigned same = __match_any_sync(0xffffffffu, g[i]);
            const int leader = __ffs(same) - 1;
            int first = 0;
            if (g[i] >= 0 && lane == leader) first = atomicAdd(&bins[g[i]], __popc(same));
            first = __shfl_sync(0xffffffffu, first, leader);
            if (g[i] >= 0) p.order[first + __popc(same & ((1u << lane) - 1))] = here + kStep * i;
        }
    };
    if (own < p.T) place(own, kept);
    for (int64_t at = own + kSortKeep * THREADS; at < p.T; at += kSortKeep * THREADS) {
        load(at, more);
        place(at, more);
    }
}

// Tile `index` of a batch of up to kInline tokens, and its tokens in `tok` (shared memory).
// False if there is no such tile. Called by a whole block. A token is first of a tile if
// no token before it has its adapter, and tiles stand in the order of their first tokens.
__device__ __forceinline__ bool find_tile(const LoraParams &p, int index, Tile &tile, int *tok, int *ids, int *found)
{
    const int tid = threadIdx.x;
    if (tid < kInline) ids[tid] = tid < p.T ? adapter_of(__ldcg(p.ids + tid), p.L) : -1;
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
    if (in) {
        int at = 0;
        for (int k = 0; k < tid; ++k) at += ids[k] == g;
        tok[at] = tid;
    }
    const int n = __syncthreads_count(in);
    tile = Tile{g, 0, n};
    return true;
}

__device__ __forceinline__ int rank_of(const LoraParams &p, int a)
{
    return p.ranks ? max(0, min(p.R, __ldcg(p.ranks + a))) : p.R;
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
    return sizeof(float) * kWarps * (T <= 8 ? 8 : (T <= 16 ? 16 : (T <= 32 ? 32 : kInline))) * (kRanks + 1);
}

template <int MT, int MOST>
__device__ __forceinline__ void shrink_tile(const LoraParams &p, const uint16_t *a, int rows, const int *tok, int count,
                                            int kb, int ke, float *red)
{
    if (count <= 8)
        shrink_steps<MT, 1>(p, a, rows, tok, count, kb, ke, red);
    else if (MOST == 16 || count <= 16)
        shrink_steps<MT, 2>(p, a, rows, tok, count, kb, ke, red);
    else if constexpr (MOST > 16) {
        if (count <= 32)
            shrink_steps<MT, 4>(p, a, rows, tok, count, kb, ke, red);
        else
            shrink_steps<MT, 8>(p, a, rows, tok, count, kb, ke, red);
    }
}

// Batches of up to MOST tokens (16: sums of two n-tiles leave registers for two blocks an SM).
// Grid: tiles x splits of K x blocks of 64 ranks.
template <int MOST>
__global__ void __launch_bounds__(kThreads, MOST == 16 ? 2 : 1) lora_shrink_few_kernel(const LoraParams p)
{
    extern __shared__ float red[];
    __shared__ int tok[kInline], ids[kInline], found[1];
    grid_dependency_wait();
    grid_launch_dependents();
    Tile tile;
    if (!find_tile(p, blockIdx.x, tile, tok, ids, found) || tile.adapter == p.L) return;
    // the adapter's ranks of this block; those it lacks are zeros
    const int rows = rank_of(p, tile.adapter) - blockIdx.z * kRanks;
    if (rows <= 0) return;                       // nobody reads sums beyond the rank
    const uint16_t *a = p.a + (static_cast<int64_t>(tile.adapter) * p.R + blockIdx.z * kRanks) * p.K;
    const int per = (p.K + 64 * p.splits - 1) / (64 * p.splits) * 64;
    const int kb = static_cast<int>(min(static_cast<int64_t>(blockIdx.y) * per, static_cast<int64_t>(p.K)));
    const int ke = static_cast<int>(min(static_cast<int64_t>(kb) + per, static_cast<int64_t>(p.K)));
    if (rows <= 16)
        shrink_tile<1, MOST>(p, a, rows, tok, tile.count, kb, ke, red);
    else if (rows <= 32)
        shrink_tile<2, MOST>(p, a, rows, tok, tile.count, kb, ke, red);
    else
        shrink_tile<4, MOST>(p, a, rows, tok, tile.count, kb, ke, red);
}

// More than kInline tokens, on the tensor core. Grid: tiles x splits of K. A stage is 64
// elements of K of 128 token rows (an MMA takes 128; what its rows beyond the tile's read is
// whatever was there) and of the adapter's rows, both in the 128-byte swizzle. Warps:
//   0-3  gather token rows by cp.async; then store the sums, a token a lane
//   4    lane 0 loads the adapter's rows by TMA
//   5    issues the MMAs (an elected lane); owns TMEM
constexpr int kLongThreads = 192;
constexpr int kLongStages = 8;
constexpr uint32_t kLongTokens = kTile * 128;
constexpr uint32_t kLongSmem = 112 * 1024;       // two blocks an SM,
constexpr uint32_t kLongSmemOne = 224 * 1024;    // one, for more than 128 ranks

struct LongParams {
    CUtensorMap tm_a;                // A as [L * R, K] bf16, box 64 elements x `rows`
    LoraParams l;
    int rows, stages;                // R rounded up to 16; stages of the ring
    uint32_t columns;                // of TMEM: a power of two
    int cluster;                     // blocks that share a tile's K as a cluster
    uint8_t *parts;                  // what a cluster leaves: u as two bf16 (see sum_cluster)
    uint64_t wait_ns;
};

struct LongShared {
    uint64_t a_full[kLongStages], x_full[kLongStages], empty[kLongStages];
    uint64_t done;
    uint32_t tmem;
    int tok[kTile];
};

// kind::f16: bf16 operands, both K-major, sums in fp32.
__host__ __device__ constexpr uint32_t idesc_bf16(int n, int m)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

__device__ __forceinline__ void mma_tc_bf16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 16 bytes from global to shared memory, of which the first `bytes` are copied and the others zeros. L2 asks for the row's next
// 128 bytes too: the whole call of 7168 -> 2112, rank 64, 32768 tokens 151.2 us, 156.8 without; 16384 87.2 and 88.4; 4096
// 31.4 and 31.6.
__device__ __forceinline__ void cp_async_or_zero(uint32_t smem_dst, const void *gsrc, uint32_t bytes)
{
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(smem_dst), "l"(gsrc), "r"(bytes) : "memory");
}

// Four numbers as two bf16 each, high and low part.
__device__ __forceinline__ void split_bf16(const float (&v)[4], uint2 &hi, uint2 &lo)
{
    uint32_t hb[2], lb[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
        hb[k] = *reinterpret_cast<const uint32_t *>(&h);
        // what rounds to infinity has no low part
        const float hx = __uint_as_float(hb[k] << 16), hy = __uint_as_float(hb[k] & 0xFFFF0000u);
        const __nv_bfloat162 l = __floats2bfloat162_rn(isinf(hx) ? 0.0f : v[2 * k] - hx, isinf(hy) ? 0.0f : v[2 * k + 1] - hy);
        lb[k] = *reinterpret_cast<const uint32_t *>(&l);
    }
    hi = make_uint2(hb[0], hb[1]);
    lo = make_uint2(lb[0], lb[1]);
}

__device__ __forceinline__ void st_cluster(uint32_t addr, const uint32_t *v)
{
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}

// Tokens of a tile whose sums a block of its cluster adds up.
__device__ __forceinline__ int cluster_tokens(const LongParams &lp, int count) { return (count <= kHalf ? kHalf : kTile) / lp.cluster; }

// Where a block keeps the sums of 64 ranks that block `from` of its cluster has of its token t: pieces of 16 bytes, spread
// over the banks.
__device__ __forceinline__ uint32_t sums_at(int from, int per, int t, int piece)
{
    return (from * per + t) * 256 + ((piece ^ (t & 15)) << 4);
}

// The sums that a cluster's blocks gave this one, added in the blocks' order, times the adapter's scale: u of
// its share of the tokens, as two bf16 a number. High parts are `parts`: a line of 64 ranks for
// every token, tokens in the order of the tiles, pieces of 16 bytes in the order that an MMA's operand has them
// in shared memory; then the low parts.
__device__ __forceinline__ void sum_cluster(const LongParams &lp, const uint8_t *smem, int4 rec, int rank, int own)
{
    const LoraParams &p = lp.l;
    const float scale = p.scales ? __ldcg(p.scales + rec.x) : 1.0f;
    const int cols = (rank + 15) / 16 * 16, per = cluster_tokens(lp, rec.z);
    for (int i = threadIdx.x; i < per * 8; i += 128) {
        const int t = own * per + (i >> 3), r = 8 * (i & 7);
        if (t >= rec.z || r >= cols) continue;
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = 0.0f;
        if (r < p.R)
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                if (s >= lp.cluster) break;
                const float4 x = *reinterpret_cast<const float4 *>(smem + sums_at(s, per, i >> 3, r >> 2));
                const float4 y = *reinterpret_cast<const float4 *>(smem + sums_at(s, per, i >> 3, (r >> 2) + 1));
                v[0] += x.x;
                v[1] += x.y;
                v[2] += x.z;
                v[3] += x.w;
                v[4] += y.x;
                v[5] += y.y;
                v[6] += y.z;
                v[7] += y.w;
            }
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = r + k < rank ? v[k] * scale : 0.0f;
        uint2 h[2], l[2];
        split_bf16({v[0], v[1], v[2], v[3]}, h[0], l[0]);
        split_bf16({v[4], v[5], v[6], v[7]}, h[1], l[1]);
        uint8_t *to = lp.parts + (static_cast<int64_t>(rec.y) + t) * 128 + (((r >> 3) ^ (t & 7)) << 4);
        *reinterpret_cast<uint4 *>(to) = make_uint4(h[0].x, h[0].y, h[1].x, h[1].y);
        *reinterpret_cast<uint4 *>(to + static_cast<int64_t>(p.T) * 128) = make_uint4(l[0].x, l[0].y, l[1].x, l[1].y);
    }
}

// CLUSTER: the blocks of a tile are a cluster and leave u; otherwise they leave its sums over their shares of K.
template <bool CLUSTER>
__global__ void __launch_bounds__(kLongThreads, 2) lora_shrink_long_kernel(const __grid_constant__ LongParams lp)
{
    extern __shared__ uint8_t smem_raw[];
    const LoraParams &p = lp.l;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int S = lp.stages;
    const uint32_t a_bytes = lp.rows * 128u, stage_bytes = kLongTokens + a_bytes;
    LongShared &sh = *reinterpret_cast<LongShared *>(smem + S * stage_bytes);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&sh.a_full[i], 1);
            mbar_init(&sh.x_full[i], 128);
            mbar_init(&sh.empty[i], 1);
        }
        mbar_init(&sh.done, 1);
        fence_mbar_init();
        tma_prefetch_desc(&lp.tm_a);
    }
    grid_dependency_wait();
    grid_launch_dependents();
    // whole blocks leave here, before TMEM is theirs
    const int4 rec = __ldcg(p.tiles + (CLUSTER ? blockIdx.x / lp.cluster : blockIdx.x));
    const int adapter = rec.x, count = rec.z;
    if (adapter == p.L || rank_of(p, adapter) == 0) return;
    const int own = CLUSTER ? static_cast<int>(cluster_ctarank()) : blockIdx.y, shares = CLUSTER ? lp.cluster : p.splits;
    const int per = (p.K + 64 * shares - 1) / (64 * shares) * 64;
    const int kb = static_cast<int>(min(static_cast<int64_t>(own) * per, static_cast<int64_t>(p.K)));
    const int ke = static_cast<int>(min(static_cast<int64_t>(kb) + per, static_cast<int64_t>(p.K)));
    const int steps = (ke - kb + 63) / 64;
    if (warp == 5) {
        tmem_alloc(&sh.tmem, lp.columns);
        tmem_relinquish();
    }
    if (tid < count) sh.tok[tid] = __ldcg(p.order + rec.y + tid);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, sh.tmem, 0);

    if (warp == 4) {
        if (lane == 0) {
            const uint64_t pol = policy_evict_last();        // other tiles of the adapter read the same rows
            bool ok = true;
            int i = 0;
            for (; i < steps; ++i) {
                const int s = i % S;
                ok = mbar_wait(&sh.empty[s], ((i / S) & 1) ^ 1u, &g_lora_error, kErrWaitEmpty, lp.wait_ns);
                if (!ok) break;
                mbar_arrive_expect_tx(&sh.a_full[s], a_bytes);
                tma_load_2d(smem + s * stage_bytes + kLongTokens, &lp.tm_a, kb + 64 * i, adapter * p.R, &sh.a_full[s], pol);
            }
            // copies in flight land before the block leaves
            for (int j = max(0, i - S); j < i; ++j)
                mbar_wait(&sh.a_full[j % S], (j / S) & 1, &g_lora_error, kErrWaitDrain);
        }
    } else if (warp == 5) {
        const uint32_t idesc = __shfl_sync(0xffffffffu, idesc_bf16(lp.rows, 128), 0);
        bool ok = true;
        for (int i = 0; i < steps; ++i) {
            const int s = i % S;
            ok = mbar_wait_warp(&sh.a_full[s], (i / S) & 1, &g_lora_error, kErrWaitFull, lp.wait_ns) &&
                 mbar_wait_warp(&sh.x_full[s], (i / S) & 1, &g_lora_error, kErrWaitOperand, lp.wait_ns);
            if (!ok) break;
            fence_proxy_async_smem();        // cp.async wrote through the generic proxy
            tc_fence_after();
            const uint64_t ad = sdesc_sw128(smem_u32(smem + s * stage_bytes));
            const uint64_t bd = sdesc_sw128(smem_u32(smem + s * stage_bytes + kLongTokens));
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < 4; ++k) mma_tc_bf16(tmem, ad + 2 * k, bd + 2 * k, idesc, i > 0 || k > 0 ? 1u : 0u);
                tc_commit(&sh.empty[s]);
            }
            __syncwarp();
        }
        // the sums are complete, or nothing of this thread runs any more; phase 0 of `done`, whichever
        if (elect_one()) tc_commit(&sh.done);
        __syncwarp();
    } else {
        // column tid % 8 of rows tid / 8 + 16 j
        const int c = tid & 7, r0 = tid >> 3;
        const uint16_t *src[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            src[j] = r0 + 16 * j < count ? p.x + static_cast<int64_t>(sh.tok[r0 + 16 * j]) * p.ldx : nullptr;
        const uint32_t dst = smem_u32(smem) + r0 * 128 + ((c ^ (r0 & 7)) << 4);
        bool ok = true;
        int i = 0;
        for (; i < steps; ++i) {
            const int s = i % S;
            ok = mbar_wait_warp(&sh.empty[s], ((i / S) & 1) ^ 1u, &g_lora_error, kErrWaitEmpty, lp.wait_ns);
            if (!ok) break;
            const int k = kb + 64 * i + 8 * c;
            const bool in = k < p.K;             // beyond the end both operands are zeros
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (src[j]) cp_async_or_zero(dst + s * stage_bytes + j * 2048, src[j] + (in ? k : 0), in ? 16u : 0u);
            cp_async_arrive(&sh.x_full[s]);
        }
        cp_async_wait_all();
        // nobody else waits for the arrivals of the last MMAs
        for (int j = max(0, i - S); j < i && ok; ++j)
            ok = mbar_wait_warp(&sh.empty[j % S], (j / S) & 1, &g_lora_error, kErrWaitDrain);
        const bool done = mbar_wait_warp(&sh.done, 0, &g_lora_error, kErrWaitAccum);
        tc_fence_after();
        const int t = 32 * warp + lane;              // this lane's token
        const uint32_t sums = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        if constexpr (CLUSTER) {
            uint32_t v[2 * 32];                      // up to 64 ranks
            if (32 * warp < count) {
                tmem_ld32(sums, *reinterpret_cast<uint32_t(*)[32]>(v));
                if (p.R > 32) tmem_ld32(sums + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
                tmem_ld_wait();
                if (!steps)
#pragma unroll
                    for (int j = 0; j < 64; ++j) v[j] = 0;
            }
            __syncwarp();
            cluster_sync();                          // every block's products are complete: the rings' memory is free
            const int per = cluster_tokens(lp, count);
            if (t < count)
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (4 * j < p.R) st_cluster(mapa_shared(smem_u32(smem) + sums_at(own, per, t % per, j), t / per), v + 4 * j);
            __syncwarp();
            cluster_sync();
            sum_cluster(lp, smem, rec, rank_of(p, adapter), own);
        } else if (ok && done && 32 * warp < count) {
            float *u = p.u + (static_cast<int64_t>(own) * p.T + (t < count ? sh.tok[t] : 0)) * p.R;
            for (int c0 = 0; c0 < p.R; c0 += 32) {
                uint32_t v[32];
                // 32 columns: those beyond the MMA's are not stored
                tmem_ld32(sums + c0, v);
                tmem_ld_wait();
                if (t < count)
#pragma unroll
                    for (int j = 0; j < 32; j += 4)
                        if (c0 + j < p.R)
                            *reinterpret_cast<uint4 *>(u + c0 + j) =
                                steps ? make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]) : make_uint4(0, 0, 0, 0);
            }
        }
    }
    __syncwarp();
    if (CLUSTER && warp >= 4) {
        cluster_sync();
        cluster_sync();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 5) {
        tc_fence_after();
        tmem_dealloc(tmem, lp.columns);
    }
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

// 16 bytes of a line that is read whole, soon after one another.
__device__ __forceinline__ uint4 load_line(const void *p)
{
    uint4 v;
    asm volatile("ld.global.L2::128B.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
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

// Rows of B of one chunk of 32 channels for 32 ranks from k0 on: 8 neighbouring ranks of four
// channels a lane. brow: this lane's first; left: channels and ranks there are from it on.
__device__ __forceinline__ void load_b(uint4 (&w)[4], const uint16_t *brow, int R, int k0, int channels, int ranks)
{
    if (channels > 6 && ranks >= 8) {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = __ldg(reinterpret_cast<const uint4 *>(brow + 2 * j * R + k0));
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w[j] = make_uint4(0, 0, 0, 0);
            if (channels > 2 * j && ranks > 0)
                w[j] = keep_first(__ldg(reinterpret_cast<const uint4 *>(brow + 2 * j * R + k0)), ranks);
        }
    }
}

// u of 16 tokens for 32 ranks in the MMAs' order: a lane's eight ranks of tokens g and g + 8,
// high and low parts.
struct RowsOfU {
    uint4 h0, h1, l0, l1;
};
__device__ __forceinline__ RowsOfU load_u(const uint32_t *hrow, const uint32_t *lrow, int ldu)
{
    return RowsOfU{*reinterpret_cast<const uint4 *>(hrow), *reinterpret_cast<const uint4 *>(hrow + 8 * ldu),
                   *reinterpret_cast<const uint4 *>(lrow), *reinterpret_cast<const uint4 *>(lrow + 8 * ldu)};
}

// d += u B^T over 32 ranks, for one chunk of channels and 16 tokens.
__device__ __forceinline__ void multiply(float (&d)[4][4], const uint4 (&w)[4], const RowsOfU &u)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        mma_bf16(d[j], u.l0.x, u.l1.x, u.l0.y, u.l1.y, w[j].x, w[j].y);
        mma_bf16(d[j], u.l0.z, u.l1.z, u.l0.w, u.l1.w, w[j].z, w[j].w);
        mma_bf16(d[j], u.h0.x, u.h1.x, u.h0.y, u.h1.y, w[j].x, w[j].y);
        mma_bf16(d[j], u.h0.z, u.h1.z, u.h0.w, u.h1.w, w[j].z, w[j].w);
    }
}

// Eight channels of base and their sums of token g (h = 0) or g + 8, rounded once.
template <bool F16>
__device__ __forceinline__ uint4 updated(const uint4 &base, const float (&d)[4][4], int h)
{
    const uint32_t v[4] = {base.x, base.y, base.z, base.w};
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 t = unpack2<F16>(v[j]);
        o[j] = pack2<F16>(t.x + d[j][2 * h], t.y + d[j][2 * h + 1]);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Columns 32c .. 32c + 31 of C for 16 tokens, c0 <= c < c1: channel of column `col` of the n-tile j
// is 32c + 8 (col / 2) + 2j + (col & 1), so lane (g, q) ends with channels 8q .. 8q + 7 of tokens g and
// g + 8. hi, lo, tok: of the first of the tokens. KEPT: the ranks are at most 32 * KEPT, and
// the next chunk's rows of B and base are on their way while one is multiplied (0: any
// rank, loaded as it goes).
template <bool F16, int KEPT>
__device__ __forceinline__ void expand_chunks(const LoraParams &p, const uint16_t *b, int rank, const uint32_t *hi,
                                              const uint32_t *lo, int ldu, const int *tok, int count, int c0, int c1)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int first = 8 * (g >> 1) + (g & 1);            // this lane's row of B in n-tile 0 of a chunk
    const uint32_t *hrow = hi + g * ldu + 4 * q, *lrow = lo + g * ldu + 4 * q;
    const uint16_t *base[2];
    uint16_t *out[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const bool has = 8 * h + g < count;
        base[h] = has ? p.base + tok[8 * h + g] * p.ldb + 8 * q : nullptr;
        out[h] = has ? p.c + tok[8 * h + g] * p.ldc + 8 * q : nullptr;
    }
    const uint16_t *brow = b + static_cast<int64_t>(32 * c0 + first) * p.R + 8 * q;
    uint4 w[KEPT ? KEPT : 1][4], old[2];
    auto fetch = [&](int c) {
        if (c >= c1) return;
        if constexpr (KEPT > 0)
#pragma unroll
            for (int k = 0; k < KEPT; ++k)
                load_b(w[k], brow, p.R, 32 * k, p.N - 32 * c - first, rank - 32 * k - 8 * q);
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (base[h] && 32 * c + 8 * q < p.N) old[h] = load_line(base[h] + 32 * c);
    };
    fetch(c0);
    for (int c = c0; c < c1; ++c) {
        float d[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) d[j][e] = 0.0f;
        if constexpr (KEPT > 0) {
#pragma unroll
            for (int k = 0; k < KEPT; ++k) multiply(d, w[k], load_u(hrow + 16 * k, lrow + 16 * k, ldu));
        } else {
            for (int k = 0; k < rank; k += 32) {
                load_b(w[0], brow, p.R, k, p.N - 32 * c - first, rank - k - 8 * q);
                multiply(d, w[0], load_u(hrow + k / 2, lrow + k / 2, ldu));
            }
        }
        const uint4 was[2] = {old[0], old[1]};
        brow += 32 * p.R;
        fetch(c + 1);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (out[h] && 32 * c + 8 * q < p.N) *reinterpret_cast<uint4 *>(out[h] + 32 * c) = updated<F16>(was[h], d, h);
        }
    }
}

// The same for more than 16 tokens and adapters of up to 64 ranks (kRanks): the `parts` warps of a lane group share
// a chunk's rows of B. kAhead chunks of B and of every warp's base are on their way to
// shared memory, by cp.async. With both in registers one chunk ahead, a warp had 1 KB of base in
// flight, and this part took 13 us at 4096 x 2112 where its bytes take 5.
constexpr int kAhead = 3;
constexpr uint32_t kRingB = 32 * 128;            // 32 channels of up to 64 ranks
constexpr uint32_t kRingBase = 32 * 32;          // 16 tokens x 32 channels

__host__ __device__ constexpr uint32_t ring_bytes() { return kAhead * (kWarps / 2 * kRingB + kWarps * kRingBase); }

template <bool F16>
__device__ __forceinline__ void expand_ring(const LoraParams &p, const uint16_t *b, int rank, const uint32_t *hi,
                                            const uint32_t *lo, int ldu, const int *tok, int count, int c0, int c1, int part,
                                            int parts, uint8_t *ring)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int group = warp / parts, in_group = part * 32 + lane, blocks = (rank + 31) / 32;
    uint8_t *bring = ring + group * kAhead * kRingB;
    uint8_t *own = ring + kAhead * (kWarps / 2 * kRingB + warp * kRingBase) + lane * 16;
    const uint32_t *hrow = hi + g * ldu + 4 * q, *lrow = lo + g * ldu + 4 * q;
    const uint16_t *base[2];
    uint16_t *out[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const bool has = 8 * h + g < count;
        base[h] = has ? p.base + tok[8 * h + g] * p.ldb + 8 * q : nullptr;
        out[h] = has ? p.c + tok[8 * h + g] * p.ldc + 8 * q : nullptr;
    }
    auto request = [&](int c, int slot) {
        if (c < c1) {
            // row r of the chunk, ranks 8v to 8v + 7: half a line further for odd rows, so that the
            // rows a load takes at once lie in different banks
            for (int i = in_group; i < 32 * 4 * blocks; i += 32 * parts) {
                const int r = blocks == 1 ? i >> 2 : i >> 3, v = blocks == 1 ? i & 3 : i & 7;
                if (32 * c + r < p.N && 8 * v < rank)
                    cp_async<16>(smem_u32(bring + slot * kRingB + r * 128 + ((16 * v) ^ ((r & 1) << 6))),
                                 b + static_cast<int64_t>(32 * c + r) * p.R + 8 * v);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (base[h] && 32 * c + 8 * q < p.N)
                    cp_async<16>(smem_u32(own + slot * kRingBase + h * 512), base[h] + 32 * c);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kAhead - 1; ++i) request(c0 + i, i);
    const uint32_t first = 8 * (g >> 1) + (g & 1);
    int slot = 0;
    for (int c = c0; c < c1; ++c) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 2) : "memory");
        // everyone's copies of this chunk have landed, and everyone is done with the one before
        asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * parts) : "memory");
        request(c + kAhead - 1, slot == 0 ? kAhead - 1 : slot - 1);
        float d[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) d[j][e] = 0.0f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (k >= blocks) break;
            uint4 w[4];
            const uint8_t *at = bring + slot * kRingB + first * 128 + ((64 * k + 16 * q) ^ ((g & 1) << 6));
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = *reinterpret_cast<const uint4 *>(at + 256 * j);
            if (32 * k + 32 > rank)
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = keep_first(w[j], rank - 32 * k - 8 * q);
            multiply(d, w, load_u(hrow + 16 * k, lrow + 16 * k, ldu));
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (!out[h] || 32 * c + 8 * q >= p.N) continue;
            const uint4 was = *reinterpret_cast<const uint4 *>(own + slot * kRingBase + h * 512);
            *reinterpret_cast<uint4 *>(out[h] + 32 * c) = updated<F16>(was, d, h);
        }
        slot = slot + 1 == kAhead ? 0 : slot + 1;
    }
}

// Words between rows of u in shared memory: 16 more than a multiple of 32, so that the
// 16-byte loads of two rows' lanes take all banks.
__host__ __device__ constexpr int u_stride(int cols) { return cols / 2 % 32 ? cols / 2 : cols / 2 + 16; }

__device__ __forceinline__ void prefetch_l2(const void *p)
{
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// C = base for some of a tile's tokens and the vectors of eight channels from v0 to v1 - 1, `step` apart.
__device__ __forceinline__ void copy_rows(const LoraParams &p, const int *tok, int count, uint32_t v0, uint32_t v1, uint32_t step)
{
    for (uint32_t i = v0; i < v1; i += step)
        for (int t0 = 0; t0 < count; t0 += 8) {
            uint4 v[8];
#pragma unroll
            for (int t = 0; t < 8; ++t)
                if (t0 + t < count) v[t] = reinterpret_cast<const uint4 *>(p.base + tok[t0 + t] * p.ldb)[i];
#pragma unroll
            for (int t = 0; t < 8; ++t)
                if (t0 + t < count) reinterpret_cast<uint4 *>(p.c + tok[t0 + t] * p.ldc)[i] = v[t];
        }
}

// Grid: halves of tiles (up to kInline tokens: tiles) x blocks of channels. Shared memory: u as
// high and low bf16, [64 tokens][ranks rounded up to 32].
template <bool INLINE, bool F16>
__global__ void __launch_bounds__(kThreads, 2) lora_expand_kernel(const LoraParams p)
{
    extern __shared__ uint32_t ushared[];
    __shared__ int tok[kHalf], ids[kInline], found[1];
    const int chunks = (p.N + 31) / 32, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Tile tile;
    // The launch before let this one start when everything before it had completed: all but u
    // is there, in L2.
    if constexpr (INLINE) {
        if (!find_tile(p, blockIdx.x, tile, tok, ids, found)) {
            grid_dependency_wait();
            return;
        }
    } else {
        const int4 r = __ldcg(p.tiles + (blockIdx.x >> 1));
        const int skip = (blockIdx.x & 1) * kHalf;
        if (r.z <= skip) {
            grid_dependency_wait();
            return;
        }
        tile = Tile{r.x, r.y + skip, min(kHalf, r.z - skip)};
        if (threadIdx.x < tile.count) tok[threadIdx.x] = __ldcg(p.order + tile.first + threadIdx.x);
        __syncthreads();
    }
    if (tile.adapter == p.L) {
        // no adapter: a copy of base, as it is
        grid_dependency_wait();
        grid_launch_dependents();
        copy_rows(p, tok, tile.count, blockIdx.y * kThreads + threadIdx.x, p.N / 8, gridDim.y * kThreads);
        return;
    }
    const int rank = rank_of(p, tile.adapter);
    const uint16_t *b = p.b + static_cast<int64_t>(tile.adapter) * p.N * p.R;
    const int rows = (tile.count + 15) / 16 * 16, cols = max(1, (rank + 31) / 32) * 32;   // 32 zeros of an adapter of rank 0
    const int ldu = u_stride((p.R + 31) / 32 * 32);
    // The block's warps share its 16-token parts (1, 2 or 4 of them) and, those of a part, its chunks.
    const int parts = tile.count <= 16 ? 1 : (tile.count <= 32 ? 2 : 4), part = warp & (parts - 1);
    // neighbouring chunks, which share lines of 128 bytes, go to one warp
    const int lanes = gridDim.y * (kWarps / parts), mine = blockIdx.y * (kWarps / parts) + warp / parts;
    const int c0 = static_cast<int>(static_cast<int64_t>(chunks) * mine / lanes);
    const int c1 = static_cast<int>(static_cast<int64_t>(chunks) * (mine + 1) / lanes);
    // this warp's part of base and, once for all parts, of B go to L2 while u is made
    if (lane < 16 && 16 * part + lane < tile.count)
        for (int n = 32 * c0; n < min(32 * c1, p.N); n += 64) prefetch_l2(p.base + tok[16 * part + lane] * p.ldb + n);
    if (part == 0)
        for (int ch = 32 * c0 + lane; ch < min(32 * c1, p.N); ch += 32)
            for (int k = 0; k < rank; k += 64) prefetch_l2(b + static_cast<int64_t>(ch) * p.R + k);
    const float scale = p.scales ? __ldcg(p.scales + tile.adapter) : 1.0f;
    grid_dependency_wait();
    grid_launch_dependents();
    uint32_t *hi = ushared, *lo = ushared + kHalf * ldu;
    // four neighbouring ranks of two tokens a thread, eight splits on their way
    for (int r = 4 * (threadIdx.x & 7); r < cols; r += 32)
        for (int t0 = threadIdx.x >> 3; t0 < rows; t0 += kThreads / 4) {
            float4 sum[2];
            const float *u[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = t0 + i * (kThreads / 8);
                sum[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                u[i] = t < tile.count && r < rank ? p.u + static_cast<int64_t>(tok[t]) * p.R + r : nullptr;
            }
            const int64_t split = static_cast<int64_t>(p.T) * p.R;
            for (int s0 = 0; s0 < p.splits; s0 += 8) {
                float4 some[2][8];
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int s = 0; s < 8; ++s)
                        if (u[i] && s0 + s < p.splits)
                            some[i][s] = __ldcg(reinterpret_cast<const float4 *>(u[i] + (s0 + s) * split));
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int s = 0; s < 8; ++s) {
                        if (!u[i] || s0 + s >= p.splits) continue;
                        sum[i].x += some[i][s].x;
                        sum[i].y += some[i][s].y;
                        sum[i].z += some[i][s].z;
                        sum[i].w += some[i][s].w;
                    }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = t0 + i * (kThreads / 8);
                if (t >= rows) continue;
                float v[4] = {sum[i].x, sum[i].y, sum[i].z, sum[i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = r + k < rank ? v[k] * scale : 0.0f;
                uint2 h, l;
                split_bf16(v, h, l);
                *reinterpret_cast<uint2 *>(hi + t * ldu + r / 2) = h;
                *reinterpret_cast<uint2 *>(lo + t * ldu + r / 2) = l;
            }
        }
    __syncthreads();
    // 64 ranks of B are what the registers hold beside the rest, and the ring
    const int left = tile.count - 16 * part, at = 16 * part * ldu;
    if (parts > 1 && p.R <= kRanks) {
        expand_ring<F16>(p, b, rank, hi + at, lo + at, ldu, tok + 16 * part, left, c0, c1, part, parts,
                         reinterpret_cast<uint8_t *>(lo + kHalf * ldu));
        return;
    }
    if (left <= 0) return;
    if (rank <= 32)
        expand_chunks<F16, 1>(p, b, rank, hi + at, lo + at, ldu, tok + 16 * part, left, c0, c1);
    else if (rank <= 64)
        expand_chunks<F16, 2>(p, b, rank, hi + at, lo + at, ldu, tok + 16 * part, left, c0, c1);
    else
        expand_chunks<F16, 0>(p, b, rank, hi + at, lo + at, ldu, tok + 16 * part, left, c0, c1);
}

// ------------------------------------------- expand, whole tiles of tokens

// Batches of well filled tiles, up to 64 ranks: u B^T by tcgen05, rows are a tile's 128 tokens, columns 64 channels
// a step. base comes to shared memory by cp.async, where a lane adds its token's sums, and leaves as C
// from there in whole lines (a lane's own row would be 32 lines a store); steps' B (TMA) and base are three ahead.
// Bound: what base and C take of HBM, a step's 32 KB in 1.3 us where two blocks an SM do the same.
// Warps:
//   0-7  base to C
//   8    lane 0 loads B, and u as sum_cluster left it
//   9    issues the MMAs; owns TMEM
constexpr int kTileThreads = kThreads + 64;
constexpr int kWide = 64;                // channels of a step
constexpr int kSteps = 3;                // of B and base in shared memory
constexpr uint32_t kUBytes = kTile * 128;            // of u's high parts (then of the low ones): 64 ranks a token
constexpr uint32_t kBAt = 2 * kUBytes, kBBytes = kWide * 128;
constexpr uint32_t kBaseAt = kBAt + kSteps * kBBytes, kBaseBytes = kTile * kWide * 2;
constexpr uint32_t kTileShared = kBaseAt + kSteps * kBaseBytes;

struct TileParams {
    CUtensorMap tm_b;                // B as [L * N, R] bf16, box 64 elements x kWide
    LoraParams l;
    const uint8_t *parts;            // u, as sum_cluster leaves it
    uint64_t wait_ns;
};

struct TileShared {
    uint64_t u_full;
    uint64_t b_full[kSteps], b_free[kSteps], acc_full[2], acc_empty[2];
    uint32_t tmem;
    int abort;
    int tok[kTile];
};
constexpr uint32_t kTileSmem = kTileShared + sizeof(TileShared) + 1024;
static_assert(kTileSmem <= 113 * 1024, "two blocks an SM");

__device__ __forceinline__ void workers_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// Grid: tiles x blocks of channels.
template <bool F16>
__global__ void __launch_bounds__(kTileThreads, 2) lora_expand_tile_kernel(const __grid_constant__ TileParams tp)
{
    extern __shared__ uint8_t smem_raw[];
    const LoraParams &p = tp.l;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    TileShared &sh = *reinterpret_cast<TileShared *>(smem + kTileShared);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    // The launch before let this one start when everything before it had completed: all but u
    // is there, in L2.
    const int4 rec = __ldcg(p.tiles + blockIdx.x);
    const int adapter = rec.x, count = rec.z;
    const int rank = adapter == p.L ? 0 : rank_of(p, adapter);
    if (tid < count) sh.tok[tid] = __ldcg(p.order + rec.y + tid);
    if (rank == 0 || count == 0) {
        __syncthreads();
        grid_dependency_wait();
        grid_launch_dependents();
        // no update: a copy of base, as it is
        if (p.copy) copy_rows(p, sh.tok, count, blockIdx.y * kTileThreads + tid, p.N / 8, gridDim.y * kTileThreads);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < kSteps; ++i) {
            mbar_init(&sh.b_full[i], 1);
            mbar_init(&sh.b_free[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.acc_full[i], 1);
            mbar_init(&sh.acc_empty[i], kWarps);
        }
        mbar_init(&sh.u_full, 1);
        sh.abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tp.tm_b);
    }
    if (warp == 9) {
        tmem_alloc(&sh.tmem, 2 * kWide);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, sh.tmem, 0);
    // this block's steps of 64 channels: whole lines of C
    const int units = (p.N + kWide - 1) / kWide;
    const int unit = static_cast<int>(static_cast<int64_t>(units) * blockIdx.y / gridDim.y), n0 = unit * kWide;
    const int steps = static_cast<int>(static_cast<int64_t>(units) * (blockIdx.y + 1) / gridDim.y) - unit;

    if (warp == 8) {
        if (lane == 0) {
            const uint64_t pol = policy_evict_last();        // other tiles of the adapter read the same rows
            int i = 0;
            bool ok = true;
            auto load_to = [&](int end) {
                for (; i < end; ++i) {
                    const int s = i % kSteps;
                    ok = mbar_wait(&sh.b_free[s], ((i / kSteps) & 1) ^ 1u, &g_lora_error, kErrWaitEmpty, tp.wait_ns);
                    if (!ok) return;
                    mbar_arrive_expect_tx(&sh.b_full[s], kBBytes);
                    tma_load_2d(smem + kBAt + s * kBBytes, &tp.tm_b, 0, adapter * p.N + n0 + i * kWide, &sh.b_full[s], pol);
                }
            };
            load_to(min(steps, kSteps));
            grid_dependency_wait();
            const uint8_t *u = tp.parts + static_cast<int64_t>(rec.y) * 128;
            mbar_arrive_expect_tx(&sh.u_full, 2 * count * 128);
            bulk_load(smem, u, count * 128, &sh.u_full, pol);
            bulk_load(smem + kUBytes, u + static_cast<int64_t>(p.T) * 128, count * 128, &sh.u_full, pol);
            if (ok) load_to(steps);
            // copies in flight land before the block leaves
            mbar_wait(&sh.u_full, 0, &g_lora_error, kErrWaitDrain);
            for (int j = max(0, i - kSteps); j < i; ++j)
                mbar_wait(&sh.b_full[j % kSteps], (j / kSteps) & 1, &g_lora_error, kErrWaitDrain);
        }
        __syncwarp();
        grid_dependency_wait();
    } else if (warp == 9) {
        grid_dependency_wait();
        const uint32_t idesc = __shfl_sync(0xffffffffu, idesc_bf16(kWide, 128), 0);
        const int ks = (rank + 15) / 16;
        const bool there = mbar_wait_warp(&sh.u_full, 0, &g_lora_error, kErrWaitOperand, tp.wait_ns);
        int i = 0;
        for (; i < steps && there; ++i) {
            const int s = i % kSteps, buf = i & 1;
            const bool ok = mbar_wait_warp(&sh.acc_empty[buf], ((i >> 1) & 1) ^ 1u, &g_lora_error, kErrWaitAccum, tp.wait_ns) &&
                            mbar_wait_warp(&sh.b_full[s], (i / kSteps) & 1, &g_lora_error, kErrWaitFull, tp.wait_ns);
            if (!ok) break;
            uint8_t *b = smem + kBAt + s * kBBytes;
            if (rank < p.R && rank < 16 * ks)
                // what B holds beyond the rank is not used, whatever it is
                for (int r = lane; r < kWide; r += 32)
                    for (int k = rank; k < 16 * ks; ++k)
                        *reinterpret_cast<uint16_t *>(b + r * 128 + (((k >> 3) ^ (r & 7)) << 4) + 2 * (k & 7)) = 0;
            fence_proxy_async_smem();
            __syncwarp();
            tc_fence_after();
            const uint64_t hi = sdesc_sw128(smem_u32(smem)), lo = sdesc_sw128(smem_u32(smem + kUBytes));
            const uint64_t bd = sdesc_sw128(smem_u32(b));
            if (elect_one()) {
                for (int k = 0; k < ks; ++k) {
                    mma_tc_bf16(tmem + buf * kWide, lo + 2 * k, bd + 2 * k, idesc, k > 0 ? 1u : 0u);
                    mma_tc_bf16(tmem + buf * kWide, hi + 2 * k, bd + 2 * k, idesc, 1u);
                }
                tc_commit(&sh.b_free[s]);
                tc_commit(&sh.acc_full[buf]);
            }
            __syncwarp();
        }
        // nobody else waits for the arrivals of the last MMAs
        for (int j = max(0, i - kSteps); j < i; ++j)
            mbar_wait_warp(&sh.b_free[j % kSteps], (j / kSteps) & 1, &g_lora_error, kErrWaitDrain);
    } else {
        // a thread's pieces of base and C: eight channels (c) of tokens row + 32 j
        const int c = tid & 7, row = tid >> 3;
        auto request = [&](int i) {
            const int n = n0 + i * kWide + 8 * c;
            if (i < steps && n < p.N) {
                const uint32_t to = smem_u32(smem + kBaseAt + i % kSteps * kBaseBytes) + row * 128 + ((c ^ (row & 7)) << 4);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (row + 32 * j < count) cp_async<16>(to + j * 4096, p.base + sh.tok[row + 32 * j] * p.ldb + n);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll
        for (int i = 0; i < kSteps; ++i) request(i);
        grid_dependency_wait();
        grid_launch_dependents();
        const int wrow = 32 * (warp & 3), t = wrow + lane, half = warp >> 2;   // this lane's token, and half of the channels
        bool ok = true;
        for (int i = 0; i < steps; ++i) {
            const int buf = i & 1;
            uint8_t *place = smem + kBaseAt + i % kSteps * kBaseBytes;
            asm volatile("cp.async.wait_group %0;" ::"n"(kSteps - 1) : "memory");
            ok = mbar_wait_warp(&sh.acc_full[buf], (i >> 1) & 1, &g_lora_error, kErrWaitAccum, tp.wait_ns);
            if (!ok) *reinterpret_cast<volatile int *>(&sh.abort) = 1;
            tc_fence_after();
            workers_sync();                  // everyone's part of base has landed
            if (*reinterpret_cast<volatile int *>(&sh.abort)) break;       // for all: it is set before this barrier only
            if (wrow < count) {
                uint32_t v[32];
                tmem_ld32(tmem + buf * kWide + 32 * half + (static_cast<uint32_t>(wrow) << 16), v);
                tmem_ld_wait();
                if (t < count)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint4 *at = reinterpret_cast<uint4 *>(place + t * 128 + (((4 * half + j) ^ (t & 7)) << 4));
                        const uint4 was = *at;
                        const uint32_t w[4] = {was.x, was.y, was.z, was.w};
                        uint32_t o[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float2 f = unpack2<F16>(w[k]);
                            const float x = __uint_as_float(v[8 * j + 2 * k]), y = __uint_as_float(v[8 * j + 2 * k + 1]);
                            o[k] = pack2<F16>(f.x + x, f.y + y);
                        }
                        *at = make_uint4(o[0], o[1], o[2], o[3]);
                    }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.acc_empty[buf]);
            workers_sync();                  // all sums are added
            const int n = n0 + i * kWide + 8 * c;
            if (n < p.N) {
                const uint8_t *from = place + row * 128 + ((c ^ (row & 7)) << 4);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (row + 32 * j < count)
                        *reinterpret_cast<uint4 *>(p.c + sh.tok[row + 32 * j] * p.ldc + n) =
                            *reinterpret_cast<const uint4 *>(from + j * 4096);
            }
            request(i + kSteps);             // a thread's own pieces again, which nobody else reads now
        }
        cp_async_wait_all();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 2 * kWide);
    }
}

template <typename Kern, typename P>
cudaError_t launch(Kern kern, dim3 grid, int threads, size_t smem, cudaStream_t stream, const P &p, int cluster = 1)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

// Tiles of a long batch that there may be (every adapter leaves half of one empty): the GPU alone knows.
int likely_tiles(const LoraParams &p) { return std::min<int>(p.max_tiles, p.T / kTile + (p.L + 1) / 2 + 1); }

template <bool F16>
cudaError_t launch_expand_tile(const LoraParams &p, const LoraLayout &l, cudaStream_t stream)
{
    static KernelOnce once;
    int sms = 0;
    const cudaError_t e = prepare_kernel(lora_expand_tile_kernel<F16>, kTileSmem, once, &sms);
    if (e != cudaSuccess) return e;
    TileParams tp;
    tp.l = p;
    tp.parts = reinterpret_cast<const uint8_t *>(p.u);
    tp.wait_ns = wait_limit_ns();
    if (!encode_map_2d(&tp.tm_b, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.b, p.R, static_cast<uint64_t>(p.L) * p.N,
                       static_cast<uint64_t>(p.R) * 2, 64u, kWide, CU_TENSOR_MAP_SWIZZLE_128B,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_128B))
        return cudaErrorInvalidValue;
    const int units = (p.N + kWide - 1) / kWide;
    // blocks a tile: as many as make the waves of blocks, two an SM, shortest (a block's start takes about three steps)
    int blocks = 1;
    int64_t best = INT64_MAX;
    for (int n = 1; n <= std::min(units, 2 * sms); ++n) {
        const int64_t waves = (static_cast<int64_t>(likely_tiles(p)) * n + 2 * sms - 1) / (2 * sms);
        const int64_t length = waves * ((units + n - 1) / n + 3);
        if (length < best) {
            best = length;
            blocks = n;
        }
    }
    return launch(lora_expand_tile_kernel<F16>, dim3(l.max_tiles, blocks), kTileThreads, kTileSmem, stream, tp);
}

template <bool INLINE, bool F16>
cudaError_t launch_expand(const LoraParams &p, const LoraLayout &l, cudaStream_t stream)
{
    static KernelOnce once;
    constexpr size_t most = sizeof(uint32_t) * 2 * kHalf * u_stride(kMaxRank) + ring_bytes();
    int sms = 0;
    const cudaError_t e = prepare_kernel(lora_expand_kernel<INLINE, F16>, most, once, &sms);
    if (e != cudaSuccess) return e;
    const size_t smem = sizeof(uint32_t) * 2 * kHalf * u_stride((p.R + 31) / 32 * 32) + (p.T > 16 && p.R <= kRanks ? ring_bytes() : 0);
    // blocks of channels: as many as give every SM two blocks, no more than one chunk a warp. How
    // many halves of tiles there are the GPU alone knows: an adapter leaves one half empty on average
    const int tiles = INLINE ? l.max_tiles : 2 * l.max_tiles, chunks = (p.N + 31) / 32;
    const int full = INLINE ? tiles : std::min<int>(tiles, p.T / kHalf + (p.L + 1) / 2 + 1);
    const int blocks = std::max(1, std::min((chunks + kWarps - 1) / kWarps, 2 * sms / full));
    return launch(lora_expand_kernel<INLINE, F16>, dim3(tiles, blocks), kThreads, smem, stream, p);
}

}  // namespace

// A tile is 128 tokens, but a block of a batch that works its tiles out itself has all of an adapter's.
LoraLayout lora_layout(int64_t T, int64_t K, int R, int L)
{
    LoraLayout l;
    // every group of tokens wastes less than one tile
    l.max_tiles = static_cast<int>(std::min<int64_t>(T, T / kTile + L + 1));
    // splits of K: two blocks an SM if all tiles are there (one of 17 to kInline tokens, by
    // registers), each with 512 elements at least (one step of every warp, or eight stages)
    const int64_t blocks = T > 16 && T <= kInline ? 152 : 304;
    l.splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({blocks / l.max_tiles, 32, (K + 511) / 512})));
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    // splits * T is at most 32 T, and at most 304 / (T / 128) * T or T: a bound that grows with T
    const int64_t most = std::min<int64_t>(32 * T, std::max<int64_t>(304 * kTile, T));
    l.u = 0;
    // or, for up to kRanks ranks, two lines of 64 bf16 a token
    l.order = l.u + up(std::max(sizeof(float) * static_cast<size_t>(most) * R, static_cast<size_t>(256) * T));
    l.tiles = l.order + up(sizeof(int) * static_cast<size_t>(T));
    l.total = l.tiles + up(sizeof(int4) * static_cast<size_t>(l.max_tiles));
    return l;
}

cudaError_t launch_lora(LoraParams p, const LoraLayout &l, bool f16, cudaStream_t stream)
{
    p.splits = l.splits;
    p.max_tiles = l.max_tiles;
    cudaError_t e;
    if (p.T <= kInline) {
        const dim3 grid(l.max_tiles, l.splits, (p.R + kRanks - 1) / kRanks);
        if (p.T <= 16) {
            e = launch(lora_shrink_few_kernel<16>, grid, kThreads, shrink_smem(p.T), stream, p);
        } else {
            static KernelOnce once;
            e = prepare_kernel(lora_shrink_few_kernel<kInline>, shrink_smem(kInline), once, nullptr);
            if (e != cudaSuccess) return e;
            e = launch(lora_shrink_few_kernel<kInline>, grid, kThreads, shrink_smem(p.T), stream, p);
        }
        if (e != cudaSuccess) return e;
        return f16 ? launch_expand<true, true>(p, l, stream) : launch_expand<true, false>(p, l, stream);
    }
    // barriers of 32 warps cost more than the rounds that they save, up to what registers keep
    const size_t bins = sizeof(int) * (p.L + 1);
    e = p.T <= 256 * kSortKeep    ? launch(lora_sort_kernel<256, false>, dim3(1), 256, bins, stream, p)
        : p.T <= 1024 * kSortKeep ? launch(lora_sort_kernel<1024, false>, dim3(1), 1024, bins, stream, p)
                                  : launch(lora_sort_kernel<1024, true>, dim3(1), 1024, bins, stream, p);
    if (e != cudaSuccess) return e;
    LongParams lp;
    lp.l = p;
    lp.rows = (p.R + 15) & ~15;
    const uint32_t smem = lp.rows <= 128 ? kLongSmem : kLongSmemOne;
    lp.stages = std::min<int>(kLongStages, (smem - 1024 - sizeof(LongShared)) / (kLongTokens + lp.rows * 128));
    lp.columns = 32;
    while (lp.columns < static_cast<uint32_t>(lp.rows)) lp.columns *= 2;
    lp.wait_ns = wait_limit_ns();
    if (!encode_map_2d(&lp.tm_a, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.a, p.K, static_cast<uint64_t>(p.L) * p.R,
                       static_cast<uint64_t>(p.K) * 2, 64u, lp.rows, CU_TENSOR_MAP_SWIZZLE_128B,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B))
        return cudaErrorInvalidValue;
    lp.parts = reinterpret_cast<uint8_t *>(p.u);
    lp.cluster = 1;
    // whole tiles of tokens: ranks that one line of u holds, rows of B that TMA's 32-bit coordinates reach, and tiles that
    // are filled well enough
    const int likely = likely_tiles(p);
    if (p.R <= kRanks && static_cast<int64_t>(p.L) * p.N <= (int64_t(1) << 31) - kWide && p.T >= kHalf * likely) {
        static KernelOnce once;
        int sms = 0;
        e = prepare_kernel(lora_shrink_long_kernel<true>, kLongSmem, once, &sms);
        if (e != cudaSuccess) return e;
        // as many blocks a tile as give every SM two, with at least four stages of K each
        lp.cluster = 8;
        while (lp.cluster > 1 && (lp.cluster * likely > 2 * sms || lp.cluster * 256 > p.K + 255)) lp.cluster /= 2;
        e = launch(lora_shrink_long_kernel<true>, dim3(l.max_tiles * lp.cluster), kLongThreads, smem, stream, lp, lp.cluster);
        if (e != cudaSuccess) return e;
        return f16 ? launch_expand_tile<true>(p, l, stream) : launch_expand_tile<false>(p, l, stream);
    }
    static KernelOnce once;
    e = prepare_kernel(lora_shrink_long_kernel<false>, kLongSmemOne, once, nullptr);
    if (e != cudaSuccess) return e;
    e = launch(lora_shrink_long_kernel<false>, dim3(l.max_tiles, l.splits), kLongThreads, smem, stream, lp);
    if (e != cudaSuccess) return e;
    return f16 ? launch_expand<false, true>(p, l, stream) : launch_expand<false, false>(p, l, stream);
}

int read_and_clear_lora_error()
{
    int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_lora_error, sizeof(int)) != cudaSuccess) return -1;
    cudaMemcpyToSymbol(g_lora_error, &zero, sizeof(int));
    return v;
}

}  // namespace mxfp4
