// The experts' products of a mixture-of-experts layer (mxfp4_moe_experts):
// MXFP8 activations x MXFP4 weights on the tensor cores (tcgen05.mma
// kind::mxf8f6f4), for row counts that only the GPU knows.
//
// Mathematics, for token t and its choice j of expert e:
//   act = MXFP8(silu(x_t G_e^T) * (x_t U_e^T)),  out_t = sum_j w_tj (act W2_e^T).
//
// Launches, each one starting while the last drains (programmatic dependent
// launch):
//   place    sorts the T * k choices by expert (counts in shared memory, prefix
//            sums, ranks): row r of the sorted order comes from token src[r],
//            choice i sits in row pos[i]; rec lists the tiles of NT rows.
//            More than kChunk choices take several blocks and a counting launch
//            before it.
//   gather   long batches only: token rows and their scales in sorted order
//   product1 epilogue silu(g) * u, MXFP8, to the workspace in sorted order
//   product2 act x W2^T, fp32 rows to the workspace
//   combine  out_t = sum_j w_tj row[pos[t, j]], in the order of j: no atomics, so
//            the result does not depend on the order of the sorted rows. The rows are
//            the accumulators as they are, so the sum is rounded once, to bf16; rows
//            of half the size would make the error of the result 1.4 times that
//            of this rounding, and more where experts cancel
//
// Both products swap the operands: the 128 rows of the MMA are weight rows, its
// columns are tokens. Weights, which dominate the traffic of a small batch, fill
// every row of the tensor core whatever the batch, and N follows the rows that an
// expert has (a multiple of 16). Product 1 puts 64 rows of G and the 64 rows of U
// of the same channels in one tile, so the epilogue has both of a channel.
//
// Bound: few rows an expert, the weights' bytes from HBM; many, the tensor core and
// the shared memory that feeds it. Measured whole (hidden size 7168, intermediate
// 2048, 32 experts, 8 choices): 1 token 53 us (187 MB, 28 us at the copy bandwidth),
// 4096 tokens 1.32 ms called one after another, 1.28 ms in a graph (2.9 TFLOP; product 1
// at 3.1 PFLOP/s).
#include <algorithm>
#include <cstring>

#include "internal.h"
#include "moe.h"
#include "mxfp8_math.cuh"
#include "ptx.cuh"

namespace mxfp4 {

__device__ int g_moe_error;

namespace {

constexpr int kMaxExperts = 512;
constexpr int kPlaceThreads = 1024;
constexpr int kPerThread = 8;
constexpr int kChunk = kPlaceThreads * kPerThread;   // choices a placing block takes

// ------------------------------------------------------------------ placing

struct PlaceParams {
    const int32_t *ids;
    int *hist;      // [chunks][E], more than one chunk only
    int *tiles;     // token tiles of all experts
    int4 *rec;      // [tiles] expert, first sorted row, rows of a token tile (a 16-byte load; the fourth word is 0)
    int *src;       // [R] token of a sorted row
    int *pos;       // [R] sorted row of a choice, -1: left out
    int R, k, E, chunks, nt;
};

__global__ void __launch_bounds__(kPlaceThreads) moe_count_kernel(const PlaceParams p)
{
    __shared__ int cnt[kMaxExperts];
    grid_dependency_wait();
    grid_launch_dependents();
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) cnt[e] = 0;
    __syncthreads();
    const int begin = blockIdx.x * kChunk;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int c = begin + i * kPlaceThreads + threadIdx.x;
        if (c < p.R) {
            const int e = p.ids[c];
            if (e >= 0 && e < p.E) atomicAdd(&cnt[e], 1);
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) p.hist[static_cast<size_t>(blockIdx.x) * p.E + e] = cnt[e];
}

__global__ void __launch_bounds__(kPlaceThreads) moe_place_kernel(const PlaceParams p)
{
    __shared__ int total[kMaxExperts];    // rows of an expert
    __shared__ int next[kMaxExperts];     // rows of it before this block's; then the next free row
    __shared__ int off[kMaxExperts];
    __shared__ int tile0[kMaxExperts];
    grid_dependency_wait();
    grid_launch_dependents();
    const int tid = threadIdx.x, begin = blockIdx.x * kChunk;
    int mine[kPerThread];
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int c = begin + i * kPlaceThreads + tid;
        const int e = c < p.R ? p.ids[c] : -1;
        mine[i] = e >= 0 && e < p.E ? e : -1;
    }
    if (p.chunks == 1) {
        for (int e = tid; e < p.E; e += blockDim.x) total[e] = next[e] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kPerThread; ++i)
            if (mine[i] >= 0) atomicAdd(&total[mine[i]], 1);
    } else {
        for (int e = tid; e < p.E; e += blockDim.x) {
            int all = 0, before = 0;
            for (int c = 0; c < p.chunks; ++c) {
                const int n = p.hist[static_cast<size_t>(c) * p.E + e];
                all += n;
                if (c < static_cast<int>(blockIdx.x)) before += n;
            }
            total[e] = all;
            next[e] = before;
        }
    }
    __syncthreads();
    if (tid < 32) {
        // prefix sums of rows and tiles: lane l takes experts [l * per, (l + 1) * per)
        const int per = (p.E + 31) / 32;
        int rows = 0, tiles = 0;
        for (int i = 0; i < per; ++i) {
            const int e = tid * per + i;
            if (e < p.E) {
                rows += total[e];
                tiles += (total[e] + p.nt - 1) / p.nt;
            }
        }
        int r0 = rows, t0 = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int a = __shfl_up_sync(0xffffffffu, r0, o), b = __shfl_up_sync(0xffffffffu, t0, o);
            if (tid >= o) {
                r0 += a;
                t0 += b;
            }
        }
        const int all_tiles = __shfl_sync(0xffffffffu, t0, 31);
        r0 -= rows;
        t0 -= tiles;
        for (int i = 0; i < per; ++i) {
            const int e = tid * per + i;
            if (e < p.E) {
                off[e] = r0;
                tile0[e] = t0;
                r0 += total[e];
                t0 += (total[e] + p.nt - 1) / p.nt;
            }
        }
        if (tid == 0 && blockIdx.x == 0) *p.tiles = all_tiles;
    }
    __syncthreads();
    for (int e = tid; e < p.E; e += blockDim.x) {
        next[e] += off[e];
        if (blockIdx.x == 0)
            for (int i = 0; i * p.nt < total[e]; ++i)
                p.rec[tile0[e] + i] = make_int4(e, off[e] + i * p.nt, min(p.nt, total[e] - i * p.nt), 0);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int c = begin + i * kPlaceThreads + tid;
        if (c < p.R) {
            int r = -1;
            if (mine[i] >= 0) {
                r = atomicAdd(&next[mine[i]], 1);
                p.src[r] = c / p.k;
            }
            p.pos[c] = r;
        }
    }
}

// ----------------------------------------------------------------- products

struct ProductParams {
    CUtensorMap tm_w;       // packed weights [E * rows, K / 2] u8, box 128 bytes x 64 rows
    CUtensorMap tm_t;       // large tiles: token rows [R, K] u8, box 128 bytes x kLargeNT / 2 rows
    CUtensorMap tm_tsf;     // large tiles: their scales [tiles * K / 128 * 2] blocks of 128 u32, box two blocks
    const uint8_t *w_sf;    // blocked weight scales, one buffer an expert
    const uint8_t *x;       // product 1: Xq, rows ldx bytes apart
    int64_t ldx;
    const uint8_t *x_sf;    // product 1: blocked scales of Xq
    uint8_t *act;           // [rows, I] E4M3 (product 1 writes, product 2 reads through tm_t)
    uint8_t *act_sf;        // [tiles][I / 128][NT / 128 rounded up][512]
    float *y;               // product 2: [rows, H]
    const int *tiles, *src;
    const int4 *rec;
    int H, I;
    uint64_t wait_ns;
};

// One unit of work: a tile of weight rows (index m) x one token tile of an expert.
struct Unit {
    int e, m, tile, row0, rows;
};

__device__ __forceinline__ void epilogue_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// --------------------------------------------------- products, few tokens
//
// Up to kSmallNT tokens a tile: what counts is the stream of weights from HBM. A
// stage is 128 weight rows x 256 elements of K. Three rings of shared memory:
//   packed  the weights as they lie in memory (16 KB), by TMA: the bytes in flight
//   wide    the same, widened to the form the tensor core takes (16 codes and 8
//           unused bytes in each 16; 32 KB)
//   token   token rows and all scales, gathered by cp.async: deep enough for their
//           latency (with three stages, those took 1350 clocks each)
// A stage costs every role some hundred clocks of waits, fences and issues, against
// 740 clocks that its 16 KB take at the HBM's rate: so two groups widen, two
// warps copy scales and two warps issue MMAs, on alternating stages (the two
// issuers into accumulators of their own, which the epilogue adds).

constexpr int kSmallNT = 32;
constexpr int kSmallThreads = 672;

constexpr int kEpiLd = 132;                       // floats of a staged column
constexpr uint32_t kEpiBytes = 16 * kEpiLd * 4;

struct SmallCfg {
    static constexpr int PACKED = 4, WIDE = 3, TOKEN = 5;
    static constexpr uint32_t PACKED_BYTES = 128 * 128;
    static constexpr uint32_t WIDE_BYTES = 2 * 128 * 128;          // two halves of 128 elements
    static constexpr uint32_t SFW_OFF = 2 * kSmallNT * 128;        // two halves of token rows, then two 512-byte blocks
    static constexpr uint32_t SFT_OFF = SFW_OFF + 1024;            // two 512-byte blocks
    static constexpr uint32_t TOKEN_BYTES = SFT_OFF + 1024;
    static constexpr uint32_t WIDE_AT = PACKED * PACKED_BYTES;
    static constexpr uint32_t TOKEN_AT = WIDE_AT + WIDE * WIDE_BYTES;
    static constexpr uint32_t EPI_AT = TOKEN_AT + TOKEN * TOKEN_BYTES;
    static constexpr uint32_t BAR_AT = EPI_AT + kEpiBytes;
    static constexpr int BARS = 2 * PACKED + 3 * TOKEN + 8;
    static constexpr uint32_t SMEM_BYTES = BAR_AT + BARS * 8 + 32 + 1024;
    static constexpr uint32_t SF_COLS = 16;                        // two blocks of weights, two of tokens, 4 columns each
    static constexpr uint32_t ACC_COLS = 4 * kSmallNT;             // [buffer][issuer]
    static constexpr uint32_t TMEM_COLS = 256;
    static_assert(TOKEN_BYTES % 1024 == 0 && SMEM_BYTES <= 232448, "shared memory budget");
    static_assert(PACKED % 2 == 0 && WIDE == 3 && TOKEN == 5, "what the waits' parities rest on");
    static_assert(WIDE <= TOKEN, "the wide ring is freed by the token ring's barriers");
    static_assert(ACC_COLS + TOKEN * SF_COLS <= TMEM_COLS, "TMEM budget");
};

// Slot (i mod N) of a ring of N and the parity of its i / N-th round.
struct Ring {
    int slot;
    uint32_t parity;
};
template <int N>
__device__ __forceinline__ Ring ring_at(int i)
{
    return Ring{i % N, static_cast<uint32_t>(i / N) & 1u};
}

// Stores the 32 accumulator columns (tokens) v of one weight row (channel) a thread:
// product 2 as it is, from registers; product 1 as MXFP8 of silu(g) * u, staged 16
// columns at a time through shared memory so that a thread gets neighbouring
// channels of one token. Called by the 128 epilogue threads; c0: first column,
// below w.rows.
template <bool FIRST>
__device__ __forceinline__ void store_columns(const uint32_t (&v)[32], float *epi, const Unit &w, int c0, int ntb,
                                              const ProductParams &p)
{
    const int t = threadIdx.x & 127;
    if constexpr (!FIRST) {
        // neighbouring lanes hold neighbouring channels: a warp stores 128 bytes of a token
        float *o = p.y + (static_cast<size_t>(w.row0) + c0) * p.H + 128 * w.m + t;
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (c0 + j < w.rows) o[static_cast<size_t>(j) * p.H] = __uint_as_float(v[j]);
        return;
    }
    const int col = t >> 3, part = t & 7;      // this thread's column and eighth of the staged rows
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
        if (c0 + 16 * pass >= w.rows) break;
#pragma unroll
        for (int j = 0; j < 16; ++j) epi[j * kEpiLd + t] = __uint_as_float(v[16 * pass + j]);
        epilogue_sync();
        const int r = c0 + 16 * pass + col;    // row of the tile
        const bool live = r < w.rows;
        const size_t row = static_cast<size_t>(w.row0) + r;
        // 8 channels a thread; four neighbours share a block of 32. silu by __expf and
        // __fdividef: off by up to (5 + 1.2 |g|) 2^-23 of itself, and 0 below -87.3 where
        // its size is under 2^-118; E4M3 keeps 2^-4, so this moves a code only next to a
        // midpoint, as the products' own fp32 sums do. expf and an IEEE division were
        // measured: 16 tokens 55 -> 64 us, 1111 ragged 105 -> 122, the others 1 to 4 %.
        const float *g = epi + col * kEpiLd + 8 * part;
        float a[8];
        uint32_t amax = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 gv = *reinterpret_cast<const float4 *>(g + 4 * i);
            const float4 uv = *reinterpret_cast<const float4 *>(g + 64 + 4 * i);
            a[4 * i] = __fdividef(gv.x, 1.0f + __expf(-gv.x)) * uv.x;
            a[4 * i + 1] = __fdividef(gv.y, 1.0f + __expf(-gv.y)) * uv.y;
            a[4 * i + 2] = __fdividef(gv.z, 1.0f + __expf(-gv.z)) * uv.z;
            a[4 * i + 3] = __fdividef(gv.w, 1.0f + __expf(-gv.w)) * uv.w;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(a[i]) & 0x7FFFFFFFu);
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const uint32_t b = mxfp8_scale_byte(amax);
        const float inv = mxfp8_scale_inverse(b);
        const uint32_t b2 = __shfl_down_sync(0xffffffffu, b, 4);
        if (live) {
            uint2 c;
            c.x = e4m3x4_rn(a[0] * inv, a[1] * inv, a[2] * inv, a[3] * inv);
            c.y = e4m3x4_rn(a[4] * inv, a[5] * inv, a[6] * inv, a[7] * inv);
            *reinterpret_cast<uint2 *>(p.act + row * p.I + 64 * w.m + 8 * part) = c;
            if (part == 0) {
                uint8_t *sf = p.act_sf + (static_cast<size_t>(w.tile) * (p.I >> 7) + (w.m >> 1)) * (ntb * 512) +
                              (r >> 7) * 512 + (r & 31) * 16 + ((r & 127) >> 5) * 4 + (w.m & 1) * 2;
                *reinterpret_cast<uint16_t *>(sf) = static_cast<uint16_t>(b | (b2 << 8));
            }
        }
        epilogue_sync();   // the staging buffer is reused
    }
}

// Walks the units first, first + step, ... of `tiles` token tiles x mw weight tiles:
// GROUP token tiles (all of them if 0) for one weight tile after another. Tiles of
// one expert are neighbours, so those at work on the same weights read them from
// L2, and a group's tokens stay there too. The record of the next unit is on its
// way while the current one is worked on.
template <int GROUP>
struct UnitWalk {
    const int4 *rec;
    int tiles, mw, units, u, step;
    int next_tile, next_m;
    int4 next;
    __device__ __forceinline__ UnitWalk(const ProductParams &p, int tiles_, int mw_, int first, int step_)
        : rec(p.rec), tiles(tiles_), mw(mw_), units(tiles_ * mw_), u(first), step(step_)
    {
        fetch();
    }
    __device__ __forceinline__ void fetch()
    {
        if (u >= units) return;
        if constexpr (GROUP == 0) {
            next_m = u / tiles;
            next_tile = u - next_m * tiles;
        } else {
            const int g = u / (GROUP * mw), local = u - g * (GROUP * mw);
            const int n = min(GROUP, tiles - g * GROUP);   // the last group may be smaller
            next_m = local / n;
            next_tile = g * GROUP + local - next_m * n;
        }
        next = __ldcg(rec + next_tile);
    }
    __device__ __forceinline__ bool more() const { return u < units; }
    // units that are left for this walker
    __device__ __forceinline__ int left() const { return u < units ? (units - u + step - 1) / step : 0; }
    __device__ __forceinline__ Unit take()
    {
        const Unit w{next.x, next_m, next_tile, next.y, next.z};
        u += step;
        fetch();
        return w;
    }
};

// FIRST: product 1 (tokens x [G; U], SwiGLU, MXFP8), else product 2. Warps:
//   0-3    epilogue of a finished tile while the next one's mainloop runs
//   4-7    copy token rows and all scales by cp.async
//   8-15   widen packed weights: groups of four on alternating stages
//   16,17  MMA issuers (an elected lane), on alternating stages of a tile; 16 owns TMEM
//   18     lane 0 loads packed weights by TMA
//   19,20  copy the scales of alternating stages to TMEM (an elected lane)
//
// A wait on a ring's barrier names the round by its parity alone, so it is right only
// if the barrier can be neither a round further nor a round behind. What makes it so
// here: a packed slot belongs to one group (PACKED is even); tokens are copied in
// order; a stage is widened only after the MMAs of the stage WIDE = 3 before it, and
// its group and its scale thread have served stage i - 2 before: so who has seen stage
// i - 2 ready knows that i - 5, whose slot it shares, was multiplied. A third group
// breaks this: a stage could then be two ahead of a slow one, and the waits fail.
// Loading weights already widened was measured too: a TMA load that unpacks moves 16
// bytes of shared memory a clock, 8-byte cp.async half of what HBM gives.
template <bool FIRST>
__global__ void __launch_bounds__(kSmallThreads, 1) moe_product_small_kernel(const __grid_constant__ ProductParams p)
{
    using Cfg = SmallCfg;
    constexpr int PACKED = Cfg::PACKED, WIDE = Cfg::WIDE, TOKEN = Cfg::TOKEN, NT = kSmallNT;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *epi = reinterpret_cast<float *>(smem + Cfg::EPI_AT);
    uint64_t *p_full = reinterpret_cast<uint64_t *>(smem + Cfg::BAR_AT);
    uint64_t *p_empty = p_full + PACKED;
    uint64_t *t_full = p_empty + PACKED;   // tokens and scales of a stage have landed
    uint64_t *ready = t_full + TOKEN;      // [TOKEN] weights widened, scales in TMEM
    uint64_t *done = ready + TOKEN;        // [TOKEN] the stage's MMAs have completed: its token and wide slots are free
    uint64_t *accf = done + TOKEN;         // [2] accumulators complete
    uint64_t *acc_empty = accf + 2;        // [2] accumulators drained
    uint64_t *cp_done = acc_empty + 2;     // [2] the scale copies of warp 19 / 20 have completed
    uint64_t *mma_done = cp_done + 2;      // [2] the MMAs of each issuer have completed
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mma_done + 2);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    volatile int *epi_go = abort_flag + 1;   // [2]

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < PACKED; ++i) {
            mbar_init(p_full + i, 1);
            mbar_init(p_empty + i, 4);      // one arrival from each warp of a widening group
        }
        for (int i = 0; i < TOKEN; ++i) {
            mbar_init(t_full + i, 128);     // one from each copying thread
            mbar_init(ready + i, 5);        // a widening group's warps and the scale copies
            mbar_init(done + i, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accf + b, 2);         // both issuers
            mbar_init(acc_empty + b, 128);
            mbar_init(cp_done + b, 1);
            mbar_init(mma_done + b, 1);
        }
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&p.tm_w);
    }
    if (warp == 16) {
        tmem_alloc(tmem_slot, Cfg::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // Product 2 starts while product 1 drains, and loads weights meanwhile: product 1
    // let it start only after everything before it had completed, so the tables of the
    // placing kernel and the weights are there; only the activations are not. (Asking L2
    // for more of the weights than the ring holds was measured slower.)
    if (FIRST) grid_dependency_wait();
    grid_launch_dependents();
    const int tiles = __ldcg(p.tiles);
    const int K = FIRST ? p.H : p.I;
    const int kc = K >> 7;                                  // blocks of 128 elements
    const int stages = (kc + 1) >> 1;                       // the last one may be half
    const int mw = FIRST ? p.I >> 6 : p.H >> 7;             // weight tiles of an expert
    const int wrows = FIRST ? 2 * p.I : p.H;                // weight rows of an expert
    // uniform across the warp, for the issuers of MMAs and scale copies
    const uint32_t tmem_u = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t wide_desc = sdesc_sw128(smem_u32(smem + Cfg::WIDE_AT));
    const uint64_t token_desc = sdesc_sw128(smem_u32(smem + Cfg::TOKEN_AT));
    UnitWalk<0> walk(p, tiles, mw, blockIdx.x, gridDim.x);

    if (warp < 4) {
        // ------------------------------------------------------------ epilogue
        int ul = 0;
        for (; walk.more(); ++ul) {
            const Unit w = walk.take();
            const int buf = ul & 1;
            if (threadIdx.x == 0) {
                const bool ok = mbar_wait(accf + buf, (ul >> 1) & 1, &g_moe_error, kErrWaitAccum, p.wait_ns);
                if (!ok) *abort_flag = 1;
                epi_go[buf] = ok && !*abort_flag;
            }
            epilogue_sync();
            if (!epi_go[buf]) break;
            tc_fence_after();
            const uint32_t trow = tmem + buf * 2 * NT + (static_cast<uint32_t>(warp * 32) << 16);
            uint32_t v[32];
            tmem_ld32(trow, v);
            tmem_ld_wait();
            if (stages > 1) {
                uint32_t v1[32];
                tmem_ld32(trow + NT, v1);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) + __uint_as_float(v1[j]));
            }
            tc_fence_before();
            mbar_arrive(acc_empty + buf);
            store_columns<FIRST>(v, epi, w, 0, 1, p);
        }
    } else if (warp < 8) {
        // -------------------------------------------------- tokens and scales
        // Thread t copies 16 bytes (column t % 8 of each half) of rows t / 8 and
        // t / 8 + 16; in the 128-byte swizzle column c of row r is at c ^ (r % 8).
        const int t = threadIdx.x - 128;
        const int r0 = t >> 3, c = t & 7;
        const uint32_t dst0 = r0 * 128 + ((c ^ (r0 & 7)) << 4);
        if (!FIRST) grid_dependency_wait();
        int gs = 0;
        bool ok = true;
        while (walk.more() && ok) {
            const Unit w = walk.take();
            // this thread's rows; what lies past the tile's last row is left as it is (its
            // columns are not stored)
            const bool one = r0 < w.rows, two = r0 + 16 < w.rows;
            const uint8_t *tok[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = w.row0 + min(r0 + 16 * i, w.rows - 1);
                tok[i] = (FIRST ? p.x + static_cast<size_t>(__ldcg(p.src + r)) * p.ldx
                                : p.act + static_cast<size_t>(r) * p.I) + c * 16;
            }
            // scales: thread t < 64 those of the weights, of product 1 from the half of the
            // 128-row blocks of G and of U that holds its 64 channels (8 of each 16
            // bytes), 64 <= t < 96 a word a token
            const uint8_t *sf = nullptr;
            uint32_t sf_dst = 0;
            if (t < 64) {
                if constexpr (FIRST) {
                    const size_t blk = static_cast<size_t>(wrows >> 7) * w.e + (w.m >> 1) + (t >= 32 ? p.I >> 7 : 0);
                    sf = p.w_sf + blk * kc * 512 + lane * 16 + (w.m & 1) * 8;
                    sf_dst = Cfg::SFW_OFF + lane * 16 + (t >= 32 ? 8 : 0);
                } else {
                    sf = p.w_sf + static_cast<size_t>(w.e * mw + w.m) * kc * 512 + (t & 31) * 16;
                    sf_dst = Cfg::SFW_OFF + (t & 31) * 16;
                }
            } else if (t < 96 && lane < w.rows) {
                const int r = lane;
                if constexpr (FIRST) {
                    const int tk = __ldcg(p.src + w.row0 + r);
                    sf = p.x_sf + static_cast<size_t>(tk >> 7) * kc * 512 + (tk & 31) * 16 + ((tk & 127) >> 5) * 4;
                } else {
                    sf = p.act_sf + static_cast<size_t>(w.tile) * kc * 512 + r * 16;
                }
                sf_dst = Cfg::SFT_OFF + lane * 16;
            }
            for (int ks = 0; ks < stages; ++ks, ++gs) {
                const Ring r = ring_at<TOKEN>(gs);
                if (gs >= TOKEN) ok = mbar_wait_warp(done + r.slot, r.parity ^ 1u, &g_moe_error, kErrWaitEmpty, p.wait_ns);
                if (!ok) {
                    *abort_flag = 1;
                    break;
                }
                const uint32_t st = smem_u32(smem + Cfg::TOKEN_AT) + r.slot * Cfg::TOKEN_BYTES;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int kb = 2 * ks + h;
                    if (kb < kc) {
                        if (one) cp_async<16>(st + dst0 + h * (NT * 128), tok[0] + kb * 128);
                        if (two) cp_async<16>(st + dst0 + h * (NT * 128) + 2048, tok[1] + kb * 128);
                        if (t < 64) {
                            if constexpr (FIRST)
                                cp_async<8>(st + sf_dst + h * 512, sf + kb * 512);
                            else if (t < 32)
                                cp_async<16>(st + sf_dst + h * 512, sf + kb * 512);
                        } else if (t < 96 && lane < w.rows) {
                            cp_async<4>(st + sf_dst + h * 512, sf + kb * 512);
                        }
                    }
                }
                cp_async_arrive(t_full + r.slot);
            }
        }
        cp_async_wait_all();   // also after an abort: nothing of this thread is in flight when the block leaves
        // nor are the arrivals of the last MMAs, which nobody else waits for
        for (int i = max(0, gs - TOKEN); i < gs && ok; ++i) {
            const Ring r = ring_at<TOKEN>(i);
            ok = mbar_wait_warp(done + r.slot, r.parity, &g_moe_error, kErrWaitDrain);
        }
    } else if (warp < 16) {
        // -------------------------------------------------- widening of weights
        // Lane l takes row l % 8 of a group of eight and 16-byte column l / 8 (+ 4): both
        // swizzles then spread eight lanes over all banks.
        const int group = (warp - 8) >> 2, w4 = (warp - 8) & 3;
        const int row8 = lane & 7, j = lane >> 3;
        bool ok = true;
        const int total = walk.left() * stages;
        for (int gs = group; gs < total; gs += 2) {
                const Ring rp = ring_at<PACKED>(gs);
                ok = mbar_wait_warp(p_full + rp.slot, rp.parity, &g_moe_error, kErrWaitFull, p.wait_ns);
                if (!ok) break;
                const uint8_t *src = smem + rp.slot * Cfg::PACKED_BYTES + w4 * 4096 + row8 * 128;
                uint4 v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = *reinterpret_cast<const uint4 *>(src + (i & 3) * 1024 + ((((i >> 2) * 4 + j) ^ row8) << 4));
                if (gs >= WIDE) {
                    // this barrier cannot complete another round before the stage at
                    // hand has been multiplied (WIDE <= TOKEN)
                    const Ring rd = ring_at<TOKEN>(gs - WIDE);
                    ok = mbar_wait_warp(done + rd.slot, rd.parity, &g_moe_error, kErrWaitEmpty, p.wait_ns);
                    if (!ok) break;
                }
                uint8_t *dst = smem + Cfg::WIDE_AT + (gs % WIDE) * Cfg::WIDE_BYTES + w4 * 4096 + row8 * 128;
                const int s0 = ((2 * j) ^ row8) << 4, s1 = ((2 * j + 1) ^ row8) << 4;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint8_t *d = dst + (i >> 2) * 16384 + (i & 3) * 1024;
                    *reinterpret_cast<uint2 *>(d + s0) = make_uint2(v[i].x, v[i].y);
                    *reinterpret_cast<uint2 *>(d + s1) = make_uint2(v[i].z, v[i].w);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(ready + gs % TOKEN);
                    // Only now: the stores needed the values. Released right after the loads,
                    // the slot was refilled before some had been executed (the compiler
                    // sinks them to the stores).
                    mbar_arrive(p_empty + rp.slot);
                }
        }
        if (!ok) *abort_flag = 1;
    } else if (warp < 18) {
        // ---------------------------------------------------------- MMA issuers
        // Whole warps walk the stages and one elected lane issues, so that descriptors
        // stay in uniform registers.
        const int me = warp - 16;
        int gs = 0, ul = 0;
        bool ok = true;
        for (; walk.more() && ok; ++ul) {
            const Unit w = walk.take();
            const int buf = ul & 1;
            if (ul >= 2)
                ok = mbar_wait_warp(acc_empty + buf, ((ul >> 1) - 1) & 1, &g_moe_error, kErrWaitAccum, p.wait_ns);
            if (!ok) break;
            tc_fence_after();
            const uint32_t idesc = __shfl_sync(0xffffffffu, idesc_w4a8((w.rows + 15) & ~15), 0);
            const uint32_t d = tmem_u + (buf * 2 + me) * NT;
            for (int ks = me; ks < stages; ks += 2) {
                const Ring r = ring_at<TOKEN>(gs + ks);
                ok = mbar_wait_warp(ready + r.slot, r.parity, &g_moe_error, kErrWaitOperand, p.wait_ns);
                if (!ok) break;
                tc_fence_after();
                const uint32_t tsf = tmem_u + Cfg::ACC_COLS + r.slot * Cfg::SF_COLS;
                const uint64_t ad = wide_desc + static_cast<uint64_t>((gs + ks) % WIDE * (Cfg::WIDE_BYTES >> 4));
                const uint64_t bd = token_desc + static_cast<uint64_t>(r.slot * (Cfg::TOKEN_BYTES >> 4));
                if (elect_one()) {
                    auto half = [&](int h, uint32_t accumulate) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_mxf8f6f4(d, ad + h * 1024 + 2 * kk, bd + h * (NT * 8) + 2 * kk,
                                         idesc_with_sf_ids(idesc, kk, kk), tsf + 4 * h, tsf + 8 + 4 * h,
                                         kk > 0 ? 1u : accumulate);
                    };
                    half(0, ks > me ? 1u : 0u);
                    if (2 * ks + 1 < kc) half(1, 1u);
                    tc_commit(done + r.slot);
                }
                __syncwarp();
            }
            gs += stages;
            if (elect_one()) tc_commit(accf + buf);
            __syncwarp();
        }
        if (!ok) *abort_flag = 1;
        // no MMA may be running when TMEM is released
        if (elect_one()) tc_commit(mma_done + me);
        __syncwarp();
        mbar_wait_warp(mma_done + me, 0, &g_moe_error, kErrWaitDrain);
    } else if (warp == 18) {
        if (lane == 0) {
            // --------------------------------------------- packed weights by TMA
            const uint64_t pol = policy_evict_first();
            int gs = 0;
            bool ok = true;
            while (walk.more() && ok && !*abort_flag) {
                const Unit w = walk.take();
                // the two halves of the tile: G and U of 64 channels, or 128 rows in a row
                const int r0 = w.e * wrows + w.m * (FIRST ? 64 : 128);
                const int r1 = r0 + (FIRST ? p.I : 64);
                for (int ks = 0; ks < stages; ++ks) {
                    const Ring r = ring_at<PACKED>(gs);
                    if (gs >= PACKED &&
                        !(ok = mbar_wait(p_empty + r.slot, r.parity ^ 1u, &g_moe_error, kErrWaitEmpty, p.wait_ns))) {
                        *abort_flag = 1;
                        break;
                    }
                    uint8_t *st = smem + r.slot * Cfg::PACKED_BYTES;
                    mbar_arrive_expect_tx(p_full + r.slot, Cfg::PACKED_BYTES);
                    tma_load_2d(st, &p.tm_w, ks * 128, r0, p_full + r.slot, pol);
                    tma_load_2d(st + 8192, &p.tm_w, ks * 128, r1, p_full + r.slot, pol);
                    ++gs;
                    if (ks == min(PACKED, stages) - 1 && walk.more()) {
                        // the weight scales of the next unit go to L2 ahead of their copies (of
                        // product 1 two runs of blocks, which two units share)
                        const size_t blk = static_cast<size_t>(wrows >> 7) * walk.next.x + walk.next_m / (FIRST ? 2 : 1);
                        prefetch_l2_bulk(p.w_sf + blk * kc * 512, kc * 512);
                        if (FIRST) prefetch_l2_bulk(p.w_sf + (blk + (p.I >> 7)) * kc * 512, kc * 512);
                    }
                }
            }
            // copies in flight land before the block leaves
            for (int i = max(0, gs - PACKED); i < gs; ++i) {
                const Ring r = ring_at<PACKED>(i);
                mbar_wait(p_full + r.slot, r.parity, &g_moe_error, kErrWaitDrain);
            }
        }
    } else {
        // ------------------------------------------------------ scales to TMEM
        // cp.async wrote the stage through the generic proxy; the fence here lets the
        // scale copies, and the MMAs that wait for them, read it through the async
        // proxy.
        const int me = warp - 19, total = walk.left() * stages;
        const uint64_t sf_desc = sdesc_scale(smem_u32(smem + Cfg::TOKEN_AT + Cfg::SFW_OFF));
        int ks = 0;                    // stage of the tile: the last one may be half
        bool ok = true;
        for (int gs = 0; gs < total; ++gs, ks = ks + 1 == stages ? 0 : ks + 1) {
            if ((gs & 1) != me) continue;
            const Ring r = ring_at<TOKEN>(gs);
            ok = mbar_wait_warp(t_full + r.slot, r.parity, &g_moe_error, kErrWaitFull, p.wait_ns);
            if (!ok) break;
            fence_proxy_async_smem();
            tc_fence_after();
            const uint64_t sd = sf_desc + static_cast<uint64_t>(r.slot * (Cfg::TOKEN_BYTES >> 4));
            const uint32_t tsf = tmem_u + Cfg::ACC_COLS + r.slot * Cfg::SF_COLS;
            if (elect_one()) {
                tc_cp_scale_block(tsf, sd);
                tc_cp_scale_block(tsf + 8, sd + 64);
                if (2 * ks + 1 < kc) {
                    tc_cp_scale_block(tsf + 4, sd + 32);
                    tc_cp_scale_block(tsf + 12, sd + 96);
                }
                tc_commit(ready + r.slot);
            }
            __syncwarp();
        }
        if (!ok) *abort_flag = 1;
        // no copy may be running when TMEM is released
        if (elect_one()) tc_commit(cp_done + me);
        __syncwarp();
        mbar_wait_warp(cp_done + me, 0, &g_moe_error, kErrWaitDrain);
    }
    __syncwarp();

    tc_fence_before();
    __syncthreads();
    if (warp == 16) {
        tc_fence_after();
        tmem_dealloc(tmem, Cfg::TMEM_COLS);
    }
}

// --------------------------------------------------- products, many tokens
//
// Tiles of 256 weight rows x up to kLargeNT tokens on CTA pairs (cta_group::2): each
// CTA holds 128 of the weight rows and half of the tokens, so an SM takes in 16 KB of
// widened weights and 14 KB of tokens for 448 clocks of MMA a stage of 128 elements.
// What bounds a stage is shared memory (128 bytes a clock): packed weights in 64
// clocks, read again 64, widened 128, tokens 112, read by the MMAs 128 + 112, together
// 608. (A single CTA's tile of 128 x 224 needs 832.) Token rows come by TMA, which
// wants them in sorted order: moe_gather_kernel copies them there. (Gathered by
// cp.async instead, 28 KB a stage took 900 clocks.)

constexpr int kLargeNT = kMoeLargeTile;
constexpr int kLargeGroups = 3;                    // widening groups of four warps
constexpr int kLargeThreads = 32 * (8 + 4 * kLargeGroups);

struct LargeCfg {
    static constexpr int PACKED = 3, OPER = 5;
    static constexpr int HALF = kLargeNT / 2;                        // token rows of a CTA
    static constexpr uint32_t PSF_OFF = 128 * 128;                   // packed stage: 256 elements of 128 rows, then scales
    static constexpr uint32_t PACKED_BYTES = PSF_OFF + 2048;         // of G and of U, or of 128 rows: 2 x 2 blocks
    static constexpr uint32_t WSF_OFF = 128 * 128;                   // widened stage: 128 elements, then their block of scales
    static constexpr uint32_t WIDE_BYTES = WSF_OFF + 1024;
    static constexpr uint32_t TSF_OFF = HALF * 128;                  // token stage: 128 elements, then two blocks of scales
    static constexpr uint32_t TOKEN_BYTES = TSF_OFF + 1024;
    static constexpr uint32_t WIDE_AT = PACKED * PACKED_BYTES;
    static constexpr uint32_t TOKEN_AT = WIDE_AT + OPER * WIDE_BYTES;
    static constexpr uint32_t EPI_AT = TOKEN_AT + OPER * TOKEN_BYTES;
    static constexpr uint32_t BAR_AT = EPI_AT + kEpiBytes;
    static constexpr int BARS = 2 * PACKED + 4 * OPER + 6;
    static constexpr uint32_t SMEM_BYTES = BAR_AT + BARS * 8 + 32 + 1024;
    static constexpr uint32_t SF_COLS = 12;                          // a block of weights, two of tokens
    static constexpr uint32_t TMEM_COLS = 512;
    static_assert(PACKED_BYTES % 1024 == 0 && WIDE_BYTES % 1024 == 0 && TOKEN_BYTES % 1024 == 0, "swizzle atoms");
    static_assert(SMEM_BYTES <= 232448, "shared memory budget");
    static_assert(2 * kLargeNT + OPER * SF_COLS <= TMEM_COLS, "TMEM budget");
    static_assert(PACKED == kLargeGroups, "a packed slot belongs to one group");
    static_assert(HALF % 16 == 0, "halves of a tile are MMA operands");
};

// FIRST: product 1 (a pair's tile: 128 channels of G and of U, 64 of each in a CTA),
// else product 2 (256 rows). Warps of each CTA:
//   0-3    epilogue of the CTA's 128 weight rows
//   4-15   widen packed weights: three groups of four take the packed stages in turn
//          (a group's two stages take it about 2700 clocks of waits, copies and
//          fences); they also see the tokens land, and tell rank 0
//   16     owns TMEM; rank 0: issues the MMAs (an elected lane)
//   17     lane 0 loads packed weights and their scales by TMA
//   18     lane 0 loads tokens and their scales by TMA
//   19     rank 0: copies the scales to both TMEMs, stage by stage (an elected lane)
//
// A wait on a ring's barrier names the round by its parity alone, so it is right only
// if the barrier can be neither a round further nor a round behind. Not behind:
// a packed slot belongs to one group (PACKED = groups); a group that waits for `done`
// of stage i - OPER has seen that of i - 2 OPER or a later one, and MMAs complete in
// order; one warp waits for `ready`, of every stage in order (two that took turns
// could find a stage's slot still in the round before: groups finish out of order).
// Not further: a stage's next round needs its MMAs, and so all who wait for it.
template <bool FIRST>
__global__ void __launch_bounds__(kLargeThreads, 1) moe_product_large_kernel(const __grid_constant__ ProductParams p)
{
    using Cfg = LargeCfg;
    constexpr int PACKED = Cfg::PACKED, OPER = Cfg::OPER, NT = kLargeNT;
    constexpr int kMmaWarp = 4 + 4 * kLargeGroups;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *epi = reinterpret_cast<float *>(smem + Cfg::EPI_AT);
    uint64_t *p_full = reinterpret_cast<uint64_t *>(smem + Cfg::BAR_AT);
    uint64_t *p_empty = p_full + PACKED;
    uint64_t *t_full = p_empty + PACKED;
    uint64_t *ready = t_full + OPER;       // rank 0: both CTAs' operands of a stage are in shared memory
    uint64_t *s_full = ready + OPER;       // rank 0: its scales are in both TMEMs
    uint64_t *done = s_full + OPER;        // its MMAs have completed
    uint64_t *accf = done + OPER;          // [2] accumulators complete
    uint64_t *acc_empty = accf + 2;        // [2] rank 0: both CTAs have drained them
    uint64_t *cp_done = acc_empty + 2;     // rank 0: the scale copies have completed
    uint64_t *mma_done = cp_done + 1;      // all MMAs have completed
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mma_done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    volatile int *epi_go = abort_flag + 1;   // [2]

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    const bool leader = rank == 0;
    if (threadIdx.x == 0) {
        for (int i = 0; i < PACKED; ++i) {
            mbar_init(p_full + i, 1);
            mbar_init(p_empty + i, 4);      // one arrival from each warp of a widening group
        }
        for (int i = 0; i < OPER; ++i) {
            mbar_init(t_full + i, 1);
            mbar_init(ready + i, 8);        // a widening group of each CTA
            mbar_init(s_full + i, 1);
            mbar_init(done + i, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accf + b, 1);
            mbar_init(acc_empty + b, 8);    // one arrival from each epilogue warp of both CTAs
        }
        mbar_init(cp_done, 1);
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&p.tm_w);
        tma_prefetch_desc(&p.tm_t);
        tma_prefetch_desc(&p.tm_tsf);
    }
    if (warp == kMmaWarp) {
        tmem_alloc_pair(tmem_slot, Cfg::TMEM_COLS);
        tmem_relinquish_pair();
    }
    // both CTAs' barriers exist before any arrival from the other CTA
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // Product 2 starts while product 1 drains, and loads weights meanwhile: product 1
    // let it start only after everything before it had completed, so the tables of the
    // placing kernel and the weights are there; only the activations are not. (Asking L2
    // for more of the weights than the ring holds was measured slower.)
    if (FIRST) grid_dependency_wait();
    grid_launch_dependents();
    const int tiles = __ldcg(p.tiles);
    const int K = FIRST ? p.H : p.I;
    const int kc = K >> 7;                                  // stages of a tile
    const int kp = (kc + 1) >> 1;                           // packed stages; the last one may be half
    const int wrows = FIRST ? 2 * p.I : p.H;                // weight rows of an expert
    const int mw = FIRST ? p.I >> 7 : (p.H + 255) >> 8;     // weight tiles of an expert
    // uniform across the warp, for the issuers of MMAs and scale copies
    const uint32_t tmem_u = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t wide_desc = sdesc_sw128(smem_u32(smem + Cfg::WIDE_AT));
    const uint64_t token_desc = sdesc_sw128(smem_u32(smem + Cfg::TOKEN_AT));
    UnitWalk<8> walk(p, tiles, mw, blockIdx.x >> 1, gridDim.x >> 1);

    if (warp < 4) {
        // ------------------------------------------------------------ epilogue
        const uint32_t acc_empty_r0 = mapa_shared(smem_u32(acc_empty), 0);
        int ul = 0;
        for (; walk.more(); ++ul) {
            Unit w = walk.take();
            const int buf = ul & 1;
            if (threadIdx.x == 0) {
                const bool ok = mbar_wait(accf + buf, (ul >> 1) & 1, &g_moe_error, kErrWaitAccum, p.wait_ns);
                if (!ok) *abort_flag = 1;
                epi_go[buf] = ok && !*abort_flag;
            }
            epilogue_sync();
            if (!epi_go[buf]) break;
            tc_fence_after();
            // this CTA's half of the tile, in units of 64 channels or 128 rows
            w.m = 2 * w.m + rank;
            const bool live = FIRST || 128 * w.m < p.H;
            const uint32_t trow = tmem + buf * NT + (static_cast<uint32_t>(warp * 32) << 16);
            for (int c0 = 0; c0 < w.rows; c0 += 32) {
                uint32_t v[32];
                tmem_ld32(trow + c0, v);
                tmem_ld_wait();
                if (c0 + 32 >= w.rows) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster_relaxed(acc_empty_r0 + buf * 8);
                }
                if (live) store_columns<FIRST>(v, epi, w, c0, 2, p);
            }
        }
    } else if (warp < kMmaWarp) {
        // -------------------------------------------------- widening of weights
        // Lane l takes row l % 8 of a group of eight and 16-byte column l / 8 of a half:
        // both swizzles then spread eight lanes over all banks.
        const int group = (warp - 4) >> 2, w4 = (warp - 4) & 3;
        const int row8 = lane & 7, j = lane >> 3;
        const uint32_t ready_r0 = mapa_shared(smem_u32(ready), 0);
        const int s0 = ((2 * j) ^ row8) << 4, s1 = ((2 * j + 1) ^ row8) << 4;
        const int n = walk.left();
        int pk = 0;
        bool ok = true;
        for (int ul = 0; ul < n && ok; ++ul)
            for (int kq = 0; kq < kp && ok; ++kq, ++pk) {
                if (pk % kLargeGroups != group) continue;
                const Ring rp = ring_at<PACKED>(pk);
                ok = mbar_wait_warp(p_full + rp.slot, rp.parity, &g_moe_error, kErrWaitFull, p.wait_ns);
                if (!ok) break;
                const uint8_t *src = smem + rp.slot * Cfg::PACKED_BYTES + w4 * 4096 + row8 * 128;
                const uint8_t *psf = smem + rp.slot * Cfg::PACKED_BYTES + Cfg::PSF_OFF + lane * 16;
                const int halves = min(2, kc - 2 * kq);
                for (int h = 0; h < halves; ++h) {
                    const int gs = ul * kc + 2 * kq + h;
                    const Ring ro = ring_at<OPER>(gs);
                    uint4 v[4], sf = make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        v[i] = *reinterpret_cast<const uint4 *>(src + i * 1024 + (((h * 4 + j) ^ row8) << 4));
                    if (w4 == 0) {
                        if constexpr (FIRST) {
                            // the half of the 128-row blocks of G and U that holds this CTA's channels
                            const uint2 g = *reinterpret_cast<const uint2 *>(psf + h * 512 + rank * 8);
                            const uint2 u = *reinterpret_cast<const uint2 *>(psf + 1024 + h * 512 + rank * 8);
                            sf = make_uint4(g.x, g.y, u.x, u.y);
                        } else {
                            sf = *reinterpret_cast<const uint4 *>(psf + h * 512);
                        }
                    }
                    if (gs >= OPER)
                        ok = mbar_wait_warp(done + ro.slot, ro.parity ^ 1u, &g_moe_error, kErrWaitEmpty, p.wait_ns);
                    if (!ok) break;
                    uint8_t *wide = smem + Cfg::WIDE_AT + ro.slot * Cfg::WIDE_BYTES;
                    uint8_t *dst = wide + w4 * 4096 + row8 * 128;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        *reinterpret_cast<uint2 *>(dst + i * 1024 + s0) = make_uint2(v[i].x, v[i].y);
                        *reinterpret_cast<uint2 *>(dst + i * 1024 + s1) = make_uint2(v[i].z, v[i].w);
                    }
                    if (w4 == 0) *reinterpret_cast<uint4 *>(wide + Cfg::WSF_OFF + lane * 16) = sf;
                    if (h + 1 == halves) {
                        // only now, when the stores have had the values (see the small tiles)
                        __syncwarp();
                        if (lane == 0) mbar_arrive(p_empty + rp.slot);
                    }
                    ok = mbar_wait_warp(t_full + ro.slot, ro.parity, &g_moe_error, kErrWaitFull, p.wait_ns);
                    if (!ok) break;
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        fence_release_own_smem_cluster();
                        mbar_arrive_cluster_relaxed(ready_r0 + ro.slot * 8);
                    }
                }
            }
        if (!ok) *abort_flag = 1;
    } else if (warp == kMmaWarp) {
        if (leader) {
            // ------------------------------------------------------- MMA issuer
            // The whole warp walks the stages and one elected lane issues, so that
            // descriptors stay in uniform registers.
            int gs = 0, ul = 0;
            bool ok = true;
            for (; walk.more() && ok; ++ul) {
                const Unit w = walk.take();
                const int buf = ul & 1;
                if (ul >= 2)
                    ok = mbar_wait_warp(acc_empty + buf, ((ul >> 1) - 1) & 1, &g_moe_error, kErrWaitAccum, p.wait_ns);
                if (!ok) break;
                tc_fence_after();
                const uint32_t idesc = __shfl_sync(0xffffffffu, idesc_w4a8((w.rows + 31) & ~31, 256), 0);
                const uint32_t d = tmem_u + buf * NT;
                for (int ks = 0; ks < kc; ++ks, ++gs) {
                    const Ring r = ring_at<OPER>(gs);
                    // s_full stands for the operands too
                    ok = mbar_wait_warp(s_full + r.slot, r.parity, &g_moe_error, kErrWaitOperand, p.wait_ns);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t ad = wide_desc + static_cast<uint64_t>(r.slot * (Cfg::WIDE_BYTES >> 4));
                    const uint64_t bd = token_desc + static_cast<uint64_t>(r.slot * (Cfg::TOKEN_BYTES >> 4));
                    const uint32_t tsf = tmem_u + 2 * NT + r.slot * Cfg::SF_COLS;
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_mxf8f6f4_pair(d, ad + 2 * kk, bd + 2 * kk, idesc_with_sf_ids(idesc, kk, kk), tsf, tsf + 4,
                                              (ks > 0 || kk > 0) ? 1u : 0u);
                        tc_commit_pair_mc(done + r.slot, 0x3);
                    }
                    __syncwarp();
                }
                if (elect_one()) tc_commit_pair_mc(accf + buf, 0x3);
                __syncwarp();
            }
            if (!ok) *abort_flag = 1;
            if (elect_one()) tc_commit_pair_mc(mma_done, 0x3);
            __syncwarp();
        }
        // no MMA may be running when the pair frees TMEM, nor an arrival of one be on its way
        mbar_wait_warp(mma_done, 0, &g_moe_error, kErrWaitDrain);
    } else if (warp == kMmaWarp + 1) {
        if (lane == 0) {
            // --------------------------------------------- packed weights by TMA
            const uint64_t pol = policy_evict_last();
            int pk = 0;
            bool ok = true;
            while (walk.more() && ok && !*abort_flag) {
                const Unit w = walk.take();
                // the two halves of this CTA's rows: G and U of 64 channels, or 128 rows in a
                // row (past the expert's last they are not stored)
                const int r0 = w.e * wrows + (FIRST ? w.m * 128 + rank * 64 : w.m * 256 + rank * 128);
                const int r1 = r0 + (FIRST ? p.I : 64);
                const size_t blk = static_cast<size_t>(wrows >> 7) * w.e +
                                   (FIRST ? w.m : min(2 * w.m + rank, (p.H >> 7) - 1));
                const uint8_t *sf0 = p.w_sf + blk * kc * 512;
                const uint8_t *sf1 = sf0 + static_cast<size_t>(p.I >> 7) * kc * 512;
                for (int kq = 0; kq < kp; ++kq, ++pk) {
                    const Ring r = ring_at<PACKED>(pk);
                    if (pk >= PACKED &&
                        !(ok = mbar_wait(p_empty + r.slot, r.parity ^ 1u, &g_moe_error, kErrWaitEmpty, p.wait_ns))) {
                        *abort_flag = 1;
                        break;
                    }
                    uint8_t *st = smem + r.slot * Cfg::PACKED_BYTES;
                    const uint32_t nsf = min(2, kc - 2 * kq) * 512;
                    mbar_arrive_expect_tx(p_full + r.slot, Cfg::PSF_OFF + (FIRST ? 2 : 1) * nsf);
                    tma_load_2d(st, &p.tm_w, kq * 128, r0, p_full + r.slot, pol);
                    tma_load_2d(st + 8192, &p.tm_w, kq * 128, r1, p_full + r.slot, pol);
                    bulk_load(st + Cfg::PSF_OFF, sf0 + kq * 1024, nsf, p_full + r.slot, pol);
                    if (FIRST) bulk_load(st + Cfg::PSF_OFF + 1024, sf1 + kq * 1024, nsf, p_full + r.slot, pol);
                }
            }
            // copies in flight land before the block leaves
            for (int i = max(0, pk - PACKED); i < pk; ++i) {
                const Ring r = ring_at<PACKED>(i);
                mbar_wait(p_full + r.slot, r.parity, &g_moe_error, kErrWaitDrain);
            }
        }
    } else if (warp == kMmaWarp + 2) {
        if (lane == 0) {
            // ----------------------------------------------------- tokens by TMA
            if (!FIRST) grid_dependency_wait();
            const uint64_t pol = policy_evict_last();
            int gs = 0;
            bool ok = true;
            while (walk.more() && ok && !*abort_flag) {
                const Unit w = walk.take();
                // rank 0 holds the first half of the MMA's columns, rank 1 the second
                const int row = w.row0 + rank * (((w.rows + 31) & ~31) >> 1);
                for (int ks = 0; ks < kc; ++ks, ++gs) {
                    const Ring r = ring_at<OPER>(gs);
                    if (gs >= OPER &&
                        !(ok = mbar_wait(done + r.slot, r.parity ^ 1u, &g_moe_error, kErrWaitEmpty, p.wait_ns))) {
                        *abort_flag = 1;
                        break;
                    }
                    uint8_t *st = smem + Cfg::TOKEN_AT + r.slot * Cfg::TOKEN_BYTES;
                    mbar_arrive_expect_tx(t_full + r.slot, Cfg::HALF * 128 + 1024);
                    tma_load_2d(st, &p.tm_t, ks * 128, row, t_full + r.slot, pol);
                    tma_load_2d(st + Cfg::TSF_OFF, &p.tm_tsf, 0, (w.tile * kc + ks) * 2, t_full + r.slot, pol);
                }
            }
            // copies in flight land before the block leaves, and so do the arrivals of the
            // last MMAs, which come from rank 0 and nobody else waits for
            for (int i = max(0, gs - OPER); i < gs; ++i) {
                const Ring r = ring_at<OPER>(i);
                mbar_wait(t_full + r.slot, r.parity, &g_moe_error, kErrWaitDrain);
            }
            for (int i = max(0, gs - OPER); i < gs && !*abort_flag; ++i) {
                const Ring r = ring_at<OPER>(i);
                if (!mbar_wait(done + r.slot, r.parity, &g_moe_error, kErrWaitDrain)) break;
            }
        }
    } else if (leader) {
        // ------------------------------------------------------ scales to TMEM
        const int total = walk.left() * kc;
        const uint64_t w_desc = sdesc_scale(smem_u32(smem + Cfg::WIDE_AT + Cfg::WSF_OFF));
        const uint64_t t_desc = sdesc_scale(smem_u32(smem + Cfg::TOKEN_AT + Cfg::TSF_OFF));
        bool ok = true;
        for (int gs = 0; gs < total; ++gs) {
            const Ring r = ring_at<OPER>(gs);
            ok = mbar_wait_warp<true>(ready + r.slot, r.parity, &g_moe_error, kErrWaitFull, p.wait_ns);
            if (!ok) break;
            tc_fence_after();
            const uint64_t wd = w_desc + static_cast<uint64_t>(r.slot * (Cfg::WIDE_BYTES >> 4));
            const uint64_t td = t_desc + static_cast<uint64_t>(r.slot * (Cfg::TOKEN_BYTES >> 4));
            const uint32_t tsf = tmem_u + 2 * NT + r.slot * Cfg::SF_COLS;
            if (elect_one()) {
                tc_cp_scale_block_pair(tsf, wd);
                tc_cp_scale_block_pair(tsf + 4, td);
                tc_cp_scale_block_pair(tsf + 8, td + 32);
                tc_commit_pair(s_full + r.slot);
            }
            __syncwarp();
        }
        if (!ok) *abort_flag = 1;
        // no copy may be running when the pair frees TMEM
        if (elect_one()) tc_commit_pair(cp_done);
        __syncwarp();
        mbar_wait_warp(cp_done, 0, &g_moe_error, kErrWaitDrain);
    }
    __syncwarp();

    // neither CTA leaves while the other may still arrive on its barriers or use
    // its shared memory and TMEM
    tc_fence_before();
    cluster_sync();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, Cfg::TMEM_COLS);
    }
}

// Token rows and their scales in sorted order, for the large tiles' TMA: block row
// blockIdx.x is a token tile, its rows shared out over warps and blockIdx.y.
struct GatherParams {
    const uint8_t *x, *x_sf;
    int64_t ldx;
    const int *tiles, *src;
    const int4 *rec;
    uint8_t *xs;        // [R, H]
    uint8_t *xs_sf;     // [tiles][H / 128][2][512]
    int H;
};

__global__ void __launch_bounds__(256) moe_gather_kernel(const GatherParams p)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int tile = blockIdx.x;
    if (tile >= __ldcg(p.tiles)) return;
    const int4 rec = __ldcg(p.rec + tile);
    const int lane = threadIdx.x & 31, kc = p.H >> 7;
    for (int r = blockIdx.y * 8 + (threadIdx.x >> 5); r < rec.z; r += gridDim.y * 8) {
        const int t = __ldcg(p.src + rec.y + r);
        const uint4 *from = reinterpret_cast<const uint4 *>(p.x + static_cast<size_t>(t) * p.ldx);
        uint4 *to = reinterpret_cast<uint4 *>(p.xs + static_cast<size_t>(rec.y + r) * p.H);
        for (int i = lane; i < p.H / 16; i += 4 * 32) {
            uint4 v[4];       // loads ahead of the stores that depend on them
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i + 32 * j < p.H / 16) v[j] = __ldg(from + i + 32 * j);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i + 32 * j < p.H / 16) to[i + 32 * j] = v[j];
        }
        const uint8_t *sf = p.x_sf + static_cast<size_t>(t >> 7) * kc * 512 + (t & 31) * 16 + ((t & 127) >> 5) * 4;
        uint8_t *sfo = p.xs_sf + static_cast<size_t>(tile) * kc * 1024 + (r >> 7) * 512 + (r & 31) * 16 + ((r & 127) >> 5) * 4;
        for (int c = lane; c < kc; c += 32)
            *reinterpret_cast<uint32_t *>(sfo + c * 1024) = *reinterpret_cast<const uint32_t *>(sf + c * 512);
    }
}

// ------------------------------------------------------------------ combine

struct CombineParams {
    const float *y;
    const int *pos;
    const float *weights;
    uint16_t *out;
    int64_t ldo;
    int k, H;
};

// out[t] = sum_j w[t, j] * y[pos[t, j]]: four channels a thread, one token a block row.
__global__ void __launch_bounds__(256) moe_combine_kernel(const CombineParams p)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t t = blockIdx.x;
    const int c = (blockIdx.y * blockDim.x + threadIdx.x) * 4;
    if (c >= p.H) return;
    float acc[4] = {};
    for (int j = 0; j < p.k; ++j) {
        const int r = __ldcg(p.pos + t * p.k + j);
        if (r < 0) continue;
        const float w = p.weights[t * p.k + j];
        const float4 v = __ldcg(reinterpret_cast<const float4 *>(p.y + static_cast<size_t>(r) * p.H + c));
        acc[0] = fmaf(w, v.x, acc[0]);
        acc[1] = fmaf(w, v.y, acc[1]);
        acc[2] = fmaf(w, v.z, acc[2]);
        acc[3] = fmaf(w, v.w, acc[3]);
    }
    const __nv_bfloat162 h[2] = {__floats2bfloat162_rn(acc[0], acc[1]), __floats2bfloat162_rn(acc[2], acc[3])};
    *reinterpret_cast<uint2 *>(p.out + t * p.ldo + c) = *reinterpret_cast<const uint2 *>(h);
}

// ------------------------------------------------------------------- launch

template <class Kern, class P>
cudaError_t launch_pdl(Kern kern, dim3 grid, dim3 block, size_t smem, cudaStream_t stream, const P &params)
{
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, params);
}

template <bool FIRST>
cudaError_t launch_product_small(const ProductParams &p, int64_t max_units, cudaStream_t stream)
{
    auto kern = moe_product_small_kernel<FIRST>;
    static KernelOnce once;
    int sms = 0;
    const cudaError_t e = prepare_kernel(kern, SmallCfg::SMEM_BYTES, once, &sms);
    if (e != cudaSuccess) return e;
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(max_units, std::max(1, sms)));
    return launch_pdl(kern, dim3(grid), dim3(kSmallThreads), SmallCfg::SMEM_BYTES, stream, p);
}

template <bool FIRST>
cudaError_t launch_product_large(const ProductParams &p, int64_t max_units, cudaStream_t stream)
{
    auto kern = moe_product_large_kernel<FIRST>;
    static KernelOnce once;
    int sms = 0;
    const cudaError_t e = prepare_kernel(kern, LargeCfg::SMEM_BYTES, once, &sms);
    if (e != cudaSuccess) return e;
    const unsigned pairs = static_cast<unsigned>(std::min<int64_t>(max_units, std::max(1, sms / 2)));
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(2 * pairs, 1, 1);
    cfg.blockDim = dim3(kLargeThreads, 1, 1);
    cfg.dynamicSmemBytes = LargeCfg::SMEM_BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

inline size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

MoeLayout moe_layout(int64_t T, int k, int E, int64_t H, int64_t I)
{
    MoeLayout out;
    const int64_t R = T * k;
    // Small tiles stream the weights of an expert once for 32 rows, large ones once for
    // 224 but with less of them in flight. Measured both ways: 256 tokens x 6 over 64
    // experts (24 rows an expert) 122 us small, 139 us large; 1111 x 5 over 40, a third
    // left out (93 rows) 166 us small, 109 us large; the border lies between and was not
    // measured. Choices that are left out count as rows, since only the GPU knows them.
    out.nt = R <= 32 * static_cast<int64_t>(E) ? kSmallNT : kLargeNT;
    out.max_tiles = static_cast<int>(R / out.nt + std::min<int64_t>(E, R));
    out.chunks = static_cast<int>((R + kChunk - 1) / kChunk);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += up256(bytes);
        return here;
    };
    out.hist = take(out.chunks > 1 ? static_cast<size_t>(out.chunks) * E * 4 : 0);
    out.tiles = take(4);
    out.rec = take(static_cast<size_t>(out.max_tiles) * 16);
    out.src = take(static_cast<size_t>(R) * 4);
    out.pos = take(static_cast<size_t>(R) * 4);
    out.act = take(static_cast<size_t>(R) * I);
    out.act_sf = take(static_cast<size_t>(out.max_tiles) * (I / 128) * ((out.nt + 127) / 128) * 512);
    out.y = take(static_cast<size_t>(R) * H * 4);
    out.xs = take(out.nt == kLargeNT ? static_cast<size_t>(R) * H : 0);
    out.xs_sf = take(out.nt == kLargeNT ? static_cast<size_t>(out.max_tiles) * (H / 128) * 1024 : 0);
    out.total = at;
    return out;
}

cudaError_t launch_moe_experts(const MoeArgs &a, const MoeLayout &l, cudaStream_t stream)
{
    PlaceParams pp;
    pp.ids = a.ids;
    pp.hist = reinterpret_cast<int *>(a.ws + l.hist);
    pp.tiles = reinterpret_cast<int *>(a.ws + l.tiles);
    pp.rec = reinterpret_cast<int4 *>(a.ws + l.rec);
    pp.src = reinterpret_cast<int *>(a.ws + l.src);
    pp.pos = reinterpret_cast<int *>(a.ws + l.pos);
    pp.R = static_cast<int>(a.T * a.k);
    pp.k = a.k;
    pp.E = a.E;
    pp.chunks = l.chunks;
    pp.nt = l.nt;
    cudaError_t e;
    if (l.chunks > 1) {
        e = launch_pdl(moe_count_kernel, dim3(l.chunks), dim3(kPlaceThreads), 0, stream, pp);
        if (e != cudaSuccess) return e;
    }
    e = launch_pdl(moe_place_kernel, dim3(l.chunks), dim3(kPlaceThreads), 0, stream, pp);
    if (e != cudaSuccess) return e;

    const bool large = l.nt == kLargeNT;
    if (large) {
        GatherParams g;
        g.x = a.xq;
        g.x_sf = a.x_sf;
        g.ldx = a.ldx;
        g.tiles = pp.tiles;
        g.src = pp.src;
        g.rec = pp.rec;
        g.xs = a.ws + l.xs;
        g.xs_sf = a.ws + l.xs_sf;
        g.H = a.H;
        e = launch_pdl(moe_gather_kernel, dim3(l.max_tiles, 14), dim3(256), 0, stream, g);
        if (e != cudaSuccess) return e;
    }

    ProductParams p;
    memset(&p, 0, sizeof(p));
    p.x = a.xq;
    p.ldx = a.ldx;
    p.x_sf = a.x_sf;
    p.act = a.ws + l.act;
    p.act_sf = a.ws + l.act_sf;
    p.y = reinterpret_cast<float *>(a.ws + l.y);
    p.tiles = pp.tiles;
    p.src = pp.src;
    p.rec = pp.rec;
    p.H = a.H;
    p.I = a.I;
    p.wait_ns = wait_limit_ns();
    p.tm_w = a.tm_w13;
    p.w_sf = a.w13_sf;
    if (large) {
        p.tm_t = a.tm_xs;
        p.tm_tsf = a.tm_xs_sf;
        e = launch_product_large<true>(p, static_cast<int64_t>(l.max_tiles) * (a.I / 128), stream);
    } else {
        e = launch_product_small<true>(p, static_cast<int64_t>(l.max_tiles) * (a.I / 64), stream);
    }
    if (e != cudaSuccess) return e;
    p.tm_w = a.tm_w2;
    p.w_sf = a.w2_sf;
    if (large) {
        p.tm_t = a.tm_act;
        p.tm_tsf = a.tm_act_sf;
        e = launch_product_large<false>(p, static_cast<int64_t>(l.max_tiles) * ((a.H + 255) / 256), stream);
    } else {
        e = launch_product_small<false>(p, static_cast<int64_t>(l.max_tiles) * (a.H / 128), stream);
    }
    if (e != cudaSuccess) return e;

    CombineParams c;
    c.y = p.y;
    c.pos = pp.pos;
    c.weights = a.weights;
    c.out = a.out;
    c.ldo = a.ldo;
    c.k = a.k;
    c.H = a.H;
    return launch_pdl(moe_combine_kernel, dim3(static_cast<unsigned>(a.T), (a.H / 4 + 255) / 256), dim3(256), 0, stream, c);
}

int read_and_clear_moe_error()
{
    int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_moe_error, sizeof(int)) != cudaSuccess) return -1;
    cudaMemcpyToSymbol(g_moe_error, &zero, sizeof(int));
    return v;
}

}  // namespace mxfp4
