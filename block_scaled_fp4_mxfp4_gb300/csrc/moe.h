// Host-side interface between the mixture-of-experts C-ABI layer (moe_api.cu)
// and its kernel translation units. Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace mxfp4 {

// ---------------------------------------------------- add_rmsnorm_quant.cu
cudaError_t launch_add_rmsnorm_mxfp8(const void *X, int64_t ldx, const void *res, int64_t ldr, const void *w, bool f16,
                                     float eps, int64_t M, int64_t K, void *H, int64_t ldh, void *Y, int64_t ldy,
                                     void *Aq, int64_t ldq, void *sf, int num_sms, cudaStream_t stream);

// ------------------------------------------------------------ moe_route.cu
struct RouteParams {
    const void *logits;
    const float *bias;      // [E] or null
    int32_t *ids;
    float *weights;
    int64_t ldl, T;
    int E, k, groups, topk_groups, group_top;
    int sigmoid, renorm;
    float scale;
    int group_lanes;        // set at launch: lanes a group fills, 0 where groups are no runs of lanes
    int vec;                // set at launch: rows allow 16-byte vectors
};
cudaError_t launch_moe_route(const RouteParams &p, int dtype, int num_sms, cudaStream_t stream);

// ---------------------------------------------------------- moe_experts.cu
// Workspace of one call, and the token tile its two products share.
struct MoeLayout {
    int nt;                 // tokens of a tile (columns of the accumulator)
    int max_tiles;          // most token tiles T * k choices can need
    int chunks;             // blocks of the placing kernel
    size_t hist, tiles, rec, src, pos, act, act_sf, y, xs, xs_sf, total;
};
constexpr int kMoeLargeTile = 224;   // nt of the layouts that need sorted token rows
MoeLayout moe_layout(int64_t T, int k, int E, int64_t H, int64_t I);

struct MoeArgs {
    const uint8_t *xq;
    int64_t ldx;
    const uint8_t *x_sf;
    const int32_t *ids;
    const float *weights;
    const uint8_t *w13_sf, *w2_sf;
    uint16_t *out;
    int64_t ldo;
    int64_t T;
    int k, E, H, I;
    uint8_t *ws;
    CUtensorMap tm_w13;     // packed weights [E * 2I, H / 2] u8, box 128 bytes x 64 rows
    CUtensorMap tm_w2;      // the same of [E * H, I / 2]
    // large tiles only: sorted token rows [R, H] and activations [R, I] (u8, box 128 bytes x half
    // a token tile), and their scales (blocks of 128 u32, box two blocks)
    CUtensorMap tm_xs, tm_xs_sf, tm_act, tm_act_sf;
};
cudaError_t launch_moe_experts(const MoeArgs &a, const MoeLayout &l, cudaStream_t stream);
int read_and_clear_moe_error();

// -------------------------------------------------------------- moe_few.cu
// The whole layer for up to kMoeFewTokens tokens: eight columns of an MMA each.
constexpr int kMoeFewTokens = 16;
struct MoeFewLayout {
    size_t counters, h, part, part_ss, xd, xsf, ids, weights, ad, asf, y, total;
};
MoeFewLayout moe_few_layout(int64_t T, int k, int E, int64_t H, int64_t I);

struct MoeFewArgs {
    const uint16_t *x, *res, *w, *router;
    uint16_t *h_out, *out;
    int64_t ldx, ldr, ldh, ldo;
    const uint8_t *w13_sf, *w2_sf;
    RouteParams route;      // logits, ldl and T unused; ids and weights may be null
    int T, H, I;
    float eps;
    uint8_t *ws;
    CUtensorMap tm_w13;     // packed weights [E * 2I, H / 2] u8, box 128 bytes x 32 rows
    CUtensorMap tm_w2;      // the same of [E * H, I / 2], box 64 rows
};
cudaError_t launch_moe_few(const MoeFewArgs &a, const MoeFewLayout &l, cudaStream_t stream);
int read_and_clear_moe_few_error();

}  // namespace mxfp4
