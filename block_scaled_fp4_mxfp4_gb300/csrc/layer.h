// Host-side interface between the C-ABI layer of mxfp4_layer.h (layer_api.cu)
// and its kernel translation units. Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace mxfp4 {

// ------------------------------------------------------- qk_norm_rope.cu
struct QkParams {
    const uint16_t *x[2];       // queries, keys
    uint16_t *out[2];
    const uint16_t *w[2];       // or null
    int64_t st[2], sh[2];       // elements between tokens, heads
    int64_t ost[2], osh[2];
    const float *table;
    const void *positions;
    int64_t T, P;
    int heads[2];
    int D, rot, pos64;
    float eps;
    int units, unit_heads;      // set at launch: units that a token's heads make, and heads of one
};
cudaError_t launch_qk_norm_rope(const QkParams &p, bool f16, bool interleaved, int num_sms, cudaStream_t stream);

// ---------------------------------------------------------------- lora.cu
struct LoraParams {
    const uint16_t *x, *a, *b;
    const int32_t *ids;
    const float *scales;
    const int32_t *ranks;
    const uint16_t *base;
    uint16_t *c;
    int64_t ldx, ldb, ldc;
    int T, K, N, R, L;
    bool copy;                  // tokens without an adapter are copied (C is not base)
    // workspace
    float *u;                   // [splits][T][R] partial sums of the first product
    int *order;                 // [T] tokens by adapter            (long batches only)
    int4 *tiles;                // adapter, first of order, tokens  (long batches only)
    int splits, max_tiles;
};
struct LoraLayout {
    int splits, max_tiles;
    size_t u, order, tiles, total;
};
LoraLayout lora_layout(int64_t T, int64_t K, int R, int L);
cudaError_t launch_lora(LoraParams p, const LoraLayout &l, bool f16, cudaStream_t stream);
int read_and_clear_lora_error();

}  // namespace mxfp4
