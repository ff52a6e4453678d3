// Parameters shared by the rotation / paged-cache kernels (qknorm_rope.cu) and
// the 4-bit cache's geometry (also used by qknorm_kv4.cu).
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace qkn {

constexpr int kKv4Group = 64;      // dims of a head that share one fp16 scale
constexpr int kKv4PageMultiple = 16;  // pages are whole 16-token tiles
constexpr int kRopeMaxHeadDim = 1024;

// Where a launch's K and V heads go.
enum Sink : int {
    kSinkRows = 0,   // rows next to Q's (no V)
    kSinkCache = 1,  // a paged cache of the element type
    kSinkKv4 = 2     // the paged 4-bit cache
};

struct RopeParams {
    // 0 = Q, 1 = K, 2 = V: token t's heads start at in[i] + t * stride[i] bytes
    const char *in[3];
    char *out[2];                // Q rows, K rows (kSinkRows), same strides as the inputs
    int64_t stride[3];
    const char *gamma[2];        // null: no norm
    int32_t heads[3];
    int32_t heads_total;
    int64_t T;
    const float *table;          // [table_rows][2 * half]: cosines, then sines
    const int64_t *positions;    // [T]
    int64_t table_rows;
    int32_t head_dim;
    int32_t half;                // rotary_dim / 2
    int32_t interleaved;         // pairs (2i, 2i + 1) instead of (i, i + half)
    int32_t units;               // vector kernel: lanes of a head = head_dim / (2 * elements per vector)
    int32_t lanes;               // vector kernel: units rounded up to a power of two
    int32_t chunks;              // vector kernel: warps per token,
    int32_t chunks_of[3];        // of which each tensor's,
    int32_t chunk_heads;         // and the heads of a warp: Q's,
    int32_t chunk_kv_heads;      // K's and V's
    float eps;
    float inv_d;                 // 1 / head_dim
    // caches (kSinkCache: bytes; kSinkKv4: codes, then scales)
    const int64_t *slots;        // [T] flat token index, negative: not written
    int64_t num_slots;
    int32_t page_size;
    char *cache[2];
    int64_t page_stride[2], token_stride[2], head_stride[2];
    __half *scales[2];
};

// Gradient of kSinkRows' forward pass; 0 = Q, 1 = K.
struct RopeGradParams {
    const char *x[2], *dy[2];
    char *dx[2];
    int64_t x_stride[2], dy_stride[2], dx_stride[2];  // bytes
    const char *gamma[2];
    float *partial;              // [grid][2][head_dim] sums of each CTA
    int32_t heads[2];
    int64_t T;
    const float *table;
    const int64_t *positions;
    int64_t table_rows;
    int32_t head_dim;
    int32_t half;
    int32_t interleaved;
    int32_t units;
    int32_t lanes;
    int32_t chunk_heads;         // vector kernel: heads a warp takes of a token at a time
    float eps;
    float inv_d;
};

}  // namespace qkn
