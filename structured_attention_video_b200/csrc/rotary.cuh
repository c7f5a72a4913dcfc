// rotary.cuh -- problem description of the rotary positions (rotary.cu).
#pragma once

#include "monarch_common.cuh"

namespace monarch {
namespace rot {

struct Strides {
    int64_t batch, head, token;   // in elements; the head dimension has stride 1
};

struct RotaryProblem {
    int B, N, H, Hkv, d;          // Hkv = 0: no keys
    int pairs, axes, end[2];      // pairs [0, end[0]) turn with axis 0, [end[0], end[1]) with 1
    int half, inverse;
    float magnitude;
    int gh, gw;                   // rows and columns of the token grid, 0: one axis
    int64_t start;
    const int32_t *starts;        // [B] or null (start)
    const int32_t *positions;     // [B][N][axes] with the two strides below, or null
    int64_t pos_batch, pos_token;
    const double *freqs;          // [pairs], radians per position
    int heads_per_block;
    Strides q, k, qo, ko;
};

cudaError_t rotary_forward(const RotaryProblem &p, monarch_dtype dtype, const void *q,
                           const void *k, void *qo, void *ko, cudaStream_t stream);

}  // namespace rot
}  // namespace monarch
