// experts_mma.h -- what the tensor-core path's kernels share: tiles of sorted rows and the activation records.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "qmm.h"

namespace qmm {

constexpr int kTileRows = 128;  // activation rows of a tile

// The activation operand of a tile, its rows made a multiple of 16 (zeros behind the last), chunk of 256 values by chunk:
//   for each of 8 blocks of 32 values, each term: rows / 8 groups of 8 rows, each 4 core matrices (8 values) of 8 rows
//   the sums of 16 values, each term: rows / 8 groups of 2 core matrices
//   the f32 scale of each row's chunk
// Q8_0 rows have two terms, Q8_K rows one.
constexpr int operand_terms(int act) { return act == QMM_Q8_0 ? 2 : 1; }
constexpr int operand_bytes(int act) { return operand_terms(act) * (512 + 32) + 4; }  // of a row's chunk

// 32-value blocks (and Q8_0 rows) stand over a power of two that a run shares.  It brings the largest scale (or minimum) below
// 2^(1 + spare), as far up as scale times code and, beside minimums, scale times the sum of 16 codes stay f16: so every f16
// scale of a run is exact where the largest is below that, and else whatever is at least 2^-(14 + spare) of it.
constexpr int weight_spare(int wt) {  // codes (Q4_1, Q5_1: centered, the minimum with them) up to 2^7, 2^3, 2^4
    return wt == QMM_Q8_0 ? 7 : wt == QMM_Q4_0 || wt == QMM_Q4_1 ? 11 : 10;
}
constexpr int act_spare(int wt) { return wt == QMM_Q4_1 || wt == QMM_Q5_1 ? 4 : 7; }
// the power that the run's values are multiplied by, from the largest scale's f16 bits (sign cleared); at least -11
__host__ __device__ constexpr int run_shift(uint32_t bits, int spare) {
    const int e = (int)(bits >> 10), s = 15 + spare - (e < 1 ? 1 : e > 30 ? 30 : e);
    return s < 15 ? s : 15;  // f16 has no larger one, and every scale is over 2^-14 by then
}

struct ExpertTile {
    int32_t expert, first, count;  // rows order[first .. first + count) of one expert
    int32_t at;                    // where its operand begins, in rows
};

struct ExpertMma {
    const uint8_t* W0;      // [E][N] rows: the product's, or the gate's
    const uint8_t* W1;      // gated: the up matrix's
    const uint8_t* operand;
    const int32_t* order;   // the rows (choices) of the tiles
    const ExpertTile* tiles;
    const int32_t* ntiles;
    float* y;               // [choices][N]
    int64_t out_values;
    int E, N, K, kind;
};

qmm_status expert_mma_32(int wt, const ExpertMma& a, bool gate, int64_t tiles_most, cudaStream_t stream);
qmm_status expert_mma_five(int wt, const ExpertMma& a, bool gate, int64_t tiles_most, cudaStream_t stream);
qmm_status expert_mma_k(int wt, const ExpertMma& a, bool gate, int64_t tiles_most, cudaStream_t stream);

}  // namespace qmm
