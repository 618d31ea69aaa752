// experts_mma.h -- what the tensor-core path's kernels share: tiles of sorted rows and the activation records.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "qmm.h"

namespace qmm {

constexpr int kTileRows = 128;  // activation rows of a tile
// 256 values of an activation row: 256 codes (plus 128); 8 f16 scales (Q8_0) or one f32 (Q8_K) at 256; the codes' sums over groups of
// 16 as f16 (whole numbers up to 2048, exact) at 272.  19 16-byte words: neighbouring rows' words fall in other banks.
constexpr int kRecord = 304;

struct ExpertTile {
    int32_t expert, first, count, unused;  // rows order[first .. first + count) of one expert
};

struct ExpertMma {
    const uint8_t* W0;      // [E][N] rows: the product's, or the gate's
    const uint8_t* W1;      // gated: the up matrix's
    const uint8_t* records; // [rows][ceil(K / 256)] records
    const int32_t* order;   // the rows (choices) of the tiles
    const ExpertTile* tiles;
    const int32_t* ntiles;
    float* y;               // [choices][N]
    int64_t out_values;
    int per_row;            // choices that share an activation row
    int E, N, K, kind;
};

qmm_status expert_mma_32(int wt, const ExpertMma& a, bool gate, int64_t tiles_most, cudaStream_t stream);
qmm_status expert_mma_five(int wt, const ExpertMma& a, bool gate, int64_t tiles_most, cudaStream_t stream);
qmm_status expert_mma_k(int wt, const ExpertMma& a, bool gate, int64_t tiles_most, cudaStream_t stream);

}  // namespace qmm
