// experts.h -- shapes, limits and the gate's activation, shared by the experts' translation units.
#pragma once

#include "qmm_device.cuh"
#include "qmm_host.h"

namespace qmm {

constexpr int kMaxChoices = 64;                // experts of one token
constexpr int64_t kMaxExperts = 1024;
constexpr int64_t kMaxRows = (int64_t)1 << 24;  // rows of a call, tokens times choices
constexpr unsigned kErrIndex = 2u;             // an expert's index beyond the last (reported as QMM_E_SHAPE)

struct ExpertShape {
    int64_t T, k, E, N, K;
};

// act(g) * u in f32: silu g / (1 + e^-g), or gelu by its tanh form, 0.5 g (1 + tanh(z)) = g / (1 + e^-2z) with
// z = sqrt(2/pi) (g + 0.044715 g^3).  Where the exponential is infinite the quotient's limit is 0, for -inf too.
__device__ __forceinline__ float gated(int kind, float g, float u) {
    float z = g;
    if (kind == QMM_GLU_GELU) z = 1.5957691216057308f * fmaf(0.044715f * g * g, g, g);
    const float e = expf(-z);
    const float v = e == INFINITY ? 0.0f : g / (1.0f + e);
    return v * u;
}

// csrc/experts_vec.cu: a launch for few rows.
qmm_status expert_vec_glu(int wt, int kind, const ExpertShape& s, const void* Wg, const void* Wu, const void* xq,
                          const int32_t* ids, float* h, cudaStream_t stream);
qmm_status expert_vec_sum(int wt, const ExpertShape& s, const void* W, const float* x, const int32_t* ids,
                          const float* weights, const float* residual, float* y, cudaStream_t stream);

}  // namespace qmm
