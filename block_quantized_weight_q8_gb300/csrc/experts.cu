// experts.cu -- the entry points of the experts' products: checks, workspaces and the choice of the path.
#include "experts.h"

namespace qmm {

static __device__ unsigned int g_experts_error = 0;  // bounds records of a bounds-checked build

static qmm_status check_experts(int wt, const ExpertShape& s) {
    if (act_type_of(wt) < 0) return QMM_E_TYPE;
    const qmm_status st = check_shape(wt, s.T, s.N, s.K);
    if (st != QMM_OK) return st;
    if (s.k < 1 || s.k > kMaxChoices || s.E < 1 || s.E > kMaxExperts || s.T * s.k > kMaxRows || s.E * s.N > kMaxDim)
        return QMM_E_SHAPE;
    return QMM_OK;
}

// The workspace: one f32 row of products for each choice.
static size_t scratch_of(int, const ExpertShape& s) { return (size_t)(s.T * s.k) * (size_t)s.N * 4; }

// y[t][n] = residual[t][n] + sum_j weights[t][j] p[t][j][n] over the choices that are there, in their order.  Bound by
// memory: 4 (k + 2) bytes a value.
__global__ void __launch_bounds__(256) combine_kernel(const float* __restrict__ p, const int32_t* __restrict__ ids,
                                                      const float* __restrict__ weights, const float* residual, float* y,
                                                      int T, int k, int E, int N) {
    pdl_launch_dependents();
    pdl_wait();
    const int64_t total = (int64_t)T * N, step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += step) {
        const int64_t t = i / N;
        const int n = (int)(i - t * N);
        float v = 0.0f;
        for (int j = 0; j < k; j++) {
            const int64_t c = t * k + j;
            const int e = ids[c];
            if (e >= 0 && e < E) v = fmaf(weights ? weights[c] : 1.0f, p[c * N + n], v);
        }
        if (QMM_IN_BOUNDS(g_experts_error, i, total)) y[i] = residual ? residual[i] + v : v;
    }
}

static qmm_status combine(const ExpertShape& s, const float* p, const int32_t* ids, const float* weights, const float* residual,
                          float* y, cudaStream_t stream) {
    DeviceInfo dev;
    const qmm_status st = current_device(&dev);
    if (st != QMM_OK) return st;
    const int64_t want = (s.T * s.N + 255) / 256, most = (int64_t)dev.sms * 8;
    return launch_pdl(combine_kernel, dim3((unsigned)(want < most ? want : most)), 256, 0, stream, p, ids, weights, residual, y,
                      (int)s.T, (int)s.k, (int)s.E, (int)s.N);
}

}  // namespace qmm

using namespace qmm;

extern "C" {

size_t qmm_experts_scratch_bytes(int wtype, int64_t T, int64_t k, int64_t E, int64_t N, int64_t K) {
    const ExpertShape s{T, k, E, N, K};
    return check_experts(wtype, s) == QMM_OK ? scratch_of(wtype, s) : 0;
}

qmm_status qmm_experts_glu(int wtype, int kind, const void* Wg, const void* Wu, const void* xq, const int32_t* ids, float* h,
                           void* scratch, size_t scratch_bytes, int64_t T, int64_t k, int64_t E, int64_t N, int64_t K,
                           qmm_stream_t stream) {
    const ExpertShape s{T, k, E, N, K};
    if (!Wg || !Wu || !xq || !ids || !h || !scratch) return QMM_E_NULL;
    const qmm_status st = check_experts(wtype, s);
    if (st != QMM_OK) return st;
    if (kind != QMM_GLU_SILU && kind != QMM_GLU_GELU) return QMM_E_TYPE;
    if (!aligned16(Wg) || !aligned16(Wu) || !aligned16(xq) || !aligned4(ids) || !aligned16(h) || !aligned16(scratch))
        return QMM_E_ALIGN;
    if (scratch_bytes < scratch_of(wtype, s)) return QMM_E_SCRATCH;
    return expert_vec_glu(wtype, kind, s, Wg, Wu, xq, ids, h, (cudaStream_t)stream);
}

qmm_status qmm_experts_sum(int wtype, const void* W, const float* h, const int32_t* ids, const float* weights,
                           const float* residual, float* y, void* scratch, size_t scratch_bytes, int64_t T, int64_t k,
                           int64_t E, int64_t N, int64_t K, qmm_stream_t stream) {
    const ExpertShape s{T, k, E, N, K};
    if (!W || !h || !ids || !y || !scratch) return QMM_E_NULL;
    const qmm_status st = check_experts(wtype, s);
    if (st != QMM_OK) return st;
    if (!aligned16(W) || !aligned16(h) || !aligned4(ids) || !aligned4(weights) || !aligned16(residual) || !aligned16(y) ||
        !aligned16(scratch))
        return QMM_E_ALIGN;
    if (scratch_bytes < scratch_of(wtype, s)) return QMM_E_SCRATCH;
    cudaStream_t cs = (cudaStream_t)stream;
    const qmm_status fused = expert_vec_sum(wtype, s, W, h, ids, weights, residual, y, cs);
    if (fused != QMM_E_SHAPE) return fused;
    // a token's rows do not fit one SM: choice by choice, then the sum
    float* p = static_cast<float*>(scratch);
    const ExpertShape each{T * k, 1, E, N, K};
    const qmm_status one = expert_vec_sum(wtype, each, W, h, ids, nullptr, nullptr, p, cs);
    return one != QMM_OK ? one : combine(s, p, ids, weights, residual, y, cs);
}

unsigned qmm_internal_experts_error(int clear) {
    unsigned v = 0;
    cudaMemcpyFromSymbol(&v, g_experts_error, sizeof(v));
    if (clear) {
        const unsigned z = 0;
        cudaMemcpyToSymbol(g_experts_error, &z, sizeof(z));
    }
    return v;
}

}  // extern "C"
