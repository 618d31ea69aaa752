// experts_mma_k.cu -- the tensor-core experts' products of Q4_K, Q6_K and Q2_K.
#include "experts_mma.cuh"

namespace qmm {

qmm_status expert_mma_k(int wt, const ExpertMma& a, bool gate, int64_t tiles_most, cudaStream_t stream) {
    switch (wt) {
    case QMM_Q4_K: return expert_mma_either<QMM_Q4_K>(a, gate, tiles_most, stream);
    case QMM_Q6_K: return expert_mma_either<QMM_Q6_K>(a, gate, tiles_most, stream);
    case QMM_Q2_K: return expert_mma_either<QMM_Q2_K>(a, gate, tiles_most, stream);
    default: return QMM_E_TYPE;
    }
}

}  // namespace qmm

extern "C" unsigned qmm_internal_expert_mma_k_error(int clear) {
    unsigned v = 0;
    cudaMemcpyFromSymbol(&v, qmm::g_expert_mma_error, sizeof(v));
    if (clear) {
        const unsigned z = 0;
        cudaMemcpyToSymbol(qmm::g_expert_mma_error, &z, sizeof(z));
    }
    return v;
}
