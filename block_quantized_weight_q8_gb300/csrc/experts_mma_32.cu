// experts_mma_32.cu -- the tensor-core experts' products of Q4_0, Q8_0 and Q4_1.
#include "experts_mma.cuh"

namespace qmm {

qmm_status expert_mma_32(int wt, const ExpertMma& a, bool gate, int64_t tiles_most, cudaStream_t stream) {
    switch (wt) {
    case QMM_Q4_0: return expert_mma_either<QMM_Q4_0>(a, gate, tiles_most, stream);
    case QMM_Q8_0: return expert_mma_either<QMM_Q8_0>(a, gate, tiles_most, stream);
    case QMM_Q4_1: return expert_mma_either<QMM_Q4_1>(a, gate, tiles_most, stream);
    default: return QMM_E_TYPE;
    }
}

}  // namespace qmm

extern "C" unsigned qmm_internal_expert_mma_32_error(int clear) {
    unsigned v = 0;
    cudaMemcpyFromSymbol(&v, qmm::g_expert_mma_error, sizeof(v));
    if (clear) {
        const unsigned z = 0;
        cudaMemcpyToSymbol(qmm::g_expert_mma_error, &z, sizeof(z));
    }
    return v;
}
