// experts_mma_five.cu -- the tensor-core experts' products of Q5_0, Q5_1 and Q5_K.
#include "experts_mma.cuh"

namespace qmm {

qmm_status expert_mma_five(int wt, const ExpertMma& a, bool gate, int64_t tiles_most, cudaStream_t stream) {
    switch (wt) {
    case QMM_Q5_0: return expert_mma_either<QMM_Q5_0>(a, gate, tiles_most, stream);
    case QMM_Q5_1: return expert_mma_either<QMM_Q5_1>(a, gate, tiles_most, stream);
    case QMM_Q5_K: return expert_mma_either<QMM_Q5_K>(a, gate, tiles_most, stream);
    default: return QMM_E_TYPE;
    }
}

}  // namespace qmm

extern "C" unsigned qmm_internal_expert_mma_five_error(int clear) {
    unsigned v = 0;
    cudaMemcpyFromSymbol(&v, qmm::g_expert_mma_error, sizeof(v));
    if (clear) {
        const unsigned z = 0;
        cudaMemcpyToSymbol(qmm::g_expert_mma_error, &z, sizeof(z));
    }
    return v;
}
