// matvec.cu -- the decode matvec (one token): y[o] = row o of the block-quantized
// W against one Q8_0 / Q8_K activation row, for Q4_0, Q8_0, Q4_K, Q6_K and Q2_K,
// and Q4_1, Q5_0, Q5_1, Q5_K.
//
// Design (GB300): the kernel is HBM-bound, so it is built around keeping the
// weight stream in flight.  Each CTA owns a contiguous range of rows (an even
// split of N over the grid).  One thread streams that range into a ring of
// shared-memory stages with 1-D bulk copies (cp.async.bulk, completing on an
// mbarrier) tagged evict-first in L2; the copies cover the 16-byte aligned
// superset of each stage's rows, so no block layout (18, 34, 84, 210 B) needs
// to be aligned.  Meanwhile the CTA unpacks the activation row once into
// shared memory (contiguous int8 codes plus f32 scales and int32 group sums).
// Each row of a stage is then owned by `lpr` lanes of one warp, which decode
// whole blocks from shared memory, take the exact integer block dot with
// __dp4a, fold it into fp32 once per block, and reduce with warp shuffles in a
// fixed order -- so every y[o] is written by one lane, identically on every
// run ([minfer] s3.3: row ownership, no split reduction).
//
// Formulas: [minfer] "10 . CPU matmul: quantized weights x Q8_0 activations"
// s3.2 (the scalar kernels, the K-quant dot walked); [ggml] "ggml Q4_0 vec_dot
// Walkthrough" s1.2 and s2.
#include <stdio.h>

#include "matvec_kernel.cuh"

namespace qmm {

constexpr int kThreads = 256;  // blocksums kernel

// ------------------------------------------------------------------ blocksums (verification)
// One CTA per (token, group of rows): copies the rows' bytes into shared memory
// with plain loads and runs the same decoders, writing the integers.
template <int WT>
__global__ void __launch_bounds__(kThreads) blocksums_kernel(const uint8_t* __restrict__ W,
                                                             const uint8_t* __restrict__ xq, int32_t* __restrict__ out,
                                                             int N, int K, int rows_per_cta, uint32_t act_bytes) {
    using F = Fmt<WT>;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* aq = smem + 128;
    const int nd = F::ACT == QMM_Q8_0 ? K / 32 : K / 256;
    const int ap = F::ACT == QMM_Q8_0 ? nd : q8k_pitch(nd);
    float* ad = reinterpret_cast<float*>(aq + act_code_bytes(F::ACT, K));
    int* as = reinterpret_cast<int*>(ad + nd);
    uint8_t* wbuf = smem + act_bytes;

    const int t = blockIdx.y;
    const int units = K / F::BV;
    const uint64_t rb = (uint64_t)units * F::BB;
    const uint64_t xrb = F::ACT == QMM_Q8_0 ? (uint64_t)(K / 32) * Q8_0_BB : (uint64_t)(K / 256) * Q8_K_BB;
    const uint8_t* xrow = xq + (uint64_t)t * xrb;
    if constexpr (F::ACT == QMM_Q8_0) unpack_q8_0_row(xrow, K, aq, ad, as);
    else unpack_q8_K_row(xrow, K, aq, ad, as);

    const int r0 = blockIdx.x * rows_per_cta;
    const int r1 = min(r0 + rows_per_cta, N);
    const uint64_t a0 = ((uint64_t)r0 * rb) & ~15ull;
    const uint64_t g1 = (uint64_t)r1 * rb;
    for (uint64_t i = a0 + threadIdx.x; i < g1; i += blockDim.x)
        if (QMM_IN_BOUNDS(g_matvec_error, i - a0, (uint64_t)rows_per_cta * rb + 16)) wbuf[i - a0] = W[i];
    __syncthreads();

    const ActView act{aq, ad, as, ap};
    const SmemBytes wv{wbuf};
    const int per = F::ACT == QMM_Q8_0 ? units : 2 * units;
    for (int i = threadIdx.x; i < (r1 - r0) * units; i += blockDim.x) {
        const int row = r0 + i / units, u = i % units;
        const uint32_t o = (uint32_t)((uint64_t)row * rb - a0) + (uint32_t)(u * F::BB);
        int32_t* dst = out + ((uint64_t)t * N + row) * per;
        if (!QMM_IN_BOUNDS(g_matvec_error, ((uint64_t)t * N + row) * per + u * (per / units), (uint64_t)gridDim.y * N * per))
            continue;
        uint32_t db, dmb;
        int v = 0, m = 0;
        if constexpr (WT == QMM_Q4_0) v = q4_0_isum(wv, o, act, u, &db);
        else if constexpr (WT == QMM_Q8_0) v = q8_0_isum(wv, o, act, u, &db);
        else if constexpr (WT == QMM_Q4_K) q4_K_isums(wv, o, act, u, &v, &m, &db, &dmb);
        else if constexpr (WT == QMM_Q2_K) q2_K_isums(wv, o, act, u, &v, &m, &db, &dmb);
        else if constexpr (WT == QMM_Q6_K) q6_K_isums(wv, o, act, u, &v, &m, &db);
        else if constexpr (WT == QMM_Q4_1) v = q4_1_isum(wv, o, act, u, &db);
        else if constexpr (WT == QMM_Q5_0) v = q5_0_isum(wv, o, act, u, &db);
        else if constexpr (WT == QMM_Q5_1) v = q5_1_isum(wv, o, act, u, &db);
        else q5_K_isums(wv, o, act, u, &v, &m, &db, &dmb);
        if constexpr (F::ACT == QMM_Q8_0) {
            dst[u] = v;
        } else {
            dst[2 * u] = v;
            dst[2 * u + 1] = m;
        }
    }
}

// ------------------------------------------------------------------ host side
qmm_status current_device(DeviceInfo* info) {
    static DeviceInfo cache[64];
    static PerDeviceOnce once;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return QMM_E_CUDA;
    const qmm_status st = once.run(dev, [&] {
        DeviceInfo d;
        d.device = dev;
        if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return QMM_E_CUDA;
        if (cudaDeviceGetAttribute(&d.max_smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess)
            return QMM_E_CUDA;
        if (cudaDeviceGetAttribute(&d.smem_per_sm, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev) != cudaSuccess)
            return QMM_E_CUDA;
        if (cudaDeviceGetAttribute(&d.smem_reserved, cudaDevAttrReservedSharedMemoryPerBlock, dev) != cudaSuccess)
            return QMM_E_CUDA;
        cache[dev] = d;
        return QMM_OK;
    });
    if (st != QMM_OK) return st;
    *info = cache[dev];
    return QMM_OK;
}

template <int WT, bool SU, int FUSE, bool SPLIT>
static qmm_status launch_matvec_k(const MatSet& set, const void* xq, const float* x, void* xq_out, int64_t K,
                                   const MatvecPlan& p, const DeviceInfo& dev, cudaStream_t stream, bool pdl) {
    static PerDeviceOnce attr_once;
    const qmm_status ast = attr_once.run(dev.device, [&] {
        if (cudaFuncSetAttribute(matvec_kernel<WT, SU, FUSE, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 dev.max_smem_optin) != cudaSuccess)
            return QMM_E_CUDA;
        // all of the SM's unified memory as shared memory, so that two small CTAs fit
        if (cudaFuncSetAttribute(matvec_kernel<WT, SU, FUSE, SPLIT>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                 (int)cudaSharedmemCarveoutMaxShared) != cudaSuccess)
            return QMM_E_CUDA;
        return QMM_OK;
    });
    if (ast != QMM_OK) return ast;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.grid);
    cfg.blockDim = dim3((unsigned)(p.nw * 32));
    cfg.dynamicSmemBytes = p.smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, matvec_kernel<WT, SU, FUSE, SPLIT>, set, (const uint8_t*)xq, x,
                                             (uint8_t*)xq_out, (int)K, p.lpr, p.pieces, p.piece_units, p.item_segs,
                                             p.depth, p.slot_bytes, p.part_off, p.act_bytes, pdl ? 1 : 0);
    return e == cudaSuccess ? QMM_OK : QMM_E_CUDA;
}

template <int WT, bool SU, int FUSE>
static qmm_status launch_matvec_su(const MatSet& set, const void* xq, const float* x, void* xq_out, int64_t K,
                                   const MatvecPlan& p, const DeviceInfo& dev, cudaStream_t stream, bool pdl) {
    if (p.pieces > 1) return launch_matvec_k<WT, SU, FUSE, true>(set, xq, x, xq_out, K, p, dev, stream, pdl);
    return launch_matvec_k<WT, SU, FUSE, false>(set, xq, x, xq_out, K, p, dev, stream, pdl);
}

// G matrices W[g] (N[g] rows each) against one activation row.  x == nullptr:
// multiply the quantized row xq.  Otherwise quantize x in the kernel (xq then
// names where CTA 0 stores the quantized row, or is null).
template <int WT>
static qmm_status launch_matvec(const void* const* W, const int64_t* N, float* const* y, int G, const void* xq,
                                const float* x, int64_t K, cudaStream_t stream, bool pdl, const float* gamma,
                                float eps) {
    if (G < 1 || G > kMaxGroup) return QMM_E_SHAPE;
    DeviceInfo dev;
    qmm_status st = current_device(&dev);
    if (st != QMM_OK) return st;
    MatvecPlan p;
    MatSet set = {};
    const bool fuse = x != nullptr;
    st = plan_matvec<WT>(N, G, K, dev, fuse, fuse && gamma != nullptr, &p, set.cta_end);
    if (st != QMM_OK) return st;
    set.G = G;
    set.gamma = fuse ? gamma : nullptr;
    set.eps = eps;
    set.norm_off = p.norm_off;
    for (int g = 0; g < G; g++) {
        set.W[g] = (const uint8_t*)W[g];
        set.y[g] = y[g];
        set.N[g] = (int)N[g];
    }
    if (fuse && gamma != nullptr) {  // RMSNorm, quantize and multiply
        if constexpr (has_su<WT>()) {
            if (p.su) return launch_matvec_su<WT, true, 2>(set, nullptr, x, (void*)xq, K, p, dev, stream, pdl);
        }
        return launch_matvec_su<WT, false, 2>(set, nullptr, x, (void*)xq, K, p, dev, stream, pdl);
    }
    if (fuse) {  // quantize and multiply
        if constexpr (has_su<WT>()) {
            if (p.su) return launch_matvec_su<WT, true, 1>(set, nullptr, x, (void*)xq, K, p, dev, stream, pdl);
        }
        return launch_matvec_su<WT, false, 1>(set, nullptr, x, (void*)xq, K, p, dev, stream, pdl);
    }
    if constexpr (has_su<WT>()) {
        if (p.su) return launch_matvec_su<WT, true, 0>(set, xq, nullptr, nullptr, K, p, dev, stream, pdl);
    }
    return launch_matvec_su<WT, false, 0>(set, xq, nullptr, nullptr, K, p, dev, stream, pdl);
}

// Public calls require 16-byte aligned bases; internal per-token calls pass rows
// of a larger buffer, which the kernel accepts at their natural alignment (W
// 16 bytes for the bulk copies, an activation row 2 bytes, y 4 bytes; an f32
// row x to quantize in the kernel 16 bytes).
static qmm_status matvec_group_checked(int wt, int G, const void* const* W, const int64_t* N, float* const* y,
                                       const void* xq, const float* x, int64_t K, cudaStream_t stream, bool pdl,
                                       bool public_call, const float* gamma = nullptr, float eps = 0.0f) {
    if (G < 1 || G > kMaxGroup) return QMM_E_SHAPE;
    if (!W || !N || !y || (!xq && !x)) return QMM_E_NULL;
    for (int g = 0; g < G; g++) {
        if (!W[g] || !y[g]) return QMM_E_NULL;
        qmm_status st = check_shape(wt, 1, N[g], K);
        if (st != QMM_OK) return st;
        if (public_call && (!aligned16(W[g]) || !aligned16(y[g]))) return QMM_E_ALIGN;
        if (!aligned16(W[g]) || ((uintptr_t)y[g] & 3u)) return QMM_E_ALIGN;
    }
    if (public_call && !aligned16(xq)) return QMM_E_ALIGN;
    if (((uintptr_t)xq & 1u) || !aligned16(x) || !aligned16(gamma)) return QMM_E_ALIGN;
    switch (wt) {
    case QMM_Q4_0: return launch_matvec<QMM_Q4_0>(W, N, y, G, xq, x, K, stream, pdl, gamma, eps);
    case QMM_Q8_0: return launch_matvec<QMM_Q8_0>(W, N, y, G, xq, x, K, stream, pdl, gamma, eps);
    case QMM_Q4_K: return launch_matvec<QMM_Q4_K>(W, N, y, G, xq, x, K, stream, pdl, gamma, eps);
    case QMM_Q6_K: return launch_matvec<QMM_Q6_K>(W, N, y, G, xq, x, K, stream, pdl, gamma, eps);
    case QMM_Q2_K: return launch_matvec<QMM_Q2_K>(W, N, y, G, xq, x, K, stream, pdl, gamma, eps);
    case QMM_Q4_1: return launch_matvec<QMM_Q4_1>(W, N, y, G, xq, x, K, stream, pdl, gamma, eps);
    case QMM_Q5_0: return launch_matvec<QMM_Q5_0>(W, N, y, G, xq, x, K, stream, pdl, gamma, eps);
    case QMM_Q5_1: return launch_matvec<QMM_Q5_1>(W, N, y, G, xq, x, K, stream, pdl, gamma, eps);
    case QMM_Q5_K: return launch_matvec<QMM_Q5_K>(W, N, y, G, xq, x, K, stream, pdl, gamma, eps);
    default: return QMM_E_TYPE;
    }
}

static qmm_status matvec_checked(int wt, const void* W, const void* xq, const float* x, float* y, int64_t N,
                                 int64_t K, cudaStream_t stream, bool pdl, bool public_call) {
    return matvec_group_checked(wt, 1, &W, &N, &y, xq, x, K, stream, pdl, public_call);
}

qmm_status matvec_dispatch(int wt, const void* W, const void* xq, float* y, int64_t N, int64_t K, cudaStream_t stream,
                           bool pdl) {
    return matvec_checked(wt, W, xq, nullptr, y, N, K, stream, pdl, false);
}

// Quantize one f32 row x and multiply, in one launch; the quantized row is also
// stored to xq_out (when not null).  Fails with QMM_E_SHAPE when the row does not
// fit the kernel's shared memory, so the caller can quantize separately instead.
qmm_status matvec_fused_dispatch(int wt, const void* W, const float* x, void* xq_out, float* y, int64_t N, int64_t K,
                                 cudaStream_t stream, bool pdl) {
    if (!x) return QMM_E_NULL;
    return matvec_checked(wt, W, xq_out, x, y, N, K, stream, pdl, false);
}

// The same for G matrices sharing the row (xq_out as above).
qmm_status matvec_group_fused_dispatch(int wt, int G, const void* const* W, const int64_t* N, float* const* y,
                                       const float* x, void* xq_out, int64_t K, cudaStream_t stream, bool pdl) {
    if (!x) return QMM_E_NULL;
    return matvec_group_checked(wt, G, W, N, y, xq_out, x, K, stream, pdl, false);
}

// The same with the row RMSNormed by gamma (eps) before it is quantized.
qmm_status matvec_group_norm_dispatch(int wt, int G, const void* const* W, const int64_t* N, float* const* y,
                                      const float* x, const float* gamma, float eps, void* xq_out, int64_t K,
                                      cudaStream_t stream, bool pdl) {
    if (!x || !gamma) return QMM_E_NULL;
    return matvec_group_checked(wt, G, W, N, y, xq_out, x, K, stream, pdl, false, gamma, eps);
}

// G matrices against one quantized row (internal: alignment as for per-token rows).
qmm_status matvec_group_dispatch(int wt, int G, const void* const* W, const int64_t* N, float* const* y,
                                 const void* xq, int64_t K, cudaStream_t stream, bool pdl) {
    return matvec_group_checked(wt, G, W, N, y, xq, nullptr, K, stream, pdl, false);
}

template <int WT>
static qmm_status launch_blocksums(const void* W, const void* xq, int32_t* s, int64_t M, int64_t N, int64_t K,
                                   cudaStream_t stream) {
    using F = Fmt<WT>;
    DeviceInfo dev;
    qmm_status st = current_device(&dev);
    if (st != QMM_OK) return st;
    const uint64_t rb = (uint64_t)(K / F::BV) * F::BB;
    const uint32_t act = 128u + act_region_bytes(F::ACT, (int)K);
    int rows = (int)(16384 / rb);
    if (rows < 1) rows = 1;
    if (rows > 64) rows = 64;
    const uint64_t smem = act + align_up((uint32_t)(rows * rb + 48), 128u);
    if (smem > (uint64_t)dev.max_smem_optin) return QMM_E_SHAPE;
    if (cudaFuncSetAttribute(blocksums_kernel<WT>, cudaFuncAttributeMaxDynamicSharedMemorySize, dev.max_smem_optin) !=
        cudaSuccess)
        return QMM_E_CUDA;
    const dim3 grid((unsigned)((N + rows - 1) / rows), (unsigned)M);
    if (M > 65535) return QMM_E_SHAPE;
    blocksums_kernel<WT><<<grid, kThreads, (size_t)smem, stream>>>((const uint8_t*)W, (const uint8_t*)xq, s, (int)N,
                                                                   (int)K, rows, act);
    return launch_status();
}

}  // namespace qmm

using namespace qmm;

extern "C" {

qmm_status qmm_matvec_q4_0(const void* W, const void* xq, float* y, int64_t N, int64_t K, qmm_stream_t stream) {
    return matvec_checked(QMM_Q4_0, W, xq, nullptr, y, N, K, (cudaStream_t)stream, true, true);
}
qmm_status qmm_matvec_q8_0(const void* W, const void* xq, float* y, int64_t N, int64_t K, qmm_stream_t stream) {
    return matvec_checked(QMM_Q8_0, W, xq, nullptr, y, N, K, (cudaStream_t)stream, true, true);
}
qmm_status qmm_matvec_q4_K(const void* W, const void* xq, float* y, int64_t N, int64_t K, qmm_stream_t stream) {
    return matvec_checked(QMM_Q4_K, W, xq, nullptr, y, N, K, (cudaStream_t)stream, true, true);
}
qmm_status qmm_matvec_q6_K(const void* W, const void* xq, float* y, int64_t N, int64_t K, qmm_stream_t stream) {
    return matvec_checked(QMM_Q6_K, W, xq, nullptr, y, N, K, (cudaStream_t)stream, true, true);
}
qmm_status qmm_matvec_q2_K(const void* W, const void* xq, float* y, int64_t N, int64_t K, qmm_stream_t stream) {
    return matvec_checked(QMM_Q2_K, W, xq, nullptr, y, N, K, (cudaStream_t)stream, true, true);
}
qmm_status qmm_matvec_q4_1(const void* W, const void* xq, float* y, int64_t N, int64_t K, qmm_stream_t stream) {
    return matvec_checked(QMM_Q4_1, W, xq, nullptr, y, N, K, (cudaStream_t)stream, true, true);
}
qmm_status qmm_matvec_q5_0(const void* W, const void* xq, float* y, int64_t N, int64_t K, qmm_stream_t stream) {
    return matvec_checked(QMM_Q5_0, W, xq, nullptr, y, N, K, (cudaStream_t)stream, true, true);
}
qmm_status qmm_matvec_q5_1(const void* W, const void* xq, float* y, int64_t N, int64_t K, qmm_stream_t stream) {
    return matvec_checked(QMM_Q5_1, W, xq, nullptr, y, N, K, (cudaStream_t)stream, true, true);
}
qmm_status qmm_matvec_q5_K(const void* W, const void* xq, float* y, int64_t N, int64_t K, qmm_stream_t stream) {
    return matvec_checked(QMM_Q5_K, W, xq, nullptr, y, N, K, (cudaStream_t)stream, true, true);
}

qmm_status qmm_blocksums(int wtype, const void* W, const void* xq, int32_t* s, int64_t M, int64_t N, int64_t K,
                         qmm_stream_t stream) {
    if (act_type_of(wtype) < 0) return QMM_E_TYPE;
    if (!W || !xq || !s) return QMM_E_NULL;
    qmm_status st = check_shape(wtype, M, N, K);
    if (st != QMM_OK) return st;
    if (!aligned16(W) || !aligned16(xq) || !aligned16(s)) return QMM_E_ALIGN;
    cudaStream_t cs = (cudaStream_t)stream;
    switch (wtype) {
    case QMM_Q4_0: return launch_blocksums<QMM_Q4_0>(W, xq, s, M, N, K, cs);
    case QMM_Q8_0: return launch_blocksums<QMM_Q8_0>(W, xq, s, M, N, K, cs);
    case QMM_Q4_K: return launch_blocksums<QMM_Q4_K>(W, xq, s, M, N, K, cs);
    case QMM_Q6_K: return launch_blocksums<QMM_Q6_K>(W, xq, s, M, N, K, cs);
    case QMM_Q2_K: return launch_blocksums<QMM_Q2_K>(W, xq, s, M, N, K, cs);
    case QMM_Q4_1: return launch_blocksums<QMM_Q4_1>(W, xq, s, M, N, K, cs);
    case QMM_Q5_0: return launch_blocksums<QMM_Q5_0>(W, xq, s, M, N, K, cs);
    case QMM_Q5_1: return launch_blocksums<QMM_Q5_1>(W, xq, s, M, N, K, cs);
    case QMM_Q5_K: return launch_blocksums<QMM_Q5_K>(W, xq, s, M, N, K, cs);
    default: return QMM_E_TYPE;
    }
}

unsigned qmm_internal_matvec_error(int clear) {
    unsigned v = 0;
    cudaMemcpyFromSymbol(&v, g_matvec_error, sizeof(v));
    if (clear) {
        const unsigned z = 0;
        cudaMemcpyToSymbol(g_matvec_error, &z, sizeof(z));
    }
    return v;
}

}  // extern "C"
