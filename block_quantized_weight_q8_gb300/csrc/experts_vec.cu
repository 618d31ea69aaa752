// experts_vec.cu -- the experts' products for a few rows: every row streams the weight rows of the matrices that its
// experts' indexes name, as the decode matvec does.
//
//   gated   h[s][n] = act(Wg[e_s][n] . x) * (Wu[e_s][n] . x)          slot s = (token, choice), legs Wg and Wu
//   summed  y[t][n] = r[t][n] + sum_j w[t][j] (W[e_tj][n] . q(h[t][j]))   one leg for each choice j of token t
//
// Bound by the weights' bytes (each slot reads its experts' rows once) and, below some 20 MB, by the launch's fixed parts:
// one token through 8 of 64 experts takes 6.9 us gated (Q4_K, 1024 x 2048 twice, 18.9 MB) and 8.3 summed (Q6_K, 2048 x
// 1024, 13.8 MB), replayed from a graph; 128 choices 60 us (5 TB/s).  The unit of work is a share of the output rows
// of one slot (gated) or token (summed): the CTA streams that share's rows of every leg through its warps' rings of bulk
// copies, with the decoders and the row geometry of the matvec, keeps each leg's sums in shared memory and joins the
// legs at the end, in the order of the choices.  So the gate's activation and the weighted sum cost no launch and no
// trip through memory, and every output comes from one fixed order of operations.
#include "experts.h"
#include "matvec_kernel.cuh"

namespace qmm {

struct ExpertVec {
    const uint8_t* W0;       // [E][N] rows: the gate's weights, or the summed product's
    const uint8_t* W1;       // the up weights (gated)
    const int32_t* ids;      // [T][k]
    const uint8_t* xq;       // gated: quantized rows [T]
    const float* x;          // summed: f32 rows [T][k]
    const float* weights;    // summed: [T][k], null: 1
    const float* residual;   // summed: [T][N] or null
    float* y;                // gated [T][k][N], summed [T][N]
    int k, E, N, K, parts;
    int kind;
    int lpr, pieces, piece_units, item_segs, depth;
    uint32_t slot_bytes, act_stride, part_off, ring_off;
};

constexpr int kMaxLegs = kMaxChoices;

template <int WT, bool SU, bool GATED, bool SPLIT>
__global__ void __launch_bounds__(kMaxWarps * 32, 1) expert_vec_kernel(const __grid_constant__ ExpertVec a) {
    using F = Fmt<WT>;
    pdl_launch_dependents();
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t leg_row[kMaxLegs];  // first weight row of the leg's expert; -1: no expert
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nw = blockDim.x >> 5, depth = a.depth;
    const int unit = (int)blockIdx.x / a.parts, share = (int)blockIdx.x - unit * a.parts;  // slot or token, its share
    const int legs = GATED ? 2 : a.k;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem) + warp * depth;
    uint8_t* acts = smem + align_up(8u * nw * depth, 128u);
    float* part = reinterpret_cast<float*>(smem + a.part_off);
    uint8_t* slots = smem + a.ring_off + (size_t)warp * depth * a.slot_bytes;
    const int K = a.K, N = a.N;
    const int nd = F::ACT == QMM_Q8_0 ? K / 32 : K / 256, nsu = K / 256;
    const int ap = F::ACT == QMM_Q8_0 ? nd : q8k_pitch(nd);
    const int qbytes = SU ? SuFmt<has_su<WT>() ? WT : QMM_Q8_0>::A * nsu : (int)act_code_bytes(F::ACT, K);

    if (lane == 0) {
        for (int i = 0; i < depth; i++) mbar_init(smem_u32(&full[i]), 1);
        fence_mbar_init();
    }
    pdl_wait();  // the indexes and the rows come from earlier kernels
    for (int j = tid; j < legs; j += blockDim.x) {  // long rows leave room for one warp, whose threads are fewer than the legs
        const int e = a.ids[(int64_t)unit * (GATED ? 1 : a.k) + (GATED ? 0 : j)];
        const bool real = e >= 0 && e < a.E;
        if (e >= a.E) atomicOr(&g_matvec_error, kErrIndex);
        leg_row[j] = real ? (int64_t)e * N : -1;
    }
    __syncthreads();

    const int units = K / F::BV;
    const uint64_t rb = (uint64_t)units * F::BB;
    const int pieces = SPLIT ? a.pieces : 1;
    const SegGeom<SPLIT> geo{rb, SU ? nsu : units, pieces, a.piece_units,
                             SU ? SuFmt<has_su<WT>() ? WT : QMM_Q8_0>::W : F::BB};
    const int rq = N / a.parts, rr = N - rq * a.parts;
    const int r_begin = share * rq + min(share, rr), rows = rq + (share < rr ? 1 : 0);
    const int nseg = rows * pieces;  // segments of one leg
    const int litems = (nseg + a.item_segs - 1) / a.item_segs;
    const int nitems = litems * legs;
    const int my_items = nitems > warp ? (nitems - warp + nw - 1) / nw : 0;
    const uint64_t total = (uint64_t)a.E * (uint64_t)N * rb;
    const uint64_t total_al = total & ~15ull;
    const uint64_t pol = policy_evict_first();

    // item `it` is segments [s0, s1) of its leg's share, counted from the share's first
    auto issue = [&](int it, int slot) {
        const int leg = it / litems, s0 = (it - leg * litems) * a.item_segs, s1 = min(s0 + a.item_segs, nseg);
        const uint8_t* W = GATED && leg ? a.W1 : a.W0;
        const int64_t row0 = leg_row[leg];
        if (row0 < 0 || !QMM_IN_BOUNDS(g_matvec_error, row0 + r_begin + rows - 1, (int64_t)a.E * N)) {
            mbar_arrive_expect_tx(smem_u32(&full[slot]), 0);
            return;
        }
        const uint64_t base = (uint64_t)(row0 + r_begin) * rb;
        issue_item(W, base + geo.off(s0), base + geo.off(s1), total_al, slots + (size_t)slot * a.slot_bytes,
                   smem_u32(&full[slot]), pol, a.slot_bytes);
    };
    if (lane == 0)
        for (int i = 0; i < depth && i < my_items; i++) issue(warp + i * nw, i);

    // the activation rows, in the layout that the decoders read
    const int nthr = blockDim.x;
    auto act_of = [&](int leg, uint8_t*& aq, float*& ad, int*& as) {
        aq = acts + (size_t)leg * a.act_stride;
        ad = reinterpret_cast<float*>(aq + qbytes);
        as = reinterpret_cast<int*>(ad + nd);
    };
    uint8_t* aq;
    float* ad;
    int* as;
    if constexpr (GATED) {
        const uint8_t* row = a.xq + (uint64_t)(unit / a.k) * nd * (F::ACT == QMM_Q8_0 ? Q8_0_BB : Q8_K_BB);
        act_of(0, aq, ad, as);
        if (leg_row[0] >= 0) {
            if constexpr (F::ACT == QMM_Q8_0) {
                for (int b = tid; b < nd; b += nthr) {
                    const unsigned short* p = reinterpret_cast<const unsigned short*>(row + (size_t)b * 34);
                    uint32_t w[8];
#pragma unroll
                    for (int i = 0; i < 8; i++) w[i] = (uint32_t)p[1 + 2 * i] | ((uint32_t)p[2 + 2 * i] << 16);
                    put_act_block<WT, SU>(w, p[0], b, nd, nsu, aq, ad, as);
                }
            } else {
                unpack_q8_K_row_by(row, nd, ap, aq, ad, as, tid, nthr);
            }
        }
    } else {
        // the legs' blocks lie side by side over all threads (Q8_0) or warps, which read four before they make the first
        const float4* x4 = reinterpret_cast<const float4*>(a.x + (int64_t)unit * a.k * K);
        if constexpr (F::ACT == QMM_Q8_0) {
            for (int i = tid; i < legs * nd; i += nthr) {
                const int leg = i / nd, b = i - leg * nd;
                if (leg_row[leg] < 0) continue;
                float4 v[8];
#pragma unroll
                for (int j = 0; j < 8; j++) v[j] = x4[(size_t)i * 8 + j];
                uint32_t w[8], dbits;
                quant_q8_0_block(v, &dbits, w);
                act_of(leg, aq, ad, as);
                put_act_block<WT, SU>(w, dbits, b, nd, nsu, aq, ad, as);
            }
        } else {
            constexpr int U = 4;
            for (int i0 = warp; i0 < legs * nd; i0 += U * nw) {
                float4 v[U][2];
#pragma unroll
                for (int u = 0; u < U; u++) {
                    const int i = i0 + u * nw;
                    if (i < legs * nd && leg_row[i / nd] >= 0) v[u][0] = x4[i * 64 + 2 * lane], v[u][1] = x4[i * 64 + 2 * lane + 1];
                }
#pragma unroll
                for (int u = 0; u < U; u++) {
                    const int i = i0 + u * nw, leg = i / nd;
                    if (i >= legs * nd || leg_row[leg] < 0) continue;
                    act_of(leg, aq, ad, as);
                    quant_q8_K_lane_put(v[u][0], v[u][1], lane, i - leg * nd, ap, aq, ad, as, nullptr);
                }
            }
        }
    }
    __syncthreads();

    const int segs_per_pass = 32 / a.lpr;
    const int ssub = lane / a.lpr, li = lane % a.lpr;
    bool failed = false;
    for (int i = 0; i < my_items; i++) {
        const int slot = i % depth, it = warp + i * nw;
        const bool ok = mbar_wait_bounded(smem_u32(&full[slot]), (uint32_t)(i / depth) & 1u, kWaitLimitNs);
        if (__any_sync(0xffffffffu, !ok)) {
            if (lane == 0) atomicOr(&g_matvec_error, kErrTimeout);
            failed = true;
            break;
        }
        const int leg = it / litems, s0 = (it - leg * litems) * a.item_segs, s1 = min(s0 + a.item_segs, nseg);
        const int64_t row0 = leg_row[leg];
        const uint64_t base = (uint64_t)((row0 < 0 ? 0 : row0) + r_begin) * rb;
        const uint64_t a0 = (base + geo.off(s0)) & ~15ull;
        uint8_t* sbuf = slots + (size_t)slot * a.slot_bytes;
        const SmemBytes wv{sbuf};
        act_of(GATED ? 0 : leg, aq, ad, as);
        const ActView act{aq, ad, as, ap};
        for (int ss = s0; ss < s1; ss += segs_per_pass) {
            const int seg = ss + ssub;
            if (row0 >= 0 && seg < s1 && total > total_al && base + geo.off(seg + 1) == total) {
                // the last < 16 bytes of the weights: not reachable by a 16-byte bulk copy
                const uint8_t* W = GATED && leg ? a.W1 : a.W0;
                for (uint64_t j = total_al + li; j < total; j += a.lpr)
                    if (QMM_IN_BOUNDS(g_matvec_error, j - a0, a.slot_bytes)) sbuf[j - a0] = W[j];
            }
            __syncwarp();
            float acc = 0.0f;
            if (seg < s1 && row0 >= 0) {
                int u0 = 0, un = geo.nunit;
                if constexpr (SPLIT) {
                    const int piece = seg - (seg / pieces) * pieces;
                    u0 = min(piece * a.piece_units, geo.nunit);
                    un = min(a.piece_units, geo.nunit - u0);
                }
                const uint32_t so = (uint32_t)(base + geo.off(seg) - a0);
                const int64_t seg_end = (int64_t)so + (int64_t)un * (SU ? geo.ubytes : F::BB);
                if (!QMM_IN_BOUNDS(g_matvec_error, seg_end - 1, a.slot_bytes)) un = 0;
                if constexpr (SU) {
                    for (int u = li; u < un; u += a.lpr) {
                        const int ug = u0 + u;
                        if constexpr (WT == QMM_Q8_0) acc += su_q8_0(sbuf + so + 272u * u, aq, nsu, ug, ad + 8 * ug);
                        else if constexpr (WT == QMM_Q4_0)
                            acc += su_q4_0(sbuf + so + 144u * u, aq, nsu, ug, ad + 8 * ug, as + 8 * ug);
                        else if constexpr (has_su<WT>())
                            acc += su_q45<WT>(sbuf + so + (uint32_t)SuFmt<WT>::W * u, aq, nsu, ug, ad + 8 * ug, as + 8 * ug);
                    }
                } else {
#pragma unroll 4
                    for (int u = li; u < un; u += a.lpr)
                        acc += unit_contrib<WT>(wv, so + (uint32_t)(u * F::BB), act, u0 + u);
                }
            }
            for (int off = a.lpr >> 1; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
            if (seg < s1 && li == 0 && QMM_IN_BOUNDS(g_matvec_error, leg * nseg + seg, legs * nseg)) part[leg * nseg + seg] = acc;
        }
        __syncwarp();
        if (lane == 0 && i + depth < my_items) issue(warp + (i + depth) * nw, slot);
    }
    if (__syncthreads_or(failed ? 1 : 0)) return;
    for (int r = tid; r < rows; r += nthr) {
        const int64_t o = (int64_t)unit * N + r_begin + r;
        auto sum = [&](int leg) {
            float v = part[leg * nseg + r * pieces];
            for (int p = 1; p < pieces; p++) v += part[leg * nseg + r * pieces + p];
            return v;
        };
        if constexpr (GATED) {
            if (QMM_IN_BOUNDS(g_matvec_error, r_begin + r, N)) a.y[o] = leg_row[0] < 0 ? 0.0f : gated(a.kind, sum(0), sum(1));
        } else {
            float v = 0.0f;
            for (int j = 0; j < legs; j++)
                if (leg_row[j] >= 0) v = fmaf(a.weights ? a.weights[(int64_t)unit * a.k + j] : 1.0f, sum(j), v);
            if (QMM_IN_BOUNDS(g_matvec_error, r_begin + r, N)) a.y[o] = a.residual ? a.residual[o] + v : v;
        }
    }
}

// The launch shape: rows are cut as the matvec cuts them (that depends on the format and K alone), and the SMs are
// shared out over the units; with more units than SMs each gets one CTA.
template <int WT>
static qmm_status plan_expert_vec(const DeviceInfo& dev, int64_t unit_count, int legs, int acts, ExpertVec* a, int* nw,
                                  uint32_t* smem, bool* su) {
    using F = Fmt<WT>;
    MatvecPlan p;
    int ends[kMaxGroup];
    const int64_t one_row = 1;  // how rows are cut goes by the format and K
    const qmm_status st = plan_matvec<WT>(&one_row, 1, a->K, dev, false, false, &p, ends);
    if (st != QMM_OK) return st;
    *su = p.su;
    a->lpr = p.lpr, a->pieces = p.pieces, a->piece_units = p.piece_units, a->item_segs = p.item_segs;
    a->slot_bytes = p.slot_bytes;
    // two CTAs share an SM: while one reads its rows or joins its legs, the other streams
    int64_t parts = unit_count >= 2 * dev.sms ? 1 : (2 * dev.sms + unit_count - 1) / unit_count;
    const int64_t most = ((int64_t)a->N * p.pieces + p.item_segs - 1) / p.item_segs;
    if (parts > most) parts = most;
    if (parts > a->N) parts = a->N;
    const uint64_t half = (uint64_t)dev.smem_per_sm / 2 - (uint64_t)dev.smem_reserved - 1024;
    const uint64_t whole = (uint64_t)dev.max_smem_optin - 1024;
    a->act_stride = align_up(matvec_act_bytes(WT, F::ACT, a->K, p.su), 128u);
    const uint64_t act_bytes = (uint64_t)acts * a->act_stride;
    // a share's sums stay in shared memory: more shares where they would take a quarter of it
    const int64_t fit = (int64_t)(half / 4) / (4 * (int64_t)legs * p.pieces);
    if (fit < 1) return QMM_E_SHAPE;
    if ((a->N + parts - 1) / parts > fit) parts = (a->N + fit - 1) / fit;
    a->parts = (int)parts;
    const int64_t rows = (a->N + parts - 1) / parts;
    const uint64_t part_bytes = align_up((uint32_t)(rows * legs * p.pieces * 4), 128u);
    const uint64_t items = (uint64_t)legs * ((rows * p.pieces + p.item_segs - 1) / p.item_segs);
    const uint64_t fixed = align_up(8u * kMaxWarps * kMaxDepth, 128u) + act_bytes + part_bytes;
    for (const uint64_t cap : {half, whole}) {
        if (cap < fixed + (cap == half ? 4 : 1) * (uint64_t)p.slot_bytes) continue;
        const uint64_t ring = (cap - fixed) / p.slot_bytes;  // slots
        uint64_t w = cap == half ? 8 : kMaxWarps;
        if (w > items) w = items;
        if (w < 4) w = 4;  // the activation is read by at least four warps
        if (w > ring) w = ring;
        uint64_t d = ring / w;
        const uint64_t per = (items + w - 1) / w;
        if (d > per) d = per;
        if (d > (uint64_t)kMaxDepth) d = kMaxDepth;
        *nw = (int)w;
        a->depth = (int)d;
        a->part_off = align_up(8u * *nw * a->depth, 128u) + (uint32_t)act_bytes;
        a->ring_off = a->part_off + (uint32_t)part_bytes;
        *smem = a->ring_off + (uint32_t)(*nw * a->depth) * a->slot_bytes;
        return QMM_OK;
    }
    return QMM_E_SHAPE;
}

template <int WT, bool SU, bool GATED, bool SPLIT>
static qmm_status launch_k(const ExpertVec& a, int nw, uint32_t smem, int64_t grid, const DeviceInfo& dev, cudaStream_t stream) {
    static PerDeviceOnce once;
    const qmm_status st = once.run(dev.device, [&] {
        auto* f = expert_vec_kernel<WT, SU, GATED, SPLIT>;
        if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, dev.max_smem_optin - 1024) != cudaSuccess ||
            cudaFuncSetAttribute(f, cudaFuncAttributePreferredSharedMemoryCarveout, (int)cudaSharedmemCarveoutMaxShared) !=
                cudaSuccess)
            return QMM_E_CUDA;
        return QMM_OK;
    });
    if (st != QMM_OK) return st;
    return launch_pdl(expert_vec_kernel<WT, SU, GATED, SPLIT>, dim3((unsigned)grid), nw * 32, smem, stream, a);
}

template <int WT, bool GATED>
static qmm_status launch(ExpertVec a, int64_t unit_count, cudaStream_t stream) {
    DeviceInfo dev;
    qmm_status st = current_device(&dev);
    if (st != QMM_OK) return st;
    int nw;
    uint32_t smem;
    bool su;
    st = plan_expert_vec<WT>(dev, unit_count, GATED ? 2 : a.k, GATED ? 1 : a.k, &a, &nw, &smem, &su);
    if (st != QMM_OK) return st;
    const int64_t grid = unit_count * a.parts;
    if (grid > 0x7FFFFFFFLL) return QMM_E_SHAPE;
    if constexpr (has_su<WT>()) {
        if (su)
            return a.pieces > 1 ? launch_k<WT, true, GATED, true>(a, nw, smem, grid, dev, stream)
                                : launch_k<WT, true, GATED, false>(a, nw, smem, grid, dev, stream);
    }
    return a.pieces > 1 ? launch_k<WT, false, GATED, true>(a, nw, smem, grid, dev, stream)
                        : launch_k<WT, false, GATED, false>(a, nw, smem, grid, dev, stream);
}

template <bool GATED>
static qmm_status by_type(int wt, const ExpertVec& a, int64_t units, cudaStream_t s) {
    switch (wt) {
    case QMM_Q4_0: return launch<QMM_Q4_0, GATED>(a, units, s);
    case QMM_Q8_0: return launch<QMM_Q8_0, GATED>(a, units, s);
    case QMM_Q4_K: return launch<QMM_Q4_K, GATED>(a, units, s);
    case QMM_Q6_K: return launch<QMM_Q6_K, GATED>(a, units, s);
    case QMM_Q2_K: return launch<QMM_Q2_K, GATED>(a, units, s);
    case QMM_Q4_1: return launch<QMM_Q4_1, GATED>(a, units, s);
    case QMM_Q5_0: return launch<QMM_Q5_0, GATED>(a, units, s);
    case QMM_Q5_1: return launch<QMM_Q5_1, GATED>(a, units, s);
    case QMM_Q5_K: return launch<QMM_Q5_K, GATED>(a, units, s);
    default: return QMM_E_TYPE;
    }
}

qmm_status expert_vec_glu(int wt, int kind, const ExpertShape& s, const void* Wg, const void* Wu, const void* xq,
                          const int32_t* ids, float* h, cudaStream_t stream) {
    ExpertVec a = {};
    a.W0 = (const uint8_t*)Wg, a.W1 = (const uint8_t*)Wu, a.ids = ids, a.xq = (const uint8_t*)xq, a.y = h;
    a.k = (int)s.k, a.E = (int)s.E, a.N = (int)s.N, a.K = (int)s.K, a.kind = kind;
    return by_type<true>(wt, a, s.T * s.k, stream);
}

qmm_status expert_vec_sum(int wt, const ExpertShape& s, const void* W, const float* x, const int32_t* ids,
                          const float* weights, const float* residual, float* y, cudaStream_t stream) {
    ExpertVec a = {};
    a.W0 = (const uint8_t*)W, a.ids = ids, a.x = x, a.weights = weights, a.residual = residual, a.y = y;
    a.k = (int)s.k, a.E = (int)s.E, a.N = (int)s.N, a.K = (int)s.K;
    return by_type<false>(wt, a, s.T, stream);
}

}  // namespace qmm

extern "C" unsigned qmm_internal_expert_vec_error(int clear) {
    unsigned v = 0;
    cudaMemcpyFromSymbol(&v, qmm::g_matvec_error, sizeof(v));
    if (clear) {
        const unsigned z = 0;
        cudaMemcpyToSymbol(qmm::g_matvec_error, &z, sizeof(z));
    }
    return v;
}
