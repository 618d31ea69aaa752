// experts.cu -- the entry points of the experts' products: checks, workspaces and the choice of the path.
#include "experts.h"
#include "experts_mma.h"

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

// The workspace of the tensor-core path: the plan (rows sorted by expert, tiles), the activation records, and one f32 row
// of products for each choice, which the other path may use too.
struct Scratch {
    size_t order, tiles, records, products, bytes;
    int64_t tiles_most;
};
static Scratch scratch_of(const ExpertShape& s) {
    const int64_t S = s.T * s.k;
    Scratch l;
    l.tiles_most = S / kTileRows + (S < s.E ? S : s.E);
    auto up = [](size_t v) { return (v + 127) / 128 * 128; };
    l.order = 128;  // the number of tiles lies at 0
    l.tiles = l.order + up((size_t)S * 4);
    l.records = l.tiles + up((size_t)l.tiles_most * sizeof(ExpertTile));
    l.products = l.records + up((size_t)S * (size_t)((s.K + 255) / 256) * kRecord);
    l.bytes = l.products + (size_t)S * (size_t)s.N * 4;
    return l;
}

// Block 0 sorts the choices by their expert and cuts each expert's into tiles; the others write the activation records
// (from 8-bit rows, or quantizing f32 rows) and, for gated products, the zero rows of choices that are not there.
// Counting and placing use shared-memory counters, one addition for a warp's choices of one expert; the order within an
// expert varies from run to run, and no result depends on it (a row's sums do not meet another row's).
struct Prepare {
    const int32_t* ids;
    const uint8_t* xq;  // [T] rows, or
    const float* x;     // [T][k] f32 rows
    float* h;           // gated: [T][k][N], else null
    int32_t* ntiles;
    int32_t* order;
    ExpertTile* tiles;
    uint8_t* records;
    int S, k, E, N, K;
};
constexpr int kPrepThreads = 512;

__device__ void plan_tiles(const Prepare& a, int* count, int* start) {
    const int tid = threadIdx.x, lane = tid & 31;
    for (int e = tid; e < a.E; e += kPrepThreads) count[e] = 0;
    __syncthreads();
    const int Sr = (a.S + 31) & ~31;  // whole warps
    for (int i = tid; i < Sr; i += kPrepThreads) {
        const int e = i < a.S ? a.ids[i] : -1;
        if (e >= a.E) atomicOr(&g_experts_error, kErrIndex);
        const bool real = e >= 0 && e < a.E;
        const unsigned same = __match_any_sync(0xffffffffu, real ? e : -1);
        if (real && lane == __ffs(same) - 1) atomicAdd(&count[e], __popc(same));
    }
    __syncthreads();
    if (tid < 32) {  // exclusive sums of the counts and of the experts' tiles
        int rows = 0, tiles = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane, c = e < a.E ? count[e] : 0, t = (c + kTileRows - 1) / kTileRows;
            int cs = c, ts = t;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int co = __shfl_up_sync(0xffffffffu, cs, off), to = __shfl_up_sync(0xffffffffu, ts, off);
                if (lane >= off) cs += co, ts += to;
            }
            if (e < a.E) start[e] = rows + cs - c;
            for (int j = 0, at = tiles + ts - t; j < t; j++)
                a.tiles[at + j] = {e, rows + cs - c + j * kTileRows, min(c - j * kTileRows, kTileRows), 0};
            rows += __shfl_sync(0xffffffffu, cs, 31), tiles += __shfl_sync(0xffffffffu, ts, 31);
        }
        if (lane == 0) *a.ntiles = tiles;
    }
    __syncthreads();
    for (int i = tid; i < Sr; i += kPrepThreads) {
        const int e = i < a.S ? a.ids[i] : -1;
        const bool real = e >= 0 && e < a.E;
        const unsigned same = __match_any_sync(0xffffffffu, real ? e : -1);
        const int first = __ffs(same) - 1;
        int at = 0;
        if (real && lane == first) at = atomicAdd(&start[e], __popc(same));
        at = __shfl_sync(0xffffffffu, at, first) + __popc(same & ((1u << lane) - 1));
        if (real && QMM_IN_BOUNDS(g_experts_error, at, a.S)) a.order[at] = i;
    }
}

template <int ACT, bool FROM_F32>
__global__ void __launch_bounds__(kPrepThreads) prepare_kernel(const __grid_constant__ Prepare a) {
    __shared__ int count[kMaxExperts], start[kMaxExperts];
    pdl_launch_dependents();
    pdl_wait();
    if (blockIdx.x == 0) {
        plan_tiles(a, count, start);
        return;
    }
    const int lane = threadIdx.x & 31;
    const int64_t warp = ((int64_t)(blockIdx.x - 1) * kPrepThreads + threadIdx.x) >> 5;
    const int64_t warps = (int64_t)(gridDim.x - 1) * (kPrepThreads / 32);
    const int nchunks = (a.K + 255) / 256;
    const int64_t total = (int64_t)(FROM_F32 ? a.S : a.S / a.k) * nchunks;
    for (int64_t i = warp; i < total; i += warps) {
        const int64_t row = i / nchunks;
        const int c = (int)(i - row * nchunks);
        if (FROM_F32) {
            const int e = a.ids[row];
            if (e < 0 || e >= a.E) continue;  // the row has no effect
        }
        // lane l: values 8l .. 8l + 7 of the chunk
        const bool in = 256 * c + 8 * lane < a.K;
        uint32_t w0 = 0, w1 = 0, dbits = 0;
        float d = 0.0f;
        if constexpr (FROM_F32) {
            const float4* x4 = reinterpret_cast<const float4*>(a.x + row * a.K) + 64 * c + 2 * lane;
            const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
            float4 v[2] = {in ? x4[0] : zero, in ? x4[1] : zero};
            if constexpr (ACT == QMM_Q8_0) {
                uint32_t w[8];
                quant_q8_0_block_lanes<4>(v, lane & 3, &dbits, w);
                // the first lane of four has all words; each lane keeps its own two
                w0 = w[0], w1 = w[1];
            } else {
                uint32_t pair;
                quant_q8_K_core(v[0], v[1], &d, &w0, &w1, &pair);
            }
        } else if constexpr (ACT == QMM_Q8_0) {
            if (in) {
                const unsigned short* p =
                    reinterpret_cast<const unsigned short*>(a.xq + (row * (a.K / 32) + 8 * c + (lane >> 2)) * Q8_0_BB);
                const unsigned short* q = p + 1 + 4 * (lane & 3);
                dbits = p[0], w0 = q[0] | (uint32_t)q[1] << 16, w1 = q[2] | (uint32_t)q[3] << 16;
            }
        } else {
            const uint32_t* p = reinterpret_cast<const uint32_t*>(a.xq + (row * nchunks + c) * Q8_K_BB);
            d = __uint_as_float(p[0]), w0 = p[1 + 2 * lane], w1 = p[2 + 2 * lane];
        }
        int sum = dp4a(w0, 0x01010101u, dp4a(w1, 0x01010101u, 0));
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        if (!QMM_IN_BOUNDS(g_experts_error, i, total)) continue;
        uint8_t* rec = a.records + i * kRecord;
        *reinterpret_cast<uint2*>(rec + 8 * lane) = make_uint2(w0 ^ 0x80808080u, w1 ^ 0x80808080u);
        if (!(lane & 1)) st_u16(rec + 272 + lane, f2h_bits((float)sum));
        if (ACT == QMM_Q8_0 && !(lane & 3)) st_u16(rec + 256 + (lane >> 1), dbits);
        if (ACT == QMM_Q8_K && lane == 0) *reinterpret_cast<float*>(rec + 256) = d;
    }
    if (a.h != nullptr)
        for (int64_t s = warp; s < a.S; s += warps) {
            const int e = a.ids[s];
            if (e >= 0 && e < a.E) continue;
            for (int n = lane; n < a.N; n += 32) a.h[s * a.N + n] = 0.0f;
        }
}

static qmm_status prepare(int act, const Prepare& a, cudaStream_t stream) {
    DeviceInfo dev;
    const qmm_status st = current_device(&dev);
    if (st != QMM_OK) return st;
    const int64_t items = (int64_t)(a.x ? a.S : a.S / a.k) * ((a.K + 255) / 256) + (a.h ? a.S / 8 : 0);
    const int64_t want = (items + kPrepThreads / 32 - 1) / (kPrepThreads / 32), most = (int64_t)dev.sms * 4 - 1;
    const dim3 grid((unsigned)(1 + (want < most ? want : most)));
    if (act == QMM_Q8_0)
        return a.x ? launch_pdl(prepare_kernel<QMM_Q8_0, true>, grid, kPrepThreads, 0, stream, a)
                   : launch_pdl(prepare_kernel<QMM_Q8_0, false>, grid, kPrepThreads, 0, stream, a);
    return a.x ? launch_pdl(prepare_kernel<QMM_Q8_K, true>, grid, kPrepThreads, 0, stream, a)
               : launch_pdl(prepare_kernel<QMM_Q8_K, false>, grid, kPrepThreads, 0, stream, a);
}

static qmm_status expert_mma(int wt, const ExpertMma& a, bool gate, int64_t tiles_most, cudaStream_t stream) {
    if (wt == QMM_Q4_0 || wt == QMM_Q8_0 || wt == QMM_Q4_1) return expert_mma_32(wt, a, gate, tiles_most, stream);
    if (wt == QMM_Q5_0 || wt == QMM_Q5_1 || wt == QMM_Q5_K) return expert_mma_five(wt, a, gate, tiles_most, stream);
    return expert_mma_k(wt, a, gate, tiles_most, stream);
}

// Both steps on the tensor-core path: h (gated) or the choices' products.
static qmm_status on_tensor_cores(int wt, int kind, const ExpertShape& s, const void* W0, const void* W1, const void* xq,
                                  const float* x, const int32_t* ids, float* out, uint8_t* scratch, cudaStream_t stream) {
    const Scratch l = scratch_of(s);
    const bool gate = W1 != nullptr;
    Prepare p = {};
    p.ids = ids, p.xq = (const uint8_t*)xq, p.x = x, p.h = gate ? out : nullptr;
    p.ntiles = reinterpret_cast<int32_t*>(scratch), p.order = reinterpret_cast<int32_t*>(scratch + l.order);
    p.tiles = reinterpret_cast<ExpertTile*>(scratch + l.tiles), p.records = scratch + l.records;
    p.S = (int)(s.T * s.k), p.k = (int)s.k, p.E = (int)s.E, p.N = (int)s.N, p.K = (int)s.K;
    const qmm_status st = prepare(act_type_of(wt), p, stream);
    if (st != QMM_OK) return st;
    ExpertMma a = {};
    a.W0 = (const uint8_t*)W0, a.W1 = (const uint8_t*)W1, a.records = p.records, a.order = p.order, a.tiles = p.tiles;
    a.ntiles = p.ntiles, a.y = out, a.out_values = s.T * s.k * s.N, a.per_row = x ? 1 : (int)s.k;
    a.E = (int)s.E, a.N = (int)s.N, a.K = (int)s.K, a.kind = kind;
    return expert_mma(wt, a, gate, l.tiles_most, stream);
}

// Which calls take the tensor cores.
static bool many_rows(const ExpertShape& s) {
    return s.T * s.k >= 32 && scratch_of(s).tiles_most * ((s.N + 63) / 64) <= kMaxDim;
}

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
    return check_experts(wtype, s) == QMM_OK ? scratch_of(s).bytes : 0;
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
    if (scratch_bytes < scratch_of(s).bytes) return QMM_E_SCRATCH;
    if (many_rows(s))
        return on_tensor_cores(wtype, kind, s, Wg, Wu, xq, nullptr, ids, h, (uint8_t*)scratch, (cudaStream_t)stream);
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
    if (scratch_bytes < scratch_of(s).bytes) return QMM_E_SCRATCH;
    cudaStream_t cs = (cudaStream_t)stream;
    float* p = reinterpret_cast<float*>((uint8_t*)scratch + scratch_of(s).products);
    if (many_rows(s)) {
        const qmm_status all = on_tensor_cores(wtype, 0, s, W, nullptr, nullptr, h, ids, p, (uint8_t*)scratch, cs);
        return all != QMM_OK ? all : combine(s, p, ids, weights, residual, y, cs);
    }
    const qmm_status fused = expert_vec_sum(wtype, s, W, h, ids, weights, residual, y, cs);
    if (fused != QMM_E_SHAPE) return fused;
    // a token's rows do not fit one SM: choice by choice, then the sum
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
