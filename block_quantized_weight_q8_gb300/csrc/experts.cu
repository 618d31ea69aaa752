// experts.cu -- the entry points of the experts' products: checks, workspaces and the choice of the path.
#include <math.h>

#include "experts.h"
#include "experts_mma.h"
#include "tc_device.cuh"

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

// The workspace of the tensor-core path: the plan (rows sorted by expert, tiles), the activation operands, and one f32 row
// of products for each choice, which the other path may use too.
struct Scratch {
    size_t order, tiles, operand, products, bytes;
    int64_t tiles_most;
};
static Scratch scratch_of(int wt, const ExpertShape& s) {
    const int64_t S = s.T * s.k;
    Scratch l;
    l.tiles_most = S / kTileRows + (S < s.E ? S : s.E);
    auto up = [](size_t v) { return (v + 127) / 128 * 128; };
    l.order = 128;  // the number of tiles lies at 0
    l.tiles = l.order + up((size_t)S * 4);
    l.operand = l.tiles + up((size_t)l.tiles_most * sizeof(ExpertTile));
    // each expert's rows are made a multiple of 16
    const size_t rows = (size_t)(S + 15 * (S < s.E ? S : s.E)), chunks = (size_t)((s.K + 255) / 256);
    l.products = l.operand + up(rows * chunks * (size_t)operand_bytes(act_type_of(wt)));
    l.bytes = l.products + (size_t)S * (size_t)s.N * 4;
    return l;
}

struct Prepare {
    const int32_t* ids;
    const uint8_t* xq;  // [T] rows, or
    const float* x;     // [T][k] f32 rows
    float* h;           // gated: [T][k][N], else null
    int32_t* ntiles;
    int32_t* order;
    ExpertTile* tiles;
    uint8_t* operand;
    int S, k, E, N, K;
    int spare;  // Q8_0 rows: act_spare of the weights
};
__device__ __forceinline__ __half2 half2_of(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }
__device__ __forceinline__ uint32_t bits_of(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
constexpr int kPlanThreads = 1024, kOperandThreads = 256;

// Sorts the choices by their expert and cuts each expert's into tiles.  Counting and placing use shared-memory counters,
// where there are few experts one addition for a warp's choices of one; the order within an expert varies from run to run,
// and no result depends on it (a row's sums do not meet another row's).  One CTA; its loads are issued eight at a time
// (one by one, each waiting for the counter of the one before, 16384 choices took 34 us; so 13.5, 256 choices 4).
constexpr int kFewExperts = 3;
__device__ __forceinline__ int next_place(int* counter, int e, int lane, int E) {
    if (E > kFewExperts) return e >= 0 ? atomicAdd(&counter[e], 1) : 0;
    int at = 0;
    for (int i = 0; i < E; i++) {
        const unsigned same = __ballot_sync(0xffffffffu, e == i);
        int base = 0;
        if (lane == 0 && same) base = atomicAdd(&counter[i], __popc(same));
        base = __shfl_sync(0xffffffffu, base, 0);
        if (e == i) at = base + __popc(same & ((1u << lane) - 1));
    }
    return at;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ Prepare a) {
    __shared__ int count[kMaxExperts], start[kMaxExperts];
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31;
    for (int e = tid; e < a.E; e += kPlanThreads) count[e] = 0;
    __syncthreads();
    constexpr int U = 8;
    auto read = [&](int i0, int (&e)[U]) {  // the choices i0 + tid, + 1024, ...; -1: none
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int64_t i = (int64_t)i0 + u * kPlanThreads + tid;
            e[u] = i < a.S ? a.ids[i] : -1;
        }
    };
    for (int64_t i0 = 0; i0 < a.S; i0 += U * kPlanThreads) {
        int e[U];
        read((int)i0, e);
#pragma unroll
        for (int u = 0; u < U; u++) {
            if (i0 + u * kPlanThreads >= a.S) break;
            if (e[u] >= a.E) atomicOr(&g_experts_error, kErrIndex);
            next_place(count, e[u] < a.E ? e[u] : -1, lane, a.E);
        }
    }
    __syncthreads();
    if (tid < 32) {  // exclusive sums of the counts, of the operands' rows and of the experts' tiles
        int rows = 0, padded = 0, tiles = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane, c = e < a.E ? count[e] : 0, p = (c + 15) & ~15, t = (c + kTileRows - 1) / kTileRows;
            int cs = c, ps = p, ts = t;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int co = __shfl_up_sync(0xffffffffu, cs, off), po = __shfl_up_sync(0xffffffffu, ps, off),
                          to = __shfl_up_sync(0xffffffffu, ts, off);
                if (lane >= off) cs += co, ps += po, ts += to;
            }
            if (e < a.E) start[e] = rows + cs - c;
            for (int j = 0, at = tiles + ts - t; j < t; j++)
                a.tiles[at + j] = {e, rows + cs - c + j * kTileRows, min(c - j * kTileRows, kTileRows), padded + ps - p + j * kTileRows};
            rows += __shfl_sync(0xffffffffu, cs, 31), padded += __shfl_sync(0xffffffffu, ps, 31);
            tiles += __shfl_sync(0xffffffffu, ts, 31);
        }
        if (lane == 0) *a.ntiles = tiles;
    }
    __syncthreads();
    for (int64_t i0 = 0; i0 < a.S; i0 += U * kPlanThreads) {
        int e[U];
        read((int)i0, e);
#pragma unroll
        for (int u = 0; u < U; u++) {
            if (i0 + u * kPlanThreads >= a.S) break;
            const int mine = e[u] < a.E ? e[u] : -1, at = next_place(start, mine, lane, a.E);
            if (mine >= 0 && QMM_IN_BOUNDS(g_experts_error, at, a.S)) a.order[at] = (int)i0 + u * kPlanThreads + tid;
        }
    }
}

// The tiles' activation operands, from 8-bit rows or from f32 rows (quantized by the activations' rule on the way), and,
// for gated products, the zero rows of choices that are not there.  A warp makes a chunk of 8 rows at a time, lane 4 r + q
// the values 8 q .. 8 q + 7 of each block of row r: its 16-byte stores lie side by side.  Bound by what it writes, 2 (Q8_K)
// or 4 bytes a value, which stays in the L2 (16384 rows of 2048 from 8-bit rows: 67 MB in 24 us), and for few rows by its
// launch (256 rows of 2048: 11 us).
template <int ACT, bool FROM_F32>
__global__ void __launch_bounds__(kOperandThreads) operand_kernel(const __grid_constant__ Prepare a) {
    constexpr int TERMS = operand_terms(ACT);
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, row = lane >> 2, kq = lane & 3;
    const int warp = (blockIdx.x * kOperandThreads + threadIdx.x) >> 5, warps = gridDim.x * (kOperandThreads / 32);
    const int nchunks = (a.K + 255) / 256;
    const int64_t total = (int64_t)*a.ntiles * (kTileRows / 8) * nchunks;
    for (int64_t item = warp; item < total; item += warps) {
        const int tile = (int)(item / (kTileRows / 8 * nchunks)), rest = (int)(item - (int64_t)tile * (kTileRows / 8 * nchunks));
        const int g = rest / nchunks, c = rest - g * nchunks;
        const ExpertTile t = a.tiles[tile];
        const int rows = (t.count + 15) & ~15;
        if (8 * g >= rows) continue;
        const bool real = 8 * g + row < t.count;
        const int64_t slot = real ? a.order[t.first + 8 * g + row] : 0;
        const int blocks = min(8, a.K / 32 - 8 * c);
        uint2 w[8];         // this lane's codes
        uint32_t dbits[8];  // Q8_0: the blocks' scales
        float d = 0.0f;     // Q8_K: the chunk's
        if constexpr (FROM_F32) {
            const float4* x4 = reinterpret_cast<const float4*>(a.x + slot * a.K) + 64 * c + 2 * kq;
            const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
            float4 v[8][2];
#pragma unroll
            for (int b = 0; b < 8; b++)
#pragma unroll
                for (int i = 0; i < 2; i++) v[b][i] = real && b < blocks ? x4[8 * b + i] : zero;
            if constexpr (ACT == QMM_Q8_0) {
#pragma unroll
                for (int b = 0; b < 8; b++) {
                    uint32_t u[8];
                    quant_q8_0_block_lanes<4>(v[b], kq, &dbits[b], u);
                    w[b] = make_uint2(u[0], u[1]);  // every lane's own two words
                }
            } else {
                float amax = 0.0f;
#pragma unroll
                for (int b = 0; b < 8; b++)
#pragma unroll
                    for (int i = 0; i < 2; i++)
                        amax = fmaxf(amax, fmaxf(fmaxf(fabsf(v[b][i].x), fabsf(v[b][i].y)), fmaxf(fabsf(v[b][i].z), fabsf(v[b][i].w))));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                d = __fdiv_rn(amax, 127.0f);
                const float id = amax != 0.0f ? __fdiv_rn(127.0f, amax) : 0.0f;
                auto code = [&](float f) { return (uint32_t)clampi(__float2int_rn(__fmul_rn(f, id)), -128, 127) & 0xFFu; };
                auto word = [&](float4 f) { return code(f.x) | code(f.y) << 8 | code(f.z) << 16 | code(f.w) << 24; };
#pragma unroll
                for (int b = 0; b < 8; b++) w[b] = make_uint2(word(v[b][0]), word(v[b][1]));
            }
        } else if constexpr (ACT == QMM_Q8_0) {
#pragma unroll
            for (int b = 0; b < 8; b++) {
                w[b] = make_uint2(0u, 0u), dbits[b] = 0;
                if (real && b < blocks) {
                    const unsigned short* p =
                        reinterpret_cast<const unsigned short*>(a.xq + (slot / a.k * (a.K / 32) + 8 * c + b) * Q8_0_BB);
                    const unsigned short* q = p + 1 + 4 * kq;
                    dbits[b] = p[0];
                    w[b] = make_uint2(q[0] | (uint32_t)q[1] << 16, q[2] | (uint32_t)q[3] << 16);
                }
            }
        } else {
            const uint32_t* p = reinterpret_cast<const uint32_t*>(a.xq + (slot / a.k * nchunks + c) * Q8_K_BB);
            if (real) d = __uint_as_float(p[0]);
#pragma unroll
            for (int b = 0; b < 8; b++) w[b] = real ? make_uint2(p[1 + 8 * b + 2 * kq], p[2 + 8 * b + 2 * kq]) : make_uint2(0u, 0u);
        }
        uint32_t f = 0;  // Q8_0: the run's power of two
        float scale = d;
        if constexpr (ACT == QMM_Q8_0) {
            uint32_t top = 0;
#pragma unroll
            for (int b = 0; b < 8; b++) top = max(top, dbits[b] & 0x7FFFu);
            const int shift = run_shift(top, a.spare);
            f = (uint32_t)(shift + 15) << 10;
            scale = __int_as_float((127 - shift) << 23);
        }
        if (!QMM_IN_BOUNDS(g_experts_error, (int64_t)t.at + 8 * g + row, (int64_t)a.S + 15 * min(a.S, a.E))) continue;
        uint8_t* const base = a.operand + ((int64_t)t.at * nchunks + (int64_t)c * rows) * operand_bytes(ACT);
        uint8_t* const at = base + g * 512 + kq * 128 + row * 16;
        uint32_t sums[8], lows[8];  // groups 2 b and 2 b + 1
#pragma unroll
        for (int b = 0; b < 8; b++) {
            int s = dp4a(w[b].x, 0x01010101u, dp4a(w[b].y, 0x01010101u, 0));
            s += __shfl_xor_sync(0xffffffffu, s, 1);
            const int other = __shfl_xor_sync(0xffffffffu, s, 2);
            sums[b] = f2h_bits((float)(kq < 2 ? s : other)) | f2h_bits((float)(kq < 2 ? other : s)) << 16;
            const uint32_t x = w[b].x ^ 0x80808080u, y = w[b].y ^ 0x80808080u;
            uint4 v = make_uint4(h2_sub(bytes_to_h2(x, 0x5140), 0x64806480u), h2_sub(bytes_to_h2(x, 0x7362), 0x64806480u),
                                 h2_sub(bytes_to_h2(y, 0x5140), 0x64806480u), h2_sub(bytes_to_h2(y, 0x7362), 0x64806480u));
            if constexpr (ACT == QMM_Q8_0) {
                const __half2 dh = __hmul2(half2_of(dbits[b] * 0x10001u), half2_of(f * 0x10001u));
                auto two = [&](uint32_t& u, uint32_t& l) {
                    const __half2 h = __hmul2(dh, half2_of(u));
                    l = bits_of(__hfma2(dh, half2_of(u), __hneg2(h)));
                    u = bits_of(h);
                };
                uint4 l;
                two(v.x, l.x), two(v.y, l.y), two(v.z, l.z), two(v.w, l.w);
                two(sums[b], lows[b]);
                if (b < blocks) *reinterpret_cast<uint4*>(at + (2 * b + 1) * 64 * rows) = l;
            }
            if (b < blocks) *reinterpret_cast<uint4*>(at + b * TERMS * 64 * rows) = v;
        }
        // the sums: lanes 0, 1 of a row write hi, 2, 3 (two terms) lo
        uint8_t* const under = base + 8 * TERMS * 64 * rows;
        if (kq < 2 * TERMS) {
            const uint32_t* from = kq < 2 ? sums : lows;
            const bool second = kq & 1;
            *reinterpret_cast<uint4*>(under + (kq >> 1) * 32 * rows + g * 256 + (kq & 1) * 128 + row * 16) =
                make_uint4(second ? from[4] : from[0], second ? from[5] : from[1], second ? from[6] : from[2], second ? from[7] : from[3]);
        }
        if (kq == 0) *reinterpret_cast<float*>(under + TERMS * 32 * rows + (8 * g + row) * 4) = scale;
    }
    if (a.h != nullptr)
        for (int64_t s = warp; s < a.S; s += warps) {
            const int e = a.ids[s];
            if (e >= 0 && e < a.E) continue;
            for (int n = lane; n < a.N; n += 32) a.h[s * a.N + n] = 0.0f;
        }
}

static qmm_status prepare(int act, const Prepare& a, int64_t tiles_most, cudaStream_t stream) {
    DeviceInfo dev;
    qmm_status st = current_device(&dev);
    if (st == QMM_OK) st = launch_pdl(plan_kernel, dim3(1), kPlanThreads, 0, stream, a);
    if (st != QMM_OK) return st;
    const int64_t items = tiles_most * (kTileRows / 8) * ((a.K + 255) / 256);
    const int64_t want = (items + kOperandThreads / 32 - 1) / (kOperandThreads / 32), most = (int64_t)dev.sms * 4;
    const dim3 grid((unsigned)(want < most ? want : most));
    if (act == QMM_Q8_0)
        return a.x ? launch_pdl(operand_kernel<QMM_Q8_0, true>, grid, kOperandThreads, 0, stream, a)
                   : launch_pdl(operand_kernel<QMM_Q8_0, false>, grid, kOperandThreads, 0, stream, a);
    return a.x ? launch_pdl(operand_kernel<QMM_Q8_K, true>, grid, kOperandThreads, 0, stream, a)
               : launch_pdl(operand_kernel<QMM_Q8_K, false>, grid, kOperandThreads, 0, stream, a);
}

static qmm_status expert_mma(int wt, const ExpertMma& a, bool gate, int64_t tiles_most, cudaStream_t stream) {
    if (wt == QMM_Q4_0 || wt == QMM_Q8_0 || wt == QMM_Q4_1) return expert_mma_32(wt, a, gate, tiles_most, stream);
    if (wt == QMM_Q5_0 || wt == QMM_Q5_1 || wt == QMM_Q5_K) return expert_mma_five(wt, a, gate, tiles_most, stream);
    return expert_mma_k(wt, a, gate, tiles_most, stream);
}

// Both steps on the tensor-core path: h (gated) or the choices' products.
static qmm_status on_tensor_cores(int wt, int kind, const ExpertShape& s, const void* W0, const void* W1, const void* xq,
                                  const float* x, const int32_t* ids, float* out, uint8_t* scratch, cudaStream_t stream) {
    const Scratch l = scratch_of(wt, s);
    const bool gate = W1 != nullptr;
    Prepare p = {};
    p.ids = ids, p.xq = (const uint8_t*)xq, p.x = x, p.h = gate ? out : nullptr;
    p.ntiles = reinterpret_cast<int32_t*>(scratch), p.order = reinterpret_cast<int32_t*>(scratch + l.order);
    p.tiles = reinterpret_cast<ExpertTile*>(scratch + l.tiles), p.operand = scratch + l.operand;
    p.spare = act_spare(wt);
    p.S = (int)(s.T * s.k), p.k = (int)s.k, p.E = (int)s.E, p.N = (int)s.N, p.K = (int)s.K;
    const qmm_status st = prepare(act_type_of(wt), p, l.tiles_most, stream);
    if (st != QMM_OK) return st;
    ExpertMma a = {};
    a.W0 = (const uint8_t*)W0, a.W1 = (const uint8_t*)W1, a.operand = p.operand, a.order = p.order, a.tiles = p.tiles;
    a.ntiles = p.ntiles, a.y = out, a.out_values = s.T * s.k * s.N;
    a.E = (int)s.E, a.N = (int)s.N, a.K = (int)s.K, a.kind = kind;
    return expert_mma(wt, a, gate, l.tiles_most, stream);
}

// Which calls take the tensor cores: those for which they take less time, by what both paths were measured to cost (us).
// The other path reads each choice's weights, 5.5 MB a us (half of what it reads several times comes from the L2), or
// decodes them block by block where 32-value rows are not of 256s, 1.5; the tensor cores go over the tiles in waves of one
// an SM, a chunk of 256 values in 1.6 (one-term weights) or 2.3.  Measured, other path / tensor cores: Q4_K, 64 experts of
// 2048 -> 1024 twice, 128 choices 60 / 70, 256 101 / 84; Q8_0, 8 experts of 4096 -> 4096 twice, 16 choices 61 / 127, 32
// 180 / 152; Q6_K, 64 experts of 1024 -> 2048, 128 choices 41 / 61, 256 111 / 73; Q5_1, 32 experts of 1408 -> 2048, 32
// choices 41 / 50, 64 74 / 61.  Of 223 calls (all types, 4 to 16 experts, rows of 768 to 4096, 2 to 2048 choices) all but
// two took at most 1.25 times the better path's time.  The rule knows the number of choices, not how they fall to the
// experts: it counts a partial tile for each of min(choices, experts).
static bool many_rows(int wt, const ExpertShape& s, bool gate) {
    DeviceInfo dev;
    if (current_device(&dev) != QMM_OK) return false;
    const double S = (double)(s.T * s.k), blocks = gate ? 64.0 : 128.0;
    const int64_t most = scratch_of(wt, s).tiles_most * ((s.N + 63) / 64);
    if (most > kMaxDim) return false;
    const double bytes = S * (gate ? 2.0 : 1.0) * (double)s.N * (double)row_bytes_of(wt, s.K);
    const double other = 6.0 + bytes / (act_type_of(wt) == QMM_Q8_0 && s.K % 256 ? 1.5e6 : 5.5e6);
    const double tiles = (S / kTileRows + (S < (double)s.E ? S : (double)s.E)) * ceil((double)s.N / blocks);
    const bool one_term = wt == QMM_Q4_K || wt == QMM_Q5_K || wt == QMM_Q2_K;
    const double tensor = 12.0 + ceil(tiles / dev.sms) * ceil((double)s.K / 256.0) * (one_term ? 1.6 : 2.3);
    return tensor < other;
}

// y[t][n] = residual[t][n] + sum_j weights[t][j] p[t][j][n] over the choices that are there, in their order.  Bound by
// memory: 4 (k + 2) bytes a value (2048 tokens of 8 choices of 2048: 168 MB in 30 us, 5.5 TB/s).  V values a thread: 4
// where N is a multiple of it.
template <int V>
__global__ void __launch_bounds__(256) combine_kernel(const float* __restrict__ p, const int32_t* __restrict__ ids,
                                                      const float* __restrict__ weights, const float* residual, float* y,
                                                      int T, int k, int E, int N) {
    pdl_launch_dependents();
    pdl_wait();
    const int64_t total = (int64_t)T * (N / V), step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += step) {
        const int64_t t = i / (N / V), at = i * V;
        const int n = (int)(at - t * N);
        float v[V] = {};
        for (int j0 = 0; j0 < k; j0 += 4) {
            float u[4][V], w[4];
#pragma unroll
            for (int j = 0; j < 4; j++) {  // four choices' loads at a time
                const int64_t c = t * k + j0 + j;
                const int e = j0 + j < k ? ids[c] : -1;
                const bool real = e >= 0 && e < E;
                w[j] = !real ? 0.0f : weights ? weights[c] : 1.0f;
                if constexpr (V == 4) {
                    const float4 q = real ? *reinterpret_cast<const float4*>(p + c * N + n) : make_float4(0.f, 0.f, 0.f, 0.f);
                    u[j][0] = q.x, u[j][1] = q.y, u[j][2] = q.z, u[j][3] = q.w;
                } else {
                    u[j][0] = real ? p[c * N + n] : 0.0f;
                }
            }
#pragma unroll
            for (int j = 0; j < 4; j++)
#pragma unroll
                for (int q = 0; q < V; q++) v[q] = fmaf(w[j], u[j][q], v[q]);
        }
        if (!QMM_IN_BOUNDS(g_experts_error, i, total)) continue;
        if constexpr (V == 4) {
            float4 r = residual ? *reinterpret_cast<const float4*>(residual + at) : make_float4(0.f, 0.f, 0.f, 0.f);
            *reinterpret_cast<float4*>(y + at) = make_float4(r.x + v[0], r.y + v[1], r.z + v[2], r.w + v[3]);
        } else {
            y[at] = residual ? residual[at] + v[0] : v[0];
        }
    }
}

static qmm_status combine(const ExpertShape& s, const float* p, const int32_t* ids, const float* weights, const float* residual,
                          float* y, cudaStream_t stream) {
    DeviceInfo dev;
    const qmm_status st = current_device(&dev);
    if (st != QMM_OK) return st;
    const int64_t each = s.N % 4 ? 1 : 4, want = (s.T * s.N / each + 255) / 256, most = (int64_t)dev.sms * 8;
    return launch_pdl(s.N % 4 ? combine_kernel<1> : combine_kernel<4>, dim3((unsigned)(want < most ? want : most)), 256, 0, stream,
                      p, ids, weights, residual, y, (int)s.T, (int)s.k, (int)s.E, (int)s.N);
}

}  // namespace qmm

using namespace qmm;

extern "C" {

size_t qmm_experts_scratch_bytes(int wtype, int64_t T, int64_t k, int64_t E, int64_t N, int64_t K) {
    const ExpertShape s{T, k, E, N, K};
    return check_experts(wtype, s) == QMM_OK ? scratch_of(wtype, s).bytes : 0;
}

int qmm_experts_path(int wtype, int gated, int64_t T, int64_t k, int64_t E, int64_t N, int64_t K) {
    const ExpertShape s{T, k, E, N, K};
    return check_experts(wtype, s) != QMM_OK ? -1 : many_rows(wtype, s, gated != 0) ? 1 : 0;
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
    if (scratch_bytes < scratch_of(wtype, s).bytes) return QMM_E_SCRATCH;
    if (many_rows(wtype, s, true))
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
    if (scratch_bytes < scratch_of(wtype, s).bytes) return QMM_E_SCRATCH;
    cudaStream_t cs = (cudaStream_t)stream;
    float* p = reinterpret_cast<float*>((uint8_t*)scratch + scratch_of(wtype, s).products);
    if (many_rows(wtype, s, false)) {
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
