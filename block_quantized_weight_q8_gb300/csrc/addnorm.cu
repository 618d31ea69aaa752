// addnorm.cu -- the residual's addition, the RMS norm and the 8-bit rows of its result in one pass:
//   y = x + r;  s = 1 / sqrt(mean(y^2) + eps);  h = (y s) w;  xq = quantized h
//
// Bound by memory: 8 bytes read and 5.06 (Q8_0) or 5.14 (Q8_K) written per value.  One CTA per row keeps the row's sum in
// registers between its two uses (rows beyond 16 values a thread of 1024 are read once more), so every value crosses
// memory once.  The quantizer's rounding makes the codes depend on the last bit of s; the squares are therefore summed as
// pairs of floats (product and its error by fma, sum and its error by the two-sum) and rounded to f32 once.  What the pairs
// lose is the roundings of the errors' own sum c.  With u = 2^-24: 16 squares a thread leave |c| at most 17 u of their sum
// and lose 169 u^2 of it, the ten joins 35 to 45 u^2 each; rows of up to 64 squares a thread settle c into the sum every
// four squares, which lose 23 u^2, and their joins 5 to 23 u^2 each.  Both stay below 2^-38 of the sum (measured: 2^-44),
// so the codes are those of the exact sum, whatever the order, but where that sum lies so near to the middle between two
// floats.
#include "qmm_device.cuh"
#include "qmm_host.h"

namespace qmm {

static __device__ unsigned int g_addnorm_error = 0;  // bounds records of a bounds-checked build

// (s, c) += (v, e): the sum's rounding error goes to c
__device__ __forceinline__ void pair_add(float& s, float& c, float v, float e) {
    const float t = __fadd_rn(s, v);
    const float z = __fsub_rn(t, s);
    c = __fadd_rn(c, __fadd_rn(__fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(v, z)), e));
    s = t;
}
// s the nearest float of s + c (an infinite sum, whose c is NaN, stays)
__device__ __forceinline__ void pair_settle(float& s, float& c) {
    const float t = __fadd_rn(s, c);
    if (t != t) return;
    c = __fsub_rn(c, __fsub_rn(t, s));
    s = t;
}
__device__ __forceinline__ void pair_square(float& s, float& c, float v) {
    const float p = __fmul_rn(v, v);
    pair_add(s, c, p, __fmaf_rn(v, v, -p));
}
__device__ __forceinline__ float4 add4(float4 a, float4 b) {
    return make_float4(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y), __fadd_rn(a.z, b.z), __fadd_rn(a.w, b.w));
}

// The row's values are dealt out in units of one warp's quantizer step: 128 values (Q8_0: a lane holds 4 of a block's 32)
// or 256 (Q8_K: a lane holds 8 of the block).  Unit u belongs to warp u % warps.  HELD: units a warp keeps in registers;
// KEEP false: the second pass reads the row again.
template <int ACT, int HELD, bool KEEP>
__global__ void add_rmsnorm_quantize_kernel(const float* x, const float* r, float* sum, const float* __restrict__ w,
                                            float eps, float* h, uint8_t* __restrict__ xq, int K) {
    constexpr int V4 = ACT == QMM_Q8_0 ? 1 : 2;  // float4 of a lane and unit
    __shared__ float ps[32], pc[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const int n4 = K / 4, units = (n4 + 32 * V4 - 1) / (32 * V4);
    const int64_t row = blockIdx.x;
    pdl_launch_dependents();
    const float4* x4 = reinterpret_cast<const float4*>(x + row * K);
    const float4* r4 = reinterpret_cast<const float4*>(r + row * K);
    const float4* w4 = reinterpret_cast<const float4*>(w);
    float4* s4 = sum != nullptr ? reinterpret_cast<float4*>(sum + row * K) : nullptr;
    float4* h4 = h != nullptr ? reinterpret_cast<float4*>(h + row * K) : nullptr;
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    pdl_wait();
    float s = 0.0f, c = 0.0f;
    float4 v[KEEP ? HELD : 1][V4];
    auto at = [&](int u, int i) { return (u * 32 + lane) * V4 + i; };
    if constexpr (KEEP) {
        float4 b[HELD][V4];
#pragma unroll
        for (int j = 0; j < HELD; j++)
#pragma unroll
            for (int i = 0; i < V4; i++) {
                const int g = at(warp + j * nw, i);
                v[j][i] = g < n4 ? x4[g] : zero;
                b[j][i] = g < n4 ? r4[g] : zero;
            }
#pragma unroll
        for (int j = 0; j < HELD; j++)
#pragma unroll
            for (int i = 0; i < V4; i++) {
                const int g = at(warp + j * nw, i);
                v[j][i] = add4(v[j][i], b[j][i]);
                if (s4 != nullptr && g < n4) s4[g] = v[j][i];
                pair_square(s, c, v[j][i].x), pair_square(s, c, v[j][i].y);
                pair_square(s, c, v[j][i].z), pair_square(s, c, v[j][i].w);
            }
    } else {
        for (int u = warp; u < units; u += nw)
#pragma unroll
            for (int i = 0; i < V4; i++) {
                const int g = at(u, i);
                if (g >= n4) continue;
                const float4 y = add4(x4[g], r4[g]);
                if (s4 != nullptr) s4[g] = y;
                pair_square(s, c, y.x), pair_square(s, c, y.y), pair_square(s, c, y.z), pair_square(s, c, y.w);
                pair_settle(s, c);
            }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const float os = __shfl_xor_sync(0xffffffffu, s, off), oc = __shfl_xor_sync(0xffffffffu, c, off);
        pair_add(s, c, os, oc);
    }
    if (lane == 0) ps[warp] = s, pc[warp] = c;
    __syncthreads();
    s = lane < nw ? ps[lane] : 0.0f, c = lane < nw ? pc[lane] : 0.0f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const float os = __shfl_xor_sync(0xffffffffu, s, off), oc = __shfl_xor_sync(0xffffffffu, c, off);
        pair_add(s, c, os, oc);
    }
    // an infinite sum has an undefined error term: the sum itself says what it is
    const float ss = isfinite(s) ? __fadd_rn(s, c) : s;
    const float sn = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss, (float)K), eps)));
    uint8_t* const orow =
        xq != nullptr ? xq + row * (ACT == QMM_Q8_0 ? (int64_t)(K / 32) * Q8_0_BB : (int64_t)(K / 256) * Q8_K_BB) : nullptr;
    auto put = [&](int u, const float4* y) {  // the whole warp: the quantizer's lanes meet
        float4 o[V4];
        bool active = true;
#pragma unroll
        for (int i = 0; i < V4; i++) {
            const int g = at(u, i);
            active = g < n4;
            o[i] = active ? norm4(y[i], sn, w4[g]) : zero;
            if (h4 != nullptr && active) h4[g] = o[i];
        }
        if (orow == nullptr || !QMM_IN_BOUNDS(g_addnorm_error, u, units)) return;
        if constexpr (ACT == QMM_Q8_0) {
            const int g = at(u, 0);
            quant_q8_0_part(o[0], active, lane & 7, orow + (active ? (int64_t)(g >> 3) * Q8_0_BB : 0));
        } else {
            quant_q8_K_lane(o[0], o[V4 - 1], lane, orow + (int64_t)u * Q8_K_BB);
        }
    };
    if constexpr (KEEP) {
#pragma unroll
        for (int j = 0; j < HELD; j++)
            if (warp + j * nw < units) put(warp + j * nw, v[j]);
    } else {
        for (int u = warp; u < units; u += nw) {
            float4 y[V4];
#pragma unroll
            for (int i = 0; i < V4; i++) {
                const int g = at(u, i);
                y[i] = g >= n4 ? zero : s4 != nullptr ? s4[g] : add4(x4[g], r4[g]);
            }
            put(u, y);
        }
    }
}

template <int ACT, int HELD, bool KEEP>
static qmm_status launch_rows(const float* x, const float* r, float* sum, const float* w, float eps, float* h, void* xq,
                              int64_t M, int64_t K, int warps, cudaStream_t stream) {
    return launch_pdl(add_rmsnorm_quantize_kernel<ACT, HELD, KEEP>, dim3((unsigned)M), warps * 32, 0, stream, x, r, sum, w,
                      eps, h, (uint8_t*)xq, (int)K);
}

template <int ACT>
static qmm_status launch_act(const float* x, const float* r, float* sum, const float* w, float eps, float* h, void* xq,
                             int64_t M, int64_t K, cudaStream_t stream) {
    constexpr int VALUES = ACT == QMM_Q8_0 ? 128 : 256;
    constexpr int H = ACT == QMM_Q8_0 ? 4 : 2;  // 16 values a lane
    // Few rows: a unit a warp, the shortest way through a row.  More rows than twice the SMs: H units a warp, so that an SM
    // holds several rows, whose loads and sums overlap (4096 rows of 4096 to the sum, f32 and Q8_0: 42 us,
    // 6.7 TB/s; a unit a warp: 58).
    const int64_t units = (K + VALUES - 1) / VALUES;
    DeviceInfo dev;
    const qmm_status st = current_device(&dev);
    if (st != QMM_OK) return st;
    if (units <= 32 && (units < H || M <= 2 * dev.sms))
        return launch_rows<ACT, 1, true>(x, r, sum, w, eps, h, xq, M, K, (int)units, stream);
    if (units <= 32 * H) return launch_rows<ACT, H, true>(x, r, sum, w, eps, h, xq, M, K, (int)((units + H - 1) / H), stream);
    return launch_rows<ACT, 1, false>(x, r, sum, w, eps, h, xq, M, K, 32, stream);
}

}  // namespace qmm

using namespace qmm;

extern "C" {

qmm_status qmm_add_rmsnorm_quantize(int act, const float* x, const float* r, float* sum, const float* w, float eps, float* h,
                                    void* xq, int64_t M, int64_t K, qmm_stream_t stream) {
    if (act != QMM_Q8_0 && act != QMM_Q8_K) return QMM_E_TYPE;
    if (!x || !r || !w || (!xq && !h)) return QMM_E_NULL;
    const qmm_status st = check_shape(act, M, 1, K);
    if (st != QMM_OK) return st;
    if (!aligned16(x) || !aligned16(r) || !aligned16(sum) || !aligned16(w) || !aligned16(h) || !aligned16(xq))
        return QMM_E_ALIGN;
    if (act == QMM_Q8_0) return launch_act<QMM_Q8_0>(x, r, sum, w, eps, h, xq, M, K, (cudaStream_t)stream);
    return launch_act<QMM_Q8_K>(x, r, sum, w, eps, h, xq, M, K, (cudaStream_t)stream);
}

unsigned qmm_internal_addnorm_error(int clear) {
    unsigned v = 0;
    cudaMemcpyFromSymbol(&v, g_addnorm_error, sizeof(v));
    if (clear) {
        const unsigned z = 0;
        cudaMemcpyToSymbol(g_addnorm_error, &z, sizeof(z));
    }
    return v;
}

}  // extern "C"
