// rope.cu -- rotary positions: the frequency table with its scalings for long
// contexts, and the rotation of f32 heads.
//
//   rope_freqs  one thread per pair, in f64 (once per model): turns per position
//               as 64-bit fractions
//   rope        a CTA per ~512 shares of eight values of neighbouring tokens: the
//               tokens' tables of (cos, sin) pairs into shared memory, then two
//               shares per thread, whose loads are issued before the tables are
//               computed
// Bound by memory: 8 bytes moved per value.
#include "qmm_host.h"
#include "rope_device.cuh"

namespace qmm {

static __device__ unsigned int g_rope_error = 0;

// keep, the share of the unscaled frequency: QMM_ROPE_BANDS, a ramp over the turns
// in orig_len positions, from lo to hi; QMM_ROPE_YARN, a ramp over the pair index,
// between the pairs that turn hi and lo times in orig_len positions
__global__ void rope_freqs_kernel(uint64_t* __restrict__ freqs, int n_rot, double base, int scaling, double factor,
                                  double orig_len, double lo, double hi) {
    pdl_wait();
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n_rot / 2) {
        double f = pow(base, -2.0 * i / n_rot);
        if (scaling != QMM_ROPE_PLAIN) {
            double keep = 0.0;
            if (scaling == QMM_ROPE_BANDS) {
                keep = (orig_len * f / (2.0 * kPi) - lo) / (hi - lo);
            } else if (scaling == QMM_ROPE_YARN) {
                const double per = n_rot / (2.0 * log(base));
                const double first = fmax(floor(per * log(orig_len / (hi * 2.0 * kPi))), 0.0);
                const double last = fmin(ceil(per * log(orig_len / (lo * 2.0 * kPi))), n_rot - 1.0);
                keep = 1.0 - (i - first) / fmax(last - first, 0.001);
            }
            keep = fmin(fmax(keep, 0.0), 1.0);
            f = (1.0 - keep) * f / factor + keep * f;
        }
        // f / 2 pi modulo 1, times 2^64: the product with 1 / 2 pi as a pair of doubles
        constexpr double kInvHi = 1.0 / (2.0 * kPi);
        const double kInvLo = fma(-kInvHi, 2.0 * kPi, 1.0) / (2.0 * kPi) - kInvHi * (2.4492935982947064e-16 / (2.0 * kPi));
        const double t = f * kInvHi, e = fma(f, kInvHi, -t) + f * kInvLo;
        const double frac = t - floor(t);
        const uint64_t whole = (uint64_t)(frac * 18446744073709551616.0);
        freqs[i] = whole + (uint64_t)(int64_t)rint(e * 18446744073709551616.0);
    }
    pdl_launch_dependents();
}

constexpr int kRopeThreads = 256;
constexpr int kRopeShares = 2 * kRopeThreads;  // shares of eight values per CTA
constexpr int kRopeTable = 1024;               // (cos, sin) entries in shared memory

// grid (groups of tpb tokens, groups of kRopeShares shares of one token when tpb
// is 1); shares: of one token, H * hd / 8
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const float* x, float* y, const int32_t* __restrict__ pos,
                                                            const uint64_t* __restrict__ freqs, int64_t T, int shares,
                                                            int hd, int64_t ldx, int64_t ldy, int tpb, RopeLayout L,
                                                            float mscale, int inverse) {
    __shared__ float4 cs[kRopeTable];
    pdl_wait();
    const int64_t t0 = (int64_t)blockIdx.x * tpb;
    const int nt = T - t0 < tpb ? (int)(T - t0) : tpb;
    const int per_head = hd >> 3, half = L.n_rot >> 1;
    const int s0 = blockIdx.y * kRopeShares;
    const int n = tpb > 1 ? nt * shares : (shares - s0 < kRopeShares ? shares - s0 : kRopeShares);
    float v[2][8];
    int token[2], share[2];
    int64_t at[2];
#pragma unroll
    for (int k = 0; k < 2; k++) {
        const int i = threadIdx.x + k * kRopeThreads;
        if (i < n) {
            token[k] = tpb > 1 ? i / shares : 0;
            const int s = s0 + i - token[k] * shares;
            const int head = s / per_head;
            share[k] = s - head * per_head;
            at[k] = (int64_t)head * hd;
            if (QMM_IN_BOUNDS(g_rope_error, (t0 + token[k]) * ldx + at[k] + hd - 1, T * ldx))
                rope_load8(L, share[k], x + (t0 + token[k]) * ldx + at[k], v[k]);
        }
    }
    for (int i = threadIdx.x; i < nt * half; i += kRopeThreads) {
        const int t = i / half;
        const uint64_t f = freqs[i - t * half];
        float4 c = turn_cos_sin((uint64_t)(int64_t)pos[t0 + t] * f, mscale);
        if (inverse) c.z = -c.z, c.w = -c.w;
        if (QMM_IN_BOUNDS(g_rope_error, i, kRopeTable)) cs[i] = c;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; k++) {
        const int i = threadIdx.x + k * kRopeThreads;
        if (i < n) {
            rope_turn8(L, share[k], v[k], cs + token[k] * half);
            if (QMM_IN_BOUNDS(g_rope_error, (t0 + token[k]) * ldy + at[k] + hd - 1, T * ldy))
                rope_store8(L, share[k], y + (t0 + token[k]) * ldy + at[k], v[k]);
        }
    }
    pdl_launch_dependents();
}

qmm_status rope_check(const qmm_rope_spec* r, int64_t hd, RopeLayout* L) {
    if (!r || !r->freqs) return QMM_E_NULL;
    if (r->layout != QMM_ROPE_HALF && r->layout != QMM_ROPE_INTERLEAVED) return QMM_E_TYPE;
    if (r->n_rot < 2 || r->n_rot > hd || r->n_rot % 2) return QMM_E_SHAPE;
    if (!aligned16(r->freqs)) return QMM_E_ALIGN;
    L->n_rot = (int)r->n_rot;
    L->halves = r->layout == QMM_ROPE_HALF;
    L->scattered = L->halves && r->n_rot % 8 != 0;
    return QMM_OK;
}

}  // namespace qmm

using namespace qmm;

extern "C" {

unsigned qmm_internal_rope_error(int clear) {
    unsigned v = 0;
    cudaMemcpyFromSymbol(&v, g_rope_error, sizeof(v));
    if (clear) {
        const unsigned z = 0;
        cudaMemcpyToSymbol(g_rope_error, &z, sizeof(z));
    }
    return v;
}

qmm_status qmm_rope_freqs(void* freqs, int64_t n_rot, double base, int scaling, double factor, double orig_len,
                          double lo, double hi, qmm_stream_t stream) {
    if (!freqs) return QMM_E_NULL;
    if (scaling < QMM_ROPE_PLAIN || scaling > QMM_ROPE_YARN) return QMM_E_TYPE;
    if (n_rot < 2 || n_rot % 2 || n_rot > kHeadMax || !(base > 1.0) || !(base <= 1e300)) return QMM_E_SHAPE;
    if (scaling != QMM_ROPE_PLAIN && !(factor > 0.0 && factor <= 1e300)) return QMM_E_SHAPE;
    if (scaling >= QMM_ROPE_BANDS && !(orig_len > 0.0 && orig_len <= 1e300 && lo > 0.0 && hi > lo && hi <= 1e300))
        return QMM_E_SHAPE;
    if (!aligned16(freqs)) return QMM_E_ALIGN;
    return launch_pdl(rope_freqs_kernel, dim3(1), kHeadMax / 2, 0, (cudaStream_t)stream, (uint64_t*)freqs, (int)n_rot,
                      base, scaling, factor, orig_len, lo, hi);
}

qmm_status qmm_rope(const qmm_rope_spec* rope, const float* x, int64_t ldx, float* y, int64_t ldy, const int32_t* pos,
                    int64_t T, int64_t H, int64_t hd, int inverse, qmm_stream_t stream) {
    if (!x || !y || !pos) return QMM_E_NULL;
    if (!head_dim_ok(hd) || T < 1 || T > kMaxDim || H < 1 || H > kHeadsMax) return QMM_E_SHAPE;
    if (!row_stride_ok(ldx, H * hd) || !row_stride_ok(ldy, H * hd) || (x == y && ldx != ldy)) return QMM_E_SHAPE;
    RopeLayout L;
    const qmm_status st = rope_check(rope, hd, &L);
    if (st != QMM_OK) return st;
    if (!aligned16(x) || !aligned16(y) || ((uintptr_t)pos & 3u)) return QMM_E_ALIGN;
    const int shares = (int)(H * hd / 8), half = L.n_rot / 2;
    int tpb = kRopeShares / shares;  // tokens per CTA
    if (tpb > kRopeTable / half) tpb = kRopeTable / half;
    if (tpb < 1) tpb = 1;
    const dim3 grid((unsigned)((T + tpb - 1) / tpb), tpb > 1 ? 1u : (unsigned)((shares + kRopeShares - 1) / kRopeShares));
    return launch_pdl(rope_kernel, grid, kRopeThreads, 0, (cudaStream_t)stream, x, y, pos, (const uint64_t*)rope->freqs,
                      T, shares, (int)hd, ldx, ldy, tpb, L, rope->mscale, inverse);
}

}  // extern "C"
