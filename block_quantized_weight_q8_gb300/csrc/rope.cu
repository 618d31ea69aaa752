// rope.cu -- rotary positions: the frequency table with its scalings for long
// contexts, and the rotation of f32 heads.
//
//   rope_freqs  one thread per pair, in f64 (once per model): turns per position
//               as 64-bit fractions
//   rope        the row kernel of the cache's store (kvpages.cu) with query rows only
#include "kvpages.cuh"
#include "rope_device.cuh"

namespace qmm {

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

qmm_status rows_launch(int type, const KvPages& c, const RowArgs& a, int hd, cudaStream_t stream);

qmm_status rope_check(const qmm_rope_spec* r, int64_t hd, RowArgs* a) {
    if (!r || !r->freqs) return QMM_E_NULL;
    if (r->layout != QMM_ROPE_HALF && r->layout != QMM_ROPE_INTERLEAVED) return QMM_E_TYPE;
    if (r->n_rot < 2 || r->n_rot > hd || r->n_rot % 2) return QMM_E_SHAPE;
    if (!aligned16(r->freqs)) return QMM_E_ALIGN;
    a->freqs = (const uint64_t*)r->freqs;
    a->mscale = r->mscale;
    a->n_rot = (int)r->n_rot;
    const bool whole = r->n_rot % 8 == 0;
    a->pairs = r->layout == QMM_ROPE_INTERLEAVED ? (whole ? kPairsNext : kPairsNextAny)
                                                 : (whole ? kPairsHalf : kPairsScattered);
    return QMM_OK;
}

}  // namespace qmm

using namespace qmm;

extern "C" {

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
    RowArgs a = {};
    const qmm_status st = rope_check(rope, hd, &a);
    if (st != QMM_OK) return st;
    if (!aligned16(x) || !aligned16(y) || !aligned4(pos)) return QMM_E_ALIGN;
    a.q = x, a.q_out = y, a.pos = pos;
    a.T = T, a.ldq = ldx, a.ldqo = ldy, a.Hq = (int)H;
    a.inverse = inverse;
    const KvPages none = {};
    return rows_launch(kNoPages, none, a, (int)hd, (cudaStream_t)stream);
}

}  // extern "C"
