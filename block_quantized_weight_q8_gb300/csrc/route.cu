// route.cu -- the routing of tokens to experts.
//
//   score_e = softmax(l)_e or 1 / (1 + e^-l_e);  key_e = score_e + bias_e
//   the `groups_kept` groups with the largest sums of their `group_top` largest keys stay open
//   ids = the k open experts with the largest keys, largest first, ties to the lower index
//   weights_j = scale * score_j, over the chosen scores' sum where they are renormalised
//
// An expert whose logit (or key) is -inf or NaN is closed to the token.  One warp per token, expert e in lane e % 32: the
// logits are read once, side by side.  Each choice is a maximum over the lane's keys, one over the warp (whole-number
// keys in the floats' order) and one of the index, so a token costs a few hundred instructions; a batch is bound by the
// launch, then by those.
//
// The choice is that of binary64.  Without a bias the scores' order is the logits' and keys are the logits themselves
// (but where groups count by two keys).  Otherwise keys carry rounding errors, bounded below; where two keys that decide
// anything lie closer than both their errors, the warp computes the token's keys again in binary64 and chooses from those
// (a few tokens in ten thousand).
#include <float.h>

#include "experts.h"

namespace qmm {

static __device__ unsigned int g_route_error = 0;  // bounds records of a bounds-checked build

struct Route {
    const float* logits;
    const float* bias;
    int32_t* ids;
    float* weights;
    int64_t ld;
    int T, E, k, groups, each, kept, top;
    int sigmoid, renorm;
    float scale;
};

// keys as whole numbers in the floats' order; 0: closed
__device__ __forceinline__ uint32_t ordered(float f) {
    const uint32_t b = __float_as_uint(f + 0.0f);  // -0 as 0
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t o) {
    return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ uint64_t ordered(double f) {
    const uint64_t b = (uint64_t)__double_as_longlong(f + 0.0);
    return b >> 63 ? ~b : b | (1ull << 63);
}
__device__ __forceinline__ double unordered(uint64_t o) {
    return __longlong_as_double((long long)(o >> 63 ? o & ~(1ull << 63) : ~o));
}
__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
    const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32));
    const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
    return (uint64_t)hi << 32 | lo;
}

// The largest key of the warp (0: none) and its expert, the lowest of equals.
template <int PER, class Key>
__device__ __forceinline__ Key best_of(const Key (&key)[PER], int lane, int* expert) {
    Key b = 0;
    int i = 0;
#pragma unroll
    for (int j = 0; j < PER; j++)
        if (key[j] > b) b = key[j], i = j;
    const Key m = warp_max(b);
    *expert = (int)__reduce_min_sync(0xffffffffu, b == m && m != 0 ? (uint32_t)(lane + 32 * i) : 0xFFFFFFFFu);
    return m;
}

// Chooses from the keys; returns false where two deciding keys lie nearer than near + rel (|a| + |b|) (near < 0: never).
// Lane j has the j-th expert in *chosen (-1: none).
template <int PER, class Key, class Value>
__device__ __forceinline__ bool choose(const Route& a, Key (&key)[PER], int lane, Value near, Value rel, int* chosen) {
    bool clear = true;
    if (a.groups > 1) {
        // the groups' worth, group g in lane g % 32 of register g / 32
        Key worth[2] = {0, 0};
        Value size[2] = {0, 0};  // the magnitudes that went into it: what its error goes by
        for (int g = 0; g < a.groups; g++) {
            const int e0 = g * a.each, e1 = e0 + a.each;
            Key b = 0, second = 0;
            int at = 0;
#pragma unroll
            for (int j = 0; j < PER; j++) {
                const int e = lane + 32 * j;
                if (e >= e0 && e < e1 && key[j] > b) second = b, b = key[j], at = e;
                else if (e >= e0 && e < e1 && key[j] > second) second = key[j];
            }
            const Key m = warp_max(b);
            Key w = m;
            Value sz = m != 0 ? fabs(unordered(m)) : (Value)0;
            if (a.top == 2 && m != 0) {
                const int win = (int)__reduce_min_sync(0xffffffffu, b == m ? (uint32_t)at : 0xFFFFFFFFu);
                const Key m2 = warp_max(b == m && at == win ? second : b);
                Value v = unordered(m);
                if (m2 != 0) v += unordered(m2), sz += fabs(unordered(m2));
                w = ordered(v);
            }
            if ((g & 31) == lane) {
                if (g < 32) worth[0] = w, size[0] = sz;
                else worth[1] = w, size[1] = sz;
            }
        }
        uint64_t open = 0;
        Value last = 0, last_size = 0;
        for (int i = 0; i < a.kept + 1; i++) {
            int g;
            const Key m = best_of(worth, lane, &g);
            if (m == 0) break;
            const Value v = unordered(m), sz = __shfl_sync(0xffffffffu, g < 32 ? size[0] : size[1], g & 31);
            // the first that stays closed against the last that is open
            if (i == a.kept && near >= 0 && !(last - v > 2 * (near + rel * (last_size + sz)))) clear = false;
            last = v, last_size = sz;
            if (i < a.kept) open |= 1ull << g;
            if ((g & 31) == lane) {
                if (g < 32) worth[0] = 0;
                else worth[1] = 0;
            }
        }
#pragma unroll
        for (int j = 0; j < PER; j++)
            if (!((open >> min((lane + 32 * j) / a.each, 63)) & 1)) key[j] = 0;
    }
    int mine = -1;
    Value last = 0;
    for (int i = 0; i < a.k + 1; i++) {
        if (i == a.k && near < 0) break;
        int e;
        const Key m = best_of(key, lane, &e);
        if (m == 0) break;
        if (near >= 0 && i > 0) {
            const Value v = unordered(m);
            if (!(last - v > near + rel * (fabs(last) + fabs(v)))) clear = false;
        }
        last = unordered(m);
        if (i < a.k && i == lane) mine = e;
#pragma unroll
        for (int j = 0; j < PER; j++)
            if (lane + 32 * j == e) key[j] = 0;
    }
    *chosen = mine;
    return clear;
}

// The token's keys in binary64, and the choice from them.
template <int PER>
__device__ __noinline__ int choose_exactly(const Route& a, const float* l, int lane, float top) {
    uint64_t key[PER];
    double total = 0.0;
    if (!a.sigmoid) {
        for (int j = 0; j < PER; j++) {
            const int e = lane + 32 * j;
            if (e < a.E && l[e] > -INFINITY) total += exp((double)fminf(l[e], FLT_MAX) - (double)top);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
    }
#pragma unroll
    for (int j = 0; j < PER; j++) {
        const int e = lane + 32 * j;
        key[j] = 0;
        if (e < a.E && l[e] > -INFINITY) {
            const double v = fminf(l[e], FLT_MAX);
            double c = a.sigmoid ? 1.0 / (1.0 + exp(-v)) : exp(v - (double)top) / total;
            if (a.bias) c += (double)a.bias[e];
            if (c > -INFINITY) key[j] = ordered(c);
        }
    }
    int mine;
    choose<PER, uint64_t, double>(a, key, lane, -1.0, 0.0, &mine);
    return mine;
}

template <int PER>
__global__ void __launch_bounds__(256) route_kernel(const __grid_constant__ Route a) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t t = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    if (t >= a.T) return;  // whole warps leave together
    const float* l = a.logits + t * a.ld;
    float v[PER];
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < PER; j++) {
        const int e = lane + 32 * j;
        float x = e < a.E && QMM_IN_BOUNDS(g_route_error, e, a.ld) ? l[e] : -INFINITY;
        x = x > -INFINITY ? fminf(x, FLT_MAX) : -INFINITY;  // NaN: closed
        v[j] = x;
        top = fmaxf(top, x);
    }
    top = unordered(warp_max(ordered(top)));
    float total = 0.0f;
    if (!a.sigmoid) {
#pragma unroll
        for (int j = 0; j < PER; j++) total += v[j] > -INFINITY ? expf(v[j] - top) : 0.0f;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
    }
    // Scores decide where there is a bias or where groups count by two keys; else the logits do.
    const bool scored = a.bias != nullptr || (a.groups > 1 && a.top == 2);
    auto score = [&](float x) { return a.sigmoid ? 1.0f / (1.0f + expf(-x)) : expf(x - top) / total; };
    uint32_t key[PER];
#pragma unroll
    for (int j = 0; j < PER; j++) {
        float c = v[j];
        if (scored && c > -INFINITY) {
            c = score(c);
            if (a.bias) c += a.bias[lane + 32 * j];
        }
        key[j] = c > -INFINITY ? ordered(c) : 0u;
    }
    int e;
    // Errors of two keys together (expf is within 2 units of 2^-23 relative): sigmoid, 2 (2^-22 s (1 - s) + 2^-23 s) and
    // the bias's addition 2^-24 |key| each; softmax, scores up to the largest, 1 / total: the exponent's rounding (its
    // size times the score at most 0.37 of the largest), the sum's 36 roundings, the quotient's.
    const float near = !scored ? -1.0f : a.sigmoid ? 6e-7f : 8e-6f / total;
    const bool sure = choose<PER, uint32_t, float>(a, key, lane, near, 1.2e-7f, &e);
    if (!sure) e = choose_exactly<PER>(a, l, lane, top);
    float w = 0.0f;
    if (e >= 0) w = score(fminf(l[e], FLT_MAX));
    if (a.renorm) {
        float sum = w;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (sum > 0.0f) w = w / sum;
    }
    if (lane < a.k && QMM_IN_BOUNDS(g_route_error, t * a.k + lane, (int64_t)a.T * a.k)) {
        a.ids[t * a.k + lane] = e;
        a.weights[t * a.k + lane] = w * a.scale;
    }
}

template <int PER>
static qmm_status launch_route(const Route& a, cudaStream_t stream) {
    // few tokens: a warp per CTA, so that they spread over the SMs
    const int warps = a.T <= 1024 ? 1 : 8;
    return launch_pdl(route_kernel<PER>, dim3((unsigned)((a.T + (int64_t)warps - 1) / warps)), warps * 32, 0, stream, a);
}

}  // namespace qmm

using namespace qmm;

extern "C" {

qmm_status qmm_route(const qmm_route_spec* spec, const float* logits, int64_t ld, const float* bias, int32_t* ids,
                     float* weights, int64_t T, int64_t E, qmm_stream_t stream) {
    if (!spec || !logits || !ids || !weights) return QMM_E_NULL;
    if (spec->score != QMM_ROUTE_SOFTMAX && spec->score != QMM_ROUTE_SIGMOID) return QMM_E_TYPE;
    const qmm_route_spec& s = *spec;
    if (T < 1 || T > kMaxDim || E < 1 || E > kMaxExperts || ld < E || ld > ((int64_t)1 << 32)) return QMM_E_SHAPE;
    if (s.groups < 1 || s.groups > 64 || E % s.groups || s.groups_kept < 1 || s.groups_kept > s.groups ||
        (s.group_top != 1 && s.group_top != 2) || !(s.scale >= -FLT_MAX && s.scale <= FLT_MAX))
        return QMM_E_SHAPE;
    if (s.k < 1 || s.k > 32 || s.k > s.groups_kept * (E / s.groups)) return QMM_E_SHAPE;
    if (!aligned4(logits) || !aligned4(bias) || !aligned4(ids) || !aligned4(weights)) return QMM_E_ALIGN;
    Route a = {};
    a.logits = logits, a.bias = bias, a.ids = ids, a.weights = weights, a.ld = ld;
    a.T = (int)T, a.E = (int)E, a.k = s.k, a.groups = s.groups, a.each = (int)(E / s.groups), a.kept = s.groups_kept;
    a.top = s.group_top, a.sigmoid = s.score == QMM_ROUTE_SIGMOID, a.renorm = s.renorm != 0, a.scale = s.scale;
    cudaStream_t cs = (cudaStream_t)stream;
    if (E <= 32) return launch_route<1>(a, cs);
    if (E <= 64) return launch_route<2>(a, cs);
    if (E <= 128) return launch_route<4>(a, cs);
    if (E <= 256) return launch_route<8>(a, cs);
    if (E <= 512) return launch_route<16>(a, cs);
    return launch_route<32>(a, cs);
}

unsigned qmm_internal_route_error(int clear) {
    unsigned v = 0;
    cudaMemcpyFromSymbol(&v, g_route_error, sizeof(v));
    if (clear) {
        const unsigned z = 0;
        cudaMemcpyToSymbol(g_route_error, &z, sizeof(z));
    }
    return v;
}

}  // extern "C"
