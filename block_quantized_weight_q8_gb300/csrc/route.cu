// route.cu -- the routing of tokens to experts.
//
//   score_e = softmax(l)_e or 1 / (1 + e^-l_e);  key_e = score_e + bias_e
//   the `groups_kept` groups with the largest sums of their `group_top` largest keys stay open
//   ids = the k open experts with the largest keys, largest first, ties to the lower index
//   weights_j = scale * score_j, over the chosen scores' sum where they are renormalised
//
// An expert whose logit (or key) is -inf or NaN is closed to the token.  One warp per token: each group has L lanes (a
// power of two, 32 where there is one group), lane l of it the group's experts l, l + L, ...; so all groups' worth comes of
// one look at a lane's keys and log2 L exchanges.  A choice is a maximum over the lane's keys, one over the warp
// (whole-number keys in the floats' order) and one of the index.  Bound by these instructions, two thousand a token:
// 8192 tokens of 256 experts, 4 of 8 groups by two keys, 8 choices take 20.4 us (25 from cold caches, the issue slots 67%
// busy; with expert e in lane e % 32 and the groups one after another, 43); a few tokens take 3.2 us.
//
// The choice is that of binary64.  Without a bias the scores' order is the logits' and keys are the logits themselves
// (but where groups count by two keys).  Otherwise keys carry rounding errors, bounded below; where two keys that decide
// anything lie closer than both their errors (a few tokens in ten thousand), the warp orders the candidates by their keys
// in binary64, or, where the groups are in doubt, chooses again from all of the token's.  Weights are f32 scores over their
// f32 sum, a few roundings each (6e-8 of the weight on the measured cases).
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
    int T, E, k, groups, each, kept, top, lanes;
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

// Lane and register of the experts.
struct Place {
    int L, per_group;  // lanes of a group; experts of a group
    int base, lane_of;  // this lane's group's first expert (-1: none), its lane in the group
    int second;         // more than 32 groups: registers from here on are those of the group 32 further on
    __device__ __forceinline__ int expert(int j) const {
        const int i = second && j >= second ? 32 * per_group + j - second : lane_of + L * j;
        return base + i;
    }
    __device__ __forceinline__ bool there(int j, int E) const {
        if (base < 0) return false;
        if (second) return j < 2 * second && expert(j) < E;
        return lane_of + L * j < per_group;
    }
};
__device__ __forceinline__ Place place_of(const Route& a, int lane) {
    if (a.groups > 32) return {1, a.each, lane * a.each, 0, a.each};
    const int g = lane / a.lanes;
    return {a.lanes, a.each, g < a.groups ? g * a.each : -1, lane - g * a.lanes, 0};
}

// Loops over a lane's keys are unrolled but for binary64 ones, which few warps of a launch run if any.
template <int PER, class Key>
constexpr int unrolled() {
    return sizeof(Key) == 8 ? 1 : PER;
}

// The largest key of the warp (0: none) and its expert, the lowest of equals; the key is cleared.
template <int PER, class Key>
__device__ __forceinline__ Key take_best(Key (&key)[PER], const Place& at, int* expert) {
    constexpr int U = unrolled<PER, Key>();
    Key b = 0;
#pragma unroll U
    for (int j = 0; j < PER; j++) b = max(b, key[j]);
    const Key m = warp_max(b);
    uint32_t e = 0xFFFFFFFFu;
    int i = 0;
    if (b == m && m != 0) {  // the lanes that have it
#pragma unroll U
        for (int j = PER - 1; j >= 0; j--)
            if (key[j] == m) i = j;
        e = (uint32_t)at.expert(i);
    }
    const uint32_t win = __reduce_min_sync(0xffffffffu, e);
    *expert = (int)win;
    if (e == win && m != 0) {
#pragma unroll U
        for (int j = 0; j < PER; j++)
            if (j == i) key[j] = 0;
    }
    return m;
}

// Chooses from the keys.  Two that lie nearer than near + rel (|a| + |b|) are not told apart (near < 0: all are).  Lane j has
// the expert of the j-th largest key in *chosen (-1: none); the result is how many lanes have one: at most k where the
// choice is sure; with *doubt more, up to where a key is surely smaller; 0 and *doubt where the groups are not sure, or
// more than 32 keys.
template <int PER, class Key, class Value>
__device__ __forceinline__ int choose(const Route& a, const Place& at, Key (&key)[PER], int lane, Value near, Value rel,
                                      int* chosen, bool* doubt) {
    constexpr int U = unrolled<PER, Key>();
    *doubt = false;
    if (a.groups > 1) {
        // the two largest keys of this lane's group (or of each of its two groups), then of the group's lanes
        Key worth[2];
        Value size[2];  // the magnitudes that went into the worth: what its error goes by
#pragma unroll
        for (int h = 0; h < 2; h++) {
            Key b = 0, s = 0;
#pragma unroll U
            for (int j = 0; j < PER; j++) {
                if (at.second && (j >= at.second) != (h == 1)) continue;
                const Key v = key[j];
                s = max(s, min(b, v));
                b = max(b, v);
            }
            for (int off = 1; off < at.L; off <<= 1) {
                const Key ob = __shfl_xor_sync(0xffffffffu, b, off), os = __shfl_xor_sync(0xffffffffu, s, off);
                s = max(min(b, ob), max(s, os));
                b = max(b, ob);
            }
            worth[h] = b, size[h] = b != 0 ? fabs(unordered(b)) : (Value)0;
            if (a.top == 2 && b != 0 && s != 0) {
                worth[h] = ordered(unordered(b) + unordered(s));
                size[h] += fabs(unordered(s));
            }
            if (h == 1 && !at.second) worth[h] = 0;
        }
        if (at.lane_of != 0 || at.base < 0) worth[0] = 0;  // one lane speaks for its group
        const Key all[2] = {worth[0], worth[1]};
        const int g = at.base < 0 ? 64 : at.base / at.per_group;
        uint64_t open = 0;
        for (int i = 0; i < a.kept; i++) {
            const Key m = warp_max(max(worth[0], worth[1]));
            if (m == 0) break;
            const uint32_t mine = worth[0] == m ? (uint32_t)g : worth[1] == m ? (uint32_t)g + 32 : 0xFFFFFFFFu;
            const uint32_t win = __reduce_min_sync(0xffffffffu, mine);
            open |= 1ull << win;
            if (mine == win) {
                if (win == (uint32_t)g) worth[0] = 0;
                else worth[1] = 0;
            }
        }
        if (near >= 0) {
            // Sure where the least that an open group can be worth is more than the most that a closed one can.  Every group
            // counts, wherever it stands: two keys of opposite signs leave a worth that is small beside its error.
            Key least = 0, most = 0;
#pragma unroll
            for (int h = 0; h < 2; h++) {
                if (all[h] == 0) continue;
                const Value v = unordered(all[h]), off = near + (Value)1.5 * rel * size[h];
                if (open >> (g + 32 * h) & 1) least = max(least, ordered(isfinite(v) ? off - v : (Value)INFINITY));
                else most = max(most, ordered(isfinite(v) ? v + off : (Value)INFINITY));
            }
            least = warp_max(least), most = warp_max(most);
            if (most != 0 && !(-unordered(least) > unordered(most))) {
                *doubt = true;
                return 0;
            }
        }
        const bool open0 = g < 64 && (open >> g) & 1, open1 = g < 32 && (open >> (g + 32)) & 1;
#pragma unroll U
        for (int j = 0; j < PER; j++)
            if (!(at.second && j >= at.second ? open1 : open0)) key[j] = 0;
    }
    int mine = -1, count = 0;
    Value last = 0;
    for (int i = 0; i <= 32; i++) {
        if (i >= a.k && near < 0) break;
        int e;
        const Key m = take_best(key, at, &e);
        if (m == 0) break;
        const Value v = unordered(m);
        if (near >= 0 && i > 0) {
            const bool apart = last - v > near + rel * (fabs(last) + fabs(v));
            if (i >= a.k && apart) break;
            if (!apart) *doubt = true;
            if (i == 32) return 0;
        }
        last = v;
        if (i == lane) mine = e;
        count = i + 1;
    }
    *chosen = mine;
    return count;
}

// The sum of the exponentials in binary64.
template <int PER>
__device__ __forceinline__ double exact_total(const Route& a, const Place& at, const float* l, float top) {
    double total = 0.0;
#pragma unroll
    for (int j = 0; j < PER; j++) {
        const int e = at.expert(j);
        if (at.there(j, a.E) && l[e] > -INFINITY) total += exp((double)fminf(l[e], FLT_MAX) - (double)top);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
    return total;
}
__device__ __forceinline__ double exact_key(const Route& a, const float* l, int e, float top, double total) {
    const double v = fminf(l[e], FLT_MAX);
    const double c = a.sigmoid ? 1.0 / (1.0 + exp(-v)) : exp(v - (double)top) / total;
    return a.bias ? c + (double)a.bias[e] : c;
}

// The order of `count` candidates, one in a lane, by their keys in binary64 (one each, where all of a token's took 20 us).
template <int PER>
__device__ __noinline__ int order_exactly(const Route& a, const float* l, int lane, float top, int candidate, int count) {
    const double total = a.sigmoid ? 1.0 : exact_total<PER>(a, place_of(a, lane), l, top);
    const double mine = lane < count ? exact_key(a, l, candidate, top, total) : 0.0;
    int rank = 0;
    for (int t = 0; t < count; t++) {
        const double other = __shfl_sync(0xffffffffu, mine, t);
        const int e = __shfl_sync(0xffffffffu, candidate, t);
        if (other > mine || (other == mine && e < candidate)) rank++;
    }
    int chosen = -1;
    for (int j = 0; j < min(a.k, count); j++) {
        const int from = __ffs(__ballot_sync(0xffffffffu, lane < count && rank == j)) - 1;
        const int e = __shfl_sync(0xffffffffu, candidate, from);
        if (lane == j) chosen = e;
    }
    return chosen;
}

// The choice from all of the token's keys in binary64: where the groups were in doubt.
template <int PER>
__device__ __noinline__ int choose_exactly(const Route& a, const float* l, int lane, float top) {
    const Place at = place_of(a, lane);
    uint64_t key[PER];
    const double total = a.sigmoid ? 1.0 : exact_total<PER>(a, at, l, top);
#pragma unroll
    for (int j = 0; j < PER; j++) {
        const int e = at.expert(j);
        key[j] = 0;
        if (at.there(j, a.E) && l[e] > -INFINITY) {
            const double c = exact_key(a, l, e, top, total);
            if (c > -INFINITY) key[j] = ordered(c);
        }
    }
    int mine;
    bool doubt;
    choose<PER, uint64_t, double>(a, at, key, lane, -1.0, 0.0, &mine, &doubt);
    return mine;
}

// Scores so small that f32 loses them, over their sum (0 where binary64 loses them too).
__device__ __noinline__ float small_weight(bool sigmoid, bool real, float v, float top) {
    const double s = !real ? 0.0 : sigmoid ? 1.0 / (1.0 + exp(-(double)v)) : exp((double)v - (double)top);
    double sum = s;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    return sum > 0.0 ? (float)(s / sum) : 0.0f;
}

constexpr int kRouteThreads = 128;

// 12 CTAs of 40 registers an SM where a lane has few keys (21.9 us without the bound, 21.5 with it).
template <int PER>
__global__ void __launch_bounds__(kRouteThreads, PER <= 8 ? 12 : 1) route_kernel(const __grid_constant__ Route a) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t t = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    if (t >= a.T) return;  // whole warps leave together
    const float* l = a.logits + t * a.ld;
    const Place at = place_of(a, lane);
    float v[PER];
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < PER; j++) {
        const int e = at.expert(j);
        float x = at.there(j, a.E) && QMM_IN_BOUNDS(g_route_error, e, a.ld) ? l[e] : -INFINITY;
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
            if (a.bias) c += a.bias[at.expert(j)];
        }
        key[j] = c > -INFINITY ? ordered(c) : 0u;
    }
    int e;
    // Errors of two keys together (expf is within 2 units of 2^-23 relative): sigmoid, 2 (2^-22 s (1 - s) + 2^-23 s), at
    // most 6 units of 2^-24, and the bias's addition 2^-24 |key| each (half of 1.2e-7); softmax, scores up to the largest,
    // 1 / total: the exponent's rounding (its size times the score at most 0.37 of the largest) and the quotient's, a few
    // units of 2^-24, and, shared by all keys, the sum's at most 69 roundings (64 keys of a lane and the warp's five).  A
    // group's worth of two keys has both their errors; its sum and the check's own addition round by 2^-24 of their sizes.
    const float near = !scored ? -1.0f : a.sigmoid ? 3.6e-7f : 8e-6f / total;
    bool doubt;
    const int count = choose<PER, uint32_t, float>(a, at, key, lane, near, 1.2e-7f, &e, &doubt);
    if (doubt) e = count > 0 ? order_exactly<PER>(a, l, lane, top, e, count) : choose_exactly<PER>(a, l, lane, top);
    else if (lane >= a.k) e = -1;
    float w = 0.0f;
    if (e >= 0) w = score(fminf(l[e], FLT_MAX));
    if (a.renorm) {
        float sum = w;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        w = sum > 1e-30f ? w / sum : small_weight(a.sigmoid, e >= 0, e >= 0 ? fminf(l[e], FLT_MAX) : 0.0f, top);
    }
    if (lane < a.k && QMM_IN_BOUNDS(g_route_error, t * a.k + lane, (int64_t)a.T * a.k)) {
        a.ids[t * a.k + lane] = e;
        a.weights[t * a.k + lane] = w * a.scale;
    }
}

template <int PER>
static qmm_status launch_route(const Route& a, cudaStream_t stream) {
    // few tokens: a warp per CTA, so that they spread over the SMs
    const int warps = a.T <= 1024 ? 1 : kRouteThreads / 32;
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
    // lanes of a group, and the experts of a lane
    a.lanes = 32;
    while (a.lanes > 1 && a.lanes * a.groups > 32) a.lanes >>= 1;
    const int per = s.groups > 32 ? 2 * a.each : (a.each + a.lanes - 1) / a.lanes;
    if (per <= 1) return launch_route<1>(a, cs);
    if (per <= 2) return launch_route<2>(a, cs);
    if (per <= 4) return launch_route<4>(a, cs);
    if (per <= 8) return launch_route<8>(a, cs);
    if (per <= 16) return launch_route<16>(a, cs);
    if (per <= 32) return launch_route<32>(a, cs);
    return launch_route<64>(a, cs);
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
