// rope_device.cuh -- rotary positions on the device: the sine and cosine of a
// position's angle as float pairs, and the rotation of a pair of values rounded
// once.  Shared by qmm_rope and qmm_kv_store, whose results therefore agree bit
// for bit.
//
// Angle.  Pair i turns F[i] / 2^64 of a full turn per position, so position p
// stands at (p * F[i]) mod 2^64: one wrapping integer product is the exact
// reduction of any angle, however far the position.  (A float product p * f has
// lost 2^-24 of up to 10^5 turns before its reduction starts.)
//
// Sine, cosine.  The phase's nearest multiple of 1/256 turn comes from a table of
// float pairs (value = hi + lo, 2^-48), the rest r, |r| <= pi/256, from the Taylor
// series sin r = r - r^3/6 + r^5/120, cos r - 1 = -r^2/2 + r^4/24 - r^6/720 (next
// terms below 2^-56 and 2^-65) with the leading terms kept as float pairs; the two
// are joined by the addition theorems.  Absolute error below 2^-42.
//
// Rotation.  x_a c - x_b s with each product's rounding error recovered by an FMA
// and the difference's by the two-sum identity (Knuth, Dekker), so the result is
// the exact value rounded once to f32 except where that lies within 2^-42 of a
// rounding border.  That is what makes a rotated key's 8-bit codes reproducible by
// any implementation that computes in 64 bits and rounds once.
// About 90 operations per pair's angle (once for the rows of a token that one CTA takes)
// and 38 per rotated pair: 64% (a rotation of part of each head) to 67% (the store) of the
// issue slots.
#pragma once

#include "qmm_device.cuh"

namespace qmm {

constexpr int kTurnSteps = 256;
struct alignas(16) TurnTable {  // an entry is read as one float4
    float v[kTurnSteps][4];       // cos hi, cos lo, sin hi, sin lo of k/256 turn
};
constexpr double kPi = 3.14159265358979323846264338327950288;

// sin and cos of k/256 turn by their Taylor series, the angle brought into
// [0, pi/4] by symmetry (so that the largest term is below 1)
constexpr double turn_series(double x, bool sine) {
    double term = sine ? x : 1.0, sum = term;
    for (int n = 1; n < 14; n++) {
        const double a = sine ? 2.0 * n : 2.0 * n - 1.0;
        term = -term * x * x / (a * (a + 1.0));
        sum += term;
    }
    return sum;
}
constexpr TurnTable make_turn_table() {
    TurnTable t{};
    for (int k = 0; k < kTurnSteps; k++) {
        const int quarter = k / 64, r = k % 64;
        const bool swap = r > 32;
        const double x = 2.0 * kPi * (swap ? 64 - r : r) / kTurnSteps;
        const double a = turn_series(x, false), b = turn_series(x, true);
        const double c0 = swap ? b : a, s0 = swap ? a : b;  // within the first quarter
        const double c = quarter == 0 ? c0 : quarter == 1 ? -s0 : quarter == 2 ? -c0 : s0;
        const double s = quarter == 0 ? s0 : quarter == 1 ? c0 : quarter == 2 ? -s0 : -c0;
        t.v[k][0] = (float)c;
        t.v[k][1] = (float)(c - (double)t.v[k][0]);
        t.v[k][2] = (float)s;
        t.v[k][3] = (float)(s - (double)t.v[k][2]);
    }
    return t;
}
static __device__ const TurnTable g_turn_table = make_turn_table();

// a + b = s + e exactly
__device__ __forceinline__ float two_sum(float a, float b, float* e) {
    const float s = __fadd_rn(a, b), bb = __fsub_rn(s, a);
    *e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb));
    return s;
}

// m * (cos, sin) of `phase` / 2^64 turns as float pairs (x, y) and (z, w)
__device__ __forceinline__ float4 turn_cos_sin(uint64_t phase, float m) {
    const uint64_t near = phase + (1ull << 55);
    const int k = (int)(near >> 56);
    const int64_t rest = (int64_t)(near & ((1ull << 56) - 1)) - (1ll << 55);
    const float4 t = *reinterpret_cast<const float4*>(g_turn_table.v[k]);
    // r = rest * 2 pi / 2^64, rest as 2^32 times its upper half (24 bits: exact) and the lower
    constexpr double kStep = 2.0 * kPi / 18446744073709551616.0;
    constexpr float kHi = (float)kStep, kLo = (float)(kStep - (double)(float)kStep);
    const float nh = 4294967296.0f * (float)(int)(rest >> 32), nl = (float)(uint32_t)rest;
    const float p = __fmul_rn(nh, kHi);
    const float pe = __fmaf_rn(nl, kHi, __fmaf_rn(nh, kLo, __fmaf_rn(nh, kHi, -p)));
    float rl;
    const float rh = two_sum(p, pe, &rl);
    const float zh = __fmul_rn(rh, rh), zl = __fmaf_rn(2.0f * rh, rl, __fmaf_rn(rh, rh, -zh));
    // sin r = rh + sl, cos r - 1 = dh + dl
    const float sl = __fmaf_rn(rh * zh, __fmaf_rn(zh, 1.0f / 120.0f, -1.0f / 6.0f), rl);
    const float dh = -0.5f * zh, dl = __fmaf_rn(zh * zh, __fmaf_rn(zh, -1.0f / 720.0f, 1.0f / 24.0f), -0.5f * zl);
    // C + (C d - S sin r) and S + (S d + C sin r)
    auto join = [&](float ah, float al, float bh, float bl) {  // a + a d + b sin r
        const float u = __fmul_rn(ah, dh), v = __fmul_rn(bh, rh);
        float low = __fadd_rn(__fmaf_rn(ah, dh, -u), __fmaf_rn(bh, rh, -v));
        low = __fmaf_rn(ah, dl, low);
        low = __fmaf_rn(bh, sl, low);
        low = __fmaf_rn(bl, rh, low);
        low = __fmaf_rn(al, dh, low);
        low = __fadd_rn(low, al);
        float e1, e2;
        const float q = two_sum(u, v, &e1);
        const float h = two_sum(ah, q, &e2);
        low = __fadd_rn(low, __fadd_rn(e1, e2));
        // times m, as a pair again
        const float g = __fmul_rn(h, m);
        return make_float2(g, __fmaf_rn(low, m, __fmaf_rn(h, m, -g)));
    };
    const float2 c = join(t.x, t.y, -t.z, -t.w), s = join(t.z, t.w, t.x, t.y);
    return make_float4(c.x, c.y, s.x, s.y);
}

// a c - b s rounded once, c and s float pairs; an infinite or NaN product is
// returned as the plain expression gives it
__device__ __forceinline__ float turn_diff(float a, float b, float ch, float cl, float sh, float sl) {
    const float p = __fmul_rn(a, ch), q = __fmul_rn(b, sh);
    const float pe = __fmaf_rn(a, cl, __fmaf_rn(a, ch, -p)), qe = __fmaf_rn(b, sl, __fmaf_rn(b, sh, -q));
    float e;
    const float r = two_sum(p, -q, &e);
    const float y = __fadd_rn(r, __fadd_rn(e, __fsub_rn(pe, qe)));
    return fabsf(y) <= 3.402823466e38f ? y : r;
}
// (a, b) turned by the angle of cs: (a c - b s, a s + b c)
__device__ __forceinline__ void turn_pair(float& a, float& b, float4 cs) {
    const float y = turn_diff(a, b, cs.x, cs.y, cs.z, cs.w);
    b = turn_diff(a, -b, cs.z, cs.w, cs.x, cs.y);
    a = y;
}

// Rows for the row kernel (kvpages.cu): f32 heads of T tokens, keys and values into a
// cache's pages, queries rotated.
constexpr int kNoPages = -1;  // in the place of a cache type: query rows only

// One thread's share of a head: eight values, of the four pairs 4o .. 4o + 3 (pair p
// < n_rot / 2 is rotated; the values behind n_rot are taken as pairs of neighbours).
// How the pairs lie:
enum RowPairs {
    kPairsNone = 0,       // nothing is rotated
    kPairsHalf = 1,       // (i, i + n_rot/2), n_rot a multiple of 8: a float4 of each half
    kPairsNext = 2,       // (2i, 2i + 1), n_rot a multiple of 8: eight neighbours
    kPairsNextAny = 3,    // the same, any even n_rot
    kPairsScattered = 4,  // (i, i + n_rot/2), any even n_rot: single values
};
struct RowArgs {
    const float* k;
    const float* v;
    const float* q;  // null: no queries
    float* q_out;
    const int32_t* pos;
    const int32_t* seq;  // null: token t belongs to sequence t
    const uint64_t* freqs;
    int64_t T, ldk, ldv, ldq, ldqo;
    int Hq, inverse;
    int n_rot, pairs;  // pairs: a RowPairs
    float mscale;
};
// Where pair p's entry of a token's table lies: the four of a share in four runs, so
// that a warp's lanes read neighbouring entries.
__host__ __device__ __forceinline__ int turn_run(int half) { return (half + 3) >> 2; }
__device__ __forceinline__ int turn_at(int half, int p) { return (p & 3) * turn_run(half) + (p >> 2); }

// The places of a share's values in its head: two float4 at first and second, or (for
// kPairsScattered) value i at a[i], value i + 4 at b[i].
struct Share {
    int first, second, turned;  // turned: pairs of the share that are rotated
};
template <int PAIRS>
__device__ __forceinline__ Share row_share(int n_rot, int o) {
    const int half = n_rot >> 1;
    Share s;
    s.turned = PAIRS == kPairsNone ? 0 : half - 4 * o;
    s.turned = s.turned < 0 ? 0 : (s.turned > 4 ? 4 : s.turned);
    const bool split = PAIRS == kPairsHalf && s.turned > 0;
    s.first = split ? 4 * o : 8 * o;
    s.second = split ? half + 4 * o : 8 * o + 4;
    return s;
}
__device__ __forceinline__ int2 scattered_at(int n_rot, int p) {
    const int half = n_rot >> 1;
    return p < half ? make_int2(p, p + half) : make_int2(2 * p, 2 * p + 1);
}
template <int PAIRS>
__device__ __forceinline__ void row_load8(const Share& s, int n_rot, int o, const float* x, float v[8]) {
    if (PAIRS == kPairsScattered) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int2 at = scattered_at(n_rot, 4 * o + i);
            v[i] = x[at.x];
            v[i + 4] = x[at.y];
        }
        return;
    }
    const float4 a = *reinterpret_cast<const float4*>(x + s.first);
    const float4 b = *reinterpret_cast<const float4*>(x + s.second);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
template <int PAIRS>
__device__ __forceinline__ void row_store8(const Share& s, int n_rot, int o, float* y, const float v[8]) {
    if (PAIRS == kPairsScattered) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int2 at = scattered_at(n_rot, 4 * o + i);
            y[at.x] = v[i];
            y[at.y] = v[i + 4];
        }
        return;
    }
    *reinterpret_cast<float4*>(y + s.first) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(y + s.second) = make_float4(v[4], v[5], v[6], v[7]);
}
// table: the token's, at this share's first pair (entry i is i * turn_run on)
template <int PAIRS>
__device__ __forceinline__ void row_turn8(const Share& s, float v[8], const float4* table, int run) {
    constexpr bool kWhole = PAIRS == kPairsHalf || PAIRS == kPairsNext;  // a share is rotated or it is not
    if constexpr (PAIRS != kPairsNone) {
        if (s.turned == 0) return;
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (kWhole || i < s.turned) {
                const float4 cs = table[i * run];
                if (PAIRS == kPairsNext || PAIRS == kPairsNextAny) turn_pair(v[2 * i], v[2 * i + 1], cs);
                else turn_pair(v[i], v[i + 4], cs);
            }
    }
}

}  // namespace qmm
