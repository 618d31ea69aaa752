// experts_mma.cuh -- the experts' products for many rows, on the 5th-generation tensor cores.
//
//   P[s][n] = W[e_s][n] . x_s        for the rows s of a call, sorted by their expert e_s
//
// sm_103a's tensor cores take no integers, and 32-value blocks have a scale each, so that a fold of every block's sum in
// registers would cost as much as the product.  Both operands are f16 instead, exact or in two terms, and f32 sums leave
// tensor memory every 256 values (128 where both operands have two terms): there one fma a sum multiplies what the row's
// 256 weights share by what the row's 256 activations share.
//   Q4_K, Q5_K, Q2_K   scale times code, a whole number up to 1953 (exact), over the block's d; the minimums over d, in
//                      two terms, times the activations' sums of 16 values (one more step of 16)
//   Q6_K               scale times code, a whole number up to 4096, in two exact terms
//   32-value blocks    the value over a power of two that the row's 256 share, in two terms, hi + lo, exact wherever the
//                      scale is (run_shift in experts_mma.h); the codes of Q4_1 and Q5_1 are centered and the minimums
//                      multiply the sums, as above
//   activations        Q8_K: the codes (exact); Q8_0: the values over a shared power of two, in two terms, likewise
// Products of two-term operands leave out lo lo, up to 2^-22 of a product.  Sums of steps are truncated to f32 by the tensor
// core; with 18 steps to a sum (Q4_K, Q5_K, Q2_K), 24 or, with minimums, 27 (32-value blocks) or 32 (Q6_K), those with a lo
// first, the errors measured are 0.04 to 0.45e-6 of the result.
//
// A tile is 128 weight rows (gated: 64 rows of the gate's and of the up matrix, row by row, so that both sums of an
// output lie in neighbouring lanes) by up to 128 rows of one expert; CTAs, one per SM, walk over the tiles, and a tile's
// last sums are added while the next one's operands are made.  The warps hand each other items, a chunk of 256 values or,
// where weights have two terms, half of one (a handover of 64 values left the issuing warp with 200 cycles an MMA of 64):
//   0-15   converters and epilogue: warp w has the 32 weight rows of lane quadrant w % 4 and of each chunk the blocks of
//          pair w / 4, turned into f16 in its tensor-memory lanes; then, for the chunk before, the sums of 32 activation
//          rows times its 32 weight rows, which it adds up in registers
//   16     issues the MMAs
//   17     copies the activation operands, which come ready made, sorted and laid out in tiles: a bulk copy an item
//          (made here from 8-bit rows by eight warps they took as many instructions as the weights)
//   18-23  copy the weight rows' bytes, 16 to a lane (a bulk copy a row left the copying warp with 84 cycles each, one
//          warp's cp.async come 65 cycles apart)
// Weights are read once per 128 rows of their expert.  What bounds a tile is the converters' warps, their conversions and
// as much again in waits, handovers and tensor-memory traffic, whatever the number of the tile's rows: 10 to 11 thousand
// warp instructions a chunk.  Measured: 16384 rows over 64 experts of Q4_K, 1024 x 2048 twice (137 GFLOP), 265 us, 520
// TFLOP/s, issue slots 72% busy, the tensor pipe 26%; over 64 of Q6_K, 2048 x 1024 (69 GFLOP), 213 us; 96 rows over 8 of
// Q8_0, 4096 x 12288, 235 us; 256 rows over 32 of Q4_0, 1408 x 2048 twice, 97 us.  Not kept, as slower: adding two sums
// with one packed fma (2 to 6%), every group of warps making a block of each item rather than two of one (12%).
#pragma once

#include <cuda.h>

#include "experts.h"
#include "experts_mma.h"
#include "tc_device.cuh"

namespace qmm {

static __device__ unsigned int g_expert_mma_error = 0;

namespace em {

constexpr int BM = 128;       // weight rows of a tile
constexpr int CONV = 16, MMA_WARP = CONV, XCOPY = MMA_WARP + 1, WCOPY = XCOPY + 1, WCOPIES = 6;
constexpr int THREADS = (WCOPY + WCOPIES) * 32;
// Registers a thread: 768 threads start with 80; the converters, with their sums, go up to what the others give away.
constexpr int REGS_CONV = 96, REGS_OTHER = 48;
static_assert(THREADS == 768 && CONV * 32 * REGS_CONV + (THREADS - CONV * 32) * REGS_OTHER <= THREADS * 80, "registers");
constexpr int A_COL0 = 2 * kTileRows;  // after two accumulators
constexpr int XOP = kTileRows * 64;    // bytes of one term of a block's activation operand: 32 values of 128 rows
constexpr int SX_RING = 8;    // chunks of activation scales

template <int WT>
struct Lay {
    using F = Fmt<WT>;
    static constexpr bool KQ = F::BV == 256;
    static constexpr bool MIN = WT == QMM_Q4_1 || WT == QMM_Q5_1 || WT == QMM_Q4_K || WT == QMM_Q5_K || WT == QMM_Q2_K;
    static constexpr int WTERMS = KQ && WT != QMM_Q6_K ? 1 : 2, XTERMS = operand_terms(F::ACT);
    // Items of a chunk, and the blocks of one.  A weight operand has 128 columns of tensor memory, each block 16 of hi and
    // (two terms) 16 of lo; there are two.
    static constexpr int ITEMS = WTERMS, BLOCKS = 8 / ITEMS, BLOCK_COLS = 16 * WTERMS;
    // activation operands: block by block, hi then lo; behind them the sums
    static constexpr int X_SLOTS = WT == QMM_Q6_K ? 4 : 2;
    static constexpr int XSUMS = BLOCKS * XTERMS * XOP, XSLOT = XSUMS + (MIN ? XTERMS * XOP / 2 : 0);
    // the minimums' operand, in shared memory: hi, lo; there are two
    static constexpr int AMIN = MIN ? 2 * BM * 32 : 0;
    // 32-value blocks without minimums: the halves of a chunk are accumulated, and have their powers of two, each for itself;
    // four chunks' powers lie in shared memory
    static constexpr bool HALVES = !KQ && !MIN;
    static constexpr int SW = HALVES ? 4 * 2 * BM * 4 : 0;
    static constexpr int CHUNK = KQ ? F::BB : 8 * F::BB;  // bytes of a row's 256 values
    // a copied row: the 16-byte superset at any offset that blocks can have, an odd number of 16-byte words
    static constexpr int ALIGN = WT == QMM_Q4_K || WT == QMM_Q5_K ? 16 : WT == QMM_Q2_K || WT == QMM_Q4_1 ? 4 : WT == QMM_Q5_1 ? 8 : 2;
    static constexpr int WORDS = (CHUNK + 16 - ALIGN + 15) / 16;
    static constexpr int PITCH = 16 * (WORDS | 1);
    static constexpr int FIXED = X_SLOTS * XSLOT + 2 * AMIN + SX_RING * kTileRows * 4 + SW + 512;
    static constexpr int FIT = (232448 - 128 - FIXED) / (BM * PITCH);
    static constexpr int WST = FIT >= 4 ? 4 : FIT;
    static_assert(FIT >= 2, "two stages of weight rows");
    static constexpr int OFF_W = 0;
    static constexpr int OFF_OP = OFF_W + WST * BM * PITCH;
    static constexpr int OFF_AMIN = OFF_OP + X_SLOTS * XSLOT;
    static constexpr int OFF_SX = OFF_AMIN + 2 * AMIN;
    static constexpr int OFF_SW = OFF_SX + SX_RING * kTileRows * 4;
    static constexpr int OFF_BAR = OFF_SW + SW;
    static constexpr int NBARS = 2 * WST + 2 * X_SLOTS + SX_RING + 2 + 4;
    static constexpr int OFF_TMEM = OFF_BAR + NBARS * 8;
    static constexpr int SMEM = OFF_TMEM + 16;
    static_assert(SMEM <= 232448 && OFF_OP % 128 == 0 && NBARS * 8 + 16 <= 512, "shared memory");
};

template <int WT>
struct Bars {
    using L = Lay<WT>;
    uint32_t base;
    __device__ uint32_t w_full(int s) const { return base + 8u * s; }                       // weight rows landed
    __device__ uint32_t w_empty(int s) const { return base + 8u * (L::WST + s); }           // converted
    __device__ uint32_t x_full(uint32_t m) const { return base + 8u * (2 * L::WST + m % L::X_SLOTS); }  // item m: activations
    __device__ uint32_t sx_full(int i) const { return base + 8u * (2 * L::WST + L::X_SLOTS + i); }  // a chunk's scales landed
    __device__ uint32_t w_op(uint32_t m) const { return base + 8u * (OPS + m % 2); }  // item m: weights written
    // Item m's MMAs are done.  Whoever waits for it has waited for the item before on this barrier: an activation slot's
    // copies are of every item, and a weight converter's items are every (second) one.
    __device__ uint32_t done(uint32_t m) const { return base + 8u * (OPS + 2 + m % L::X_SLOTS); }
    __device__ uint32_t acc_full(int i) const { return base + 8u * (OPS + 2 + L::X_SLOTS + i); }
    __device__ uint32_t acc_empty(int i) const { return base + 8u * (OPS + 2 + L::X_SLOTS + 2 + i); }
    static constexpr int OPS = 2 * L::WST + L::X_SLOTS + SX_RING;
};

__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (mbar_wait_bounded(bar, parity, kWaitLimitNs)) return true;
    atomicOr(&g_expert_mma_error, kErrTimeout);
    *abort_flag = 1;
    return false;
}
// the same for a whole warp, which stays together
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    return __all_sync(0xffffffffu, wait_or_abort(bar, parity, abort_flag));
}

__device__ __forceinline__ uint32_t h2_mul(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t h2_fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t h2_neg(uint32_t a) {
    uint32_t d;
    asm("neg.f16x2 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
// 16 bytes (of which `bytes` are read, zeros behind them) into shared memory; the arrival is counted when this thread's
// copies so far have landed.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ uint32_t h2_dup(uint32_t h) { return (h & 0xFFFFu) * 0x10001u; }
// v as two f16, each in both halves of a word
__device__ __forceinline__ void split2(float v, uint32_t* hi, uint32_t* lo) {
    const uint32_t h = f2h_bits(v);
    *hi = h2_dup(h);
    *lo = h2_dup(f2h_bits(v - h2f(h)));
}
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }
__device__ __forceinline__ uint32_t pow2_half(int e) { return (uint32_t)(e + 15) << 10; }  // -14 <= e <= 15

// What the blocks of a row's chunk share: what their sums are multiplied by; the power that 32-value blocks are multiplied
// by, or what the scales and minimums are multiplied by over it (K-quants); the first 16 bytes of a Q4_K or
// Q5_K block.
struct WRow {
    float scale;
    int shift;
    float value, min;
    uint4 head;
};
// What is taken from the codes of Q4_1 and Q5_1, so that neither the products nor the minimums' share are much larger than
// their sum (the minimum gets it back times the scale).
template <int WT>
constexpr int center() {
    return WT == QMM_Q4_1 ? 8 : WT == QMM_Q5_1 ? 16 : 0;
}

// The 32 codes of block kb of the chunk at byte `o` of the row, in K order, four to a word (Q4_K: 16 times those of odd
// blocks), and the f16 offset word.
template <int WT>
__device__ __forceinline__ uint32_t codes_of(const SmemBytes& w, uint32_t o, int kb, uint32_t (&c)[8]) {
    if constexpr (WT == QMM_Q8_0) {
        w.words<8>(o + 34 * kb + 2, c);
#pragma unroll
        for (int i = 0; i < 8; i++) c[i] ^= 0x80808080u;
        return 0x64806480u;
    } else if constexpr (WT == QMM_Q4_0 || WT == QMM_Q4_1 || WT == QMM_Q5_0 || WT == QMM_Q5_1) {
        constexpr bool FIVE = WT == QMM_Q5_0 || WT == QMM_Q5_1;
        const uint32_t b = o + Fmt<WT>::BB * kb;
        uint32_t q[5];
        uint32_t qh = 0;
        if constexpr (WT == QMM_Q4_0) w.words<4>(b + 2, q);
        if constexpr (WT == QMM_Q4_1) w.words_aligned<4>(b + 4, q);
        if constexpr (WT == QMM_Q5_0) {
            w.words<5>(b + 2, q);
            qh = q[0], q[0] = q[1], q[1] = q[2], q[2] = q[3], q[3] = q[4];
        }
        if constexpr (WT == QMM_Q5_1) {
            qh = w.w32(b + 4);
            w.words_aligned<4>(b + 8, q);
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
            c[i] = q[i] & 0x0F0F0F0Fu;
            c[4 + i] = (q[i] >> 4) & 0x0F0F0F0Fu;
            if constexpr (FIVE) {
                c[i] |= spread4(qh >> (4 * i)) << 4;
                c[4 + i] |= spread4(qh >> (16 + 4 * i)) << 4;
            }
        }
        return WT == QMM_Q4_0 || WT == QMM_Q4_1 ? 0x64086408u : 0x64106410u;
    } else if constexpr (WT == QMM_Q4_K || WT == QMM_Q5_K) {
        const uint32_t b = o + (WT == QMM_Q4_K ? 16 : 48) + 32 * (kb >> 1);
        const uint4 q0 = *reinterpret_cast<const uint4*>(w.base + b), q1 = *reinterpret_cast<const uint4*>(w.base + b + 16);
        const uint32_t q[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
#pragma unroll
        for (int i = 0; i < 8; i++)
            c[i] = WT == QMM_Q4_K ? q[i] & (kb & 1 ? 0xF0F0F0F0u : 0x0F0F0F0Fu) : (q[i] >> (4 * (kb & 1))) & 0x0F0F0F0Fu;
        if constexpr (WT == QMM_Q5_K) {
            const uint4 h0 = *reinterpret_cast<const uint4*>(w.base + o + 16), h1 = *reinterpret_cast<const uint4*>(w.base + o + 32);
            const uint32_t h[8] = {h0.x, h0.y, h0.z, h0.w, h1.x, h1.y, h1.z, h1.w};
#pragma unroll
            for (int i = 0; i < 8; i++) c[i] |= ((h[i] >> kb) & 0x01010101u) << 4;
        }
        return 0x64006400u;
    } else if constexpr (WT == QMM_Q2_K) {
        uint32_t q[8];
        w.words_aligned<8>(o + 16 + 32 * (kb >> 2), q);
        const int sh = 2 * (kb & 3);
#pragma unroll
        for (int i = 0; i < 8; i++) c[i] = (q[i] >> sh) & 0x03030303u;
        return 0x64006400u;
    } else {  // Q6_K
        const int half = kb >> 2, part = kb & 3;
        uint32_t q[8], h[8];
        w.words<8>(o + 64 * half + 32 * (part & 1), q);
        w.words<8>(o + 128 + 32 * half, h);
        const int sh = 4 * (part >> 1), hs = 2 * part;
#pragma unroll
        for (int i = 0; i < 8; i++) c[i] = ((q[i] >> sh) & 0x0F0F0F0Fu) | (((h[i] >> hs) & 0x03030303u) << 4);
        return 0x64206420u;
    }
}

// A K-quant block's sums are over its d, unless its minimums' scale m is over 1000 times that (hardly any weights have that)
// and not all minimums are zero: then over d times such a power of two, 2^-10 to 2^-8 of m, that minimums up to 63 times
// their scale stay f16.  Minimums, two f16, keep 2^-22 of themselves or 2^-25 of what the sums are over.  Scale times code
// is exact where that power is at most 2^20, m at most 2^29 d; beyond, the scale (Q4_K: a 16th of it, times 16 code) is
// rounded by up to 2^-25 of what the sums are over, and scale times code by up to 2^-25 m.
template <class None>
__device__ __forceinline__ WRow shared_scale(float d, float m, None none) {
    float D = d, value = 1.0f;
    if (!(fabsf(m) <= 1000.0f * fabsf(d)) && !(isfinite(m) && none())) {
        if (d == 0.0f) {
            D = m, value = 0.0f;
        } else {
            const int p = ((__float_as_int(m) >> 23) & 255) - ((__float_as_int(d) >> 23) & 255) - 9;
            const int up = p < 0 ? 0 : p > 60 ? 60 : p;
            D = d * pow2(up), value = pow2(-up);
        }
    }
    const float inv = D != 0.0f ? __fdividef(1.0f, D) : 0.0f;  // 2 units of 2^-23, of what is 2^-22 in two terms
    return {D, 0, value, -(m * inv), make_uint4(0u, 0u, 0u, 0u)};
}

template <int WT>
__device__ __forceinline__ WRow row_scale(const SmemBytes& w, uint32_t o, int half, int blocks) {
    if constexpr (WT == QMM_Q4_K || WT == QMM_Q5_K) {
        const uint4 head = *reinterpret_cast<const uint4*>(w.base + o);
        WRow r = shared_scale(h2f(head.x), h2f(head.x >> 16), [&] { return (head.z | (head.w & 0xF0F0F0F0u)) == 0u; });
        r.head = head;
        return r;
    } else if constexpr (WT == QMM_Q2_K) {
        const uint32_t dd = w.w32(o + 80);
        return shared_scale(h2f(dd), h2f(dd >> 16), [&] {
            uint32_t sc[4];
            w.words_aligned<4>(o, sc);
            return ((sc[0] | sc[1] | sc[2] | sc[3]) & 0xF0F0F0F0u) == 0u;
        });
    } else if constexpr (WT == QMM_Q6_K) {
        return {h2f(w.u16(o + 208)), 0, 1.0f, 0.0f, make_uint4(0u, 0u, 0u, 0u)};
    } else {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < (Lay<WT>::HALVES ? 4 : 8); i++) {
            const int kb = (Lay<WT>::HALVES ? 4 * half : 0) + i;
            if (kb >= blocks) break;
            const uint32_t b = o + Fmt<WT>::BB * kb;
            if constexpr (Lay<WT>::MIN) {
                const uint32_t dm = w.w32(b);
                top = max(top, max(dm & 0x7FFFu, (dm >> 16) & 0x7FFFu));
            } else {
                top = max(top, w.u16(b) & 0x7FFFu);
            }
        }
        const int shift = run_shift(top, weight_spare(WT));
        return {pow2(-shift), shift, 0.0f, 0.0f, make_uint4(0u, 0u, 0u, 0u)};
    }
}

// 6-bit field b (0-7) of a Q4_K header: low six bits of byte b of `first` for b < 4; else four low bits of byte b - 4 of
// `second` under the two top bits of that byte of `top`.
__device__ __forceinline__ uint32_t six_bits(int b, uint32_t first, uint32_t second, uint32_t top) {
    const int sh = 8 * (b & 3);
    return b < 4 ? (first >> sh) & 63u : ((second >> sh) & 15u) | (((top >> sh) >> 6) & 3u) << 4;
}

// Block kb of a row's chunk as f16 words in K order: hi and (two terms) lo.
template <int WT>
__device__ __forceinline__ void convert_block(const SmemBytes& w, uint32_t o, int kb, const WRow& row, uint32_t (&hi)[16],
                                              uint32_t (&lo)[16]) {
    uint32_t c[8];
    const uint32_t magic = codes_of<WT>(w, o, kb, c);
    // the scales of the block's two halves
    uint32_t d0, d1;
    if constexpr (WT == QMM_Q4_K || WT == QMM_Q5_K) {
        const float over = WT == QMM_Q4_K && (kb & 1) ? 0.0625f : 1.0f;
        d0 = d1 = h2_dup(f2h_bits(row.value * over * (float)six_bits(kb, row.head.y, row.head.w, row.head.y)));
    } else if constexpr (WT == QMM_Q2_K) {
        const uint32_t sc = w.u16(o + 2 * kb);
        d0 = h2_dup(f2h_bits(row.value * (float)(sc & 15u))), d1 = h2_dup(f2h_bits(row.value * (float)((sc >> 8) & 15u)));
    } else if constexpr (WT == QMM_Q6_K) {
        const uint32_t sc = w.u16(o + 192 + 2 * kb);
        d0 = h2_dup(f2h_bits((float)(int8_t)(sc & 0xFFu))), d1 = h2_dup(f2h_bits((float)(int8_t)(sc >> 8)));
    } else {
        d0 = d1 = h2_mul(h2_dup(w.u16(o + Fmt<WT>::BB * kb)), h2_dup(pow2_half(row.shift)));
    }
    if constexpr (Lay<WT>::WTERMS == 1) {
        // scale (1024 + code) - 1024 scale: every part is an f16 and so is the result
        const uint32_t c0 = h2_mul(d0, 0xE400E400u), c1 = h2_mul(d1, 0xE400E400u);
#pragma unroll
        for (int i = 0; i < 8; i++) {
            hi[2 * i] = h2_fma(i < 4 ? d0 : d1, bytes_to_h2(c[i], 0x5140), i < 4 ? c0 : c1);
            hi[2 * i + 1] = h2_fma(i < 4 ? d0 : d1, bytes_to_h2(c[i], 0x7362), i < 4 ? c0 : c1);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const uint32_t d = i < 4 ? d0 : d1;
            const uint32_t q0 = h2_sub(bytes_to_h2(c[i], 0x5140), magic), q1 = h2_sub(bytes_to_h2(c[i], 0x7362), magic);
            hi[2 * i] = h2_mul(d, q0), hi[2 * i + 1] = h2_mul(d, q1);
            lo[2 * i] = h2_fma(d, q0, h2_neg(hi[2 * i])), lo[2 * i + 1] = h2_fma(d, q1, h2_neg(hi[2 * i + 1]));
        }
    }
}

// The chunk's minimums over 16 groups of 16 values (Q4_1, Q5_1: with what the codes gave away), as hi and lo: what an
// activation group's sum is multiplied by.
template <int WT>
__device__ __forceinline__ void convert_min(const SmemBytes& w, uint32_t o, int blocks, const WRow& row, uint32_t (&hi)[8],
                                            uint32_t (&lo)[8]) {
    if constexpr (WT == QMM_Q4_1 || WT == QMM_Q5_1) {
        const float f = pow2(row.shift);
#pragma unroll
        for (int b = 0; b < 8; b++) {
            const uint32_t dm = b < blocks ? w.w32(o + Fmt<WT>::BB * b) : 0u;
            split2(fmaf((float)center<WT>(), h2f(dm), h2f(dm >> 16)) * f, &hi[b], &lo[b]);
        }
    } else if constexpr (WT == QMM_Q4_K || WT == QMM_Q5_K) {
#pragma unroll
        for (int b = 0; b < 8; b++)
            split2(row.min * (float)six_bits(b, row.head.z, row.head.w >> 4, row.head.z), &hi[b], &lo[b]);
    } else if constexpr (WT == QMM_Q2_K) {
        uint32_t sc[4];
        w.words_aligned<4>(o, sc);
#pragma unroll
        for (int b = 0; b < 8; b++) {
            const uint32_t two = sc[b >> 1] >> (16 * (b & 1));
            uint32_t h0, l0, h1, l1;
            split2(row.min * (float)((two >> 4) & 15u), &h0, &l0);
            split2(row.min * (float)((two >> 12) & 15u), &h1, &l1);
            hi[b] = (h0 & 0xFFFFu) | (h1 << 16), lo[b] = (l0 & 0xFFFFu) | (l1 << 16);
        }
    }
}

// The MMA with A in tensor memory and B in shared memory, K-major core matrices 128 bytes apart along K and `sbo` along N:
// `x` is B's address over 16.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t x, uint32_t sbo, uint32_t idesc, bool add) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 b;\n mov.b64 b, {%2, %3};\n setp.ne.u32 p, %5, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n}\n" ::"r"(d),
        "r"(a), "r"(x | 128u >> 4 << 16), "r"(sbo >> 4 | 1u << 14), "r"(idesc), "r"(add ? 1u : 0u)
        : "memory");
}
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}
template <int WT, bool GATED>
__global__ void __launch_bounds__(THREADS, 1) expert_mma_kernel(const __grid_constant__ ExpertMma a) {
    using L = Lay<WT>;
    pdl_launch_dependents();
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    if (!QMM_IN_BOUNDS(g_expert_mma_error, L::SMEM - 1, dynamic_smem_bytes())) return;
    const Bars<WT> bars{sbase + L::OFF_BAR};
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_TMEM);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_TMEM + 8);
    float* const sx = reinterpret_cast<float*>(smem + L::OFF_SX);
    float* const sw = reinterpret_cast<float*>(smem + L::OFF_SW);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < L::WST; i++) mbar_init(bars.w_full(i), WCOPIES * 32), mbar_init(bars.w_empty(i), CONV);
        for (int i = 0; i < L::X_SLOTS; i++) mbar_init(bars.x_full(i), 1), mbar_init(bars.done(i), 1);
        for (int i = 0; i < SX_RING; i++) mbar_init(bars.sx_full(i), 1);
        for (int i = 0; i < 2; i++) mbar_init(bars.w_op(i), CONV / L::ITEMS);
        for (int i = 0; i < 2; i++) mbar_init(bars.acc_full(i), 1), mbar_init(bars.acc_empty(i), CONV);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == MMA_WARP) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();  // the tiles and the activation records come from the kernel before

    constexpr int NROWS = GATED ? BM / 2 : BM;  // output columns of a tile
    const int N = a.N;
    const int nt = (N + NROWS - 1) / NROWS;
    const int nb = a.K / 32;
    const int nchunks = (a.K + 255) / 256;
    const int ntiles = *a.ntiles * nt;
    const uint64_t rb = (uint64_t)(a.K / Fmt<WT>::BV) * Fmt<WT>::BB;
    const uint64_t total = (uint64_t)a.E * (uint64_t)N * rb;
    auto blocks_of = [&](int c) { return L::KQ ? 8 : min(8, nb - 8 * c); };
    // the weight row of tile row r (rows behind the last repeat it)
    auto weight_row = [&](const ExpertTile& t, int n0, int r) {
        const int n = min(n0 + (GATED ? r >> 1 : r), N - 1);
        return (int64_t)t.expert * N + n;
    };

    if (warp < CONV) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_CONV));
        // ------------------------------------------------------------ weight operands, sums
        const int quad = warp & 3, grp = warp >> 2;
        const int r = quad * 32 + lane;  // tile row
        const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
        float acc[32];
#pragma unroll
        for (int j = 0; j < 32; j++) acc[j] = 0.0f;
        uint32_t gc = 0, folded = 0;  // chunks, accumulations
        bool ok = true;
        // The chunk before: its sums are added while the MMAs of the next run, also across tiles.
        bool pending = false, pending_last = false;
        float pending_scale = 0.0f;
        int pending_halves = 0, pending_n0 = 0, pending_count = 0, pending_slot = 0;  // lane j: the choice of row 32 grp + j
        // adds the next accumulation of the pending chunk, times its scales, to the registers
        auto fold = [&](int half) {
            const uint32_t buf = folded & 1, of = gc - 1;
            if (!warp_wait(bars.acc_full((int)buf), (folded / 2) & 1u, abort_flag)) return false;
            if (!warp_wait(bars.sx_full((int)(of % SX_RING)), (of / SX_RING) & 1u, abort_flag)) return false;
            folded++;
            tc_fence_after();
            if (grp * 32 < pending_count) {
                const uint32_t cols = lanes + buf * kTileRows + (uint32_t)(grp * 32);
                const uint4* s4 = reinterpret_cast<const uint4*>(sx + of % SX_RING * kTileRows + grp * 32);
                const uint32_t sb = __float_as_uint(L::HALVES ? sw[((of & 3) * 2 + half) * BM + r] : pending_scale);
                const uint64_t s2 = f2_pack(sb, sb);
                uint32_t v[2][8];
                tmem_ld8(cols, v[0]);
                tmem_ld_wait_regs8(v[0]);
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    if (q < 3) tmem_ld8(cols + 8 * (q + 1), v[(q + 1) & 1]);
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        const uint4 s = s4[2 * q + h];
                        const uint32_t* u = v[q & 1] + 4 * h;
                        float* o = acc + 8 * q + 4 * h;
                        const uint64_t p0 = f2_mul(s2, f2_pack(s.x, s.y)), p1 = f2_mul(s2, f2_pack(s.z, s.w));
                        o[0] = fmaf(__uint_as_float(u[0]), __uint_as_float((uint32_t)p0), o[0]);
                        o[1] = fmaf(__uint_as_float(u[1]), __uint_as_float((uint32_t)(p0 >> 32)), o[1]);
                        o[2] = fmaf(__uint_as_float(u[2]), __uint_as_float((uint32_t)p1), o[2]);
                        o[3] = fmaf(__uint_as_float(u[3]), __uint_as_float((uint32_t)(p1 >> 32)), o[3]);
                    }
                    if (q < 3) tmem_ld_wait_regs8(v[(q + 1) & 1]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.acc_empty((int)buf));
            return true;
        };
        // writes the finished sums of a tile
        auto finish = [&] {
            const int n0 = pending_n0;
            if constexpr (GATED) {
                const int col = n0 + quad * 16 + (lane >> 1);
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    if (grp * 32 + j >= pending_count) break;  // the whole warp
                    // even lanes hold the gate's sum and take token j, odd ones the up sum and token j + 1
                    const float other = __shfl_xor_sync(0xffffffffu, lane & 1 ? acc[j] : acc[j + 1], 1);
                    const float g = lane & 1 ? other : acc[j], u = lane & 1 ? acc[j + 1] : other;
                    const int64_t o = (int64_t)__shfl_sync(0xffffffffu, pending_slot, j + (lane & 1)) * N + col;
                    if (grp * 32 + j + (lane & 1) < pending_count && col < N) {
                        if (QMM_IN_BOUNDS(g_expert_mma_error, o, a.out_values)) a.y[o] = gated(a.kind, g, u);
                    }
                }
            } else {
                const int col = n0 + r;
#pragma unroll
                for (int j = 0; j < 32; j++) {
                    if (grp * 32 + j >= pending_count) break;
                    const int64_t o = (int64_t)__shfl_sync(0xffffffffu, pending_slot, j) * N + col;
                    if (col < N && QMM_IN_BOUNDS(g_expert_mma_error, o, a.out_values)) a.y[o] = acc[j];
                }
            }
#pragma unroll
            for (int j = 0; j < 32; j++) acc[j] = 0.0f;
        };
        ExpertTile next = blockIdx.x < ntiles ? a.tiles[blockIdx.x / nt] : ExpertTile{};
        for (int ti = blockIdx.x; ti < ntiles && ok; ti += gridDim.x) {
            const ExpertTile t = next;
            if (ti + (int)gridDim.x < ntiles) next = a.tiles[(ti + gridDim.x) / nt];
            const int n0 = ti % nt * NROWS;
            const uint32_t row = (uint32_t)((uint64_t)weight_row(t, n0, r) * rb);  // modulo 2^32: its low bits are used
            const int slot_of = grp * 32 + lane < t.count ? a.order[t.first + grp * 32 + lane] : 0;
            for (int c = 0; c < nchunks; c++, gc++) {
                const uint32_t s = gc % L::WST;
                const int blocks = blocks_of(c);
                if (!(ok = warp_wait(bars.w_full(s), (gc / L::WST) & 1u, abort_flag))) break;
                const SmemBytes w{smem + L::OFF_W + (s * BM + r) * L::PITCH};
                const uint32_t o = (row + (uint32_t)(c * L::CHUNK)) & 15u;
                const WRow ws = row_scale<WT>(w, o, grp >> 1, blocks);
                if (L::HALVES && !(grp & 1)) sw[((gc & 3) * 2 + (grp >> 1)) * BM + r] = ws.scale;
                // this warp's blocks of its item, once the MMAs of the one before in its place are done
                const uint32_t m = L::ITEMS * gc + (L::ITEMS == 2 ? grp >> 1 : 0);
                if (m >= 2 && !(ok = warp_wait(bars.done(m - 2), ((m - 2) / L::X_SLOTS) & 1u, abort_flag))) break;
                tc_fence_after();
                const uint32_t slot = lanes + (uint32_t)A_COL0 + (m & 1) * 128 + (2 * grp % L::BLOCKS) * L::BLOCK_COLS;
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    if (L::KQ || 2 * grp + h < blocks) {
                        uint32_t hi[16], lo[16];
                        convert_block<WT>(w, o, 2 * grp + h, ws, hi, lo);
                        tmem_st16(slot + L::BLOCK_COLS * h, hi);
                        if constexpr (L::WTERMS == 2) tmem_st16(slot + L::BLOCK_COLS * h + 16, lo);
                    }
                    // in between, the first half of the chunk before: the MMAs of this one wait for it
                    if (!L::KQ && h == 0 && ok && pending && pending_halves == 2) ok = fold(0);
                }
                if (!ok) break;
                if constexpr (L::MIN) {
                    // the minimums go with the chunk's last item, by one of its groups in turn
                    if (grp == (L::ITEMS == 1 ? (int)(gc & 3) : 2 * (blocks > 4) + (int)(gc & 1))) {
                        uint32_t hi[8], lo[8];
                        convert_min<WT>(w, o, blocks, ws, hi, lo);
                        uint8_t* const at = smem + L::OFF_AMIN + (gc & 1) * L::AMIN + (r >> 3) * 256 + (r & 7) * 16;
                        *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4*>(at + 128) = make_uint4(hi[4], hi[5], hi[6], hi[7]);
                        *reinterpret_cast<uint4*>(at + BM * 32) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                        *reinterpret_cast<uint4*>(at + BM * 32 + 128) = make_uint4(lo[4], lo[5], lo[6], lo[7]);
                        fence_proxy_async_smem();
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bars.w_op(m)), mbar_arrive(bars.w_empty(s));
                if (pending) {
                    if (!(ok = fold(pending_halves - 1))) break;
                    if (pending_last) finish();
                }
                pending = true, pending_last = c + 1 == nchunks, pending_scale = ws.scale;
                pending_halves = !L::KQ && blocks > 4 ? 2 : 1, pending_count = t.count, pending_n0 = n0, pending_slot = slot_of;
            }
        }
        if (ok && pending && (pending_halves == 1 || fold(0)) && fold(pending_halves - 1)) finish();
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OTHER));
        if (warp >= WCOPY) {
            // -------------------------------------------------------- the weight rows' bytes
            // Lanes 0-15 and 16-31 have a row each (gated: of the gate's and of the up matrix), a lane the 16-byte word
            // lane % 16 of the row's aligned superset, four instructions a step: the words of all 128 rows are copied,
            // also behind a row's end or the expert's last row, where the next ones' bytes lie.  Only tiles near the last
            // row of all leave out what is not there.
            const int half = lane >> 4, p = lane & 15, me = warp - WCOPY;
            const uint8_t* const W = GATED && half ? a.W1 : a.W0;
            const uint32_t step = (uint32_t)rb * (GATED ? 1 : 2);  // warp j takes steps j, j + 3, ...
            uint32_t gc = 0;
            bool ok = true;
            for (int ti = blockIdx.x; ti < ntiles && ok; ti += gridDim.x) {
                const int expert = a.tiles[ti / nt].expert, n0 = ti % nt * NROWS;
                const uint64_t first = ((uint64_t)expert * N + n0) * rb;  // of the tile's rows
                for (int c = 0; c < nchunks; c++, gc++) {
                    const uint32_t s = gc % L::WST;
                    if (gc >= L::WST && !warp_wait(bars.w_empty(s), (gc / L::WST - 1) & 1u, abort_flag)) {
                        ok = false;
                        break;
                    }
                    const uint64_t at = first + (uint64_t)c * L::CHUNK;
                    const uint32_t stage = sbase + L::OFF_W + s * (BM * L::PITCH);
                    if (at + (uint64_t)(NROWS - 1) * rb + 16 * L::WORDS <= total) {
                        const uint64_t from = at & ~15ull;
                        const uint8_t* const src = W + from + 16 * p;
                        uint32_t off = (uint32_t)(at - from) + (GATED ? 0u : half * (uint32_t)rb) + me * step;
                        const uint32_t dst = stage + (2 * me + half) * L::PITCH + 16 * p;
                        if (p < L::WORDS)
#pragma unroll 11
                            for (int i = 0; i < (BM / 2 + WCOPIES - 1) / WCOPIES; i++) {
                                if (WCOPIES * i + me < BM / 2)
                                    copy16(dst + i * (2 * WCOPIES * L::PITCH), src + (off & ~15u), 16u);
                                off += WCOPIES * step;
                            }
                        if constexpr (L::WORDS > 16) {  // the words behind the 16th: lanes 2 i and 2 i + 1 have row i's
                            static_assert(L::WORDS == 18, "two words are left");
                            const int q = lane >> 1;
                            const uint8_t* const src2 = (GATED && (q & 1) ? a.W1 : a.W0) + from + 256 + 16 * (lane & 1);
                            uint32_t off2 = (uint32_t)(at - from) + (uint32_t)(GATED ? q >> 1 : q) * (uint32_t)rb;
                            const uint32_t dst2 = stage + q * L::PITCH + 256 + 16 * (lane & 1);
#pragma unroll
                            for (int i = 0; i < BM / 16; i++) {
                                if (i % WCOPIES == me) copy16(dst2 + i * (16 * L::PITCH), src2 + (off2 & ~15u), 16u);
                                off2 += 8 * step;
                            }
                        }
                    } else {
                        const uint32_t bytes = L::KQ ? L::CHUNK : blocks_of(c) * Fmt<WT>::BB;
                        for (int i = 32 * me + lane; i < BM * L::WORDS; i += 32 * WCOPIES) {
                            const int r = i / L::WORDS, w = i - r * L::WORDS, n = GATED ? r >> 1 : r;
                            const uint64_t g0 = at + (uint64_t)n * rb, from = (g0 & ~15ull) + 16 * w;
                            if (n0 + n < N && from < g0 + bytes && QMM_IN_BOUNDS(g_expert_mma_error, from, total))
                                copy16(stage + r * L::PITCH + 16 * w, (GATED && (r & 1) ? a.W1 : a.W0) + from,
                                       (uint32_t)min((uint64_t)16, total - from));
                        }
                    }
                    copies_arrive(bars.w_full(s));
                }
            }
            copies_wait();
        } else if (warp == MMA_WARP) {
            // -------------------------------------------------------- the MMAs
            // The whole warp walks, so that addresses and descriptors stay in uniform registers; one lane issues.
            const bool leader = elect_one();
            uint32_t acc = 0, m = 0, c0 = 0;  // accumulations, items, chunks of the tiles before
            bool ok = true;
            for (int ti = blockIdx.x; ti < ntiles && ok; ti += gridDim.x) {
                const uint32_t rows = (uint32_t)(a.tiles[ti / nt].count + 15) & ~15u;
                const uint32_t idesc = instr_desc_f16(BM, (int)rows);
                const uint32_t term = rows * 64 >> 4;  // of a block's activations, in descriptor units
                for (int c = 0; c < nchunks && ok; c++) {
                    const int blocks = blocks_of(c);
#pragma unroll
                    for (int h = 0; h < L::ITEMS; h++, m++) {
                        const int mine = min(blocks - h * L::BLOCKS, L::BLOCKS);  // a last chunk's second item may be empty
                        const bool last = L::ITEMS == 1 || (blocks > 4) == h;     // of the chunk's
                        const uint32_t d = tmem + (acc & 1) * kTileRows;
                        if ((!L::KQ || h == 0) && mine > 0 && acc >= 2 &&
                            !(ok = warp_wait(bars.acc_empty(acc & 1), (acc / 2 - 1) & 1u, abort_flag)))
                            break;
                        if (!(ok = warp_wait(bars.x_full(m), (m / L::X_SLOTS) & 1u, abort_flag)) ||
                            !(ok = warp_wait(bars.w_op(m), (m / 2) & 1u, abort_flag)))
                            break;
                        tc_fence_after();
                        const uint32_t ah = tmem + (uint32_t)A_COL0 + (m & 1) * 128;
                        const uint32_t op = sbase + L::OFF_OP + m % L::X_SLOTS * L::XSLOT;
                        if (leader) {
                            // the accumulation's first MMA starts its sums
                            bool add = L::KQ && h > 0;
                            // the products with a lo come first: small sums lose less to truncation (half the error of
                            // hi and lo in turn, at the same speed)
                            if constexpr (L::WTERMS == 2) {
                                uint32_t x = op >> 4;
#pragma unroll
                                for (int b = 0; b < L::BLOCKS; b++) {
                                    if (!L::KQ && b >= mine) break;
#pragma unroll
                                    for (int k = 0; k < 2; k++) {
                                        const uint32_t al = ah + L::BLOCK_COLS * b + 8 * k, xh = x + 16 * k;
                                        mma_ts(d, al + 16, xh, 512, idesc, add);
                                        add = true;
                                        if constexpr (L::XTERMS == 2) mma_ts(d, al, xh + term, 512, idesc, true);
                                    }
                                    x += L::XTERMS * term;
                                }
                            }
                            const uint64_t min = smem_desc(sbase + L::OFF_AMIN + ((c0 + c) & 1) * L::AMIN, 128, 256);
                            const uint64_t sums = smem_desc(op + L::XSUMS, 128, 256);
                            if (L::MIN && L::WTERMS == 2 && last) {
                                mma_f16(d, min + (BM * 32 >> 4), sums, idesc, 1);
                                mma_f16(d, min, sums + (rows * 32 >> 4), idesc, 1);
                            }
                            uint32_t x = op >> 4;
#pragma unroll
                            for (int b = 0; b < L::BLOCKS; b++) {
                                if (!L::KQ && b >= mine) break;
#pragma unroll
                                for (int k = 0; k < 2; k++) {
                                    mma_ts(d, ah + L::BLOCK_COLS * b + 8 * k, x + 16 * k, 512, idesc, add);
                                    add = true;
                                }
                                x += L::XTERMS * term;
                            }
                            if (L::MIN && last) {  // hi and lo of the minimums, 16 sums a row
                                if constexpr (L::WTERMS == 1) mma_f16(d, min + (BM * 32 >> 4), sums, idesc, 1);
                                mma_f16(d, min, sums, idesc, 1);
                            }
                            mma_commit(bars.done(m));
                            if (L::KQ ? last : mine > 0) mma_commit(bars.acc_full(acc & 1));
                        }
                        if (L::KQ ? last : mine > 0) acc++;
                        __syncwarp();
                    }
                }
                c0 += nchunks;
            }
            // the last commits land before the CTA ends
            for (uint32_t i = m > L::X_SLOTS ? m - L::X_SLOTS : 0; i < m; i++)
                mbar_wait_bounded(bars.done(i), (i / L::X_SLOTS) & 1u, kWaitLimitNs);
        } else if (elect_one()) {
            // -------------------------------------------------------- the activation operands' copies
            uint32_t gc = 0, m = 0;
            bool ok = true;
            for (int ti = blockIdx.x; ti < ntiles && ok; ti += gridDim.x) {
                const ExpertTile t = a.tiles[ti / nt];
                const uint32_t rows = (uint32_t)(t.count + 15) & ~15u;
                constexpr uint32_t ROW = operand_bytes(Fmt<WT>::ACT);  // of a row's chunk
                const uint8_t* src = a.operand + (uint64_t)t.at * (uint64_t)nchunks * ROW;
                for (int c = 0; c < nchunks && ok; c++, gc++, src += rows * ROW) {
                    const int blocks = blocks_of(c);
                    const uint8_t* const sums = src + 8 * L::XTERMS * 64 * rows;
                    for (int h = 0; h < L::ITEMS; h++, m++) {
                        if (m >= L::X_SLOTS && !(ok = wait_or_abort(bars.done(m), (m / L::X_SLOTS - 1) & 1u, abort_flag))) break;
                        if (h == 0) {
                            const uint32_t bar = bars.sx_full((int)(gc % SX_RING));
                            mbar_arrive_expect_tx(bar, rows * 4);
                            bulk_g2s_nohint(sbase + L::OFF_SX + gc % SX_RING * (kTileRows * 4),
                                            sums + L::XTERMS * 32 * rows, rows * 4, bar);
                        }
                        const uint32_t dst = sbase + L::OFF_OP + m % L::X_SLOTS * L::XSLOT;
                        const uint32_t bytes = L::XTERMS * 64 * rows * (uint32_t)max(0, min(blocks - h * L::BLOCKS, L::BLOCKS));
                        const uint32_t sbytes = L::MIN && (L::ITEMS == 1 || (blocks > 4) == h) ? L::XTERMS * 32 * rows : 0u;
                        mbar_arrive_expect_tx(bars.x_full(m), bytes + sbytes);
                        if (bytes) bulk_g2s_nohint(dst, src + h * L::BLOCKS * L::XTERMS * 64 * rows, bytes, bars.x_full(m));
                        if (sbytes) bulk_g2s_nohint(dst + L::XSUMS, sums, sbytes, bars.x_full(m));
                    }
                }
            }
            if (!ok) {  // after a timeout: the copies in flight land before the CTA ends
                for (uint32_t i = m > L::X_SLOTS ? m - L::X_SLOTS : 0; i < m; i++)
                    mbar_wait_bounded(bars.x_full(i), (i / L::X_SLOTS) & 1u, kWaitLimitNs);
                for (uint32_t i = gc > 2 ? gc - 2 : 0; i < gc; i++)
                    mbar_wait_bounded(bars.sx_full((int)(i % SX_RING)), (i / SX_RING) & 1u, kWaitLimitNs);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == MMA_WARP) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

}  // namespace em

template <int WT, bool GATED>
static qmm_status expert_mma_launch(const ExpertMma& a, int64_t tiles_most, cudaStream_t stream) {
    using L = em::Lay<WT>;
    DeviceInfo dev;
    qmm_status st = current_device(&dev);
    if (st != QMM_OK) return st;
    static PerDeviceOnce once;
    st = once.run(dev.device, [] {
        auto* f = em::expert_mma_kernel<WT, GATED>;
        // the converters' registers come out of what the launch has
        cudaFuncAttributes at;
        if (cudaFuncGetAttributes(&at, f) != cudaSuccess) return QMM_E_CUDA;
        if (at.numRegs * em::THREADS < em::CONV * 32 * em::REGS_CONV + (em::THREADS - em::CONV * 32) * em::REGS_OTHER)
            return QMM_E_CUDA;
        return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM) == cudaSuccess ? QMM_OK : QMM_E_CUDA;
    });
    if (st != QMM_OK) return st;
    const int64_t most = tiles_most * ((a.N + (GATED ? 63 : 127)) / (GATED ? 64 : 128));
    const int64_t grid = most < dev.sms ? most : dev.sms;
    return launch_pdl(em::expert_mma_kernel<WT, GATED>, dim3((unsigned)grid), em::THREADS, L::SMEM, stream, a);
}

template <int WT>
static qmm_status expert_mma_either(const ExpertMma& a, bool gate, int64_t tiles_most, cudaStream_t stream) {
    return gate ? expert_mma_launch<WT, true>(a, tiles_most, stream) : expert_mma_launch<WT, false>(a, tiles_most, stream);
}

}  // namespace qmm
