// attend.cu -- attention of one new token per sequence over a paged key-value
// cache: out[h] = sum_p w_p v_p, w = softmax_p(scale * q_h . k_p), p over the
// sequence's positions (or the last `window` of them), h's KV head shared by the
// G = Hq / Hkv query heads of its group.
//
// Bound by the cache's bytes, each read once: 2 (hd + 4) per position and KV head
// (8-bit rows), against 4 G hd operations, which is more than the f32 units do at
// the memory's rate for G = 8 -- so both products run on the tensor cores, as
// m16n8k16 f16 products with f32 sums (mma.sync: eight query heads fill a
// sixteen-row tile; a tcgen05 tile has 64 rows at least, and its operands would
// have to be stored to shared memory again after their conversion).
//   codes   int8 is exact in f16; the row's scale multiplies the f32 sum (keys) or
//           the softmax weight (values)
//   f32     a query, and the weights times the value scales, are split into two
//           f16 (hi + lo, 22 bits) and take two rows of the tile: rows 0-7 are
//           the heads' hi, rows 8-15 their lo, and one thread holds both sums.
//           Each is first brought near f16's upper end by a power of two (of a head's
//           query; of the head's largest weight times scale in the tile), so that lo
//           stays in f16's range; what is below 2^-12 of that largest, with lo at f16's
//           least step, is off by 2^-39 of it at most.  The power is the tile's own: one
//           kept from earlier tiles let a single large row without weight cost all later
//           ones their low bits
//   layout  the order of the 16 values within a step is free as long as both
//           operands share it, so a lane takes its operand straight from 16-byte
//           loads of natural rows, and a tile's scores are in the registers where
//           the second product wants its weights: nothing is shuffled but the
//           row maximum
// Running maximum and sum of a softmax (in base 2) per warp: one pass.  The reference
// is a whole number near the maximum, so rescaling by it is exact and rare.
//
// Split.  The work is the list of (row, unit, tile): a unit is a KV head and up to
// eight of its query heads, a tile 32 (16) positions; each unit counts as unit_cost
// tiles more than it has, which is what starting and finishing one takes.  A fixed
// number of teams each take an equal run of the list, found by a scan of the lengths on
// the device: a captured launch serves any lengths, ragged batches are balanced to a
// tile, and a long sequence is spread over the whole GPU.  A unit inside one run is
// written at once; else its parts go to the workspace (at most two per run), and the
// second kernel joins them in order.  Nothing is added by atomics: results do not vary.
// A team is a CTA whose four warps take tiles in turn and meet in shared memory, or,
// where there are many units, a single warp, which meets nobody (kTeamUnits).
//
// Measured (32 query heads on 8 KV heads of 128, 8-bit): 64 rows of up to 8192
// positions, 380 MB, 70 us = 5.4 TB/s; two rows of 131072 and 32768 (64 query heads),
// 346 MB, 64 us, of which the same copies without any arithmetic take 54, the start
// (lengths, pages, first copies, one after the other) 3.6 and the join 2 to 4.  Nine to
// 16 query heads per KV head are two units that copy and convert the same rows: 125 us
// and 677 MB for the 64 rows with 128 query heads, 72 us and 380 MB with 64.  Rows that do
// not fill 64, 128 or 256 values, and pages of fewer than 16 positions, take the slower
// copies: 91 us for the 64 rows with heads of 80, 96 or 112, or with pages of 8.
#include <type_traits>

#include "kvpages.cuh"

namespace qmm {

static __device__ unsigned int g_attend_error = 0;

constexpr int kAttendWarps = 4;
constexpr int kAttendThreads = 32 * kAttendWarps;
constexpr int kAttendSms = 152;
constexpr int kAttendHeads = 8;  // query heads per unit
constexpr int kJoinThreads = 128;
constexpr int kJoinFew = 8;  // parts that one CTA joins for all heads
// Up to so many units, a team is a CTA (the first tokens of one request: 4.9 us, a single
// warp per unit 6.3; a row of 4096 positions 8.7 and 9.6); with more, a warp (1000 rows
// of 40 positions, 8 units each: 104 us by CTAs, 48 by warps; 64 ragged rows, 512 units:
// 72 and 70).
constexpr int64_t kTeamUnits = 152;
// what a unit costs a team besides its tiles, in tiles
__host__ __device__ constexpr uint32_t unit_cost(int team) { return team == 1 ? 2 : 12; }
constexpr float kSlack = 4.0f;  // what scores may be over the running reference, in powers of two

template <int TYPE, int HDT>
struct AttendShape {
    static constexpr int kRow = HDT * (TYPE == QMM_KV_F16 ? 2 : 1);  // bytes of a row
    static constexpr int kTile = kRow <= 128 ? 32 : 16;              // positions
    // A warp's ring has three slots of one tile's keys or values, with their scales and the
    // mask: two are on their way while one is read.
    static constexpr int kSlots = 3;
    static constexpr int kSlot = kTile * kRow + 4 * kTile + 16;
    static constexpr int kRing = kSlots * kSlot;  // of a warp
    static constexpr int kSmem = kAttendWarps * kRing;
    // CTAs per SM such that about 68 KB are on their way for rows of up to 256 bytes: more
    // queue up in the memory system, which then serves the SMs unevenly (two rows of 131072
    // and 64 ragged ones of 128-byte rows: 63.5 and 70.0 us; with a third CTA 75.7 and 82.1,
    // with a fourth slot 63.7 and 71.3).  512-byte rows have 132 KB on their way, but with a
    // single CTA four warps cannot keep up (a window of 1024: 52 us instead of 47; 60000
    // positions 92 instead of 85).
    static constexpr int kCtas = kRow <= 64 ? 4 : 2;
};

// Runs at most, of single warps: what the workspace has room for.  Rows of more than 64
// bytes, which 8-bit heads over 64 and all 16-bit ones have, get half as many.
inline int64_t attend_max_runs(int64_t hd) {
    static_assert(AttendShape<QMM_KV_Q8, 64>::kCtas == 4 && AttendShape<QMM_KV_F16, 64>::kCtas == 2 &&
                  AttendShape<QMM_KV_Q8, 128>::kCtas == 2 && AttendShape<QMM_KV_F16, 128>::kCtas == 2 &&
                  AttendShape<QMM_KV_Q8, 256>::kCtas == 2 && AttendShape<QMM_KV_F16, 256>::kCtas == 2, "CTAs per SM");
    return (hd <= 64 ? 4 : 2) * kAttendSms * kAttendWarps;
}

struct AttendArgs {
    const float* q;
    const int32_t* lens;
    const int32_t* seq;  // may be null: row r reads sequence r
    float* out;
    float* lse;  // may be null
    float* parts;
    int4* joins;
    int64_t R, ldq, ldo, window;
    int G, blocks;  // query heads per KV head, units per KV head
    uint32_t chunk, chunks;  // rows per chunk, at most kAttendThreads chunks
    uint32_t runs;           // of the launch: two parts and two notes each in the workspace
    float scale;
};

// What row r reads: positions first .. len - 1 of sequence seq.
struct RowRange {
    int64_t seq;
    int first, len;
};
__device__ __forceinline__ RowRange attend_row(const KvPages& c, const AttendArgs& a, int64_t r) {
    RowRange x;
    x.len = __ldg(a.lens + r);
    x.seq = a.seq ? (int64_t)__ldg(a.seq + r) : r;
    x.first = 0;
    if (x.len > 0) {
        const int64_t room = c.max_pages << c.page_shift;
        if (x.seq < 0 || x.seq >= c.num_seqs) {
            atomicOr(&g_attend_error, kErrPlace);
            x.len = 0;
        } else if (x.len > room) {
            atomicOr(&g_attend_error, kErrPlace);
            x.len = (int)room;
        }
        if (a.window > 0 && x.len > a.window) x.first = x.len - (int)a.window;
    }
    return x;
}
template <int TILE>
__device__ __forceinline__ uint32_t row_tiles(const RowRange& x) {
    return x.len > 0 ? (uint32_t)(x.len - 1) / TILE + 1u - (uint32_t)x.first / TILE : 0u;
}
// A unit's share of the list: its cost, then its tiles.
template <int TEAM>
__device__ __forceinline__ uint32_t unit_weight(uint32_t tiles) {
    return tiles ? tiles + unit_cost(TEAM) : 0u;
}

// n / d for 0 <= n < 2^31, d > 0, by the approximate reciprocal (relative error below 2^-21
// with the conversions') and two corrections: the whole-number division takes twice as
// long, and these stand one behind the other before the first byte is fetched.
__device__ __forceinline__ uint32_t quick_div(uint32_t n, uint32_t d) {
    const float by = __fdividef(1.0f, (float)d);
    uint32_t q = (uint32_t)((float)n * by);
    int rest = (int)(n - q * d);  // within 2^11 d of 0, modulo 2^32
    q += (int)floorf((float)rest * by);
    rest = (int)(n - q * d);
    return rest < 0 ? q - 1 : (rest >= (int)d ? q + 1 : q);
}

// The list cut into `count` runs whose lengths differ by one at most; no more runs than
// leave each a tile per warp.
template <int TEAM>
struct Runs {
    uint32_t count, q, rem;
    __device__ __forceinline__ Runs(uint32_t work, uint32_t most) {
        const uint32_t fill = work / TEAM;
        count = fill < 1 ? 1 : (fill < most ? fill : most);
        q = quick_div(work, count);
        rem = work - q * count;
    }
    __device__ __forceinline__ uint32_t begin(uint32_t c) const { return c * q + (c < rem ? c : rem); }
    __device__ __forceinline__ uint32_t of(uint32_t g) const {  // the run that holds position g
        const uint32_t cut = rem * (q + 1);
        return g < cut ? quick_div(g, q + 1) : rem + quick_div(g - cut, q);
    }
};

// Sum over the block of each thread's v; *before: over the threads before this one.
template <int THREADS>
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* before, uint32_t* sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t incl = v;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, incl, m);
        if (lane >= m) incl += o;
    }
    __syncthreads();  // sums may still be read from the scan before
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    uint32_t base = 0, total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; w++) {
        if (w < warp) base += sums[w];
        total += sums[w];
    }
    *before = base + incl - v;
    return total;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4z(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ float exp2_approx(float x) {  // within 2 units in the last place; 0 at -inf
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void mma_f16(float d[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the same from a zero sum
__device__ __forceinline__ void mma_f16_first(float d[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
// (lo, hi) to two f16, the first in the low half
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// the two f16 of hi, and of what they leave of (x, y)
__device__ __forceinline__ void split_h2(float x, float y, uint32_t* hi, uint32_t* lo) {
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    *hi = *reinterpret_cast<const uint32_t*>(&h);
    *lo = pack_h2(x - f.x, y - f.y);
}
// The sum of a hi and a lo row.  An infinity in an f16 row makes the lo row's sum a NaN (0
// or the other sign times it), where the hi row's is the definition's.
template <int TYPE>
__device__ __forceinline__ float add_rows(float hi, float lo) {
    return TYPE == QMM_KV_F16 && fabsf(hi) == INFINITY ? hi : hi + lo;
}
// biased bytes (code + 128) sel of w as two f16: 1024 + byte, less 1152
__device__ __forceinline__ uint32_t codes_h2(uint32_t w, uint32_t sel) {
    const uint32_t b = __byte_perm(w, 0x64646464u, sel);
    const uint32_t bias = 0x64806480u;
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&b), *reinterpret_cast<const __half2*>(&bias));
    return *reinterpret_cast<const uint32_t*>(&r);
}
// 2^e
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }
// |x|'s exponent field (e + 127 with 2^e <= |x| < 2^(e + 1)), at least kExpLow so that
// 2^(14 - e) and 2^(e - 14) are normal
constexpr int kExpLow = 20;
__device__ __forceinline__ int exponent_of(float x) {
    const int e = (int)((__float_as_uint(x) & 0x7FFFFFFFu) >> 23);
    return e < kExpLow ? kExpLow : e;
}
// Where an exchanged value quad q of head h lies in its head's row: what the eight
// lanes of two heads write at once (quads 4 apart) goes to different banks.
__device__ __forceinline__ int exchange_quad(int h, int q) { return q ^ ((q >> 3) & 1) ^ ((h & 1) << 1); }

template <int TYPE, int HDT, int TEAM>
__global__ void __launch_bounds__(kAttendThreads, AttendShape<TYPE, HDT>::kCtas)
    attend_kernel(KvPages c, AttendArgs a) {
    using S = AttendShape<TYPE, HDT>;
    constexpr int TILE = S::kTile, ROW = S::kRow;
    constexpr int kChunks = ROW / 16;                    // 16-byte chunks of a row
    constexpr int kSize = TYPE == QMM_KV_F16 ? 2 : 1;    // bytes of a value
    constexpr int kPer = 16 / kSize;                     // values of a chunk
    constexpr int kGroups = kChunks / 4, kSteps = HDT / 16;
    constexpr int kVB = 8 * kSize, kSets = ROW / (8 * kVB);  // a lane takes eight values of a row at once
    constexpr int kChains = TILE == 16 ? 2 : 1;  // sums of the first product that run side by side
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ uint32_t scan[kAttendWarps], ends[kAttendThreads];
    __shared__ RowRange rows[kAttendThreads];
    __shared__ float part_m[kAttendWarps][kAttendHeads], part_l[kAttendWarps][kAttendHeads];
    __shared__ float part_f[kAttendWarps][kAttendHeads], unit_l[kAttendHeads];
    pdl_wait();
    pdl_launch_dependents();  // the join is launched now and waits for this grid
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = lane >> 2, j = lane & 3;
    const uint32_t units = c.Hkv * a.blocks;
    const int Hq = a.G * c.Hkv;

    // The list's length up to each of (at most) 128 chunks of rows, read once per block:
    // a load of lens by every warp of the grid meets in one line of the L2 (1.5 us of a
    // single row's 10).
    const uint32_t R = (uint32_t)a.R, chunk = a.chunk, chunks = a.chunks;
    const bool held = chunk == 1;  // every row's range fits in shared memory
    uint32_t total, before, mine = 0;
    for (uint32_t i = threadIdx.x * chunk; i < R && i < (threadIdx.x + 1) * chunk; i++) {
        const RowRange x = attend_row(c, a, i);
        if (held) rows[i] = x;
        mine += unit_weight<TEAM>(row_tiles<TILE>(x));
    }
    if (R <= 32) {
        if (warp == 0) {
            before = mine;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, before, m);
                if (lane >= m) before += v;
            }
            ends[lane] = before;
        }
        __syncthreads();
        total = ends[31];
    } else {
        total = block_scan<kAttendThreads>(mine, &before, scan);
        ends[threadIdx.x] = before + mine;
        __syncthreads();
    }
    auto row_of = [&](uint32_t i) { return held ? rows[i] : attend_row(c, a, i); };

    // Rows without positions, shared out among all warps.  CTA teams write them last: the
    // pass stands between a call's start and its first byte (first tokens of a request
    // 5.17 us, 5.47 with the pass first); single warps first, while the others' copies
    // start (64 ragged rows, heads of 64: 44.7 us, 45.6 with the pass last).
    auto empty_rows = [&]() {
        for (uint32_t i = blockIdx.x * kAttendWarps + warp; i < R; i += gridDim.x * kAttendWarps)
            if (row_of(i).len == 0) {
                for (int d = lane; d < Hq * (c.hd >> 2); d += 32)
                    if (QMM_IN_BOUNDS(g_attend_error, i * a.ldo + 4 * d + 3, a.R * a.ldo))
                        reinterpret_cast<float4*>(a.out + i * a.ldo)[d] = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int h = lane; a.lse && h < Hq; h += 32)
                    if (QMM_IN_BOUNDS(g_attend_error, (int64_t)i * Hq + h, a.R * Hq)) a.lse[(int64_t)i * Hq + h] = -INFINITY;
            }
    };
    if (TEAM == 1) empty_rows();

    // The team's run, and the row r in which it begins.  joins: for the second kernel,
    // the unit that the run continues and the one that it leaves unfinished.
    const uint32_t run = TEAM == 1 ? blockIdx.x * kAttendWarps + warp : blockIdx.x;
    const int member = TEAM == 1 ? 0 : warp;
    if (member == 0 && lane < 2 && QMM_IN_BOUNDS(g_attend_error, 2 * run + lane, 2 * a.runs))
        a.joins[2 * run + lane] = make_int4(0, 0, 0, 0);
    __syncwarp();
    const Runs<TEAM> runs(total * units, gridDim.x * (kAttendWarps / TEAM));
    const bool idle = total == 0 || run >= runs.count;
    const uint32_t begin = idle ? 0 : runs.begin(run), end = idle ? 0 : runs.begin(run + 1);
    uint32_t r = 0, g = begin, row_start;  // row_start: the row's first position in the list
    {
        uint32_t at = 0;
        for (uint32_t k = 0; k < chunks; k += 32) {
            const uint32_t found = __ballot_sync(0xFFFFFFFFu, k + lane < chunks && begin < ends[k + lane] * units);
            if (found) {
                at = k + __ffs(found) - 1;
                break;
            }
        }
        r = at * chunk;
        row_start = at ? ends[at - 1] * units : 0;
    }

    constexpr uint32_t kFull = TILE == 32 ? 0xFFFFFFFFu : 0xFFFFu;
    uint8_t* ring = smem + warp * S::kRing;
    const uint32_t ring_u = smem_u32(ring);
    // where this lane's chunk of the it-th copy goes in a tile (swizzled so that both
    // products' 16-byte loads are free of bank conflicts), but for the part of the
    // swizzle that depends on `it`
    constexpr int kRowsPer = 32 / kChunks > 0 ? 32 / kChunks : 1;  // rows of one copy instruction
    const int c_row = lane / kChunks, c_ch = lane % kChunks;
    auto put_k = [&](int it) {
        const int row = it * kRowsPer + c_row;
        return row * ROW + (ROW >= 128 ? c_ch ^ ((row >> 2 & 1) << 2) : c_ch) * 16;
    };
    auto put_v = [&](int it) {
        const int row = it * kRowsPer + c_row;
        return row * ROW + (ROW >= 128 ? c_ch ^ ((row & 3) << 1) : c_ch ^ ((row >> 1 & 1) << 1)) * 16;
    };
    const bool wide = c.hd == HDT && c.page_shift >= 4;  // rows fill their tile's, sixteen of them share a page
    const int mask_o = (1 << c.page_shift) - 1;
    while (g < end) {
        const RowRange x = row_of(r);
        const uint32_t tiles = row_tiles<TILE>(x), weight = unit_weight<TEAM>(tiles);
        if (tiles == 0 || g >= row_start + weight * units) {
            row_start += weight * units;
            r++;
            continue;
        }
        const uint32_t u = quick_div(g - row_start, weight), off = g - row_start - u * weight;
        const uint32_t take = weight - off < end - g ? weight - off : end - g;
        constexpr uint32_t kCost = unit_cost(TEAM);
        const int ta = off > kCost ? (int)(off - kCost) : 0;
        const int tb = off + take > kCost ? (int)(off + take - kCost) : 0;
        g += take;
        if (ta == tb) continue;
        const int kvh = a.blocks == 1 ? (int)u : (int)u / a.blocks, hb = (int)u - kvh * a.blocks;
        const int head0 = kvh * a.G + hb * kAttendHeads;
        const int heads = a.G - hb * kAttendHeads < kAttendHeads ? a.G - hb * kAttendHeads : kAttendHeads;
        const int tile0 = x.first / TILE;
        const int32_t* pages = c.table + x.seq * c.max_pages;

        // This lane's position in the next tile to look up, less x.first; positions
        // of this piece are those below `span`.
        const int last_p = (tile0 + tb) * TILE < x.len ? (tile0 + tb) * TILE : x.len;
        const unsigned span = (unsigned)(last_p - x.first);
        int look = lane < TILE ? (tile0 + ta + member) * TILE + lane - x.first : -(1 << 30) - 4096;
        // the page there as the table has it; -1: no position
        auto page_at = [&](int at) -> int {
            if ((unsigned)at >= span) return -1;
            const int pg = (at + x.first) >> c.page_shift;
            return QMM_IN_BOUNDS(g_attend_error, x.seq * c.max_pages + pg, c.num_seqs * c.max_pages) ? __ldg(pages + pg) : -1;
        };
        // its row in the pools, from their start; -1: none
        const int64_t head_at = (int64_t)(kvh << c.page_shift) * c.row_bytes;
        auto row_at = [&](int at, int id) -> int64_t {
            if ((unsigned)id < (unsigned)c.num_pages)
                return id * c.stride + head_at + (int64_t)((at + x.first) & mask_o) * c.row_bytes;
            if ((unsigned)at < span) atomicOr(&g_attend_error, kErrPlace);
            return -1;
        };
        // from there to its scale: as far behind the page's scales as the row behind the page
        auto scale_by = [&](int at) -> uint32_t {
            const int64_t row = (kvh << c.page_shift) + ((at + x.first) & mask_o);
            return (uint32_t)(c.scales - row * (c.row_bytes - 4));
        };
        // one half of a tile, its keys or its values, into a slot of the ring; at: this
        // lane's position's row, by: from there to its scale, live: the positions that have one
        auto issue = [&](bool there, int64_t at, uint32_t by, uint32_t live, bool values, int slot) {
            if (there) {
                const uint8_t* pool = values ? c.v : c.k;
                const uint32_t dst = ring_u + slot * S::kSlot;
                if (!values && lane == 0)
                    *reinterpret_cast<uint32_t*>(ring + slot * S::kSlot + TILE * ROW + 4 * TILE) = live;
                if (wide && live == kFull) {
#pragma unroll
                    for (int b = 0; b < TILE / 16; b++) {
                        const int64_t from = __shfl_sync(0xFFFFFFFFu, at, 16 * b) + c_row * ROW + c_ch * 16;
                        constexpr int kN = kChunks / 2;  // copies of sixteen rows
#pragma unroll
                        for (int i = 0; i < kN; i++) {
                            if (!QMM_IN_BOUNDS(g_attend_error, from + i * 512 + 15, c.num_pages * c.stride)) continue;
                            const uint32_t to = dst + (values ? put_v(b * kN + i) : put_k(b * kN + i));
                            cp_async16(to, pool + from + i * 512, 16);
                        }
                    }
                } else {
#pragma unroll 1
                    for (int it = 0; it < TILE * kChunks / 32; it++) {
                        int64_t from = __shfl_sync(0xFFFFFFFFu, at, it * kRowsPer + c_row);
                        int bytes = (from >= 0 && c_ch * 16 < c.row_bytes) ? 16 : 0;
                        from = bytes ? from + c_ch * 16 : 0;
                        if (!QMM_IN_BOUNDS(g_attend_error, from + 15, c.num_pages * c.stride)) from = 0, bytes = 0;
                        cp_async16(dst + (values ? put_v(it) : put_k(it)), pool + from, bytes);
                    }
                }
                if (TYPE == QMM_KV_Q8 && lane < TILE) {  // position p's scale at (p % 4) (TILE / 4) + p / 4
                    int bytes = at >= 0 ? 4 : 0;
                    int64_t from = bytes ? at + by : 0;
                    if (!QMM_IN_BOUNDS(g_attend_error, from + 3, c.num_pages * c.stride)) from = 0, bytes = 0;
                    cp_async4z(dst + TILE * ROW + 4 * ((lane & 3) * (TILE / 4) + (lane >> 2)), pool + from, bytes);
                }
            }
            cp_async_commit();  // an empty group where there is no tile: the wait counts groups
        };

        const int id0 = page_at(look);
        int id1 = page_at(look + TEAM * TILE);  // the page of the tile after
        // A operand of the first product: step s of lane j holds values
        // kPer * (j + 4 * (s / (kPer / 4))) + 4 * (s % (kPer / 4)) .. + 3 of head n
        float4 qv[kSteps];
        {
            const float* qh = a.q + r * a.ldq + (int64_t)(head0 + n) * c.hd;
#pragma unroll
            for (int s = 0; s < kSteps; s++) {
                const int d = kPer * (j + 4 * (s / (kPer / 4))) + 4 * (s % (kPer / 4));
                qv[s] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (n < heads && d < c.hd &&
                    QMM_IN_BOUNDS(g_attend_error, r * a.ldq + (int64_t)(head0 + n) * c.hd + d + 3, a.R * a.ldq))
                    qv[s] = __ldg(reinterpret_cast<const float4*>(qh + d));
            }
        }
        // Fill two slots.  While half q of the tiles' halves is read, q + 1 and q + 2 are on
        // their way.
        int64_t at1 = row_at(look, id0);
        uint32_t live1 = __ballot_sync(0xFFFFFFFFu, at1 >= 0), by1 = scale_by(look);
        auto next_tile = [&]() {  // at1, by1 and live1 to the tile after, whose page is in id1
            look += TEAM * TILE;
            at1 = row_at(look, id1), by1 = scale_by(look);
            live1 = __ballot_sync(0xFFFFFFFFu, at1 >= 0);
            id1 = page_at(look + TEAM * TILE);
        };
        issue(ta + member < tb, at1, by1, live1, false, 0);
        issue(ta + member < tb, at1, by1, live1, true, 1);

        const bool whole = ta == 0 && tb == (int)tiles;
        if (!whole && member == 0 && lane == 0) {
            const uint32_t g0 = row_start + u * weight + kCost;  // the unit's first tile
            const uint32_t c0 = ta == 0 ? run : runs.of(g0), c1 = tb == (int)tiles ? run : runs.of(g0 + tiles - 1);
            const uint32_t to = 2 * run + (ta == 0 ? 1 : 0);
            if (QMM_IN_BOUNDS(g_attend_error, to, 2 * a.runs)) a.joins[to] = make_int4((int)r, (int)u, (int)c0, (int)(c1 - c0 + 1));
        }

        uint32_t qf[kSteps][4];
        float q_scale;
        {
            float amax = 0.0f;
#pragma unroll
            for (int s = 0; s < kSteps; s++)
                amax = fmaxf(amax, fmaxf(fmaxf(fabsf(qv[s].x), fabsf(qv[s].y)), fmaxf(fabsf(qv[s].z), fabsf(qv[s].w))));
            amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
            const int e = exponent_of(amax) - 127;
            const float by = pow2i(14 - e);
            q_scale = a.scale * 1.44269504088896341f * pow2i(e - 14);  // scores in base 2
#pragma unroll
            for (int s = 0; s < kSteps; s++) {
                split_h2(qv[s].x * by, qv[s].y * by, &qf[s][0], &qf[s][1]);
                split_h2(qv[s].z * by, qv[s].w * by, &qf[s][2], &qf[s][3]);
            }
        }

        // Of head n: m_run, a whole number that no score so far is over by more than kSlack,
        // the sum of weights 2^(score - m_run) of this lane's positions, and the weighted
        // values.  The slack makes raising m_run rare; as it is whole, rescaling is exact.
        float m_run = -INFINITY, l_run = 0.0f;
        float o[kSets][8][2];
#pragma unroll
        for (int s = 0; s < kSets; s++)
#pragma unroll
            for (int t = 0; t < 8; t++) o[s][t][0] = o[s][t][1] = 0.0f;

        int slot = 0;
        auto turn = [&](int by) { return slot + by >= S::kSlots ? slot + by - S::kSlots : slot + by; };
        for (int t = ta + member; t < tb; t += TEAM) {
            cp_async_wait<S::kSlots - 2>();
            __syncwarp();  // the keys are here for every lane, and the slot before is read out
            next_tile();
            issue(t + TEAM < tb, at1, by1, live1, false, turn(2));
            const uint32_t st = ring_u + slot * S::kSlot;
            const uint8_t* tail = ring + slot * S::kSlot + TILE * ROW;  // scales, then the mask
            const uint32_t live = *reinterpret_cast<const uint32_t*>(tail + 4 * TILE);

            // scores: column i of n-tile m is position 8 m + i / 2 + 4 (i % 2)
            float sc[TILE / 8][kChains][4];
#pragma unroll
            for (int cg = 0; cg < kGroups; cg++) {
                uint4 kw[TILE / 8];
#pragma unroll
                for (int m = 0; m < TILE / 8; m++) {
                    const int row = 8 * m + (n >> 1) + 4 * (n & 1);
                    const int ch = ROW >= 128 ? (4 * cg + j) ^ ((n & 1) << 2) : 4 * cg + j;
                    kw[m] = lds128(st + row * ROW + ch * 16);
                }
#pragma unroll
                for (int w = 0; w < kPer / 4; w++) {
                    const int step = cg * (kPer / 4) + w;
#pragma unroll
                    for (int m = 0; m < TILE / 8; m++) {
                        const uint32_t* f = reinterpret_cast<const uint32_t*>(&kw[m]);
                        uint32_t b0, b1;
                        if (TYPE == QMM_KV_Q8) {
                            const uint32_t y = f[w] ^ 0x80808080u;
                            b0 = codes_h2(y, 0x4140u), b1 = codes_h2(y, 0x4342u);
                        } else {
                            b0 = f[2 * w], b1 = f[2 * w + 1];
                        }
                        if (step < kChains) mma_f16_first(sc[m][step % kChains], qf[step], b0, b1);
                        else mma_f16(sc[m][step % kChains], qf[step], b0, b1);
                    }
                }
            }
            // this lane's positions of head n: 4 i + j
            constexpr int kMine = TILE / 4;
            float wt[kMine], top = -INFINITY;
#pragma unroll
            for (int i = 0; i < kMine; i += 4) {
                const float* y0 = sc[i >> 1][0];
                const float* y1 = sc[(i >> 1) + 1][0];
                wt[i] = add_rows<TYPE>(y0[0], y0[2]), wt[i + 1] = add_rows<TYPE>(y0[1], y0[3]);
                wt[i + 2] = add_rows<TYPE>(y1[0], y1[2]), wt[i + 3] = add_rows<TYPE>(y1[1], y1[3]);
                if (kChains == 2) {
                    const float* z0 = sc[i >> 1][kChains - 1];
                    const float* z1 = sc[(i >> 1) + 1][kChains - 1];
                    wt[i] += add_rows<TYPE>(z0[0], z0[2]), wt[i + 1] += add_rows<TYPE>(z0[1], z0[3]);
                    wt[i + 2] += add_rows<TYPE>(z1[0], z1[2]), wt[i + 3] += add_rows<TYPE>(z1[1], z1[3]);
                }
                if (TYPE == QMM_KV_Q8) {
                    const float4 ks = *reinterpret_cast<const float4*>(tail + 4 * (j * kMine + i));
                    wt[i] *= ks.x * q_scale, wt[i + 1] *= ks.y * q_scale;
                    wt[i + 2] *= ks.z * q_scale, wt[i + 3] *= ks.w * q_scale;
                } else {
                    wt[i] *= q_scale, wt[i + 1] *= q_scale, wt[i + 2] *= q_scale, wt[i + 3] *= q_scale;
                }
            }
            if (live != kFull) {
#pragma unroll
                for (int i = 0; i < kMine; i++)
                    if (!(live >> (4 * i + j) & 1u)) wt[i] = -INFINITY;
            }
#pragma unroll
            for (int i = 0; i < kMine; i++) top = fmaxf(top, wt[i]);
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            slot = turn(1);
            cp_async_wait<S::kSlots - 2>();
            __syncwarp();  // the values are here, the keys are read out
            issue(t + TEAM < tb, at1, by1, live1, true, turn(2));
            const uint32_t sv = ring_u + slot * S::kSlot;
            const float* vs = reinterpret_cast<const float*>(ring + slot * S::kSlot + TILE * ROW);
            if (__any_sync(0xFFFFFFFFu, top > m_run + kSlack)) {
                const float m_new = top > m_run + kSlack ? ceilf(top) : m_run;
                const float keep = exp2_approx(m_run - (m_new == -INFINITY ? 0.0f : m_new));
                m_run = m_new;
                l_run *= keep;
#pragma unroll
                for (int s = 0; s < kSets; s++)
#pragma unroll
                    for (int t2 = 0; t2 < 8; t2++) o[s][t2][0] *= keep, o[s][t2][1] *= keep;
            }
            const float m_at = m_run == -INFINITY ? 0.0f : m_run;  // nothing seen yet: every weight is 0
            float big = 0.0f;
#pragma unroll
            for (int i = 0; i < kMine; i += 4) {
                const float w0 = exp2_approx(wt[i] - m_at), w1 = exp2_approx(wt[i + 1] - m_at);
                const float w2 = exp2_approx(wt[i + 2] - m_at), w3 = exp2_approx(wt[i + 3] - m_at);
                l_run += (w0 + w1) + (w2 + w3);
                wt[i] = w0, wt[i + 1] = w1, wt[i + 2] = w2, wt[i + 3] = w3;
                if (TYPE == QMM_KV_Q8) {
                    const float4 v4 = *reinterpret_cast<const float4*>(vs + j * kMine + i);
                    wt[i] *= v4.x, wt[i + 1] *= v4.y, wt[i + 2] *= v4.z, wt[i + 3] *= v4.w;
                    big = fmaxf(big, fmaxf(fmaxf(fabsf(wt[i]), fabsf(wt[i + 1])), fmaxf(fabsf(wt[i + 2]), fabsf(wt[i + 3]))));
                }
            }
            int e;  // the head's largest is below 2^(e + 1) (f16 rows: its weight, known from the score)
            if (TYPE == QMM_KV_Q8) {
                big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, 1));
                big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, 2));
                e = exponent_of(big) - 127;
            } else {
                e = max(__float2int_rd(top - m_at), kExpLow - 127);
            }
            const float up = pow2i(14 - e), down = pow2i(e - 14);
            uint32_t pf[TILE / 16][4];
#pragma unroll
            for (int i = 0; i < kMine; i += 4) {
                split_h2(wt[i] * up, wt[i + 1] * up, &pf[i >> 2][0], &pf[i >> 2][1]);
                split_h2(wt[i + 2] * up, wt[i + 3] * up, &pf[i >> 2][2], &pf[i >> 2][3]);
            }
            // Values: column n of n-tile (set, t) is value 64 set + 8 n + t.  Fresh sums per
            // tile, added to the running ones by f32 FMAs: the tensor core's own additions cut
            // off instead of rounding, which over a long cache would add up.
#pragma unroll
            for (int s = 0; s < kSets; s++) {
                float acc[8][4];
#pragma unroll
                for (int b = 0; b < TILE / 16; b++) {
                    uint32_t vw[4][kVB / 4];
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const uint32_t vr = sv + (16 * b + j + 4 * i) * ROW;
                        if (kVB == 16) {
                            const uint4 y = lds128(vr + (((8 * s + n) ^ (j << 1)) << 4));
                            vw[i][0] = y.x, vw[i][1] = y.y, vw[i][kVB / 4 - 2] = y.z, vw[i][kVB / 4 - 1] = y.w;
                        } else {
                            const int ch = (4 * s + (n >> 1)) ^ (ROW >= 128 ? j << 1 : j & 2);
                            const uint2 y = lds64(vr + (ch << 4) + ((n & 1) << 3));
                            vw[i][0] = y.x, vw[i][1] = y.y;
                        }
                    }
                    auto mma = [&](int t2, uint32_t b0, uint32_t b1) {
                        if (b == 0) mma_f16_first(acc[t2 & 7], pf[b], b0, b1);
                        else mma_f16(acc[t2 & 7], pf[b], b0, b1);
                    };
#pragma unroll
                    for (int w = 0; w < kVB / 4; w++) {
                        if (TYPE == QMM_KV_Q8) {
                            const uint32_t w0 = vw[0][w] ^ 0x80808080u, w1 = vw[1][w] ^ 0x80808080u;
                            const uint32_t w2 = vw[2][w] ^ 0x80808080u, w3 = vw[3][w] ^ 0x80808080u;
                            const uint32_t al = __byte_perm(w0, w1, 0x5140u), ah = __byte_perm(w0, w1, 0x7362u);
                            const uint32_t bl = __byte_perm(w2, w3, 0x5140u), bh = __byte_perm(w2, w3, 0x7362u);
                            mma(4 * w, codes_h2(al, 0x4140u), codes_h2(bl, 0x4140u));
                            mma(4 * w + 1, codes_h2(al, 0x4342u), codes_h2(bl, 0x4342u));
                            mma(4 * w + 2, codes_h2(ah, 0x4140u), codes_h2(bh, 0x4140u));
                            mma(4 * w + 3, codes_h2(ah, 0x4342u), codes_h2(bh, 0x4342u));
                        } else {
                            mma(2 * w, __byte_perm(vw[0][w], vw[1][w], 0x5410u),
                                __byte_perm(vw[2][w], vw[3][w], 0x5410u));
                            mma(2 * w + 1, __byte_perm(vw[0][w], vw[1][w], 0x7632u),
                                __byte_perm(vw[2][w], vw[3][w], 0x7632u));
                        }
                    }
                }
#pragma unroll
                for (int t2 = 0; t2 < 8; t2++)
#pragma unroll
                    for (int i = 0; i < 2; i++)
                        o[s][t2][i] = __fmaf_rn(add_rows<TYPE>(acc[t2][i], acc[t2][i + 2]), down, o[s][t2][i]);
            }
            slot = turn(1);
        }

        cp_async_wait<0>();
        l_run += __shfl_xor_sync(0xFFFFFFFFu, l_run, 1);
        l_run += __shfl_xor_sync(0xFFFFFFFFu, l_run, 2);
        const int64_t part_at = (2 * (int64_t)run + (ta == 0 ? 1 : 0)) * (kAttendHeads * (c.hd + 2));
        [[maybe_unused]] const int64_t parts_end = 2 * (int64_t)a.runs * (kAttendHeads * (c.hd + 2));
        float* part = a.parts + part_at;
        float* out = a.out + r * a.ldo + (int64_t)head0 * c.hd;
        auto put_ml = [&](int h, float m, float l) {
            if (!whole) {
                if (!QMM_IN_BOUNDS(g_attend_error, part_at + kAttendHeads * (c.hd + 1) + h, parts_end)) return;
                part[kAttendHeads * c.hd + h] = m, part[kAttendHeads * (c.hd + 1) + h] = l;
            } else if (a.lse && QMM_IN_BOUNDS(g_attend_error, r * Hq + head0 + h, a.R * Hq)) {
                a.lse[(int64_t)r * Hq + head0 + h] = (m + log2f(l)) * 0.693147180559945309f;
            }
        };
        auto put = [&](int h, int d, float4 y) {
            if (!whole) {
                if (QMM_IN_BOUNDS(g_attend_error, part_at + h * c.hd + d + 3, parts_end))
                    *reinterpret_cast<float4*>(part + h * c.hd + d) = y;
            } else if (QMM_IN_BOUNDS(g_attend_error, r * a.ldo + (int64_t)(head0 + h) * c.hd + d + 3, a.R * a.ldo)) {
                *reinterpret_cast<float4*>(out + h * c.hd + d) = y;
            }
        };
        if (TEAM == 1) {
            const float by = !whole ? 1.0f : (l_run == 0.0f ? 0.0f : __fdiv_rn(1.0f, l_run));
#pragma unroll
            for (int s = 0; s < kSets; s++)
#pragma unroll
                for (int i = 0; i < 2; i++)
#pragma unroll
                    for (int t = 0; t < 8; t += 4) {
                        const int d = 64 * s + 8 * (2 * j + i) + t;
                        if (n < heads && d < c.hd)
                            put(n, d, make_float4(o[s][t][i] * by, o[s][t + 1][i] * by, o[s][t + 2][i] * by,
                                                  o[s][t + 3][i] * by));
                    }
            if (j == 0 && n < heads) put_ml(n, m_run, l_run);
            __syncwarp();  // the ring is free for the next unit
            continue;
        }
        // the warps meet: running references and sums, then the values through shared memory
        if (j == 0) part_m[warp][n] = m_run, part_l[warp][n] = l_run;
        __syncthreads();  // every ring is read out: its memory is the exchange now
        float* xo = reinterpret_cast<float*>(smem) + (warp * kAttendHeads + n) * HDT;
#pragma unroll
        for (int s = 0; s < kSets; s++)
#pragma unroll
            for (int i = 0; i < 2; i++)
#pragma unroll
                for (int t = 0; t < 8; t += 4)
                    *reinterpret_cast<float4*>(xo + 4 * exchange_quad(n, (64 * s + 8 * (2 * j + i) + t) / 4)) =
                        make_float4(o[s][t][i], o[s][t + 1][i], o[s][t + 2][i], o[s][t + 3][i]);
        if (threadIdx.x < heads) {
            const int h = threadIdx.x;
            float m = -INFINITY, l = 0.0f;
#pragma unroll
            for (int w = 0; w < kAttendWarps; w++) m = fmaxf(m, part_m[w][h]);
            const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
            for (int w = 0; w < kAttendWarps; w++) {
                part_f[w][h] = exp2_approx(part_m[w][h] - ref);
                l += part_l[w][h] * part_f[w][h];
            }
            unit_l[h] = l;
            put_ml(h, m, l);
        }
        __syncthreads();
        const int quads = c.hd >> 2;
        for (int i = threadIdx.x; i < heads * quads; i += kAttendThreads) {
            const int h = i / quads, q = i - h * quads;
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kAttendWarps; w++) {
                const float* xw = reinterpret_cast<float*>(smem) + (w * kAttendHeads + h) * HDT;
                const float4 z = *reinterpret_cast<const float4*>(xw + 4 * exchange_quad(h, q));
                const float f = part_f[w][h];
                y.x = __fmaf_rn(z.x, f, y.x), y.y = __fmaf_rn(z.y, f, y.y);
                y.z = __fmaf_rn(z.z, f, y.z), y.w = __fmaf_rn(z.w, f, y.w);
            }
            if (whole) {
                const float by = unit_l[h] == 0.0f ? 0.0f : __fdiv_rn(1.0f, unit_l[h]);
                y.x *= by, y.y *= by, y.z *= by, y.w *= by;
            }
            put(h, 4 * q, y);
        }
        __syncthreads();  // the exchange is read out
    }

    if (TEAM > 1) empty_rows();
}

// One CTA per run, for the unit that its team continued and the one that it began and
// left unfinished (a.joins: row, unit, first run, number of runs).  Up to kJoinFew parts
// are joined by the first run's CTA, a thread per four values; the values of a unit in
// more parts are shared out among its runs' CTAs, 32 values at a time, with 4 threads
// side by side over the parts and four such pieces in hand at once (one at a time: 66.6 us
// instead of 64 for the two long rows above, 71 instead of 70 for the ragged ones), or 16
// threads where there is a single piece, as for a unit in more parts than it has pieces.
// The order of the sums depends on the runs alone.
struct JoinUnit {
    const float* parts;
    int n, row, head0, heads;
};
__global__ void __launch_bounds__(kJoinThreads) attend_join_kernel(KvPages c, AttendArgs a) {
    constexpr int kLanes = kJoinThreads / 8;  // threads that share four neighbouring values' column
    constexpr int kBatch = 4;                 // parts that a thread fetches at once
    static_assert(kLanes == 16, "side, below");
    __shared__ __align__(16) float4 sum[kLanes][8];
    __shared__ float fold_m[kLanes], fold_l[kLanes];
    pdl_wait();
    pdl_launch_dependents();
    const int Hq = a.G * c.Hkv, size = kAttendHeads * (c.hd + 2), per_head = (c.hd + 31) >> 5;
    if (!QMM_IN_BOUNDS(g_attend_error, blockIdx.x, a.runs)) return;
    const int4 jobs[2] = {a.joins[2 * blockIdx.x], a.joins[2 * blockIdx.x + 1]};
    if (jobs[0].w == 0 && jobs[1].w == 0) return;
    auto unit_of = [&](const int4& job) {
        JoinUnit x;
        const int kvh = a.blocks == 1 ? job.y : job.y / a.blocks, hb = job.y - kvh * a.blocks;
        x.parts = a.parts + 2 * (int64_t)job.z * size;
        x.n = job.w, x.row = job.x, x.head0 = kvh * a.G + hb * kAttendHeads;
        x.heads = a.G - hb * kAttendHeads < kAttendHeads ? a.G - hb * kAttendHeads : kAttendHeads;
        return x;
    };
    // the unit begins in its first run, the others continue it
    auto part = [&](const JoinUnit& x, int i) -> const float* {
        const float* p = x.parts + (2 * i + (i == 0 ? 1 : 0)) * (int64_t)size;
        return QMM_IN_BOUNDS(g_attend_error, p - a.parts + size - 1, 2 * (int64_t)a.runs * size) ? p : a.parts;
    };
    auto put = [&](const JoinUnit& x, int h, int d, float4 y, float m, float l) {
        const float by = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
        const int64_t to = x.row * a.ldo + (int64_t)(x.head0 + h) * c.hd + d, lse_to = (int64_t)x.row * Hq + x.head0 + h;
        if (QMM_IN_BOUNDS(g_attend_error, to + 3, a.R * a.ldo))
            *reinterpret_cast<float4*>(a.out + to) = make_float4(y.x * by, y.y * by, y.z * by, y.w * by);
        if (a.lse && d == 0 && QMM_IN_BOUNDS(g_attend_error, lse_to, a.R * Hq))
            a.lse[lse_to] = (m + log2f(l)) * 0.693147180559945309f;
    };
    auto add = [](float4& y, float& l, const float4& z, float pl, float f) {
        l = __fmaf_rn(pl, f, l);
        y.x = __fmaf_rn(z.x, f, y.x), y.y = __fmaf_rn(z.y, f, y.y);
        y.z = __fmaf_rn(z.z, f, y.z), y.w = __fmaf_rn(z.w, f, y.w);
    };
    if (jobs[1].w > 0 && jobs[1].w <= kJoinFew) {
        const JoinUnit x = unit_of(jobs[1]);
        const int quads = c.hd >> 2;
        for (int e = threadIdx.x; e < x.heads * quads; e += kJoinThreads) {
            const int h = e / quads, d = 4 * (e - h * quads);
            float4 z[kJoinFew];
            float pm[kJoinFew], pl[kJoinFew], m = -INFINITY, l = 0.0f;
#pragma unroll
            for (int i = 0; i < kJoinFew; i++) {
                const float* p = part(x, i < x.n ? i : 0);
                z[i] = *reinterpret_cast<const float4*>(p + h * c.hd + d);
                pm[i] = p[kAttendHeads * c.hd + h], pl[i] = p[kAttendHeads * (c.hd + 1) + h];
            }
#pragma unroll
            for (int i = 0; i < kJoinFew; i++)
                if (i < x.n) m = fmaxf(m, pm[i]);
            const float ref = m == -INFINITY ? 0.0f : m;
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < kJoinFew; i++)
                if (i < x.n) add(y, l, z[i], pl[i], exp2_approx(pm[i] - ref));
            put(x, h, d, y, m, l);
        }
    }
    // this CTA's pieces of both units
    int pieces[2];
#pragma unroll
    for (int k = 0; k < 2; k++) {
        const int4 job = jobs[k];
        pieces[k] = 0;
        if (job.w > kJoinFew) {
            const int all = unit_of(job).heads * per_head, first = blockIdx.x - job.z;
            pieces[k] = first < all ? (int)quick_div(all - first - 1, job.w) + 1 : 0;
        }
    }
    const int lg = pieces[0] + pieces[1] == 1 ? 4 : 2, side = 1 << lg, q = threadIdx.x & 7, at = threadIdx.x >> 3, s = at & (side - 1);
    const int slots = kLanes >> lg;
    for (int e0 = 0; e0 < pieces[0] + pieces[1]; e0 += slots) {
        const int e = e0 + (at >> lg);
        const bool there = e < pieces[0] + pieces[1];
        const int4 job = e < pieces[0] ? jobs[0] : jobs[1];
        const JoinUnit x = unit_of(job);
        const int piece = there ? (int)blockIdx.x - job.z + (e < pieces[0] ? e : e - pieces[0]) * job.w : 0;
        const int h = (int)quick_div(piece, per_head), d = 32 * (piece - h * per_head) + 4 * q;
        // each thread's parts about their own maximum, then the threads' about theirs
        float m = -INFINITY, l = 0.0f;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i0 = s; there && i0 < x.n; i0 += kBatch * side) {
            float4 z[kBatch];
            float pm[kBatch], pl[kBatch], top = m;
#pragma unroll
            for (int k = 0; k < kBatch; k++) {
                const int i = i0 + k * side;
                const float* p = part(x, i < x.n ? i : s);
                z[k] = *reinterpret_cast<const float4*>(p + h * c.hd + (d < c.hd ? d : 0));
                pm[k] = p[kAttendHeads * c.hd + h], pl[k] = p[kAttendHeads * (c.hd + 1) + h];
            }
#pragma unroll
            for (int k = 0; k < kBatch; k++)
                if (i0 + k * side < x.n) top = fmaxf(top, pm[k]);
            const float ref = top == -INFINITY ? 0.0f : top, keep = exp2_approx(m - ref);
            m = top;
            l *= keep, y.x *= keep, y.y *= keep, y.z *= keep, y.w *= keep;
#pragma unroll
            for (int k = 0; k < kBatch; k++)
                if (i0 + k * side < x.n) add(y, l, z[k], pl[k], exp2_approx(pm[k] - ref));
        }
        sum[at][q] = y;
        if (q == 0) fold_m[at] = m, fold_l[at] = l;
        __syncthreads();
        if (s == 0 && there) {
            float top = -INFINITY, all = 0.0f;
            for (int k = at; k < at + side; k++) top = fmaxf(top, fold_m[k]);
            const float ref = top == -INFINITY ? 0.0f : top;
            y = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = at; k < at + side; k++) add(y, all, sum[k][q], fold_l[k], exp2_approx(fold_m[k] - ref));
            if (d < c.hd) put(x, h, d, y, top, all);
        }
        __syncthreads();
    }
}

}  // namespace qmm

using namespace qmm;

extern "C" {

unsigned qmm_internal_attend_error(int clear) {
    unsigned v = 0;
    cudaMemcpyFromSymbol(&v, g_attend_error, sizeof(v));
    if (clear) {
        const unsigned z = 0;
        cudaMemcpyToSymbol(g_attend_error, &z, sizeof(z));
    }
    return v;
}

size_t qmm_kv_attend_scratch_bytes(int64_t Hq, int64_t Hkv, int64_t hd) {
    if (!head_dim_ok(hd) || Hkv < 1 || Hkv > 1024 || Hq < 1 || Hq % Hkv || Hq / Hkv > 64) return 0;
    return (size_t)attend_max_runs(hd) * 2 * (kAttendHeads * (size_t)(hd + 2) * sizeof(float) + sizeof(int4));
}

qmm_status qmm_kv_attend(const qmm_kv_pages* cache, const float* q, int64_t ldq, const int32_t* lens,
                         const int32_t* seq, float* out, int64_t ldo, float* lse, void* scratch, size_t scratch_bytes,
                         int64_t R, int64_t Hq, float scale, int64_t window, qmm_stream_t stream) {
    if (!q || !lens || !out || !scratch) return QMM_E_NULL;
    KvPages c;
    qmm_status st = kv_pages_check(cache, &c);
    if (st != QMM_OK) return st;
    const size_t need = qmm_kv_attend_scratch_bytes(Hq, c.Hkv, c.hd);
    if (need == 0 || R < 1 || R > kMaxDim || R * Hq > kMaxDim || (!seq && R > c.num_seqs) || window < 0 ||
        !row_stride_ok(ldq, Hq * c.hd) || !row_stride_ok(ldo, Hq * c.hd))
        return QMM_E_SHAPE;
    // the list of tiles is counted in 32 bits
    const int64_t room = c.max_pages << c.page_shift, seen = window > 0 && window < room ? window + 16 : room;
    const int64_t blocks = (Hq / c.Hkv + kAttendHeads - 1) / kAttendHeads;
    if (room > ((int64_t)1 << 30) || R * c.Hkv * blocks > kMaxDim / (seen / 16 + 2 + unit_cost(kAttendWarps)))
        return QMM_E_SHAPE;
    if (!aligned16(q) || !aligned16(out) || !aligned4(lens) || !aligned4(seq) || !aligned4(lse) || !aligned16(scratch))
        return QMM_E_ALIGN;
    if (scratch_bytes < need) return QMM_E_SCRATCH;
    AttendArgs a;
    a.q = q, a.lens = lens, a.seq = seq, a.out = out, a.lse = lse;
    a.joins = (int4*)scratch;
    a.parts = (float*)(a.joins + 2 * attend_max_runs(c.hd));
    a.R = R, a.ldq = ldq, a.ldo = ldo, a.window = window;
    a.G = (int)(Hq / c.Hkv);
    a.blocks = (int)blocks;
    a.chunk = (uint32_t)((R + kAttendThreads - 1) / kAttendThreads);
    a.chunks = (uint32_t)((R + a.chunk - 1) / a.chunk);
    a.scale = scale;
    DeviceInfo dev;
    st = current_device(&dev);
    if (st != QMM_OK) return st;
    const cudaStream_t cs = (cudaStream_t)stream;
    const bool ctas = R * c.Hkv * blocks <= kTeamUnits;
    auto go = [&](auto type, auto hdt, auto team) -> qmm_status {
        constexpr int TYPE = decltype(type)::value, HDT = decltype(hdt)::value, TEAM = decltype(team)::value;
        using S = AttendShape<TYPE, HDT>;
        static PerDeviceOnce once;
        const qmm_status set = once.run(dev.device, [&] {
            return cudaFuncSetAttribute(attend_kernel<TYPE, HDT, TEAM>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        S::kSmem) == cudaSuccess ? QMM_OK : QMM_E_CUDA;
        });
        if (set != QMM_OK) return set;
        // no more CTAs than the runs of rows that fill the table's room (or the window): the list
        // of any lengths is cut the same, and fewer are started
        constexpr int kRuns = kAttendWarps / TEAM;  // of a CTA
        const int64_t tiles = window > 0 && window < room ? (window - 1) / S::kTile + 2 : (room - 1) / S::kTile + 1;
        const int64_t most = (R * c.Hkv * blocks * (tiles + unit_cost(TEAM)) / TEAM + kRuns - 1) / kRuns;
        const unsigned grid = (unsigned)(most < S::kCtas * kAttendSms ? most : S::kCtas * kAttendSms);
        a.runs = grid * kRuns;
        return launch_pdl(attend_kernel<TYPE, HDT, TEAM>, dim3(grid), kAttendThreads, S::kSmem, cs, c, a);
    };
    using std::integral_constant;
    auto by_team = [&](auto type, auto hdt) -> qmm_status {
        return ctas ? go(type, hdt, integral_constant<int, kAttendWarps>()) : go(type, hdt, integral_constant<int, 1>());
    };
    auto by_width = [&](auto type) -> qmm_status {
        if (c.hd <= 64) return by_team(type, integral_constant<int, 64>());
        if (c.hd <= 128) return by_team(type, integral_constant<int, 128>());
        return by_team(type, integral_constant<int, 256>());
    };
    st = cache->type == QMM_KV_Q8 ? by_width(integral_constant<int, QMM_KV_Q8>())
                                  : by_width(integral_constant<int, QMM_KV_F16>());
    if (st != QMM_OK) return st;
    return launch_pdl(attend_join_kernel, dim3(a.runs), kJoinThreads, 0, cs, c, a);
}

}  // extern "C"
