// kvpages.cu -- keys and values into the pages of a cache, and back; the rotation of
// heads (qmm_rope) is the same kernel with query rows only.
//
//   rows      a CTA per few tokens: their places and rotation tables into shared
//             memory, then a group of lanes per head row, eight values a lane, which
//             keeps its row of each token in turn (the next one's loads ahead) -- key
//             rows are rotated and quantized, value rows quantized, query rows
//             rotated and written as f32.  One launch for all three, each value read
//             once
//   kv_load   four values a thread, its column of each token in turn: 4 (8) bytes of
//             codes in, 16 bytes out
// The 8-bit rule is qmm_kv_quantize's, step by step.  The load is bound by memory: 32768
// positions of 8 x 128 in 61 us, 5.5 TB/s (16-bit rows 72 us, 5.6 TB/s).  So is a rotation
// alone (4096 x 32 x 128 in 25.8 us, 5.2 TB/s; a bare product of the same size takes 21.4).
// The store fills neither the issue slots (67%) nor the memory's rate (28%): a thread has
// one token ahead in flight, and of about 320 instructions for 8 values of a warp's lanes
// half are the rotation's pairs and a quarter the quantizing (8192 tokens of 8 + 8 rows
// of 128 in 27 us; 17 without the rotation, 12.6 at the memory's rate; 16-bit rows 22 and
// 19.5, 15 at the memory's rate).
#include <type_traits>

#include "kvpages.cuh"
#include "rope_device.cuh"

namespace qmm {

static __device__ unsigned int g_pages_error = 0;

constexpr int kSms = 152;
constexpr int kRowThreads = 256;
constexpr int kRowCtas = 4;     // per SM
constexpr int kRowTable = 512;  // (cos, sin) entries of one block of tokens
constexpr int kRowTokens = 32;  // tokens of a block at most

// What a token's rows need to know of its place: the page's offset in the pools (-1:
// it has none) and the position in it (-1: a padding token).
struct __align__(16) Place {
    int64_t page;
    int o;
};
__device__ __forceinline__ Place place_of(const KvPages& c, const int32_t* pos, const int32_t* seq, int64_t t) {
    Place x;
    const int p = pos[t];
    x.o = p < 0 ? -1 : p & ((1 << c.page_shift) - 1);
    x.page = -1;
    if (p >= 0) {
        const int id = kv_page_of(c, seq ? (int64_t)seq[t] : t, p);
        if (id < 0) atomicOr(&g_pages_error, kErrPlace);
        else x.page = id * c.stride;
    }
    return x;
}

// The tokens of a CTA, `par` side by side: neighbouring CTAs take neighbouring tokens,
// so that what is read and written at one time lies together in memory.
struct CtaTokens {
    int par, count;
    __device__ __forceinline__ CtaTokens(int64_t T, int p) : par(p) {
        const int64_t whole = T / p, rest = T - whole * p;  // groups of par, and the last few
        const int64_t b = blockIdx.x, n = whole > b ? (whole - b - 1) / gridDim.x + 1 : 0;
        count = (int)n * p + (rest && whole % gridDim.x == b ? (int)rest : 0);
    }
    __device__ __forceinline__ int64_t at(int i) const {
        if (par == 1) return blockIdx.x + (int64_t)i * gridDim.x;
        const int g = i / par;
        return (blockIdx.x + (int64_t)g * gridDim.x) * par + (i - g * par);
    }
};

// Grid (CTAs that share the tokens, parts of a token's rows).  width: lanes per row, hd / 8
// (for 8-bit rows rounded up to a power of two: the largest value goes round by
// shuffles); rows_per: rows of a CTA; par: tokens side by side (more than one where a
// token has fewer rows than a CTA takes); block: tokens whose places and tables are in
// shared memory, the next block's prepared ahead.
template <int TYPE, int PAIRS>
__global__ void __launch_bounds__(kRowThreads, kRowCtas) rows_kernel(KvPages c, RowArgs a, int hd, int width,
                                                                     int rows_per, int par, int block) {
    __shared__ float4 tables[2][kRowTable];
    __shared__ Place places[2][TYPE == kNoPages ? 1 : kRowTokens];
    pdl_wait();
    pdl_launch_dependents();  // every kernel here waits before it touches memory: the next may be placed now
    const CtaTokens own(a.T, par);
    const int nt = own.count;
    const int Hkv = TYPE == kNoPages ? 0 : c.Hkv, rows = 2 * Hkv + a.Hq;
    const int group = threadIdx.x / width, o = threadIdx.x - group * width;
    const int tl = group / rows_per, row = blockIdx.y * rows_per + group - tl * rows_per;
    const bool live = tl < par && row < rows && 8 * o < hd;
    const bool query = row >= 2 * Hkv, value = !query && row >= Hkv;
    const int h = query ? row - 2 * Hkv : (value ? row - Hkv : row);
    const int half = a.n_rot >> 1, run = turn_run(half);
    Share share = row_share<PAIRS>(a.n_rot, o);
    if (PAIRS != kPairsScattered && value) share = row_share<kPairsNone>(0, o);  // eight neighbours, as they are
    if (value) share.turned = 0;
    const int side = TYPE == kNoPages ? 2 : (!live ? 0 : (query ? 2 : (value ? 1 : 0)));
    const int64_t ld = side == 2 ? a.ldq : (side == 1 ? a.ldv : a.ldk);
    // Fetches are free of branches (a lane out of range reads the row's first share, and
    // the last token is read again): a load inside a branch is waited for at its end.
    const int64_t step = (int64_t)gridDim.x * par;  // tokens from one of this thread's to its next
    const int64_t first = own.at(tl < nt ? tl : nt - 1);
    const float* x = (side == 2 ? a.q : (side == 1 ? a.v : a.k)) + first * ld + (live ? (int64_t)h * hd : 0);
    [[maybe_unused]] const float* x_end = (side == 2 ? a.q : (side == 1 ? a.v : a.k)) + a.T * ld;
    float* y = query ? a.q_out + first * a.ldqo + (int64_t)h * hd : nullptr;
    const int o_read = live ? o : 0;
    const Share from = live ? share : row_share<kPairsNone>(0, 0);
    auto fetch = [&](float v[8]) {
        if (!QMM_IN_BOUNDS(g_pages_error, hd - 1, x_end - x)) return;
        row_load8<PAIRS>(from, a.n_rot, o_read, x, v);
    };
    // where this thread's row lies in a page
    uint8_t* pool = (value ? c.v : c.k) + (int64_t)(h << c.page_shift) * c.row_bytes;
    uint8_t* pool_scale = (value ? c.v : c.k) + c.scales + 4 * (int64_t)(h << c.page_shift);
    auto prepare = [&](int b0, int buf) {  // places and tables of the block that begins at the CTA's token b0
        const int n = nt - b0 < block ? nt - b0 : block;
        if (TYPE != kNoPages && (int)threadIdx.x < n)
            places[buf][threadIdx.x] = place_of(c, a.pos, a.seq, own.at(b0 + threadIdx.x));
        for (int i = threadIdx.x; i < n * half; i += blockDim.x) {
            const int t = i / half;
            float4 e = turn_cos_sin((uint64_t)(int64_t)a.pos[own.at(b0 + t)] * a.freqs[i - t * half], a.mscale);
            if (a.inverse) e.z = -e.z, e.w = -e.w;
            const int to = t * 4 * run + turn_at(half, i - t * half);
            if (QMM_IN_BOUNDS(g_pages_error, to, kRowTable)) tables[buf][to] = e;
        }
    };
    float v[8] = {}, ahead[8] = {};
    fetch(v);
    prepare(0, 0);
    __syncthreads();

    const bool codes = TYPE == QMM_KV_Q8 && __any_sync(0xFFFFFFFFu, live && !query);  // the warp quantizes
    for (int b0 = 0, buf = 0; b0 < nt; b0 += block, buf ^= 1) {
        if (b0 > 0) __syncthreads();  // the block before is done, and this one prepared
        if (b0 + block < nt) prepare(b0 + block, buf ^ 1);
        const int bn = nt - b0 < block ? nt - b0 : block;
        for (int i0 = 0; i0 < bn; i0 += par) {  // the same count for every lane: the shuffles need whole warps
            const int tb = i0 + tl, t = b0 + tb;  // of the block, of the CTA
            if (t + par < nt) x += step * ld;
            fetch(ahead);
            const bool here = live && tb < bn;
            Place p;
            p.page = -1, p.o = 0;
            if (TYPE != kNoPages) p = places[buf][here ? tb : 0];
            if (here) row_turn8<PAIRS>(share, v, tables[buf] + tb * 4 * run + o, run);
            if (query) {
                if (here && p.o >= 0 && QMM_IN_BOUNDS(g_pages_error, (y - a.q_out) + hd - 1, a.T * a.ldqo))
                    row_store8<PAIRS>(share, a.n_rot, o, y, v);
                y += step * a.ldqo;
            }
            if (TYPE != kNoPages) {
                float amax = 0.0f;
                if (codes) {
#pragma unroll
                    for (int i = 0; i < 8; i++) amax = fmaxf(amax, fabsf(v[i]));
                    amax = here ? amax : 0.0f;
                    for (int m = width >> 1; m > 0; m >>= 1)
                        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, m));
                }
                if (here && !query && p.page >= 0) {
                    const int64_t at = p.page + (int64_t)p.o * c.row_bytes;
                    if (!QMM_IN_BOUNDS(g_pages_error, at + (int64_t)(h << c.page_shift) * c.row_bytes + c.row_bytes - 1,
                                       c.num_pages * c.stride)) {
                    } else if (TYPE == QMM_KV_Q8) {
                        // |x * (127 / amax)| rounds beyond 127 only where the quotient is infinite
                        const float inv = amax != 0.0f ? __fdiv_rn(127.0f, amax) : 0.0f;
                        uint32_t b[8];
#pragma unroll
                        for (int i = 0; i < 8; i++) b[i] = (uint32_t)__float2int_rn(__fmul_rn(v[i], inv));
                        if (inv == INFINITY) {
#pragma unroll
                            for (int i = 0; i < 8; i++) b[i] = (uint32_t)clampi((int)b[i], -128, 127);
                        }
                        if (PAIRS == kPairsScattered) {
#pragma unroll
                            for (int i = 0; i < 4; i++) {
                                const int2 e = scattered_at(a.n_rot, 4 * o + i);
                                pool[at + e.x] = (uint8_t)b[i];
                                pool[at + e.y] = (uint8_t)b[i + 4];
                            }
                        } else {
                            const uint32_t w0 = __byte_perm(__byte_perm(b[0], b[1], 0x0040u),
                                                            __byte_perm(b[2], b[3], 0x0040u), 0x5410u);
                            const uint32_t w1 = __byte_perm(__byte_perm(b[4], b[5], 0x0040u),
                                                            __byte_perm(b[6], b[7], 0x0040u), 0x5410u);
                            *reinterpret_cast<uint32_t*>(pool + at + share.first) = w0;
                            *reinterpret_cast<uint32_t*>(pool + at + share.second) = w1;
                        }
                        if (o == 0 && QMM_IN_BOUNDS(g_pages_error, p.page + c.scales + 4 * ((int64_t)(h << c.page_shift) + p.o) + 3,
                                                    c.num_pages * c.stride))
                            *reinterpret_cast<float*>(pool_scale + p.page + 4 * p.o) = __fdiv_rn(amax, 127.0f);
                    } else {
                        __half* to = reinterpret_cast<__half*>(pool + at);
                        if (PAIRS == kPairsScattered) {
#pragma unroll
                            for (int i = 0; i < 4; i++) {
                                const int2 e = scattered_at(a.n_rot, 4 * o + i);
                                to[e.x] = __float2half_rn(v[i]);
                                to[e.y] = __float2half_rn(v[i + 4]);
                            }
                        } else {
                            const uint32_t w0 = f2h_bits(v[0]) | f2h_bits(v[1]) << 16;
                            const uint32_t w1 = f2h_bits(v[2]) | f2h_bits(v[3]) << 16;
                            const uint32_t w2 = f2h_bits(v[4]) | f2h_bits(v[5]) << 16;
                            const uint32_t w3 = f2h_bits(v[6]) | f2h_bits(v[7]) << 16;
                            *reinterpret_cast<uint2*>(to + share.first) = make_uint2(w0, w1);
                            *reinterpret_cast<uint2*>(to + share.second) = make_uint2(w2, w3);
                        }
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 8; i++) v[i] = ahead[i];
        }
    }
}

// CTAs that share T tokens, `par` at a time: one wave of `ctas` per SM at most.
static unsigned token_ctas(int64_t T, int64_t parts, int ctas, int par) {
    const int64_t most = (int64_t)ctas * kSms / parts, groups = (T + par - 1) / par;
    return (unsigned)(most < 1 ? 1 : (groups < most ? groups : most));
}

qmm_status rows_launch(int type, const KvPages& c, const RowArgs& a, int hd, cudaStream_t stream) {
    int width = hd / 8;
    if (type == QMM_KV_Q8)
        for (width = 2; 8 * width < hd;) width *= 2;
    const int groups = kRowThreads / width, rows = (type == kNoPages ? 0 : 2 * c.Hkv) + a.Hq;
    int block = kRowTokens;  // the tables and places in shared memory
    if (a.n_rot && block > kRowTable / (4 * turn_run(a.n_rot / 2))) block = kRowTable / (4 * turn_run(a.n_rot / 2));
    const int parts = (rows + groups - 1) / groups, rows_per = (rows + parts - 1) / parts;
    int par = parts > 1 ? 1 : groups / rows;
    if (par > block) par = block;
    if (par > a.T) par = (int)a.T;
    block -= block % par;
    const int threads = (par * rows_per * width + 31) / 32 * 32;
    const dim3 grid(token_ctas(a.T, parts, kRowCtas * kRowThreads / threads, par), (unsigned)parts);
    auto go = [&](auto kern) {
        return launch_pdl(kern, grid, threads, 0, stream, c, a, hd, width, rows_per, par, block);
    };
    auto by_pairs = [&](auto t) -> qmm_status {
        constexpr int TYPE = decltype(t)::value;
        switch (a.pairs) {
        case kPairsHalf: return go(rows_kernel<TYPE, kPairsHalf>);
        case kPairsNext: return go(rows_kernel<TYPE, kPairsNext>);
        case kPairsNextAny: return go(rows_kernel<TYPE, kPairsNextAny>);
        case kPairsScattered: return go(rows_kernel<TYPE, kPairsScattered>);
        default: return TYPE == kNoPages ? QMM_E_TYPE : go(rows_kernel<TYPE == kNoPages ? QMM_KV_Q8 : TYPE, kPairsNone>);
        }
    };
    using std::integral_constant;
    if (type == QMM_KV_Q8) return by_pairs(integral_constant<int, QMM_KV_Q8>());
    if (type == QMM_KV_F16) return by_pairs(integral_constant<int, QMM_KV_F16>());
    return by_pairs(integral_constant<int, kNoPages>());
}

constexpr int kLoadThreads = 256;
constexpr int kLoadCtas = 5;     // per SM
constexpr int kLoadUnroll = 4;   // tokens whose codes are fetched before the first is converted
constexpr int kLoadTokens = 64;  // of a block at most

// int8 byte k of w (biased by 128) as a float: placed in the low mantissa bits of
// 2^23, less 2^23 + 128
__device__ __forceinline__ float code_f(uint32_t biased, uint32_t sel) {
    return __fsub_rn(__uint_as_float(__byte_perm(biased, 0x4B000000u, sel)), 8388736.0f);
}

// Loads that stay where they are written.
__device__ __forceinline__ uint32_t ld_here(const uint32_t* p) {
    uint32_t v;
    asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ uint2 ld_here(const uint2* p) {
    uint2 v;
    asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
    return v;
}

// Grid (CTAs that share the tokens, groups of kLoadThreads columns); a column is four values
// of one head of the keys or the values; par: tokens side by side; block: tokens whose
// places are in shared memory, the next block's looked up ahead.
template <int TYPE>
__global__ void __launch_bounds__(kLoadThreads, kLoadCtas)
    kv_load_kernel(KvPages c, const int32_t* __restrict__ pos, const int32_t* __restrict__ seq, float* k_out, int64_t ldk,
                   float* v_out, int64_t ldv, int64_t T, int par, int block) {
    __shared__ Place places[2][kLoadTokens];
    pdl_wait();
    pdl_launch_dependents();  // every kernel here waits before it touches memory: the next may be placed now
    const CtaTokens own(T, par);
    const int nt = own.count;
    const int quads = c.hd >> 2, side = c.Hkv * quads, columns = (k_out ? side : 0) + (v_out ? side : 0);
    const int tl = par > 1 ? threadIdx.x / columns : 0;
    const int col = blockIdx.y * kLoadThreads + threadIdx.x - tl * columns;
    const bool live = tl < par && col < columns;
    const bool value = !k_out || col >= side;
    const int e = value && k_out ? col - side : col, h = e / quads, quad = e - h * quads;
    const int64_t ld = value ? ldv : ldk;
    float* out = (value ? v_out : k_out) + (int64_t)h * c.hd + 4 * quad;
    constexpr int kQuad = TYPE == QMM_KV_Q8 ? 4 : 8;  // bytes
    const int head = h << c.page_shift;
    const uint8_t* pool = (value ? c.v : c.k) + (int64_t)head * c.row_bytes + kQuad * quad;
    const uint8_t* scales = (value ? c.v : c.k) + c.scales + 4 * (int64_t)head;
    if ((int)threadIdx.x < block && (int)threadIdx.x < nt)
        places[0][threadIdx.x] = place_of(c, pos, seq, own.at(threadIdx.x));
    __syncthreads();
    for (int b0 = 0, buf = 0; b0 < nt; b0 += block, buf ^= 1) {
        if (b0 > 0) __syncthreads();  // the block before is done, and this one's places are here
        const int n = nt - b0 < block ? nt - b0 : block, ahead = b0 + block + threadIdx.x;
        if ((int)threadIdx.x < block && ahead < nt) places[buf ^ 1][threadIdx.x] = place_of(c, pos, seq, own.at(ahead));
        if (!live) continue;
        for (int ta = tl; ta < n; ta += kLoadUnroll * par) {
            uint2 w[kLoadUnroll];
            float d[kLoadUnroll];
            int64_t page[kLoadUnroll];
#pragma unroll
            for (int u = 0; u < kLoadUnroll; u++) {
                // No branches: with one around each load a thread has a single load in flight (32768 tokens
                // of 8 x 128 values: 92 us then, 60 us so, 5.6 TB/s).
                const int t = ta + u * par;
                const Place p = places[buf][t < n ? t : n - 1];
                page[u] = p.page;
                int64_t at = p.page < 0 ? 0 : p.page + (int64_t)p.o * c.row_bytes, sat = p.page < 0 ? 0 : p.page + 4 * p.o;
                if (!QMM_IN_BOUNDS(g_pages_error, at + (int64_t)head * c.row_bytes + kQuad * quad + kQuad - 1,
                                   c.num_pages * c.stride))
                    at = 0;
                if (TYPE == QMM_KV_Q8 && !QMM_IN_BOUNDS(g_pages_error, sat + c.scales + 4 * (int64_t)head + 3, c.num_pages * c.stride))
                    sat = 0;
                if (TYPE == QMM_KV_Q8) {
                    w[u].x = ld_here(reinterpret_cast<const uint32_t*>(pool + at));
                    d[u] = __uint_as_float(ld_here(reinterpret_cast<const uint32_t*>(scales + sat)));
                } else {
                    w[u] = ld_here(reinterpret_cast<const uint2*>(pool + at));
                }
            }
#pragma unroll
            for (int u = 0; u < kLoadUnroll; u++) {
                const int t = ta + u * par;
                if (t >= n || places[buf][t].o < 0) continue;
                if (!QMM_IN_BOUNDS(g_pages_error, own.at(b0 + t) * ld + (int64_t)h * c.hd + 4 * quad + 3, T * ld)) continue;
                float4 y;
                if (TYPE == QMM_KV_Q8) {  // d * code, rounded once
                    const uint32_t b = w[u].x ^ 0x80808080u;
                    y.x = __fmul_rn(d[u], code_f(b, 0x7640u));
                    y.y = __fmul_rn(d[u], code_f(b, 0x7641u));
                    y.z = __fmul_rn(d[u], code_f(b, 0x7642u));
                    y.w = __fmul_rn(d[u], code_f(b, 0x7643u));
                } else {
                    y = make_float4(h2f(w[u].x), h2f(w[u].x >> 16), h2f(w[u].y), h2f(w[u].y >> 16));
                }
                if (page[u] < 0) y = make_float4(0.f, 0.f, 0.f, 0.f);
                *reinterpret_cast<float4*>(out + own.at(b0 + t) * ld) = y;
            }
        }
    }
}

qmm_status rope_check(const qmm_rope_spec* r, int64_t hd, RowArgs* a);

}  // namespace qmm

using namespace qmm;

extern "C" {

unsigned qmm_internal_pages_error(int clear) {
    unsigned v = 0;
    cudaMemcpyFromSymbol(&v, g_pages_error, sizeof(v));
    if (clear) {
        const unsigned z = 0;
        cudaMemcpyToSymbol(g_pages_error, &z, sizeof(z));
    }
    return v;
}

size_t qmm_kv_page_bytes(int type, int64_t Hkv, int64_t page_size, int64_t hd) {
    const int64_t rb = kv_row_bytes_of(type, hd);
    if (rb == 0 || !head_dim_ok(hd) || Hkv < 1 || Hkv > 1024 || page_size < 1 || page_size > 4096 ||
        kv_log2(page_size) < 0)
        return 0;
    return (size_t)(Hkv * page_size * (rb + (type == QMM_KV_Q8 ? 4 : 0)));
}

qmm_status qmm_kv_store(const qmm_kv_pages* cache, const float* k, int64_t ldk, const float* v, int64_t ldv,
                        const int32_t* pos, const int32_t* seq, int64_t T, const qmm_rope_spec* rope, const float* q,
                        int64_t ldq, float* q_out, int64_t ldqo, int64_t Hq, qmm_stream_t stream) {
    if (!k || !v || !pos || (q && (!q_out || !rope))) return QMM_E_NULL;
    KvPages c;
    qmm_status st = kv_pages_check(cache, &c);
    if (st != QMM_OK) return st;
    const int64_t row = (int64_t)c.Hkv * c.hd;
    if (T < 1 || T > kMaxDim || !row_stride_ok(ldk, row) || !row_stride_ok(ldv, row)) return QMM_E_SHAPE;
    if (!seq && T > c.num_seqs) return QMM_E_SHAPE;
    if (q && (Hq < 1 || Hq > kHeadsMax || !row_stride_ok(ldq, Hq * c.hd) || !row_stride_ok(ldqo, Hq * c.hd) ||
              (q == q_out && ldq != ldqo)))
        return QMM_E_SHAPE;
    RowArgs a = {};
    if (rope) {
        st = rope_check(rope, c.hd, &a);
        if (st != QMM_OK) return st;
    }
    if (!aligned16(k) || !aligned16(v) || !aligned4(pos) || !aligned4(seq) || !aligned16(q) || (q && !aligned16(q_out)))
        return QMM_E_ALIGN;
    a.k = k, a.v = v, a.q = q, a.q_out = q_out, a.pos = pos, a.seq = seq;
    a.T = T, a.ldk = ldk, a.ldv = ldv, a.ldq = ldq, a.ldqo = ldqo;
    a.Hq = q ? (int)Hq : 0;
    return rows_launch(cache->type, c, a, c.hd, (cudaStream_t)stream);
}

qmm_status qmm_kv_load(const qmm_kv_pages* cache, const int32_t* pos, const int32_t* seq, int64_t T, float* k_out,
                       int64_t ldk, float* v_out, int64_t ldv, qmm_stream_t stream) {
    if (!pos || (!k_out && !v_out)) return QMM_E_NULL;
    KvPages c;
    const qmm_status st = kv_pages_check(cache, &c);
    if (st != QMM_OK) return st;
    const int64_t row = (int64_t)c.Hkv * c.hd;
    if (T < 1 || T > kMaxDim || (k_out && !row_stride_ok(ldk, row)) || (v_out && !row_stride_ok(ldv, row)))
        return QMM_E_SHAPE;
    if (!seq && T > c.num_seqs) return QMM_E_SHAPE;
    if (!aligned4(pos) || !aligned4(seq) || !aligned16(k_out) || !aligned16(v_out)) return QMM_E_ALIGN;
    const int columns = (int)(row / 4) * ((k_out ? 1 : 0) + (v_out ? 1 : 0));
    const int par = columns < kLoadThreads ? kLoadThreads / columns : 1;
    const int64_t parts = (columns + kLoadThreads - 1) / kLoadThreads;
    const int side_by_side = par < kLoadTokens ? par : kLoadTokens, block = kLoadTokens - kLoadTokens % side_by_side;
    const dim3 grid(token_ctas(T, parts, kLoadCtas, side_by_side), (unsigned)parts);
    auto go = [&](auto kern) {
        return launch_pdl(kern, grid, kLoadThreads, 0, (cudaStream_t)stream, c, pos, seq, k_out, ldk, v_out, ldv, T,
                          side_by_side, block);
    };
    return cache->type == QMM_KV_Q8 ? go(kv_load_kernel<QMM_KV_Q8>) : go(kv_load_kernel<QMM_KV_F16>);
}

}  // extern "C"
