// kvpages.cu -- keys and values into the pages of a cache, and back.
//
//   kv_store  a CTA per few tokens: the tokens' rotation tables into shared memory,
//             then a group of lanes per head row, eight values a lane -- key rows
//             are rotated and quantized, value rows quantized, query rows rotated
//             and written as f32.  One launch for all three, each value read once
//   kv_load   four values a thread: 4 (8) bytes of codes in, 16 bytes out
// Both are bound by memory; the 8-bit rule is qmm_kv_quantize's, step by step.
#include "kvpages.cuh"
#include "rope_device.cuh"

namespace qmm {

static __device__ unsigned int g_pages_error = 0;

constexpr int kStoreThreads = 256;
constexpr int kStoreTable = 1024;  // (cos, sin) entries in shared memory

struct StoreArgs {
    const float* k;
    const float* v;
    const float* q;  // may be null: no queries
    float* q_out;
    const int32_t* pos;
    const int32_t* seq;  // may be null: token t belongs to sequence t
    const uint64_t* freqs;
    int64_t T, ldk, ldv, ldq, ldqo;
    int Hq;
    float mscale;
    RopeLayout L;
};

// width: lanes per row, hd / 8 rounded up to a power of two; tpb: tokens per CTA
template <int TYPE>
__global__ void __launch_bounds__(kStoreThreads) kv_store_kernel(KvPages c, StoreArgs a, int width, int tpb) {
    __shared__ float4 cs[kStoreTable];
    pdl_wait();
    const int64_t t0 = (int64_t)blockIdx.x * tpb;
    const int nt = a.T - t0 < tpb ? (int)(a.T - t0) : tpb;
    const int half = a.L.n_rot >> 1;
    for (int i = threadIdx.x; i < nt * half; i += kStoreThreads) {
        const int t = i / half;
        const float4 e = turn_cos_sin((uint64_t)(int64_t)a.pos[t0 + t] * a.freqs[i - t * half], a.mscale);
        if (QMM_IN_BOUNDS(g_pages_error, i, kStoreTable)) cs[i] = e;
    }
    __syncthreads();
    const int rows = 2 * c.Hkv + a.Hq;  // of a token: keys, values, queries
    const int groups = kStoreThreads / width, group = threadIdx.x / width, o = threadIdx.x - group * width;
    const int total = nt * rows, rounds = (total + gridDim.y * groups - 1) / (gridDim.y * groups);
    for (int it = 0; it < rounds; it++) {  // the same count for every lane: the shuffles need whole warps
        const int i = (it * gridDim.y + blockIdx.y) * groups + group;
        const int tl = i / rows, r = i - tl * rows;
        const int64_t t = t0 + tl;
        const bool live = i < total && 8 * o < c.hd;
        const int pos = i < total ? a.pos[t] : -1;
        const bool query = r >= 2 * c.Hkv, value = !query && r >= c.Hkv;
        const int h = query ? r - 2 * c.Hkv : (value ? r - c.Hkv : r);
        RopeLayout L = a.L;
        if (value) L.n_rot = L.halves = L.scattered = 0;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = 0.0f;
        if (live && pos >= 0) {
            const int64_t ld = query ? a.ldq : (value ? a.ldv : a.ldk);
            const float* x = query ? a.q : (value ? a.v : a.k);
            if (QMM_IN_BOUNDS(g_pages_error, t * ld + (int64_t)h * c.hd + c.hd - 1, a.T * ld))
                rope_load8(L, o, x + t * ld + (int64_t)h * c.hd, v);
            rope_turn8(L, o, v, cs + tl * half);
        }
        int id = -1;
        if (live && pos >= 0 && !query) {
            const int64_t s = a.seq ? (int64_t)a.seq[t] : t;
            id = kv_page_of(c, s, pos);
            if (id < 0) atomicOr(&g_pages_error, kErrPlace);
        }
        const int off = pos & ((1 << c.page_shift) - 1);
        uint8_t* pool = value ? c.v : c.k;
        if (query) {
            if (live && pos >= 0 && QMM_IN_BOUNDS(g_pages_error, t * a.ldqo + (int64_t)h * c.hd + c.hd - 1, a.T * a.ldqo))
                rope_store8(L, o, a.q_out + t * a.ldqo + (int64_t)h * c.hd, v);
        }
        if (TYPE == QMM_KV_Q8) {
            float amax = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; j++) amax = fmaxf(amax, fabsf(v[j]));
            for (int m = width >> 1; m > 0; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, m));
            if (id >= 0) {
                const float inv = amax != 0.0f ? __fdiv_rn(127.0f, amax) : 0.0f;
                uint32_t b[8];
#pragma unroll
                for (int j = 0; j < 8; j++)
                    b[j] = (uint32_t)clampi(__float2int_rn(__fmul_rn(v[j], inv)), -128, 127) & 0xFFu;
                const int64_t at = kv_row_at(c, id, h, off), sat = kv_scale_at(c, id, h, off);
                if (QMM_IN_BOUNDS(g_pages_error, at + c.hd - 1, c.num_pages * c.stride) &&
                    QMM_IN_BOUNDS(g_pages_error, sat + 3, c.num_pages * c.stride)) {
                    if (L.scattered) {
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            const int2 e = rope_pair(L, 4 * o + j);
                            pool[at + e.x] = (uint8_t)b[j];
                            pool[at + e.y] = (uint8_t)b[j + 4];
                        }
                    } else {
                        const uint32_t w0 = b[0] | b[1] << 8 | b[2] << 16 | b[3] << 24;
                        const uint32_t w1 = b[4] | b[5] << 8 | b[6] << 16 | b[7] << 24;
                        *reinterpret_cast<uint32_t*>(pool + at + rope_first(L, o)) = w0;
                        *reinterpret_cast<uint32_t*>(pool + at + rope_second(L, o)) = w1;
                    }
                    if (o == 0) *reinterpret_cast<float*>(pool + sat) = __fdiv_rn(amax, 127.0f);
                }
            }
        } else if (id >= 0) {
            const int64_t at = kv_row_at(c, id, h, off);
            if (QMM_IN_BOUNDS(g_pages_error, at + 2 * c.hd - 1, c.num_pages * c.stride)) {
                __half* row = reinterpret_cast<__half*>(pool + at);
                if (L.scattered) {
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const int2 e = rope_pair(L, 4 * o + j);
                        row[e.x] = __float2half_rn(v[j]);
                        row[e.y] = __float2half_rn(v[j + 4]);
                    }
                } else {
                    const uint32_t w0 = f2h_bits(v[0]) | f2h_bits(v[1]) << 16, w1 = f2h_bits(v[2]) | f2h_bits(v[3]) << 16;
                    const uint32_t w2 = f2h_bits(v[4]) | f2h_bits(v[5]) << 16, w3 = f2h_bits(v[6]) | f2h_bits(v[7]) << 16;
                    *reinterpret_cast<uint2*>(row + rope_first(L, o)) = make_uint2(w0, w1);
                    *reinterpret_cast<uint2*>(row + rope_second(L, o)) = make_uint2(w2, w3);
                }
            }
        }
    }
    pdl_launch_dependents();
}

constexpr int kLoadThreads = 256;
constexpr int kLoadUnroll = 4;

// A thread's quads of four values are kLoadThreads apart in the list (token, pool,
// head, quad) of the CTA's tpb tokens; the loads of kLoadUnroll of them are issued
// before the first is converted.
template <int TYPE>
__global__ void __launch_bounds__(kLoadThreads) kv_load_kernel(KvPages c, const int32_t* __restrict__ pos,
                                                               const int32_t* __restrict__ seq, float* k_out, int64_t ldk,
                                                               float* v_out, int64_t ldv, int64_t T, int tpb) {
    pdl_wait();
    const int64_t t0 = (int64_t)blockIdx.x * tpb;
    const int nt = T - t0 < tpb ? (int)(T - t0) : tpb;
    const int quads = c.hd >> 2, row = c.Hkv * quads;  // per head row; per token and pool
    const int pools = (k_out ? 1 : 0) + (v_out ? 1 : 0);
    const int total = nt * pools * row, step = gridDim.y * kLoadThreads;
    for (int i0 = blockIdx.y * kLoadThreads + threadIdx.x; i0 < total; i0 += kLoadUnroll * step) {
        uint2 w[kLoadUnroll];
        float d[kLoadUnroll];
        float* dst[kLoadUnroll];
#pragma unroll
        for (int u = 0; u < kLoadUnroll; u++) {
            const int i = i0 + u * step;
            dst[u] = nullptr;
            if (i >= total) continue;
            const int tp = i / row, e = i - tp * row, h = e / quads, quad = e - h * quads;
            const int tl = pools == 2 ? tp >> 1 : tp;
            const bool value = pools == 2 ? (tp & 1) : !k_out;
            const int64_t t = t0 + tl;
            const int p = pos[t];
            if (p < 0) continue;
            const int64_t ld = value ? ldv : ldk;
            if (!QMM_IN_BOUNDS(g_pages_error, t * ld + (int64_t)h * c.hd + 4 * quad + 3, T * ld)) continue;
            dst[u] = (value ? v_out : k_out) + t * ld + (int64_t)h * c.hd + 4 * quad;
            const int id = kv_page_of(c, seq ? (int64_t)seq[t] : t, p);
            w[u] = make_uint2(0u, 0u);
            d[u] = 0.0f;
            if (id < 0) {  // a zero row, and the status
                atomicOr(&g_pages_error, kErrPlace);
                continue;
            }
            const uint8_t* pool = value ? c.v : c.k;
            const int off = p & ((1 << c.page_shift) - 1);
            const int64_t at = kv_row_at(c, id, h, off) + (TYPE == QMM_KV_Q8 ? 4 : 8) * quad;
            if (!QMM_IN_BOUNDS(g_pages_error, at + 7, c.num_pages * c.stride)) continue;
            if (TYPE == QMM_KV_Q8) {
                w[u].x = *reinterpret_cast<const uint32_t*>(pool + at);
                d[u] = *reinterpret_cast<const float*>(pool + kv_scale_at(c, id, h, off));
            } else {
                w[u] = *reinterpret_cast<const uint2*>(pool + at);
            }
        }
#pragma unroll
        for (int u = 0; u < kLoadUnroll; u++) {
            if (!dst[u]) continue;
            float4 y;
            if (TYPE == QMM_KV_Q8) {  // d * code, rounded once
                y.x = __fmul_rn(d[u], (float)(int8_t)(w[u].x & 0xFFu));
                y.y = __fmul_rn(d[u], (float)(int8_t)(w[u].x >> 8 & 0xFFu));
                y.z = __fmul_rn(d[u], (float)(int8_t)(w[u].x >> 16 & 0xFFu));
                y.w = __fmul_rn(d[u], (float)(int8_t)(w[u].x >> 24));
            } else {
                y = make_float4(h2f(w[u].x), h2f(w[u].x >> 16), h2f(w[u].y), h2f(w[u].y >> 16));
            }
            *reinterpret_cast<float4*>(dst[u]) = y;
        }
    }
    pdl_launch_dependents();
}

qmm_status rope_check(const qmm_rope_spec* r, int64_t hd, RopeLayout* L);

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
    StoreArgs a = {};
    if (rope) {
        st = rope_check(rope, c.hd, &a.L);
        if (st != QMM_OK) return st;
        a.freqs = (const uint64_t*)rope->freqs;
        a.mscale = rope->mscale;
    }
    if (!aligned16(k) || !aligned16(v) || !aligned4(pos) || !aligned4(seq) || !aligned16(q) || (q && !aligned16(q_out)))
        return QMM_E_ALIGN;
    a.k = k, a.v = v, a.q = q, a.q_out = q_out, a.pos = pos, a.seq = seq;
    a.T = T, a.ldk = ldk, a.ldv = ldv, a.ldq = ldq, a.ldqo = ldqo;
    a.Hq = q ? (int)Hq : 0;
    int width = 2;
    while (8 * width < c.hd) width *= 2;
    const int groups = kStoreThreads / width, rows = 2 * c.Hkv + a.Hq;
    int tpb = 2 * groups / rows;  // tokens per CTA: about two rows per group
    if (a.L.n_rot && tpb > 2 * kStoreTable / a.L.n_rot) tpb = 2 * kStoreTable / a.L.n_rot;
    if (tpb < 1) tpb = 1;
    int64_t parts = tpb > 1 ? 1 : (rows + 2 * groups - 1) / (2 * groups);  // CTAs that share a token's rows
    const int64_t blocks = (T + tpb - 1) / tpb;
    const dim3 grid((unsigned)blocks, (unsigned)parts);
    const cudaStream_t cs = (cudaStream_t)stream;
    if (cache->type == QMM_KV_Q8)
        return launch_pdl(kv_store_kernel<QMM_KV_Q8>, grid, kStoreThreads, 0, cs, c, a, width, tpb);
    return launch_pdl(kv_store_kernel<QMM_KV_F16>, grid, kStoreThreads, 0, cs, c, a, width, tpb);
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
    const int per = (int)(row / 4) * ((k_out ? 1 : 0) + (v_out ? 1 : 0));  // quads of a token
    constexpr int want = kLoadThreads * kLoadUnroll;
    int tpb = want / per;
    if (tpb < 1) tpb = 1;
    const int64_t parts = tpb > 1 ? 1 : (per + want - 1) / want;
    const dim3 grid((unsigned)((T + tpb - 1) / tpb), (unsigned)parts);
    const cudaStream_t cs = (cudaStream_t)stream;
    if (cache->type == QMM_KV_Q8)
        return launch_pdl(kv_load_kernel<QMM_KV_Q8>, grid, kLoadThreads, 0, cs, c, pos, seq, k_out, ldk, v_out, ldv, T,
                          tpb);
    return launch_pdl(kv_load_kernel<QMM_KV_F16>, grid, kLoadThreads, 0, cs, c, pos, seq, k_out, ldk, v_out, ldv, T,
                      tpb);
}

}  // extern "C"
