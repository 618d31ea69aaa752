// kvpages.cuh -- the paged key-value cache: its description as the kernels take
// it, the host's checks of it, and the page of a position.
//
// A page holds page_size positions (a power of two) of every KV head.  Codes come
// first, head by head: row (head h, position o) at (h * page_size + o) * row_bytes,
// hd bytes of int8 or 2 hd of f16.  8-bit rows keep their f32 scales behind all
// codes, in the same order.  Against rows of 4 + hd bytes with the scale in front
// (qmm_kv_quantize's), this keeps every row on a 16-byte boundary, so that the
// attention fetches it with 16-byte asynchronous copies, and a head's positions
// side by side, so that a CTA that reads one head reads whole lines.
#pragma once

#include "qmm_device.cuh"
#include "qmm_host.h"

namespace qmm {

struct KvPages {
    uint8_t* k;
    uint8_t* v;
    const int32_t* table;
    int64_t stride;    // bytes from one page to the next
    int64_t num_seqs;
    int64_t max_pages;
    int64_t scales;    // byte offset of the scales in a page (8-bit rows)
    int num_pages;
    int Hkv, hd;
    int row_bytes;     // of a row's codes
    int page_shift;    // log2 of page_size
};

// The page of position pos of sequence seq, or -1 where the table holds none.
__device__ __forceinline__ int kv_page_of(const KvPages& c, int64_t seq, int64_t pos) {
    const int64_t pg = pos >> c.page_shift;
    if (seq < 0 || seq >= c.num_seqs || pg >= c.max_pages) return -1;
    const int id = __ldg(c.table + seq * c.max_pages + pg);
    return (unsigned)id < (unsigned)c.num_pages ? id : -1;
}

constexpr unsigned kErrPlace = 2u;  // a position without a page, a sequence outside the table

inline int kv_log2(int64_t n) {
    int s = 0;
    while (s < 31 && ((int64_t)1 << s) < n) s++;
    return ((int64_t)1 << s) == n ? s : -1;
}
inline int64_t kv_row_bytes_of(int type, int64_t hd) {
    return type == QMM_KV_Q8 ? hd : (type == QMM_KV_F16 ? 2 * hd : 0);
}

// Checks a cache's description and lays it out for the kernels.
inline qmm_status kv_pages_check(const qmm_kv_pages* c, KvPages* d) {
    if (!c || !c->k || !c->v || !c->table) return QMM_E_NULL;
    if (c->type != QMM_KV_Q8 && c->type != QMM_KV_F16) return QMM_E_TYPE;
    const size_t bytes = qmm_kv_page_bytes(c->type, c->Hkv, c->page_size, c->hd);
    if (bytes == 0 || c->num_pages < 1 || c->num_pages > kMaxDim || c->num_seqs < 1 || c->num_seqs > kMaxDim ||
        c->max_pages < 1 || c->max_pages > kMaxDim || c->page_stride < (int64_t)bytes || c->page_stride % 16 ||
        c->page_stride > ((int64_t)1 << 36))
        return QMM_E_SHAPE;
    if (!aligned16(c->k) || !aligned16(c->v) || !aligned4(c->table)) return QMM_E_ALIGN;
    d->k = (uint8_t*)c->k;
    d->v = (uint8_t*)c->v;
    d->table = c->table;
    d->stride = c->page_stride;
    d->num_seqs = c->num_seqs;
    d->max_pages = c->max_pages;
    d->num_pages = (int)c->num_pages;
    d->Hkv = (int)c->Hkv;
    d->hd = (int)c->hd;
    d->row_bytes = (int)kv_row_bytes_of(c->type, c->hd);
    d->scales = c->Hkv * c->page_size * (int64_t)d->row_bytes;
    d->page_shift = kv_log2(c->page_size);
    return QMM_OK;
}

}  // namespace qmm
