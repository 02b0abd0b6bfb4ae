// A paged cache's layout, shared by the kernels that read and write it.
#ifndef SGEMV_KV_H
#define SGEMV_KV_H

#include "internal.h"

// What every workspace of these calls begins with: arrival counters, zero
// between calls, whichever call it is, so that one workspace serves them all.
constexpr size_t kSgemvCounterBytes = (size_t)1 << 18;

inline bool sgemv_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline int sgemv_size_of(int type) { return type == SGEMV_F32 ? 4 : type == SGEMV_E4M3 ? 1 : 2; }

// SGEMV_OK when kv describes a cache that the kernels can address.
inline int sgemv_check_kv(const sgemv_kv& kv) {
    if (!kv.k || !kv.v || kv.reserved) return SGEMV_EINVAL;
    if (kv.type != SGEMV_F16 && kv.type != SGEMV_BF16 && kv.type != SGEMV_E4M3) return SGEMV_EINVAL;
    if (kv.type != SGEMV_E4M3 && (kv.k_scale || kv.v_scale)) return SGEMV_EINVAL;
    if (kv.pages < 1 || kv.page_size < 1 || kv.page_size > 65536 || kv.heads < 1 || kv.heads > SGEMV_MAX_HEADS)
        return SGEMV_ESIZE;
    if (kv.dim < 8 || kv.dim > SGEMV_MAX_DIM || kv.dim % 8) return SGEMV_ESIZE;
    if ((int64_t)kv.pages * kv.page_size > 0x7FFFFFFF) return SGEMV_ESIZE;
    // a place's offset stays below 2^62 bytes
    const int64_t strides[6] = {kv.k_page, kv.k_token, kv.k_head, kv.v_page, kv.v_token, kv.v_head};
    const int64_t counts[3] = {kv.pages, kv.page_size, kv.heads};
    for (int i = 0; i < 6; ++i)
        if (strides[i] < 0 || (counts[i % 3] > 1 && (strides[i] < kv.dim || strides[i] > ((int64_t)1 << 60) / counts[i % 3])))
            return SGEMV_ESIZE;
    const int per = 8;   // elements: 16 bytes, or 8 of SGEMV_E4M3
    if (!sgemv_aligned(kv.k, kv.type == SGEMV_E4M3 ? 8 : 16) || !sgemv_aligned(kv.v, kv.type == SGEMV_E4M3 ? 8 : 16) ||
        !sgemv_aligned(kv.k_scale, 4) || !sgemv_aligned(kv.v_scale, 4))
        return SGEMV_EALIGN;
    for (int i = 0; i < 6; ++i)
        if (counts[i % 3] > 1 && strides[i] % per) return SGEMV_EALIGN;
    return SGEMV_OK;
}

// Bytes from the first to past the last value of the keys (or values).
inline int64_t sgemv_kv_bytes(const sgemv_kv& kv, bool keys) {
    const int64_t last = (int64_t)(kv.pages - 1) * (keys ? kv.k_page : kv.v_page) +
                         (int64_t)(kv.page_size - 1) * (keys ? kv.k_token : kv.v_token) +
                         (int64_t)(kv.heads - 1) * (keys ? kv.k_head : kv.v_head) + kv.dim;
    return last * sgemv_size_of(kv.type);
}

inline SgemvRows sgemv_kv_rows(const sgemv_kv& kv, bool keys) {
    return SgemvRows{keys ? kv.k : kv.v, 1, 0, sgemv_kv_bytes(kv, keys)};
}

// Division of 0 <= n < 2^31 by a fixed d in 1 .. 2^16: (n * m) >> s.  With
// 2^(s-31) >= d, m = floor(2^s / d) + 1 is off from 2^s / d by at most 1, and n
// times that stays below 2^s / d.
struct SgemvDiv {
    uint32_t m, d;
    int32_t s;
};

inline SgemvDiv sgemv_div(int d) {
    SgemvDiv r;
    r.d = (uint32_t)d;
    r.s = 31;
    while (((int64_t)1 << (r.s - 31)) < d) ++r.s;
    r.m = (uint32_t)((((uint64_t)1 << r.s) / (uint64_t)d) + 1);
    return r;
}

#endif
