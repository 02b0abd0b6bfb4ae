// Shared by the library's source files; nothing here is exported.
#ifndef SGEMV_INTERNAL_H
#define SGEMV_INTERNAL_H

#include <cstdint>

#include "sgemv.h"

// Rows of len bytes in memory, step bytes apart.
struct SgemvRows {
    const void* p;
    int64_t rows, step, len;
};

// Whether two buffers (either may be absent) share bytes.  Ranges that meet
// count as sharing, except where both are columns of one wider buffer.
inline bool sgemv_overlap(const SgemvRows& a, const SgemvRows& b) {
    if (!a.p || !b.p) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    const uintptr_t a1 = a0 + (uintptr_t)(a.rows - 1) * (uintptr_t)a.step + (uintptr_t)a.len;
    const uintptr_t b1 = b0 + (uintptr_t)(b.rows - 1) * (uintptr_t)b.step + (uintptr_t)b.len;
    if (a1 <= b0 || b1 <= a0) return false;
    if (a.rows > 1 && b.rows > 1 && a.step == b.step) {
        const uintptr_t step = (uintptr_t)a.step, off = b0 > a0 ? (b0 - a0) % step : (step - (a0 - b0) % step) % step;
        return !(off >= (uintptr_t)a.len && off + (uintptr_t)b.len <= step);
    }
    return true;
}

// Keep a failed HIP call's hipError_t for sgemv_last_hip_error.
__attribute__((visibility("hidden"))) int sgemv_hip_failed(int hip_error);

// SGEMV_OK when *d is a description that the q4 packer makes.
__attribute__((visibility("hidden"))) int sgemv_q4_check_desc(const sgemv_q4_desc* d);

#endif
