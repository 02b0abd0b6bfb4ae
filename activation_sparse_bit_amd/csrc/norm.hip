// The norms before and after a block, with its gate and residual scale.
//
//   u = y or norm(y),  r = residual + scale * gate * u,  x = norm(r)
//   norm(v) = (v - c) / sqrt(mean((v - c)^2) + eps) * w + b
//
// One workgroup (one wavefront for short rows) owns a row and keeps it in
// registers as fp32 from the first load to the last store, so every byte
// moves once and both norms see unrounded values.  Means and squared
// deviations are two sums over the row each (the deviations are taken from
// the mean, not from a difference of large sums), added over the lanes of a
// wavefront and then over the wavefronts in a fixed order.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "internal.h"

namespace {

typedef uint32_t uint4_t __attribute__((ext_vector_type(4)));
typedef uint32_t uint4_u2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t uint4_u4 __attribute__((ext_vector_type(4), aligned(4)));

// Eight elements as loaded: 16 bytes of 16-bit types, 32 bytes of fp32.
template <int BYTES>
struct Raw {
    uint4_t v[BYTES / 2];
};

// Elements e0 .. e0 + 8 of a row, zero beyond D.
template <int BYTES>
__device__ __forceinline__ Raw<BYTES> load8(const void* p, int64_t row, int e0, int D) {
    Raw<BYTES> r;
#pragma unroll
    for (int i = 0; i < BYTES / 2; ++i) r.v[i] = uint4_t{0, 0, 0, 0};
    if constexpr (BYTES == 2) {
        const uint16_t* q = static_cast<const uint16_t*>(p) + row + e0;
        if (e0 + 8 <= D) {
            r.v[0] = *reinterpret_cast<const uint4_u2*>(q);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (e0 + i < D) r.v[0][i >> 1] |= (uint32_t)q[i] << (16 * (i & 1));
        }
    } else {
        const uint32_t* q = static_cast<const uint32_t*>(p) + row + e0;
        if (e0 + 8 <= D) {
            r.v[0] = *reinterpret_cast<const uint4_u4*>(q);
            r.v[1] = *reinterpret_cast<const uint4_u4*>(q + 4);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (e0 + i < D) r.v[i >> 2][i & 3] = q[i];
        }
    }
    return r;
}

template <int BYTES>
__device__ __forceinline__ void to_f32(const Raw<BYTES>& r, bool bf16, float* f) {
    if constexpr (BYTES == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t e = r.v[i >> 2][i & 3];   // by value: a bit cast of the vector element itself reads element 0
            f[i] = __builtin_bit_cast(float, e);
        }
    } else if (bf16) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = __builtin_bit_cast(float, (i & 1) ? r.v[0][i >> 1] & 0xFFFF0000u : r.v[0][i >> 1] << 16);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = (float)__builtin_bit_cast(_Float16, (uint16_t)(r.v[0][i >> 1] >> (16 * (i & 1))));
    }
}

// A vector of length D (weights, a shared gate) in any type.
__device__ __forceinline__ void load8_any(const void* p, int type, int64_t row, int e0, int D, float* f) {
    if (type == SGEMV_F32) to_f32<4>(load8<4>(p, row, e0, D), false, f);
    else to_f32<2>(load8<2>(p, row, e0, D), type == SGEMV_BF16, f);
}

__device__ __forceinline__ void store8(void* p, int type, int64_t row, int e0, int D, const float* f) {
    if (type == SGEMV_F32) {
        float* q = static_cast<float*>(p) + row + e0;
        if (e0 + 8 <= D) {
            uint4_t a, b;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = __builtin_bit_cast(uint32_t, f[i]);
                b[i] = __builtin_bit_cast(uint32_t, f[4 + i]);
            }
            *reinterpret_cast<uint4_u4*>(q) = a;
            *reinterpret_cast<uint4_u4*>(q + 4) = b;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (e0 + i < D) q[i] = f[i];
        }
        return;
    }
    uint16_t h[8];
    if (type == SGEMV_BF16) {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = __builtin_bit_cast(uint16_t, (__bf16)f[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = __builtin_bit_cast(uint16_t, (_Float16)f[i]);
    }
    uint16_t* q = static_cast<uint16_t*>(p) + row + e0;
    if (e0 + 8 <= D) {
        uint4_t a;
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = (uint32_t)h[2 * i] | (uint32_t)h[2 * i + 1] << 16;
        *reinterpret_cast<uint4_u2*>(q) = a;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (e0 + i < D) q[i] = h[i];
    }
}

// Sum of v over the T threads of a row, the same value in each.  `slot`
// names the call: two calls in a row use two places, so one barrier each.
template <int T>
__device__ __forceinline__ float row_sum(float v, float (*part)[16], int slot) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
    if constexpr (T > 64) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) part[slot][wave] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < T / 64; ++w) v += part[slot][w];
    }
    return v;
}

// v <- (v - c) / sqrt(mean((v - c)^2) + eps) over the row; elements beyond D
// (zero on entry) do not count.
template <int T, int CH>
__device__ __forceinline__ void normalize(float (&v)[CH * 8], int tid, const sgemv_norm& a, float (*part)[16],
                                          int slot) {
    const float inv_d = 1.0f / (float)a.D;
    if (a.flags & SGEMV_NORM_CENTER) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < CH * 8; ++i) s += v[i];
        const float mean = row_sum<T>(s, part, slot) * inv_d;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if ((c * T + tid) * 8 + i < a.D) v[c * 8 + i] -= mean;
    }
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < CH * 8; ++i) q = fmaf(v[i], v[i], q);
    const float inv = 1.0f / sqrtf(row_sum<T>(q, part, slot + 1) * inv_d + a.eps);
#pragma unroll
    for (int i = 0; i < CH * 8; ++i) v[i] *= inv;
}

// v <- v * w + b for the eight elements from e0 on.
__device__ __forceinline__ void affine(float* v, const void* w, const void* b, const sgemv_norm& a, int e0) {
    float t[8];
    if (w) {
        load8_any(w, a.w_type, 0, e0, a.D, t);
        const float one = (a.flags & SGEMV_NORM_PLUS_ONE) ? 1.0f : 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= t[i] + one;
    }
    if (b) {
        load8_any(b, a.w_type, 0, e0, a.D, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += t[i];
    }
}

// T threads a row, CH chunks of eight elements a thread (D <= 8 * T * CH).
// RB, YB: bytes of an element of the residual and of y.
template <int T, int CH, int RB, int YB>
__global__ __launch_bounds__(T < 256 ? 256 : T) void k_norm(sgemv_norm a) {
    __shared__ float part[4][16];
    constexpr int kRows = T < 256 ? 256 / T : 1;   // rows per workgroup
    const int tid = threadIdx.x % T;
    const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / T;
    if (row >= a.rows) return;   // only where a wavefront owns a row: no barrier follows there
    const int D = a.D;

    Raw<RB> rr[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) rr[c] = load8<RB>(a.residual, row * a.ld_residual, (c * T + tid) * 8, D);
    float r[CH * 8];
    if (a.y) {
        Raw<YB> yr[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) yr[c] = load8<YB>(a.y, row * a.ld_y, (c * T + tid) * 8, D);
        float u[CH * 8];
#pragma unroll
        for (int c = 0; c < CH; ++c) to_f32<YB>(yr[c], a.y_type == SGEMV_BF16, u + c * 8);
        if (a.flags & SGEMV_NORM_POST) {
            normalize<T, CH>(u, tid, a, part, 0);
#pragma unroll
            for (int c = 0; c < CH; ++c) affine(u + c * 8, a.post_weight, a.post_bias, a, (c * T + tid) * 8);
        }
        if (a.gate) {
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                float g[8];
                load8_any(a.gate, a.y_type, row * a.ld_gate, (c * T + tid) * 8, D, g);
#pragma unroll
                for (int i = 0; i < 8; ++i) u[c * 8 + i] *= g[i];
            }
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) to_f32<RB>(rr[c], a.residual_type == SGEMV_BF16, r + c * 8);
#pragma unroll
        for (int i = 0; i < CH * 8; ++i) r[i] = fmaf(a.scale, u[i], r[i]);
    } else {
#pragma unroll
        for (int c = 0; c < CH; ++c) to_f32<RB>(rr[c], a.residual_type == SGEMV_BF16, r + c * 8);
    }
    if (a.residual_out) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
            if ((c * T + tid) * 8 < D)
                store8(a.residual_out, a.residual_type, row * a.ld_residual_out, (c * T + tid) * 8, D, r + c * 8);
    }
    // elements beyond D are not zero here where a shift or scale moved them
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if ((c * T + tid) * 8 + i >= D) r[c * 8 + i] = 0.0f;
    normalize<T, CH>(r, tid, a, part, 2);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int e0 = (c * T + tid) * 8;
        if (e0 < D) {
            affine(r + c * 8, a.weight, a.bias, a, e0);
            store8(a.x, a.x_type, row * a.ld_x, e0, D, r + c * 8);
        }
    }
}

typedef void (*Kernel)(sgemv_norm);

template <int T, int CH>
Kernel pick_types(int RB, int YB) {
    if (RB == 2) return YB == 2 ? k_norm<T, CH, 2, 2> : k_norm<T, CH, 2, 4>;
    return YB == 2 ? k_norm<T, CH, 4, 2> : k_norm<T, CH, 4, 4>;
}

int size_of(int type) { return type == SGEMV_F32 ? 4 : 2; }
bool type_ok(int type) { return type >= SGEMV_F16 && type <= SGEMV_F32; }
bool aligned_to(const void* p, int a) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(a - 1)) == 0; }

// Rows of D elements in memory.
struct Rows {
    const void* p;
    int64_t rows, ld;
    int size;
    bool whole;   // may be the same buffer as an output
};

// Whether an output and another buffer share bytes in a way that the kernel
// does not allow for.
bool clash(const Rows& out, const Rows& b, int64_t D) {
    if (!out.p || !b.p) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(out.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    const uintptr_t step_a = (uintptr_t)out.ld * out.size, step_b = (uintptr_t)b.ld * b.size;
    const uintptr_t len_a = (uintptr_t)D * out.size, len_b = (uintptr_t)D * b.size;
    const uintptr_t a1 = a0 + (uintptr_t)(out.rows - 1) * step_a + len_a;
    const uintptr_t b1 = b0 + (uintptr_t)(b.rows - 1) * step_b + len_b;
    if (a1 <= b0 || b1 <= a0) return false;
    if (a0 == b0 && out.size == b.size && (out.rows == 1 || step_a == step_b)) return !b.whole;
    if (out.rows > 1 && b.rows > 1 && step_a == step_b) {   // columns of one wider buffer
        const uintptr_t off = b0 > a0 ? (b0 - a0) % step_a : (step_a - (a0 - b0) % step_a) % step_a;
        return !(off >= len_a && off + len_b <= step_a);
    }
    return true;
}

}  // namespace

extern "C" int sgemv_block_norm(const sgemv_norm* args, void* stream) {
    if (!args) return SGEMV_EINVAL;
    sgemv_norm a = *args;
    if (a.rows < 0 || a.rows > 0x7FFFFFFF || a.D < 1 || a.D > SGEMV_MAX_K) return SGEMV_ESIZE;
    if (a.rows == 0) return SGEMV_OK;   // an empty buffer has no address
    if (!a.residual || !a.x) return SGEMV_EINVAL;
    if (a.flags & ~(SGEMV_NORM_POST | SGEMV_NORM_CENTER | SGEMV_NORM_PLUS_ONE)) return SGEMV_EINVAL;
    if (!a.y && (a.gate || (a.flags & SGEMV_NORM_POST))) return SGEMV_EINVAL;
    if (!(a.flags & SGEMV_NORM_POST) && (a.post_weight || a.post_bias)) return SGEMV_EINVAL;
    if (!type_ok(a.residual_type) || !type_ok(a.y_type) || !type_ok(a.w_type) || !type_ok(a.x_type))
        return SGEMV_EINVAL;
    if (!(a.eps >= 0.0f) || std::isinf(a.eps)) return SGEMV_EINVAL;
    const int64_t max_ld = (int64_t)1 << 31;   // rows * ld * 4 stays below 2^64
    if (a.ld_residual < a.D || a.ld_residual > max_ld || a.ld_x < a.D || a.ld_x > max_ld) return SGEMV_ESIZE;
    if (a.y && (a.ld_y < a.D || a.ld_y > max_ld)) return SGEMV_ESIZE;
    if (a.gate && a.ld_gate && (a.ld_gate < a.D || a.ld_gate > max_ld)) return SGEMV_ESIZE;
    if (a.residual_out && (a.ld_residual_out < a.D || a.ld_residual_out > max_ld)) return SGEMV_ESIZE;
    const int rb = size_of(a.residual_type), yb = size_of(a.y_type), wb = size_of(a.w_type), xb = size_of(a.x_type);
    if (!aligned_to(a.residual, rb) || !aligned_to(a.residual_out, rb) || !aligned_to(a.y, yb) ||
        !aligned_to(a.gate, yb) || !aligned_to(a.x, xb) || !aligned_to(a.post_weight, wb) ||
        !aligned_to(a.post_bias, wb) || !aligned_to(a.weight, wb) || !aligned_to(a.bias, wb))
        return SGEMV_EALIGN;

    const Rows outs[2] = {{a.x, a.rows, a.ld_x, xb, false}, {a.residual_out, a.rows, a.ld_residual_out, rb, false}};
    const Rows others[] = {{a.residual, a.rows, a.ld_residual, rb, true},
                           {a.y, a.rows, a.ld_y, yb, true},
                           {a.gate, a.ld_gate ? a.rows : 1, a.ld_gate, yb, a.ld_gate != 0},
                           {a.post_weight, 1, a.D, wb, false},
                           {a.post_bias, 1, a.D, wb, false},
                           {a.weight, 1, a.D, wb, false},
                           {a.bias, 1, a.D, wb, false}};
    if (clash(outs[0], outs[1], a.D)) return SGEMV_EINVAL;
    for (const Rows& o : outs)
        for (const Rows& b : others)
            if (clash(o, b, a.D)) return SGEMV_EINVAL;

    Kernel k;
    int T, rows_per = 1;
    if (a.D <= 512) { T = 64; k = pick_types<64, 1>(rb, yb); rows_per = 4; }
    else if (a.D <= 2048) { T = 256; k = pick_types<256, 1>(rb, yb); }
    else if (a.D <= 4096) { T = 256; k = pick_types<256, 2>(rb, yb); }
    else if (a.D <= 8192) { T = 256; k = pick_types<256, 4>(rb, yb); }
    else if (a.D <= 16384) { T = 512; k = pick_types<512, 4>(rb, yb); }
    else if (a.D <= 32768) { T = 1024; k = pick_types<1024, 4>(rb, yb); }
    else { T = 1024; k = pick_types<1024, 8>(rb, yb); }
    void* kargs[] = {&a};
    const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(k), dim3((unsigned)((a.rows + rows_per - 1) / rows_per)),
                                         dim3(T < 256 ? 256 : T), kargs, 0, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? SGEMV_OK : sgemv_hip_failed((int)e);
}
