// The norms before and after a block, with its gate and residual scale.
//
//   u = y or norm(y),  r = residual + scale * gate * u,  x = norm(r)
//   norm(v) = (v - c) / sqrt(mean((v - c)^2) + eps) * w + b
//
// One workgroup (one wavefront for short rows) owns a row and keeps it as fp32
// from the first load to the last store, so every byte moves once and both
// norms see unrounded values.  In registers, that is, of which a thread has
// 128: by the compiler's report four runs a thread of an odd width (from 16392
// elements on, from 8200 with more than 256 rows) leave 8 bytes a lane in
// scratch, 200 with an fp32 residual and 16-bit y, and eight runs (from 32776
// on) 132 to 844.  Means and squared deviations are two sums over the row each
// (the deviations are taken from the mean, not from a difference of large
// sums), added over the lanes of a wavefront and then over the wavefronts in a
// fixed order.
//
// A thread owns runs of eight elements, moved as 16-byte pieces at whatever
// address the row has (pieces off a 16-byte boundary cost 3 to 7 % here), and
// the first threads own one element each of what a width that is no multiple
// of eight leaves over.  No element has two owners, so outputs may take the
// place of inputs.
//
// Many rows are bound by HBM: 16384 x 4096 (bf16, both norms, 537 MB) in 94 to
// 99 us, 5.4 to 5.7 TB/s, with an fp32 residual (805 MB) in 143; a library copy
// reaches 5.3.  Few rows are latency: 1 x 4096 in 2.5 us, 16 x 8192 with both
// norms in 5.0, each sum over a row about 0.5 of it.  Odd widths, whose rows are
// few and long, wait at four sums a row: 777 x 5001 in 14.4 us (2.7 TB/s), 300 x
// 12003 with an fp32 residual 19.0 (300 x 12000: 13.1), 300 x 20001 33.8 (20000:
// 20.9).  Above 32768 elements: 300 x 65536 95.8 us, 1.6 TB/s.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "internal.h"

namespace {

typedef uint32_t uint4_t __attribute__((ext_vector_type(4)));
typedef uint32_t uint4_u2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t uint4_u4 __attribute__((ext_vector_type(4), aligned(4)));

// N elements (a run of eight, or one) as loaded: words of BYTES-wide elements.
template <int BYTES, int N>
struct Raw {
    uint4_t v[N == 8 ? BYTES / 2 : 1];

    __device__ __forceinline__ void load(const void* p, int64_t at) {
        if constexpr (N == 1) {
            if constexpr (BYTES == 2) v[0][0] = static_cast<const uint16_t*>(p)[at];
            else v[0][0] = static_cast<const uint32_t*>(p)[at];
        } else if constexpr (BYTES == 2) {
            v[0] = *reinterpret_cast<const uint4_u2*>(static_cast<const uint16_t*>(p) + at);
        } else {
            const uint32_t* q = static_cast<const uint32_t*>(p) + at;
            v[0] = *reinterpret_cast<const uint4_u4*>(q);
            v[1] = *reinterpret_cast<const uint4_u4*>(q + 4);
        }
    }

    __device__ __forceinline__ void get(int type, float (&f)[N]) const {
        // words by value: a bit cast of a vector element itself reads element 0
        if constexpr (BYTES == 4) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint32_t e = v[i >> 2][i & 3];
                f[i] = __builtin_bit_cast(float, e);
            }
        } else if (type == SGEMV_BF16) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint32_t e = v[0][i >> 1];
                f[i] = __builtin_bit_cast(float, (i & 1) ? e & 0xFFFF0000u : e << 16);
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint32_t e = v[0][i >> 1];
                f[i] = (float)__builtin_bit_cast(_Float16, (uint16_t)(e >> (16 * (i & 1))));
            }
        }
    }
};

// The same for a vector (weights, biases) whose type is known at run time
// only; absent where p is NULL.
template <int N>
struct RawAny {
    uint4_t v[N == 8 ? 2 : 1];

    __device__ __forceinline__ void load(const void* p, int type, int64_t at) {
        if (!p) return;
        if (type == SGEMV_F32) {
            Raw<4, N> r;
            r.load(p, at);
#pragma unroll
            for (int i = 0; i < (N == 8 ? 2 : 1); ++i) v[i] = r.v[i];
        } else {
            Raw<2, N> r;
            r.load(p, at);
            v[0] = r.v[0];
        }
    }
    __device__ __forceinline__ void get(int type, float (&f)[N]) const {
        if (type == SGEMV_F32) {
            Raw<4, N> r;
#pragma unroll
            for (int i = 0; i < (N == 8 ? 2 : 1); ++i) r.v[i] = v[i];
            r.get(type, f);
        } else {
            Raw<2, N> r;
            r.v[0] = v[0];
            r.get(type, f);
        }
    }
};

template <int N>
__device__ __forceinline__ void store(void* p, int type, int64_t at, const float (&f)[N]) {
    if (type == SGEMV_F32) {
        float* q = static_cast<float*>(p) + at;
        if constexpr (N == 1) {
            q[0] = f[0];
        } else {
            uint4_t a, b;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = __builtin_bit_cast(uint32_t, f[i]);
                b[i] = __builtin_bit_cast(uint32_t, f[4 + i]);
            }
            *reinterpret_cast<uint4_u4*>(q) = a;
            *reinterpret_cast<uint4_u4*>(q + 4) = b;
        }
        return;
    }
    uint16_t h[N];
    if (type == SGEMV_BF16) {
#pragma unroll
        for (int i = 0; i < N; ++i) h[i] = __builtin_bit_cast(uint16_t, (__bf16)f[i]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) h[i] = __builtin_bit_cast(uint16_t, (_Float16)f[i]);
    }
    uint16_t* q = static_cast<uint16_t*>(p) + at;
    if constexpr (N == 1) {
        q[0] = h[0];
    } else {
        uint4_t a;
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = (uint32_t)h[2 * i] | (uint32_t)h[2 * i + 1] << 16;
        *reinterpret_cast<uint4_u2*>(q) = a;
    }
}

template <int CTRL>
__device__ __forceinline__ float add_lane(float v) {
    return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false));
}

// Sum over each sixteen lanes, in every one of them: pairs, fours, then the
// mirrored halves.  Register moves within the vector unit; shuffles through
// LDS took 0.4 us a sum longer.
__device__ __forceinline__ float sum16(float v) {
    v = add_lane<0xB1>(v);       // quad_perm 1 0 3 2
    v = add_lane<0x4E>(v);       // quad_perm 2 3 0 1
    v = add_lane<0x141>(v);      // row_half_mirror
    return add_lane<0x140>(v);   // row_mirror
}

// Sum of v over a row's threads, the same value in each.  `slot` names the
// call: calls that follow each other use different places, so one barrier
// each.
template <bool WAVE>
__device__ __forceinline__ float row_sum(float v, float (*part)[16], int slot) {
    v = sum16(v);
    const auto lane_value = [&](int l) {
        return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l));
    };
    v = (lane_value(0) + lane_value(16)) + (lane_value(32) + lane_value(48));
    if constexpr (!WAVE) {
        if ((threadIdx.x & 63) == 0) part[slot][threadIdx.x >> 6] = v;
        __syncthreads();
        const int w = threadIdx.x & 15;   // a wavefront's sum a lane, at most sixteen
        v = sum16(w < (int)(blockDim.x >> 6) ? part[slot][w] : 0.0f);
    }
    return v;
}

// Everything a thread holds of a row and where it is: CH runs, and with ODD
// one element more.
template <int CH, bool ODD>
struct Mine {
    int run0, step;       // element of the first run, distance of the runs
    int full, D;          // D rounded down to a multiple of eight
    int odd_at;           // the odd element
    bool has_odd;

    __device__ __forceinline__ int at(int c) const { return run0 + c * step; }
    __device__ __forceinline__ bool in(int c) const { return at(c) < full; }
    // where to load from: threads behind the last run read it again
    __device__ __forceinline__ int from(int c) const { return min(at(c), full - 8); }
    __device__ __forceinline__ int odd_from() const { return min(odd_at, D - 1); }
};

template <int CH>
struct Values {
    float v[CH][8];
    float odd[1];

    // zero what is not the row's (most wavefronts have nothing of the kind)
    template <bool ODD>
    __device__ __forceinline__ void clear_outside(const Mine<CH, ODD>& my) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
            if (!my.in(c)) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[c][i] = 0.0f;
            }
        if (ODD && !my.has_odd) odd[0] = 0.0f;
    }
};

// v <- (v - c) / sqrt(mean((v - c)^2) + eps) over the row.  What lies outside
// the row has to be zero on entry, and does not count.
template <bool WAVE, int CH, bool ODD>
__device__ __forceinline__ void normalize(Values<CH>& x, const Mine<CH, ODD>& my, const sgemv_norm& a,
                                          float (*part)[16], int slot) {
    const float inv_d = 1.0f / (float)a.D;
    if (a.flags & SGEMV_NORM_CENTER) {
        float s = ODD ? x.odd[0] : 0.0f;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) s += x.v[c][i];
        const float mean = row_sum<WAVE>(s, part, slot) * inv_d;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const float m = my.in(c) ? mean : 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) x.v[c][i] -= m;
        }
        if (ODD && my.has_odd) x.odd[0] -= mean;
    }
    float q = ODD ? x.odd[0] * x.odd[0] : 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) q = fmaf(x.v[c][i], x.v[c][i], q);
    const float inv = 1.0f / sqrtf(row_sum<WAVE>(q, part, slot + 1) * inv_d + a.eps);
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) x.v[c][i] *= inv;
    if (ODD) x.odd[0] *= inv;
}

// A weight and a bias of N elements.
template <int N>
struct Affine {
    RawAny<N> w, b;
    __device__ __forceinline__ void load(const void* pw, const void* pb, int type, int64_t at) {
        w.load(pw, type, at);
        b.load(pb, type, at);
    }
    __device__ __forceinline__ void apply(float (&v)[N], const void* pw, const void* pb, const sgemv_norm& a) const {
        float t[N];
        if (pw) {
            w.get(a.w_type, t);
            const float one = (a.flags & SGEMV_NORM_PLUS_ONE) ? 1.0f : 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] *= t[i] + one;
        }
        if (pb) {
            b.get(a.w_type, t);
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += t[i];
        }
    }
};

// A row's threads (a wavefront with WAVE, four rows a workgroup; a workgroup
// otherwise) own CH runs each.  RB, YB: bytes of an element of the residual
// and of y.  ODD: D is no multiple of eight.  A thread with one run loads all
// that it will need at once, so that a lone row waits for memory once; one
// with many loads what it has registers for.
template <bool WAVE, int CH, int RB, int YB, bool ODD>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void k_norm(sgemv_norm a) {
    __shared__ float part[4][16];
    constexpr bool kAll = CH == 1, kBoth = CH <= 2;   // every vector, or the residual beside y, loaded up front
    // The vectors of a later step: all runs' at once where there are registers for them (2048 x 28672: 105 us instead
    // of 119), otherwise run by run, and where the registers are full nothing is moved ahead of its run.  (With two
    // runs a thread fewer registers leave room for more rows: 777 x 5001 14.1 us run by run, 16.8 at once.)
    constexpr bool kTogether = CH == 4 && !ODD, kFenced = CH > 2 && !kTogether;
    const int tid = WAVE ? threadIdx.x & 63 : threadIdx.x;
    const int64_t row = WAVE ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : (int64_t)blockIdx.x;
    if (WAVE && row >= a.rows) return;   // no barrier follows with WAVE
    Mine<CH, ODD> my;
    my.run0 = tid * 8;
    my.step = (WAVE ? 64 : blockDim.x) * 8;
    my.D = a.D;
    my.full = a.D & ~7;
    my.odd_at = my.full + tid;
    my.has_odd = ODD && my.odd_at < a.D;
    const int64_t rrow = row * a.ld_residual, yrow = row * a.ld_y, grow = row * a.ld_gate;
    const int64_t orow = row * a.ld_residual_out, xrow = row * a.ld_x;

    Raw<RB, 8> rr[CH];
    Raw<YB, 8> yr[CH], gr[CH];
    Affine<8> post[kTogether ? CH : 1], pre[kTogether ? CH : 1];
    Raw<RB, 1> rr1;
    Raw<YB, 1> yr1, gr1;
    Affine<1> post1, pre1;
    if (!ODD || my.full) {   // a row of fewer than eight has no run
        if (a.y) {
#pragma unroll
            for (int c = 0; c < CH; ++c) yr[c].load(a.y, yrow + my.from(c));
        }
        if (kBoth || !a.y) {
#pragma unroll
            for (int c = 0; c < CH; ++c) rr[c].load(a.residual, rrow + my.from(c));
        }
        if (kBoth && a.gate) {
#pragma unroll
            for (int c = 0; c < CH; ++c) gr[c].load(a.gate, grow + my.from(c));
        }
        if (kAll) {
            post[0].load(a.post_weight, a.post_bias, a.w_type, my.from(0));
            pre[0].load(a.weight, a.bias, a.w_type, my.from(0));
        }
    }
    if (ODD) {
        if (a.y) yr1.load(a.y, yrow + my.odd_from());
        rr1.load(a.residual, rrow + my.odd_from());
        if (a.gate) gr1.load(a.gate, grow + my.odd_from());
        post1.load(a.post_weight, a.post_bias, a.w_type, my.odd_from());
        pre1.load(a.weight, a.bias, a.w_type, my.odd_from());
    }

    Values<CH> r;
    if (a.y) {
#pragma unroll
        for (int c = 0; c < CH; ++c) yr[c].get(a.y_type, r.v[c]);
        if (ODD) yr1.get(a.y_type, r.odd);
        if (a.flags & SGEMV_NORM_POST) {
            r.clear_outside(my);
            normalize<WAVE, CH, ODD>(r, my, a, part, 0);
            if (kTogether) {
#pragma unroll
                for (int c = 0; c < CH; ++c) post[c].load(a.post_weight, a.post_bias, a.w_type, my.from(c));
            }
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                if (kFenced) asm volatile("" ::: "memory");
                if (!kAll && !kTogether) post[0].load(a.post_weight, a.post_bias, a.w_type, my.from(c));
                post[kTogether ? c : 0].apply(r.v[c], a.post_weight, a.post_bias, a);
            }
            if (ODD) post1.apply(r.odd, a.post_weight, a.post_bias, a);
        }
        if (kTogether) {
#pragma unroll
            for (int c = 0; c < CH; ++c) rr[c].load(a.residual, rrow + my.from(c));
            if (a.gate) {
#pragma unroll
                for (int c = 0; c < CH; ++c) gr[c].load(a.gate, grow + my.from(c));
            }
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            if (kFenced) {
                asm volatile("" ::: "memory");
                rr[c].load(a.residual, rrow + my.from(c));
                if (a.gate) gr[c].load(a.gate, grow + my.from(c));
            }
            float t[8];
            if (a.gate) {
                gr[c].get(a.y_type, t);
#pragma unroll
                for (int i = 0; i < 8; ++i) r.v[c][i] *= t[i];
            }
            rr[c].get(a.residual_type, t);
#pragma unroll
            for (int i = 0; i < 8; ++i) r.v[c][i] = fmaf(a.scale, r.v[c][i], t[i]);
        }
        if (ODD) {
            float t[1];
            if (a.gate) {
                gr1.get(a.y_type, t);
                r.odd[0] *= t[0];
            }
            rr1.get(a.residual_type, t);
            r.odd[0] = fmaf(a.scale, r.odd[0], t[0]);
        }
    } else {
#pragma unroll
        for (int c = 0; c < CH; ++c) rr[c].get(a.residual_type, r.v[c]);
        if (ODD) rr1.get(a.residual_type, r.odd);
    }
    if (a.residual_out) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
            if (my.in(c)) store(a.residual_out, a.residual_type, orow + my.at(c), r.v[c]);
        if (ODD && my.has_odd) store(a.residual_out, a.residual_type, orow + my.odd_at, r.odd);
    }
    r.clear_outside(my);
    normalize<WAVE, CH, ODD>(r, my, a, part, 2);
    if (kTogether) {
#pragma unroll
        for (int c = 0; c < CH; ++c) pre[c].load(a.weight, a.bias, a.w_type, my.from(c));
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        if (my.in(c)) {
            if (kFenced) asm volatile("" ::: "memory");
            if (!kAll && !kTogether) pre[0].load(a.weight, a.bias, a.w_type, my.at(c));
            pre[kTogether ? c : 0].apply(r.v[c], a.weight, a.bias, a);
            store(a.x, a.x_type, xrow + my.at(c), r.v[c]);
        }
    }
    if (ODD && my.has_odd) {
        pre1.apply(r.odd, a.weight, a.bias, a);
        store(a.x, a.x_type, xrow + my.odd_at, r.odd);
    }
}

typedef void (*Kernel)(sgemv_norm);

template <bool WAVE, int CH, bool ODD>
Kernel pick_types(int RB, int YB) {
    if (RB == 2) return YB == 2 ? k_norm<WAVE, CH, 2, 2, ODD> : k_norm<WAVE, CH, 2, 4, ODD>;
    return YB == 2 ? k_norm<WAVE, CH, 4, 2, ODD> : k_norm<WAVE, CH, 4, 4, ODD>;
}

template <bool WAVE, int CH>
Kernel pick(int RB, int YB, bool odd) {
    return odd ? pick_types<WAVE, CH, true>(RB, YB) : pick_types<WAVE, CH, false>(RB, YB);
}

int size_of(int type) { return type == SGEMV_F32 ? 4 : 2; }
bool type_ok(int type) { return type >= SGEMV_F16 && type <= SGEMV_F32; }
bool aligned_to(const void* p, int a) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(a - 1)) == 0; }

// Whether an output shares bytes with another buffer otherwise than by taking
// its place whole, where that is allowed.
bool clash(const SgemvRows& out, const SgemvRows& b, bool may_replace) {
    if (may_replace && out.p == b.p && out.len == b.len && (out.rows == 1 || out.step == b.step)) return false;
    return sgemv_overlap(out, b);
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

    const auto rows_of = [&](const void* p, int64_t rows, int64_t ld, int size) {
        return SgemvRows{p, rows, ld * size, (int64_t)a.D * size};
    };
    const SgemvRows outs[2] = {rows_of(a.x, a.rows, a.ld_x, xb), rows_of(a.residual_out, a.rows, a.ld_residual_out, rb)};
    if (sgemv_overlap(outs[0], outs[1])) return SGEMV_EINVAL;
    for (const SgemvRows& o : outs)
        if (clash(o, rows_of(a.residual, a.rows, a.ld_residual, rb), true) ||
            clash(o, rows_of(a.y, a.rows, a.ld_y, yb), true) ||
            clash(o, rows_of(a.gate, a.ld_gate ? a.rows : 1, a.ld_gate, yb), a.ld_gate != 0) ||
            clash(o, rows_of(a.post_weight, 1, 0, wb), false) || clash(o, rows_of(a.post_bias, 1, 0, wb), false) ||
            clash(o, rows_of(a.weight, 1, 0, wb), false) || clash(o, rows_of(a.bias, 1, 0, wb), false))
            return SGEMV_EINVAL;

    const bool odd = a.D % 8 != 0;
    const int runs = a.D / 8;
    Kernel k;
    unsigned block = 256, rows_per = 1;
    if (runs <= 64) {
        k = pick<true, 1>(rb, yb, odd);
        rows_per = 4;
    } else {
        // Runs a thread.  One is fastest for a few rows, where only latency counts (16 x 5001: 4.8 us, 5.7 with two;
        // 16 x 14336, too long for one: 5.7 with two, 7.4 with four); many long rows want several runs in flight a
        // thread and room for more rows on a compute unit (8192 x 8192: 104 us with two runs, 112 with one, 115 with
        // four; 512 x 14336: 13.2 us with four, 16.8 with two).
        int CH = 1;
        if (runs > 1024 || (runs > 512 && a.rows > 256) || (runs > 256 && a.rows > 512)) CH = 2;
        if (runs > 2048 || (runs > 1024 && a.rows > 256)) CH = 4;
        if (runs > 4096) CH = 8;
        block = (unsigned)((runs + CH * 64 - 1) / (CH * 64) * 64);
        k = CH == 1   ? pick<false, 1>(rb, yb, odd)
            : CH == 2 ? pick<false, 2>(rb, yb, odd)
            : CH == 4 ? pick<false, 4>(rb, yb, odd)
                      : pick<false, 8>(rb, yb, odd);
    }
    // A launch has fewer than 2^32 threads: many rows take several, of 2^21 rows each.
    const int64_t all = a.rows, most = (int64_t)1 << 21;
    const auto advance = [&](const void* p, int64_t ld, int size) -> const void* {
        return p ? static_cast<const uint8_t*>(p) + most * ld * size : nullptr;
    };
    for (int64_t done = 0; done < all; done += most) {
        a.rows = all - done < most ? all - done : most;
        void* kargs[] = {&a};
        const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(k),
                                             dim3((unsigned)((a.rows + rows_per - 1) / rows_per)), dim3(block), kargs, 0,
                                             static_cast<hipStream_t>(stream));
        if (e != hipSuccess) return sgemv_hip_failed((int)e);
        a.residual = advance(a.residual, a.ld_residual, rb);
        a.y = advance(a.y, a.ld_y, yb);
        a.gate = advance(a.gate, a.ld_gate, yb);
        a.residual_out = const_cast<void*>(advance(a.residual_out, a.ld_residual_out, rb));
        a.x = const_cast<void*>(advance(a.x, a.ld_x, xb));
    }
    return SGEMV_OK;
}
