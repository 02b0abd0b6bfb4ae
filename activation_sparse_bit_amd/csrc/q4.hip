// 4-bit products that read every weight: sgemv_q4_run, sgemv_q4_run_gated.
//
//   y[m][n] = sum over groups g of s[n][g] * sum_{k in g} (q[n][k] - z[n][g]) x[m][k]
//
// Everything runs on the matrix cores, for one row as for sixteen: the codes
// of 16 outputs and 32 inputs are one operand of v_mfma_f32_16x16x32, the
// activations of up to 16 rows the other, so the vector units only unpack
// codes (about nine instructions for eight weights) and scale one sum per
// group, output and row.  A lane of the weight operand holds eight inputs of
// one output, and a lane of the result holds that same output, so a lane
// needs the scale and the zero-point of one output only.
//
// Row m of x is row (m % 4) * 4 + m / 4 of its operand: result register i of
// a lane then is row lane / 16 + 4 i, and with at most four rows only the
// first of the four result registers is scaled and summed.
//
// fp16 activations: codes become exact fp16 integers q - z (bits 0x6400 | q
// are 1024 + q, and (1024 + 16 q) / 16 - 64 for the upper nibbles).  bf16
// activations: bits 0x4180 | q << 3 are 16 + q, and the group's sum loses
// (16 + z) * sum x afterwards, sum x being one more matrix product with ones.
//
// A workgroup owns whole outputs: its wavefronts split the inputs, keep
// their sums in registers, and add them over LDS in wavefront order, so there
// is nothing to hand from one workgroup to another and the result does not
// depend on timing.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "internal.h"

namespace {

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf8_t __attribute__((ext_vector_type(8)));
typedef float float4_t __attribute__((ext_vector_type(4)));
typedef uint32_t uint4_t __attribute__((ext_vector_type(4)));
typedef uint32_t uint4_u __attribute__((ext_vector_type(4), aligned(2)));   // 16 bytes at any element

constexpr int kTileN = 16;
constexpr int kBlockK = 128;

struct Q4Args {
    const uint8_t* w;    // codes
    const uint8_t* s;    // scales
    const uint8_t* z;    // zero-points (NULL: 8)
    const uint16_t* x;
    const uint16_t* bias[2];
    void* y;
    int64_t ldx, ldy;
    int32_t N, K, M;
    int32_t tiles;       // tiles of 16 matrix rows (gate and up counted apart)
    int32_t blocks;      // blocks of 128 inputs
    int32_t gated, act;
    int32_t x_bf16, y_f32, s_bf16;
};

__device__ __forceinline__ float bf16_f32(uint32_t b) { return __builtin_bit_cast(float, b << 16); }
__device__ __forceinline__ float f16_f32(uint32_t b) { return (float)__builtin_bit_cast(_Float16, (uint16_t)b); }

// Eight inputs of one activation row from k0 on, zero beyond K.
__device__ __forceinline__ uint4_t load_x(const uint16_t* row, int k0, int K) {
    uint4_t v = {0, 0, 0, 0};
    if (k0 + 8 <= K) {
        v = *reinterpret_cast<const uint4_u*>(row + k0);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (k0 + i < K) v[i >> 1] |= (uint32_t)row[k0 + i] << (16 * (i & 1));
    }
    return v;
}

// One word of eight codes as the fp16 integers q - z; zl is 1024 + z and zh
// is 64 + z, twice each.
__device__ __forceinline__ half8_t unpack_f16(uint32_t w, half2_t zl, half2_t zh) {
    const half2_t sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f};
    half2_t p[4];
    p[0] = __builtin_bit_cast(half2_t, (w & 0x000F000Fu) | 0x64006400u) - zl;
    p[1] = __builtin_elementwise_fma(__builtin_bit_cast(half2_t, (w & 0x00F000F0u) | 0x64006400u), sixteenth, -zh);
    w >>= 8;
    p[2] = __builtin_bit_cast(half2_t, (w & 0x000F000Fu) | 0x64006400u) - zl;
    p[3] = __builtin_elementwise_fma(__builtin_bit_cast(half2_t, (w & 0x00F000F0u) | 0x64006400u), sixteenth, -zh);
    return half8_t{p[0][0], p[0][1], p[1][0], p[1][1], p[2][0], p[2][1], p[3][0], p[3][1]};
}

// The same as the bf16 integers q + 16.
__device__ __forceinline__ bf8_t unpack_bf16(uint32_t w) {
    uint4_t v;
    v[0] = ((w << 3) & 0x00780078u) | 0x41804180u;
    v[1] = ((w >> 1) & 0x00780078u) | 0x41804180u;
    v[2] = ((w >> 5) & 0x00780078u) | 0x41804180u;
    v[3] = ((w >> 9) & 0x00780078u) | 0x41804180u;
    return __builtin_bit_cast(bf8_t, v);
}

__device__ __forceinline__ float gate_of(float v, int act) {
    if (act == SGEMV_ACT_SILU) return v / (1.0f + expf(-v));
    if (act == SGEMV_ACT_GELU) return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
    return v < 0.0f ? 0.0f : v;   // a NaN stays
}

// BF: bf16 activations.  NT: tiles per workgroup (even when gated: a gate
// tile, then its up tile).  MR: result registers in use, ceil(M / 4).
// P: groups per block of 128 inputs.
template <bool BF, int NT, int MR, int P>
__global__ __launch_bounds__(1024) void k_q4(Q4Args a) {
    extern __shared__ float red[];   // [wavefront][NT][MR][64]
    const int lane = threadIdx.x & 63;
    const int wave = threadIdx.x >> 6;
    const int waves = blockDim.x >> 6;
    const int n16 = lane & 15;
    const int c = lane >> 4;
    const int row = (n16 >> 2) + (n16 & 3) * 4;   // the activation row this lane feeds
    const int tile0 = blockIdx.x * NT;
    const uint16_t* xrow = a.x + (int64_t)row * a.ldx;
    const bool feeds = row < a.M;

    int cell[NT];   // first cell of each tile (a tile past the end rereads the last one)
#pragma unroll
    for (int t = 0; t < NT; ++t) cell[t] = min(tile0 + t, a.tiles - 1) * a.blocks;

    float sum[NT][MR];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < MR; ++i) sum[t][i] = 0.0f;

    for (int b = wave; b < a.blocks; b += waves) {
        uint4_t x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[j] = uint4_t{0, 0, 0, 0};
            if (feeds) x[j] = load_x(xrow, b * kBlockK + 32 * j + 8 * c, a.K);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int64_t cl = cell[t] + b;
            const uint4_t w = reinterpret_cast<const uint4_t*>(a.w + cl * 1024)[lane];
            const int64_t sx = (cl * kTileN + n16) * P;   // scale index of this lane's first group
#pragma unroll
            for (int g = 0; g < P; ++g) {
                const uint32_t sb = reinterpret_cast<const uint16_t*>(a.s)[sx + g];
                const float s = a.s_bf16 ? bf16_f32(sb) : f16_f32(sb);
                uint32_t z = 8;
                if (a.z) z = (a.z[(sx + g) >> 1] >> (((sx + g) & 1) * 4)) & 15u;
                float4_t acc = {0, 0, 0, 0};
                if constexpr (BF) {
                    float4_t ones = {0, 0, 0, 0};
                    const uint4_t one = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
#pragma unroll
                    for (int j = g * 4 / P; j < (g + 1) * 4 / P; ++j) {
                        const bf8_t xv = __builtin_bit_cast(bf8_t, x[j]);
                        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv, unpack_bf16(w[j]), acc, 0, 0, 0);
                        ones = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv, __builtin_bit_cast(bf8_t, one), ones, 0, 0, 0);
                    }
                    const float off = -(float)(16u + z);
#pragma unroll
                    for (int i = 0; i < MR; ++i) sum[t][i] = fmaf(s, fmaf(off, ones[i], acc[i]), sum[t][i]);
                } else {
                    const half2_t zl = __builtin_bit_cast(half2_t, (0x6400u | z) * 0x10001u);   // 1024 + z
                    const half2_t zh = zl - half2_t{(_Float16)960.0f, (_Float16)960.0f};        // 64 + z
#pragma unroll
                    for (int j = g * 4 / P; j < (g + 1) * 4 / P; ++j)
                        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, x[j]),
                                                                     unpack_f16(w[j], zl, zh), acc, 0, 0, 0);
#pragma unroll
                    for (int i = 0; i < MR; ++i) sum[t][i] = fmaf(s, acc[i], sum[t][i]);
                }
            }
        }
    }

#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < MR; ++i) red[((wave * NT + t) * MR + i) * 64 + lane] = sum[t][i];
    __syncthreads();

    const int per_wave = NT * MR * 64;
    const int outs = a.gated ? per_wave / 2 : per_wave;
    for (int o = threadIdx.x; o < outs; o += blockDim.x) {
        const int l = o & 63, i = (o >> 6) % MR, t = (o >> 6) / MR;
        const int m = (l >> 4) + 4 * i;
        const int tile = a.gated ? (tile0 >> 1) + t : tile0 + t;   // tile of the output
        const int n = tile * kTileN + (l & 15);
        if (m >= a.M || n >= a.N) continue;
        float v[2];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            v[p] = 0.0f;
            if (p && !a.gated) break;
            const float* src = red + (((a.gated ? 2 * t + p : t) * MR + i) * 64 + l);
            for (int w = 0; w < waves; ++w) v[p] += src[w * per_wave];
            if (a.bias[p]) v[p] += BF ? bf16_f32(a.bias[p][n]) : f16_f32(a.bias[p][n]);
        }
        const float r = a.gated ? gate_of(v[0], a.act) * v[1] : v[0];
        const int64_t at = (int64_t)m * a.ldy + n;
        if (a.y_f32) static_cast<float*>(a.y)[at] = r;
        else if constexpr (BF) static_cast<__bf16*>(a.y)[at] = (__bf16)r;
        else static_cast<_Float16*>(a.y)[at] = (_Float16)r;
    }
}

typedef void (*Kernel)(Q4Args);

template <bool BF, int NT, int MR>
Kernel pick_p(int P) {
    return P == 1 ? k_q4<BF, NT, MR, 1> : P == 2 ? k_q4<BF, NT, MR, 2> : k_q4<BF, NT, MR, 4>;
}

template <bool BF, int NT>
Kernel pick_mr(int MR, int P) {
    return MR == 1 ? pick_p<BF, NT, 1>(P) : MR == 2 ? pick_p<BF, NT, 2>(P) : pick_p<BF, NT, 4>(P);
}

bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int run(const sgemv_q4_desc* d, const void* packed, const void* x, int x_type, int M, int ldx, const void* bias0,
        const void* bias1, int act, void* y, int y_type, int ldy, bool gated, void* stream) {
    if (!d || !packed || !x || !y) return SGEMV_EINVAL;
    const int st = sgemv_q4_check_desc(d);
    if (st) return st;
    if (((d->flags & SGEMV_Q4_GATED) != 0) != gated) return SGEMV_EINVAL;
    if (x_type != SGEMV_F16 && x_type != SGEMV_BF16) return SGEMV_EINVAL;
    if (y_type != x_type && y_type != SGEMV_F32) return SGEMV_EINVAL;
    if (act < SGEMV_ACT_SILU || act > SGEMV_ACT_RELU) return SGEMV_EINVAL;
    if (M < 1 || M > SGEMV_MAX_BATCH || ldx < d->K || ldy < d->N) return SGEMV_ESIZE;
    if (!aligned_to(packed, 256) || !aligned_to(x, 2) || !aligned_to(y, y_type == SGEMV_F32 ? 4 : 2) ||
        !aligned_to(bias0, 2) || !aligned_to(bias1, 2))
        return SGEMV_EALIGN;

    const uint8_t* blob = static_cast<const uint8_t*>(packed);
    Q4Args a;
    std::memset(&a, 0, sizeof a);
    a.w = blob + d->w_off;
    a.s = blob + d->s_off;
    a.z = (d->flags & SGEMV_Q4_ZEROS) ? blob + d->z_off : nullptr;
    a.x = static_cast<const uint16_t*>(x);
    a.bias[0] = static_cast<const uint16_t*>(bias0);
    a.bias[1] = static_cast<const uint16_t*>(bias1);
    a.y = y;
    a.ldx = ldx;
    a.ldy = ldy;
    a.N = d->N;
    a.K = d->K;
    a.M = M;
    a.tiles = (d->N + kTileN - 1) / kTileN * (gated ? 2 : 1);
    a.blocks = (d->K + kBlockK - 1) / kBlockK;
    a.gated = gated;
    a.act = act;
    a.x_bf16 = x_type == SGEMV_BF16;
    a.y_f32 = y_type == SGEMV_F32;
    a.s_bf16 = (d->flags & SGEMV_Q4_BF16_SCALES) != 0;

    const int NT = gated ? 2 : 1;
    const int MR = M <= 4 ? 1 : M <= 8 ? 2 : 4;
    const int P = kBlockK / d->group;
    int waves = 4;
    while (waves > 1 && waves > a.blocks) waves /= 2;
    Kernel k;
    if (a.x_bf16) k = NT == 1 ? pick_mr<true, 1>(MR, P) : pick_mr<true, 2>(MR, P);
    else k = NT == 1 ? pick_mr<false, 1>(MR, P) : pick_mr<false, 2>(MR, P);
    const size_t lds = (size_t)waves * NT * MR * 64 * sizeof(float);
    void* args[] = {&a};
    const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(k), dim3((a.tiles + NT - 1) / NT),
                                         dim3(waves * 64), args, lds, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? SGEMV_OK : sgemv_hip_failed((int)e);
}

}  // namespace

extern "C" int sgemv_q4_run(const sgemv_q4_desc* d, const void* packed, const void* x, int32_t x_type, int32_t M,
                            int32_t ldx, const void* bias, void* y, int32_t y_type, int32_t ldy, void* stream) {
    return run(d, packed, x, x_type, M, ldx, bias, nullptr, SGEMV_ACT_SILU, y, y_type, ldy, false, stream);
}

extern "C" int sgemv_q4_run_gated(const sgemv_q4_desc* d, const void* packed, const void* x, int32_t x_type,
                                  int32_t M, int32_t ldx, const void* bias_gate, const void* bias_up, int32_t act,
                                  void* h, int32_t h_type, int32_t ldh, void* stream) {
    return run(d, packed, x, x_type, M, ldx, bias_gate, bias_up, act, h, h_type, ldh, true, stream);
}
