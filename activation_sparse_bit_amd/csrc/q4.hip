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
// Up to four rows: operand row 4 r + j holds row r's inputs of step j, so one
// 16-byte load a lane brings what four steps need; step j's products are read
// from result register j.  Up to eight rows two steps share a load, up to
// sixteen each step has its own.  Activations are read in row order and put
// into operand order through the wavefront's own LDS: loaded directly, the 64
// lanes of a load would touch 64 pieces in 16 lines (28672 x 8192 gated, 16
// rows: 62 us instead of 58).
//
// fp16 activations: codes become exact fp16 integers q - z (bits 0x6400 | q
// are 1024 + q, and (1024 + 16 q) / 16 - 64 for the upper nibbles).  bf16
// activations: bits 0x4180 | q << 3 are 16 + q, and the group's sum loses
// (16 + z) * sum x afterwards, sum x being one more matrix product with ones.
// Where that leaves fp32 (an infinity in x, or 31 times a value), a wavefront
// goes over its inputs again with exact bf16 integers q - z, for the sums
// concerned only.
//
// A workgroup owns whole outputs: its wavefronts split the inputs, keep
// their sums in registers, and add them over LDS in wavefront order, so there
// is nothing to hand from one workgroup to another and the result does not
// depend on timing.
//
// Bound by HBM where the matrix is large: 100003 x 4096 (four rows, 219 MB) in
// 35 to 42 us, 5.2 to 6.2 TB/s, the vector units 66 to 80 % busy; 28672 x 8192
// gated (16 rows, 251 MB) in 50 to 52 us.  With sixteen rows the L2 counts too:
// 8192 x 28672 (123 MB) in 32 us, its activations read 256 times (235 MB).  A
// matrix that stays in the 256 MB cache is read from there, and then its start
// and end count: 4096 x 14336 takes 7.4 us warm and 10.8 cold, 14336 x 4096
// gated 12.3 and 14.7.  A small one (2048 x 2048, 2.6 us warm, 4.0 cold) is
// launch and latency.  Many resident wavefronts hide the latency, not
// prefetching: two blocks in flight a wavefront cost registers and gained 3 % at
// most.
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
    const uint8_t* z;    // zero-points, z_stride bytes a cell
    const uint16_t* x;
    const uint16_t* bias[2];
    void* y;
    int64_t ldx, ldy;
    int32_t N, K, M;
    int32_t tiles;       // tiles of 16 matrix rows (gate and up counted apart)
    int32_t blocks;      // blocks of 128 inputs
    int32_t gated, act;
    int32_t x_bf16, y_f32, s_bf16;
    uint32_t z_stride;   // 0: no zero-points, all 8
};

__device__ __forceinline__ float bf16_f32(uint32_t b) { return __builtin_bit_cast(float, b << 16); }
__device__ __forceinline__ float f16_f32(uint32_t b) { return (float)__builtin_bit_cast(_Float16, (uint16_t)b); }

// Masks and exponents of the unpacking, in registers that the compiler takes
// as unknown: with literals it emits an AND and an OR where one v_and_or_b32
// does (a third of the unpacking).
template <bool Z_IN_VECTOR>
struct Unpack {
    uint32_t lo, hi, exp, z_mask, z_exp;   // codes; zero-points: without any, the mask is 0 and the 8 in z_exp
    __device__ __forceinline__ Unpack(bool bf, bool zeros)
        : lo(bf ? 0x00780078u : 0x000F000Fu), hi(0x00F000F0u), exp(bf ? 0x41804180u : 0x64006400u),
          z_mask(!zeros ? 0u : bf ? 15u << 19 : 15u),
          z_exp((bf ? 0x41800000u : 0x6400u) | (zeros ? 0u : bf ? 8u << 19 : 8u)) {
        asm("" : "+s"(lo));
        asm("" : "+s"(hi));
        asm("" : "+v"(exp));
        // one v_and_or_b32 for a zero-point too, where it shows: several groups a block, or bf16 (28672 x 8192 gated, 16
        // rows: 53.2 -> 51.4 us); with one group and fp16 the scalar form is as fast or faster (12.7 against 12.9)
        if constexpr (Z_IN_VECTOR) asm("" : "+v"(z_exp));
        else asm("" : "+s"(z_exp));
    }
};

// One word of eight codes as the fp16 integers q - z; zl is 1024 + z and zh
// is 64 + z, twice each.
template <class U>
__device__ __forceinline__ half8_t unpack_f16(const U& u, uint32_t w, half2_t zl, half2_t zh) {
    const half2_t sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f};
    half2_t p[4];
    p[0] = __builtin_bit_cast(half2_t, (w & u.lo) | u.exp) - zl;
    p[1] = __builtin_elementwise_fma(__builtin_bit_cast(half2_t, (w & u.hi) | u.exp), sixteenth, -zh);
    w >>= 8;
    p[2] = __builtin_bit_cast(half2_t, (w & u.lo) | u.exp) - zl;
    p[3] = __builtin_elementwise_fma(__builtin_bit_cast(half2_t, (w & u.hi) | u.exp), sixteenth, -zh);
    return half8_t{p[0][0], p[0][1], p[1][0], p[1][1], p[2][0], p[2][1], p[3][0], p[3][1]};
}

// The same as the bf16 integers q + 16.
template <class U>
__device__ __forceinline__ bf8_t unpack_bf16(const U& u, uint32_t w) {
    uint4_t v;
    v[0] = ((w << 3) & u.lo) | u.exp;
    v[1] = ((w >> 1) & u.lo) | u.exp;
    v[2] = ((w >> 5) & u.lo) | u.exp;
    v[3] = ((w >> 9) & u.lo) | u.exp;
    return __builtin_bit_cast(bf8_t, v);
}

__device__ __forceinline__ float gate_of(float v, int act) {
    if (act == SGEMV_ACT_SILU) {   // v / (1 + e^-v), below zero v e^v / (1 + e^v): e^-v is infinite from -88.7 on
        const float e = expf(-fabsf(v));
        return (v < 0.0f ? v * e : v) / (1.0f + e);
    }
    // erfc(-t) is 1 + erf(t) without its cancellation (at v = -5 the sum has lost 4 % of the value)
    if (act == SGEMV_ACT_GELU) return 0.5f * v * erfcf(v * -0.70710678118654752f);
    return v < 0.0f ? 0.0f : v;   // a NaN stays
}

// The scales of a lane's output in one block of 128 inputs (P of them) and
// their zero-points, as loaded: whole words, of which a lane takes its part
// when it uses them.  (Loads of 8 or 16 bits are widened by the compiler where
// they meet the loop, which waits for them there and leaves nothing in flight.)
template <int P>
struct Meta {
    typedef uint32_t words __attribute__((ext_vector_type(P == 4 ? 2 : 1)));
    words s;
    uint32_t z;
    // Without zero-points every lane rereads one line of the scales (stride 0): no branch, so that the number of
    // loads in flight is known where they are waited for.
    __device__ __forceinline__ void load(const Q4Args& a, int64_t cell, int n16) {
        s = reinterpret_cast<const words*>(a.s + cell * 32 * P)[P == 1 ? n16 >> 1 : n16];
        z = reinterpret_cast<const uint32_t*>(a.z + cell * a.z_stride)[n16 * P >> 3];
    }
    __device__ __forceinline__ float scale(int g, int n16, bool bf16) const {
        const uint32_t word = P == 4 ? s[g >> 1] : s[0];
        const uint32_t b = word >> (P == 1 ? (n16 & 1) * 16 : (g & 1) * 16);
        const float f = f16_f32(b & 0xFFFFu), h = bf16_f32(b);
        return bf16 ? h : f;
    }
    // The zero-point's nibble moved to bit `to` of the word.
    __device__ __forceinline__ uint32_t moved(int g, int n16, int to) const {
        const int at = (n16 * P & 7) * 4 + g * 4;
        return to ? __builtin_amdgcn_alignbit(z, z, (at - to) & 31) : z >> at;
    }
};

// A wavefront's share of one tile's sums from bf16 activations and the exact
// integers q - z, for sums that came out of the kernel's own way as no number
// or an infinity.  Operand row 4 c + i holds row MR c + i of x, so that a lane
// gets the outputs that it has there.  Rare, so its loop stays rolled: unrolled
// it would set the kernel's register count (50 -> 85) and with it how many
// wavefronts hide each other's loads.  8192 x 28672 with 16 rows takes 60 us
// with an infinity in one row, 125 with a row of NaN, 33 without.
template <int MR, int P>
__device__ __forceinline__ float4_t exact_sums(const Q4Args& a, int cell, int wave, int waves) {
    const int lane = threadIdx.x & 63, n16 = lane & 15, c = lane >> 4;
    const uint16_t* row = a.x + (int64_t)min((n16 >> 2) * MR + min(n16 & 3, MR - 1), a.M - 1) * a.ldx;
    float4_t sum = {0, 0, 0, 0};
#pragma unroll 1
    for (int step = wave * 4; step < a.blocks * 4; step += (step & 3) == 3 ? waves * 4 - 3 : 1) {
        const int64_t at = cell + (step >> 2);
        const int meta = n16 * P + (step & 3) * P / 4;   // the group's place in its cell
        const uint32_t w = reinterpret_cast<const uint32_t*>(a.w + at * 1024)[lane * 4 + (step & 3)];
        const uint32_t sb = reinterpret_cast<const uint16_t*>(a.s)[at * (kTileN * P) + meta];
        const uint32_t zb = a.z_stride ? a.z[at * a.z_stride + (meta >> 1)] >> (4 * (meta & 1)) & 15u : 8u;
        const float z = (float)zb;
        const int k0 = step * 32 + 8 * c;
        uint4_t x = {0, 0, 0, 0}, q;
        if (k0 + 8 <= a.K) {
            x = *reinterpret_cast<const uint4_u*>(row + k0);
        } else {
#pragma unroll 1
            for (int k = k0; k < k0 + 8; k += 2) {   // two inputs a turn, moved in from above
                const uint32_t lo = k < a.K ? row[k] : 0u, hi = k + 1 < a.K ? row[k + 1] : 0u;
                x = uint4_t{x[1], x[2], x[3], lo | hi << 16};
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // small integers: the lower half of their fp32 is zero
            const float q0 = (float)(w >> (4 * i) & 15u) - z, q1 = (float)(w >> (4 * i + 16) & 15u) - z;
            q[i] = __builtin_bit_cast(uint32_t, q0) >> 16 | __builtin_bit_cast(uint32_t, q1);
        }
        const float4_t zero = {0, 0, 0, 0};
        const float4_t d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8_t, x), __builtin_bit_cast(bf8_t, q),
                                                                   zero, 0, 0, 0);
        const float s = a.s_bf16 ? bf16_f32(sb) : f16_f32(sb);
#pragma unroll
        for (int i = 0; i < MR; ++i) {
            float v = fmaf(s, d[i], sum[i]);
            asm volatile("" : "+v"(v));   // consumed before the loop's branch, as in the kernel
            sum[i] = v;
        }
    }
    return sum;
}

// BF: bf16 activations.  NT: tiles per workgroup (even when gated: a gate
// tile, then its up tile).  MR: result registers in use: 1, 2, 4 for up to
// 4, 8, 16 rows.  P: groups per block of 128 inputs.  ST: codes are read past the
// caches.
template <bool BF, int NT, int MR, int P, bool ST>
__global__ __launch_bounds__(1024) void k_q4(Q4Args a) {
    constexpr int J = 4 / MR;   // steps that share an operand of activations
    extern __shared__ uint4_t lds[];   // MR * 64 for each wavefront: activations, then its sums [NT][MR][64]
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6;
    const int n16 = lane & 15;
    const int c = lane >> 4;
    const int tile0 = blockIdx.x * NT;
    // Load l of a block's activations: row 4 l + c, its inputs from 8 * n16 on (the last row again beyond M: those
    // results are not stored).
    const uint16_t* xlane[MR];
    uint4_t *put[MR], *get[MR];   // where this lane writes what it loads, and reads what it feeds
#pragma unroll
    for (int l = 0; l < MR; ++l) {
        const int r = 4 * l + c, j = n16 >> 2;
        xlane[l] = a.x + (int64_t)min(r, a.M - 1) * a.ldx + 8 * n16;
        put[l] = lds + wave * MR * 64 + r * 16 + ((J * (r + (n16 & 3) + 4 * (j / J)) + j % J) & 15);
        get[l] = lds + wave * MR * 64 + n16 / J * 16 + ((n16 + J * (c + 4 * l)) & 15);
    }

    int cell[NT];   // first cell of each tile (a tile past the end rereads the last one)
#pragma unroll
    for (int t = 0; t < NT; ++t) cell[t] = min(tile0 + t, a.tiles - 1) * a.blocks;

    float sum[NT][MR];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < MR; ++i) sum[t][i] = 0.0f;

    const auto fetch_weights = [&](uint4_t (&w)[NT], Meta<P> (&md)[NT], int b) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const uint4_t* from = reinterpret_cast<const uint4_t*>(a.w + (int64_t)(cell[t] + b) * 1024) + lane;
            if constexpr (ST) w[t] = __builtin_nontemporal_load(from);
            else w[t] = *from;
            md[t].load(a, cell[t] + b, n16);
        }
    };
    const Unpack<BF || (P > 1)> u(BF, a.z_stride != 0);
    const auto multiply = [&](const uint4_t (&w)[NT], const Meta<P> (&md)[NT], const uint4_t (&raw)[MR]) {
        // From rows to operands through the wavefront's own LDS (its accesses are in order; the fences hold the
        // compiler to it).
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int l = 0; l < MR; ++l) *put[l] = raw[l];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        uint4_t x[MR];
#pragma unroll
        for (int h = 0; h < MR; ++h) x[h] = *get[h];
#pragma unroll
        for (int g = 0; g < P; ++g) {
            constexpr int kSteps = 4 / P;                    // steps of a group
            constexpr int kPhases = kSteps < J ? kSteps : J;   // ... of different operand rows
            float ones[MR];   // BF: the group's sum of activations
            if constexpr (BF) {
                const uint4_t one = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
                float4_t o = {0, 0, 0, 0};
#pragma unroll
                for (int h = g * kSteps / J; h <= ((g + 1) * kSteps - 1) / J; ++h)
                    o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8_t, x[h]),
                                                                __builtin_bit_cast(bf8_t, one), o, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < MR; ++i) {
                    ones[i] = o[i * J + g * kSteps % J];
#pragma unroll
                    for (int q = 1; q < kPhases; ++q) ones[i] += o[i * J + (g * kSteps + q) % J];
                }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const float s = md[t].scale(g, n16, a.s_bf16);
                // 16 + z in fp32 for bf16 activations; 1024 + z and 64 + z in fp16, twice each, for fp16
                const uint32_t zb = (md[t].moved(g, n16, BF ? 19 : 0) & u.z_mask) | u.z_exp;
                const half2_t zl = __builtin_bit_cast(half2_t, zb << 16 | zb);
                const half2_t zh = zl - half2_t{(_Float16)960.0f, (_Float16)960.0f};
                float4_t acc[kPhases];
#pragma unroll
                for (int q = 0; q < kPhases; ++q) acc[q] = float4_t{0, 0, 0, 0};
#pragma unroll
                for (int e = 0; e < kSteps; ++e) {
                    const int j = g * kSteps + e;
                    float4_t& d = acc[e % kPhases];
                    if constexpr (BF)
                        d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8_t, x[j / J]),
                                                                    unpack_bf16(u, w[t][j]), d, 0, 0, 0);
                    else
                        d = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, x[j / J]),
                                                                   unpack_f16(u, w[t][j], zl, zh), d, 0, 0, 0);
                }
#pragma unroll
                for (int i = 0; i < MR; ++i) {
                    float v = acc[0][i * J + g * kSteps % J];
#pragma unroll
                    for (int q = 1; q < kPhases; ++q) v += acc[q][i * J + (g * kSteps + q) % J];
                    if constexpr (BF) v = fmaf(-__builtin_bit_cast(float, zb), ones[i], v);
                    sum[t][i] = fmaf(s, v, sum[t][i]);
                }
            }
        }
        // Consume the products here: moved behind a branch, the first read of a result can come too soon after the
        // matrix instruction (seen with this compiler: the last block's product was lost).
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < MR; ++i) asm volatile("" : "+v"(sum[t][i]));
    };

    const int full = a.K / kBlockK;
    uint4_t w[NT], raw[MR];
    Meta<P> md[NT];
    if (full < a.blocks && wave == full % waves) {   // the inputs behind the last full block
        fetch_weights(w, md, full);
        const int k0 = full * kBlockK + 8 * n16;
#pragma unroll
        for (int l = 0; l < MR; ++l) {
            const uint16_t* row = xlane[l] - 8 * n16;
            uint32_t e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = row[min(k0 + i, a.K - 1)];
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = k0 + i < a.K ? e[i] : 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) raw[l][i] = e[2 * i] | e[2 * i + 1] << 16;
        }
        multiply(w, md, raw);
    }
    // wavefront w multiplies blocks w, w + waves, ...: the workgroup reads
    // one contiguous run at a time
    for (int b = wave; b < full; b += waves) {
        fetch_weights(w, md, b);
#pragma unroll
        for (int l = 0; l < MR; ++l) raw[l] = *reinterpret_cast<const uint4_u*>(xlane[l] + b * kBlockK);
        multiply(w, md, raw);
    }

    // a wavefront's sums take the place of its activations
    float* red = reinterpret_cast<float*>(lds);
    constexpr int kStride = MR * 256;   // floats of a wavefront's LDS
    static_assert(NT * MR * 64 <= kStride, "sums fit");
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < MR; ++i) red[wave * kStride + (t * MR + i) * 64 + lane] = sum[t][i];
    if constexpr (BF) {
        bool left = false;   // fp32, for one of this lane's sums
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < MR; ++i) left |= !__builtin_isfinite(sum[t][i]);
        if (__any(left)) {
#pragma unroll 1
            for (int t = 0; t < NT; ++t) {
                const float4_t e = exact_sums<MR, P>(a, min(tile0 + t, a.tiles - 1) * a.blocks, wave, waves);
#pragma unroll
                for (int i = 0; i < MR; ++i) {
                    float& s = red[wave * kStride + (t * MR + i) * 64 + lane];
                    if (!__builtin_isfinite(s)) s = e[i];
                }
            }
        }
    }
    __syncthreads();

    const int per_wave = NT * MR * 64;
    const int outs = a.gated ? per_wave / 2 : per_wave;
    for (int o = threadIdx.x; o < outs; o += blockDim.x) {
        const int l = o & 63, i = (o >> 6) % MR, t = (o >> 6) / MR;
        const int m = (l >> 4) * MR + i;
        const int tile = a.gated ? (tile0 >> 1) + t : tile0 + t;   // tile of the output
        const int n = tile * kTileN + (l & 15);
        if (m >= a.M || n >= a.N) continue;
        float v[2];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            v[p] = 0.0f;
            if (p && !a.gated) break;
            const float* src = red + (((a.gated ? 2 * t + p : t) * MR + i) * 64 + l);
            for (int w = 0; w < waves; ++w) v[p] += src[w * kStride];
            if (a.bias[p]) v[p] += BF ? bf16_f32(a.bias[p][n]) : f16_f32(a.bias[p][n]);
        }
        const float r = a.gated ? gate_of(v[0], a.act) * v[1] : v[0];
        const int64_t at = (int64_t)m * a.ldy + n;
        if (a.y_f32) static_cast<float*>(a.y)[at] = r;
        else if constexpr (BF) static_cast<__bf16*>(a.y)[at] = (__bf16)r;
        else static_cast<_Float16*>(a.y)[at] = (_Float16)r;
    }
}

// ---------------------------------------------------------------------------
// packing on the device
// ---------------------------------------------------------------------------
struct PackArgs {
    const uint8_t* q[2];
    const uint16_t* s[2];
    const uint8_t* z[2];
    uint8_t* blob;
    sgemv_q4_desc d;
};

// Sixteen bytes of the blob: the codes of one lane in one cell, the header,
// or scales and zero-points.  Bound by reading a byte a code; rows are read
// in pieces of eight bytes, which the caches put together.
__device__ __forceinline__ void pack_16(const PackArgs& a, uint64_t id) {
    const uint64_t blocks = (a.d.K + kBlockK - 1) / kBlockK, parts = (a.d.flags & SGEMV_Q4_GATED) ? 2 : 1;
    const uint64_t slots = a.d.w_bytes / 16, P = kBlockK / a.d.group;
    const uint64_t N = a.d.N, K = a.d.K, G = (K + a.d.group - 1) / a.d.group;
    if (id < slots) {
        const uint64_t cell = id >> 6, r = id & 15, c = id >> 4 & 3;
        const uint64_t b = cell % blocks, tile = cell / blocks, n = tile / parts * kTileN + r;
        const uint8_t* row = a.q[tile % parts] + n * K;
        uint4_t out = {0, 0, 0, 0};
        if (n < N) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint64_t k0 = b * kBlockK + 32 * j + 8 * c;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (k0 + i < K) out[j] |= (uint32_t)(row[k0 + i] & 15) << (4 * ((i >> 1) + 4 * (i & 1)));
            }
        }
        reinterpret_cast<uint4_t*>(a.blob + a.d.w_off)[id] = out;
        return;
    }
    // the bytes outside the codes, 16 at a time: the header, then scales and zero-points up to the end
    const uint64_t rest = id - slots;
    const uint64_t at = rest < 16 ? rest * 16 : a.d.s_off + (rest - 16) * 16;
    if (at >= a.d.total_bytes) return;
    uint8_t byte[16];
    for (int i = 0; i < 16; ++i) {
        const uint64_t o = at + i;
        uint32_t v = 0;
        const auto index = [&](uint64_t m, uint64_t& n, uint64_t& g, uint64_t& part) {
            const uint64_t cell = m / (kTileN * P), tile = cell / blocks;
            n = tile / parts * kTileN + m / P % kTileN;
            g = cell % blocks * P + m % P;
            part = tile % parts;
            return n < N && g < G;
        };
        uint64_t n, g, part;
        if (o < 80) {
            const uint32_t word[20] = {0x31514753u, 1u, (uint32_t)a.d.N, (uint32_t)a.d.K, (uint32_t)a.d.group, a.d.flags,
                                       (uint32_t)a.d.w_off, (uint32_t)(a.d.w_off >> 32), (uint32_t)a.d.w_bytes,
                                       (uint32_t)(a.d.w_bytes >> 32), (uint32_t)a.d.s_off, (uint32_t)(a.d.s_off >> 32),
                                       (uint32_t)a.d.s_bytes, (uint32_t)(a.d.s_bytes >> 32), (uint32_t)a.d.z_off,
                                       (uint32_t)(a.d.z_off >> 32), (uint32_t)a.d.z_bytes, (uint32_t)(a.d.z_bytes >> 32),
                                       (uint32_t)a.d.total_bytes, (uint32_t)(a.d.total_bytes >> 32)};
            v = word[o >> 2] >> (8 * (o & 3));
        } else if (o >= a.d.s_off && o < a.d.s_off + a.d.s_bytes) {
            const uint64_t m = (o - a.d.s_off) >> 1;
            if (index(m, n, g, part)) v = a.s[part][n * G + g] >> (8 * (o & 1));
        } else if (o >= a.d.z_off && o < a.d.z_off + a.d.z_bytes) {
            const uint64_t m = (o - a.d.z_off) << 1;
            if (index(m, n, g, part)) v = a.z[part][n * G + g] & 15;
            if (index(m + 1, n, g, part)) v |= (uint32_t)(a.z[part][n * G + g] & 15) << 4;
        }
        byte[i] = (uint8_t)v;
    }
    for (int i = 0; i < 16; ++i) a.blob[at + i] = byte[i];
}

__global__ __launch_bounds__(256) void k_q4_pack(PackArgs a, uint64_t n) {
    for (uint64_t id = (uint64_t)blockIdx.x * 256 + threadIdx.x; id < n; id += (uint64_t)gridDim.x * 256) pack_16(a, id);
}

typedef void (*Kernel)(Q4Args);

template <bool BF, int NT, int MR, bool ST>
Kernel pick_p(int P) {
    return P == 1 ? k_q4<BF, NT, MR, 1, ST> : P == 2 ? k_q4<BF, NT, MR, 2, ST> : k_q4<BF, NT, MR, 4, ST>;
}

template <bool BF, int NT, bool ST>
Kernel pick_mr(int MR, int P) {
    return MR == 1 ? pick_p<BF, NT, 1, ST>(P) : MR == 2 ? pick_p<BF, NT, 2, ST>(P) : pick_p<BF, NT, 4, ST>(P);
}

template <bool BF>
Kernel pick(int NT, int MR, int P, bool streamed) {
    if (NT == 1) return pick_mr<BF, 1, false>(MR, P);
    if (NT == 2) return streamed ? pick_mr<BF, 2, true>(MR, P) : pick_mr<BF, 2, false>(MR, P);
    return streamed ? pick_p<BF, 4, 4, true>(P) : pick_p<BF, 4, 4, false>(P);
}

int launch(const Q4Args& a, Kernel k, int NT, int waves, hipStream_t stream) {
    const int MR = a.M <= 4 ? 1 : a.M <= 8 ? 2 : 4;
    const size_t lds = (size_t)waves * MR * 1024;
    Q4Args copy = a;
    void* args[] = {&copy};
    const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(k), dim3((a.tiles + NT - 1) / NT),
                                         dim3(waves * 64), args, lds, stream);
    return e == hipSuccess ? SGEMV_OK : sgemv_hip_failed((int)e);
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
    const int ys = y_type == SGEMV_F32 ? 4 : 2;
    const SgemvRows out{y, M, (int64_t)ldy * ys, (int64_t)d->N * ys};
    if (sgemv_overlap(out, {x, M, (int64_t)ldx * 2, (int64_t)d->K * 2}) ||
        sgemv_overlap(out, {packed, 1, 0, (int64_t)d->total_bytes}) ||
        sgemv_overlap(out, {bias0, 1, 0, (int64_t)d->N * 2}) || sgemv_overlap(out, {bias1, 1, 0, (int64_t)d->N * 2}))
        return SGEMV_EINVAL;

    const uint8_t* blob = static_cast<const uint8_t*>(packed);
    Q4Args a;
    std::memset(&a, 0, sizeof a);
    a.w = blob + d->w_off;
    a.s = blob + d->s_off;
    const bool zeros = (d->flags & SGEMV_Q4_ZEROS) != 0;
    a.z = zeros ? blob + d->z_off : a.s;
    a.z_stride = zeros ? kTileN / 2 * (kBlockK / d->group) : 0;
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

    const int MR = M <= 4 ? 1 : M <= 8 ? 2 : 4;
    // Tiles per workgroup.  More tiles share one reading of the activations, fewer leave no compute unit idle: below
    // 512 tiles one each (4096 x 14336: 7.3 us against 10.2 with two), from there two (8192 x 28672, eight rows: 26.7
    // against 31.9 with one), and with more than eight rows, whose activations weigh most, four from 1024 tiles on
    // (28672 x 8192, 16 rows: 29.4 against 34.5 with two).
    int NT = a.tiles < 512 ? 1 : MR == 4 && a.tiles >= 1024 ? 4 : 2;
    if (gated && NT == 1) NT = 2;
    // Wavefronts, which split the inputs: sixteen where the workgroups alone do not fill the card (4096 x 14336: 7.3 us
    // against 9.4 with eight; 28672 x 8192, one row, 896 workgroups: 23.8 against 25.3), eight otherwise
    // (14336 x 4096, 16 rows, gated: 13.8 against 15.3 with sixteen), four for many short rows
    // (100003 x 1024: 10.7 against 11.5 with eight).
    const int grid = (a.tiles + NT - 1) / NT;
    int waves = 8;
    if (MR == 4 ? grid <= 256 && a.blocks >= 32 : (grid <= 512 && a.blocks >= 32) || (grid <= 1024 && a.blocks >= 64))
        waves = 16;
    else if (a.blocks <= 8 && grid > 1024) waves = 4;
    while (waves > 1 && waves > a.blocks) waves /= 2;
    const int P = kBlockK / d->group;
    // A matrix that takes a good part of the 256 MB cache is gone from it before its next use: its codes are read past
    // the caches (warm, three matrices in turn: 100003 x 4096 42.0 -> 39.2 us, 28672 x 8192 gated, 16 rows, 56.9 -> 52.2;
    // cold, more than 600 MB in turn: 44.2 -> 41.4 and 62.2 -> 56.2).  Smaller ones may stay from one token to the next,
    // and reading past the caches would lose more then than it gains when they are cold: 4096 x 14336 7.4 -> 8.8 us warm,
    // 10.7 -> 10.2 cold; 8192 x 14336 12.1 -> 13.0 and 14.6 -> 14.0; 14336 x 4096 gated 12.8 -> 13.6 and 14.7 -> 14.3.
    // Workgroups of one tile read through the caches whatever the size (that many codes in fewer than 512 tiles take
    // more than 24000 inputs): 7168 x 28672 past the caches 22.1 -> 21.1 us warm, 26.4 -> 25.8 cold, 16 rows 44.2 -> 43.2
    // and 46.8 -> 42.2, not worth 18 more kernels.
    const bool streamed = d->w_bytes >= (96ull << 20);
    const Kernel k = a.x_bf16 ? pick<true>(NT, MR, P, streamed) : pick<false>(NT, MR, P, streamed);
    return launch(a, k, NT, waves, static_cast<hipStream_t>(stream));
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

extern "C" int sgemv_q4_pack_device(const uint8_t* q, const uint16_t* scales, const uint8_t* zeros, const uint8_t* q_up,
                                    const uint16_t* scales_up, const uint8_t* zeros_up, int32_t N, int32_t K,
                                    int32_t group, uint32_t flags, void* packed, size_t capacity,
                                    sgemv_q4_desc* desc_out, void* stream) {
    PackArgs a;
    std::memset(&a, 0, sizeof a);
    const bool gated = (flags & SGEMV_Q4_GATED) != 0, with_zeros = (flags & SGEMV_Q4_ZEROS) != 0;
    const int st = gated ? sgemv_q4_pack_gated(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, N, K, group, flags,
                                               nullptr, 0, &a.d)
                         : sgemv_q4_pack(nullptr, nullptr, nullptr, N, K, group, flags, nullptr, 0, &a.d);
    if (st) return st;
    if (!q || !scales || (with_zeros && !zeros)) return SGEMV_EINVAL;
    if (gated && (!q_up || !scales_up || (with_zeros && !zeros_up))) return SGEMV_EINVAL;
    if (!packed) return SGEMV_EINVAL;
    if (capacity < a.d.total_bytes) return SGEMV_ESIZE;
    if (!aligned_to(packed, 256) || !aligned_to(scales, 2) || !aligned_to(scales_up, 2)) return SGEMV_EALIGN;
    const int64_t codes = (int64_t)N * K, groups = (int64_t)N * ((K + group - 1) / group);
    const SgemvRows out{packed, 1, 0, (int64_t)a.d.total_bytes};
    const SgemvRows in[6] = {{q, 1, 0, codes}, {scales, 1, 0, 2 * groups}, {with_zeros ? zeros : nullptr, 1, 0, groups},
                             {gated ? q_up : nullptr, 1, 0, codes}, {gated ? scales_up : nullptr, 1, 0, 2 * groups},
                             {gated && with_zeros ? zeros_up : nullptr, 1, 0, groups}};
    for (const SgemvRows& i : in)
        if (sgemv_overlap(out, i)) return SGEMV_EINVAL;
    a.q[0] = q;
    a.q[1] = q_up;
    a.s[0] = scales;
    a.s[1] = scales_up;
    a.z[0] = zeros;
    a.z[1] = zeros_up;
    a.blob = static_cast<uint8_t*>(packed);
    uint64_t n = a.d.w_bytes / 16 + 16 + (a.d.total_bytes - a.d.s_off + 15) / 16;
    const uint64_t grid = (n + 255) / 256, most = 1u << 22;   // a launch has fewer than 2^32 threads
    void* args[] = {&a, &n};
    const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(k_q4_pack), dim3((unsigned)(grid < most ? grid : most)),
                                         dim3(256), args, 0, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return sgemv_hip_failed((int)e);
    if (desc_out) *desc_out = a.d;
    return SGEMV_OK;
}
