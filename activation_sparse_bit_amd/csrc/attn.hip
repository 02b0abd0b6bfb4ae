// Attention of one new token per sequence over a paged cache: sgemv_attn_paged.
//
//   z_i = scale q . k_i,   out = sum_i e^(z_i - m) v_i / sum_i e^(z_i - m)
//
// One pass over the keys and values with a running maximum m, sum and output.
// The query heads that share a key head (up to 16, more take several passes)
// are the columns of v_mfma_f32_16x16x32: keys as the rows give z for 16
// tokens and 16 heads, values as the rows give 16 output elements for 16
// heads.  A lane's four scores of each of two products belong to one head and
// eight tokens, and those eight tokens are just what its slots of the second
// product's operand want, so probabilities never leave their lane, and the
// running maximum, its correction and the output belong to the lane's head.
// A probability is given to the second product as the sum of two numbers of the
// inputs' type (16 bits of it in bf16, 22 in fp16): twice its matrix instructions,
// which the stream hides (48 x 24000 tokens 676 us with one, 673 with two; one
// sequence of 640 tokens 9.3 and 9.6), and an output that is rounded once.
// Values are read in rows (16 bytes a lane, whole rows by neighbouring lanes);
// a lane that reads eight tokens' eight elements turns them by byte permutes
// into eight operands of eight tokens each.  Keys are read in whole lines of 128
// bytes too, eight tokens a load, and two loads exchange half their lanes (eight
// apart) to become the operands of 16 tokens.  Loads of whole lines can be
// marked as used once (48 x 24000 tokens in bf16, 64 heads of 128 on 8: 742 us,
// 675 marked); where a row is no whole number of lines, or several workgroups
// read it, that costs more than it gives (16 x 8192 tokens, 64 heads of 96 on 8: 97
// us, 116 marked; 160 heads of 128 on 8: 135 and 157).
//
// Work is split evenly whatever the lengths: the units of 128 tokens of all
// sequences form one line that is cut into equal runs, and a workgroup takes
// one run for one key head.  Neighbouring workgroups take the same run for
// neighbouring heads, so rows of memory that hold several heads are read at
// one time.  A run's first and last piece may be part of a sequence; such
// pieces go to the workspace, and the last workgroup of that sequence and head
// to arrive joins them in the order of the tokens (above 2 * 16 pieces, each 16
// of them first: one key head over 131000 tokens 27 us, in one step 86).  The
// cut follows from the lengths alone, so results do not depend on timing.
//
// Bound by HBM: 48 x 20011..24000 tokens, 64 heads of 128 on 8, 4.32 GB in 673-676
// us, 6.4 TB/s; 16 sequences of up to 32768 tokens 61 us, 4.4 TB/s, since some
// 15 us go to the first loads, the last steps of uneven workgroups and the
// join.  Loads alone, without the products, take the same times.  A short
// sequence (640 tokens, 9.5 us) waits for a launch, two dependent reads (table,
// keys), one hand-off and a join.
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdint>

#include "kv.h"

namespace {

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf8_t __attribute__((ext_vector_type(8)));
typedef float float4_t __attribute__((ext_vector_type(4)));
typedef uint32_t uint2_t __attribute__((ext_vector_type(2)));
typedef uint32_t uint4_t __attribute__((ext_vector_type(4)));
typedef uint32_t uint2_u __attribute__((ext_vector_type(2), aligned(4)));
typedef uint32_t uint4_u __attribute__((ext_vector_type(4), aligned(8)));

constexpr int kWaves = 4;
constexpr int kTile = 32;                 // tokens of a wavefront's step
constexpr int kUnit = kWaves * kTile;     // tokens of a workgroup's step
constexpr int kRows = 16;                 // query heads of one key head at a time
constexpr int kMaxRuns = 256;             // that the line is cut into, and so pieces of one head
constexpr int kParty = 16;                // pieces that are joined to one where there are more than twice as many
constexpr int kMaxHeads = 2048;           // heads (of all sequences) of one launch
constexpr int kCounterStep = 32;          // words between heads' arrival counters: one, and one for each party
constexpr int kGrid = 512;                // workgroups that the GPU holds at once, two on a compute unit
static_assert((size_t)kMaxHeads * kCounterStep * 4 <= kSgemvCounterBytes, "counters");
constexpr uint32_t kCacheSC1 = 16;        // cache policy: coherent at device scope
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

struct Args {
    const uint8_t* k;
    const uint8_t* v;
    const float* k_scale;
    const float* v_scale;
    int64_t k_page, k_token, k_head, v_page, v_token, v_head;   // bytes
    const uint16_t* q;
    uint16_t* out;
    float* lse;
    const int32_t* table;
    const int32_t* lengths;
    uint32_t* counters;
    void* partial;
    int64_t q_row, q_head, out_row, out_head, ld_table;
    SgemvDiv page;
    int32_t pages, capacity;      // pages of the cache, tokens that a table's row can list
    int32_t batch, heads, groups, group, kv_heads;   // groups: key heads x tiles of 16; group: query heads of a key head
    int32_t dim, window;
    int32_t q_vector;             // whether q can be read in 16 bytes
    uint32_t partial_bytes, slot_bytes;
    float scale, softcap;
};

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ float as_float(uint32_t v) { return __builtin_bit_cast(float, v); }
__device__ __forceinline__ uint32_t as_u32(float v) { return __builtin_bit_cast(uint32_t, v); }
__device__ __forceinline__ int divide(int n, const SgemvDiv& d) { return (int)(((uint64_t)(uint32_t)n * d.m) >> d.s); }

// Largest and sum over the four lanes that hold one head (16 and 32 apart).
__device__ __forceinline__ float head_max(float v) {
    const auto a = __builtin_amdgcn_permlane16_swap(as_u32(v), as_u32(v), false, false);
    v = fmaxf(as_float(a[0]), as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(as_u32(v), as_u32(v), false, false);
    return fmaxf(as_float(b[0]), as_float(b[1]));
}
__device__ __forceinline__ float head_sum(float v) {
    const auto a = __builtin_amdgcn_permlane16_swap(as_u32(v), as_u32(v), false, false);
    v = as_float(a[0]) + as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(as_u32(v), as_u32(v), false, false);
    return as_float(b[0]) + as_float(b[1]);
}

struct F16 {
    using pair = half2_t;
    using frag = half8_t;
    // Probabilities are held 2^15 times their size: of two numbers of fp16 the first then keeps those down to 2^-29 of the
    // largest as well as it keeps the largest, and the second is never off by more than 2^-40 of it.
    static constexpr float kLift = 15.0f;
    static __device__ __forceinline__ float4_t mfma(frag a, frag b, float4_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ uint32_t two(float a, float b) {
        return __builtin_bit_cast(uint32_t, half2_t{(_Float16)a, (_Float16)b});
    }
    static __device__ __forceinline__ float low(uint32_t w) { return (float)__builtin_bit_cast(half2_t, w)[0]; }
    static __device__ __forceinline__ float high(uint32_t w) { return (float)__builtin_bit_cast(half2_t, w)[1]; }
    static __device__ __forceinline__ uint16_t one(float a) { return __builtin_bit_cast(uint16_t, (_Float16)a); }
    template <bool HIGH>
    static __device__ __forceinline__ uint32_t from_e4m3(uint32_t w) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HIGH));
    }
};

struct BF16 {
    using pair = bf2_t;
    using frag = bf8_t;
    static constexpr float kLift = 0.0f;
    static __device__ __forceinline__ float4_t mfma(frag a, frag b, float4_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ uint32_t two(float a, float b) {
        return __builtin_bit_cast(uint32_t, bf2_t{(__bf16)a, (__bf16)b});
    }
    static __device__ __forceinline__ float low(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
    static __device__ __forceinline__ float high(uint32_t w) { return __builtin_bit_cast(float, w & 0xFFFF0000u); }
    static __device__ __forceinline__ uint16_t one(float a) { return __builtin_bit_cast(uint16_t, (__bf16)a); }
    template <bool HIGH>
    static __device__ __forceinline__ uint32_t from_e4m3(uint32_t w) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HIGH));
    }
};

// Tokens of a sequence: [lo, len) are seen; units count from `first`.
struct Span {
    int len, lo, first, units;
    bool bad;
};
__device__ __forceinline__ Span span_of(int len, const Args& a) {
    Span s;
    s.bad = len < 0 || len > a.capacity;
    s.len = s.bad ? 0 : len;
    s.lo = a.window > 0 && s.len > a.window ? s.len - a.window : 0;
    s.first = s.lo & ~(kTile - 1);
    s.units = (s.len - s.first + kUnit - 1) / kUnit;
    if (s.units < 1) s.units = 1;   // an empty sequence's output is written too
    return s;
}

// PAIRS: 64s of elements that a head's keys are padded to.  VW: value elements
// of a lane, VB blocks of 16 of them.  WHOLE: page_size is a multiple of 16, so
// 16 tokens from a multiple of 16 on lie in one page.  LINES: heads of PAIRS * 64
// elements, whole lines, each read once.
template <class T, bool E4M3, int PAIRS, int VW, int VB, bool WHOLE, bool LINES>
struct Attention {
    static constexpr int STEPS = 2 * PAIRS;
    static constexpr int KLOADS = E4M3 ? PAIRS : STEPS;   // 16-byte loads of a token's row by four lanes
    static constexpr int DPAD = VB * 16 * VW;
    static constexpr int VBYTES = VW * (E4M3 ? 1 : 2);
    static constexpr int VWORDS = VBYTES / 4;
    static constexpr int ES = E4M3 ? 1 : 2;
    static constexpr int LDO = 16 * VW + 4;               // floats between rows of the exchange

    struct Shared {
        union {
            float o[kWaves][kRows][LDO];
            struct {
                float2 join[kRows][2 * kParty];           // weight (first the maximum) and sum of every part
                float4_t sums[kRows][DPAD / 4];
            };
        };
        float m[kWaves][kRows], l[kWaves][kRows];
        float row_m[kRows], row_l[kRows];
        float4_t shares[256];
        int scan[kWaves], found[2];
        int last;
    };

    // A step's keys and values as they come.
    struct Tile {
        uint4_t kr[2][KLOADS];
        uint32_t vr[8][VB][VWORDS];
    };
    // Where a step's tokens are: the pages of its halves and the places there, or each lane's own page and place.
    struct Where {
        int id[2], in[2];
        bool bad;
    };

    typename T::frag qf[STEPS];
    float4_t o[VB][VW];
    float m, l;

    static __device__ __forceinline__ uint4_t load16(const uint8_t* p) {
        return __builtin_bit_cast(uint4_t, *reinterpret_cast<const uint4_u*>(p));
    }

    static __device__ __forceinline__ uint4_t load16nt(const uint8_t* p) {
        return __builtin_bit_cast(uint4_t, __builtin_nontemporal_load(reinterpret_cast<const uint4_u*>(p)));
    }
    // First element of a lane's eight of step s.
    static __device__ __forceinline__ int key_dim(int s, int g) {
        return E4M3 ? 64 * (s >> 1) + 16 * g + 8 * (s & 1) : 32 * s + 8 * g;
    }
    // Loads that pair up to whole lines; an odd one is loaded by token.
    static constexpr int PAIRED = KLOADS / 2 * 2;

    // 16 bytes of a key from element d on, zero beyond a head's end, since what stands there may be anything.
    template <bool LAST, bool ONCE>
    static __device__ __forceinline__ uint4_t key_piece(const Args& a, const uint8_t* row, int d) {
        constexpr int n = E4M3 ? 16 : 8;
        if (LINES || !LAST || a.dim == PAIRS * 64 || d + n <= a.dim) return ONCE && LINES ? load16nt(row + d * ES) : load16(row + d * ES);
        uint4_t w = {0, 0, 0, 0};
        if (E4M3 && d + 8 <= a.dim) {
            const uint2_t half = __builtin_bit_cast(uint2_t, *reinterpret_cast<const uint2_u*>(row + d));
            w[0] = half[0];
            w[1] = half[1];
        }
        return w;
    }

    __device__ __forceinline__ void load_q(const Args& a, int b, int head, int g) {
        const uint16_t* q = a.q + b * a.q_row + head * a.q_head;
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int d = key_dim(s, g);
            uint4_t w = {0, 0, 0, 0};
            if (d < a.dim) {
                if (a.q_vector) {
                    w = *reinterpret_cast<const uint4_t*>(q + d);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[j] = q[d + 2 * j] | (uint32_t)q[d + 2 * j + 1] << 16;
                }
            }
            qf[s] = __builtin_bit_cast(typename T::frag, w);
        }
    }

    // The keys of 16 tokens: low is the lane's token of the first eight, high that of the second, own that of its number.
    static __device__ __forceinline__ void load_key(const Args& a, uint4_t (&kr)[KLOADS], const uint8_t* low, const uint8_t* high,
                                                    const uint8_t* own, int c, int g) {
        constexpr int n = E4M3 ? 16 : 8;
#pragma unroll
        for (int s = 0; s < PAIRED; s += 2) {
            const int d = 4 * n * (s + (c >> 3)) + n * g;
            if (s + 2 < KLOADS) {
                kr[s] = key_piece<false, true>(a, low, d);
                kr[s + 1] = key_piece<false, true>(a, high, d);
            } else {
                kr[s] = key_piece<true, true>(a, low, d);
                kr[s + 1] = key_piece<true, true>(a, high, d);
            }
        }
        if constexpr (KLOADS > PAIRED) kr[PAIRED] = key_piece<true, false>(a, own, 4 * n * PAIRED + n * g);
    }

    // A pair of loads as the operands that they stand for: lanes 8..15 of each 16 of the one, 0..7 of the other change places.
    static __device__ __forceinline__ void pair_up(uint4_t& even, uint4_t& odd) {
        uint4_t x, y;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = (int)even[i], o = (int)odd[i];
            x[i] = (uint32_t)__builtin_amdgcn_update_dpp(e, o, 0x128 /* row_ror:8 */, 0xF, 0xC, false);
            y[i] = (uint32_t)__builtin_amdgcn_update_dpp(o, e, 0x128, 0xF, 0x3, false);
        }
        even = x;
        odd = y;
    }

    static __device__ __forceinline__ void load_value(const Args& a, uint32_t (&vr)[VB][VWORDS], const uint8_t* row, int c) {
#pragma unroll
        for (int nb = 0; nb < VB; ++nb) {
            const int d = (nb * 16 + c) * VW;
            const uint8_t* p = row + (LINES || d < a.dim ? d : 0) * ES;   // beyond a head's end: rows of the result that nobody reads
            if constexpr (VWORDS == 4) {
                const uint4_t w = LINES ? load16nt(p) : load16(p);
#pragma unroll
                for (int i = 0; i < 4; ++i) vr[nb][i] = w[i];
            } else if constexpr (VWORDS == 2) {
                const uint2_u* q = reinterpret_cast<const uint2_u*>(p);
                const uint2_t w = __builtin_bit_cast(uint2_t, LINES ? __builtin_nontemporal_load(q) : *q);
                vr[nb][0] = w[0];
                vr[nb][1] = w[1];
            } else {
                vr[nb][0] = *reinterpret_cast<const uint32_t*>(p);
            }
        }
    }

    // The pages of 32 tokens from t0 on, some of them in [lo, len).  Entries that no such token is in are not looked at, they
    // may be those of pages that were given back: what is asked for beside is read from a seen token's page.
    static __device__ __forceinline__ Where find(const Args& a, const int32_t* pages, int t0, const Span& span) {
        Where w;
        w.bad = false;
        if constexpr (WHOLE) {   // a page holds all 16 of a half or none
            const int ta = t0 + 16 <= span.lo ? t0 + 16 : t0, tb = t0 + 16 < span.len ? t0 + 16 : t0;
            const int pa = divide(ta, a.page), pb = divide(tb, a.page);
            w.id[0] = pages[pa];
            w.id[1] = pages[pb];
            w.in[0] = ta - pa * (int)a.page.d;
            w.in[1] = tb - pb * (int)a.page.d;
        } else {
            int t = t0 + (int)(threadIdx.x & 31);
            t = t < span.lo ? span.lo : t < span.len ? t : span.len - 1;
            const int p = divide(t, a.page);
            w.id[0] = pages[p];
            w.in[0] = t - p * (int)a.page.d;
        }
        return w;
    }

    // Starts a step's loads.  An id that is no page becomes page 0, and `bad` says so.
    static __device__ __forceinline__ void load(const Args& a, Tile& tile, Where w, int64_t k_off, int64_t v_off, bool& bad) {
        const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
        if constexpr (WHOLE) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if ((uint32_t)w.id[h] >= (uint32_t)a.pages) {
                    bad = true;
                    w.id[h] = 0;
                }
                const uint8_t* k = a.k + k_off + w.id[h] * a.k_page + w.in[h] * a.k_token;
                load_key(a, tile.kr[h], k + (c & 7) * a.k_token, k + (8 + (c & 7)) * a.k_token, k + c * a.k_token, c, g);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint8_t* v = a.v + v_off + w.id[h] * a.v_page + w.in[h] * a.v_token;
#pragma unroll
                for (int j = 0; j < 4; ++j) load_value(a, tile.vr[4 * h + j], v + (4 * g + j) * a.v_token, c);
            }
        } else {
            const bool out = (uint32_t)w.id[0] >= (uint32_t)a.pages;
            bad |= __ballot(out) != 0;
            if (out) w.id[0] = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint8_t* row[3];
#pragma unroll
                for (int x = 0; x < 3; ++x) {
                    const int from = 16 * h + (x == 0 ? c & 7 : x == 1 ? 8 + (c & 7) : c);
                    const int i = __shfl(w.id[0], from), t = __shfl(w.in[0], from);
                    row[x] = a.k + k_off + i * a.k_page + t * a.k_token;
                }
                load_key(a, tile.kr[h], row[0], row[1], row[2], c, g);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int from = 16 * (j >> 2) + 4 * g + (j & 3);
                const int i = __shfl(w.id[0], from), t = __shfl(w.in[0], from);
                load_value(a, tile.vr[j], a.v + v_off + i * a.v_page + t * a.v_token, c);
            }
        }
    }

    // One step with keys and values that were loaded: 32 tokens from t0 on, some of them in [lo, len).
    __device__ __forceinline__ void step(const Args& a, Tile& tile, const Span& span, int t0, float z_scale, bool twice) {
        const int lane = threadIdx.x & 63, g = lane >> 4;
        uint4_t (&kr)[2][KLOADS] = tile.kr;
        uint32_t (&vr)[8][VB][VWORDS] = tile.vr;
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int s = 0; s < PAIRED; s += 2) pair_up(kr[w][s], kr[w][s + 1]);
        float4_t z[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                uint4_t f;
                if constexpr (E4M3) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t x = kr[w][s >> 1][2 * (s & 1) + i];
                        f[2 * i] = T::template from_e4m3<false>(x);
                        f[2 * i + 1] = T::template from_e4m3<true>(x);
                    }
                } else {
                    f = kr[w][s];
                }
                z[w] = T::mfma(__builtin_bit_cast(typename T::frag, f), qf[s], z[w]);
            }
        // a result has to be read in the block that makes it: a read behind a branch can miss its wait states
        asm volatile("" : "+v"(z[0]), "+v"(z[1]));

        const bool edge = t0 < span.lo || t0 + kTile > span.len;
        float t[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = z[j >> 2][j & 3] * z_scale;
        if (a.softcap > 0.0f) {   // in units of log2(e), as without it
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float x = t[j] * (1.0f / a.softcap);
                t[j] = a.softcap * tanhf(x) * kLog2e;   // a cap's own product would be infinite above 2.36e38
            }
        }
        if (edge) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int tok = t0 + 16 * (j >> 2) + 4 * g + (j & 3);
                const bool seen = tok >= span.lo && tok < span.len;
                if (!seen) {
                    t[j] = -INFINITY;
#pragma unroll
                    for (int nb = 0; nb < VB; ++nb)
#pragma unroll
                        for (int i = 0; i < VWORDS; ++i) vr[j][nb][i] = 0;
                }
            }
        }
        float top = t[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) top = fmaxf(top, t[j]);
        top = fmaxf(m, head_max(top));
        const float base = top == -INFINITY ? 0.0f : top;
        if (__ballot(top != m)) {
            const float by = __builtin_amdgcn_exp2f(m - base);
            l *= by;
#pragma unroll
            for (int nb = 0; nb < VB; ++nb)
#pragma unroll
                for (int r = 0; r < VW; ++r) o[nb][r] *= by;
            m = top;
        }
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            t[j] = __builtin_amdgcn_exp2f(t[j] - base + T::kLift);
            sum += t[j];
        }
        l += sum;
        // A probability meets the values as the sum of two numbers of the type, the second what the first leaves off: 16 bits
        // of it (bf16) or 22 (fp16).  One alone, 8 or 11 bits, was off by up to half a step of the output more.  The second
        // may be zero or below, which an infinite value would make NaN: there the first is taken twice, and the sums halved.
        uint4_t pw, rw;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            pw[i] = T::two(t[2 * i], t[2 * i + 1]);
            rw[i] = twice ? pw[i] : T::two(t[2 * i] - T::low(pw[i]), t[2 * i + 1] - T::high(pw[i]));
        }
        const auto pf = __builtin_bit_cast(typename T::frag, pw), rf = __builtin_bit_cast(typename T::frag, rw);
#pragma unroll
        for (int nb = 0; nb < VB; ++nb)
#pragma unroll
            for (int r2 = 0; r2 < VW / 2; ++r2) {   // elements 2 r2 and 2 r2 + 1 of the lane's
                uint32_t x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if constexpr (E4M3) {
                        const uint32_t w = vr[j][nb][r2 >> 1];
                        x[j] = r2 & 1 ? T::template from_e4m3<true>(w) : T::template from_e4m3<false>(w);
                    } else {
                        x[j] = vr[j][nb][r2];
                    }
                }
                uint4_t lo, hi;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    lo[i] = __builtin_amdgcn_perm(x[2 * i + 1], x[2 * i], 0x05040100u);
                    hi[i] = __builtin_amdgcn_perm(x[2 * i + 1], x[2 * i], 0x07060302u);
                }
                const auto v0 = __builtin_bit_cast(typename T::frag, lo), v1 = __builtin_bit_cast(typename T::frag, hi);
                o[nb][2 * r2] = T::mfma(v0, rf, o[nb][2 * r2]);
                o[nb][2 * r2 + 1] = T::mfma(v1, rf, o[nb][2 * r2 + 1]);
                o[nb][2 * r2] = T::mfma(v0, pf, o[nb][2 * r2]);
                o[nb][2 * r2 + 1] = T::mfma(v1, pf, o[nb][2 * r2 + 1]);
            }
#pragma unroll
        for (int nb = 0; nb < VB; ++nb)
#pragma unroll
            for (int r = 0; r < VW; ++r) asm volatile("" : "+v"(o[nb][r]));
    }

    static __device__ __forceinline__ void store4(const Args& a, int b, int head, int d, float4_t v, float by) {
        uint16_t* p = a.out + b * a.out_row + head * a.out_head + d;
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = T::one(v[i] * by);
    }

    // Joins `count` parts of a head, in the order of their tokens: weights of the parts in LDS, then outputs, of which
    // out(row, element, four of them) takes the sums.  The first parts' outputs are under way while the weights are made.
    template <class Slot, class Out>
    static __device__ __forceinline__ void join(const Args& a, Shared& sh, __amdgpu_buffer_rsrc_t rs, int count, int rows,
                                                Slot slot, Out out) {
        constexpr int kAtOnce = 8;
        const int tid = threadIdx.x;
        const int quads = a.dim / 4, items = rows * quads;
        int split = 1;   // threads that share an item's parts
        while (split < 8 && items * split * 2 <= 256) split *= 2;
        const int share = split > 1 ? tid / items : 0;
        const auto fetch = [&](int row, int d, int from, uint4_t (&w)[kAtOnce]) {
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const int i = from + k * split;
                if (i < count) w[k] = __builtin_amdgcn_raw_buffer_load_b128(rs, slot(i) + (uint32_t)(row * DPAD + d) * 4, 0, kCacheSC1);
            }
        };
        uint4_t w[kAtOnce];
        const int first = split > 1 ? tid - share * items : tid;
        const bool takes = split > 1 ? share < split : tid < items;
        const int first_row = first / quads, first_d = 4 * (first - first_row * quads);
        if (takes) fetch(first_row, first_d, share, w);

        const int row = tid >> 4, sub = tid & 15;
        float top = -INFINITY;
        if (row < rows) {
            for (int i = sub; i < count; i += 16) {
                const auto ml = __builtin_amdgcn_raw_buffer_load_b64(rs, slot(i) + kRows * DPAD * 4 + row * 8, 0, kCacheSC1);
                const float pm = as_float(ml[0]), pl = as_float(ml[1]);
                sh.join[row][i] = make_float2(pm, pl);
                top = fmaxf(top, pm);
            }
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
            const float base = top == -INFINITY ? 0.0f : top;
            float sum = 0.0f;
            for (int i = sub; i < count; i += 16) {
                const float2 p = sh.join[row][i];
                const float by = __builtin_amdgcn_exp2f(p.x - base);
                sh.join[row][i].x = by;
                sum += by * p.y;
            }
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) sum += __shfl_xor(sum, d);
            if (sub == 0) {
                sh.row_m[row] = top;
                sh.row_l[row] = sum;
            }
        }
        __syncthreads();
        for (int x = first; takes && x < items; x += 256) {
            const int r = x == first ? first_row : x / quads, d = x == first ? first_d : 4 * (x - r * quads);
            float4_t sum = {0, 0, 0, 0};
            for (int from = share; from < count; from += kAtOnce * split) {
                if (x != first || from >= split) fetch(r, d, from, w);
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k)
                    if (from + k * split < count) sum += __builtin_bit_cast(float4_t, w[k]) * sh.join[r][from + k * split].x;
            }
            if (split == 1) out(r, d, sum);
            else sh.shares[tid] = sum;
        }
        if (split > 1) {
            __syncthreads();
            if (tid < items) {
                float4_t sum = sh.shares[tid];
                for (int k = 1; k < split; ++k) sum += sh.shares[k * items + tid];
                out(first_row, first_d, sum);
            }
        }
    }

    // Counts the workgroup as one of n that have published; whether it is the last, which leaves the counter at zero.
    static __device__ __forceinline__ bool arrive(Shared& sh, uint32_t* counter, int n) {
        __builtin_amdgcn_s_waitcnt(0);   // this thread's stores acknowledged
        __syncthreads();                 // ... and every thread's, before the count
        if (threadIdx.x == 0) {
            const bool last = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)(n - 1);
            if (last) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            sh.last = last;
        }
        __syncthreads();
        return uniform(sh.last) != 0;
    }

    static __device__ __forceinline__ void publish_sums(Shared& sh, __amdgpu_buffer_rsrc_t rs, uint32_t slot, int rows) {
        if ((int)threadIdx.x < rows) {
            const uint32_t at = slot + kRows * DPAD * 4 + threadIdx.x * 8;
            __builtin_amdgcn_raw_buffer_store_b32(as_u32(sh.row_m[threadIdx.x]), rs, at, 0, kCacheSC1);
            __builtin_amdgcn_raw_buffer_store_b32(as_u32(sh.row_l[threadIdx.x]), rs, at + 4, 0, kCacheSC1);
        }
    }

    __device__ void run(const Args& a, Shared& sh) {
        const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), c = lane & 15, g = lane >> 4;

        // the cut: this workgroup's head, the units before every sequence, and the sequence of its run's first unit
        const int runs = (int)gridDim.x / a.groups, which = (int)blockIdx.x / a.groups, h = (int)blockIdx.x - which * a.groups;
        int b, base, total, run;
        if (a.batch <= 64) {   // every wavefront for itself
            const int mine = lane < a.batch ? span_of(a.lengths[lane], a).units : 0;
            int scan = mine;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int up = __shfl_up(scan, d);
                if (lane >= d) scan += up;
            }
            total = __builtin_amdgcn_readlane(scan, 63);
            run = (total + runs - 1) / runs;
            const uint64_t past = __ballot(scan > which * run);
            if (!past) return;   // beyond the last unit
            b = __builtin_ctzll(past);
            base = __builtin_amdgcn_readlane(scan - mine, b);
        } else {
            const int each = (a.batch + 255) / 256;
            int mine = 0;
            for (int i = 0; i < each; ++i)
                if (tid * each + i < a.batch) mine += span_of(a.lengths[tid * each + i], a).units;
            int scan = mine;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int up = __shfl_up(scan, d);
                if (lane >= d) scan += up;
            }
            if (lane == 63) sh.scan[wave] = scan;
            __syncthreads();
            int before = scan - mine;
            total = 0;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                if (w < wave) before += sh.scan[w];
                total += sh.scan[w];
            }
            total = uniform(total);
            run = (total + runs - 1) / runs;
            const int at = which * run;
            if (at >= total) return;
            for (int i = 0; i < each; ++i) {
                const int n = tid * each + i < a.batch ? span_of(a.lengths[tid * each + i], a).units : 0;
                if (before <= at && at < before + n) {
                    sh.found[0] = tid * each + i;
                    sh.found[1] = before;
                }
                before += n;
            }
            __syncthreads();
            b = uniform(sh.found[0]);
            base = uniform(sh.found[1]);
        }
        int u = which * run;
        const int end = u + run < total ? u + run : total;
        const int kvh = h % a.kv_heads, tile = h / a.kv_heads;
        const int rows = a.group - kRows * tile < kRows ? a.group - kRows * tile : kRows;
        const int head0 = kvh * a.group + kRows * tile;
        Span span = span_of(uniform(a.lengths[b]), a);
        const __amdgpu_buffer_rsrc_t rs =
            __builtin_amdgcn_make_buffer_rsrc(a.partial, (short)0, (int)a.partial_bytes, 0x00020000);
        int piece = 0;

        while (u < end) {
            const int c0 = u - base, c1 = span.units < c0 + (end - u) ? span.units : c0 + (end - u);
            load_q(a, b, head0 + (c < rows ? c : 0), g);
            float z_scale = a.scale * kLog2e;
            if (a.softcap > 0.0f) z_scale = a.scale;
            if (E4M3 && a.k_scale) z_scale *= a.k_scale[kvh];
            bool bad = span.bad;
            const int32_t* pages = a.table + b * a.ld_table;
            // this wavefront's steps of the piece: tokens t0, t0 + kUnit, ... below `last`
            const int64_t k_off = kvh * a.k_head, v_off = kvh * a.v_head;
            const int start = span.first + c0 * kUnit + wave * kTile;
            const int last = span.first + c1 * kUnit < span.len ? span.first + c1 * kUnit : span.len;
            for (bool twice = false;; twice = true) {   // once more only where the first time made NaN
                m = -INFINITY;
                l = 0.0f;
#pragma unroll
                for (int nb = 0; nb < VB; ++nb)
#pragma unroll
                    for (int r = 0; r < VW; ++r) o[nb][r] = float4_t{0, 0, 0, 0};
                for (int t0 = start; t0 < last; t0 += kUnit) {
                    Tile tile;
                    load(a, tile, find(a, pages, t0, span), k_off, v_off, bad);
                    step(a, tile, span, t0, z_scale, twice);
                }
                bool nan = false;
#pragma unroll
                for (int nb = 0; nb < VB; ++nb)
#pragma unroll
                    for (int r = 0; r < VW; ++r)
#pragma unroll
                        for (int i = 0; i < 4; ++i) nan |= o[nb][r][i] != o[nb][r][i];
                if (twice) {
#pragma unroll
                    for (int nb = 0; nb < VB; ++nb)
#pragma unroll
                        for (int r = 0; r < VW; ++r) o[nb][r] *= 0.5f;
                    break;
                }
                if (!__ballot(nan)) break;
            }
            l = head_sum(l);
            if (bad) l = NAN;

            // the workgroup's wavefronts
            if (g == 0) {
                sh.m[wave][c] = m;
                sh.l[wave][c] = l;
            }
            __syncthreads();
            float top = sh.m[0][c];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) top = fmaxf(top, sh.m[w][c]);
            const float from = top == -INFINITY ? 0.0f : top;
            const float by = __builtin_amdgcn_exp2f(m - from);
            if (wave == 0 && g == 0) {
                float sum = 0.0f;
#pragma unroll
                for (int w = 0; w < kWaves; ++w) sum += sh.l[w][c] * __builtin_amdgcn_exp2f(sh.m[w][c] - from);
                sh.row_m[c] = top;
                sh.row_l[c] = sum;
            }
            const bool whole = c1 - c0 == span.units;
            const float v_by = E4M3 && a.v_scale ? a.v_scale[kvh] : 1.0f;
            const uint32_t slot = (uint32_t)(2 * (int)blockIdx.x + (piece ? 1 : 0)) * a.slot_bytes;
#pragma unroll
            for (int nb = 0; nb < VB; ++nb) {
                if (nb) __syncthreads();
                if (c < rows) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int r = 0; r < VW; r += 4)
                            *reinterpret_cast<float4_t*>(&sh.o[wave][c][VW * (4 * g + i) + r]) =
                                float4_t{o[nb][r][i] * by, o[nb][r + 1][i] * by, o[nb][r + 2][i] * by, o[nb][r + 3][i] * by};
                }
                __syncthreads();
                for (int x = tid; x < rows * 4 * VW; x += 256) {
                    const int row = x / (4 * VW), d = 4 * (x % (4 * VW));
                    float4_t sum = *reinterpret_cast<const float4_t*>(&sh.o[0][row][d]);
#pragma unroll
                    for (int w = 1; w < kWaves; ++w) sum += *reinterpret_cast<const float4_t*>(&sh.o[w][row][d]);
                    const int dim = nb * 16 * VW + d;
                    if (whole) {
                        const float total_l = sh.row_l[row];
                        const bool none = span.len == 0 && !span.bad;
                        if (dim < a.dim) store4(a, b, head0 + row, dim, sum, none ? 0.0f : v_by / total_l);
                    } else {
                        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(uint4_t, sum), rs,
                                                               slot + (uint32_t)(row * DPAD + dim) * 4, 0, kCacheSC1);
                    }
                }
            }
            if (whole) {
                if (a.lse && tid < rows)
                    a.lse[(int64_t)b * a.heads + head0 + tid] =
                        span.len == 0 && !span.bad ? -INFINITY
                                                   : kLn2 * (sh.row_m[tid] - T::kLift) + logf(sh.row_l[tid]);
                __syncthreads();   // the next piece writes what this one reads
            } else {
                publish_sums(sh, rs, slot, rows);
                const int w0 = base / run, pieces = (base + span.units - 1) / run - w0 + 1;
                const auto piece_slot = [&](int i) {   // a run that starts before this sequence ends with it: its second slot
                    const int w = w0 + i;
                    return (uint32_t)(2 * (w * a.groups + h) + (w * run < base ? 1 : 0)) * a.slot_bytes;
                };
                const auto final = [&](int row, int d, float4_t sum) { store4(a, b, head0 + row, d, sum, v_by / sh.row_l[row]); };
                uint32_t* counter = a.counters + (b * a.groups + h) * kCounterStep;
                bool joined = false;
                if (pieces <= 2 * kParty) {
                    if (arrive(sh, counter, pieces)) {
                        join(a, sh, rs, pieces, rows, piece_slot, final);
                        joined = true;
                    }
                } else {   // in two steps, the first of them by many workgroups side by side; a party's sum replaces its first piece
                    const int party = (which - w0) / kParty, parties = (pieces + kParty - 1) / kParty;
                    const int members = pieces - party * kParty < kParty ? pieces - party * kParty : kParty;
                    if (arrive(sh, counter + 1 + party, members)) {
                        const uint32_t to = piece_slot(party * kParty);
                        join(a, sh, rs, members, rows, [&](int i) { return piece_slot(party * kParty + i); },
                             [&](int row, int d, float4_t sum) { sh.sums[row][d / 4] = sum; });
                        __syncthreads();   // every piece has been read
                        for (int x = tid; x < rows * (a.dim / 4); x += 256) {
                            const int row = x / (a.dim / 4), d = 4 * (x - row * (a.dim / 4));
                            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(uint4_t, sh.sums[row][d / 4]), rs,
                                                                   to + (uint32_t)(row * DPAD + d) * 4, 0, kCacheSC1);
                        }
                        publish_sums(sh, rs, to, rows);
                        if (arrive(sh, counter, parties)) {
                            join(a, sh, rs, parties, rows, [&](int i) { return piece_slot(i * kParty); }, final);
                            joined = true;
                        }
                    }
                }
                if (joined && a.lse && tid < rows)
                    a.lse[(int64_t)b * a.heads + head0 + tid] = kLn2 * (sh.row_m[tid] - T::kLift) + logf(sh.row_l[tid]);
                __syncthreads();
            }
            u += c1 - c0;
            ++piece;
            if (u < end) {
                base = u;
                ++b;
                span = span_of(uniform(a.lengths[b]), a);
            }
        }
    }
};

template <class T, bool E4M3, int PAIRS, int VW, int VB, bool WHOLE, bool LINES>
__global__ __launch_bounds__(256, PAIRS <= 2 ? 2 : 1) void k_attn(Args a) {
    using Op = Attention<T, E4M3, PAIRS, VW, VB, WHOLE, LINES>;
    __shared__ typename Op::Shared sh;
    Op op;
    op.run(a, sh);
}

typedef void (*Kernel)(Args);

template <class T, bool E4M3, bool WHOLE>
Kernel pick_dim(int dim, bool once) {
    const bool lines = once && dim % (E4M3 ? 128 : 64) == 0;
    if (dim <= 64) {
        if constexpr (!E4M3)
            if (lines) return k_attn<T, E4M3, 1, 4, 1, WHOLE, true>;
        return k_attn<T, E4M3, 1, 4, 1, WHOLE, false>;
    }
    if (dim <= 128) return lines ? k_attn<T, E4M3, 2, 8, 1, WHOLE, true> : k_attn<T, E4M3, 2, 8, 1, WHOLE, false>;
    if (dim <= 192) {
        if constexpr (!E4M3)
            if (lines) return k_attn<T, E4M3, 3, 4, 3, WHOLE, true>;
        return k_attn<T, E4M3, 3, 4, 3, WHOLE, false>;
    }
    return lines ? k_attn<T, E4M3, 4, 8, 2, WHOLE, true> : k_attn<T, E4M3, 4, 8, 2, WHOLE, false>;
}

template <class T>
Kernel pick(bool e4m3, bool whole, int dim, bool once) {
    if (e4m3) return whole ? pick_dim<T, true, true>(dim, once) : pick_dim<T, true, false>(dim, once);
    return whole ? pick_dim<T, false, true>(dim, once) : pick_dim<T, false, false>(dim, once);
}

int padded(int dim) { return (dim + 63) / 64 * 64; }
uint32_t slot_bytes(int dim) { return (uint32_t)(kRows * padded(dim) * 4 + kRows * 8); }

}  // namespace

extern "C" size_t sgemv_attn_workspace_bytes(int32_t batch, int32_t heads, int32_t heads_kv, int32_t dim) {
    if (batch < 0 || heads < 1 || heads > SGEMV_MAX_HEADS || heads_kv < 1 || heads % heads_kv || dim < 8 ||
        dim > SGEMV_MAX_DIM || dim % 8)
        return 0;
    const int64_t groups = (int64_t)heads_kv * ((heads / heads_kv + kRows - 1) / kRows);
    return kSgemvCounterBytes + (size_t)2 * (groups > kGrid ? groups : kGrid) * slot_bytes(dim);
}

extern "C" int sgemv_attn_paged(const sgemv_attn_args* args, const sgemv_kv* cache, void* stream) {
    if (!args || !cache) return SGEMV_EINVAL;
    const sgemv_attn_args& p = *args;
    const sgemv_kv& kv = *cache;
    if (p.reserved || (p.type != SGEMV_F16 && p.type != SGEMV_BF16)) return SGEMV_EINVAL;
    if (p.batch < 0 || p.heads < 1 || p.heads > SGEMV_MAX_HEADS) return SGEMV_ESIZE;
    if (int e = sgemv_check_kv(kv)) return e;
    if (kv.type != p.type && kv.type != SGEMV_E4M3) return SGEMV_EINVAL;
    if (p.heads % kv.heads || !std::isfinite(p.scale) || (p.softcap != 0.0f && !(p.softcap >= FLT_MIN && p.softcap <= FLT_MAX)))
        return SGEMV_EINVAL;
    if (p.window < 0 || p.max_pages < 1 || (int64_t)p.max_pages * kv.page_size > 0x7FFFFFFF - 256) return SGEMV_ESIZE;
    if (p.batch == 0) return SGEMV_OK;
    if (!p.q || !p.out || !p.table || !p.lengths || !p.workspace) return SGEMV_EINVAL;
    const int64_t most = (int64_t)1 << 40;
    if (p.ld_table < p.max_pages || p.ld_table > most || p.q_row < 0 || p.q_head < 0 || p.out_row < 0 || p.out_head < 0 ||
        p.q_row > most || p.q_head > most || p.out_row > most || p.out_head > most)
        return SGEMV_ESIZE;
    if ((p.heads > 1 && (p.q_head < kv.dim || p.out_head < kv.dim)) ||
        (p.batch > 1 && (p.q_row < kv.dim || p.out_row < kv.dim)))
        return SGEMV_ESIZE;
    // rows outside of heads or heads outside of rows; nothing of out is written twice
    const int64_t heads_span = (int64_t)(p.heads - 1) * p.out_head + kv.dim, rows_span = (int64_t)(p.batch - 1) * p.out_row + kv.dim;
    if (p.batch > 1 && p.heads > 1 && p.out_row < heads_span && p.out_head < rows_span) return SGEMV_ESIZE;
    const size_t need = sgemv_attn_workspace_bytes(p.batch, p.heads, kv.heads, kv.dim);
    if (p.workspace_bytes < need) return SGEMV_ESIZE;
    if (!sgemv_aligned(p.q, 2) || !sgemv_aligned(p.out, 2) || !sgemv_aligned(p.lse, 4) || !sgemv_aligned(p.table, 4) ||
        !sgemv_aligned(p.lengths, 4) || !sgemv_aligned(p.workspace, 256))
        return SGEMV_EALIGN;
    const auto whole = [&](const void* at, int64_t row, int64_t head) {
        return SgemvRows{at, 1, 0, ((int64_t)(p.batch - 1) * row + (int64_t)(p.heads - 1) * head + kv.dim) * 2};
    };
    const SgemvRows q = whole(p.q, p.q_row, p.q_head), out = whole(p.out, p.out_row, p.out_head);
    const SgemvRows lse = {p.lse, 1, 0, (int64_t)p.batch * p.heads * 4};
    const SgemvRows ins[] = {{p.table, 1, 0, ((int64_t)(p.batch - 1) * p.ld_table + p.max_pages) * 4},
                             {p.lengths, 1, 0, (int64_t)p.batch * 4},
                             {p.workspace, 1, 0, (int64_t)need},
                             {kv.k_scale, 1, 0, kv.heads * 4},
                             {kv.v_scale, 1, 0, kv.heads * 4},
                             sgemv_kv_rows(kv, true),
                             sgemv_kv_rows(kv, false),
                             q};
    if (sgemv_overlap(out, lse)) return SGEMV_EINVAL;
    for (const SgemvRows& in : ins)
        if (sgemv_overlap(out, in) || sgemv_overlap(lse, in)) return SGEMV_EINVAL;

    const int es = kv.type == SGEMV_E4M3 ? 1 : 2;
    Args a;
    a.k = static_cast<const uint8_t*>(kv.k);
    a.v = static_cast<const uint8_t*>(kv.v);
    a.k_scale = kv.k_scale;
    a.v_scale = kv.v_scale;
    a.k_page = kv.k_page * es; a.k_token = kv.k_token * es; a.k_head = kv.k_head * es;
    a.v_page = kv.v_page * es; a.v_token = kv.v_token * es; a.v_head = kv.v_head * es;
    a.counters = static_cast<uint32_t*>(p.workspace);
    a.partial = static_cast<uint8_t*>(p.workspace) + kSgemvCounterBytes;
    a.q_row = p.q_row; a.q_head = p.q_head; a.out_row = p.out_row; a.out_head = p.out_head; a.ld_table = p.ld_table;
    a.page = sgemv_div(kv.page_size);
    a.pages = kv.pages;
    a.capacity = p.max_pages * kv.page_size;
    a.heads = p.heads;
    a.group = p.heads / kv.heads;
    a.kv_heads = kv.heads;
    a.groups = kv.heads * ((a.group + kRows - 1) / kRows);
    a.dim = kv.dim;
    a.window = p.window;
    a.q_vector = sgemv_aligned(p.q, 16) && p.q_row % 8 == 0 && p.q_head % 8 == 0;
    a.slot_bytes = slot_bytes(kv.dim);
    // a run for each workgroup that fits, for every head
    int runs = kGrid / a.groups;
    runs = runs < 1 ? 1 : runs > kMaxRuns ? kMaxRuns : runs;
    const unsigned grid = (unsigned)(runs * a.groups);
    a.partial_bytes = 2 * grid * a.slot_bytes;
    a.scale = p.scale;
    a.softcap = p.softcap;
    const bool whole_pages = kv.page_size % 16 == 0, e4m3 = kv.type == SGEMV_E4M3;
    const bool once = a.groups == kv.heads;   // a key head's query heads fit one tile
    const Kernel kernel = p.type == SGEMV_F16 ? pick<F16>(e4m3, whole_pages, kv.dim, once) : pick<BF16>(e4m3, whole_pages, kv.dim, once);
    // a launch counts its units in 30 bits and its heads by kMaxHeads counters
    const int64_t units = a.capacity / kUnit + 2;
    int64_t per = kMaxHeads / a.groups;
    if (per > 0x3FFFFFFF / units) per = 0x3FFFFFFF / units;
    if (per < 1) return SGEMV_ESIZE;
    for (int64_t b = 0; b < p.batch; b += per) {
        a.batch = (int)(p.batch - b < per ? p.batch - b : per);
        a.q = static_cast<const uint16_t*>(p.q) + b * p.q_row;
        a.out = static_cast<uint16_t*>(p.out) + b * p.out_row;
        a.lse = p.lse ? p.lse + b * p.heads : nullptr;
        a.table = p.table + b * p.ld_table;
        a.lengths = p.lengths + b;
        void* kargs[] = {&a};
        const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(kernel), dim3(grid), dim3(256), kargs, 0,
                                             static_cast<hipStream_t>(stream));
        if (e != hipSuccess) return sgemv_hip_failed((int)e);
    }
    return SGEMV_OK;
}
