// Rotary positions with several axes, and the write into a paged cache:
// sgemv_rotary.
//
//   (a, b) -> scale (a cos - b sin, a sin + b cos),  angle = position * inv_freq
//
// A workgroup takes one token (and, for few tokens, a part of its heads): it
// forms the token's cosines and sines once, in LDS, and turns every head with
// them.  Angles are reduced in 64 bits, which three roundings leave off by at most
// 2^-51 of the number of turns: a position up to 2^31 with an inv_freq up to 1 is
// under 2^28.4 turns, and off by less than 2^-22 of one; with larger ones, by
// more in proportion.  Cosine and sine follow in fp32 from the part of a turn that
// is left.
//
// Nothing is computed on the way that a stream of q, k and v does not hide:
// bound by HBM for a prompt (16384 tokens, 64 query and 8 key heads of 128, three
// axes: 124 us for 671 MB read and written, 5.4 TB/s, where a copy reaches 5.2 to
// 5.7), by the launch for a token (4.3 us).  One workgroup a token, so that
// its angles are formed once; from 512 workgroups on a token's heads are no
// longer split, which would form them again.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "kv.h"

namespace {

typedef uint32_t uint2_t __attribute__((ext_vector_type(2)));
typedef uint32_t uint4_t __attribute__((ext_vector_type(4)));
typedef float float4_t __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kMaxPairs = SGEMV_MAX_DIM / 2;

struct Args {
    const uint8_t *q, *k, *v;
    uint8_t *q_out, *k_out;
    const int32_t* positions;
    const float* inv_freq;
    const int32_t* slots;
    uint8_t *cache_k, *cache_v;
    const float *k_scale, *v_scale;
    int64_t q_row, q_head, q_out_row, q_out_head, k_row, k_head, k_out_row, k_out_head, v_row, v_head;   // bytes
    int64_t ck_page, ck_token, ck_head, cv_page, cv_token, cv_head;                                      // bytes
    int64_t ld_positions;
    SgemvDiv page;
    int32_t places;           // slots of the cache
    int32_t heads_q, heads_k, heads_v, dim, pairs;
    int32_t cache_type;
    int32_t e4m3_scaled;
    float scale;
    uint32_t axis[kMaxPairs / 16];   // two bits a pair
};

__device__ __forceinline__ int divide(int n, const SgemvDiv& d) { return (int)(((uint64_t)(uint32_t)n * d.m) >> d.s); }

template <int TYPE>
__device__ __forceinline__ float widen(uint32_t bits) {
    if (TYPE == SGEMV_F16) return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
    if (TYPE == SGEMV_BF16) return __builtin_bit_cast(float, bits << 16);
    return __builtin_bit_cast(float, bits);
}
__device__ __forceinline__ uint32_t narrow(float v, int type) {
    if (type == SGEMV_F16) return __builtin_bit_cast(uint16_t, (_Float16)v);
    if (type == SGEMV_BF16) return __builtin_bit_cast(uint16_t, (__bf16)v);
    return __builtin_bit_cast(uint32_t, v);
}
// Two values as e4m3, held at +-448 (the conversion itself would give NaN beyond); NaN stays.
__device__ __forceinline__ float held(float v) { return v != v ? v : fminf(fmaxf(v, -448.0f), 448.0f); }
__device__ __forceinline__ uint32_t e4m3_two(float a, float b) {
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(held(a), held(b), 0, false) & 0xFFFFu;
}

// Eight values from a 16-byte aligned address.
template <int TYPE>
__device__ __forceinline__ void load8(const uint8_t* p, float (&v)[8]) {
    if (TYPE == SGEMV_F32) {
        const float4_t a = *reinterpret_cast<const float4_t*>(p), b = *reinterpret_cast<const float4_t*>(p + 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = a[i];
            v[4 + i] = b[i];
        }
    } else {
        const uint4_t w = *reinterpret_cast<const uint4_t*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = widen<TYPE>(w[i] & 0xFFFFu);
            v[2 * i + 1] = widen<TYPE>(w[i] >> 16);
        }
    }
}
__device__ __forceinline__ void store8(uint8_t* p, int type, const float (&v)[8]) {
    if (type == SGEMV_F32) {
        *reinterpret_cast<float4_t*>(p) = float4_t{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<float4_t*>(p + 16) = float4_t{v[4], v[5], v[6], v[7]};
    } else if (type == SGEMV_E4M3) {
        *reinterpret_cast<uint2_t*>(p) = uint2_t{e4m3_two(v[0], v[1]) | e4m3_two(v[2], v[3]) << 16,
                                                 e4m3_two(v[4], v[5]) | e4m3_two(v[6], v[7]) << 16};
    } else {
        uint4_t w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = narrow(v[2 * i], type) | narrow(v[2 * i + 1], type) << 16;
        *reinterpret_cast<uint4_t*>(p) = w;
    }
}
template <int TYPE>
__device__ __forceinline__ float load1(const uint8_t* p, int d) {
    return TYPE == SGEMV_F32 ? reinterpret_cast<const float*>(p)[d]
                             : widen<TYPE>(reinterpret_cast<const uint16_t*>(p)[d]);
}
__device__ __forceinline__ void store1(uint8_t* p, int type, int d, float v) {
    if (type == SGEMV_F32) reinterpret_cast<float*>(p)[d] = v;
    else if (type == SGEMV_E4M3) p[d] = (uint8_t)e4m3_two(v, v);
    else reinterpret_cast<uint16_t*>(p)[d] = (uint16_t)narrow(v, type);
}

__device__ __forceinline__ int size_of(int type) { return type == SGEMV_F32 ? 4 : type == SGEMV_E4M3 ? 1 : 2; }

// VECTOR: eight elements (of each half) at a time; every address is a multiple
// of 16 bytes, and so are the halves.  Otherwise a pair at a time.
template <int TYPE, bool ADJACENT, bool VECTOR>
__global__ __launch_bounds__(kThreads) void k_rotary(Args a) {
    __shared__ float2 cs[kMaxPairs];
    constexpr int ES = TYPE == SGEMV_F32 ? 4 : 2;
    const int64_t t = blockIdx.x;
    const int tid = threadIdx.x;
    if (tid < a.dim / 2) {
        float2 w = {1.0f, 0.0f};   // elements beyond the pairs pass
        if (tid < a.pairs) {
            const int axis = (a.axis[tid >> 4] >> (2 * (tid & 15))) & 3;
            const double turns = (double)a.positions[axis * a.ld_positions + t] * (double)a.inv_freq[tid] * 0.15915494309189533577;
            const float part = (float)(turns - rint(turns));
            float s, c;
            sincospif(2.0f * part, &s, &c);
            w = {c * a.scale, s * a.scale};
        }
        cs[tid] = w;
    }
    int slot = -1;
    if (a.cache_k) slot = a.slots[t];
    const bool cached = slot >= 0 && slot < a.places;
    const int page = cached ? divide(slot, a.page) : 0, in = cached ? slot - page * (int)a.page.d : 0;
    __syncthreads();

    const int half = a.pairs, rot = 2 * a.pairs;
    // pieces of a head: pairs of runs of eight, then runs of eight that pass; or runs of eight; or pairs
    const int runs = VECTOR ? (ADJACENT ? a.dim / 8 : half / 8) : a.dim / 2;
    const int pieces = VECTOR && !ADJACENT ? runs + (a.dim - rot) / 8 : runs;
    const int straight = VECTOR ? a.dim / 8 : a.dim / 2;   // pieces of a head of v
    const int turned = (a.heads_q + a.heads_k) * pieces;
    const int all = turned + (cached ? a.heads_v * straight : 0);
    for (int x = blockIdx.y * kThreads + tid; x < all; x += gridDim.y * kThreads) {
        const bool is_v = x >= turned;
        const int y = is_v ? x - turned : x, per = is_v ? straight : pieces;
        int h = y / per;
        const int i = y - h * per;
        const bool is_q = !is_v && h < a.heads_q;
        if (!is_v && !is_q) h -= a.heads_q;
        const uint8_t* from = is_q   ? a.q + t * a.q_row + h * a.q_head
                              : is_v ? a.v + t * a.v_row + h * a.v_head
                                     : a.k + t * a.k_row + h * a.k_head;
        uint8_t* to = is_q ? a.q_out + t * a.q_out_row + h * a.q_out_head
                           : !is_v && a.k_out ? a.k_out + t * a.k_out_row + h * a.k_out_head : nullptr;
        uint8_t* keep = nullptr;
        float by = 1.0f;
        if (!is_q && cached) {
            keep = is_v ? a.cache_v + page * a.cv_page + in * a.cv_token + h * a.cv_head
                        : a.cache_k + page * a.ck_page + in * a.ck_token + h * a.ck_head;
            const float* scales = is_v ? a.v_scale : a.k_scale;
            if (scales) by = scales[h];
        }
        const int ks = size_of(a.cache_type);
        if constexpr (VECTOR) {
            const bool two = !ADJACENT && !is_v && i < runs;   // a run of the first half and one of the second
            const int d0 = ADJACENT || is_v || two ? 8 * i : rot + 8 * (i - runs);
            float u[8], w[8];
            load8<TYPE>(from + d0 * ES, u);
            if (two) {
                load8<TYPE>(from + (half + d0) * ES, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 f = cs[d0 + j];
                    const float p = u[j] * f.x - w[j] * f.y, r = u[j] * f.y + w[j] * f.x;
                    u[j] = p;
                    w[j] = r;
                }
            } else if (ADJACENT && !is_v) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = cs[d0 / 2 + j];
                    const float p = u[2 * j] * f.x - u[2 * j + 1] * f.y, r = u[2 * j] * f.y + u[2 * j + 1] * f.x;
                    if (d0 / 2 + j < a.pairs) {
                        u[2 * j] = p;
                        u[2 * j + 1] = r;
                    }
                }
            }
            if (to) {
                store8(to + d0 * ES, TYPE, u);
                if (two) store8(to + (half + d0) * ES, TYPE, w);
            }
            if (keep) {
                if (a.e4m3_scaled) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) u[j] /= by;
                }
                store8(keep + d0 * ks, a.cache_type, u);
                if (two) {
                    if (a.e4m3_scaled) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) w[j] /= by;
                    }
                    store8(keep + (half + d0) * ks, a.cache_type, w);
                }
            }
        } else {
            const bool pair = !is_v && i < a.pairs;
            const int d0 = ADJACENT || !pair ? 2 * i : i, d1 = pair && !ADJACENT ? half + i : d0 + 1;
            float u = load1<TYPE>(from, d0), w = load1<TYPE>(from, d1);
            if (pair) {
                const float2 f = cs[i];
                const float p = u * f.x - w * f.y, r = u * f.y + w * f.x;
                u = p;
                w = r;
            }
            if (to) {
                store1(to, TYPE, d0, u);
                store1(to, TYPE, d1, w);
            }
            if (keep) {
                if (a.e4m3_scaled) {
                    u /= by;
                    w /= by;
                }
                store1(keep, a.cache_type, d0, u);
                store1(keep, a.cache_type, d1, w);
            }
        }
    }
}

typedef void (*Kernel)(Args);

template <int TYPE>
Kernel pick(bool adjacent, bool vector) {
    if (adjacent) return vector ? k_rotary<TYPE, true, true> : k_rotary<TYPE, true, false>;
    return vector ? k_rotary<TYPE, false, true> : k_rotary<TYPE, false, false>;
}

// One operand's tokens x heads of dim elements, as rows for overlap checks.
struct Operand {
    const void* p;
    int64_t row, head;   // elements
    int heads;
};

SgemvRows extent(const Operand& o, int64_t tokens, int dim, int size) {
    // tokens as rows where a token's heads lie together, else one range
    const int64_t span = (int64_t)(o.heads - 1) * o.head + dim;
    if (tokens == 1 || o.row >= span) return SgemvRows{o.p, tokens, o.row * size, span * size};
    return SgemvRows{o.p, 1, 0, ((tokens - 1) * o.row + span) * size};
}

// Whether two operands share bytes.  Heads that lie between each other's (queries, keys and values side by side head by
// head) are told apart by their places within the smallest stride, where both have the same strides, all multiples of it.
bool share(const Operand& a, const Operand& b, int64_t tokens, int dim, int size) {
    if (!a.p || !b.p) return false;
    if (a.heads > 1 && b.heads > 1 && a.head == b.head && (tokens == 1 || a.row == b.row)) {
        const int64_t step = tokens > 1 && a.row < a.head ? a.row : a.head;
        if (a.head % step == 0 && (tokens == 1 || a.row % step == 0)) {
            const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
            const int64_t bytes = step * size, width = (int64_t)dim * size;
            const int64_t off = pb > pa ? (int64_t)((pb - pa) % (uintptr_t)bytes)
                                        : (int64_t)(((uintptr_t)bytes - (pa - pb) % (uintptr_t)bytes) % (uintptr_t)bytes);
            if (off >= width && off + width <= bytes) return false;
        }
    }
    return sgemv_overlap(extent(a, tokens, dim, size), extent(b, tokens, dim, size));
}

}  // namespace

extern "C" int sgemv_rotary(const sgemv_rotary_args* args, const sgemv_kv* cache, void* stream) {
    if (!args) return SGEMV_EINVAL;
    const sgemv_rotary_args& p = *args;
    if (p.type != SGEMV_F16 && p.type != SGEMV_BF16 && p.type != SGEMV_F32) return SGEMV_EINVAL;
    if (p.flags & ~(SGEMV_ROTARY_ADJACENT | SGEMV_ROTARY_STRIPED) || !std::isfinite(p.scale)) return SGEMV_EINVAL;
    if (p.tokens < 0 || p.tokens > 0x7FFFFFFF || p.heads_q < 0 || p.heads_q > SGEMV_MAX_HEADS || p.heads_kv < 0 ||
        p.heads_kv > SGEMV_MAX_HEADS)
        return SGEMV_ESIZE;
    if (p.dim < 8 || p.dim > SGEMV_MAX_DIM || p.dim % 8 || p.pairs < 1 || p.pairs > p.dim / 2) return SGEMV_ESIZE;
    if (p.axes < 1 || p.axes > SGEMV_MAX_AXES) return SGEMV_ESIZE;
    int64_t sum = 0;
    for (int i = 0; i < SGEMV_MAX_AXES; ++i) {
        if (p.sections[i] < 0 || (i >= p.axes && p.sections[i])) return SGEMV_EINVAL;
        sum += p.sections[i];
    }
    if (sum != p.pairs) return SGEMV_EINVAL;
    if (cache) {
        if (int e = sgemv_check_kv(*cache)) return e;
        if (!p.k || cache->heads != p.heads_kv || cache->dim != p.dim) return SGEMV_EINVAL;
    }
    if (p.tokens == 0) return SGEMV_OK;
    if (!p.positions || !p.inv_freq || (!p.q && !p.k)) return SGEMV_EINVAL;
    if ((!p.q) != (!p.q_out) || (p.q && p.heads_q < 1) || (p.k && p.heads_kv < 1)) return SGEMV_EINVAL;
    if (cache ? !p.slots : (p.v || p.slots || (p.k && !p.k_out))) return SGEMV_EINVAL;
    if (!p.k && p.k_out) return SGEMV_EINVAL;
    const int64_t most = (int64_t)1 << 40;
    if (p.ld_positions < 0 || p.ld_positions > most || (p.axes > 1 && p.ld_positions < p.tokens)) return SGEMV_ESIZE;
    const int size = sgemv_size_of(p.type);
    const Operand q = {p.q, p.q_row, p.q_head, p.heads_q}, q_out = {p.q_out, p.q_out_row, p.q_out_head, p.heads_q};
    const Operand k = {p.k, p.k_row, p.k_head, p.heads_kv}, k_out = {p.k_out, p.k_out_row, p.k_out_head, p.heads_kv};
    const Operand v = {p.v, p.v_row, p.v_head, p.heads_kv};
    bool vector = true;
    for (const Operand* o : {&q, &q_out, &k, &k_out, &v}) {
        if (!o->p) continue;
        if (o->row < 0 || o->head < 0 || o->row > most || o->head > most) return SGEMV_ESIZE;
        if ((o->heads > 1 && o->head < p.dim) || (p.tokens > 1 && o->row < p.dim)) return SGEMV_ESIZE;
        if (o->heads > 1 && p.tokens > 1 && o->row < (o->heads - 1) * o->head + p.dim &&
            o->head < (p.tokens - 1) * o->row + p.dim)
            return SGEMV_ESIZE;
        if (!sgemv_aligned(o->p, (uintptr_t)size)) return SGEMV_EALIGN;
        vector = vector && sgemv_aligned(o->p, 16) && o->row * size % 16 == 0 && o->head * size % 16 == 0;
    }
    if (!sgemv_aligned(p.positions, 4) || !sgemv_aligned(p.inv_freq, 4) || !sgemv_aligned(p.slots, 4)) return SGEMV_EALIGN;
    const bool adjacent = p.flags & SGEMV_ROTARY_ADJACENT;
    if (!adjacent && (p.pairs % 8 || (p.dim - 2 * p.pairs) % 8)) vector = false;

    const auto ext = [&](const Operand& o) { return extent(o, p.tokens, p.dim, size); };
    SgemvRows outs[4] = {ext(q_out), ext(k_out), {nullptr, 1, 0, 0}, {nullptr, 1, 0, 0}};
    if (cache) {
        outs[2] = sgemv_kv_rows(*cache, true);
        outs[3] = sgemv_kv_rows(*cache, false);
    }
    const SgemvRows ins[] = {ext(q), ext(k), ext(v), {p.positions, 1, 0, ((int64_t)(p.axes - 1) * p.ld_positions + p.tokens) * 4},
                             {p.inv_freq, 1, 0, (int64_t)p.pairs * 4}, {p.slots, 1, 0, p.tokens * 4},
                             {cache ? cache->k_scale : nullptr, 1, 0, (int64_t)p.heads_kv * 4},
                             {cache ? cache->v_scale : nullptr, 1, 0, (int64_t)p.heads_kv * 4}};
    const auto replaces = [&](const Operand& out, const Operand& in) {   // the very same elements
        return out.p == in.p && (p.tokens == 1 || out.row == in.row) && (in.heads == 1 || out.head == in.head);
    };
    const Operand* const turned[2] = {&q_out, &k_out};
    const Operand* const read[3] = {&q, &k, &v};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 8; ++j) {
            if (i == 0 && j == 0 && replaces(q_out, q)) continue;
            if (i == 1 && j == 1 && replaces(k_out, k)) continue;
            if (i < 2 && j < 3 ? share(*turned[i], *read[j], p.tokens, p.dim, size) : sgemv_overlap(outs[i], ins[j]))
                return SGEMV_EINVAL;
        }
        // keys and values may be parts of one buffer: the caller's strides keep them apart
        for (int j = i + 1; j < 4; ++j)
            if (i == 0 && j == 1 ? share(q_out, k_out, p.tokens, p.dim, size) : i < 2 && sgemv_overlap(outs[i], outs[j]))
                return SGEMV_EINVAL;
    }

    Args a = {};
    const auto bytes = [&](int64_t n) { return n * size; };
    a.q = static_cast<const uint8_t*>(p.q); a.k = static_cast<const uint8_t*>(p.k); a.v = static_cast<const uint8_t*>(p.v);
    a.q_out = static_cast<uint8_t*>(p.q_out); a.k_out = static_cast<uint8_t*>(p.k_out);
    a.positions = p.positions; a.inv_freq = p.inv_freq; a.slots = p.slots;
    a.q_row = bytes(p.q_row); a.q_head = bytes(p.q_head); a.q_out_row = bytes(p.q_out_row); a.q_out_head = bytes(p.q_out_head);
    a.k_row = bytes(p.k_row); a.k_head = bytes(p.k_head); a.k_out_row = bytes(p.k_out_row); a.k_out_head = bytes(p.k_out_head);
    a.v_row = bytes(p.v_row); a.v_head = bytes(p.v_head);
    a.ld_positions = p.ld_positions;
    a.page = sgemv_div(1);
    if (cache) {
        const int es = sgemv_size_of(cache->type);
        a.cache_k = static_cast<uint8_t*>(cache->k); a.cache_v = static_cast<uint8_t*>(cache->v);
        a.k_scale = cache->k_scale; a.v_scale = cache->v_scale;
        a.ck_page = cache->k_page * es; a.ck_token = cache->k_token * es; a.ck_head = cache->k_head * es;
        a.cv_page = cache->v_page * es; a.cv_token = cache->v_token * es; a.cv_head = cache->v_head * es;
        a.page = sgemv_div(cache->page_size);
        a.places = cache->pages * cache->page_size;
        a.cache_type = cache->type;
        a.e4m3_scaled = cache->k_scale || cache->v_scale;
    }
    a.heads_q = p.q ? p.heads_q : 0;
    a.heads_k = p.k ? p.heads_kv : 0;
    a.heads_v = p.v ? p.heads_kv : 0;
    a.dim = p.dim;
    a.pairs = p.pairs;
    a.scale = p.scale;
    int left[SGEMV_MAX_AXES], axis = 0;
    for (int i = 0; i < SGEMV_MAX_AXES; ++i) left[i] = p.sections[i];
    for (int i = 0; i < p.pairs; ++i) {
        while (!left[axis]) axis = (axis + 1) % SGEMV_MAX_AXES;   // some axis has pairs left: their sum is pairs
        --left[axis];
        a.axis[i >> 4] |= (uint32_t)axis << (2 * (i & 15));
        if (p.flags & SGEMV_ROTARY_STRIPED) axis = (axis + 1) % SGEMV_MAX_AXES;
    }
    const Kernel kernel = p.type == SGEMV_F16    ? pick<SGEMV_F16>(adjacent, vector)
                          : p.type == SGEMV_BF16 ? pick<SGEMV_BF16>(adjacent, vector)
                                                 : pick<SGEMV_F32>(adjacent, vector);
    // few tokens: a token's heads over several workgroups
    const int pieces = (a.heads_q + a.heads_k + a.heads_v) * (vector ? p.dim / 8 : p.dim / 2);
    int64_t split = 512 / p.tokens;
    if (split > (pieces + kThreads - 1) / kThreads) split = (pieces + kThreads - 1) / kThreads;
    if (split < 1) split = 1;
    // a launch has fewer than 2^32 threads
    const int64_t per = (int64_t)1 << 22;
    for (int64_t t = 0; t < p.tokens; t += per) {
        const int64_t n = p.tokens - t < per ? p.tokens - t : per;
        void* kargs[] = {&a};
        const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(kernel), dim3((unsigned)n, (unsigned)split),
                                             dim3(kThreads), kargs, 0, static_cast<hipStream_t>(stream));
        if (e != hipSuccess) return sgemv_hip_failed((int)e);
        a.q += per * a.q_row; a.q_out += per * a.q_out_row; a.k += per * a.k_row; a.v += per * a.v_row;
        if (a.k_out) a.k_out += per * a.k_out_row;
        a.positions += per;
        if (a.slots) a.slots += per;
    }
    return SGEMV_OK;
}
