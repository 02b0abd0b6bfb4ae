// Beam selection: sgemv_beam_select.
//
//   s(w, v) = score[w] + logit[w][v] - log sum_u e^logit[w][u]
//
// One pass over the logits in one launch.  A workgroup takes a part of one
// beam's vocabulary into registers and leaves the part's maximum, its sum of
// exponentials and its best candidates; the last workgroup of a batch entry to
// arrive has every beam's normaliser and picks among the parts' candidates.
//
// The best n of a part: every lane has its largest value, and the k-th largest
// of a wavefront's 64 is found bit by bit with ballots.  With k = n / 4, n values
// reach the smallest of the four wavefronts' bounds; the few dozen values that
// do are ranked, each by counting those above it.  Where equal values make them
// too many, the threads' best are told apart by their places, and the n-th best
// of those is a bound that only the values of n threads can reach.  Much the
// same picks the parts that matter by their best values, and of the part that is
// r-th by its best only the first n - r values can be among the best n.
// Within a beam the logits' order is that of s, and equal values go by their
// place, so every key is unique and the answer does not depend on timing.
//
// Bound by latency: one request with 4 beams of 32003 takes 10.9 us, of which
// 5 go to the last workgroup's choice (three dependent reads past the caches and
// some ten barriers).  48 x 8 beams of 100003 in bf16, 63 MB without
// those that have ended, take 34 us, vector units half busy: loads and sums alone take 19, the parts' choices 7, the last
// entries' 8; smaller parts (2048 or 4096 values each) take 44, since each
// part's choice costs much the same whatever its size.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "kv.h"

namespace {

typedef uint32_t uint4_t __attribute__((ext_vector_type(4)));
typedef uint32_t uint4_h __attribute__((ext_vector_type(4), aligned(2)));   // 16 bytes at any element
typedef uint32_t uint4_w __attribute__((ext_vector_type(4), aligned(4)));

constexpr int kThreads = 256;
constexpr int kMaxBatch = 2048;        // entries of one launch
constexpr int kMostTied = 6 * kThreads; // a part's values to be ranked, before their places tell them apart
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kFar = 67108864.0f;    // 2^26: as far from zero a float may be off from v L by 2, and ever more beyond
constexpr int kCounterStep = 16;       // words between arrival counters
static_assert((size_t)kMaxBatch * kCounterStep * 4 <= kSgemvCounterBytes, "counters");

struct Args {
    const uint8_t* logits;
    const float* scores;
    const uint8_t* finished;
    int32_t *tokens, *parents;
    float* scores_out;
    uint32_t* counters;
    uint64_t* parts_out;          // per beam and part: choices keys, then maximum and sum
    int64_t ld_batch, ld_beam;    // elements
    int32_t beams, vocab, choices, parts, slice, end_token;
};

// Bits of a widened value that are always the same.
template <int TYPE>
constexpr int kFixed = TYPE == SGEMV_F16 ? 13 : TYPE == SGEMV_BF16 ? 16 : 0;

// A value's bits as a number that grows with it, without the fixed ones; 0 for
// NaN and -infinity.
template <int TYPE>
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v + 0.0f);   // -0 is 0
    const uint32_t k = u & 0x80000000u ? ~u : u | 0x80000000u;
    return v > -INFINITY ? k >> kFixed<TYPE> : 0u;               // false for NaN
}
template <int TYPE>
__device__ __forceinline__ float value_of(uint32_t key) {
    const uint32_t k = key << kFixed<TYPE>;
    return __builtin_bit_cast(float, k & 0x80000000u ? k & 0x7FFFFFFFu : ~k & ~((1u << kFixed<TYPE>) - 1u));
}
__device__ __forceinline__ uint64_t key_of(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return u >> 63 ? ~u : u | 1ull << 63;
}
__device__ __forceinline__ double score_of(uint64_t k) {
    return __builtin_bit_cast(double, k >> 63 ? k & ~(1ull << 63) : ~k);
}

// What is handed from workgroup to workgroup goes past the caches of an XCD.
__device__ __forceinline__ void publish(uint64_t* p, uint64_t v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t fetch(const uint64_t* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

template <int TYPE>
__device__ __forceinline__ float widen(uint32_t bits) {
    if (TYPE == SGEMV_F16) return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
    if (TYPE == SGEMV_BF16) return __builtin_bit_cast(float, bits << 16);
    return __builtin_bit_cast(float, bits);
}

// Eight values from any element on.
template <int TYPE>
struct Run {
    uint4_t a, b;
    __device__ __forceinline__ void load(const uint8_t* p) {
        if constexpr (TYPE == SGEMV_F32) {
            a = *reinterpret_cast<const uint4_w*>(p);
            b = *reinterpret_cast<const uint4_w*>(p + 16);
        } else {
            a = *reinterpret_cast<const uint4_h*>(p);
        }
    }
    __device__ __forceinline__ float get(int j) const {
        if constexpr (TYPE == SGEMV_F32) return widen<TYPE>(j < 4 ? a[j] : b[j - 4]);
        else return widen<TYPE>(j & 1 ? a[j >> 1] >> 16 : a[j >> 1] & 0xFFFFu);
    }
};

// Sums and maxima over 16 lanes (by rotations) and over all 64, by moves within
// the vector unit.
template <int N>
__device__ __forceinline__ float turned(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x120 + N, 0xF, 0xF, false));
}
template <int N>
__device__ __forceinline__ double turned(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, 0x120 + N, 0xF, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), 0x120 + N, 0xF, 0xF, false);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ float row_max(float v) {
    v = fmaxf(v, turned<1>(v));
    v = fmaxf(v, turned<2>(v));
    v = fmaxf(v, turned<4>(v));
    return fmaxf(v, turned<8>(v));
}
template <class V>
__device__ __forceinline__ V row_sum(V v) {
    v += turned<1>(v);
    v += turned<2>(v);
    v += turned<4>(v);
    return v + turned<8>(v);
}
// (A bit cast of a vector's element itself reads element 0: these take it as a number.)
__device__ __forceinline__ float as_float(uint32_t v) { return __builtin_bit_cast(float, v); }
__device__ __forceinline__ uint32_t as_u32(float v) { return __builtin_bit_cast(uint32_t, v); }
__device__ __forceinline__ float wave_max(float v) {
    v = row_max(v);
    const auto x = __builtin_amdgcn_permlane16_swap(as_u32(v), as_u32(v), false, false);
    v = fmaxf(as_float(x[0]), as_float(x[1]));
    const auto y = __builtin_amdgcn_permlane32_swap(as_u32(v), as_u32(v), false, false);
    return fmaxf(as_float(y[0]), as_float(y[1]));
}
__device__ __forceinline__ float wave_sum(float v) {
    v = row_sum(v);
    const auto x = __builtin_amdgcn_permlane16_swap(as_u32(v), as_u32(v), false, false);
    v = as_float(x[0]) + as_float(x[1]);
    const auto y = __builtin_amdgcn_permlane32_swap(as_u32(v), as_u32(v), false, false);
    return as_float(y[0]) + as_float(y[1]);
}

// The largest of three; where one is NaN, possibly NaN (fmaxf would take two more instructions for that).
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}

// One beam's candidate: beam, logit and token in one number, larger for the one to prefer among equal s.
__device__ __forceinline__ uint64_t place_of(int beam, uint64_t key) {
    return (uint64_t)(63 - beam) << 52 | (key >> 32) << 20 | (0xFFFFFu - (~(uint32_t)key & 0xFFFFFu));
}

__device__ __forceinline__ int lanes(bool v) { return __popcll(__ballot(v)); }

// The n-th largest of the wavefront's 64 keys, or 0 where fewer than n are
// above it.
template <int BITS>
__device__ __forceinline__ uint32_t nth_of_wave(uint32_t key, int n) {
    uint32_t t = 0;
#pragma unroll 4
    for (int bit = BITS - 1; bit >= 0; --bit) {
        const uint32_t trial = t | 1u << bit;
        if (lanes(key >= trial) >= n) t = trial;
    }
    return t;
}

struct Candidate {
    uint64_t s, place;
};
__device__ __forceinline__ bool above(const Candidate& a, const Candidate& b) {
    return (a.s > b.s) | ((a.s == b.s) & (a.place > b.place));   // without branches
}

// Rank of item i of a list of `count` in LDS, counted by `per` neighbouring
// threads together (a power of two up to 64).
template <class V, class F>
__device__ __forceinline__ int rank_of(const V* list, int count, const V& item, int per, F above_it) {
    int rank = 0;
#pragma unroll 8
    for (int k = (int)threadIdx.x & (per - 1); k < count; k += per) rank += above_it(list[k], item);
    for (int d = 1; d < per; d <<= 1) rank += __shfl_xor(rank, d);
    return rank;
}
// Threads that count together for each of `count` items.
__device__ __forceinline__ int threads_per(int count) {
    int per = 1;
    while (per < 64 && count * per * 2 <= kThreads) per *= 2;
    return per;
}

// Drops items that cannot be among the n best of a list of up to PER * kThreads
// in LDS: every wavefront finds the n/4-th largest key of its share, bit by bit,
// and n items reach the smallest of these.  Ranking is quadratic, so it pays from
// some dozen items on.  Returns the new count.
template <int PER, class V, class F>
__device__ __forceinline__ int tighten(V* list, int count, int most, int n, uint32_t* bounds, uint32_t* left, F key) {
    if (count <= most) return count;   // most is at least n, so every wavefront's share has n/4 items
    __syncthreads();                   // `count` may come from *left: every thread has read it before it is cleared
    const int tid = threadIdx.x;
    constexpr int kWaves = kThreads / 64;
    const int at = (tid & 63) * kWaves + tid / 64;   // neighbours, which are alike, over the wavefronts
    V mine[PER];
    uint32_t k[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        k[i] = 0;
        if (at + i * kThreads < count) {
            mine[i] = list[at + i * kThreads];
            k[i] = key(mine[i]);
        }
    }
    uint32_t t = 0;
    const int need = (n + kWaves - 1) / kWaves;
    for (int bit = 31; bit >= 0; --bit) {
        const uint32_t trial = t | 1u << bit;
        int here = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (i * kThreads < count) here += lanes(k[i] >= trial);
        if (here >= need) t = trial;
    }
    if ((tid & 63) == 0) bounds[tid / 64] = t;
    if (tid == 0) *left = 0;
    __syncthreads();
    t = bounds[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) t = t < bounds[w] ? t : bounds[w];
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (at + i * kThreads < count && k[i] >= t) list[atomicAdd(left, 1u)] = mine[i];
    __syncthreads();
    return (int)*left;
}

// The n best of the candidates found, best first; the entry's counter is free again.
template <int PER>
__device__ __forceinline__ void finish(const Args& a, Candidate* found, int there, int n, int entry, uint32_t* bounds,
                                       uint32_t* left, uint32_t* counter) {
    const int tid = threadIdx.x;
    const int count = tighten<PER>(found, there, 2 * n + 96, n, bounds, left, [](const Candidate& c) { return (uint32_t)(c.s >> 32); });
    const int per = threads_per(count);
    const int64_t out = (int64_t)entry * n;
    for (int i = tid / per; i < count; i += kThreads / per) {
        const Candidate c = found[i];
        const int r = rank_of(found, count, c, per, above);
        if (r < n && (tid & (per - 1)) == 0) {
            a.tokens[out + r] = (int32_t)(0xFFFFFu - (uint32_t)(c.place & 0xFFFFFu));
            a.parents[out + r] = 63 - (int32_t)(c.place >> 52);
            a.scores_out[out + r] = (float)score_of(c.s);
        }
    }
    if (tid >= count && tid < n) {
        a.tokens[out + tid] = -1;
        a.parents[out + tid] = -1;
        a.scores_out[out + tid] = -INFINITY;
    }
    if (tid == 0) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// RUNS runs of eight values a thread, at most N choices.  Six workgroups a compute unit hide each other's waits (48 x 8 x
// 100003: 33.9 us, five 36.3, eight 34); with 64 choices that would spill more.
template <int TYPE, int RUNS, int N>
__global__ __launch_bounds__(kThreads, N <= 16 ? 6 : 5) void k_beam(Args a) {
    extern __shared__ uint64_t lds[];
    __shared__ float part_m[kThreads / 64], part_s[kThreads / 64], part_t[kThreads / 64];
    __shared__ double offset[SGEMV_MAX_BEAMS], largest[SGEMV_MAX_BEAMS];   // s = (logit - largest) + offset
    __shared__ uint32_t left, bounds[kThreads / 64], wave_bound[kThreads / 64], order[N];
    __shared__ uint64_t part_bound;
    __shared__ Candidate bound;
    constexpr int ES = TYPE == SGEMV_F32 ? 4 : 2;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = a.choices;
    const int part = blockIdx.x % a.parts, beam = (int)(blockIdx.x / a.parts) % a.beams;
    const int entry = (int)(blockIdx.x / a.parts) / a.beams;
    const int record = n + 1;
    uint64_t* mine = a.parts_out + (int64_t)blockIdx.x * record;
    const auto order_of = [](uint64_t x, uint64_t y) { return x > y; };

    const bool done = a.finished && a.finished[entry * a.beams + beam];
    if (!done) {
        const uint8_t* row = a.logits + (entry * a.ld_batch + beam * a.ld_beam) * ES;
        const int first = part * a.slice, end = first + a.slice < a.vocab ? first + a.slice : a.vocab;
        float v[RUNS][8];
        int base[RUNS];   // place of a run's first value
        if (a.vocab >= 8) {
            // a run that passes the end is read from eight before it, and what belongs to others is left out: loads
            // without a branch are all in flight at once
            Run<TYPE> raw[RUNS];
#pragma unroll
            for (int r = 0; r < RUNS; ++r) {
                const int at = first + (r * kThreads + tid) * 8;
                base[r] = at < end - 8 ? at : end - 8;
                raw[r].load(row + (int64_t)base[r] * ES);
            }
#pragma unroll
            for (int r = 0; r < RUNS; ++r) {
                const int at = first + (r * kThreads + tid) * 8;
#pragma unroll
                for (int j = 0; j < 8; ++j) v[r][j] = raw[r].get(j);
                if (base[r] < at) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (base[r] + j < at) v[r][j] = -INFINITY;
                }
            }
        } else {
#pragma unroll
            for (int r = 0; r < RUNS; ++r) {
                base[r] = (r * kThreads + tid) * 8;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[r][j] = -INFINITY;
                    if (base[r] + j < end)
                        v[r][j] = TYPE == SGEMV_F32 ? widen<TYPE>(reinterpret_cast<const uint32_t*>(row)[base[r] + j])
                                                    : widen<TYPE>(reinterpret_cast<const uint16_t*>(row)[base[r] + j]);
                }
            }
        }
        float top = -INFINITY;
#pragma unroll
        for (int r = 0; r < RUNS; ++r) {
            top = max3(top, v[r][0], v[r][1]);
            top = max3(top, v[r][2], v[r][3]);
            top = max3(top, v[r][4], v[r][5]);
            top = max3(top, v[r][6], v[r][7]);
        }
        const float wm = wave_max(top);
        // wavefronts whose 64 lanes all have values; where there is none, the first one's may do alone
        const int full = end - first >= 4 * 512 ? 4 : end - first >= 512 ? (end - first) / 512 : 1;
        const uint32_t nth = nth_of_wave<32 - kFixed<TYPE>>(key_of<TYPE>(top), (n + full - 1) / full);
        if (lane == 0) {
            part_m[wave] = wm;
            part_t[wave] = nth ? value_of<TYPE>(nth) : -3.4028234664e38f;   // no bound: any finite value
        }
        if (tid == 0) {
            left = 0;
            part_bound = 0;
        }
        __syncthreads();
        float m = part_m[0], least = part_t[0];
#pragma unroll
        for (int w = 1; w < kThreads / 64; ++w) {
            m = fmaxf(m, part_m[w]);
            least = w < full ? fminf(least, part_t[w]) : least;
        }
        // 2^(v L - c), c the largest v L as a float: one rounding each, and none of the largest logit's own
        const float c = m == -INFINITY ? 0.0f : m * kLog2e;
        float sum = 0.0f;
#pragma unroll
        for (int r = 0; r < RUNS; ++r)
#pragma unroll
            for (int j = 0; j < 8; ++j) sum += __builtin_amdgcn_exp2f(fmaf(v[r][j], kLog2e, -c));
        sum = wave_sum(sum);
        if (lane == 0) part_s[wave] = sum;
        __syncthreads();
        sum = part_s[0];
#pragma unroll
        for (int w = 1; w < kThreads / 64; ++w) sum += part_s[w];
        if (sum != sum || !(fabsf(c) <= kFar)) {
            // the same in every thread: NaN among the logits is left out, an infinity stays; and far from zero, where
            // logits are whole numbers, differences are taken first
            m = -INFINITY;
#pragma unroll
            for (int r = 0; r < RUNS; ++r)
#pragma unroll
                for (int j = 0; j < 8; ++j) m = v[r][j] > m ? v[r][j] : m;
            m = wave_max(m);
            __syncthreads();
            if (lane == 0) part_m[wave] = m;
            __syncthreads();
            m = part_m[0];
#pragma unroll
            for (int w = 1; w < kThreads / 64; ++w) m = fmaxf(m, part_m[w]);
            const float near = m == -INFINITY ? 0.0f : m * kLog2e;
            const bool far = !(fabsf(near) <= kFar);
            sum = 0.0f;
#pragma unroll
            for (int r = 0; r < RUNS; ++r)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (v[r][j] == v[r][j])
                        sum += __builtin_amdgcn_exp2f(far ? (v[r][j] - m) * kLog2e : fmaf(v[r][j], kLog2e, -near));
            sum = wave_sum(sum);
            if (lane == 0) part_s[wave] = sum;
            __syncthreads();
            sum = part_s[0];
#pragma unroll
            for (int w = 1; w < kThreads / 64; ++w) sum += part_s[w];
        }
        const auto place = [&](int r, int j) { return ~(uint32_t)(base[r] + j); };
        // values that reach the bound, each wavefront's in a place of its own
        constexpr uint32_t kRoom = kMostTied / (kThreads / 64);
        uint32_t many = 0;
#pragma unroll
        for (int r = 0; r < RUNS; ++r)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint64_t reach = __ballot(v[r][j] >= least);
                if (reach) {
                    if (v[r][j] >= least) {
                        const uint32_t to = many + __builtin_amdgcn_mbcnt_hi((uint32_t)(reach >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)reach, 0));
                        if (to < kRoom) lds[wave * kRoom + to] = (uint64_t)key_of<TYPE>(v[r][j]) << 32 | place(r, j);
                    }
                    many += (uint32_t)__popcll(reach);
                }
            }
        if (lane == 0) wave_bound[wave] = many;
        __syncthreads();
        uint32_t of_wave[kThreads / 64], all = 0;
        bool over = false;
#pragma unroll
        for (int w = 0; w < kThreads / 64; ++w) {
            of_wave[w] = wave_bound[w];
            over = over || of_wave[w] > kRoom;
            all += of_wave[w];
        }
        if (over) {   // the same in every thread
            __syncthreads();
            uint64_t best = 0;
#pragma unroll
            for (int r = 0; r < RUNS; ++r)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint64_t k = key_of<TYPE>(v[r][j]), key = k << 32 | place(r, j);
                    if (k && key > best) best = key;
                }
            lds[tid] = best;
            if (tid == 0) left = 0;
            __syncthreads();
            const int rank = rank_of(lds, kThreads, best, 1, order_of);
            if (rank == n - 1 && best) part_bound = best;
            __syncthreads();
            const uint64_t bound_key = part_bound;
            if (best && best >= bound_key) {
#pragma unroll
                for (int r = 0; r < RUNS; ++r)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint64_t k = key_of<TYPE>(v[r][j]), key = k << 32 | place(r, j);
                        if (k && key >= bound_key) lds[atomicAdd(&left, 1u)] = key;
                    }
            }
            __syncthreads();
            all = left;
        } else {      // side by side
            constexpr int kEach = kMostTied / kThreads;
            uint64_t mine_of[kEach];
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                uint32_t x = tid + i * kThreads, w = 0;
                if (x >= all) break;
#pragma unroll
                for (int k = 0; k < kThreads / 64 - 1; ++k)
                    if (w == (uint32_t)k && x >= of_wave[k]) {
                        x -= of_wave[k];
                        ++w;
                    }
                mine_of[i] = lds[w * kRoom + x];
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                if (tid + i * kThreads < (int)all) lds[tid + i * kThreads] = mine_of[i];
            __syncthreads();
        }
        constexpr int kMost = N * RUNS * 8 > kMostTied ? N * RUNS * 8 : kMostTied;
        const int count = tighten<kMost / kThreads>(lds, (int)all, 256, n, bounds, &left, [](uint64_t k) { return (uint32_t)(k >> 32); });
        const int per = threads_per(count);
        for (int i = tid / per; i < count; i += kThreads / per) {
            const uint64_t key = lds[i];
            const int rank = rank_of(lds, count, key, per, order_of);
            if (rank < n && (tid & (per - 1)) == 0) publish(mine + rank, key);
        }
        if (tid >= count && tid < n) publish(mine + tid, 0ull);
        if (tid == 0) publish(mine + n, (uint64_t)as_u32(m) << 32 | as_u32(sum));
    }

    // the last workgroup of this entry goes on
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    uint32_t* counter = a.counters + entry * kCounterStep;
    const int lists = a.beams * a.parts;
    if (tid == 0)
        left = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)(lists - 1);
    __syncthreads();
    const bool last = left != 0;
    __syncthreads();
    if (!last) return;

    const uint64_t* records = a.parts_out + (int64_t)entry * lists * record;
    const auto ended = [&](int w) { return a.finished && a.finished[entry * a.beams + w]; };
    // the parts' sums, and at the same time each thread's first list's best
    const uint64_t first_key = tid < lists ? fetch(records + (int64_t)tid * record) : 0;
    for (int i = tid; i < lists; i += kThreads) lds[i] = fetch(records + (int64_t)i * record + n);
    if (tid == 0) left = 0;
    __syncthreads();
    for (int w0 = 0; w0 < a.beams; w0 += kThreads / 16) {   // 16 lanes a beam
        const int w = w0 + tid / 16;
        if (w < a.beams) {
            double off = (double)a.scores[entry * a.beams + w];
            float m = -INFINITY;
            if (!ended(w)) {
                for (int p = tid & 15; p < a.parts; p += 16) m = fmaxf(m, __builtin_bit_cast(float, (uint32_t)(lds[w * a.parts + p] >> 32)));
                m = row_max(m);
                double s = 0.0;
                for (int p = tid & 15; p < a.parts; p += 16) {
                    const uint64_t ms = lds[w * a.parts + p];
                    const float pm = __builtin_bit_cast(float, (uint32_t)(ms >> 32)), ps = __builtin_bit_cast(float, (uint32_t)ms);
                    if (pm > -INFINITY) {   // what the part's exponents were taken from
                        const float c = pm * kLog2e;
                        const double from = fabsf(c) <= kFar ? (double)c : (double)pm * (double)kLog2e;
                        s += (double)(ps * __builtin_amdgcn_exp2f((float)(from - (double)m * (double)kLog2e)));
                    }
                }
                s = row_sum(s);
                // back by the factor that the exponents were taken with; not finite where no logit or an infinite one is there
                off -= log2(s) / (double)kLog2e;
            }
            if ((tid & 15) == 0) {
                offset[w] = off;
                largest[w] = (double)m;
            }
        }
    }
    __syncthreads();

    Candidate* found = reinterpret_cast<Candidate*>(lds);   // lists by their best, later the values that may be chosen
    uint32_t* found_list = reinterpret_cast<uint32_t*>(found + lists);
    const auto candidate = [&](int list, int i, uint64_t key) {
        const int w = list / a.parts;
        Candidate c = {0, 0};
        const double off = offset[w];
        if (!(off - off == 0.0)) return c;                  // not finite: no candidates
        if (ended(w)) {
            if (i == 0 && list == w * a.parts) c = Candidate{key_of(off), (uint64_t)(63 - w) << 52 | (0xFFFFFu - (uint32_t)a.end_token)};
            return c;
        }
        if (key) c = Candidate{key_of(((double)value_of<TYPE>((uint32_t)(key >> 32)) - largest[w]) + off), place_of(w, key)};
        return c;
    };
    const auto kth = [&](int list, int i) { return fetch(records + (int64_t)list * record + i); };
    // a bound that n of the lists' best reach: the n-th of a wavefront's threads
    const Candidate first = tid < lists ? candidate(tid, 0, first_key) : Candidate{0, 0};
    uint64_t best = first.s;
    for (int i = tid + kThreads; i < lists; i += kThreads) {
        const uint64_t c = candidate(i, 0, kth(i, 0)).s;
        best = best > c ? best : c;
    }
    const uint32_t nth = nth_of_wave<32>((uint32_t)(best >> 32), n);
    if (lane == 0) wave_bound[wave] = nth;
    __syncthreads();
    uint32_t reach = wave_bound[0];
#pragma unroll
    for (int w = 1; w < kThreads / 64; ++w) reach = reach > wave_bound[w] ? reach : wave_bound[w];
    const auto enlist = [&](int i, const Candidate& c) {
        if (c.s && (uint32_t)(c.s >> 32) >= reach) {
            const uint32_t at = atomicAdd(&left, 1u);
            found[at] = c;
            found_list[at] = (uint32_t)i;
        }
    };
    enlist(tid, first);
    for (int i = tid + kThreads; i < lists; i += kThreads) enlist(i, candidate(i, 0, kth(i, 0)));
    if (tid == 0) bound = Candidate{0, 0};
    __syncthreads();
    // their order
    const int holders = (int)left, per_holder = threads_per(holders);
    for (int i = tid / per_holder; i < holders; i += kThreads / per_holder) {
        const Candidate c = found[i];
        const int r = rank_of(found, holders, c, per_holder, above);
        if (r < n) order[r] = found_list[i];
        if (r == n - 1) bound = c;
    }
    __syncthreads();
    const int used = holders < n ? holders : n;
    const Candidate least = bound;
    // pair (r, j): value j of the r-th list
    constexpr int kPairs = (N * N + kThreads - 1) / kThreads;
    if (tid == 0) left = 0;
    __syncthreads();
    uint64_t key[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        const int x = tid + i * kThreads, r = x / n, j = x - r * n;
        key[i] = r < used && r + j < n ? kth((int)order[r], j) : 0;
    }
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        const int x = tid + i * kThreads, r = x / n, j = x - r * n;
        if (r >= used || r + j >= n) continue;
        const Candidate c = candidate((int)order[r], j, key[i]);
        if (c.s && !above(least, c)) found[atomicAdd(&left, 1u)] = c;
    }
    __syncthreads();
    finish<(N * (N + 1) / 2 + kThreads - 1) / kThreads>(a, found, (int)left, n, entry, bounds, &left, counter);
}

int64_t parts_of(int vocab, int runs) { return (vocab + runs * kThreads * 8 - 1) / (runs * kThreads * 8); }

// How a beam's vocabulary is cut: parts of RUNS * 2048 values at most, equal
// and whole runs of eight.
struct Cut {
    int runs, parts, slice;
};
Cut cut_of(int64_t rows, int beams, int vocab) {
    Cut c;
    for (c.runs = 1; c.runs < 4; c.runs *= 2) {
        const int64_t parts = parts_of(vocab, c.runs);
        if (rows * parts <= 512 && beams * parts <= kThreads) break;
    }
    c.parts = (int)parts_of(vocab, c.runs);
    c.slice = ((vocab + c.parts - 1) / c.parts + 7) / 8 * 8;
    c.parts = (vocab + c.slice - 1) / c.slice;
    return c;
}

typedef void (*Kernel)(Args);
template <int TYPE, int N>
Kernel pick_runs(int runs) {
    return runs == 4 ? k_beam<TYPE, 4, N> : runs == 2 ? k_beam<TYPE, 2, N> : k_beam<TYPE, 1, N>;
}
template <int TYPE>
Kernel pick(int runs, int choices) {
    return choices <= 16 ? pick_runs<TYPE, 16>(runs) : pick_runs<TYPE, SGEMV_MAX_CHOICES>(runs);
}

bool sizes_ok(int32_t batch, int32_t beams, int32_t vocab, int32_t choices) {
    return batch >= 0 && beams >= 1 && beams <= SGEMV_MAX_BEAMS && vocab >= 1 && vocab <= SGEMV_MAX_VOCAB && choices >= 1 &&
           choices <= SGEMV_MAX_CHOICES;
}

}  // namespace

extern "C" size_t sgemv_beam_workspace_bytes(int32_t batch, int32_t beams, int32_t vocab, int32_t choices) {
    if (!sizes_ok(batch, beams, vocab, choices)) return 0;
    // launches of at most kMaxBatch entries; the last may have few and so a finer cut
    const int64_t entries = batch < kMaxBatch ? batch : kMaxBatch;
    int64_t records = entries * beams * parts_of(vocab, 4);
    const int64_t finer = 512 < entries * beams * parts_of(vocab, 1) ? 512 : entries * beams * parts_of(vocab, 1);
    if (finer > records) records = finer;
    return kSgemvCounterBytes + (size_t)records * (choices + 1) * 8;
}

extern "C" int sgemv_beam_select(const sgemv_beam_args* args, void* stream) {
    if (!args) return SGEMV_EINVAL;
    const sgemv_beam_args& p = *args;
    if (p.type != SGEMV_F16 && p.type != SGEMV_BF16 && p.type != SGEMV_F32) return SGEMV_EINVAL;
    if (!sizes_ok(p.batch, p.beams, p.vocab, p.choices)) return SGEMV_ESIZE;
    if (p.batch == 0) return SGEMV_OK;
    if (!p.logits || !p.scores || !p.tokens || !p.parents || !p.scores_out || !p.workspace) return SGEMV_EINVAL;
    if (p.finished && (p.end_token < 0 || p.end_token >= p.vocab)) return SGEMV_EINVAL;
    const int64_t most = (int64_t)1 << 40;
    if (p.ld_batch < 0 || p.ld_batch > most || p.ld_beam < 0 || p.ld_beam > most) return SGEMV_ESIZE;
    const size_t need = sgemv_beam_workspace_bytes(p.batch, p.beams, p.vocab, p.choices);
    if (p.workspace_bytes < need) return SGEMV_ESIZE;
    const int size = sgemv_size_of(p.type);
    if (!sgemv_aligned(p.logits, (uintptr_t)size) || !sgemv_aligned(p.scores, 4) || !sgemv_aligned(p.tokens, 4) ||
        !sgemv_aligned(p.parents, 4) || !sgemv_aligned(p.scores_out, 4) || !sgemv_aligned(p.workspace, 256))
        return SGEMV_EALIGN;
    const int64_t rows = (int64_t)p.batch * p.beams, chosen = (int64_t)p.batch * p.choices;
    const SgemvRows outs[3] = {{p.tokens, 1, 0, chosen * 4}, {p.parents, 1, 0, chosen * 4}, {p.scores_out, 1, 0, chosen * 4}};
    const SgemvRows ins[4] = {
        {p.logits, 1, 0, ((p.batch - 1) * p.ld_batch + (p.beams - 1) * p.ld_beam + p.vocab) * size},
        {p.scores, 1, 0, rows * 4}, {p.finished, 1, 0, rows}, {p.workspace, 1, 0, (int64_t)need}};
    for (int i = 0; i < 3; ++i) {
        for (const SgemvRows& in : ins)
            if (sgemv_overlap(outs[i], in)) return SGEMV_EINVAL;
        for (int j = i + 1; j < 3; ++j)
            if (sgemv_overlap(outs[i], outs[j])) return SGEMV_EINVAL;
    }
    Args a;
    a.counters = static_cast<uint32_t*>(p.workspace);
    a.parts_out = reinterpret_cast<uint64_t*>(static_cast<uint8_t*>(p.workspace) + kSgemvCounterBytes);
    a.ld_batch = p.ld_batch;
    a.ld_beam = p.ld_beam;
    a.beams = p.beams;
    a.vocab = p.vocab;
    a.choices = p.choices;
    a.end_token = p.end_token;
    for (int64_t b = 0; b < p.batch; b += kMaxBatch) {
        const int64_t entries = p.batch - b < kMaxBatch ? p.batch - b : kMaxBatch;
        const Cut cut = cut_of(entries * p.beams, p.beams, p.vocab);
        a.logits = static_cast<const uint8_t*>(p.logits) + b * p.ld_batch * size;
        a.scores = p.scores + b * p.beams;
        a.finished = p.finished ? p.finished + b * p.beams : nullptr;
        a.tokens = p.tokens + b * p.choices;
        a.parents = p.parents + b * p.choices;
        a.scores_out = p.scores_out + b * p.choices;
        a.parts = cut.parts;
        a.slice = cut.slice;
        const int lists = p.beams * cut.parts, n = p.choices;
        // in LDS: the values of n threads or kMostTied of them (8 bytes); the lists by their best (20); the values that may
        // be chosen (16)
        const int cap = n * cut.runs * 8 > kMostTied ? n * cut.runs * 8 : kMostTied;
        size_t shared = (size_t)cap * 8;
        if (shared < (size_t)lists * 20) shared = (size_t)lists * 20;
        if (shared < (size_t)n * (n + 1) / 2 * 16) shared = (size_t)n * (n + 1) / 2 * 16;
        const Kernel kernel = p.type == SGEMV_F16    ? pick<SGEMV_F16>(cut.runs, n)
                              : p.type == SGEMV_BF16 ? pick<SGEMV_BF16>(cut.runs, n)
                                                     : pick<SGEMV_F32>(cut.runs, n);
        void* kargs[] = {&a};
        const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(kernel), dim3((unsigned)(entries * lists)),
                                             dim3(kThreads), kargs, shared, static_cast<hipStream_t>(stream));
        if (e != hipSuccess) return sgemv_hip_failed((int)e);
    }
    return SGEMV_OK;
}
