// Beam selection: sgemv_beam_select.
//
//   s(w, v) = score[w] + logit[w][v] - log sum_u e^logit[w][u]
//
// One pass over the logits in one launch.  A workgroup takes a part of one
// beam's vocabulary into registers and leaves the part's maximum, its sum of
// exponentials and its best candidates; the last workgroup of a batch entry to
// arrive has every beam's normaliser and picks among the parts' candidates.
//
// The best n of a part: every lane has its best value, and the n-th best of a
// wavefront's 64 is found bit by bit with ballots.  n values reach that bound,
// and so they do the largest of the four wavefronts' bounds; the few dozen
// values that reach it are ranked, each by counting those above it.  Where
// they are too many (sorted or equal logits), the n-th best of all 256 threads
// is taken instead, which the values of n threads only can reach.  The same
// bound over the parts' best values leaves n parts, and of the part that is
// r-th best by its first value only the first n - r can be among the best n.
// Within a beam the logits' order is that of s, and equal values go by their
// place, so every key is unique and the answer does not depend on timing.
//
// Bound by HBM for a batch of large vocabularies, by latency for one request.
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
constexpr int kCounterStep = 16;       // words between arrival counters
constexpr size_t kCounterBytes = (size_t)kMaxBatch * kCounterStep * 4;

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
    int32_t cap, lists;           // candidates and lists that LDS has room for
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

template <int TYPE>
__device__ __forceinline__ void load8(const uint8_t* p, float (&v)[8]) {
    if (TYPE == SGEMV_F32) {
        const uint4_t a = *reinterpret_cast<const uint4_w*>(p), b = *reinterpret_cast<const uint4_w*>(p + 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = widen<TYPE>(a[i]);
            v[4 + i] = widen<TYPE>(b[i]);
        }
    } else {
        const uint4_t a = *reinterpret_cast<const uint4_h*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = widen<TYPE>(a[i] & 0xFFFFu);
            v[2 * i + 1] = widen<TYPE>(a[i] >> 16);
        }
    }
}

template <class V>
__device__ __forceinline__ V wave_max(V v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const V o = __shfl_xor(v, d);
        v = v > o ? v : o;
    }
    return v;
}
template <class V>
__device__ __forceinline__ V wave_sum(V v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
    return v;
}

// One beam's candidate: beam, logit and token in one number, larger for the one to prefer among equal s.
__device__ __forceinline__ uint64_t place_of(int beam, uint64_t key) {
    return (uint64_t)(63 - beam) << 52 | (key >> 32) << 20 | (0xFFFFFu - (~(uint32_t)key & 0xFFFFFu));
}

__device__ __forceinline__ int lanes(bool v) { return __popcll(__ballot(v)); }

// The n-th best of the wavefront's 64 keys (value above place; 0 is none), or 0
// where fewer than n are there.
template <int TYPE>
__device__ __forceinline__ uint64_t nth_of_wave(uint64_t key, int n) {
    const uint32_t value = (uint32_t)(key >> 32), place = (uint32_t)key;
    uint32_t t = 0, p = 0;
    for (int bit = 31 - kFixed<TYPE>; bit >= 0; --bit)
        if (lanes(value >= (t | 1u << bit)) >= n) t |= 1u << bit;
    if (t == 0) return 0;
    const int need = n - lanes(value > t);
    if (lanes(value == t) > need)
        for (int bit = 31; bit >= 0; --bit)
            if (lanes(value == t && place >= (p | 1u << bit)) >= need) p |= 1u << bit;
    return (uint64_t)t << 32 | p;
}

struct Candidate {
    uint64_t s, place;
};
__device__ __forceinline__ bool above(const Candidate& a, const Candidate& b) {
    return a.s > b.s || (a.s == b.s && a.place > b.place);
}

// RUNS runs of eight values a thread.
template <int TYPE, int RUNS>
__global__ __launch_bounds__(kThreads) void k_beam(Args a) {
    extern __shared__ uint64_t lds[];
    __shared__ float part_m[kThreads / 64], part_s[kThreads / 64];
    __shared__ double offset[SGEMV_MAX_BEAMS];
    __shared__ uint32_t left;
    __shared__ uint64_t wave_bound[kThreads / 64];
    __shared__ Candidate bound;
    constexpr int ES = TYPE == SGEMV_F32 ? 4 : 2;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = a.choices;
    const int part = blockIdx.x % a.parts, beam = (int)(blockIdx.x / a.parts) % a.beams;
    const int entry = (int)(blockIdx.x / a.parts) / a.beams;
    const int record = n + 1;
    uint64_t* mine = a.parts_out + (int64_t)blockIdx.x * record;

    const bool done = a.finished && a.finished[entry * a.beams + beam];
    if (!done) {
        const uint8_t* row = a.logits + (entry * a.ld_batch + beam * a.ld_beam) * ES;
        const int first = part * a.slice, end = first + a.slice < a.vocab ? first + a.slice : a.vocab;
        float v[RUNS][8];
#pragma unroll
        for (int r = 0; r < RUNS; ++r) {
            const int at = first + (r * kThreads + tid) * 8;
            if (at + 8 <= end) {
                load8<TYPE>(row + (int64_t)at * ES, v[r]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[r][j] = at + j >= end ? -INFINITY
                              : TYPE == SGEMV_F32
                                  ? widen<TYPE>(reinterpret_cast<const uint32_t*>(row)[at + j])
                                  : widen<TYPE>(reinterpret_cast<const uint16_t*>(row)[at + j]);
            }
        }
        float top = -INFINITY;
        int top_at = 0;   // the first of a thread's values that is its largest
#pragma unroll
        for (int r = 0; r < RUNS; ++r)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (v[r][j] > top) {
                    top = v[r][j];
                    top_at = first + (r * kThreads + tid) * 8 + j;
                }
        const float wm = wave_max(top);
        // a thread's best, with the place turned round so that the lowest wins among equals
        const uint32_t top_key = key_of<TYPE>(top);
        const uint64_t best = top_key ? (uint64_t)top_key << 32 | ~(uint32_t)top_at : 0ull;
        const uint64_t nth = nth_of_wave<TYPE>(best, n);
        if (lane == 0) {
            part_m[wave] = wm;
            wave_bound[wave] = nth;
        }
        if (tid == 0) left = 0;
        __syncthreads();
        float m = part_m[0];
        uint64_t least = wave_bound[0];
#pragma unroll
        for (int w = 1; w < kThreads / 64; ++w) {
            m = fmaxf(m, part_m[w]);
            least = least > wave_bound[w] ? least : wave_bound[w];
        }
        const float from = m == -INFINITY ? 0.0f : m;
        float sum = 0.0f;
        int reach = 0;
#pragma unroll
        for (int r = 0; r < RUNS; ++r)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float d = v[r][j] - from;
                // log2(e) in two parts: what its rounding takes from far logits would add up
                const float e = __builtin_amdgcn_exp2f(fmaf(d, 1.44269502e+0f, d * 1.92596299e-8f));
                if (v[r][j] == v[r][j]) sum += e;
                const uint64_t key = (uint64_t)key_of<TYPE>(v[r][j]) << 32 | ~(uint32_t)(first + (r * kThreads + tid) * 8 + j);
                reach += key >> 32 && key >= least;
            }
        sum = wave_sum(sum);
        reach = wave_sum(reach);
        if (lane == 0) {
            part_s[wave] = sum;
            if (reach) atomicAdd(&left, (uint32_t)reach);
        }
        __syncthreads();
        const bool many = left > (uint32_t)(2 * a.cap);
        __syncthreads();
        if (many) {
            if (tid == 0) wave_bound[0] = 0;
            lds[tid] = best;
            __syncthreads();
            int rank = 0;
            for (int i = 0; i < kThreads; ++i) rank += lds[i] > best;
            if (rank == n - 1 && best) wave_bound[0] = best;
            __syncthreads();
            least = wave_bound[0];
        }
        if (tid == 0) left = 0;
        __syncthreads();
        if (best && best >= least) {
#pragma unroll
            for (int r = 0; r < RUNS; ++r)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint64_t key = (uint64_t)key_of<TYPE>(v[r][j]) << 32 | ~(uint32_t)(first + (r * kThreads + tid) * 8 + j);
                    if (key >> 32 && key >= least) lds[atomicAdd(&left, 1u)] = key;
                }
        }
        __syncthreads();
        const int count = (int)left;
        for (int i = tid; i < count; i += kThreads) {
            const uint64_t key = lds[i];
            int above_it = 0;
            for (int k = 0; k < count; ++k) above_it += lds[k] > key;
            if (above_it < n) publish(mine + above_it, key);
        }
        if (tid >= count && tid < n) publish(mine + tid, 0ull);
        if (tid == 0) {
            float s = part_s[0];
#pragma unroll
            for (int w = 1; w < kThreads / 64; ++w) s += part_s[w];
            publish(mine + n, (uint64_t)__builtin_bit_cast(uint32_t, m) << 32 | __builtin_bit_cast(uint32_t, s));
        }
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
    for (int w = wave; w < a.beams; w += kThreads / 64) {
        const float score = a.scores[entry * a.beams + w];
        double off = (double)score;
        if (!(a.finished && a.finished[entry * a.beams + w])) {
            float m = -INFINITY;
            for (int p = lane; p < a.parts; p += 64)
                m = fmaxf(m, __builtin_bit_cast(float, (uint32_t)(fetch(records + (int64_t)(w * a.parts + p) * record + n) >> 32)));
            m = wave_max(m);
            double s = 0.0;
            for (int p = lane; p < a.parts; p += 64) {
                const uint64_t ms = fetch(records + (int64_t)(w * a.parts + p) * record + n);
                const float pm = __builtin_bit_cast(float, (uint32_t)(ms >> 32)), ps = __builtin_bit_cast(float, (uint32_t)ms);
                if (pm > -INFINITY) s += (double)ps * exp((double)pm - (double)m);
            }
            s = wave_sum(s);
            off = (double)score - ((double)m + log(s));   // not finite where no logit or an infinite one is there
        }
        if (lane == 0) offset[w] = off;
    }
    if (tid == 0) {
        left = 0;
        bound = Candidate{0, 0};
    }
    __syncthreads();

    Candidate* found = reinterpret_cast<Candidate*>(lds);                       // cap of them
    Candidate* head = found + a.cap;                                            // the parts' first values
    uint32_t* head_list = reinterpret_cast<uint32_t*>(head + a.lists);
    const auto candidate = [&](int list, int i) {
        const int w = list / a.parts;
        Candidate c = {0, 0};
        const double off = offset[w];
        if (!(off - off == 0.0)) return c;                                      // not finite: no candidates
        if (a.finished && a.finished[entry * a.beams + w]) {
            if (i == 0 && list == w * a.parts) c = Candidate{key_of(off), (uint64_t)(63 - w) << 52 | (0xFFFFFu - (uint32_t)a.end_token)};
            return c;
        }
        const uint64_t key = fetch(records + (int64_t)list * record + i);
        if (key) c = Candidate{key_of((double)value_of<TYPE>((uint32_t)(key >> 32)) + off), place_of(w, key)};
        return c;
    };
    // a bound on the parts' first values, and those that reach it
    Candidate best = {0, 0};
    for (int i = tid; i < lists; i += kThreads) {
        const Candidate c = candidate(i, 0);
        if (above(c, best)) best = c;
    }
    found[tid] = best;
    __syncthreads();
    int rank = 0;
    for (int i = 0; i < kThreads; ++i) rank += above(found[i], best);
    if (rank == n - 1 && best.s) bound = best;
    __syncthreads();
    Candidate least = bound;
    for (int i = tid; i < lists; i += kThreads) {
        if (!(rank < n && best.s)) break;
        const Candidate c = candidate(i, 0);
        if (c.s && !above(least, c)) {
            const uint32_t at = atomicAdd(&left, 1u);
            head[at] = c;
            head_list[at] = (uint32_t)i;
        }
    }
    __syncthreads();
    const int heads = (int)left;
    __syncthreads();
    // their order: of the r-th, the first n - r values can be among the best n
    uint32_t* order = reinterpret_cast<uint32_t*>(found);
    for (int i = tid; i < heads; i += kThreads) {
        const Candidate c = head[i];
        int r = 0;
        for (int k = 0; k < heads; ++k) r += above(head[k], c);
        if (r < n) order[r] = head_list[i];
        if (r == n - 1) bound = c;
    }
    if (tid == 0) left = 0;
    __syncthreads();
    const int used = heads < n ? heads : n;
    least = bound;
    // pair (r, j): value j of the r-th part.  A thread's parts are read before found, which order shares, is written
    constexpr int kPairs = (SGEMV_MAX_CHOICES * SGEMV_MAX_CHOICES + kThreads - 1) / kThreads;
    uint32_t list[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        const int x = tid + i * kThreads;
        list[i] = x < used * n ? order[x / n] : 0;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        const int x = tid + i * kThreads, r = x / n, j = x - r * n;
        if (r >= used || r + j >= n) continue;
        const Candidate c = candidate((int)list[i], j);
        if (c.s && !above(least, c)) found[atomicAdd(&left, 1u)] = c;
    }
    __syncthreads();
    const int count = (int)left;
    const int64_t out = (int64_t)entry * n;
    for (int i = tid; i < count; i += kThreads) {
        const Candidate c = found[i];
        int r = 0;
        for (int k = 0; k < count; ++k) r += above(found[k], c);
        if (r < n) {
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

// How a beam's vocabulary is cut: parts of RUNS * 2048 values at most, equal
// and whole runs of eight.
struct Cut {
    int runs, parts, slice;
};
Cut cut_of(int64_t rows, int vocab) {
    Cut c;
    const int64_t large = (vocab + 8191) / 8192;
    c.runs = rows * large >= 512 ? 4 : 1;
    const int most = c.runs * kThreads * 8;
    c.parts = (vocab + most - 1) / most;
    c.slice = ((vocab + c.parts - 1) / c.parts + 7) / 8 * 8;
    c.parts = (vocab + c.slice - 1) / c.slice;
    return c;
}

typedef void (*Kernel)(Args);
template <int TYPE>
Kernel pick(int runs) {
    return runs == 4 ? k_beam<TYPE, 4> : k_beam<TYPE, 1>;
}

bool sizes_ok(int32_t batch, int32_t beams, int32_t vocab, int32_t choices) {
    return batch >= 0 && beams >= 1 && beams <= SGEMV_MAX_BEAMS && vocab >= 1 && vocab <= SGEMV_MAX_N && choices >= 1 &&
           choices <= SGEMV_MAX_CHOICES;
}

}  // namespace

extern "C" size_t sgemv_beam_workspace_bytes(int32_t batch, int32_t beams, int32_t vocab, int32_t choices) {
    if (!sizes_ok(batch, beams, vocab, choices)) return 0;
    // launches of at most kMaxBatch entries; the finest cut of any batch up to this one
    const int64_t entries = batch < kMaxBatch ? batch : kMaxBatch;
    const int64_t fine = (vocab + kThreads * 8 - 1) / (kThreads * 8), coarse = (vocab + 8191) / 8192;
    int64_t records = entries * beams * coarse;
    const int64_t few = 511 < entries * beams * coarse ? 511 : entries * beams * coarse;   // rows * coarse of a fine cut
    if (few / coarse * fine > records) records = few / coarse * fine;
    return kCounterBytes + (size_t)records * (choices + 1) * 8;
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
    a.parts_out = reinterpret_cast<uint64_t*>(static_cast<uint8_t*>(p.workspace) + kCounterBytes);
    a.ld_batch = p.ld_batch;
    a.ld_beam = p.ld_beam;
    a.beams = p.beams;
    a.vocab = p.vocab;
    a.choices = p.choices;
    a.end_token = p.end_token;
    for (int64_t b = 0; b < p.batch; b += kMaxBatch) {
        const int64_t entries = p.batch - b < kMaxBatch ? p.batch - b : kMaxBatch;
        const Cut cut = cut_of(entries * p.beams, p.vocab);
        a.logits = static_cast<const uint8_t*>(p.logits) + b * p.ld_batch * size;
        a.scores = p.scores + b * p.beams;
        a.finished = p.finished ? p.finished + b * p.beams : nullptr;
        a.tokens = p.tokens + b * p.choices;
        a.parents = p.parents + b * p.choices;
        a.scores_out = p.scores_out + b * p.choices;
        a.parts = cut.parts;
        a.slice = cut.slice;
        const int lists = p.beams * cut.parts, n = p.choices;
        a.cap = n * (n + 1) / 2 > kThreads ? n * (n + 1) / 2 : kThreads;
        if (a.cap * 2 < n * cut.runs * 8) a.cap = n * cut.runs * 4;   // the values of n threads, half as large
        a.lists = n * ((lists + kThreads - 1) / kThreads);
        const size_t shared = (size_t)a.cap * 16 + (size_t)a.lists * 20;
        const Kernel kernel = p.type == SGEMV_F16    ? pick<SGEMV_F16>(cut.runs)
                              : p.type == SGEMV_BF16 ? pick<SGEMV_BF16>(cut.runs)
                                                     : pick<SGEMV_F32>(cut.runs);
        void* kargs[] = {&a};
        const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(kernel), dim3((unsigned)(entries * lists)),
                                             dim3(kThreads), kargs, shared, static_cast<hipStream_t>(stream));
        if (e != hipSuccess) return sgemv_hip_failed((int)e);
    }
    return SGEMV_OK;
}
