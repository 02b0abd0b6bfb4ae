// Pages of a cache: sgemv_pages_fork, sgemv_pages_compact, sgemv_pages_copy.
//
// Whole numbers and copies.  A fork adds (children - 1) to the count of every
// page of every row, once for all of a row's children, and then plans: who
// copies a shared page, how many pages each row needs (a sum over the rows
// before it), which free pages there are, lowest first.  Where the counts fit
// one workgroup's LDS, that is one workgroup's work; else a workgroup for each
// row adds, and the last one to arrive plans (after a launch that copies the
// counts, where they go to another array).  The last launch writes tables,
// slots and lengths, and copies.  A compaction counts the used pages of every
// 4096, then ranks movers and free places with those sums, then renames and
// copies.
//
// Copies are bound by HBM: 16 bytes a lane, every pair, layer, keys and values
// cut into pieces of 16 KiB over one fixed grid, since only the device knows
// how many pairs there are (1500 pages, a quarter of them moved, 389 MB read and
// written: 89 us, of which the copies 80, 4.9 TB/s).  The plan is bound by
// latency, a few dependent loads: 4 rows 5.3 us in LDS and 4.6 for the copies and
// tables, 256 rows 11.5 and 11.5 (together 15 and 26 by the plan in memory).  In
// large pools the last workgroup's search for free pages, from page 0 on, is nearly
// all of it: 64 rows that need a page each in a pool of 20000 pages, 95 % of them
// used at the low ids, take 27 us, of 200000 152, of a million 713.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "kv.h"

namespace {

typedef uint32_t uint2_t __attribute__((ext_vector_type(2)));
typedef uint32_t uint4_t __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kBlock = 4096;               // pages of a block of a compaction
constexpr int kDeep = 4;                   // vectors of a thread and piece
constexpr int kPiece = kThreads * kDeep;   // vectors of a piece of a copy

constexpr int kSmallThreads = 1024;        // of a plan in LDS, and its most rows
constexpr int kSmallPages = 6144;          // 8 bytes of LDS each
constexpr int kSmallEntries = 1 << 16;     // of its table

// What the kernels copy: one geometry, the addresses of every layer.
struct Copy {
    int64_t k_page, k_token, k_head, v_page, v_token, v_head;   // bytes
    SgemvDiv vectors, heads, tokens;   // vectors of a head's row, heads, tokens of a page
    int32_t layers, pages, page_size;
    int32_t pieces;                    // of one page, keys or values
    int32_t wide;                      // 16-byte vectors, else 8
    int32_t heads_outside;             // heads before tokens in memory
    uint8_t* k[SGEMV_MAX_LAYERS];
    uint8_t* v[SGEMV_MAX_LAYERS];
};

// A row after a fork: what it took over, by how much it grows, its first fresh
// page (its place in the list of free pages; before that is known, the page
// that it may have to copy) and whether that one is a copy.
struct Row {
    int32_t length, grow, start, copied;
};

struct Fork {
    const int32_t *table, *lengths, *refs, *parents, *grow;
    int32_t *table_out, *lengths_out, *refs_out, *slots, *pairs, *count, *status;
    uint32_t* counter;
    int32_t *staged, *free_list, *mark;   // mark: growing rows of a page, the highest of them
    Row* row;
    int64_t ld_table, ld_table_out;
    SgemvDiv page;
    int32_t rows, max_pages, pages, max_grow;
};

struct Compact {
    const int32_t *table, *lengths, *refs;
    int32_t *table_out, *refs_out, *pairs, *count;
    uint32_t* counter;
    int32_t *before, *target, *source, *rank;   // used pages before each block (and in all), free places, movers, a mover's rank
    int64_t ld_table, ld_table_out;
    SgemvDiv page;
    int32_t rows, max_pages, pages, blocks;
};

__device__ __forceinline__ int divide(int n, const SgemvDiv& d) { return (int)(((uint64_t)(uint32_t)n * d.m) >> d.s); }
__device__ __forceinline__ int parts(int n, const SgemvDiv& d) { return n ? divide(n - 1, d) + 1 : 0; }

// What workgroups of one launch tell each other goes past the caches of an XCD.
__device__ __forceinline__ int peek(const int32_t* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ void poke(int32_t* p, int v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ void add(int32_t* p, int v) { __hip_atomic_fetch_add(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

// Sum over the workgroup's threads before this one; `all` gets the whole sum.
template <int THREADS = kThreads>
__device__ __forceinline__ int block_before(int v, int* shared, int& all) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int scan = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int up = __shfl_up(scan, d);
        if (lane >= d) scan += up;
    }
    __syncthreads();   // an earlier sum has been read
    if (lane == 63) shared[wave] = scan;
    __syncthreads();
    int before = scan - v;
    all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) {
        if (w < wave) before += shared[w];
        all += shared[w];
    }
    return before;
}

// Whether the calling workgroup is the last of n; resets the counter.
__device__ __forceinline__ bool last_of(uint32_t* counter, int n, int* shared) {
    __builtin_amdgcn_s_waitcnt(0);   // this thread's stores and atomics acknowledged
    __syncthreads();                 // ... and every thread's
    if (threadIdx.x == 0) {
        const bool last = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)(n - 1);
        if (last) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        shared[0] = last;
    }
    __syncthreads();
    const bool last = shared[0] != 0;
    __syncthreads();
    return last;
}

// ONCE: whole pages, which nobody reads again soon, past the caches (1500 pages of 64 tokens, a quarter of them moved:
// 97.5 us, 88.4 so; parts of pages that are read next: 26.5, 28.8 so).
template <bool ONCE, class T>
__device__ __forceinline__ void copy_piece(const Copy& c, bool keys, uint8_t* base, int source, int target, int tokens, int first) {
    const int64_t page = keys ? c.k_page : c.v_page, token = keys ? c.k_token : c.v_token, head = keys ? c.k_head : c.v_head;
    const uint8_t* from = base + source * page;
    uint8_t* to = base + target * page;
    const int per = (int)c.vectors.d, rows = (int)c.heads.d * (c.heads_outside ? c.page_size : tokens);
    T got[kDeep];
    int64_t at[kDeep];
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
        const int x = first + i * kThreads + (int)threadIdx.x;
        const int r = divide(x, c.vectors), piece = x - r * per;
        int t, h;
        if (c.heads_outside) {
            h = divide(r, c.tokens);
            t = r - h * c.page_size;
        } else {
            t = divide(r, c.heads);
            h = r - t * (int)c.heads.d;
        }
        at[i] = r < rows && t < tokens ? t * token + h * head + piece * (int64_t)sizeof(T) : -1;
        if (at[i] >= 0) {
            const T* p = reinterpret_cast<const T*>(from + at[i]);
            got[i] = ONCE ? __builtin_nontemporal_load(p) : *p;
        }
    }
#pragma unroll
    for (int i = 0; i < kDeep; ++i)
        if (at[i] >= 0) {
            T* p = reinterpret_cast<T*>(to + at[i]);
            if (ONCE) __builtin_nontemporal_store(got[i], p);
            else *p = got[i];
        }
}

// Pieces of all pairs over the grid; pair(j, source, target, tokens).
template <bool ONCE, class F>
__device__ __forceinline__ void copy_pairs(const Copy& c, int count, F pair) {
    const int64_t per = (int64_t)c.layers * 2 * c.pieces, all = per * count;
    for (int64_t x = blockIdx.x; x < all; x += gridDim.x) {
        const int j = (int)(x / per);
        int rest = (int)(x - j * per);
        const int layer = rest / (2 * c.pieces);
        rest -= layer * 2 * c.pieces;
        const bool keys = rest < c.pieces;
        const int first = (keys ? rest : rest - c.pieces) * kPiece;
        int source, target, tokens;
        pair(j, source, target, tokens);
        if (tokens > c.page_size) tokens = c.page_size;
        if ((uint32_t)source >= (uint32_t)c.pages || (uint32_t)target >= (uint32_t)c.pages || tokens <= 0 || source == target) continue;
        uint8_t* base = keys ? c.k[layer] : c.v[layer];
        if (c.wide) copy_piece<ONCE, uint4_t>(c, keys, base, source, target, tokens, first);
        else copy_piece<ONCE, uint2_t>(c, keys, base, source, target, tokens, first);
    }
}

__global__ __launch_bounds__(kThreads) void k_copy(Copy c, const int32_t* pairs, const int32_t* count, int most) {
    int n = most;
    if (count) n = count[0] < most ? count[0] : most;
    if (n > 0)
        copy_pairs<false>(c, n, [&](int j, int& source, int& target, int& tokens) {
            source = pairs[3 * (int64_t)j];
            target = pairs[3 * (int64_t)j + 1];
            tokens = pairs[3 * (int64_t)j + 2];
        });
}

__global__ __launch_bounds__(kThreads) void k_move(const int32_t* from, int32_t* to, int n) {
    const int i = blockIdx.x * kThreads + threadIdx.x;
    if (i < n) to[i] = from[i];
}

__device__ __forceinline__ int length_of(const Fork& a, int row) {
    const int n = a.lengths[row];
    return n < 0 || n > a.max_pages * (int)a.page.d ? 0 : n;
}
// Length that row r takes over.
__device__ __forceinline__ int inherited(const Fork& a, int r, int& parent) {
    parent = a.parents ? a.parents[r] : r;
    if ((uint32_t)parent >= (uint32_t)a.rows) {
        parent = r;
        return 0;
    }
    return length_of(a, parent);
}

__global__ __launch_bounds__(kThreads) void k_fork(Fork a) {
    __shared__ int shared[kThreads / 64];
    __shared__ int bad_rows;
    const int tid = threadIdx.x;
    if (a.parents) {
        const int r = blockIdx.x;
        int children = 0;
        for (int i = tid; i < a.rows; i += kThreads) children += a.parents[i] == r;
        int all;
        block_before(children, shared, all);
        const int32_t* mine = a.table + r * a.ld_table;
        if (all != 1) {
            const int used = parts(length_of(a, r), a.page);
            for (int c = tid; c < used; c += kThreads) {
                const int id = mine[c];
                if ((uint32_t)id < (uint32_t)a.pages) add(a.refs_out + id, all - 1);
            }
        }
        if (a.staged) {   // the table is written in place: what is taken over is kept aside
            int parent;
            const int used = parts(inherited(a, r, parent), a.page);
            const int32_t* from = a.table + parent * a.ld_table;
            for (int c = tid; c < used; c += kThreads) a.staged[r * (int64_t)a.max_pages + c] = from[c];
        }
        if (!last_of(a.counter, a.rows, shared)) return;
    }

    // the plan: a thread has `each` rows in a row
    constexpr int kDeepScan = 8;
    const int each = (a.rows + kThreads - 1) / kThreads, r0 = tid * each;
    const int r1 = r0 + each < a.rows ? r0 + each : a.rows;
    if (tid == 0) bad_rows = 0;
    __syncthreads();
    for (int r = r0; r < r1; ++r) {
        int parent;
        const int grow = a.grow ? a.grow[r] : 0, length = inherited(a, r, parent), at = divide(length, a.page);
        int id = -1;   // the partly filled last page of a growing row
        if (grow > 0 && at * (int)a.page.d != length) id = a.table[parent * a.ld_table + at];
        if ((uint32_t)id >= (uint32_t)a.pages) id = -1;
        if (grow < 0 || (a.slots && grow > a.max_grow) || (int64_t)length + grow > (int64_t)a.max_pages * (int)a.page.d)
            atomicAdd(&bad_rows, 1);
        if (id >= 0) {
            poke(a.mark + 2 * (int64_t)id, 0);
            poke(a.mark + 2 * (int64_t)id + 1, -1);
        }
        a.row[r] = Row{length, grow, id, 0};
    }
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    for (int r = r0; r < r1; ++r) {
        const int id = a.row[r].start;
        if (id >= 0) {
            add(a.mark + 2 * (int64_t)id, 1);
            __hip_atomic_fetch_max(a.mark + 2 * (int64_t)id + 1, r, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    }
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    const bool bad = bad_rows != 0;
    int need = 0, copied = 0;
    for (int r = r0; r < r1 && !bad; ++r) {
        Row row = a.row[r];
        if (row.start >= 0) {   // a shared page is copied, but by its last holder where all of them grow
            const int32_t* mark = a.mark + 2 * (int64_t)row.start;
            const int held = peek(a.refs_out + row.start);
            row.copied = held > 1 && !(peek(mark) == held && peek(mark + 1) == r);
        }
        copied += row.copied;
        need += row.copied + parts(row.length + row.grow, a.page) - parts(row.length, a.page);
        a.row[r].copied = row.copied;
    }
    int needed, pairs;
    int start = block_before(need, shared, needed);
    int pair = block_before(copied, shared, pairs);
    // the lowest free pages
    int have = 0;
    for (int64_t base = 0; base < a.pages && have < needed; base += kThreads * kDeepScan) {
        const int64_t at = base + tid * kDeepScan;
        int free_here[kDeepScan], n = 0;
#pragma unroll
        for (int i = 0; i < kDeepScan; ++i) free_here[i] = peek(a.refs_out + (at + i < a.pages ? at + i : a.pages - 1));
#pragma unroll
        for (int i = 0; i < kDeepScan; ++i) {
            free_here[i] = at + i < a.pages && free_here[i] <= 0;
            n += free_here[i];
        }
        int all, rank = have + block_before(n, shared, all);
#pragma unroll
        for (int i = 0; i < kDeepScan; ++i)
            if (free_here[i]) {
                if (rank < needed) a.free_list[rank] = (int32_t)(at + i);
                ++rank;
            }
        have += all;
    }
    const int missing = needed > have ? needed - have : 0;
    const bool grows = !bad && missing == 0;
    if (tid == 0) {
        a.status[0] = missing;
        a.status[1] = bad_rows;
        a.count[0] = grows ? pairs : 0;
    }
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();   // the fresh pages, by this workgroup's other threads
    for (int r = r0; r < r1; ++r) {
        Row row = a.row[r];
        const int id = row.start;
        row.start = start;
        if (grows) {
            const int fresh = row.copied + parts(row.length + row.grow, a.page) - parts(row.length, a.page);
            for (int i = 0; i < fresh; ++i) poke(a.refs_out + a.free_list[start + i], 1);
            if (row.copied) {
                add(a.refs_out + id, -1);
                a.pairs[3 * (int64_t)pair] = id;
                a.pairs[3 * (int64_t)pair + 1] = a.free_list[start];
                a.pairs[3 * (int64_t)pair + 2] = row.length - divide(row.length, a.page) * (int)a.page.d;
                ++pair;
            }
            start += fresh;
        } else {
            row.grow = row.copied = 0;
        }
        a.row[r] = row;
    }
    for (int i = (grows ? pairs : 0) + tid; i < a.rows; i += kThreads)
#pragma unroll
        for (int k = 0; k < 3; ++k) a.pairs[3 * (int64_t)i + k] = -1;
}

// The same by one workgroup, a thread for each row, with the counts in LDS (and beside them a word for every page: how many
// growing rows have it, and the highest of them plus one).
__global__ __launch_bounds__(kSmallThreads) void k_fork_small(Fork a, SgemvDiv width) {
    extern __shared__ int counts[];
    __shared__ int shared[kSmallThreads / 64], children[kSmallThreads], lengths[kSmallThreads], parents[kSmallThreads];
    __shared__ int bad_rows;
    uint32_t* mark = reinterpret_cast<uint32_t*>(counts + a.pages);
    const int tid = threadIdx.x;
    const bool is_row = tid < a.rows;
    for (int i = tid; i < a.pages; i += kSmallThreads) counts[i] = a.refs[i];
    int parent = tid, grow = 0, own = 0;
    if (is_row) {
        if (a.parents) parent = a.parents[tid];
        if (a.grow) grow = a.grow[tid];
        own = length_of(a, tid);
    }
    children[tid] = 0;
    lengths[tid] = own;
    if (tid == 0) bad_rows = 0;
    __syncthreads();
    const bool alive = is_row && (uint32_t)parent < (uint32_t)a.rows;
    const int length = alive ? lengths[parent] : 0;
    parents[tid] = alive ? parent : tid;
    if (alive) atomicAdd(&children[parent], 1);
    const int at = divide(length, a.page);
    int id = -1;   // the partly filled last page of a growing row
    if (grow > 0 && at * (int)a.page.d != length) id = a.table[parent * a.ld_table + at];
    if ((uint32_t)id >= (uint32_t)a.pages) id = -1;
    if (is_row && (grow < 0 || (a.slots && grow > a.max_grow) || (int64_t)length + grow > (int64_t)a.max_pages * (int)a.page.d))
        atomicAdd(&bad_rows, 1);
    if (id >= 0) mark[id] = 0;
    __syncthreads();
    if (a.parents) {
        constexpr int kDeepRows = 4;
        const int all = a.rows * a.max_pages;
        for (int x0 = tid; x0 < all; x0 += kSmallThreads * kDeepRows) {
            int own_id[kDeepRows], more[kDeepRows], taken[kDeepRows];
#pragma unroll
            for (int i = 0; i < kDeepRows; ++i) {
                const int x = x0 + i * kSmallThreads, r = x < all ? divide(x, width) : 0, c = x - r * a.max_pages;
                more[i] = x < all && c < parts(lengths[r], a.page) ? children[r] - 1 : 0;
                own_id[i] = more[i] ? a.table[r * a.ld_table + c] : -1;
                if (a.staged && x < all) taken[i] = a.table[parents[r] * a.ld_table + c];
            }
#pragma unroll
            for (int i = 0; i < kDeepRows; ++i) {
                if ((uint32_t)own_id[i] < (uint32_t)a.pages) atomicAdd(&counts[own_id[i]], more[i]);
                if (a.staged && x0 + i * kSmallThreads < all) a.staged[x0 + i * kSmallThreads] = taken[i];
            }
        }
    }
    if (id >= 0) atomicAdd(&mark[id], 1u << 16);
    __syncthreads();
    if (id >= 0) atomicMax(&mark[id], (mark[id] & 0xFFFF0000u) | (uint32_t)(tid + 1));
    __syncthreads();
    const bool bad = bad_rows != 0;
    int copied = 0, need = 0;
    if (is_row && !bad) {
        if (id >= 0) copied = counts[id] > 1 && !((int)(mark[id] >> 16) == counts[id] && (int)(mark[id] & 0xFFFFu) == tid + 1);
        need = copied + parts(length + grow, a.page) - parts(length, a.page);
    }
    int needed, pairs, have = 0;
    const int start = block_before<kSmallThreads>(need, shared, needed);
    const int pair = block_before<kSmallThreads>(copied, shared, pairs);
    for (int base = 0; base < a.pages && have < needed; base += kSmallThreads) {
        const bool is_free = base + tid < a.pages && counts[base + tid] <= 0;
        int all;
        const int rank = have + block_before<kSmallThreads>(is_free, shared, all);
        if (is_free && rank < needed) a.free_list[rank] = base + tid;
        have += all;
    }
    const int missing = needed > have ? needed - have : 0;
    const bool grows = !bad && missing == 0;
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();   // the fresh pages, by other threads; the counts have been read
    if (is_row) {
        if (grows) {
            for (int i = 0; i < need; ++i) counts[a.free_list[start + i]] = 1;
            if (copied) {
                atomicSub(&counts[id], 1);
                a.pairs[3 * pair] = id;
                a.pairs[3 * pair + 1] = a.free_list[start];
                a.pairs[3 * pair + 2] = length - at * (int)a.page.d;
            }
        }
        a.row[tid] = grows ? Row{length, grow, start, copied} : Row{length, 0, 0, 0};
    }
    const int listed = grows ? pairs : 0;
    for (int i = 3 * listed + tid; i < 3 * a.rows; i += kSmallThreads) a.pairs[i] = -1;
    if (tid == 0) {
        a.status[0] = missing;
        a.status[1] = bad_rows;
        a.count[0] = listed;
    }
    __syncthreads();
    for (int i = tid; i < a.pages; i += kSmallThreads) a.refs_out[i] = counts[i];
}

__global__ __launch_bounds__(kThreads) void k_fork_write(Fork a, Copy c) {
    copy_pairs<false>(c, a.count[0], [&](int j, int& source, int& target, int& tokens) {
        source = a.pairs[3 * (int64_t)j];
        target = a.pairs[3 * (int64_t)j + 1];
        tokens = a.pairs[3 * (int64_t)j + 2];
    });
    const int64_t stride = (int64_t)gridDim.x * kThreads, from = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const auto entry = [&](int r, const Row& row, int col) {
        const int used = parts(row.length, a.page);
        if (col < used) {
            if (row.copied && col == used - 1) return a.free_list[row.start];
            if (a.staged && a.parents) return a.staged[r * (int64_t)a.max_pages + col];
            int parent = a.parents ? a.parents[r] : r;
            return a.table[parent * a.ld_table + col];   // a length above 0: the parent is a row
        }
        if (col < parts(row.length + row.grow, a.page)) return a.free_list[row.start + row.copied + col - used];
        return -1;
    };
    for (int64_t x = from; x < (int64_t)a.rows * a.max_pages; x += stride) {
        const int r = (int)(x / a.max_pages), col = (int)(x - (int64_t)r * a.max_pages);
        a.table_out[r * a.ld_table_out + col] = entry(r, a.row[r], col);
    }
    for (int64_t x = from; x < a.rows; x += stride) a.lengths_out[x] = a.row[x].length + a.row[x].grow;
    if (a.slots)
        for (int64_t x = from; x < (int64_t)a.rows * a.max_grow; x += stride) {
            const int r = (int)(x / a.max_grow), j = (int)(x - (int64_t)r * a.max_grow);
            const Row row = a.row[r];
            int slot = -1;
            if (j < row.grow) {
                const int token = row.length + j, col = divide(token, a.page), id = entry(r, row, col);
                if ((uint32_t)id < (uint32_t)a.pages) slot = (id - col) * (int)a.page.d + token;
            }
            a.slots[x] = slot;
        }
}

// Used pages from x on, below end and in x's block: this thread's share.  Loads without a branch are in flight at once.
__device__ __forceinline__ int used_in(const Compact& a, int x, int end) {
    int held[kBlock / kThreads], n = 0;
#pragma unroll
    for (int i = 0; i < kBlock / kThreads; ++i) {
        const int at = x + (int)threadIdx.x + i * kThreads;
        held[i] = a.refs[at < end ? at : end - 1];
    }
#pragma unroll
    for (int i = 0; i < kBlock / kThreads; ++i) n += x + (int)threadIdx.x + i * kThreads < end && held[i] > 0;
    return n;
}

__global__ __launch_bounds__(kThreads) void k_count_used(Compact a) {
    __shared__ int shared[kThreads / 64];
    const int tid = threadIdx.x;
    const int n = used_in(a, blockIdx.x * kBlock, a.pages);
    int all;
    block_before(n, shared, all);
    if (tid == 0) poke(a.before + blockIdx.x, all);
    if (!last_of(a.counter, a.blocks, shared)) return;
    int sum = 0;
    for (int base = 0; base < a.blocks; base += kThreads) {
        const int i = base + tid, v = i < a.blocks ? peek(a.before + i) : 0;
        const int before = sum + block_before(v, shared, all);
        if (i < a.blocks) poke(a.before + i, before);
        sum += all;
    }
    if (tid == 0) poke(a.before + a.blocks, sum);
}

__global__ __launch_bounds__(kThreads) void k_rank(Compact a) {
    __shared__ int shared[kThreads / 64];
    const int tid = threadIdx.x;
    constexpr int kEach = kBlock / kThreads;
    const int64_t at = (int64_t)blockIdx.x * kBlock + tid * kEach;
    int held[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) held[i] = a.refs[at + i < a.pages ? at + i : a.pages - 1];
    const int used = a.before[a.blocks], edge = used / kBlock * kBlock;   // the block that the border is in
    int all, stay = used;                                                // used pages below `used`
    if (used < a.pages) {
        block_before(used > edge ? used_in(a, edge, used) : 0, shared, all);
        stay = a.before[edge / kBlock] + all;
    }
    bool in_use[kEach];
    int n = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        in_use[i] = at + i < a.pages && held[i] > 0;
        n += in_use[i];
    }
    int before = a.before[blockIdx.x] + block_before(n, shared, all);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int64_t x = at + i;
        if (x < a.pages) {
            if (x < used) {
                if (!in_use[i]) a.target[x - before] = (int32_t)x;
            } else {
                a.rank[x] = in_use[i] ? before - stay : -1;
                if (in_use[i]) a.source[before - stay] = (int32_t)x;
            }
        }
        before += in_use[i];
    }
    if (blockIdx.x == 0 && tid == 0) a.count[0] = used - stay;
}

__global__ __launch_bounds__(kThreads) void k_compact_write(Compact a, Copy c) {
    const int64_t stride = (int64_t)gridDim.x * kThreads, from = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int used = a.before[a.blocks], moves = a.count[0];
    for (int64_t x = from; x < (int64_t)a.rows * a.max_pages; x += stride) {
        const int r = (int)(x / a.max_pages), col = (int)(x - (int64_t)r * a.max_pages);
        const int length = a.lengths[r];
        const bool fine = length >= 0 && length <= a.max_pages * (int)a.page.d;
        int id = -1;
        if (fine && col < parts(length, a.page)) {
            id = a.table[r * a.ld_table + col];
            if (id >= used && id < a.pages) {
                const int j = a.rank[id];
                if (j >= 0) id = a.target[j];
            }
        }
        a.table_out[r * a.ld_table_out + col] = id;
    }
    for (int64_t x = from; x < a.pages; x += stride) {
        const int j = (int)x;
        int source = -1, target = -1;
        if (j < moves) {
            source = a.source[j];
            target = a.target[j];
            a.refs_out[target] = a.refs[source];
            a.refs_out[source] = 0;
        }
        a.pairs[3 * x] = source;
        a.pairs[3 * x + 1] = target;
        a.pairs[3 * x + 2] = j < moves ? (int)a.page.d : -1;
        if (a.refs_out != a.refs) {   // the pages that stay as they are: used ones in front, free ones behind
            const int held = a.refs[x];
            if ((held > 0) == (x < used)) a.refs_out[x] = held;
        }
    }
    copy_pairs<true>(c, moves, [&](int j, int& source, int& target, int& tokens) {
        source = a.source[j];
        target = a.target[j];
        tokens = (int)a.page.d;
    });
}

constexpr size_t up(size_t n) { return (n + 255) / 256 * 256; }

// SGEMV_OK, or why the caches cannot be copied in together.
int make_copy(const sgemv_kv* caches, int32_t layers, Copy& c) {
    if (layers < 0 || layers > SGEMV_MAX_LAYERS) return SGEMV_ESIZE;
    c.layers = layers;
    if (layers == 0) return SGEMV_OK;
    if (!caches) return SGEMV_EINVAL;
    const sgemv_kv& f = caches[0];
    for (int i = 0; i < layers; ++i) {
        const sgemv_kv& kv = caches[i];
        if (int e = sgemv_check_kv(kv)) return e;
        if (kv.type != f.type || kv.pages != f.pages || kv.page_size != f.page_size || kv.heads != f.heads || kv.dim != f.dim ||
            kv.k_page != f.k_page || kv.k_token != f.k_token || kv.k_head != f.k_head || kv.v_page != f.v_page ||
            kv.v_token != f.v_token || kv.v_head != f.v_head)
            return SGEMV_EINVAL;
        c.k[i] = static_cast<uint8_t*>(kv.k);
        c.v[i] = static_cast<uint8_t*>(kv.v);
    }
    const int es = sgemv_size_of(f.type), row = f.dim * es;
    c.k_page = f.k_page * es; c.k_token = f.k_token * es; c.k_head = f.k_head * es;
    c.v_page = f.v_page * es; c.v_token = f.v_token * es; c.v_head = f.v_head * es;
    // 8-bit rows may be odd multiples of 8 bytes, and so may their addresses
    bool wide = row % 16 == 0;
    for (const int64_t s : {c.k_page, c.k_token, c.k_head, c.v_page, c.v_token, c.v_head}) wide = wide && s % 16 == 0;
    for (int i = 0; i < layers; ++i) wide = wide && sgemv_aligned(c.k[i], 16) && sgemv_aligned(c.v[i], 16);
    c.wide = wide;
    const int vectors = row / (wide ? 16 : 8);
    if ((int64_t)vectors * f.heads * f.page_size > 0x7FFFFFFF - 2 * kPiece) return SGEMV_ESIZE;
    c.vectors = sgemv_div(vectors);
    c.heads = sgemv_div(f.heads);
    c.tokens = sgemv_div(f.page_size);
    c.pages = f.pages;
    c.page_size = f.page_size;
    c.pieces = (int)(((int64_t)vectors * f.heads * f.page_size + kPiece - 1) / kPiece);
    c.heads_outside = f.heads > 1 && f.page_size > 1 && c.k_head > c.k_token;
    return SGEMV_OK;
}

unsigned grid_for(int64_t entries, int64_t most_pieces) {
    int64_t g = (entries + kThreads - 1) / kThreads;
    if (most_pieces > g) g = most_pieces;
    return (unsigned)(g < 1 ? 1 : g > 2048 ? 2048 : g);
}

int launch(const void* kernel, unsigned grid, void** args, void* stream) {
    const hipError_t e = hipLaunchKernel(kernel, dim3(grid), dim3(kThreads), args, 0, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? SGEMV_OK : sgemv_hip_failed((int)e);
}

bool sizes_ok(int32_t rows, int32_t max_pages, int32_t pages) {
    return rows >= 1 && rows <= SGEMV_MAX_ROWS && max_pages >= 1 && pages >= 1 && pages <= (1 << 24) &&
           (int64_t)rows * max_pages <= 0x7FFFFFFF;
}

// What both calls check; `fork` has more operands.
int check(const sgemv_pages_args& p, const sgemv_kv* caches, bool fork, Copy& c) {
    if (!sizes_ok(p.rows, p.max_pages, p.pages)) return SGEMV_ESIZE;
    if (p.page_size < 1 || p.page_size > 65536 || (int64_t)p.pages * p.page_size > 0x7FFFFFFF ||
        (int64_t)p.max_pages * p.page_size > 0x7FFFFFFF - 65536)
        return SGEMV_ESIZE;
    const int64_t most = (int64_t)1 << 40;
    if (p.ld_table < p.max_pages || p.ld_table_out < p.max_pages || p.ld_table > most || p.ld_table_out > most) return SGEMV_ESIZE;
    if (fork && (p.max_grow < 0 || p.max_grow > 65536)) return SGEMV_ESIZE;
    if (!p.table || !p.lengths || !p.refs || !p.table_out || !p.refs_out || !p.pairs || !p.count || !p.workspace) return SGEMV_EINVAL;
    if (fork && (!p.lengths_out || !p.status)) return SGEMV_EINVAL;
    if (int e = make_copy(caches, p.layers, c)) return e;
    if (c.layers && (caches[0].pages != p.pages || caches[0].page_size != p.page_size)) return SGEMV_EINVAL;
    const size_t need = sgemv_pages_workspace_bytes(p.rows, p.max_pages, p.pages);
    if (p.workspace_bytes < need) return SGEMV_ESIZE;
    const void* words[] = {p.table, p.lengths, p.refs, p.table_out, p.refs_out, p.pairs, p.count};
    for (const void* w : words)
        if (!sgemv_aligned(w, 4)) return SGEMV_EALIGN;
    if (fork && (!sgemv_aligned(p.lengths_out, 4) || !sgemv_aligned(p.parents, 4) || !sgemv_aligned(p.grow, 4) ||
                 !sgemv_aligned(p.slots, 4) || !sgemv_aligned(p.status, 4)))
        return SGEMV_EALIGN;
    if (!sgemv_aligned(p.workspace, 256)) return SGEMV_EALIGN;

    const int64_t rows = p.rows;
    const auto table = [&](const void* at, int64_t ld) { return SgemvRows{at, rows, ld * 4, (int64_t)p.max_pages * 4}; };
    const auto flat = [](const void* at, int64_t n) { return SgemvRows{at, 1, 0, n * 4}; };
    const SgemvRows ins[] = {table(p.table, p.ld_table), flat(p.lengths, rows), flat(p.refs, p.pages),
                             flat(fork ? p.parents : nullptr, rows), flat(fork ? p.grow : nullptr, rows),
                             {p.workspace, 1, 0, (int64_t)need}};
    const SgemvRows outs[] = {table(p.table_out, p.ld_table_out), flat(fork ? p.lengths_out : nullptr, rows),
                              flat(p.refs_out, p.pages), flat(p.pairs, 3 * (fork ? rows : (int64_t)p.pages)), flat(p.count, 1),
                              flat(fork && p.max_grow ? p.slots : nullptr, rows * p.max_grow), flat(fork ? p.status : nullptr, 2)};
    for (int i = 0; i < 7; ++i) {
        for (int j = 0; j < 6; ++j) {
            const bool itself = i < 3 && i == j && outs[i].p == ins[j].p && outs[i].step == ins[j].step;
            if (!itself && sgemv_overlap(outs[i], ins[j])) return SGEMV_EINVAL;
        }
        for (int j = i + 1; j < 7; ++j)
            if (sgemv_overlap(outs[i], outs[j])) return SGEMV_EINVAL;
        for (int l = 0; l < c.layers; ++l)
            if (sgemv_overlap(outs[i], sgemv_kv_rows(caches[l], true)) || sgemv_overlap(outs[i], sgemv_kv_rows(caches[l], false)))
                return SGEMV_EINVAL;
    }
    for (const SgemvRows& in : ins)
        for (int l = 0; l < c.layers; ++l)
            if (sgemv_overlap(in, sgemv_kv_rows(caches[l], true)) || sgemv_overlap(in, sgemv_kv_rows(caches[l], false)))
                return SGEMV_EINVAL;
    return SGEMV_OK;
}

}  // namespace

extern "C" size_t sgemv_pages_workspace_bytes(int32_t rows, int32_t max_pages, int32_t pages) {
    if (!sizes_ok(rows, max_pages, pages)) return 0;
    const size_t fork = up((size_t)rows * max_pages * 4) + up((size_t)pages * 4) + up((size_t)pages * 8) + up((size_t)rows * 16);
    const size_t compact = up(((size_t)pages / kBlock + 2) * 4) + 3 * up((size_t)pages * 4);
    return kSgemvCounterBytes + (fork > compact ? fork : compact);
}

extern "C" int sgemv_pages_fork(const sgemv_pages_args* args, const sgemv_kv* caches, void* stream) {
    if (!args) return SGEMV_EINVAL;
    const sgemv_pages_args& p = *args;
    Copy c = {};
    if (int e = check(p, caches, true, c)) return e;
    Fork a;
    uint8_t* w = static_cast<uint8_t*>(p.workspace);
    const auto take = [&](size_t n) {
        uint8_t* at = w;
        w += up(n);
        return at;
    };
    a.counter = reinterpret_cast<uint32_t*>(take(kSgemvCounterBytes));
    a.staged = reinterpret_cast<int32_t*>(take((size_t)p.rows * p.max_pages * 4));
    a.free_list = reinterpret_cast<int32_t*>(take((size_t)p.pages * 4));
    a.mark = reinterpret_cast<int32_t*>(take((size_t)p.pages * 8));
    a.row = reinterpret_cast<Row*>(take((size_t)p.rows * 16));
    if (p.table_out != p.table) a.staged = nullptr;
    a.table = p.table; a.lengths = p.lengths; a.refs = p.refs; a.parents = p.parents; a.grow = p.grow;
    a.table_out = p.table_out; a.lengths_out = p.lengths_out; a.refs_out = p.refs_out;
    a.slots = p.max_grow ? p.slots : nullptr;
    a.pairs = p.pairs; a.count = p.count; a.status = p.status;
    a.ld_table = p.ld_table; a.ld_table_out = p.ld_table_out;
    a.page = sgemv_div(p.page_size);
    a.rows = p.rows; a.max_pages = p.max_pages; a.pages = p.pages; a.max_grow = p.max_grow;
    if (p.rows <= kSmallThreads && p.pages <= kSmallPages && (int64_t)p.rows * p.max_pages <= kSmallEntries) {
        SgemvDiv width = sgemv_div(p.max_pages);
        void* plan[] = {&a, &width};
        const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(k_fork_small), dim3(1), dim3(kSmallThreads), plan,
                                             (size_t)p.pages * 8, static_cast<hipStream_t>(stream));
        if (e != hipSuccess) return sgemv_hip_failed((int)e);
    } else {
        if (p.refs_out != p.refs) {
            void* kargs[] = {(void*)&a.refs, &a.refs_out, &a.pages};
            if (int e = launch(reinterpret_cast<const void*>(k_move), (unsigned)((p.pages + kThreads - 1) / kThreads), kargs, stream)) return e;
        }
        void* plan[] = {&a};
        if (int e = launch(reinterpret_cast<const void*>(k_fork), a.parents ? (unsigned)p.rows : 1u, plan, stream)) return e;
    }
    void* write[] = {&a, &c};
    return launch(reinterpret_cast<const void*>(k_fork_write),
                  grid_for((int64_t)p.rows * p.max_pages, (int64_t)p.rows * c.layers * 2 * c.pieces), write, stream);
}

extern "C" int sgemv_pages_compact(const sgemv_pages_args* args, const sgemv_kv* caches, void* stream) {
    if (!args) return SGEMV_EINVAL;
    const sgemv_pages_args& p = *args;
    Copy c = {};
    if (int e = check(p, caches, false, c)) return e;
    Compact a;
    uint8_t* w = static_cast<uint8_t*>(p.workspace);
    const auto take = [&](size_t n) {
        uint8_t* at = w;
        w += up(n);
        return at;
    };
    a.blocks = (p.pages + kBlock - 1) / kBlock;
    a.counter = reinterpret_cast<uint32_t*>(take(kSgemvCounterBytes));
    a.before = reinterpret_cast<int32_t*>(take(((size_t)p.pages / kBlock + 2) * 4));
    a.target = reinterpret_cast<int32_t*>(take((size_t)p.pages * 4));
    a.source = reinterpret_cast<int32_t*>(take((size_t)p.pages * 4));
    a.rank = reinterpret_cast<int32_t*>(take((size_t)p.pages * 4));
    a.table = p.table; a.lengths = p.lengths; a.refs = p.refs;
    a.table_out = p.table_out; a.refs_out = p.refs_out; a.pairs = p.pairs; a.count = p.count;
    a.ld_table = p.ld_table; a.ld_table_out = p.ld_table_out;
    a.page = sgemv_div(p.page_size);
    a.rows = p.rows; a.max_pages = p.max_pages; a.pages = p.pages;
    void* kargs[] = {&a};
    if (int e = launch(reinterpret_cast<const void*>(k_count_used), (unsigned)a.blocks, kargs, stream)) return e;
    if (int e = launch(reinterpret_cast<const void*>(k_rank), (unsigned)a.blocks, kargs, stream)) return e;
    void* write[] = {&a, &c};
    const int64_t entries = (int64_t)p.rows * p.max_pages > p.pages ? (int64_t)p.rows * p.max_pages : p.pages;
    return launch(reinterpret_cast<const void*>(k_compact_write),
                  grid_for(entries, (int64_t)p.pages * c.layers * 2 * c.pieces), write, stream);
}

extern "C" int sgemv_pages_copy(const sgemv_kv* caches, int32_t layers, const int32_t* pairs, const int32_t* count,
                                int32_t max_pairs, void* stream) {
    Copy c = {};
    if (max_pairs < 0) return SGEMV_ESIZE;
    if (layers < 1) return SGEMV_ESIZE;
    if (int e = make_copy(caches, layers, c)) return e;
    if (max_pairs == 0) return SGEMV_OK;
    if (!pairs) return SGEMV_EINVAL;
    if (!sgemv_aligned(pairs, 4) || !sgemv_aligned(count, 4)) return SGEMV_EALIGN;
    for (int l = 0; l < layers; ++l)
        for (const bool keys : {true, false})
            if (sgemv_overlap(SgemvRows{pairs, 1, 0, (int64_t)max_pairs * 12}, sgemv_kv_rows(caches[l], keys)) ||
                sgemv_overlap(SgemvRows{count, 1, 0, 4}, sgemv_kv_rows(caches[l], keys)))
                return SGEMV_EINVAL;
    void* kargs[] = {&c, (void*)&pairs, (void*)&count, &max_pairs};
    return launch(reinterpret_cast<const void*>(k_copy), grid_for(1, (int64_t)max_pairs * layers * 2 * c.pieces), kargs, stream);
}
