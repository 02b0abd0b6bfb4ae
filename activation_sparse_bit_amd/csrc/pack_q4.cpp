// Host packer of the 4-bit weights of sgemv_q4_run and sgemv_q4_run_gated
// (no HIP calls).
//
// These products read every weight, so the layout is made for streaming: the
// matrix is cut into tiles of 16 outputs by 128 inputs, and the 1024 bytes of
// a tile hold, lane by lane, exactly what each of the 64 lanes of a
// wavefront feeds to four matrix-core steps.  One 16-byte load per lane
// fetches a tile in one contiguous KiB, and nothing is exchanged between
// lanes afterwards.  The byte formulas are documented in sgemv.h.
#include "internal.h"

#include <cstring>

namespace {

constexpr uint64_t kHeader = 256;
constexpr int kTileN = 16;
constexpr int kBlockK = 128;

uint64_t roundup(uint64_t v, uint64_t a) { return (v + a - 1) / a * a; }

int fill_desc(int32_t N, int32_t K, int32_t group, uint32_t flags, sgemv_q4_desc* d) {
    if (group != 32 && group != 64 && group != 128) return SGEMV_EINVAL;
    if (flags & ~(SGEMV_Q4_GATED | SGEMV_Q4_ZEROS | SGEMV_Q4_BF16_SCALES)) return SGEMV_EINVAL;
    if (N < 1 || N > SGEMV_MAX_N || K < 1 || K > SGEMV_MAX_K) return SGEMV_ESIZE;
    const uint64_t tiles = roundup((uint64_t)N, kTileN) / kTileN * ((flags & SGEMV_Q4_GATED) ? 2 : 1);
    const uint64_t cells = tiles * (roundup((uint64_t)K, kBlockK) / kBlockK);   // 16 x 128 blocks
    std::memset(d, 0, sizeof *d);
    d->N = N;
    d->K = K;
    d->group = group;
    d->flags = flags;
    d->w_off = kHeader;
    d->w_bytes = cells * 1024;
    d->s_off = d->w_off + d->w_bytes;
    d->s_bytes = cells * (kTileN * 2) * (kBlockK / group);
    d->z_off = roundup(d->s_off + d->s_bytes, 256);
    d->z_bytes = (flags & SGEMV_Q4_ZEROS) ? cells * (kTileN / 2) * (kBlockK / group) : 0;
    d->total_bytes = roundup(d->z_off + d->z_bytes, 256);
    return SGEMV_OK;
}

struct Part {
    const uint8_t* q;
    const uint16_t* s;
    const uint8_t* z;   // NULL: symmetric
};

// Whether any byte of p[0 .. n) is above 15.
bool any_above_15(const uint8_t* p, uint64_t n) {
    uint64_t bad = 0, v;
    uint64_t i = 0;
    for (; i + 8 <= n; i += 8) {
        std::memcpy(&v, p + i, 8);
        bad |= v;
    }
    for (; i < n; ++i) bad |= p[i];
    return (bad & 0xF0F0F0F0F0F0F0F0ull) != 0;
}

bool all_finite(const uint16_t* p, uint64_t n, uint16_t exp_mask) {
    for (uint64_t i = 0; i < n; ++i)
        if ((p[i] & exp_mask) == exp_mask) return false;
    return true;
}

// Eight codes (one byte each, input order) into one word: inputs 2h and
// 2h + 1 at nibbles h and h + 4, so that masking a word of two 16-bit halves
// yields the pair (2h, 2h + 1).
uint32_t pack8(uint64_t v) {
    const uint64_t e = v & 0x000F000F000F000Full;
    const uint64_t o = (v >> 8) & 0x000F000F000F000Full;
    const uint32_t lo = (uint32_t)((e | e >> 12 | e >> 24 | e >> 36) & 0xFFFF);
    const uint32_t hi = (uint32_t)((o | o >> 12 | o >> 24 | o >> 36) & 0xFFFF);
    return lo | hi << 16;
}

int pack(const Part* parts, int n_parts, const sgemv_q4_desc& d, void* out, size_t cap) {
    if (!out) return SGEMV_OK;   // size query
    const bool zeros = (d.flags & SGEMV_Q4_ZEROS) != 0;
    for (int p = 0; p < n_parts; ++p)
        if (!parts[p].q || !parts[p].s || (zeros && !parts[p].z)) return SGEMV_EINVAL;
    if (cap < d.total_bytes) return SGEMV_ESIZE;
    const uint64_t N = d.N, K = d.K, G = (K + d.group - 1) / d.group;
    const uint16_t exp_mask = (d.flags & SGEMV_Q4_BF16_SCALES) ? 0x7F80 : 0x7C00;
    for (int p = 0; p < n_parts; ++p) {   // validate everything before writing anything
        if (any_above_15(parts[p].q, N * K)) return SGEMV_EINVAL;
        if (!all_finite(parts[p].s, N * G, exp_mask)) return SGEMV_EINVAL;
        if (zeros && any_above_15(parts[p].z, N * G)) return SGEMV_EINVAL;
    }

    uint8_t* blob = static_cast<uint8_t*>(out);
    std::memset(blob, 0, kHeader);
    const uint32_t version = 1;
    std::memcpy(blob, "SGQ1", 4);
    std::memcpy(blob + 4, &version, 4);
    std::memcpy(blob + 8, &d.N, 4);
    std::memcpy(blob + 12, &d.K, 4);
    std::memcpy(blob + 16, &d.group, 4);
    std::memcpy(blob + 20, &d.flags, 4);
    std::memcpy(blob + 24, &d.w_off, 8);
    std::memcpy(blob + 32, &d.w_bytes, 8);
    std::memcpy(blob + 40, &d.s_off, 8);
    std::memcpy(blob + 48, &d.s_bytes, 8);
    std::memcpy(blob + 56, &d.z_off, 8);
    std::memcpy(blob + 64, &d.z_bytes, 8);
    std::memcpy(blob + 72, &d.total_bytes, 8);
    std::memset(blob + d.s_off, 0, d.total_bytes - d.s_off);

    const uint64_t blocks = (K + kBlockK - 1) / kBlockK;
    const uint64_t tiles = (N + kTileN - 1) / kTileN;
    const int per_block = kBlockK / d.group;   // groups per 128 inputs
    uint8_t* w = blob + d.w_off;
    uint16_t* sc = reinterpret_cast<uint16_t*>(blob + d.s_off);
    uint8_t* zp = blob + d.z_off;
    for (uint64_t t = 0; t < tiles; ++t)
        for (int p = 0; p < n_parts; ++p) {
            const uint64_t cell0 = (t * n_parts + p) * blocks;
            for (uint64_t b = 0; b < blocks; ++b) {
                uint8_t* cell = w + (cell0 + b) * 1024;
                for (uint64_t r = 0; r < kTileN; ++r) {
                    const uint64_t n = t * kTileN + r;
                    uint8_t codes[kBlockK];
                    const uint8_t* src = codes;
                    const uint64_t left = n < N ? K - b * kBlockK : 0;
                    if (left >= (uint64_t)kBlockK) {
                        src = parts[p].q + n * K + b * kBlockK;
                    } else {
                        std::memset(codes, 0, sizeof codes);
                        if (left) std::memcpy(codes, parts[p].q + n * K + b * kBlockK, left);
                    }
                    for (int j = 0; j < 4; ++j)
                        for (int c = 0; c < 4; ++c) {
                            uint64_t v;
                            std::memcpy(&v, src + 32 * j + 8 * c, 8);
                            const uint32_t word = pack8(v);
                            std::memcpy(cell + (16 * c + r) * 16 + 4 * j, &word, 4);
                        }
                    if (n >= N) continue;
                    for (int i = 0; i < per_block; ++i) {
                        const uint64_t g = b * per_block + i;
                        if (g >= G) break;
                        const uint64_t at = ((cell0 + b) * kTileN + r) * per_block + i;
                        sc[at] = parts[p].s[n * G + g];
                        if (zeros) zp[at >> 1] |= (uint8_t)(parts[p].z[n * G + g] << ((at & 1) * 4));
                    }
                }
            }
        }
    return SGEMV_OK;
}

}  // namespace

// Whether d is a description that the packer makes.
int sgemv_q4_check_desc(const sgemv_q4_desc* d) {
    if (!d) return SGEMV_EINVAL;
    sgemv_q4_desc e;
    const int st = fill_desc(d->N, d->K, d->group, d->flags, &e);
    if (st) return st;
    return std::memcmp(d, &e, sizeof e) ? SGEMV_EINVAL : SGEMV_OK;
}

extern "C" int sgemv_q4_pack(const uint8_t* q, const uint16_t* scales, const uint8_t* zeros, int32_t N, int32_t K,
                             int32_t group, uint32_t flags, void* out, size_t out_capacity, sgemv_q4_desc* desc_out) {
    if (flags & SGEMV_Q4_GATED) return SGEMV_EINVAL;
    sgemv_q4_desc d;
    int st = fill_desc(N, K, group, flags, &d);
    if (st) return st;
    const Part part{q, scales, zeros};
    st = pack(&part, 1, d, out, out_capacity);
    if (st == SGEMV_OK && desc_out) *desc_out = d;
    return st;
}

extern "C" int sgemv_q4_pack_gated(const uint8_t* q_gate, const uint16_t* scales_gate, const uint8_t* zeros_gate,
                                   const uint8_t* q_up, const uint16_t* scales_up, const uint8_t* zeros_up, int32_t N,
                                   int32_t K, int32_t group, uint32_t flags, void* out, size_t out_capacity,
                                   sgemv_q4_desc* desc_out) {
    sgemv_q4_desc d;
    int st = fill_desc(N, K, group, flags | SGEMV_Q4_GATED, &d);
    if (st) return st;
    const Part parts[2] = {{q_gate, scales_gate, zeros_gate}, {q_up, scales_up, zeros_up}};
    st = pack(parts, 2, d, out, out_capacity);
    if (st == SGEMV_OK && desc_out) *desc_out = d;
    return st;
}

extern "C" int sgemv_q4_desc_from_header(const void* header, size_t bytes, sgemv_q4_desc* desc_out) {
    if (!header || !desc_out || bytes < 80) return SGEMV_EINVAL;
    const uint8_t* h = static_cast<const uint8_t*>(header);
    uint32_t version;
    std::memcpy(&version, h + 4, 4);
    if (std::memcmp(h, "SGQ1", 4) || version != 1) return SGEMV_EINVAL;
    sgemv_q4_desc d;
    std::memset(&d, 0, sizeof d);
    std::memcpy(&d.N, h + 8, 4);
    std::memcpy(&d.K, h + 12, 4);
    std::memcpy(&d.group, h + 16, 4);
    std::memcpy(&d.flags, h + 20, 4);
    std::memcpy(&d.w_off, h + 24, 8);
    std::memcpy(&d.w_bytes, h + 32, 8);
    std::memcpy(&d.s_off, h + 40, 8);
    std::memcpy(&d.s_bytes, h + 48, 8);
    std::memcpy(&d.z_off, h + 56, 8);
    std::memcpy(&d.z_bytes, h + 64, 8);
    std::memcpy(&d.total_bytes, h + 72, 8);
    if (sgemv_q4_check_desc(&d)) return SGEMV_EINVAL;
    *desc_out = d;
    return SGEMV_OK;
}
