/*
 * sgemv.h - C ABI of the dynamically sparse int4 GEMV for MI355X (gfx950).
 *
 * The operation ("Enabling Dynamic Sparsity in Quantized LLM Inference",
 * Abstract): during decode the activation vector x is dynamically sparse;
 * entries with small magnitude are dropped, and only the weight columns that
 * match the surviving indices are read, from a group-wise low-bit quantized
 * weight matrix stored in a layout that keeps those reads local.  The page
 * names three parts - a sparsity-consistent quantized weight layout, a GEMV
 * kernel for it, and a run-time step that gathers the active indices - and
 * this library provides one call for each, plus the batched variant:
 *
 *   sgemv_pack_layout     host: int4 codes + fp16 scale/zero -> packed blob
 *                         (sgemv_pack_layout_z4: the same with 4-bit zeros;
 *                         sgemv_pack_layout_ng: groups along the outputs)
 *   sgemv_gather_indices  device: threshold x, emit the ascending list of
 *                         active indices and its length
 *   sgemv_run             device: y = W . x over the listed columns (M = 1)
 *   sgemv_run_batched     device: M <= 16 rows over the union list, each row
 *                         masked by its own threshold
 *   sgemv_run_fused       device: threshold, union, compact and GEMV in one
 *                         launch (M <= 16), the list optional
 *
 * Weights.  W is [N][K] (output x input, like a Linear weight), quantized
 * asymmetrically to 4 bits with one fp16 scale s and one fp16 zero-point z
 * per output row n and group g of 128 consecutive inputs (k / 128):
 *   w^[n][k] = s[n][k/128] * (q[n][k] - z[n][k/128]),  q in 0..15,
 * z an integer 0..15 stored as fp16 (the GPTQ-style format that the page
 * cites; the page itself fixes no format, so this is our reading).
 *
 * Selection.  Entry k of row m is active iff float32(|x[m][k]|) >= t[m]:
 * ties are kept, NaN is never active, -0 and +0 are active when t == 0.  The
 * page does not state the rule; magnitude thresholding with a calibrated
 * per-call scalar follows "Training-Free Activation Sparsity in Large
 * Language Models", which the page builds on.
 *
 * Conventions for every call.
 *   - Every pointer marked "device" is device memory; "host" is host memory.
 *     The caller owns all buffers; the library allocates nothing and keeps
 *     no state between calls except a thread-local last HIP error.
 *   - `stream` is a hipStream_t passed as void* (NULL = the null stream).
 *     Device work is enqueued on it asynchronously; the host never waits.
 *   - Arguments are validated before any HIP call.  On a bad argument the
 *     call returns a negative status and enqueues nothing.  A failed launch
 *     returns SGEMV_EHIP (details: sgemv_last_hip_error).  Faults while a
 *     kernel runs surface at the caller's next synchronisation.
 *   - Nothing is printed, nothing throws across the ABI.
 *   - Calls are re-entrant; calls that share a workspace must not run
 *     concurrently on different streams.
 */
#ifndef SGEMV_H
#define SGEMV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Description of one packed matrix; produced by sgemv_pack_layout or
 * sgemv_desc_from_header, read by the device calls (host memory). */
typedef struct sgemv_desc {
    int32_t  N;            /* outputs (rows of W)                          */
    int32_t  K;            /* inputs (columns of W), multiple of 128       */
    int32_t  group;        /* quantization group along K, always 128       */
    int32_t  tile_n;       /* outputs per tile of the layout               */
    uint64_t w_off;        /* byte offset of the weight region (= 256)     */
    uint64_t w_bytes;      /* N*K/2                                        */
    uint64_t m_off;        /* byte offset of the scale/zero region         */
    uint64_t m_bytes;      /* (K/128)*N*4, or (K/128)*N*5/2 for version 2  */
    uint64_t total_bytes;  /* size of the whole blob                       */
    uint32_t version;      /* SGEMV_LAYOUT_PAIRS, _Z4 or _NG               */
    uint32_t reserved;     /* 0                                            */
} sgemv_desc;

enum sgemv_status {
    SGEMV_OK           = 0,
    SGEMV_EINVAL       = -1,  /* NULL pointer, bad value, bad flag          */
    SGEMV_ESIZE        = -2,  /* a size out of range or capacity too small  */
    SGEMV_EALIGN       = -3,  /* pointer or leading dimension misaligned    */
    SGEMV_EUNSUPPORTED = -4,  /* valid layout the kernels do not implement  */
    SGEMV_EHIP         = -5   /* a HIP call failed                          */
};

#define SGEMV_GROUP       128
#define SGEMV_MAX_BATCH   16
#define SGEMV_MAX_K       65536
#define SGEMV_MAX_N       (1 << 20)
#define SGEMV_TILE_N      512   /* the tile width the device kernels run   */
#define SGEMV_OUT_F32     1u    /* flag: y is fp32 instead of fp16         */
#define SGEMV_LAYOUT_PAIRS 1u   /* layout version 1: (s, z) fp16 pairs     */
#define SGEMV_LAYOUT_Z4    2u   /* layout version 2: fp16 s, 4-bit z       */
#define SGEMV_LAYOUT_NG    3u   /* layout version 3: groups along N        */

/*
 * sgemv_pack_layout - re-lay int4 weights so that each active input index
 * maps to contiguous bytes (host only, no HIP call).
 *
 * Realises the sparsity-aware weight layout asked for by the page's
 * Abstract (weights arranged to match activation sparsity, for memory
 * locality on the GPU); the page does not give its pattern, so the pattern
 * is ours:
 *
 *   blob = header (256 B) | weights | scale/zero metadata, little-endian
 *   header 0: "SGV1", 4: u32 version 1, 8: i32 N, 12: i32 K, 16: i32 group,
 *          20: i32 tile_n, 24: u64 w_off, 32: u64 w_bytes, 40: u64 m_off,
 *          48: u64 m_bytes, 56: u64 total_bytes, 64..255 zero
 *   w_off = 256; m_off = w_off + roundup(w_bytes, 256);
 *   total = m_off + roundup(m_bytes, 256)
 *   weight byte  w_off + (t*K + k)*(tile_n/2) + j
 *                = q[t*tile_n + 2j][k] | q[t*tile_n + 2j + 1][k] << 4
 *   metadata     m_off + ((t*(K/128) + g)*tile_n + i)*4 = s bits, z bits of
 *                row t*tile_n + i, group g (two little-endian u16)
 *
 * So for every tile of tile_n outputs, one input index k is one contiguous
 * run of tile_n/2 bytes (256 B for tile_n = 512), and one group's scales
 * and zeros are one contiguous run of tile_n*4 bytes.
 *
 *   q          host uint8 [N][K], row-major, values 0..15
 *   scales_f16 host uint16 [N][K/128], fp16 bit patterns of finite values
 *   zeros_f16  host uint16 [N][K/128], fp16 bit patterns of integers 0..15
 *   group      must be 128
 *   tile_n     power of two in [64, 1024] dividing N (the device calls run
 *              tile_n = SGEMV_TILE_N only)
 *   out        host buffer of out_capacity bytes, or NULL for a size query
 *   desc_out   receives the description (may be NULL when out == NULL)
 * Returns SGEMV_OK; EINVAL for NULL inputs, a code > 15, a bad scale or
 * zero-point, group != 128; ESIZE for bad N/K/tile_n or out_capacity <
 * total_bytes.  The blob is self-describing and may be saved and reloaded.
 */
int sgemv_pack_layout(const uint8_t* q, const uint16_t* scales_f16,
                      const uint16_t* zeros_f16, int32_t N, int32_t K,
                      int32_t group, int32_t tile_n, void* out,
                      size_t out_capacity, sgemv_desc* desc_out);

/*
 * sgemv_pack_layout_z4 - the same layout with compact metadata (version 2).
 *
 * The weight region is byte for byte that of sgemv_pack_layout.  The
 * zero-points are integers 0..15, so they take 4 bits: the run of one
 * (tile, group) pair holds the tile_n fp16 scales, then tile_n/2 bytes of
 * zero-points, two per byte.  Same numbers, 2.5 instead of 4 bytes per row
 * and group: this carries the page's sparsity-consistent layout (Abstract)
 * to the metadata, which every touched group still reads in full.
 *
 *   header as above with version 2 and m_bytes = (K/128)*N*5/2
 *   scale       m_off + (t*(K/128) + g)*(5*tile_n/2) + 2i : fp16 bits of
 *               s[t*tile_n + i][g] (little-endian u16)
 *   zero-points m_off + (t*(K/128) + g)*(5*tile_n/2) + 2*tile_n + j
 *               = z[t*tile_n + 2j][g] | z[t*tile_n + 2j + 1][g] << 4
 *
 * Arguments, ownership and errors as for sgemv_pack_layout.  Every device
 * call takes either version (desc->version) and computes bit for bit the
 * same y from both.
 */
int sgemv_pack_layout_z4(const uint8_t* q, const uint16_t* scales_f16,
                         const uint16_t* zeros_f16, int32_t N, int32_t K,
                         int32_t group, int32_t tile_n, void* out,
                         size_t out_capacity, sgemv_desc* desc_out);

/*
 * sgemv_pack_layout_ng - layout version 3, for weights quantized with their
 * groups along the outputs: one fp16 scale s and one integer zero-point z
 * per input column k and group b of 128 consecutive outputs,
 *   w^[n][k] = s[n/128][k] * (q[n][k] - z[n/128][k]).
 * The page asks for a quantization layout consistent with activation
 * sparsity (Abstract); with groups along the outputs a column's scale and
 * zero-point belong to that column alone, so they are read only when the
 * column is active and the metadata bytes fall with the sparsity, as the
 * weight bytes do.
 *
 *   header as above with version 3; m_bytes = (N/128)*K*4
 *   weight bytes exactly those of sgemv_pack_layout
 *   metadata     m_off + ((h*K + k)*2 + e)*4 : fp16 bits of s[2h + e][k],
 *                then fp16 bits of z[2h + e][k]  (h < N/256, e in {0, 1}):
 *                per 256 outputs and column, 8 contiguous bytes
 *
 *   q          host uint8 [N][K], row-major, values 0..15
 *   scales_f16 host uint16 [N/128][K], fp16 bit patterns of finite values
 *   zeros_f16  host uint16 [N/128][K], fp16 bit patterns of integers 0..15
 *   tile_n     power of two in [256, 1024] dividing N
 * Other arguments, ownership and errors as for sgemv_pack_layout (ESIZE
 * also for tile_n < 256).  Every device call takes this version.  The
 * kernels fold each column's scale into its activation (s * x rounded once
 * to fp16) and subtract the zero-point exactly, so y differs from the exact
 * product by at most 2^-11 * sum_k |w^[n][k]| |x[k]| plus fp32 accumulation
 * before the final rounding of y (versions 1 and 2: fp32 accumulation
 * error only).
 */
int sgemv_pack_layout_ng(const uint8_t* q, const uint16_t* scales_f16,
                         const uint16_t* zeros_f16, int32_t N, int32_t K,
                         int32_t group, int32_t tile_n, void* out,
                         size_t out_capacity, sgemv_desc* desc_out);

/*
 * sgemv_pack_layout_parts - one blob for several projections that read the
 * same activations (the query, key and value projections of an attention
 * block; the gate and up projections of a gated feed-forward block), their
 * rows stacked along N in the order given, so that one device call
 * thresholds x once and computes all of them.  The blob is exactly the one
 * sgemv_pack_layout (version SGEMV_LAYOUT_PAIRS), sgemv_pack_layout_z4
 * (SGEMV_LAYOUT_Z4) or sgemv_pack_layout_ng (SGEMV_LAYOUT_NG) writes for the
 * row-concatenated matrix; projection p's
 * outputs are y[off_p .. off_p + n_part[p]) with off_p the sum of the
 * earlier n_part.  Host only, no HIP call.
 *
 *   parts      number of projections, >= 1
 *   q          host array of `parts` pointers, part p: uint8 [n_part[p]][K]
 *   scales_f16 host array of `parts` pointers, part p: uint16 [n_part[p]][K/128]
 *              ([n_part[p]/128][K] for SGEMV_LAYOUT_NG)
 *   zeros_f16  likewise for the zero-points
 *   n_part     host int32 [parts]: rows of each part, each a multiple of
 *              tile_n (no tile mixes two projections)
 *   K, group, tile_n, out, out_capacity, desc_out as for sgemv_pack_layout
 *   version    SGEMV_LAYOUT_PAIRS, SGEMV_LAYOUT_Z4 or SGEMV_LAYOUT_NG
 * Returns SGEMV_OK; EINVAL for parts < 1, NULL arrays or parts, a bad code,
 * scale or zero-point, a bad version; ESIZE for a part that is not whole
 * tiles, a total N out of range, or too small a capacity.  With out == NULL
 * it is a size query (q, scales and zeros may then be NULL).
 */
int sgemv_pack_layout_parts(int32_t parts, const uint8_t* const* q,
                            const uint16_t* const* scales_f16,
                            const uint16_t* const* zeros_f16, const int32_t* n_part,
                            int32_t K, int32_t group, int32_t tile_n, uint32_t version,
                            void* out, size_t out_capacity, sgemv_desc* desc_out);

/* Parse and check the 64-byte header of a blob held in host memory (for a
 * blob that was saved and reloaded; version 1, 2 or 3).  EINVAL on a bad magic,
 * version or inconsistent offsets. */
int sgemv_desc_from_header(const void* header, size_t bytes, sgemv_desc* desc_out);

/*
 * sgemv_gather_indices - the run-time step of the page's Abstract that
 * collects the indices of the surviving activations at low cost: threshold
 * every row, OR the rows' masks, and compact the union into an ascending
 * list.  A few workgroups (one per 4096 columns, or per 8192 with more
 * rows), each over its own column range; every workgroup counts the active
 * columns below its range straight from x, so they need no scratch memory
 * and no communication; wavefront ballots and bit counts give each lane its
 * rank, an LDS scan orders the wavefronts.
 *
 *   x_f16      device fp16 [M][ldx]; 16-byte aligned
 *   M          rows, 1..SGEMV_MAX_BATCH
 *   K          columns, multiple of 128, <= SGEMV_MAX_K
 *   ldx        row stride in elements, >= K, multiple of 8
 *   thresholds host float [M], each finite and >= 0
 *   idx        device int32 [K]: receives the active indices ascending in
 *              idx[0 .. count); entries beyond count are left untouched
 *   count      device int32 [1]: receives the number of active indices
 * Deterministic: the list is unique for given inputs.
 */
int sgemv_gather_indices(const void* x_f16, int32_t M, int32_t K, int32_t ldx,
                         const float* thresholds, int32_t* idx, int32_t* count,
                         void* stream);

/*
 * sgemv_run - y = W . x over the listed columns (the page's specialised
 * GEMV for the sparse layout, Abstract):
 *   y[n] = sum over j < *count of w^[n][idx[j]] * x[idx[j]]
 * accumulated in fp32 (products exact, per-lane partial sums, fixed-order
 * tree across lanes, wavefronts and workgroups), rounded once to fp16 with
 * round-to-nearest-even (or stored as fp32 with SGEMV_OUT_F32).  x is used
 * unmasked at the listed indices.  With idx == NULL every column is used
 * (the dense int4 GEMV) and count is ignored.  count == 0 gives y = +0.
 * The result is bitwise reproducible for given inputs.
 *
 *   d          host description of the packed matrix (tile_n = 512)
 *   packed     device blob from sgemv_pack_layout, 256-byte aligned
 *   x_f16      device fp16 [K], 16-byte aligned
 *   idx        device int32 buffer of K entries, 4-byte aligned, whose
 *              first *count entries are ascending, unique and < K (as
 *              produced by sgemv_gather_indices); or NULL for all columns.
 *              Entries beyond *count may hold anything.
 *   count      device int32 [1], 0 <= *count <= K (clamped to that range)
 *   y          device fp16 [N] (fp32 with SGEMV_OUT_F32), 16-byte aligned
 *   flags      0 or SGEMV_OUT_F32
 *   workspace  device, sgemv_workspace_bytes(d, 1) bytes, 256-byte
 *              aligned, zero-filled once by the caller.  It holds one
 *              arrival counter per 256 outputs, which every call returns to
 *              zero, then scratch (lists, sums) that needs no clearing, at
 *              offsets that depend on N: so it can be reused by any later
 *              call on the same stream for a matrix with the same N (sized
 *              for the largest K and row count among them).  A workspace
 *              that has served one N must be zero-filled again before it
 *              serves another.  May be NULL when the call has a single
 *              column segment (K up to 512 for one or two rows, 1024 for
 *              more); the call returns SGEMV_EINVAL when it needs one.
 */
int sgemv_run(const sgemv_desc* d, const void* packed, const void* x_f16,
              const int32_t* idx, const int32_t* count, void* y,
              uint32_t flags, void* workspace, void* stream);

/*
 * sgemv_run_batched - M rows against one matrix over the union list
 * (batched contextual sparsity as in "Polar Sparsity: High Throughput
 * Batched LLM Inferencing with Scalable Contextual Sparsity", which the
 * page builds on: the batch reads the union of its rows' active columns
 * once):
 *   y[m][n] = sum over j < *count of w^[n][idx[j]] * xe[m][idx[j]],
 *   xe[m][k] = x[m][k] if float32(|x[m][k]|) >= thresholds[m], else 0
 * With thresholds == NULL every row uses x unmasked at every listed index.
 * With idx == NULL every column is listed.
 *
 *   x_f16 device fp16 [M][ldx], 16-byte aligned, ldx >= K, ldx % 8 == 0
 *   y     device fp16/fp32 [M][ldy], 16-byte aligned, ldy >= N, ldy % 8 == 0
 *   workspace: sgemv_workspace_bytes(d, M) bytes, same contract as above.
 * Other arguments as in sgemv_run.  SGEMV_ESIZE when the call's partial
 * sums would exceed 4 GiB - 1 (half tiles x segments x M x 1 KiB; only
 * near the largest N, K and M), which the kernels address with 32-bit
 * offsets.
 */
int sgemv_run_batched(const sgemv_desc* d, const void* packed,
                      const void* x_f16, int32_t M, int32_t ldx,
                      const float* thresholds, const int32_t* idx,
                      const int32_t* count, void* y, int32_t ldy,
                      uint32_t flags, void* workspace, void* stream);

/*
 * sgemv_run_fused - the gathering step and the GEMV in one launch, so that
 * no kernel boundary and no round trip through a global list separate the
 * thresholding from the weight reads (the page's Abstract asks for index
 * gathering with minimal overhead).  Each wavefront thresholds one
 * 128-column group of every row, compacts the columns active in any row in
 * LDS and reads only their weight bytes; the workgroups of the column
 * segments (512 or 1024 columns) are summed as in sgemv_run.
 *   y[m][n] = sum over active k of w^[n][k] * xe[m][k]
 * with xe and the union of active columns as in sgemv_run_batched (with
 * thresholds), which it equals within the same error bound (the order of
 * the fp32 additions differs, so the bits may differ).
 *
 *   M          1..SGEMV_MAX_BATCH.  One or two rows run on the vector
 *              units; 3 to 16 rows run on the matrix cores
 *              (v_mfma_f32_16x16x32_f16 over exactly dequantized fp16
 *              q - z, fp32 accumulation), each row masked by its own
 *              threshold over the union of the rows' active columns
 *   thresholds host float [M], each finite and >= 0 (required)
 *   idx, count both NULL, or both device int32 ([K] and [1], 4-byte
 *              aligned): then they receive exactly what
 *              sgemv_gather_indices writes for the same x and thresholds
 *   workspace  sgemv_workspace_bytes(d, M) bytes, same contract as above
 * Other arguments as in sgemv_run_batched.  Bitwise reproducible.
 */
int sgemv_run_fused(const sgemv_desc* d, const void* packed, const void* x_f16,
                    int32_t M, int32_t ldx, const float* thresholds,
                    int32_t* idx, int32_t* count, void* y, int32_t ldy,
                    uint32_t flags, void* workspace, void* stream);

/*
 * sgemv_run_fused_static - sgemv_run_fused without a workspace argument, for
 * callers that cannot allocate device memory (code under graph capture,
 * tight serving loops, harnesses that forbid allocation).  The scratch
 * (arrival counters, the list workgroups' line and list, partial sums) is a
 * fixed 16 MiB device array inside the library, one per GPU, held until the
 * process ends; its address is taken once per GPU (on the first call there,
 * which also clears its counters on `stream`); nothing is allocated.
 *   - Sizes beyond the array: N above 262144 (1024 half tiles), or partial
 *     sums above its 15.5 MiB (half tiles x segments x M x 1 KiB; segments
 *     of 512 columns for one or two rows, 1024 for more) return
 *     SGEMV_ESIZE before any HIP call.  Every configuration of 8192- to
 *     28672-wide Llama-3 projections with up to 16 rows fits.
 *   - Every call on a GPU shares that GPU's array and leaves its counters
 *     at zero again; calls that overlap on one GPU (other streams, other host
 *     threads) race and must not be made.
 * Other arguments, results and errors as for sgemv_run_fused, which it
 * equals bit for bit.
 */
int sgemv_run_fused_static(const sgemv_desc* d, const void* packed, const void* x_f16,
                           int32_t M, int32_t ldx, const float* thresholds,
                           int32_t* idx, int32_t* count, void* y, int32_t ldy,
                           uint32_t flags, void* stream);

/* Bytes of workspace needed by sgemv_run (M = 1), sgemv_run_batched or
 * sgemv_run_fused with up to M rows on matrix d; 0 for an invalid
 * description. */
size_t sgemv_workspace_bytes(const sgemv_desc* d, int32_t M);

/* ------------------------------------------------------------------------
 * Beside the sparse projections: 4-bit products that read every weight, and
 * the norms around a block.
 *
 * The calls above skip the columns that a thresholded input leaves out.  A
 * decode step also has projections whose input is dense (an attention
 * output, the head that gives the logits), weights quantized in other groups
 * and widths, the gate between the up and down projections, and the norms
 * and residual additions between the blocks.  These calls serve them with
 * the same conventions: the caller owns every buffer, arguments are checked
 * before any HIP call, work is enqueued on `stream` (NULL = the null stream)
 * on the current device, which has to be the one that holds the buffers, and
 * results are bitwise reproducible.  They need no workspace and keep no
 * state, so calls on different streams do not disturb each other, and they
 * may be captured into a graph.
 * ------------------------------------------------------------------------ */

enum sgemv_type {            /* element types of x, y, residuals and weights */
    SGEMV_F16  = 0,
    SGEMV_BF16 = 1,
    SGEMV_F32  = 2
};

enum sgemv_act {             /* gate functions of sgemv_q4_run_gated         */
    SGEMV_ACT_SILU = 0,      /* v / (1 + e^-v)                               */
    SGEMV_ACT_GELU = 1,      /* v (1 + erf(v / sqrt 2)) / 2                  */
    SGEMV_ACT_RELU = 2       /* max(v, 0)                                    */
};

#define SGEMV_Q4_GATED       1u   /* a gate and an up projection, interleaved  */
#define SGEMV_Q4_ZEROS       2u   /* zero-points stored (else every z is 8)    */
#define SGEMV_Q4_BF16_SCALES 4u   /* scales are bf16 instead of fp16           */

/* Description of one matrix (or gate/up pair) packed by sgemv_q4_pack or
 * sgemv_q4_pack_gated (host memory). */
typedef struct sgemv_q4_desc {
    int32_t  N;            /* outputs (of each of the two, when gated)     */
    int32_t  K;            /* inputs                                       */
    int32_t  group;        /* inputs per scale: 32, 64 or 128              */
    uint32_t flags;        /* SGEMV_Q4_*                                   */
    uint64_t w_off;        /* byte offset of the codes (= 256)             */
    uint64_t w_bytes;
    uint64_t s_off;        /* byte offset of the scales                    */
    uint64_t s_bytes;
    uint64_t z_off;        /* byte offset of the zero-points               */
    uint64_t z_bytes;      /* 0 without SGEMV_Q4_ZEROS                     */
    uint64_t total_bytes;  /* size of the whole blob                       */
} sgemv_q4_desc;

/*
 * sgemv_q4_pack - lay 4-bit weights out for sgemv_q4_run (host only).
 *   w^[n][k] = s[n][k/group] * (q[n][k] - z[n][k/group])
 *
 *   blob = header (256 B) | codes | scales | zero-points, little-endian
 *   header 0: "SGQ1", 4: u32 version 1, 8: i32 N, 12: i32 K, 16: i32 group,
 *          20: u32 flags, 24: u64 w_off, 32: u64 w_bytes, 40: u64 s_off,
 *          48: u64 s_bytes, 56: u64 z_off, 64: u64 z_bytes,
 *          72: u64 total_bytes, 80..255 zero
 *   The matrix is cut into cells of 16 outputs by 128 inputs, zero beyond N
 *   and K: B = ceil(K/128) cells per 16 outputs, cell (t, b) at index
 *   t*B + b (sgemv_q4_pack_gated: the gate's cells of 16 outputs, then the
 *   up projection's: index (2t + p)*B + b).
 *   codes        w_off + cell*1024 + (16c + r)*16 + 4j, c, j < 4, r < 16: a
 *                u32 whose nibble (i>>1) + 4*(i&1) is
 *                q[16t + r][128b + 32j + 8c + i], i < 8
 *   scales       u16 index (cell*16 + r)*P + i, P = 128/group, i < P:
 *                s[16t + r][b*P + i], at s_off
 *   zero-points  nibble index as for the scales, even index in the low half
 *                of a byte, at z_off
 *   s_off = w_off + w_bytes; z_off and total_bytes are rounded up to 256
 *
 *   q        host uint8 [N][K], values 0..15
 *   scales   host uint16 [N][ceil(K/group)]: finite fp16 bits (bf16 bits with
 *            SGEMV_Q4_BF16_SCALES)
 *   zeros    host uint8 [N][ceil(K/group)], values 0..15, used with
 *            SGEMV_Q4_ZEROS only; without it every zero-point is 8
 *   N, K     1..SGEMV_MAX_N, 1..SGEMV_MAX_K, any value (the last group and
 *            the last cells may be partial)
 *   out      host buffer of out_capacity bytes, or NULL for a size query
 *   desc_out receives the description (may be NULL)
 * EINVAL for a bad group, flag, code, scale or zero-point or a NULL array;
 * ESIZE for N, K out of range or too small a capacity.
 */
int sgemv_q4_pack(const uint8_t* q, const uint16_t* scales, const uint8_t* zeros,
                  int32_t N, int32_t K, int32_t group, uint32_t flags, void* out,
                  size_t out_capacity, sgemv_q4_desc* desc_out);

/* sgemv_q4_pack_gated - the same for a gate and an up projection of equal
 * shape and format that share their input (SGEMV_Q4_GATED is set in the
 * description), for sgemv_q4_run_gated. */
int sgemv_q4_pack_gated(const uint8_t* q_gate, const uint16_t* scales_gate,
                        const uint8_t* zeros_gate, const uint8_t* q_up,
                        const uint16_t* scales_up, const uint8_t* zeros_up,
                        int32_t N, int32_t K, int32_t group, uint32_t flags,
                        void* out, size_t out_capacity, sgemv_q4_desc* desc_out);

/*
 * sgemv_q4_pack_device - the same blob, byte for byte, made on the device from
 * codes, scales and zero-points that are there already (the up projection's
 * with SGEMV_Q4_GATED in flags, else NULL).
 *   packed   device buffer of `capacity` bytes, 256-byte aligned (a size query
 *            is sgemv_q4_pack or sgemv_q4_pack_gated with out == NULL)
 * Shapes and types as above, in device memory.  Codes and zero-points are not
 * checked: their low four bits are taken.  EINVAL, ESIZE and EALIGN as above;
 * EINVAL also where an input shares bytes with the blob.
 */
int sgemv_q4_pack_device(const uint8_t* q, const uint16_t* scales, const uint8_t* zeros,
                         const uint8_t* q_up, const uint16_t* scales_up,
                         const uint8_t* zeros_up, int32_t N, int32_t K, int32_t group,
                         uint32_t flags, void* packed, size_t capacity,
                         sgemv_q4_desc* desc_out, void* stream);

/* Parse and check the header (at least 80 bytes) of a blob of either call.
 * EINVAL on a bad magic, version or inconsistent fields. */
int sgemv_q4_desc_from_header(const void* header, size_t bytes,
                              sgemv_q4_desc* desc_out);

/*
 * sgemv_q4_run - y[m][n] = sum_k w^[n][k] x[m][k] + bias[n] for 1 to
 * SGEMV_MAX_BATCH rows, every weight read once.
 *
 *   d       host description without SGEMV_Q4_GATED
 *   packed  device blob, 256-byte aligned
 *   x       device [M][ldx] of x_type: SGEMV_F16 or SGEMV_BF16
 *   bias    device [N] of x_type, or NULL
 *   y       device [M][ldy] of y_type: x_type or SGEMV_F32; refused where it
 *           overlaps an input (columns of one wider buffer do not)
 *   ldx, ldy  row strides in elements, >= K and >= N.  Pointers need the
 *           alignment of their elements only.
 * Products are exact and sums are held in fp32, one group of inputs at a
 * time; the group's scale, the bias and the one rounding to y_type follow.
 * fp16 activations multiply q - z, so y is within fp32 accumulation of the
 * exact value.  bf16 activations multiply q + 16 (four bits more than a code
 * fit bf16's mantissa, and CDNA4 has no packed bf16 subtraction) and
 * (z + 16) * sum x is taken off each group's sum in fp32: the accumulation
 * error is relative to sum |s| (q + 16) |x| instead, at most a few 2^-24 of
 * it per group.  Sums that leave fp32 on this way but not by the formula, and
 * those with an infinity, are computed again from q - z in the same launch, as
 * fp16 ones are; a call with such a row takes 2 to 5 times as long.
 * EINVAL for NULL, a bad type or description or an overlap; ESIZE for M, ldx
 * or ldy; EALIGN for pointers.
 */
int sgemv_q4_run(const sgemv_q4_desc* d, const void* packed, const void* x,
                 int32_t x_type, int32_t M, int32_t ldx, const void* bias,
                 void* y, int32_t y_type, int32_t ldy, void* stream);

/*
 * sgemv_q4_run_gated - the gated product of a feed-forward block in one
 * launch:
 *   h[m][n] = act(gate[n] . x[m] + bias_gate[n]) * (up[n] . x[m] + bias_up[n])
 * both sums and the gate function in fp32, one rounding to h_type.  h is
 * what the down projection takes: sgemv_q4_run, or sgemv_run_fused, which
 * skips the columns of small h and takes fp16 only.
 *
 *   d    host description with SGEMV_Q4_GATED
 *   act  SGEMV_ACT_*
 *   bias_gate, bias_up  device [N] of x_type, each may be NULL
 *   h    device [M][ldh] of h_type: x_type or SGEMV_F32
 * Everything else as for sgemv_q4_run.
 */
int sgemv_q4_run_gated(const sgemv_q4_desc* d, const void* packed, const void* x,
                       int32_t x_type, int32_t M, int32_t ldx, const void* bias_gate,
                       const void* bias_up, int32_t act, void* h, int32_t h_type,
                       int32_t ldh, void* stream);

#define SGEMV_NORM_POST     1u   /* y is normed before it is added            */
#define SGEMV_NORM_CENTER   2u   /* subtract the mean (layer norm)            */
#define SGEMV_NORM_PLUS_ONE 4u   /* weights are stored around 0: factor 1 + w */

/* Arguments of sgemv_block_norm (host memory, read during the call). */
typedef struct sgemv_norm {
    int64_t     rows;             /* 0 .. 2^31 - 1; 0 enqueues nothing (the
                                     buffers may then be NULL)                */
    int32_t     D;                /* 1 .. SGEMV_MAX_K                         */
    uint32_t    flags;            /* SGEMV_NORM_*                             */
    const void* residual;         /* device [rows][ld_residual]               */
    const void* y;                /* device [rows][ld_y], or NULL             */
    const void* gate;             /* device [rows][ld_gate] of y_type, or [D]
                                     with ld_gate == 0, or NULL               */
    const void* post_weight;      /* device [D] of w_type, each may be NULL   */
    const void* post_bias;
    const void* weight;
    const void* bias;
    void*       residual_out;     /* device [rows][ld_residual_out] of
                                     residual_type, or NULL                   */
    void*       x;                /* device [rows][ld_x] of x_type            */
    int64_t     ld_residual, ld_y, ld_gate, ld_residual_out, ld_x;
    float       scale;
    float       eps;              /* >= 0, finite                             */
    int32_t     residual_type, y_type, w_type, x_type;   /* SGEMV_F16/BF16/F32 */
} sgemv_norm;

/*
 * sgemv_block_norm - from the output y of one block to the input x of the
 * next, in one pass over the rows (one launch for up to 2^21 of them):
 *   u  = y, or norm(y; post_weight, post_bias) with SGEMV_NORM_POST
 *   r  = residual + scale * gate * u      (gate 1 when NULL)
 *   residual_out = r
 *   x  = norm(r; weight, bias)
 *   norm(v; w, b) = (v - c) / sqrt(mean((v - c)^2) + eps) * w + b
 * with c = 0, or the mean of v with SGEMV_NORM_CENTER; a NULL weight is a
 * factor 1, a NULL bias 0, and SGEMV_NORM_PLUS_ONE adds 1 to weights that
 * are given.  With y == NULL, r = residual (gate and SGEMV_NORM_POST are
 * then refused).  Everything is computed in fp32 and rounded once on the way
 * out; x is the norm of r before its rounding to residual_type.  A row's sum
 * of squares has to fit fp32 (values below 7 * 10^16 do at any width).
 *
 * Row strides are at least D and pointers need the alignment of their
 * elements only.  An output may be the very buffer of residual, y or a
 * per-row gate (same address, row stride and element size), and columns of one
 * wider buffer may be different operands; any other meeting of an output's
 * byte range with another buffer's is refused.
 * EINVAL for NULL residual or x, a bad flag, type, eps or overlap; ESIZE for
 * rows, D or a stride; EALIGN for pointers.
 */
int sgemv_block_norm(const sgemv_norm* a, void* stream);

/* Static string for a status code. */
const char* sgemv_strerror(int status);

/* hipError_t of the last failed HIP call on this thread (0 if none). */
int sgemv_last_hip_error(void);

#ifdef __cplusplus
}
#endif

#endif /* SGEMV_H */
