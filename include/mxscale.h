/*
 * mxscale.h -- C ABI of libmxscale: MXFP8 E8M0 scale factors -> per-group
 * 128x4 blocked ("swizzled") layout, on NVIDIA B200 (sm_100a).
 *
 * The operation (pytorch/ao pull requests on MXFP8 MoE training):
 *   - "[mxfp8 moe training] compute prefix sum of group sizes inside kernel
 *     intead of precomputing" (#3285), Context and Changes: the padded start
 *     of every group is a prefix sum of padded group sizes, computed inside
 *     the kernel, with no host precompute and no device-to-host copy.
 *   - "[mxfp8 moe training] fallback cuda kernel for when input doesn't meet 2d
 *     TMA constraints" (#3708), Context: groups along M; a pipelined TMA kernel
 *     when the row stride is a multiple of 16 bytes, a simpler kernel for any
 *     other width (e.g. 44 columns), chosen per input.
 *   - "[mxfp8 moe training] add bench script for scale conversion to blocked
 *     format kernels for groups along K" (#3604): groups along K, each group
 *     made of 128x4 scale-factor tiles.
 *   - "Add CuTeDSL MXFP8 K-groups scale rearrange kernel" (#4704), review,
 *     "Additional findings": padding is zero; empty groups add nothing; the
 *     grid is over-provisioned by one chunk per group.
 *
 * Layout.  Scales are uint8 (E8M0), row-major (rows x cols) with a row
 * stride in bytes; one scale per 32 data elements.  A group's padded matrix
 * is cut into 128x4 tiles of 512 bytes, ordered row-block-major then
 * column-block-minor; element (r, c) of a tile sits at byte
 * (r%32)*16 + (r/32)*4 + c.
 *   - Groups along M (forward / dgrad): group g is rows [E'[g-1], E'[g]),
 *     padded to a multiple of 128 rows and roundup(cols, 4) columns; group g's
 *     blocked rows start at row P_g = sum_{h<g} roundup(n_h, 128) of one
 *     matrix roundup(cols, 4) wide.
 *   - Groups along K (wgrad): group g is columns [E'[g-1], E'[g]), padded to
 *     W_g = roundup(w_g, 4) columns and R = roundup(rows, 128) rows; group g's
 *     blocked matrix (R x W_g) is stored contiguously at byte R * sum_{h<g} W_h.
 *   Group ends E are int32 in device memory, cumulative (end of group g), in
 *   rows (M) or scale columns (K).  They are read only on the device and are
 *   clamped there, never rejected: E'[-1] = 0, E'[g] = min(max(E[g], E'[g-1]), T)
 *   with T = rows (M) or cols (K).  Rows (M) or columns (K) past E'[G-1] are
 *   ignored.  Every byte of the output allocation is written: real bytes,
 *   zero padding, and a zero tail after the last group; the caller need not
 *   clear `out`.
 *
 * Ownership and streams.  The caller owns every buffer.  The library never
 * allocates, frees or synchronises, never reads device memory on the host,
 * and launches only on `stream`, so every call may be captured in a CUDA
 * graph (the pointers and shapes are then frozen into the graph).  The first
 * call on a device sets kernel attributes and queries the device once; make
 * that first call before any stream capture.  Calls are thread-safe.
 *
 * Errors.  Argument faults the host can see return a status and launch
 * nothing.  A failed CUDA call returns MX_ERR_CUDA (mx_last_cuda_error gives
 * the CUDA code).
 * Bad device-side offsets are clamped as stated above.  Every wait of a
 * kernel's copy pipeline has a time limit (about 2^31 SM clocks); a kernel
 * whose wait runs out sets bit 0 of the device flags and returns early, and
 * the output of that call is then undefined (partly written).  The call
 * itself has already returned MX_OK by then: the flags (mx_device_flags) are
 * the only record, and they are shared by every call on the device, so check
 * them after a batch of calls, not per call.
 *
 * Contexts.  The library uses the CUDA context current in the calling
 * thread.  Only when no context is current does it bind the current
 * device's primary context (as the CUDA runtime would); a context the caller
 * made current, primary or not, is left in place.  Kernel attributes (the
 * shared-memory sizes) are set once per device, in the context current at
 * the library's first call on that device: make every call on a device from
 * that same context (normally the primary one).
 */
#ifndef MXSCALE_H
#define MXSCALE_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MX_OK = 0,
    MX_ERR_INVALID_ARG = 1,  /* null pointer, G outside [1, 64], negative size, stride < cols, sizes too large */
    MX_ERR_MISALIGNED = 2,   /* `out` not 16-byte aligned, or a forced path whose alignment rule fails */
    MX_ERR_UNSUPPORTED = 3,  /* shape beyond the kernels' index range */
    MX_ERR_CUDA = 4          /* a CUDA runtime or driver call failed */
} mx_status;

typedef enum { MX_GROUPS_M = 0, MX_GROUPS_K = 1 } mx_group_dim;

/* Kernel choice.  AUTO takes, in order of preference:
 *   TMA   2-D tensor-map loads: `scales` 16-byte aligned, row stride a multiple of 16;
 *   FLAT  1-D tensor-map loads of whole row blocks (groups along M only): `scales`
 *         16-byte aligned, row stride and cols multiples of 4, row stride <= 256;
 *   WORD  32-bit loads: `scales` and the row stride multiples of 4;
 *   BYTE  byte loads: anything else.
 * Forcing a path whose alignment rule fails returns MX_ERR_MISALIGNED; forcing
 * FLAT for groups along K or a stride above 256 returns MX_ERR_UNSUPPORTED. */
typedef enum { MX_PATH_AUTO = 0, MX_PATH_TMA = 1, MX_PATH_WORD = 2, MX_PATH_BYTE = 3, MX_PATH_FLAT = 4 } mx_path;

#define MX_MAX_GROUPS 64

/* Bytes the caller must allocate for `out`:
 *   M: (rows + 128 * num_groups) * roundup(cols, 4)
 *   K: roundup(rows, 128) * (cols + 4 * num_groups)
 * an upper bound on the padded output for any split of the groups, known on
 * the host without reading the offsets.  Host-only.  Returns 0 for invalid
 * arguments (and for shapes whose allocation is genuinely empty). */
size_t mx_rearranged_size(mx_group_dim dim, int64_t rows, int64_t cols, int32_t num_groups);

/* Groups along M.
 *   scales             device, uint8, element (i, j) at scales[i * row_stride + j];
 *                      any alignment; may be NULL when rows == 0 or cols == 0
 *   rows, cols         >= 0, each at most 2^31 - 2^14
 *   row_stride         bytes between rows, >= cols
 *   group_end_offsets  device, int32[num_groups], cumulative row ends
 *   num_groups         1..64
 *   out                device, 16-byte aligned, mx_rearranged_size(MX_GROUPS_M, ...) bytes,
 *                      must not overlap `scales`
 *   stream             CUDA stream (0 = legacy default stream)
 */
mx_status mx_rearrange_m_groups(const uint8_t *scales, int64_t rows, int64_t cols, int64_t row_stride,
                                const int32_t *group_end_offsets, int32_t num_groups, uint8_t *out,
                                cudaStream_t stream);

/* Groups along K: as mx_rearrange_m_groups, with group_end_offsets holding
 * cumulative scale-column ends and `out` sized by mx_rearranged_size(MX_GROUPS_K, ...). */
mx_status mx_rearrange_k_groups(const uint8_t *scales, int64_t rows, int64_t cols, int64_t row_stride,
                                const int32_t *group_end_offsets, int32_t num_groups, uint8_t *out,
                                cudaStream_t stream);

/* Either dimension with an explicit kernel choice (tests and benchmarks). */
mx_status mx_rearrange_ex(mx_group_dim dim, const uint8_t *scales, int64_t rows, int64_t cols,
                          int64_t row_stride, const int32_t *group_end_offsets, int32_t num_groups,
                          uint8_t *out, mx_path path, cudaStream_t stream);

/* Inverse of mx_rearrange_m_groups: read a blocked buffer (16-byte aligned, laid
 * out as mx_rearrange_m_groups writes it for the same rows, cols and group
 * ends) and write the row-major scales: element (i, j) at
 * scales[i * row_stride + j], any alignment.  Elements that no group covers
 * (rows at or past the last clamped end) are written as 0; bytes between
 * cols and row_stride are not touched.  The values of `blocked`'s padding
 * bytes do not matter (whole tiles are read, padding included, and ignored).
 * Same limits, clamping and stream rules as the forward call; the blocked
 * buffer must not overlap `scales`.  (The other side of the layout
 * the pytorch/ao pages convert to: #3604, 128x4 tiles in each group.) */
mx_status mx_unrearrange_m_groups(const uint8_t *blocked, int64_t rows, int64_t cols,
                                  const int32_t *group_end_offsets, int32_t num_groups, uint8_t *scales,
                                  int64_t row_stride, cudaStream_t stream);

/* Inverse of mx_rearrange_k_groups (groups along columns; uncovered columns
 * at or past the last clamped end are written as 0). */
mx_status mx_unrearrange_k_groups(const uint8_t *blocked, int64_t rows, int64_t cols,
                                  const int32_t *group_end_offsets, int32_t num_groups, uint8_t *scales,
                                  int64_t row_stride, cudaStream_t stream);

/* Padded group starts as the blocked layout uses them (pytorch/ao #3285,
 * Context: the new start of each padded group), for a consumer that would
 * otherwise rescan: starts[g] = sum_{h<g} roundup(n_h, 128) rows (M) or
 * sum_{h<g} roundup(w_h, 4) columns (K), and starts[G] = the padded total.
 * `starts` is device int32[num_groups + 1]; one warp computes it on `stream`
 * from the device offsets (clamped as above).  Group g's blocked bytes start
 * at starts[g] * roundup(cols, 4) (M) or roundup(rows, 128) * starts[g] (K). */
mx_status mx_padded_group_starts(mx_group_dim dim, int64_t rows, int64_t cols, const int32_t *group_end_offsets,
                                 int32_t num_groups, int32_t *starts, cudaStream_t stream);

/* The path AUTO would take for these arguments (host-only, no device access). */
mx_path mx_select_path(mx_group_dim dim, const void *scales, int64_t rows, int64_t cols, int64_t row_stride);

/* Static description of a status code. */
const char *mx_status_string(mx_status status);

/* Device-side error flags of the current device (bit 0: a pipeline wait ran
 * past its time limit and the kernel returned early; the output of the call
 * that set it is undefined).  The flags accumulate over every call of every
 * thread on the device until cleared, so a set bit names no call.
 * Synchronises the device: for tests and debugging, never on a hot path.
 * `clear` != 0 resets the flags after reading. */
mx_status mx_device_flags(uint32_t *flags, int clear);

/* Failure-detection self-test: launches one CTA that waits, with the same
 * bounded mbarrier wait the pipelines use, on a barrier nothing arrives at.
 * The wait gives up after `limit_cycles` SM clocks (1 .. 2^32) and sets bit 0
 * of the device flags; read them with mx_device_flags.  The kernel returns
 * normally and the context stays usable.  Asynchronous on `stream`. */
mx_status mx_selftest_bounded_wait(int64_t limit_cycles, cudaStream_t stream);

/* The CUDA error code behind the calling thread's most recent MX_ERR_CUDA
 * (0 if none): a cudaError_t, or the CUresult of a failed tensor-map encode.  The library reports launch failures from the launch's own
 * return code and never reads or clears the thread's pending CUDA error. */
int mx_last_cuda_error(void);

/* Library version, major * 10000 + minor * 100 + patch. */
int mx_version(void);

/* ---------------------------------------------------------------------------
 * Mixture-of-experts operators around the scales: slots sorted by expert,
 * token rows into expert order and back, 8-bit quantization, and the grouped
 * 8-bit product that reads both kinds of scales.
 *
 * A slot is one (token, choice) pair, slot = token * choices + choice.  The
 * rows of all experts follow one another, expert by expert, and each expert's
 * in the order of their slots; group_ends (int32[num_experts], cumulative) are
 * the group ends of every entry point here, clamped like group_end_offsets
 * above.  Slots whose expert id is outside [0, num_experts) have no row (an
 * expert of another rank): the rows behind the last group belong to nobody and
 * are written as zeros.  Indexes in device memory that are out of range are
 * skipped, never followed.
 *
 * Strides are in elements, and below 2^40 bytes (MX_ERR_UNSUPPORTED).  Outputs must not overlap inputs.  Streams, graphs,
 * contexts and the bounded waits are as described above.  Pointers
 * are aligned to their elements (MX_ERR_MISALIGNED) and rows are at least their
 * length apart (MX_ERR_INVALID_ARG); beyond that any alignment and stride is taken.
 * Rows that start on 16-byte boundaries are moved 16 bytes at a time, others less,
 * and nothing is written beside the rows of an output.  The product alone asks for 16-byte
 * aligned operand rows; its contraction is at most 2^25 long, and a row of its
 * output 2^31 - 1 bytes (MX_ERR_UNSUPPORTED). */
typedef enum { MX_F32 = 0, MX_BF16 = 1, MX_F16 = 2, MX_E4M3 = 3, MX_E5M2 = 4 } mx_dtype;

/* Bytes of workspace that mx_expert_sort needs (0 for few slots). Host-only. */
size_t mx_expert_sort_workspace(int64_t tokens, int32_t choices);

/* Sorts slots by expert, stable.
 *   expert_ids   device, int32 or int64 (id_bytes 4 or 8) [tokens, choices]
 *   group_ends   out, int32[num_experts], num_experts 1..64
 *   row_of_slot  out, int32[tokens * choices]: the slot's row, -1 if it has none
 *   slot_of_row  out, int32[tokens * choices]: the row's slot, -1 behind the last group
 *   workspace    device, 4-byte aligned; of one call at a time (two streams, or two
 *                captured graphs that may run at once, need one each) */
mx_status mx_expert_sort(const void *expert_ids, int32_t id_bytes, int64_t tokens, int32_t choices, int32_t num_experts,
                         int32_t *group_ends, int32_t *row_of_slot, int32_t *slot_of_row, void *workspace,
                         cudaStream_t stream);

/* out[row_of_slot[t, j]] = x[t] for tokens * choices rows of out (f32, bf16 or
 * f16).  Its gradient is mx_combine_rows without weights.  Rows off 8-byte boundaries
 * have less than 2^32 - 2^15 bytes (MX_ERR_UNSUPPORTED). */
mx_status mx_dispatch_rows(const void *x, mx_dtype dtype, int64_t tokens, int64_t cols, int64_t x_stride,
                           const int32_t *row_of_slot, int32_t choices, const int32_t *group_ends, int32_t num_experts,
                           void *out, int64_t out_stride, cudaStream_t stream);

/* y[t] = sum over j of weights[t, j] * rows[row_of_slot[t, j]], over slots that
 * have a row, in the order of j, in 32 bits, rounded once; weights float32
 * [tokens, choices], or NULL for ones. */
mx_status mx_combine_rows(const void *rows, mx_dtype dtype, int64_t tokens, int64_t cols, int64_t rows_stride,
                          const int32_t *row_of_slot, int32_t choices, const float *weights, void *y, int64_t y_stride,
                          cudaStream_t stream);

/* Gradient of mx_combine_rows: d_rows[row_of_slot[t, j]] = weights[t, j] * grad[t]
 * and d_weights[t, j] = <grad[t], rows[row_of_slot[t, j]]> (0 for slots without a row). */
mx_status mx_combine_rows_backward(const void *grad, mx_dtype dtype, int64_t tokens, int64_t cols, int64_t grad_stride,
                                   const void *rows, int64_t rows_stride, const int32_t *row_of_slot, int32_t choices,
                                   const int32_t *group_ends, int32_t num_experts, const float *weights, void *d_rows,
                                   int64_t d_rows_stride, float *d_weights, cudaStream_t stream);

/* 8-bit values q (e4m3 or e5m2) and E8M0 scales: the scale of a block is the
 * smallest power of two with which nothing in the block saturates, at least
 * 2^-127 (byte 0, also that of a block of zeros); q is rounded to nearest, ties
 * to even.  A block that holds a NaN or an infinity gets the scale byte 255 and
 * NaN values.
 *
 * Rows: blocks of `block` (128 or 32) consecutive columns of a row; the scale of
 * block i of row r at scales[r * scale_row_stride + i * scale_block_stride].
 * With row_of_slot (else NULL, and choices, group_ends, num_experts unused)
 * row t is quantized once and written to the rows row_of_slot[t, :] of q and
 * scales: mx_dispatch_rows and quantization in one pass. */
mx_status mx_quantize_rows(const void *x, mx_dtype dtype, int64_t rows, int64_t cols, int64_t x_stride, int32_t block,
                           mx_dtype out_dtype, const int32_t *row_of_slot, int32_t choices, const int32_t *group_ends,
                           int32_t num_experts, uint8_t *q, int64_t q_stride, uint8_t *scales, int64_t scale_row_stride,
                           int64_t scale_block_stride, cudaStream_t stream);

/* Rows that mx_quantize_cols writes: roundup(rows, 128) + 128 * num_groups.  Host-only; 0 for invalid arguments. */
int64_t mx_padded_rows(int64_t rows, int32_t num_groups);

/* Columns: blocks of 128 consecutive rows of a group in one column.  Group g
 * starts at row P_g (a multiple of 128, see mx_padded_group_starts) of q; rows
 * of q that hold no data are zeros.  q is mx_padded_rows(...) x cols, the scale
 * of rows [128 i, 128 i + 128) of column c at scales[i * scale_stride + c]. */
mx_status mx_quantize_cols(const void *x, mx_dtype dtype, int64_t rows, int64_t cols, int64_t x_stride,
                           const int32_t *group_ends, int32_t num_groups, mx_dtype out_dtype, uint8_t *q, int64_t q_stride,
                           uint8_t *scales, int64_t scale_stride, cudaStream_t stream);

/* Square blocks of 128 x 128 of `groups` matrices; scales are contiguous,
 * [groups, roundup(rows, 128) / 128, roundup(cols, 128) / 128]. */
mx_status mx_quantize_blocks(const void *x, mx_dtype dtype, int64_t groups, int64_t rows, int64_t cols, int64_t x_group_stride,
                             int64_t x_stride, mx_dtype out_dtype, uint8_t *q, int64_t q_group_stride, int64_t q_stride,
                             uint8_t *scales, cudaStream_t stream);

/* How the weights of a grouped product lie in memory. */
typedef enum { MX_B_NK = 0, MX_B_KN = 1 } mx_b_layout;

/* Grouped product, groups along the rows (forward, and the input gradient):
 *   out[r, n] = sum_k a[r, k] * b[g(r), n, k], each value times its scale,
 * accumulated in 32 bits by the tensor cores.  rows of a behind the last group
 * give rows of zeros.  a and b are e4m3 or e5m2 (each its own), 16-byte aligned
 * with row (and, of b, group) strides that are multiples of 16; out is f32,
 * bf16 or f16.
 *   b_layout  MX_B_NK: b is [G, n, k]; MX_B_KN: b is [G, k, n], the forward
 *             weights as they are stored, read for the gradient of the input
 *   block 128 a's scales cover 128 values of a row (a_scales[r * row_stride +
 *             i * block_stride]); b's cover 128 x 128 (b_scales[g * group_stride +
 *             (n / 128) * n_stride + (k / 128) * k_stride])
 *   block 32  both scales lie in the blocked layout, 16-byte aligned, strides
 *             unused: a's as mx_rearrange_m_groups writes [rows, k / 32] for
 *             group_ends, b's as it writes [G * n, k / 32] for groups of n rows;
 *             MX_B_NK only */
mx_status mx_grouped_matmul_m(const void *a, mx_dtype a_dtype, int64_t a_stride, const uint8_t *a_scales,
                              int64_t a_scale_row_stride, int64_t a_scale_block_stride, const void *b, mx_dtype b_dtype,
                              mx_b_layout b_layout, int64_t b_group_stride, int64_t b_stride, const uint8_t *b_scales,
                              int64_t b_scale_group_stride, int64_t b_scale_n_stride, int64_t b_scale_k_stride,
                              int32_t block, int64_t rows, int64_t n, int64_t k, const int32_t *group_ends,
                              int32_t num_groups, void *out, mx_dtype out_dtype, int64_t out_stride, cudaStream_t stream);

/* Grouped product, groups along the contraction (the weight gradient):
 *   out[g, m, n] = sum over the rows r of group g of a[r, m] * b[r, n]
 * with a [padded_rows, m] and b [padded_rows, n] and their scales as
 * mx_quantize_cols lays them out (groups at padded starts, zeros between).
 * group_ends are the ends without padding.  A group without rows gives zeros. */
mx_status mx_grouped_matmul_k(const void *a, mx_dtype a_dtype, int64_t a_stride, const uint8_t *a_scales,
                              int64_t a_scale_stride, const void *b, mx_dtype b_dtype, int64_t b_stride,
                              const uint8_t *b_scales, int64_t b_scale_stride, int64_t padded_rows, int64_t m, int64_t n,
                              const int32_t *group_ends, int32_t num_groups, void *out, mx_dtype out_dtype,
                              int64_t out_group_stride, int64_t out_stride, cudaStream_t stream);

/* How a grouped product is spread over the SMs: 128 x 128 tiles of one CTA each, or of
 * 2, 4 or 8 CTAs that share a tile's contraction; 128 x 256 tiles; 256 x 256 tiles of
 * pairs of CTAs, or of the transposed product (weight gradients only). */
typedef enum { MX_TILES_NONE = 0, MX_TILES_NARROW = 1, MX_TILES_SPLIT_2 = 2, MX_TILES_SPLIT_4 = 4, MX_TILES_SPLIT_8 = 8,
               MX_TILES_WIDE = 16, MX_TILES_PAIRS = 32, MX_TILES_PAIRS_ACROSS = 33 } mx_tiles;

/* The tiles that the grouped products take on a device of `sms` SMs (host-only):
 * MX_GROUPS_M for mx_grouped_matmul_m (m its rows), MX_GROUPS_K for
 * mx_grouped_matmul_k (k its padded rows).  MX_TILES_NONE for invalid arguments. */
mx_tiles mx_select_tiles(mx_group_dim dim, int64_t m, int64_t n, int64_t k, int32_t num_groups, int32_t sms);

#ifdef __cplusplus
}
#endif
#endif /* MXSCALE_H */
