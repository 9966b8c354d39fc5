/*
 * fp8q.h -- C ABI of libfp8q, FP8 / MXFP8 quantization for sm_103a (GB300).
 *
 * The library quantizes BF16 or FP32 tensors to 8-bit floats, the step that
 * runs before each Fprop / Dgrad / Wgrad matmul of FP8 training:
 *   - per-tensor amax, current scaling and delayed scaling, each followed by
 *     a saturating round-to-nearest-even cast to E4M3 or E5M2;
 *   - MXFP8: 1x32 blocks with one E8M0 scale each (exponent rounded up),
 *     rowwise and columnwise (transposed), optionally per ragged group;
 * and the steps around it: dequantization, blockwise FP8, NVFP4, the
 * SQNR / zero-rate statistics of a quantized copy, the products of blockwise
 * copies, the expert layer that feeds and joins them, and what stands around
 * it in a block: the norm with the residual, the gated activation, the layer
 * for a few tokens in one call, the gradients' norm and clip.
 *
 * Conventions for every entry point:
 *   - Pointers documented as "device" are CUDA device pointers owned by the
 *     caller; the library never frees them and never allocates on these
 *     calls (only fp8q_delayed_create allocates, for its own state).
 *   - All work is asynchronous on `stream` (a cudaStream_t passed as void*,
 *     NULL = the legacy default stream).  Return codes report argument
 *     validation and launch errors only; fp8q_last_error_string() gives the
 *     message of the most recent failure on the calling thread.
 *   - Inputs are contiguous row-major tensors; x must be 16-byte aligned.
 *     dt selects the element type: FP8Q_IN_BF16 (raw BF16 bits) or
 *     FP8Q_IN_FP32.  Outputs are raw 8-bit codes (uint8).
 *   - Groups: group_offsets is a device int64 array of num_groups + 1 row
 *     offsets, non-decreasing, from 0 to rows; group g is rows
 *     [offsets[g], offsets[g+1]).  NULL means one group of all rows
 *     (num_groups must then be 1).  Offsets that break these rules give
 *     unspecified values but never an out-of-bounds access.
 *   - num_groups is at most FP8Q_MAX_GROUPS.
 *
 * Readings of the source pages that fix bit-level results (the same as the
 * CPU oracle's): a NaN input encodes to 0x7F in both formats; +-Inf and any
 * overflow saturate to +-max; the sign of zero is kept except in an all-zero
 * MX block; amax compares magnitude bits, so NaN inputs make amax NaN.
 */
#ifndef FP8Q_H
#define FP8Q_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define FP8Q_MAX_GROUPS 4096

#if defined(__GNUC__)
#define FP8Q_API __attribute__((visibility("default")))
#else
#define FP8Q_API
#endif

typedef enum {
    FP8Q_OK = 0,
    FP8Q_ERR_INVALID_ARG = 1, /* a pointer, size, enum or alignment is invalid */
    FP8Q_ERR_UNSUPPORTED = 2, /* valid request the library does not handle (e.g. cols % 32 for MX) */
    FP8Q_ERR_CUDA = 3,        /* a CUDA call or kernel launch failed */
    FP8Q_ERR_TIMEOUT = 4      /* a bounded device-side wait gave up */
} fp8q_status;

typedef enum { FP8Q_IN_BF16 = 0, FP8Q_IN_FP32 = 1 } fp8q_in_dtype;

/* E4M3: bias 7, no Inf, max 448.  E5M2: IEEE style, bias 15, max 57344.
 * ("混合精度与 FP8 训练", 2.2; "Blackwell GPU MXFP8 预训练最佳实践", 3.1)
 * MX element formats below 8 bits, for mx_quantize_fp4_fp6 only: E2M1
 * (MXFP4: 0, 0.5, 1, 1.5, 2, 3, 4, 6; "混合精度与 FP8 训练" 13.2) and the
 * MXFP6 pair E2M3 (bias 1, max 7.5) and E3M2 (bias 3, max 28), read as the
 * OCP microscaling formats that "Blackwell GPU MXFP8 预训练最佳实践" 3.2
 * names without defining.  None has Inf or NaN. */
typedef enum { FP8Q_E4M3 = 0, FP8Q_E5M2 = 1, FP8Q_E2M1 = 2, FP8Q_E2M3 = 3, FP8Q_E3M2 = 4 } fp8q_format;

typedef enum { MXFP8_ROW = 1, MXFP8_COL = 2, MXFP8_BOTH = 3 } mxfp8_dir;

/* MX scale rule.  FP8Q_MX_RULE_UP: X = ceil(log2(amax / destmax)), the
 * round-up rule ("Blackwell GPU MXFP8 预训练最佳实践" 4.1, Algorithm 1);
 * FP8Q_MX_RULE_OCP: X = floor(log2(amax)) - e_max, the OCP rule ("混合精度与
 * FP8 训练" 13.1; e_max = 8 for E4M3, 15 for E5M2), which can put elements
 * above the format maximum (they saturate).  Both saturate X to [-127, 127]. */
typedef enum { FP8Q_MX_RULE_UP = 0, FP8Q_MX_RULE_OCP = 1 } fp8q_mx_rule;

/* Blockwise group shapes.  FP8Q_BLOCK_1X128: 1x128 groups (one token's 128
 * channels) for the rowwise copy, 128x1 groups for the transposed copy;
 * FP8Q_BLOCK_128X128: 128x128 blocks, whose transposed copy is the same
 * blocks transposed. */
typedef enum { FP8Q_BLOCK_1X128 = 1, FP8Q_BLOCK_128X128 = 128 } fp8q_block;

/* Scores of the routing: over all experts of a token, or of each alone. */
typedef enum { FP8Q_SCORE_SOFTMAX = 0, FP8Q_SCORE_SIGMOID = 1 } fp8q_score;

/* Output type of the dequantizers and of the products. */
typedef enum { FP8Q_OUT_BF16 = 0, FP8Q_OUT_FP32 = 1 } fp8q_out_dtype;

/* Library version (major * 10000 + minor * 100 + patch). */
FP8Q_API int32_t fp8q_version(void);

/* Message of the last failed call on this thread ("" if none). */
FP8Q_API const char* fp8q_last_error_string(void);

/*
 * Synchronizes `stream`, then reports and clears device-side failures that
 * earlier calls on this device recorded: FP8Q_ERR_TIMEOUT when a bounded
 * wait inside a kernel (the shared-memory barriers of the MXFP8, the
 * blockwise and the products' pipelines, the grid-wide wait for the scale in the single-launch
 * current scaling) gave up, in which case that call's outputs are
 * incomplete.  FP8Q_OK otherwise.
 */
FP8Q_API fp8q_status fp8q_check_device(void* stream);

/*
 * Time budget of every bounded device-side wait, in nanoseconds (default
 * 1e9), for kernels launched afterwards on the current device.  No wait
 * gives up before its budget is over, nor spins much longer: the clock is
 * read every 16 tries, in the products from some 100 us on.  A stalled
 * pipeline ends its kernel and is reported by fp8q_check_device.
 */
FP8Q_API fp8q_status fp8q_set_wait_budget_ns(uint64_t ns);

/*
 * Test hook for the failure path above (the pages have no counterpart).
 * While `on` is nonzero, the BF16 MXFP8 kernel's producer warp issues no
 * loads, so its consumers' waits for data can never complete: each gives up
 * after the wait budget, the call's outputs are left unwritten and
 * fp8q_check_device reports FP8Q_ERR_TIMEOUT.  No copy is in flight when
 * the kernel ends.  Applies to kernels launched afterwards on the current
 * device; leave it off (the default) outside such tests.
 */
FP8Q_API fp8q_status fp8q_debug_stall_mx_producer(int32_t on);

/*
 * Test hook for the same failure path in the single-launch current scaling
 * of fp8q_cast_per_tensor (taken for an ungrouped tensor of more than 2 MB
 * and up to about 160M BF16 elements; smaller ones take a one-cluster
 * kernel that has no grid-wide wait).  While `on` is nonzero, the CTA
 * that should publish the scale does not, so every other CTA's wait for it
 * gives up after the wait budget: no codes are written, fp8q_check_device
 * reports FP8Q_ERR_TIMEOUT, and the workspace is zero-filled again by the
 * last CTA to leave.  Applies to kernels launched afterwards on the current
 * device; leave it off (the default) outside such tests.
 */
FP8Q_API fp8q_status fp8q_debug_stall_scale_publish(int32_t on);

/*
 * Test hook for the same failure path in the products.  While `on` is
 * nonzero, fp8q_matmul_blockwise and the grouped products issue no loads, so
 * their waits for data run out: fp8q_check_device reports FP8Q_ERR_TIMEOUT,
 * and the call's output is worthless.  Applies to kernels launched
 * afterwards on the current device; leave it off (the default) outside such
 * tests.
 */
FP8Q_API fp8q_status fp8q_debug_stall_matmul_loads(int32_t on);

/*
 * amax_out[g] = max |x| over group g, bit-exact: the FP32 value whose bits
 * are the largest magnitude bits in the group (BF16 widened exactly), so a
 * NaN makes the result NaN and an empty group gives 0.
 * ("HiFloat8：高性能训练之路" 1.2, ComputeAmax; "混合精度与 FP8 训练" 8.1.)
 *   x           device, rows*cols elements of type dt
 *   amax_out    device float[num_groups]
 * One reduction pass over x (2 or 4 bytes per element read).
 */
FP8Q_API fp8q_status fp8q_amax(const void* x, int32_t dt, int64_t rows, int64_t cols,
                      const int64_t* group_offsets, int32_t num_groups, float* amax_out,
                      void* stream);

/*
 * scale_out[g] = fl32(fl32(F8max / amax[g]) * 2^-margin) and
 * scale_inv_out[g] = fl32(1 / scale_out[g]), with the same special cases as
 * current scaling (amax 0 or non-finite -> scale 1; a quotient above FLT_MAX
 * -> FLT_MAX).  ("HiFloat8：高性能训练之路" 1.2, eqs. 1 and 3; "混合精度与 FP8
 * 训练" 8.2, the margin.)  It is the scale step of current scaling on its
 * own, for a tensor split across devices: each device takes fp8q_amax of
 * its part, the amaxes are combined with a MAX all-reduce (on the FP32 bit
 * patterns as int32, which keeps NaN), and each device casts its part with
 * fp8q_cast_per_tensor(scale_in = scale_out).
 *   amax           device float[num_groups] (taken by magnitude)
 *   scale_out      device float[num_groups]
 *   scale_inv_out  device float[num_groups] or NULL
 */
FP8Q_API fp8q_status fp8q_scale_from_amax(const float* amax, int32_t num_groups, int32_t fmt,
                                          int32_t margin, float* scale_out, float* scale_inv_out,
                                          void* stream);

/*
 * Bytes of workspace fp8q_cast_per_tensor needs for num_groups groups.
 */
FP8Q_API size_t fp8q_cast_workspace_bytes(int32_t num_groups);

/*
 * Per-tensor (per-group) scaled cast:  q = RNE_sat(fl32(x * scale[g])).
 *
 * scale_in == NULL: current scaling ("HiFloat8：高性能训练之路" 1.2, eqs.
 *   1-2; "混合精度与 FP8 训练" 8.2): amax[g] is reduced first, then
 *   scale[g] = fl32(fl32(F8max / amax[g]) * 2^-margin), with amax = 0 giving
 *   scale 1, a non-finite amax giving scale 1, and an overflowing quotient
 *   giving FLT_MAX.  Two passes over x (read, read + write) in two
 *   launches, except for an ungrouped tensor of up to about 160M BF16
 *   elements on a GB300, which takes one launch: up to 2 MB of x, one
 *   thread-block cluster of 16 CTAs holds it in shared memory and
 *   exchanges the amax between them; beyond that, the 32 KB slices that
 *   fit one or two per resident CTA (about 20M elements) stay on chip
 *   (registers, shared memory) while the scale is published and are read
 *   once, and the rest of the tensor is streamed by the same CTAs and read
 *   twice, partly from L2.
 * scale_in != NULL: device float[num_groups] scales are used as given; if
 *   amax_out is non-NULL the amax of x is reduced in the same single pass.
 *
 *   x              device, rows*cols elements of type dt
 *   fmt            FP8Q_E4M3 or FP8Q_E5M2
 *   margin         0..63
 *   q              device uint8[rows*cols], same layout as x
 *   amax_out       device float[G] or NULL
 *   scale_out      device float[G] or NULL: the scale used
 *   scale_inv_out  device float[G] or NULL: fl32(1 / scale)
 *   sat_count_out  device uint64[G] or NULL: elements with |fl32(x*scale)|
 *                  > F8max (NaN not counted), i.e. clamped by the cast
 *   workspace      device, >= fp8q_cast_workspace_bytes(num_groups) bytes,
 *                  8-byte aligned, zero-filled before its first use; every
 *                  successful call leaves it zero-filled again (after a
 *                  call that fp8q_check_device reports as timed out, fill
 *                  it with zeros again).  Calls that may overlap on the GPU
 *                  need separate workspaces.
 */
FP8Q_API fp8q_status fp8q_cast_per_tensor(const void* x, int32_t dt, int64_t rows, int64_t cols,
                                 const int64_t* group_offsets, int32_t num_groups,
                                 int32_t fmt, int32_t margin, const float* scale_in,
                                 uint8_t* q, float* amax_out, float* scale_out,
                                 float* scale_inv_out, unsigned long long* sat_count_out,
                                 void* workspace, size_t workspace_bytes, void* stream);

/*
 * fp8q_cast_per_tensor without a caller workspace.  The source pages have
 * no counterpart to this entry point; it exists for callers that cannot
 * allocate device memory where they quantize (a plugin inside a host
 * application whose allocator owns all device memory, or a step where a
 * cudaMalloc / cudaFree would synchronize the device).  It allocates
 * nothing: the workspace is a fixed 8 KB array in the library's device
 * memory, present on every GPU that loads the library until the process
 * exits.
 *   - Arguments and results are those of fp8q_cast_per_tensor, minus the
 *     workspace; num_groups must be at most 256 (FP8Q_ERR_INVALID_ARG
 *     otherwise).
 *   - The first call on each device looks up the array's device address
 *     and keeps it; make that first call before any stream capture.  A
 *     context reset (cudaDeviceReset) is not supported afterwards: the
 *     array may be reloaded at another address.
 *   - All calls on a device share the array.  A call checks its arguments
 *     first (a rejected call touches nothing), then clears the part it
 *     uses (one small zeroing kernel on `stream`).  Calls whose work may
 *     overlap on the GPU race on it: order them on one stream.
 */
FP8Q_API fp8q_status fp8q_cast_per_tensor_static_ws(const void* x, int32_t dt, int64_t rows, int64_t cols,
                                                    const int64_t* group_offsets, int32_t num_groups,
                                                    int32_t fmt, int32_t margin, const float* scale_in,
                                                    uint8_t* q, float* amax_out, float* scale_out,
                                                    float* scale_inv_out, unsigned long long* sat_count_out,
                                                    void* stream);

/*
 * Delayed scaling ("HiFloat8：高性能训练之路" 1.2 eqs. 3-4 and section 3;
 * "混合精度与 FP8 训练" 8.2): a library-owned state holds an amax history
 * ring of history_len entries.  Step t:
 *   - if the history is empty (after create or reset): current scaling with
 *     no margin on x_t;
 *   - else scale = fl32(fl32(F8max / max(filled history)) * 2^-margin);
 *   - q_t = RNE_sat(fl32(x_t * scale));
 *   - if t % interval == 0 (t counted from create/reset), amax(x_t) is
 *     computed in the same pass and appended, dropping the oldest entry when
 *     the ring is full; a non-finite amax raises the state's flag.
 * The host keeps step, head and count, so the call never synchronizes.
 */
typedef struct fp8q_delayed_state fp8q_delayed_state;

/* Allocates the state on the current device (history_len 1..1024,
 * interval >= 1, margin 0..63).  That device owns the state: reset and step
 * must be called with it current (FP8Q_ERR_INVALID_ARG otherwise); get, set
 * and destroy switch to it themselves and restore the caller's device. */
FP8Q_API fp8q_status fp8q_delayed_create(int32_t history_len, int32_t interval, int32_t margin,
                                int32_t fmt, fp8q_delayed_state** out);
FP8Q_API fp8q_status fp8q_delayed_destroy(fp8q_delayed_state* st);
/* Empties the history and clears the flag (async on stream); step = 0. */
FP8Q_API fp8q_status fp8q_delayed_reset(fp8q_delayed_state* st, void* stream);
/*
 *   x, n            device, n elements of type dt
 *   q               device uint8[n]
 *   scale_used_out  device float[1] or NULL; scale_inv_out likewise
 *   amax_out        device float[1] or NULL: written on recording steps only
 *   sat_count_out   device uint64[1] or NULL
 * Consecutive steps on one state must be issued on one stream (or ordered).
 */
FP8Q_API fp8q_status fp8q_delayed_step(fp8q_delayed_state* st, const void* x, int32_t dt, int64_t n,
                              uint8_t* q, float* scale_used_out, float* scale_inv_out,
                              float* amax_out, unsigned long long* sat_count_out,
                              void* stream);
/* Copies the state to the host (synchronizes the state's device): history_host
 * float[history_len] (ring order), head (next slot), count (filled entries),
 * step, nonfinite flag.  Any output pointer may be NULL. */
FP8Q_API fp8q_status fp8q_delayed_get(const fp8q_delayed_state* st, float* history_host, int32_t* head,
                             int32_t* count, int64_t* step, int32_t* nonfinite);
/* Restores a state saved by fp8q_delayed_get (checkpoint resume); clears
 * the flag.  Synchronous. */
FP8Q_API fp8q_status fp8q_delayed_set(fp8q_delayed_state* st, const float* history_host, int32_t head,
                             int32_t count, int64_t step);

/*
 * Number of columnwise MX blocks per column: sum over groups of
 * ceil(n_g / 32), from HOST offsets (NULL: ceil(rows / 32)).  Returns -1 for
 * invalid offsets.
 */
FP8Q_API int64_t mxfp8_col_blocks(const int64_t* group_offsets_host, int32_t num_groups, int64_t rows);

/*
 * MXFP8 quantization ("Blackwell GPU MXFP8 预训练最佳实践" 4.1-4.2;
 * "混合精度与 FP8 训练" 13.1; "HiFloat8：高性能训练之路" 2), one pass over x.
 * Each block of k <= 32 values gets X = ceil(log2(amax / destmax)) computed
 * exactly and saturated to [-127, 127] (destmax 448 for E4M3, 57344 for
 * E5M2); the scale byte is X + 127 (E8M0), elements are RNE_sat(v / 2^X).
 * amax = 0 gives byte 0x00 and all-zero elements; a block holding Inf or
 * NaN gives byte 0xFF and elements 0x7F.
 *   rowwise (dir & MXFP8_ROW): blocks x[r, 32j .. 32j+31]
 *     q_row  device uint8[rows * cols]          (row-major, like x)
 *     s_row  device uint8[rows * (cols / 32)]   (row-major)
 *   columnwise (dir & MXFP8_COL): per group, blocks of 32 consecutive rows
 *     from the group's first row, the last one possibly shorter; taken from
 *     x itself, not from the rowwise copy; output transposed:
 *     q_col  device uint8[cols * rows]          q_col[c * rows + r]
 *     s_col  device uint8[cols * s_col_ld]      s_col[c * s_col_ld + b], b
 *            numbering the column blocks of all groups in order; s_col_ld
 *            must be >= mxfp8_col_blocks(...) for the offsets used (blocks
 *            past s_col_ld are not written); an s_col_ld that is a
 *            multiple of 16 keeps every scale row 16-byte aligned, which
 *            the grouped path stores faster
 * cols % 32 == 0 is required (FP8Q_ERR_UNSUPPORTED otherwise); rows is any.
 * x is 16-byte aligned and q_row 32-byte aligned (a block's 32 codes leave
 * in one 32-byte store; FP8Q_ERR_INVALID_ARG otherwise).  Pointers of the
 * unused direction may be NULL.  A rejected call writes nothing.
 */
FP8Q_API fp8q_status mxfp8_quantize(const void* x, int32_t dt, int64_t rows, int64_t cols,
                           const int64_t* group_offsets, int32_t num_groups, int32_t fmt,
                           int32_t dir, uint8_t* q_row, uint8_t* s_row, uint8_t* q_col,
                           uint8_t* s_col, int64_t s_col_ld, void* stream);

/*
 * mxfp8_quantize with a choice of scale rule (fp8q_mx_rule) and an optional
 * count of saturated elements: those whose scaled magnitude |v / 2^X|
 * exceeds the format maximum and are clamped to it ("Blackwell GPU MXFP8
 * 预训练最佳实践" 4.1 compares the two rules by exactly this saturation).
 *   sat_count  device uint64[2] or NULL: [0] rowwise copy, [1] columnwise
 *              copy; zeroed by the call, then accumulated on the stream.
 * Never saturates under FP8Q_MX_RULE_UP.  Other arguments as mxfp8_quantize.
 */
FP8Q_API fp8q_status mxfp8_quantize_rule(const void* x, int32_t dt, int64_t rows, int64_t cols,
                                         const int64_t* group_offsets, int32_t num_groups, int32_t fmt,
                                         int32_t dir, int32_t scale_rule, uint8_t* q_row, uint8_t* s_row,
                                         uint8_t* q_col, uint8_t* s_col, int64_t s_col_ld,
                                         unsigned long long* sat_count, void* stream);

/*
 * Scale layouts of mxfp8_quantize_ex.  FP8Q_SCALES_ROW_MAJOR is the layout of
 * mxfp8_quantize.  FP8Q_SCALES_MMA_128X4 writes the same scales straight into
 * the 128 x 4 block layout that block-scaled tensor-core MMA reads, the
 * layout mx_scales_to_mma_layout produces from row-major scales (the pages
 * give none; "Blackwell GPU MXFP8 预训练最佳实践" 3.2 only says the tensor
 * cores take the MX types natively): the scale matrix is padded to 128-row
 * and 4-column multiples and cut into 512-byte blocks, stored block row by
 * block row; scale (r, c) sits at byte (r % 32) * 16 + (r / 32 % 4) * 4 +
 * c % 4 of its block.  Padding bytes are 0.
 */
typedef enum { FP8Q_SCALES_ROW_MAJOR = 0, FP8Q_SCALES_MMA_128X4 = 1 } fp8q_scale_layout;

/* Bytes of a scale matrix of rows x scale_cols in the 128 x 4 block layout:
 * ceil(rows / 128) * 128 * ceil(scale_cols / 4) * 4 (-1 for negative sizes). */
FP8Q_API int64_t mxfp8_mma_scale_bytes(int64_t rows, int64_t scale_cols);

/*
 * mxfp8_quantize_rule with a choice of scale layout (fp8q_scale_layout).
 * Under FP8Q_SCALES_MMA_128X4:
 *   s_row  device uint8[mxfp8_mma_scale_bytes(rows, cols / 32)]
 *   s_col  device uint8[mxfp8_mma_scale_bytes(cols, s_col_ld)], the columnwise
 *          scales as a cols x s_col_ld matrix; s_col_ld must be the column
 *          block count itself (mxfp8_col_blocks; checked without groups, a
 *          precondition with groups), so that no block index is padding
 * Both are written in full: the kernels store every scale and, for shapes
 * with padding (rows or cols not a multiple of 128, cols / 32 or s_col_ld
 * not a multiple of 4) and for FP32 input, the call clears the buffer with
 * one cudaMemsetAsync first.  Other arguments as mxfp8_quantize_rule.
 */
FP8Q_API fp8q_status mxfp8_quantize_ex(const void* x, int32_t dt, int64_t rows, int64_t cols,
                                       const int64_t* group_offsets, int32_t num_groups, int32_t fmt,
                                       int32_t dir, int32_t scale_rule, int32_t scale_layout, uint8_t* q_row,
                                       uint8_t* s_row, uint8_t* q_col, uint8_t* s_col, int64_t s_col_ld,
                                       unsigned long long* sat_count, void* stream);

/*
 * MXFP4 / MXFP6 quantization ("混合精度与 FP8 训练" 13.1-13.2; "Blackwell
 * GPU MXFP8 预训练最佳实践" 3.2 and 4.1): blocks of 32 elements with one E8M0
 * scale, as mxfp8_quantize_rule but with element format elem (FP8Q_E2M1,
 * FP8Q_E2M3 or FP8Q_E3M2): destmax 6, 7.5 or 28 under FP8Q_MX_RULE_UP, e_max
 * 2, 2 or 4 under FP8Q_MX_RULE_OCP.  Elements are the nearest codes of
 * v / 2^X, saturating.  A block whose amax is 0 gets scale byte 0 and +0
 * codes; one holding Inf or NaN gets 0xFF and +0 codes.  One pass over x
 * writes both copies.  No groups.
 *   rowwise (dir & MXFP8_ROW):
 *     q_row  E2M1: device uint8 [rows][cols / 2], two codes per byte, the
 *                  even element in the low nibble; FP6: [rows][cols], one
 *                  code per byte in bits 0-5
 *     s_row  device uint8 [rows][cols / 32]
 *   columnwise (dir & MXFP8_COL): blocks of 32 rows (the last one shorter),
 *   stored transposed:
 *     q_col  E2M1: [cols][rows / 2] (rows must be even); FP6: [cols][rows]
 *     s_col  device uint8 [cols][ceil(rows / 32)]
 *   sat_count  device uint64[2] or NULL: elements whose |v / 2^X| exceeds
 *              destmax (clamped), [0] rowwise, [1] columnwise; zeroed by
 *              the call.  Never nonzero under FP8Q_MX_RULE_UP.
 * cols % 32 == 0 (FP8Q_ERR_UNSUPPORTED otherwise); q_row and q_col 16-byte
 * aligned; pointers of an unused copy may be NULL.
 */
FP8Q_API fp8q_status mx_quantize_fp4_fp6(const void* x, int32_t dt, int64_t rows, int64_t cols, int32_t elem,
                                         int32_t dir, int32_t scale_rule, uint8_t* q_row, uint8_t* s_row,
                                         uint8_t* q_col, uint8_t* s_col, unsigned long long* sat_count,
                                         void* stream);

/*
 * Blockwise FP8 with one FP32 scale per group ("混合精度与 FP8 训练" 10.2:
 * activations in 1x128 groups, weights in 128x128 blocks, along the GEMM
 * reduction dimension; 10.3: scales taken online from each group's amax;
 * 10.4: optionally integer powers of two; 10.5: the transposed copy of a
 * 1x128-grouped tensor is quantized from x in 128x1 groups, never from the
 * rowwise codes).  Per group: scale = fl32(F8max / amax) with the
 * per-tensor special cases (amax 0 or non-finite -> 1, overflow -> FLT_MAX),
 * rounded down to a power of two when pow2_scales is set; q =
 * RNE_sat(fl32(x * scale)); scale_inv = fl32(1 / scale) is stored.
 *   x            device BF16 [rows][cols]; cols % 16 == 0, and rows % 16 == 0
 *                for the transposed copy (FP8Q_ERR_UNSUPPORTED otherwise,
 *                and for FP32 input)
 *   block        fp8q_block
 *   dir          MXFP8_ROW, MXFP8_COL or MXFP8_BOTH
 *   q            device uint8 [rows][cols] (rowwise copy)
 *   scale_inv    device float: 1x128 -> [rows][ceil(cols/128)];
 *                128x128 -> [ceil(rows/128)][ceil(cols/128)]
 *   q_t          device uint8 [cols][rows] (transposed copy)
 *   scale_inv_t  device float: 128x1 -> [cols][ceil(rows/128)];
 *                128x128 -> [ceil(cols/128)][ceil(rows/128)]
 * Pointers of the unused copy may be NULL; x, q and q_t 16-byte aligned.
 */
FP8Q_API fp8q_status fp8q_quantize_blockwise(const void* x, int32_t dt, int64_t rows, int64_t cols, int32_t fmt,
                                             int32_t block, int32_t pow2_scales, int32_t dir, uint8_t* q,
                                             float* scale_inv, uint8_t* q_t, float* scale_inv_t, void* stream);

/*
 * The product of two blockwise FP8 tensors, both stored with the reduction
 * last (the copies fp8q_quantize_blockwise writes):
 *   out[i][j] = sum_kb sa[i][kb] * sb(j, kb) * sum_{k in block kb} A[i][k] * B[j][k]
 * with A, B the values of the codes and sa, sb their scale_inv ("混合精度与
 * FP8 训练" 10.2-10.5: 1x128 activations, 128x128 weights, blocks along the
 * reduction).  The inner sums are the tensor core's, the outer sum is FP32;
 * BF16 output is rounded once, to nearest even.  The three products of a
 * linear layer y = x W^T (x [T][K], W [N][K]):
 *   Fprop  a = x.q     b = W.q    (128x128)   out [T][N]
 *   Dgrad  a = dy.q    b = W.q_t  (128x128)   out [T][K]
 *   Wgrad  a = dy.q_t  b = x.q_t  (1x128)     out [N][K]
 *   a            device uint8 [m][k], 16-byte aligned, a_fmt codes
 *   a_scale_inv  device float [m][ceil(k/128)]
 *   b            device uint8 [n][k], 16-byte aligned, b_fmt codes (the
 *                formats may differ)
 *   b_scale_inv  device float: FP8Q_BLOCK_1X128 -> [n][ceil(k/128)];
 *                FP8Q_BLOCK_128X128 -> [ceil(n/128)][ceil(k/128)]
 *   out          device BF16 or FP32 [m][n] (out_dt, fp8q_out_dtype)
 *   accumulate   nonzero: out += the product (FP32 output only)
 * m and n are any, k % 16 == 0 (FP8Q_ERR_UNSUPPORTED otherwise); k == 0
 * gives zeros.  NaN and Inf codes propagate as in the sum above.  sa * sb is
 * formed first, in FP32: where that product leaves FP32's normal range a block
 * loses digits or overflows, even if its sum would not have.
 */
FP8Q_API fp8q_status fp8q_matmul_blockwise(const uint8_t* a, const float* a_scale_inv, int32_t a_fmt,
                                           const uint8_t* b, const float* b_scale_inv, int32_t b_fmt,
                                           int32_t b_block, int64_t m, int64_t n, int64_t k, int32_t out_dt,
                                           int32_t accumulate, void* out, void* stream);

/*
 * The experts' products: rows of group g of a times the g-th matrix of b,
 *   out[i][j] = sum_k A[i][k] * B[g][j][k],  group_offsets[g] <= i < group_offsets[g + 1],
 * with the scales of fp8q_matmul_blockwise (b in 128x128 blocks).  Groups
 * may start at any row and be empty; rows in no group are not written.
 *   a              device uint8 [rows][k];  a_scale_inv [rows][ceil(k/128)]
 *   b              device uint8 [num_groups][n][k]
 *   b_scale_inv    device float [num_groups][ceil(n/128)][ceil(k/128)]
 *   group_offsets  device int64 [num_groups + 1], required
 *   out            device BF16 or FP32 [rows][n]
 */
FP8Q_API fp8q_status fp8q_matmul_grouped(const uint8_t* a, const float* a_scale_inv, int32_t a_fmt,
                                         const uint8_t* b, const float* b_scale_inv, int32_t b_fmt,
                                         const int64_t* group_offsets, int32_t num_groups, int64_t rows, int64_t n,
                                         int64_t k, int32_t out_dt, void* out, void* stream);

/*
 * The experts' weight gradients: a reduction over each group's rows of two
 * transposed copies,
 *   out[g][i][j] = sum over the rows r of group g of A[i][r] * B[j][r].
 *   a_t            device uint8 [m][rows];  a_scale_inv_t [m][ceil(rows/128)]
 *   b_t            device uint8 [n][rows];  b_scale_inv_t [n][ceil(rows/128)]
 *   group_offsets  device int64 [num_groups + 1]: multiples of 128, so that
 *                  no 128x1 scale group spans two groups; the last may be
 *                  rows itself.  (Others give unspecified values.)
 *   out            device BF16 or FP32 [num_groups][m][n]; an empty group's
 *                  matrix is zero (left as it is with accumulate)
 * rows % 16 == 0 (FP8Q_ERR_UNSUPPORTED otherwise); accumulate as above.
 */
FP8Q_API fp8q_status fp8q_matmul_grouped_wgrad(const uint8_t* a_t, const float* a_scale_inv_t, int32_t a_fmt,
                                               const uint8_t* b_t, const float* b_scale_inv_t, int32_t b_fmt,
                                               const int64_t* group_offsets, int32_t num_groups, int64_t rows,
                                               int64_t m, int64_t n, int32_t out_dt, int32_t accumulate, void* out,
                                               void* stream);

/*
 * Routing of tokens to experts (the pages' MoE workload takes its group
 * offsets as given; this and the plan below make them).  Scores s are a
 * softmax of a token's logits, or 1 / (1 + exp(-x)) of each.  Keys are
 * s + bias, or the logits themselves when there is neither a bias nor more
 * than one group (the same order).  With num_groups > 1, a group of
 * experts / num_groups consecutive experts is worth the sum of its two best
 * keys (its only one if it has one expert) and only the top_groups best
 * groups stay.  The top_k best keys are chosen, best first; equal keys and
 * equal groups go to the lowest index.  Weights are
 *   weight_scale * s_j / (sum of the chosen s)   with renormalize,
 *   weight_scale * s_j                           without.
 * A logit that is -inf or NaN, or whose key is, is never chosen (its key
 * counts as -inf in its group); where fewer than top_k are left, the last
 * ids are -1 and their weights 0.  Weights are 0, too, where renormalize finds
 * that all chosen sigmoid scores are 0 in FP32 (logits below -88).  A NaN logit, under softmax also +inf,
 * makes all the token's weights NaN.  Arithmetic is FP32.
 *   logits   device BF16 or FP32 (dt) [tokens][experts], experts <= 1024
 *   top_k    1..32, at most experts / num_groups * top_groups
 *   bias     device float [experts] or NULL
 *   num_groups  1..32, divides experts
 *   weights  device float [tokens][top_k]
 *   ids      device int32 [tokens][top_k]
 */
FP8Q_API fp8q_status fp8q_moe_route(const void* logits, int32_t dt, int64_t tokens, int32_t experts, int32_t top_k,
                                    int32_t score, const float* bias, int32_t num_groups, int32_t top_groups,
                                    int32_t renormalize, float weight_scale, float* weights, int32_t* ids,
                                    void* stream);

/*
 * The gradient of fp8q_moe_route's weights with respect to the logits; the
 * choice (ids) and the bias are constants.  Slots with id -1 add nothing.  A
 * token whose weights a NaN (under softmax also a +inf) logit made NaN gets NaN
 * for every logit.
 *   ids        device int32 [tokens][top_k], as routing wrote them
 *   d_weights  device float [tokens][top_k]
 *   d_logits   device, type dt, [tokens][experts]: written in full
 */
FP8Q_API fp8q_status fp8q_moe_route_backward(const void* logits, int32_t dt, int64_t tokens, int32_t experts,
                                             int32_t top_k, int32_t score, int32_t renormalize, float weight_scale,
                                             const int32_t* ids, const float* d_weights, void* d_logits,
                                             void* stream);

/* Rows that always hold `slots` rows when each expert's are padded to a
 * multiple of align: (slots + min(slots, experts) * (align - 1)) rounded down
 * to one (-1 for invalid arguments). */
FP8Q_API int64_t fp8q_moe_rows(int64_t slots, int32_t experts, int32_t align);

/* Bytes of workspace fp8q_moe_plan needs (contents do not matter); 0 for up
 * to 1024 slots, whose workspace may be NULL. */
FP8Q_API size_t fp8q_moe_plan_workspace_bytes(int64_t slots, int32_t experts);

/*
 * The experts' row order.  Slot t * top_k + j is token t's j-th expert; slots
 * are sorted by expert, those of one expert in slot order, and each expert's
 * segment is padded to a multiple of align rows (1 for none; 128 for
 * transposed copies and weight gradients).
 *   ids        device int32 [slots]; one that is no expert's (-1) drops its slot
 *   experts    1..1024
 *   rows       rows of the padded order, >= fp8q_moe_rows()
 *   offsets    device int64 [experts + 1]: the segments' first rows (the
 *              group offsets of every grouped entry point)
 *   row_of     device int32 [slots]: a slot's row, -1 if dropped
 *   src        device int32 [rows]: a row's slot, -1 for padding and for the
 *              rows from offsets[experts] on
 *   workspace  device, >= fp8q_moe_plan_workspace_bytes(), 4-byte aligned
 */
FP8Q_API fp8q_status fp8q_moe_plan(const int32_t* ids, int64_t slots, int32_t experts, int32_t align, int64_t rows,
                                   int64_t* offsets, int32_t* row_of, int32_t* src, void* workspace,
                                   size_t workspace_bytes, void* stream);

/*
 * The tokens' rows in the plan's order, quantized as fp8q_quantize_blockwise
 * quantizes the gathered matrix with 1x128 groups, in one pass: row r is
 * token src[r] / top_k, zeros where src[r] is -1.
 *   x    device BF16 [tokens][cols], 16-byte aligned; cols % 16 == 0
 *   src  device int32 [rows]
 *   q, scale_inv, q_t, scale_inv_t, dir: as there, with `rows` rows (rows %
 *   16 == 0 for the transposed copy; align 128 keeps its 128x1 groups inside
 *   one expert)
 */
FP8Q_API fp8q_status fp8q_moe_dispatch(const void* x, int32_t dt, int64_t tokens, int64_t cols, int32_t top_k,
                                       const int32_t* src, int64_t rows, int32_t fmt, int32_t pow2_scales,
                                       int32_t dir, uint8_t* q, float* scale_inv, uint8_t* q_t, float* scale_inv_t,
                                       void* stream);

/*
 * The experts' rows back to the tokens:
 *   out[t] = sum_j weights[t][j] * y[row_of[t][j]]
 * summed in FP32 in the order of j and rounded once; dropped slots add
 * nothing.  weights NULL counts every slot once: the gradient of the
 * dispatch.
 *   y        device, type dt (BF16 or FP32), [rows][cols]
 *   row_of   device int32 [tokens][top_k], top_k <= 32
 *   weights  device float [tokens][top_k] or NULL
 *   out      device, type dt, [tokens][cols]
 */
FP8Q_API fp8q_status fp8q_moe_combine(const void* y, int32_t dt, int64_t rows, int64_t cols, const int32_t* row_of,
                                      const float* weights, int64_t tokens, int32_t top_k, void* out, void* stream);

/*
 * The gradients of fp8q_moe_combine:
 *   d_y[row_of[t][j]] = weights[t][j] * d_out[t],  0 for padding rows;
 *   d_weights[t][j] = sum over columns of d_out[t] * y[row_of[t][j]],  0 for
 *   dropped slots.
 * Types and sizes as there; weights, src and d_weights are required.
 */
FP8Q_API fp8q_status fp8q_moe_combine_backward(const void* d_out, const void* y, int32_t dt, int64_t rows,
                                               int64_t cols, const int32_t* row_of, const int32_t* src,
                                               const float* weights, int64_t tokens, int32_t top_k, void* d_y,
                                               float* d_weights, void* stream);

/* Bytes of workspace fp8q_moe_decode needs (contents do not matter). */
FP8Q_API size_t fp8q_moe_decode_workspace_bytes(int64_t tokens, int32_t top_k, int64_t inner);

/*
 * The whole expert layer for a few tokens (1 to 64), as one serving step has
 * them:
 *   out[t] = sum_j weights[t][j] * W2[e] a,  e = ids[t][j],
 *   a = gate * up / (1 + exp(-gate)),  gate = W1[e][:inner] x[t],  up = W1[e][inner:] x[t]
 * with W1, W2 the values of blockwise codes (128x128 blocks).  Unlike the
 * path over fp8q_moe_dispatch and the grouped products, tokens and inner
 * values are not quantized: products and sums are FP32's.  Inner values are off
 * by 2^-22 of themselves for FP32 output and by 2^-11 for BF16, or by 2^-38 of
 * the largest of their 32; a token's values are exact down to 2^-32 of the
 * largest of their 128.  Where such a largest value times its scale_inv is
 * below some 2^-111 all of them lose digits.  A slot whose id is no expert's
 * (-1) adds nothing; an expert that a token names twice counts with the sum of
 * the weights.  Sums have a fixed order.  Each chosen expert's weights are read
 * once for up to 8 of its tokens.
 *   x             device BF16 [tokens][hidden], 16-byte aligned
 *   ids, weights  device int32, float [tokens][top_k], as fp8q_moe_route
 *                 writes them; top_k <= 32
 *   w1            device uint8 [experts][2 * inner][hidden], 16-byte aligned;
 *                 w1_scale_inv [experts][ceil(2 * inner / 128)][ceil(hidden / 128)]
 *   w2            device uint8 [experts][hidden][inner], 16-byte aligned;
 *                 w2_scale_inv [experts][ceil(hidden / 128)][ceil(inner / 128)]
 *   out           device BF16 or FP32 (out_dt) [tokens][hidden]
 *   workspace     device, 16-byte aligned; calls that may overlap on the GPU
 *                 need separate ones
 * hidden and inner are multiples of 16, experts <= 1024.
 */
FP8Q_API fp8q_status fp8q_moe_decode(const void* x, int64_t tokens, int64_t hidden, int64_t inner, int32_t experts,
                                     int32_t top_k, const int32_t* ids, const float* weights, const uint8_t* w1,
                                     const float* w1_scale_inv, const uint8_t* w2, const float* w2_scale_inv,
                                     int32_t w_fmt, int32_t out_dt, void* out, void* workspace, size_t workspace_bytes,
                                     void* stream);

/*
 * Root-mean-square norm of the rows, with the residual's addition before it
 * and the 8-bit copies that the next product reads (the pages quantize a
 * product's input; this makes that input):
 *   h = x + residual, rounded to the residual's type; x itself without one
 *   rstd[r] = 1 / sqrt(sum_c h[r][c]^2 / cols + eps)
 *   y[r][c] = h[r][c] * rstd[r] * weight[c]
 * The copies are those of fp8q_quantize_blockwise with 1x128 groups for the
 * FP32 values of y.  Arithmetic is FP32: a row whose sum of squares passes
 * FP32's largest number (equal values from some 1.8e19 / sqrt(cols) on) gives
 * rstd 0 and so y 0; squares below 2^-126 (of values below some 1e-19) lose
 * digits, which shows where eps is no larger; a row without any nonzero value
 * gives y 0 (NaN with eps 0).
 *   x          device, type dt (BF16 or FP32), [rows][cols], 1 <= cols <= 32768
 *   residual   device, type residual_dt, [rows][cols], or NULL
 *   weight     device, type weight_dt, [cols]
 *   dir        0 (no copy), MXFP8_ROW, MXFP8_COL or MXFP8_BOTH
 *   h          device, type residual_dt, [rows][cols]: required with a
 *              residual, which it may overwrite; not written without
 *   rstd       device float [rows]
 *   y          device, type dt, [rows][cols], or NULL
 *   q, scale_inv, q_t, scale_inv_t: as fp8q_quantize_blockwise; cols % 16 ==
 *   0 for a copy, rows % 16 == 0 for the transposed one, and every tensor
 *   but rstd and the scales 16-byte aligned.  Without a copy any sizes and
 *   alignments do.  Other outputs overlap no input.
 */
FP8Q_API fp8q_status fp8q_rmsnorm(const void* x, int32_t dt, const void* residual, int32_t residual_dt,
                                  const void* weight, int32_t weight_dt, int64_t rows, int64_t cols, float eps,
                                  int32_t fmt, int32_t dir, int32_t pow2_scales, void* h, float* rstd, void* y,
                                  uint8_t* q, float* scale_inv, uint8_t* q_t, float* scale_inv_t, void* stream);

/* Bytes of workspace fp8q_rmsnorm_backward needs (contents do not matter). */
FP8Q_API size_t fp8q_rmsnorm_backward_workspace_bytes(int64_t rows, int64_t cols);

/*
 * The gradients of fp8q_rmsnorm, with g = d_y * weight and u = h * rstd:
 *   d_x[r][c] = rstd[r] * (g - u * mean_c(g * u)) + d_h[r][c]
 *   d_weight[c] = sum_r d_y[r][c] * u[r][c]
 * d_x is the gradient of x and of the residual alike.  Sums are FP32 in a
 * fixed order; no rows give d_weight 0.
 *   d_y        device, type dt, [rows][cols]
 *   h          device, type h_dt, [rows][cols]: the call's h (x without a
 *              residual), with its rstd
 *   d_h        device, type h_dt, [rows][cols], or NULL: the gradient that
 *              reaches h past the norm
 *   d_x        device, type h_dt, [rows][cols]; may overwrite d_h
 *   d_weight   device float [cols]
 *   workspace  device, 16-byte aligned; calls that may overlap on the GPU
 *              need separate ones
 */
FP8Q_API fp8q_status fp8q_rmsnorm_backward(const void* d_y, int32_t dt, const void* h, int32_t h_dt,
                                           const void* weight, int32_t weight_dt, const float* rstd, const void* d_h,
                                           int64_t rows, int64_t cols, void* d_x, float* d_weight, void* workspace,
                                           size_t workspace_bytes, void* stream);

/*
 * The gated activation between the two products of a block, and its copies:
 *   a[r][j] = gate * up / (1 + exp(-gate)),  gate = h[r][j], up = h[r][inner + j]
 * The copies are those of fp8q_quantize_blockwise with 1x128 groups for the
 * FP32 values of a.  1 / (1 + exp(-gate)) counts as 0 below 2^-126 (gates
 * below some -87.3); a gate of -Inf gives NaN, as -Inf * 0 does.
 *   h    device, type dt (BF16 or FP32), [rows][2 * inner]
 *   dir  0 (no copy), MXFP8_ROW, MXFP8_COL or MXFP8_BOTH
 *   a    device, type dt, [rows][inner], or NULL
 *   q, scale_inv, q_t, scale_inv_t: as there; inner % 16 == 0 for a copy,
 *   rows % 16 == 0 for the transposed one, h and a 16-byte aligned.  Without
 *   a copy any sizes and alignments do.  Outputs overlap no input.
 */
FP8Q_API fp8q_status fp8q_swiglu(const void* h, int32_t dt, int64_t rows, int64_t inner, int32_t fmt, int32_t dir,
                                 int32_t pow2_scales, void* a, uint8_t* q, float* scale_inv, uint8_t* q_t,
                                 float* scale_inv_t, void* stream);

/*
 * The gradient of fp8q_swiglu with respect to h, with s = 1 / (1 + exp(-gate)):
 *   d_h[r][j] = d_a * up * s * (1 + gate * (1 - s)),  d_h[r][inner + j] = d_a * gate * s
 * and its copies (of the [rows][2 * inner] matrix; inner % 8 == 0).  The slope
 * of the activation reaches 1.1: the gate's half may be Inf where up or d_a is
 * beyond 3e38 and the other one below 1.
 *   d_a  device, type dt, [rows][inner]
 *   d_h  device, type dt, [rows][2 * inner], or NULL
 */
FP8Q_API fp8q_status fp8q_swiglu_backward(const void* h, const void* d_a, int32_t dt, int64_t rows, int64_t inner,
                                          int32_t fmt, int32_t dir, int32_t pow2_scales, void* d_h, uint8_t* q,
                                          float* scale_inv, uint8_t* q_t, float* scale_inv_t, void* stream);

/* Bytes of workspace fp8q_clip_grads needs for `count` tensors (contents do not matter). */
FP8Q_API size_t fp8q_clip_grads_workspace_bytes(int32_t count);

/*
 * The norm of all gradients together, and the gradients scaled to a largest
 * norm (what follows the weight gradients of a step):
 *   norm = sqrt(sum over tensors and values of g^2)
 *   scale = min(1, max_norm / (norm + 1e-6)),  out[i] = grads[i] * scale
 * Squares are added in FP32 over up to 64 values and in FP64 beyond, in a
 * fixed order: values from some 1e18 on overflow, those below some 1e-20
 * count as 0.  A norm of NaN or Inf is reported as it is; Inf gives scale 0
 * (NaN where max_norm is Inf too), NaN gives NaN.
 *   grads, out  host arrays of `count` device pointers; a tensor may be
 *               overwritten by its own output (out[i] == grads[i]; with
 *               scale 1 it is then left alone); an output that overlaps
 *               another tensor is refused; the same gradient twice counts twice
 *   sizes       host int64 [count]: values of each tensor (0 for none)
 *   dts         host int32 [count]: FP8Q_IN_BF16 or FP8Q_IN_FP32, of the
 *               gradient and its output
 *   out         NULL: the norm alone (and the scale, if asked for)
 *   norm        device float[1]
 *   scale       device float[1], or NULL without out
 *   workspace   device, 8-byte aligned; calls that may overlap on the GPU
 *               need separate ones
 * The arrays are read before the call returns.
 */
FP8Q_API fp8q_status fp8q_clip_grads(const void* const* grads, const int64_t* sizes, const int32_t* dts, int32_t count,
                                     float max_norm, void* const* out, float* norm, float* scale, void* workspace,
                                     size_t workspace_bytes, void* stream);

/*
 * NVFP4 ("混合精度与 FP8 训练" 13.2): E2M1 elements (0, 0.5, 1, 1.5, 2, 3,
 * 4, 6 and negatives), one E4M3 scale per 16 elements along a row, and one
 * FP32 scale for the tensor.  Each step is one IEEE single operation:
 *   S = 448 * 6 / amax(tensor)   (amax 0 or non-finite -> 1; overflow -> FLT_MAX)
 *   block code = RNE_sat_E4M3(amax_b * fl32(S / 6)), d = its value
 *   element = RNE_sat_E2M1(x * fl32(S / d)), all +0 when d is 0 or NaN
 * The value a code stands for is e2m1(q) * d / S.
 *   x          device BF16 or FP32 [rows][cols], cols % 16 == 0
 *   q          device uint8 [rows][cols / 2], two codes per byte, the even
 *              element in the low nibble (8-byte aligned)
 *   s          device uint8 [rows][cols / 16], E4M3 codes
 *   amax_out   device float[1], required: receives the tensor amax (it is
 *              the reduction's accumulator, zeroed by the call)
 *   scale_out  device float[1] or NULL: receives S
 * Two passes over x: the amax, then the quantization.
 */
FP8Q_API fp8q_status fp8q_quantize_nvfp4(const void* x, int32_t dt, int64_t rows, int64_t cols, uint8_t* q,
                                         uint8_t* s, float* amax_out, float* scale_out, void* stream);

/*
 * Block scales rearranged for block-scaled tensor-core MMA.  The pages give
 * no layout ("Blackwell GPU MXFP8 预训练最佳实践" 3.2 says only that the
 * tensor cores take the MX types natively); this is NVIDIA's public one.
 * The rows x scale_cols scale array is padded to multiples of 128 rows and
 * 4 columns and cut into 128 x 4 blocks of 512 bytes, stored block row by
 * block row; inside a block, scale (r, c) is byte (r % 32) * 16 + (r / 32)
 * * 4 + c.  Padding bytes are 0.
 *   s     device uint8 [rows][s_ld], the first scale_cols bytes of each row
 *         used (e.g. s_row [rows][cols / 32], s_col [cols][s_col_ld] with
 *         scale_cols = its block count, NVFP4 s [rows][cols / 16])
 *   out   device uint8 [ceil(rows / 128) * 128 * ceil(scale_cols / 4) * 4],
 *         4-byte aligned, fully written
 */
FP8Q_API fp8q_status mx_scales_to_mma_layout(const uint8_t* s, int64_t rows, int64_t scale_cols, int64_t s_ld,
                                             uint8_t* out, void* stream);

/*
 * Dequantization.  ("HiFloat8：高性能训练之路" 1.1-1.2: a quantized tensor is
 * de-scaled by scale_inv = 1 / Scale; "Blackwell GPU MXFP8 预训练最佳实践"
 * 4.1 and 4.3: an MX element stands for value * 2^X, X = byte - 127, and
 * without MX hardware the blocks are dequantized to BF16 for a BF16
 * matmul.)  Codes are decoded exactly.  BF16 output rounds to nearest, ties
 * to even; every NaN result is the canonical quiet NaN (BF16 0x7FC0, FP32
 * 0x7FC00000).  q and y must be 16-byte aligned; out_dt is FP8Q_OUT_BF16
 * (2 bytes per element) or FP8Q_OUT_FP32 (4 bytes).
 */

/*
 * y[i] = fl_out(fl32(value(q[i]) * scale_inv[g])) for the rows of group g.
 *   q          device uint8[rows*cols], the codes of fp8q_cast_per_tensor
 *   scale_inv  device float[num_groups]
 *   y          device BF16 or FP32 [rows*cols]
 */
FP8Q_API fp8q_status fp8q_dequantize_per_tensor(const uint8_t* q, int64_t rows, int64_t cols,
                                                const int64_t* group_offsets, int32_t num_groups,
                                                int32_t fmt, const float* scale_inv, int32_t out_dt,
                                                void* y, void* stream);

/*
 * One MX copy back to high precision: y = fl_out(value(q) * 2^(s - 127)),
 * scale byte 0xFF -> NaN.  rows x cols is the original tensor (cols % 32 ==
 * 0).
 *   dir MXFP8_ROW: q = q_row [rows][cols], s = s_row [rows][cols/32]
 *                  (s_ld ignored), y [rows][cols].
 *   dir MXFP8_COL: q = q_col [cols][rows], s = s_col [cols][s_ld] with the
 *                  column blocks of all groups in order, as mxfp8_quantize
 *                  wrote them; y [cols][rows], the copy's own (transposed)
 *                  layout.  Blocks past s_ld dequantize to NaN.
 */
FP8Q_API fp8q_status mxfp8_dequantize(const uint8_t* q, const uint8_t* s, int64_t rows, int64_t cols,
                                      const int64_t* group_offsets, int32_t num_groups, int32_t fmt,
                                      int32_t dir, int64_t s_ld, int32_t out_dt, void* y, void* stream);

/*
 * Quantization-error statistics of a quantized copy against the tensor it
 * was made from ("昇腾 Ascend 950 低精度格式", appendix 3.4: formats are
 * compared by the per-layer SQNR and zero-rate of weights, activations and
 * KV cache).  xh is the FP32 value a code stands for: per-tensor
 * fl32(value(q) * scale_inv[g]); MX value(q) * 2^X rounded to FP32 (exact
 * unless it reaches 2^128, which gives Inf; scale byte 0xFF gives NaN).
 * Over the elements where x and xh are both finite:
 *   SQNR = 10 log10(signal / noise) dB,  zero-rate = n_flushed / n,
 * both computed on the device from the sums and counts (SQNR +inf for an
 * exact copy of a nonzero signal, NaN when signal and noise are both 0;
 * zero-rate 0 for an empty tensor).  Sums are exact to about 2e-6 relative
 * (FP32 sums of 32 elements added in FP64) and repeat exactly from run to
 * run on one GPU.
 */
typedef struct fp8q_qstats {
    double signal;                   /* sum of x^2 over the finite pairs */
    double noise;                    /* sum of (x - xh)^2 over the finite pairs */
    unsigned long long n;            /* elements compared */
    unsigned long long n_zero;       /* elements with xh == 0 */
    unsigned long long n_flushed;    /* xh == 0 while x != 0 (a NaN x is not 0) */
    unsigned long long n_nonfinite;  /* x or xh Inf or NaN: left out of the sums */
    double sqnr_db;                  /* 10 log10(signal / noise) */
    double zero_rate;                /* n_flushed / n */
} fp8q_qstats;

/* Bytes of workspace the statistics calls need (a constant, under 100 KB). */
FP8Q_API size_t fp8q_qstats_workspace_bytes(void);

/*
 * Statistics of a per-tensor (per-group) copy, one pass over x and q.
 *   x          device BF16 or FP32 [rows][cols] (16-byte aligned)
 *   q          device uint8 [rows][cols], 16-byte aligned (the codes of
 *              fp8q_cast_per_tensor)
 *   scale_inv  device float[num_groups]
 *   out        device fp8q_qstats, 8-byte aligned: written by the call
 *   workspace  device, >= fp8q_qstats_workspace_bytes() bytes, 16-byte
 *              aligned, zero-filled before its first use; every call leaves
 *              it ready for the next.  Calls that may overlap on the GPU
 *              need separate workspaces.
 * Rows outside every group are not compared.
 */
FP8Q_API fp8q_status fp8q_qstats_per_tensor(const void* x, int32_t dt, int64_t rows, int64_t cols,
                                            const int64_t* group_offsets, int32_t num_groups, int32_t fmt,
                                            const uint8_t* q, const float* scale_inv, fp8q_qstats* out,
                                            void* workspace, size_t workspace_bytes, void* stream);

/*
 * Statistics of one MX copy of x (cols % 32 == 0), one pass over x and the
 * copy.  Layouts as mxfp8_quantize wrote them:
 *   dir MXFP8_ROW: q = q_row [rows][cols] (16-byte aligned), s = s_row
 *                  [rows][cols/32]; group_offsets and s_ld are not used.
 *   dir MXFP8_COL: q = q_col [cols][rows], s = s_col [cols][s_ld] with the
 *                  column blocks of all groups in order; element (c, r) of
 *                  the copy is compared with x[r][c].  Blocks past s_ld
 *                  count as NaN scales.
 * Other arguments as fp8q_qstats_per_tensor.
 */
FP8Q_API fp8q_status mxfp8_qstats(const void* x, int32_t dt, int64_t rows, int64_t cols,
                                  const int64_t* group_offsets, int32_t num_groups, int32_t fmt, int32_t dir,
                                  const uint8_t* q, const uint8_t* s, int64_t s_ld, fp8q_qstats* out,
                                  void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8Q_H */
