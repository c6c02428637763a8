/*
 * nvfp4.h -- C ABI of libnvfp4.so: NVFP4 quantisers and block-scaled GEMMs
 * for one GB300 (sm_103a), the hot path of an NVFP4 linear / MLP layer.
 *
 * The method is the NVFP4 pretraining recipe of the "NVFP4 pretraining
 * recipe" page (re-post of NVIDIA's blog on NVFP4 in TransformerEngine and
 * MaxText).  Each entry point below cites the passage of that page that
 * defines what it computes.
 *
 * Conventions shared by every entry point
 *  - Pointers named "device" are CUDA device pointers on the current device;
 *    host pointers are marked "host".  The caller owns every buffer, including
 *    workspaces and the per-tensor scalars; the library never allocates,
 *    frees or synchronises on the hot path (nvfp4_check_device_errors is the
 *    one call that synchronises).
 *  - All work is enqueued asynchronously on `stream` (a cudaStream_t; NULL is
 *    the legacy default stream).  Nothing on the hot path allocates or
 *    synchronises, so a sequence of calls can be captured into a CUDA graph
 *    and replayed (after one uncaptured call of each, which configures the
 *    kernels).  The quantiser, amax and GEMM kernels are launched with
 *    programmatic stream serialization: a kernel may be scheduled while the
 *    previous one on the stream finishes, and waits for it to complete before
 *    it touches global memory, so stream order is kept.
 *  - Argument errors are reported by the return value before anything is
 *    launched; a failed launch returns NVFP4_ERR_CUDA.  Device-side wait
 *    timeouts (a hung pipeline) are recorded in a device error word and
 *    reported by nvfp4_check_device_errors.
 *  - Matrices are row-major.  A "K-major" NVFP4 operand [rows, K] stores the
 *    E2M1 codes of row r in bytes r*K/2 .. r*K/2 + K/2 - 1, element 2i in the
 *    low nibble and element 2i+1 in the high nibble.
 *  - Scale tensors (E4M3, one byte per 16 elements) are stored in the layout
 *    the block-scaled MMA reads: 512-byte atoms of 128 rows x 4 scale
 *    columns, the byte of (row r, scale column c) at
 *        atom(r/128, c/4) * 512 + (r%32)*16 + ((r/32)%4)*4 + c%4,
 *    atoms row-block major, rows padded to 128 and scale columns to 4 with
 *    zero bytes.  Size: pad128(rows) * pad4(cols/16) bytes.
 */
#ifndef NVFP4_H
#define NVFP4_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef void* nvfp4_stream; /* a cudaStream_t */

typedef enum {
  NVFP4_OK = 0,
  NVFP4_ERR_INVALID_ARG = 1,    /* null pointer, bad enum or flag combination   */
  NVFP4_ERR_SHAPE = 2,          /* a dimension breaks the rules stated per call */
  NVFP4_ERR_ALIGN = 3,          /* a pointer or leading dimension is misaligned */
  NVFP4_ERR_ARCH = 4,           /* the current device is not sm_103             */
  NVFP4_ERR_WORKSPACE = 5,      /* workspace missing or smaller than required   */
  NVFP4_ERR_CUDA = 6,           /* a CUDA runtime/driver call failed            */
  NVFP4_ERR_DEVICE_TIMEOUT = 7  /* a kernel's bounded wait expired              */
} nvfp4_status;

typedef enum { NVFP4_IN_BF16 = 0, NVFP4_IN_FP32 = 1 } nvfp4_in_dtype;

/* Quantisation geometry ("NVFP4 pretraining recipe", bullets 1 and 4).
 *  ROW_1X16   : 1x16 blocks along the contiguous dim; output [rows, cols].
 *  COL_1X16   : 1x16 blocks along the rows; output is the transpose
 *               [cols, rows] (K-major along the original rows), the form the
 *               WGRAD GEMM consumes.
 *  BLOCK_16X16: one scale per 16x16 tile (weights); output [rows, cols], and
 *               with NVFP4_EMIT_T also the transpose [cols, rows] built from
 *               the same codes (no requantisation). */
typedef enum { NVFP4_ROW_1X16 = 0, NVFP4_COL_1X16 = 1, NVFP4_BLOCK_16X16 = 2 } nvfp4_mode;

enum {
  NVFP4_RHT = 1u,        /* 16-point random Hadamard transform along the blocks (bullet 3) */
  NVFP4_SR = 2u,         /* stochastic rounding of the elements (bullet 5); else RNE       */
  NVFP4_EMIT_T = 4u,     /* BLOCK_16X16 only: also write the transposed operand            */
  NVFP4_AMAX_GIVEN = 8u, /* use *out->amax (device, set by the caller) as the tensor amax   */
  /* with NVFP4_SR: `offset` is the device address (8-byte aligned) of a uint64
   * that holds the offset, read when the kernel runs.  A captured CUDA graph
   * keeps the arguments of its calls, so with a plain offset every replay
   * rounds with the same random numbers; with this one a replay takes what the
   * caller has advanced the counter to. */
  NVFP4_OFFSET_DEVICE = 32u
};

/* A quantised NVFP4 operand.  The caller fills the pointers; nvfp4_quantize
 * fills rows/cols/mode/flags.  rows x cols is the logical K-major operand
 * (cols = contraction length).
 *   codes    device uint8 [rows][cols/2]
 *   scales   device uint8, MMA layout for [rows, cols]
 *   codes_t  device uint8 [cols][rows/2]     (BLOCK_16X16 + EMIT_T, else NULL)
 *   scales_t device uint8, MMA layout for [cols, rows] (likewise)
 *   amax     device float: tensor amax (output; input with AMAX_GIVEN)
 *   s_dec    device float: per-tensor decode scale 1/s_enc (output)        */
typedef struct nvfp4_tensor {
  void* codes;
  void* scales;
  void* codes_t;
  void* scales_t;
  float* amax;
  float* s_dec;
  int64_t rows;
  int64_t cols;
  int32_t mode;
  uint32_t flags;
} nvfp4_tensor;

/* ---------------------------------------------------------------------- */
/* Status and device                                                       */
/* ---------------------------------------------------------------------- */
const char* nvfp4_status_string(nvfp4_status s);
/* Library version as major*10000 + minor*100 + patch. */
int nvfp4_version(void);
/* NVFP4_OK when `device` is an sm_103 GPU this library's kernels run on. */
nvfp4_status nvfp4_device_check(int device);
/* Synchronises `stream`, then reads and clears the device error word that
 * kernels set when a bounded wait expires.  Returns NVFP4_ERR_DEVICE_TIMEOUT
 * if it was set, NVFP4_ERR_CUDA if the stream reported an error. */
nvfp4_status nvfp4_check_device_errors(nvfp4_stream stream);

/* Failure injection for tests of the bounded waits; the pages have no
 * counterpart (they describe no failure handling).  While a STALL bit of
 * stall_mask is set, the producer of every launch of that kernel family
 * issues no loads, so the consumers' first pipeline wait runs out; nothing is
 * in flight when the kernel gives up, and it returns after recording the
 * timeout (nvfp4_check_device_errors then reports NVFP4_ERR_DEVICE_TIMEOUT):
 *   NVFP4_STALL_QUANTIZE  the quantise passes of nvfp4_quantize, and the row
 *                         loads of nvfp4_residual_norm_fwd / _bwd
 *   NVFP4_STALL_GEMM      every GEMM kernel (single-SM and CTA-pair tiles;
 *                         on a pair a timeout in either CTA stops both)
 * With a LOSE bit the loads are issued and each block's first wait is for 16
 * bytes more than will come, so the kernel gives up with loads behind it; with
 * a QUIT bit it gives up before its first wait, its loads in flight:
 *   NVFP4_LOSE_NORM       nvfp4_residual_norm_fwd / _bwd (rows to 8192 columns,
 *                         forward 16384: the others load no rows ahead)
 *   NVFP4_QUIT_GEMM       every GEMM kernel
 * wait_limit_ns sets how long those kernels' pipeline waits last before they
 * give up (0: the default, 2 s); the waits that drain copies and MMAs
 * already issued keep their own 2 s limit.  Synchronises the device, then
 * applies to later launches until changed; call it with nothing of this
 * library in flight.  Returns NVFP4_ERR_INVALID_ARG for unknown bits,
 * NVFP4_ERR_CUDA if the device cannot be reached. */
enum { NVFP4_STALL_QUANTIZE = 1u, NVFP4_STALL_GEMM = 2u, NVFP4_LOSE_NORM = 16u,
       NVFP4_QUIT_GEMM = 32u };
nvfp4_status nvfp4_debug_inject(uint32_t stall_mask, uint64_t wait_limit_ns);

/* ---------------------------------------------------------------------- */
/* Quantiser                                                               */
/* ---------------------------------------------------------------------- */
/* Byte sizes for quantising an input x [rows, cols]: the codes (and, with
 * EMIT_T, the same again for codes_t), the MMA-layout scales (scales_t has
 * the size of the transposed operand's scales), and the workspace
 * nvfp4_quantize needs.  Any output pointer may be NULL. */
nvfp4_status nvfp4_quantize_sizes(int64_t rows, int64_t cols, int32_t mode, uint32_t flags,
                                  size_t* codes_bytes, size_t* scales_bytes,
                                  size_t* scales_t_bytes, size_t* workspace_bytes);

/* NVFP4 quantisation of x [rows, cols] (row-major, leading dim ld elements),
 * per "NVFP4 pretraining recipe", bullets 1-5:
 *   amax_T = max |v| over the (RHT-transformed, if NVFP4_RHT) operand v;
 *   s_enc = 6*448 / amax_T (1 if amax_T == 0, FLT_MAX if not finite),
 *   s_dec = 1 / s_enc;
 *   per block b (16 elements, or a 16x16 tile): a_b = max |v|,
 *   S_b = E4M3_rn_satfinite((a_b / 6) * s_enc);
 *   per element: y = v * (S_b == 0 ? 0 : s_enc / S_b), encoded to E2M1 by
 *   round-to-nearest-even with saturation to +-6, or with NVFP4_SR by
 *   stochastic rounding: round |y| up to the next grid value iff
 *   r < floor(frac * 2^32), frac = (|y| - lo) / (hi - lo), where r is word
 *   idx%4 of Philox4x32-10(key = seed, counter = (idx/4 lo, idx/4 hi, 0,
 *   offset lo)) and idx = row*cols + col in the output layout.
 *   NVFP4_RHT (1x16 modes): each block becomes (1/4) H16 diag(s) v, signs s_i
 *   = -1 where bit i of word 0 of Philox(key = seed, counter = (0,0,1,0)) is
 *   set -- one sign vector per seed, so both WGRAD operands quantised with the
 *   same seed share it (bullet 3: RHT on the WGRAD inputs only).
 * Shapes: ROW_1X16 needs cols % 16 == 0; COL_1X16 rows % 16 == 0 and
 * cols % 8 == 0; BLOCK_16X16 rows % 16 == 0, cols % 16 == 0, no NVFP4_RHT.
 * x must be 16-byte aligned and ld * element size a multiple of 16 bytes.
 * The workspace (device, >= the size nvfp4_quantize_sizes gives, 16-byte
 * aligned) holds per-CTA partial maxima; with NVFP4_AMAX_GIVEN it may be NULL.
 * Outputs: out->codes/scales (+ codes_t/scales_t), out->amax, out->s_dec;
 * padding bytes of the scale tensors are written as zero. */
nvfp4_status nvfp4_quantize(const void* x, int32_t in_dtype, int64_t rows, int64_t cols,
                            int64_t ld, int32_t mode, uint32_t flags, uint64_t seed,
                            uint64_t offset, nvfp4_tensor* out, void* workspace,
                            size_t workspace_bytes, nvfp4_stream stream);

/* The per-tensor amax of nvfp4_quantize ("NVFP4 pretraining recipe", bullet
 * 4: amax_T over the operand as quantised) for the two quantisations a
 * training step makes of X and of dY -- the row-wise operand (ROW_1X16, no
 * transform) and the column-wise WGRAD operand (COL_1X16 with NVFP4_RHT) --
 * from one read of x [rows, cols] (leading dim ld, bf16 or fp32):
 *   amax_plain = max |x|                            (if amax_plain != NULL),
 *   amax_rht   = max |(1/4) H16 diag(s) v| over every 16-row block v of every
 *                column, signs s from `seed` as in nvfp4_quantize
 *                                                   (if amax_rht != NULL).
 * Both are device floats; each equals, bit for bit, the amax the matching
 * nvfp4_quantize call computes itself, so passing it with NVFP4_AMAX_GIVEN
 * (out->amax pointing at it) gives identical codes and scales.  At least one
 * output must be non-NULL; amax_rht needs rows % 16 == 0.  x: 16-byte
 * aligned, ld * element size a multiple of 16 bytes, cols % 8 == 0.  The
 * workspace is as for nvfp4_quantize (partial maxima; contents on return
 * unspecified).  Two kernel launches on `stream`; nothing is allocated.
 * Returns NVFP4_ERR_INVALID_ARG, _SHAPE, _ALIGN, _WORKSPACE, _ARCH, _CUDA as
 * nvfp4_quantize does. */
nvfp4_status nvfp4_amax(const void* x, int32_t in_dtype, int64_t rows, int64_t cols, int64_t ld,
                        uint64_t seed, float* amax_plain, float* amax_rht, void* workspace,
                        size_t workspace_bytes, nvfp4_stream stream);

/* Both quantisations a training step makes of one bf16 activation or
 * gradient x [rows, cols] (leading dim ld), from one read of x -- bit for bit
 * what two nvfp4_quantize calls give ("NVFP4 pretraining recipe", bullets
 * 1-5: the FPROP / DGRAD operand is quantised row-wise, the WGRAD operand
 * column-wise with the RHT on the WGRAD inputs only, SR on gradients):
 *   row_out: nvfp4_quantize(x, ROW_1X16, row_flags, seed, row_offset)
 *   col_out: nvfp4_quantize(x, COL_1X16, col_flags, seed, col_offset)
 * row_flags: NVFP4_AMAX_GIVEN, optionally | NVFP4_SR; col_flags:
 * NVFP4_AMAX_GIVEN, optionally | NVFP4_RHT | NVFP4_SR (each SR also with
 * | NVFP4_OFFSET_DEVICE).  Both amaxes are given
 * (*row_out->amax = max |x|, *col_out->amax = the column operand's amax, e.g.
 * both from one nvfp4_amax call), so nothing needs a workspace.  Shapes:
 * rows % 16 == 0, cols % 16 == 0.  x, the codes and scales buffers 16-byte
 * aligned, ld * 2 a multiple of 16; bf16 input only.  One kernel launch on
 * `stream`; nothing is allocated.  Returns NVFP4_ERR_INVALID_ARG (a NULL
 * pointer, fp32 input, a flag outside those above or AMAX_GIVEN missing),
 * _SHAPE, _ALIGN, _ARCH, _CUDA. */
nvfp4_status nvfp4_quantize_rowcol(const void* x, int32_t in_dtype, int64_t rows, int64_t cols,
                                   int64_t ld, uint32_t row_flags, uint32_t col_flags,
                                   uint64_t seed, uint64_t row_offset, uint64_t col_offset,
                                   nvfp4_tensor* row_out, nvfp4_tensor* col_out,
                                   nvfp4_stream stream);

/* nvfp4_quantize without a workspace argument; the pages have no counterpart
 * to this entry point.  It is for callers that cannot provide device scratch
 * memory -- code running during CUDA graph capture (where cudaMalloc is not
 * allowed), plugins given only input and output pointers, or programs whose
 * allocator owns all device memory.  The per-CTA partial maxima of the amax
 * pass go to a fixed 4 KB array (1024 floats) inside the library, held on
 * every GPU that loads the library until the process exits.  The caller still
 * passes x and the output buffers of `out`, exactly as for nvfp4_quantize, and
 * gets the same results.
 * Every call made outside stream capture looks up the array's device address
 * on the current device (after a cudaDeviceReset the array may move); a call
 * made while `stream` is being captured reuses the address the last
 * uncaptured call on that device found, so make the first call on a device
 * before any stream capture.  The call itself allocates and frees nothing.
 * All calls share the one array: calls that can overlap on the GPU
 * (different streams, no ordering between them) race and must not be issued
 * that way.  Each call's amax pass rewrites every partial its quantise pass
 * reads, so nothing needs clearing between calls.  The array holds the
 * partial maxima of the largest amax grid the library launches (1024 CTAs),
 * so every device and shape nvfp4_quantize accepts is accepted; the statuses
 * are those of nvfp4_quantize. */
nvfp4_status nvfp4_quantize_noalloc(const void* x, int32_t in_dtype, int64_t rows, int64_t cols,
                                    int64_t ld, int32_t mode, uint32_t flags, uint64_t seed,
                                    uint64_t offset, nvfp4_tensor* out, nvfp4_stream stream);

/* ---------------------------------------------------------------------- */
/* MX comparison formats                                                   */
/* ---------------------------------------------------------------------- */
/* "NVFP4 pretraining recipe" page, "NVFP4 format and advantages": MXFP4
 * scales 32-element blocks by powers of two (E8M0), against NVFP4's 16-element
 * E4M3 blocks under a per-tensor scale; the same page quotes MXFP8 and MXFP4
 * block-scaled GEMMs on Blackwell.  These quantisers produce those formats
 * for comparison with NVFP4 (error studies), following the OCP Microscaling
 * specification the page links. */
typedef enum { NVFP4_MXFP4 = 0, NVFP4_MXFP8 = 1 } nvfp4_mx_format;
enum {
  NVFP4_MX_ROW = 0,  /* blocks of 32 along the columns; output [rows, cols]            */
  NVFP4_MX_COL = 1   /* blocks of 32 along the rows; output transposed [cols, rows]    */
};

/* Byte sizes of the outputs of nvfp4_mx_quantize for x [rows, cols]:
 * codes = out_rows * out_cols / 2 (MXFP4) or out_rows * out_cols (MXFP8),
 * scales = out_rows * out_cols / 32, scales_sw = the same scales in the MMA
 * layout (512-byte atoms of 128 rows x 4 scale columns, rows padded to 128
 * and scale columns to 4).  Any pointer may be NULL.  Returns
 * NVFP4_ERR_SHAPE unless the blocked dimension is a multiple of 32 (and, for
 * NVFP4_MX_COL, cols a multiple of 8). */
nvfp4_status nvfp4_mx_sizes(int64_t rows, int64_t cols, int32_t mode, int32_t fmt,
                            size_t* codes_bytes, size_t* scales_bytes, size_t* scales_sw_bytes);

/* MXFP4 / MXFP8 quantisation of x [rows, cols] (bf16 or fp32, row-major,
 * leading dim ld elements).  Per block of 32 consecutive output elements:
 *   shared = clamp(floor(log2(amax)) - emax, -127, 127), emax = 2 (E2M1) or
 *            8 (E4M3); scale byte = shared + 127 (E8M0, value 2^shared);
 *            0 when the block is all zero; 0xFF (NaN) when it holds a value
 *            that is not finite, with zero codes;
 *   element = v / 2^shared rounded to nearest-even and saturated to the
 *            element format's largest finite value (6 or 448), sign kept.
 * Outputs (device, caller-owned, sizes from nvfp4_mx_sizes): codes row-major
 * [out_rows][out_cols] -- MXFP4 packed two per byte, element 2i in the low
 * nibble of byte i; MXFP8 one E4M3 byte each -- and scales row-major
 * [out_rows][out_cols / 32], and, if scales_sw is not NULL, the same
 * scale bytes in the MMA layout nvfp4_mx_gemm reads (offset
 * ((r/128) * (padded scale cols / 4) + c/4) * 512 + (r%32)*16 + ((r/32)%4)*4
 * + c%4 for row r, scale column c; padding written as zero).  x and codes
 * must be 16-byte aligned and ld * element size a multiple of 16 bytes.  One
 * kernel launch on `stream` (plus a memset of scales_sw when it has
 * padding); nothing is allocated.  Returns NVFP4_ERR_INVALID_ARG, _SHAPE,
 * _ALIGN, _ARCH, _CUDA. */
nvfp4_status nvfp4_mx_quantize(const void* x, int32_t in_dtype, int64_t rows, int64_t cols,
                               int64_t ld, int32_t mode, int32_t fmt, void* codes, void* scales,
                               void* scales_sw, nvfp4_stream stream);

/* D bf16 [M, N] = A . B^T for MX operands, the comparison GEMMs (the page's
 * quote of MXFP8 and MXFP4 block-scaled GEMMs on Blackwell):
 *   D[m][n] = bf16_rn( sum_k deq(A)[m][k] * deq(B)[n][k] ),
 *   deq = element value * 2^(scale byte - 127) over its 32-element block.
 * A: a_codes [M][K] K-major as nvfp4_mx_quantize writes them (MXFP4: K/2
 * bytes per row, MXFP8: K), a_scales_sw its scales in the MMA layout (the
 * scales_sw output of nvfp4_mx_quantize); B likewise [N][K].  The WGRAD
 * operands are the NVFP4_MX_COL outputs.  Shapes: K % 128 == 0, N % 8 == 0.
 * All pointers device, 16-byte aligned.  One launch (the CTA-pair kernel,
 * tcgen05 kind::mxf4nvf4 scale_vec::2X or kind::mxf8f6f4 scale_vec::1X).
 * Returns NVFP4_ERR_INVALID_ARG, _SHAPE, _ALIGN, _ARCH, _CUDA. */
nvfp4_status nvfp4_mx_gemm(const void* a_codes, const void* a_scales_sw, const void* b_codes,
                           const void* b_scales_sw, int32_t fmt, void* D, int64_t M, int64_t N,
                           int64_t K, nvfp4_stream stream);

/* ---------------------------------------------------------------------- */
/* Block-scaled GEMM                                                       */
/* ---------------------------------------------------------------------- */
/* Output modes of nvfp4_gemm. */
enum {
  NVFP4_D_BF16 = 0,        /* D bf16 [M,N] = bf16(alpha * acc)                            */
  NVFP4_D_F32_ACCUM = 1,   /* D fp32 [M,N] += float(bf16(alpha * acc)) (master gradient)   */
  NVFP4_D_BF16_ADD_C = 2   /* D bf16 [M,N] = bf16(alpha * acc + float(C)), C bf16 [M,N]    */
};

/* D = alpha * A . B^T with A [M, K] and B [N, K] NVFP4 K-major operands and
 * alpha = (*A->s_dec) * (*B->s_dec) read on the device; FP32 accumulation in
 * tensor memory, BF16 output ("NVFP4 pretraining recipe", Figure 1 text:
 * FPROP, DGRAD and WGRAD consume NVFP4 inputs and emit BF16 outputs, later
 * folded into the FP32 master weight -- NVFP4_D_F32_ACCUM).
 * a_view / b_view: 0 reads codes/scales, 1 reads codes_t/scales_t (the
 * transpose written by BLOCK_16X16 + EMIT_T: DGRAD reads W this way, bullet 4).
 * The operand's logical shape must match (rows, cols) = (M, K) / (N, K).
 * Shapes: M, N >= 1, K % 64 == 0, N % 8 == 0.  D (and C) 16-byte aligned.
 * workspace: unused (may be NULL). */
nvfp4_status nvfp4_gemm(const nvfp4_tensor* A, int32_t a_view, const nvfp4_tensor* B,
                        int32_t b_view, void* D, int32_t d_mode, const void* C, int64_t M,
                        int64_t N, int64_t K, void* workspace, size_t workspace_bytes,
                        nvfp4_stream stream);

/* Output-tile configurations of nvfp4_gemm_ex. */
enum {
  NVFP4_TILE_AUTO = 0,          /* 128 x 128 when N <= 128; else the CTA pair when its     *
                                 * 256 x 256 tiles number at least half the SMs (256 x 384 *
                                 * where its rounds of tiles per pair cost less, not with  *
                                 * NVFP4_D_BF16_ADD_C); else 128 x 256 on one SM           */
  NVFP4_TILE_128X128 = 1,       /* one SM per 128 x 128 tile                               */
  NVFP4_TILE_128X256 = 2,       /* one SM per 128 x 256 tile                               */
  NVFP4_TILE_PAIR_256X256 = 3,  /* a cluster of two SMs per 256 x 256 tile (cta_group::2) */
  /* 4 is retired (rejected with NVFP4_ERR_INVALID_ARG)                                    */
  NVFP4_TILE_128X256_K128 = 5,  /* one SM per 128 x 256 tile, 8 stages of K = 128          */
  NVFP4_TILE_PAIR_256X384 = 6   /* a cluster of two SMs per 256 x 384 tile: an N = 256 and *
                                 * an N = 128 MMA per K step, 4 stages; not with           *
                                 * NVFP4_D_BF16_ADD_C (NVFP4_ERR_INVALID_ARG)              */
};

/* As nvfp4_gemm with an explicit output-tile configuration (NVFP4_TILE_*).
 * For tuning and tests; results are identical up to FP32 summation order. */
nvfp4_status nvfp4_gemm_ex(const nvfp4_tensor* A, int32_t a_view, const nvfp4_tensor* B,
                           int32_t b_view, void* D, int32_t d_mode, const void* C, int64_t M,
                           int64_t N, int64_t K, int32_t tile, nvfp4_stream stream);

/* ---------------------------------------------------------------------- */
/* SwiGLU MLP (gate, up, down projections) with NVFP4 GEMMs                */
/* ---------------------------------------------------------------------- */
/* "NVFP4 pretraining recipe", Figure 1 text: the MLP's GEMMs run in NVFP4.
 * Forward: G = X Wg^T, U = X Wu^T, H = silu(G) * U, Y = H Wd^T; backward:
 * dH = dY Wd, dWd += dY^T H, dG/dU from the SwiGLU derivative, dX = dG Wg +
 * dU Wu, dWg += dG^T X, dWu += dU^T X.  Quantisation per operand: X, H and W
 * with RNE (1x16 / 16x16), dY, dG, dU with SR; the WGRAD operands (X^T, H^T,
 * dY^T, dG^T, dU^T) COL_1X16 with the RHT when flags has NVFP4_RHT.
 * Dimensions: M tokens, D hidden, F ffn; Wg, Wu fp32 [F, D], Wd fp32 [D, F]
 * (device, the FP32 master weights, quantised 16x16 every forward).
 * flags: NVFP4_RHT, and NVFP4_AMAX_GIVEN for a forward whose weight amaxes
 * are already in the weight operands' amax slots in `saved`
 * (nvfp4_mlp_operand: Q_WG / Q_WU / Q_WD, .amax), e.g. written there by the
 * previous optimizer step (nvfp4_sgd_step): the three weights are then
 * quantised without their amax passes, with codes and scales identical to a
 * forward that takes the amaxes itself.  The backward ignores
 * NVFP4_AMAX_GIVEN. */
typedef struct nvfp4_mlp_params {
  int64_t M, D, F;
  const float* Wg;
  const float* Wu;
  const float* Wd;
  uint64_t seed;   /* RHT signs and SR key                           */
  uint64_t step;   /* SR counter offsets 8*step + 0..5 (per tensor); a  *
                    * captured graph keeps it                          */
  uint32_t flags;  /* NVFP4_RHT | NVFP4_AMAX_GIVEN, or 0             */
} nvfp4_mlp_params;

/* SwiGLU between the gate/up and down projections, with the tensor amaxes of
 * its outputs for the NVFP4 quantisations that follow ("NVFP4 pretraining
 * recipe" page, Figure 1 text and bullets 3-5: each output is quantised
 * row-wise for FPROP / DGRAD and column-wise, with the RHT when enabled, for
 * WGRAD; both need its per-tensor amax).  Computed in FP32 with the CUDA
 * expf, each output rounded once to bf16:
 *   forward   H  = silu(G) * U,               silu(g) = g sigmoid(g)
 *   backward  dU = dH * silu(G),  dG = dH * U * sigmoid(G) (1 + G (1 - sigmoid(G)))
 * All tensors bf16 [rows, cols], contiguous, 16-byte aligned; rows % 16 == 0,
 * cols % 8 == 0.  For each output T the kernel writes two device floats,
 * taken from the bf16 values it stores (no second read of T):
 *   amax_*_row = max |T|, the amax of T's ROW_1X16 quantisation;
 *   amax_*_col = with NVFP4_RHT in flags, max |(1/4) H16 diag(s) v| over every
 *                16-row block v of every column of T, signs s from `seed`
 *                as in nvfp4_quantize; otherwise max |T| again.
 * Each equals, bit for bit, what nvfp4_amax returns for T, so it can be given
 * to nvfp4_quantize with NVFP4_AMAX_GIVEN.  workspace: device scratch of at
 * least nvfp4_swiglu_workspace_bytes(), 16-byte aligned, contents on return
 * unspecified.  Two kernel launches on `stream`; nothing is allocated.
 * Returns NVFP4_ERR_INVALID_ARG (a NULL pointer, unknown flag bits),
 * _SHAPE, _ALIGN, _WORKSPACE, _ARCH, _CUDA. */
size_t nvfp4_swiglu_workspace_bytes(void);
nvfp4_status nvfp4_swiglu_fwd(const void* G, const void* U, void* H, int64_t rows, int64_t cols,
                              uint32_t flags, uint64_t seed, float* amax_h_row,
                              float* amax_h_col, void* workspace, size_t workspace_bytes,
                              nvfp4_stream stream);
nvfp4_status nvfp4_swiglu_bwd(const void* dH, const void* G, const void* U, void* dG, void* dU,
                              int64_t rows, int64_t cols, uint32_t flags, uint64_t seed,
                              float* amax_dg_row, float* amax_dg_col, float* amax_du_row,
                              float* amax_du_col, void* workspace, size_t workspace_bytes,
                              nvfp4_stream stream);

/* Device bytes of the saved-activation buffer (forward -> backward) and of
 * the workspace either call needs. */
nvfp4_status nvfp4_mlp_sizes(int64_t M, int64_t D, int64_t F, size_t* saved_bytes,
                             size_t* workspace_bytes);

/* X bf16 [M, D] -> Y bf16 [M, D]; fills `saved` (device) for the backward.
 * Shapes: M, D, F multiples of 128. */
nvfp4_status nvfp4_mlp_fwd(const nvfp4_mlp_params* p, const void* X, void* Y, void* saved,
                           size_t saved_bytes, void* workspace, size_t workspace_bytes,
                           nvfp4_stream stream);

/* dY bf16 [M, D] -> dX bf16 [M, D]; dWg, dWu fp32 [F, D] and dWd fp32 [D, F]
 * (device) are accumulated: += float(bf16(WGRAD)). */
nvfp4_status nvfp4_mlp_bwd(const nvfp4_mlp_params* p, const void* dY, const void* saved,
                           void* dX, float* dWg, float* dWu, float* dWd, void* workspace,
                           size_t workspace_bytes, nvfp4_stream stream);

/* Where nvfp4_mlp_fwd / nvfp4_mlp_bwd keep the intermediates of one MLP
 * step inside the caller's `saved` and workspace buffers, so a caller can
 * read them after a call (to inspect or check each stage of the step); the
 * same Figure 1 text passage as the MLP calls.  The bf16 tensors (row-major):
 *   G, U       [M, F]  in saved      (gate and up projections, forward)
 *   H          [M, F]  in workspace  (silu(G) * U, forward)
 *   DH, DG, DU [M, F]  in workspace  (backward: dY Wd, the SwiGLU derivative)
 *   DX_GATE    [M, D]  in workspace  (backward: bf16(dG Wg), which the
 *                                     second DGRAD adds to dU Wu)
 * Contents are those the last fwd (G, U, H) or bwd (the others) call wrote.
 */
enum {
  NVFP4_MLP_G = 0, NVFP4_MLP_U = 1, NVFP4_MLP_H = 2, NVFP4_MLP_DH = 3, NVFP4_MLP_DG = 4,
  NVFP4_MLP_DU = 5, NVFP4_MLP_DX_GATE = 6
};
/* *data = device address of tensor `which` inside saved / workspace (the
 * buffer that holds it must not be NULL; the other may be), *rows, *cols its
 * shape.  Returns NVFP4_ERR_SHAPE as nvfp4_mlp_sizes, NVFP4_ERR_INVALID_ARG for
 * an unknown `which` or a NULL pointer.  Nothing is launched. */
nvfp4_status nvfp4_mlp_tensor(int64_t M, int64_t D, int64_t F, const void* saved,
                              const void* workspace, int32_t which, void** data, int64_t* rows,
                              int64_t* cols);

/* The quantised operands of the nine GEMMs (descriptors with rows x cols the
 * logical K-major operand, as nvfp4_quantize fills them):
 *   Q_WG, Q_WU [F, D], Q_WD [D, F]  in saved  16x16 with the transpose
 *                                             (codes_t / scales_t)
 *   Q_XC [D, M], Q_HC [F, M]        in saved  the forward's WGRAD operands
 *   Q_X [M, D], Q_H [M, F]          in workspace (FPROP operands)
 *   Q_DY [M, D], Q_DG, Q_DU [M, F]  in workspace (DGRAD operands, SR)
 *   Q_DYC [D, M], Q_DGC, Q_DUC [F, M] in workspace (WGRAD operands)
 * *out receives the pointers into the buffers; amax and s_dec point at the
 * device floats the quantiser wrote.  Returns as nvfp4_mlp_tensor. */
enum {
  NVFP4_MLP_Q_WG = 16, NVFP4_MLP_Q_WU = 17, NVFP4_MLP_Q_WD = 18, NVFP4_MLP_Q_X = 19,
  NVFP4_MLP_Q_XC = 20, NVFP4_MLP_Q_H = 21, NVFP4_MLP_Q_HC = 22, NVFP4_MLP_Q_DY = 23,
  NVFP4_MLP_Q_DYC = 24, NVFP4_MLP_Q_DG = 25, NVFP4_MLP_Q_DGC = 26, NVFP4_MLP_Q_DU = 27,
  NVFP4_MLP_Q_DUC = 28
};
nvfp4_status nvfp4_mlp_operand(int64_t M, int64_t D, int64_t F, const void* saved,
                               const void* workspace, int32_t which, nvfp4_tensor* out);

/* ---------------------------------------------------------------------- */
/* Optimizer step of an FP32 master weight                                  */
/* ---------------------------------------------------------------------- */
/* "NVFP4 pretraining recipe" page, Figure 1 text: the MLP GEMMs' BF16
 * outputs are folded into FP32 master weights on the optimizer step, and
 * each step quantises the weights 16x16 under a per-tensor FP32 scale taken
 * from the tensor's amax.  This call is that step for one weight, fused with
 * the amax of the updated weight, so the next quantisation needs no amax
 * pass.  The pages name no optimizer: plain SGD on the FP32 master weight W
 * and the FP32 master gradient G (the WGRAD results the GEMM's
 * NVFP4_D_F32_ACCUM mode or nvfp4_mlp_bwd folded into it), elementwise in
 * binary32, the product rounded first:
 *   W[i]  = W[i] - lr * G[i]
 *   G[i]  = 0                  with NVFP4_ZERO_GRAD in flags
 *   *amax = max_i |W[i]|       of the updated W, when amax is not NULL: bit
 *                              for bit what nvfp4_amax returns for W, so it
 *                              can be given to the 16x16 quantiser
 *                              (NVFP4_AMAX_GIVEN), or written straight into
 *                              an MLP weight operand's amax slot for an
 *                              nvfp4_mlp_fwd with NVFP4_AMAX_GIVEN.
 * W, G: device float [n], 16-byte aligned, not overlapping; n > 0, n % 4 == 0;
 * lr finite.  amax: device float, 4-byte aligned, or NULL.  workspace:
 * device scratch of at least the nvfp4_quantize_sizes workspace size
 * (16-byte aligned) when amax is not NULL, else unused (may be NULL);
 * contents on return unspecified.  One read of W and G, one write of W (and
 * of G with NVFP4_ZERO_GRAD); two kernel launches on `stream` (one without
 * amax); nothing is allocated.  Returns NVFP4_ERR_INVALID_ARG (NULL W or G,
 * W and G overlapping, unknown flag bits, lr not finite), _SHAPE, _ALIGN,
 * _WORKSPACE, _ARCH, _CUDA. */
enum { NVFP4_ZERO_GRAD = 16u };
nvfp4_status nvfp4_sgd_step(float* W, float* G, int64_t n, float lr, uint32_t flags, float* amax,
                            void* workspace, size_t workspace_bytes, nvfp4_stream stream);

/* ---------------------------------------------------------------------- */
/* Orthogonalised momentum of matrices                                      */
/* ---------------------------------------------------------------------- */
/* The optimiser step for weights that are matrices (or a stack of them, such
 * as the experts' projections): a momentum, whose matrix is replaced by one
 * with nearly the same singular vectors and singular values near 1, by an
 * iteration of products (Newton-Schulz).  For each of `batch` matrices
 * [rows, cols]:
 *   V <- mu V + G,   U = G + mu V (nesterov) or V
 *   X <- U / max(||U||_F, eps, 1e-18)
 *   `steps` times, with the step's (a, b, c):
 *     A = X X^T,  B = b A + c A A,  X <- a X + B X
 *     (rows > cols: A = X^T X,  X <- a X + X B, the same polynomial)
 *   update = X
 * G the gradient (grad_dtype), V the FP32 momentum, U, X, A and B internal:
 * the products take f16 operands with what f16 would lose of X and of the
 * diagonals carried beside them, and FP32 accumulators; the update is within
 * about 1.5e-3 of that of 64 bits (2-norm of the difference) plus its one
 * rounding to bf16.  A matrix of zeros gives zeros.  NaN or infinities in a
 * matrix make its update (and momentum) unspecified, not the others'; a norm's
 * squares are summed in FP32, so norms below 1e-18 count as that, and above 1e18 as
 * infinity.  The entries of X, A and B must stay below 16 in magnitude, which they
 * do for every input with coefficients that keep X's singular values below 2 and
 * |b s + c s^2| below 16 on their squares s, as the usual (3.4445, -4.7750,
 * 2.0315) do. */
enum { NVFP4_MUON_MAX_STEPS = 32 };
typedef struct nvfp4_muon_params {
  int64_t batch, rows, cols;
  int32_t grad_dtype; /* nvfp4_in_dtype                                    */
  int32_t nesterov;   /* 0 or 1                                            */
  int32_t steps;      /* 1 .. NVFP4_MUON_MAX_STEPS                         */
  float mu;           /* momentum                                          */
  float eps;          /* > 0                                               */
  const float* coefs; /* host, [steps][3]; read before the call returns    */
} nvfp4_muon_params;

/* *workspace_bytes (may be NULL) = what nvfp4_muon_update needs: up to 21 MB where
 * min(rows, cols) <= 128, else about 6 bytes an element and 4 min(rows, cols)^2 a
 * matrix, and 11 MB.  NVFP4_ERR_SHAPE unless
 * 1 <= batch <= 65535, rows, cols >= 1, rows cols < 2^31 and
 * min(rows, cols) <= 32768. */
nvfp4_status nvfp4_muon_sizes(int64_t batch, int64_t rows, int64_t cols,
                              size_t* workspace_bytes);

/* grad [batch, rows, cols] (zeroed with NVFP4_ZERO_GRAD in flags), momentum float
 * [batch, rows, cols] (read and written), update bf16 [batch, rows, cols]; all
 * contiguous, 16-byte aligned, not overlapping.  Any rows and cols; rows of a
 * multiple of 8 elements take the fast loads and stores.  The result is the same
 * on every call.  workspace: device, 16-byte aligned, at least
 * nvfp4_muon_sizes gives; contents on return unspecified.  On `stream`, with nothing
 * allocated: one launch for matrices with a side of at most 128 and for a few of some
 * hundred rows or columns (with it, where CTAs meet by counters, a small memset; such
 * a launch is cooperative), else 2 + 3 steps.  Returns NVFP4_ERR_INVALID_ARG (NULL pointers,
 * overlaps, unknown flags or types, steps, mu, eps or coefs out of range),
 * _SHAPE, _ALIGN, _WORKSPACE, _ARCH, _CUDA. */
nvfp4_status nvfp4_muon_update(const nvfp4_muon_params* p, void* grad, float* momentum,
                               void* update, uint32_t flags, void* workspace,
                               size_t workspace_bytes, nvfp4_stream stream);

/* Applies an update to an FP32 master weight, elementwise in binary32:
 *   W[i]  = (1 - lr decay) W[i] - (lr scale) update[i]
 *   *amax = max_i |W[i]|  of the updated W, when amax is not NULL, as
 *           nvfp4_sgd_step gives it (NaN is left out, as there).
 * The factors are computed in binary64 and rounded once.  update bf16 [n], W
 * float [n], both 16-byte aligned, not overlapping; n > 0.  lr, scale, decay
 * finite.  workspace: as nvfp4_sgd_step.  One read of both, one write of W. */
nvfp4_status nvfp4_muon_apply(float* W, const void* update, int64_t n, float lr, float scale,
                              float decay, float* amax, void* workspace, size_t workspace_bytes,
                              nvfp4_stream stream);

/* ---------------------------------------------------------------------- */
/* Mixture of experts: routing, grouped products, norms                     */
/* ---------------------------------------------------------------------- */
/* The pages describe a dense MLP; these calls build the mixture-of-experts
 * form of it from the same quantisers and NVFP4 operands.  A block is
 *   nvfp4_residual_norm_fwd -> nvfp4_route_fwd -> nvfp4_dispatch ->
 *   quantise, nvfp4_group_gemm (gate, up), nvfp4_swiglu_fwd, quantise,
 *   nvfp4_group_gemm (down) -> nvfp4_combine -> nvfp4_residual_norm_fwd.
 *
 * Groups: expert e owns rows offsets[e] .. offsets[e] + sizes[e] - 1 of a
 * [rows, .] tensor.  The offsets are multiples of 128 (the rows of a scale
 * atom), rows is a multiple of 128, and the rows of a group's last block of
 * 128 past its size, and those from offsets[groups] on, are padding, which
 * every producer here writes as zero.  Groups do not overlap.  sizes [groups]
 * and offsets [groups + 1] are device int32 arrays: nothing of a plan is known
 * to the host, so a whole block can be captured into a graph. */

/* How the weights of the chosen experts are normalised. */
enum {
  NVFP4_ROUTE_ALL = 0,   /* softmax over all experts, the chosen ones' entries kept */
  NVFP4_ROUTE_CHOSEN = 1 /* softmax over the chosen experts                         */
};

/* *rows = the rows of a plan's tensors, a multiple of 128 that holds every
 * assignment of `tokens` tokens to `top` of `experts` experts:
 * floor((n + 127 min(experts, n)) / 128) 128 with n = tokens top; source has
 * as many entries.  *workspace_bytes = what nvfp4_route_fwd needs.  Either may
 * be NULL.  NVFP4_ERR_SHAPE unless tokens >= 1, 1 <= experts <= 512,
 * 1 <= top <= min(16, experts) and *rows <= INT32_MAX. */
nvfp4_status nvfp4_route_sizes(int64_t tokens, int64_t experts, int32_t top, int64_t* rows,
                               size_t* workspace_bytes);

/* Routes each token to `top` experts by its logits [tokens, experts] (bf16 or
 * FP32, leading dimension ld elements): the largest logits, the largest first,
 * the lowest index among equals.  A logit of -inf or NaN is never chosen;
 * +inf counts as the largest finite value.  Outputs (device, caller-owned):
 *   expert [tokens, top] int32  the chosen experts; -1 in the slots of a token
 *                               with fewer than `top` logits to choose from
 *   weight [tokens, top] float  their weights (mode NVFP4_ROUTE_*), 0 for -1
 *   sizes [experts], offsets [experts + 1] int32   the groups
 *   row [tokens, top] int32     the row of each slot among the groups, -1 for -1
 *   source [rows] int32         the slot (token top + j) of each row, -1: padding
 * A group's rows are in the order of the slots.  The result is the same on
 * every call.  workspace: device, 4-byte aligned, >= nvfp4_route_sizes gives, not
 * touched up to 64 tokens.  One launch up to 64 tokens, else three.  Returns NVFP4_ERR_INVALID_ARG,
 * _SHAPE, _ALIGN, _WORKSPACE, _ARCH, _CUDA. */
nvfp4_status nvfp4_route_fwd(const void* logits, int32_t in_dtype, int64_t tokens,
                             int64_t experts, int64_t ld, int32_t top, int32_t mode,
                             int32_t* expert, float* weight, int32_t* sizes, int32_t* offsets,
                             int32_t* row, int32_t* source, void* workspace,
                             size_t workspace_bytes, nvfp4_stream stream);

/* dlogits [tokens, experts] (contiguous, the logits' type) from dweight
 * [tokens, top]: w_i sum_j w_j (dw_i - dw_j) over a token's slots, with
 * NVFP4_ROUTE_ALL also the unchosen experts' share; exact zeros where an
 * expert could not be chosen.  expert, weight: as nvfp4_route_fwd wrote them
 * for the same logits and mode.  One launch. */
nvfp4_status nvfp4_route_bwd(const void* logits, int32_t in_dtype, int64_t tokens,
                             int64_t experts, int64_t ld, int32_t top, int32_t mode,
                             const int32_t* expert, const float* weight, const float* dweight,
                             void* dlogits, nvfp4_stream stream);

/* The same plan by scores, with a bias for balance and groups of experts.  For
 * each token, over the experts whose logit is not -inf or NaN (+inf counts as the
 * largest finite value):
 *   s_e = sigmoid(l_e), or softmax(l)_e
 *   a group's worth is the sum of the group_top largest s_e + bias_e among its
 *     experts (of one, where it has one); the groups_kept groups of the largest
 *     worth are kept
 *   the `top` experts of the largest s_e + bias_e in them are chosen, the largest
 *     first
 *   weight_i = scale s_i / (renormalise: sum of the chosen s; else 1)
 * The bias decides the choice alone.  Everything is compared as 64 bits have it,
 * equals by the lowest index; without a bias experts are compared by their
 * logits.  Groups are consecutive experts, all of one size.  Empty slots, plan and
 * workspace as nvfp4_route_fwd; launches too.  bias: device float [experts], finite,
 * or NULL.
 * NVFP4_ERR_SHAPE unless nvfp4_route_sizes accepts the sizes, groups is a power of
 * two up to 32 that divides experts, 1 <= groups_kept <= groups, group_top is 1 or
 * 2, and the kept groups have `top` experts; NVFP4_ERR_INVALID_ARG unless scale is
 * finite and above 0.  The rest as nvfp4_route_fwd. */
enum { NVFP4_SCORE_SOFTMAX = 0, NVFP4_SCORE_SIGMOID = 1 };
typedef struct nvfp4_route_params {
  int64_t tokens, experts, ld;
  int32_t in_dtype;    /* nvfp4_in_dtype of the logits (and their gradient)  */
  int32_t top;
  int32_t score;       /* NVFP4_SCORE_*                                      */
  int32_t renormalise; /* 0 or 1                                             */
  int32_t groups, groups_kept, group_top;
  float scale;
} nvfp4_route_params;
nvfp4_status nvfp4_route_scored_fwd(const nvfp4_route_params* p, const void* logits,
                                    const float* bias, int32_t* expert, float* weight,
                                    int32_t* sizes, int32_t* offsets, int32_t* row,
                                    int32_t* source, void* workspace, size_t workspace_bytes,
                                    nvfp4_stream stream);

/* dlogits [tokens, experts] (contiguous, the logits' type) from dweight [tokens,
 * top], over a token's slots i, j, with v = weight / scale:
 *   softmax, renormalised   dl_i = w_i sum_j v_j (dw_i - dw_j)
 *   softmax                 the same plus the unchosen experts' share, who get
 *                           -s_e sum_j w_j dw_j
 *   sigmoid, renormalised   dl_i = w_i (1 - s_i) sum_j v_j (dw_i - dw_j)
 *   sigmoid                 dl_i = w_i (1 - s_i) dw_i
 * and zero elsewhere.  expert, weight: as nvfp4_route_scored_fwd wrote them for the
 * same logits and parameters (those of the groups are not read, but checked).  One
 * launch. */
nvfp4_status nvfp4_route_scored_bwd(const nvfp4_route_params* p, const void* logits,
                                    const int32_t* expert, const float* weight,
                                    const float* dweight, void* dlogits, nvfp4_stream stream);

/* bias_e += rate sign(mean of the loads - sizes[e]), the loads a plan's sizes
 * [experts] or the sum of several plans': experts with more than their share lose
 * rate, the others gain it, and one at the mean keeps its bias.  1 <= experts <=
 * 512.  One launch. */
nvfp4_status nvfp4_route_balance(const int32_t* sizes, int64_t experts, float rate, float* bias,
                                 nvfp4_stream stream);

/* xe [rows, cols] bf16: row row[t, j] is x[t], x bf16 [tokens, cols]; rows whose
 * source is -1 are zero.  cols % 8 == 0, all tensors contiguous and 16-byte
 * aligned.  Entries of `row` outside [0, rows) are skipped.  The gradient is
 * nvfp4_combine without weights.  One launch. */
nvfp4_status nvfp4_dispatch(const void* x, const int32_t* row, const int32_t* source,
                            int64_t tokens, int64_t cols, int32_t top, int64_t rows, void* xe,
                            nvfp4_stream stream);

/* y[t] = sum_j weight[t, j] o[row[t, j]] (weight NULL: all ones) in FP32,
 * rounded once to bf16; a token without rows gets zeros.  Shapes as
 * nvfp4_dispatch. */
nvfp4_status nvfp4_combine(const void* o, const int32_t* row, const float* weight,
                           int64_t tokens, int64_t cols, int32_t top, int64_t rows, void* y,
                           nvfp4_stream stream);

/* The gradients of nvfp4_combine from dy bf16 [tokens, cols]: d_o [rows, cols]
 * bf16, row row[t, j] is weight[t, j] dy[t] and padding rows are zero;
 * dweight[t, j] = sum_c dy[t, c] o[row[t, j], c] (0 for a slot without a row).
 * d_o may not be o.  One launch. */
nvfp4_status nvfp4_combine_bwd(const void* dy, const void* o, const int32_t* row,
                               const int32_t* source, const float* weight, int64_t tokens,
                               int64_t cols, int32_t top, int64_t rows, void* d_o,
                               float* dweight, nvfp4_stream stream);

/* Products grouped by expert: D[r, :] = alpha A[r, :] . B_e^T for the rows r of
 * group e, alpha = *A->s_dec * *B->s_dec.  A [rows, K] is a row-wise operand.
 *   b_view 0: B [groups * N, K], expert e's weights in rows e N .. (FPROP)
 *   b_view 1: B [groups * K, N] quantised 16x16 with NVFP4_EMIT_T, expert e in
 *             rows e K ..; codes_t / scales_t are read (DGRAD)
 * d_mode NVFP4_D_BF16 or NVFP4_D_BF16_ADD_C (adds C bf16 [rows, N] in FP32
 * before the rounding).  D bf16 [rows, N]: padding rows are written as zero
 * whatever A (or C) holds there.  tile: NVFP4_TILE_AUTO, or for tuning and
 * tests NVFP4_TILE_PAIR_256X256 or _PAIR_256X384.  Shapes: rows % 128 == 0, N % 128 == 0,
 * K % 64 == 0, 1 <= groups <= 512.  A group that does not lie in [0, rows) or
 * does not start on a multiple of 128 counts as empty.  One launch.  Returns
 * NVFP4_ERR_INVALID_ARG, _SHAPE, _ALIGN, _ARCH, _CUDA. */
nvfp4_status nvfp4_group_gemm(const nvfp4_tensor* A, const nvfp4_tensor* B, int32_t b_view,
                              const int32_t* sizes, const int32_t* offsets, int32_t groups,
                              void* D, int32_t d_mode, const void* C, int64_t rows, int64_t N,
                              int64_t K, int32_t tile, nvfp4_stream stream);

/* Weight gradients grouped by expert: D_e [M, N] = alpha A[:, rows of e] .
 * B[:, rows of e]^T for A [M, rows], B [N, rows] column-wise operands
 * (NVFP4_COL_1X16 of the [rows, M] and [rows, N] tensors, with the RHT on both
 * or on neither); the padding rows of those tensors must have been zero.
 *   NVFP4_D_BF16       D bf16 [groups, M, N], zeros for an empty group
 *   NVFP4_D_F32_ACCUM  D fp32 [groups, M, N] += the FP32 product, not rounded
 *                      to bf16 in between (an empty group's D stays as it is);
 *                      one addition an element, in L2, which flushes
 *                      subnormal operands and results to zero
 * tile: NVFP4_TILE_AUTO, _PAIR_256X256, or with NVFP4_D_BF16 _PAIR_256X384.
 * Shapes: rows, M, N multiples of 128, 1 <= groups <= 512.  One launch. */
nvfp4_status nvfp4_group_wgrad(const nvfp4_tensor* A, const nvfp4_tensor* B,
                               const int32_t* sizes, const int32_t* offsets, int32_t groups,
                               void* D, int32_t d_mode, int64_t M, int64_t N, int64_t rows,
                               int32_t tile, nvfp4_stream stream);

/* The gate of a block's output in nvfp4_residual_norm_*. */
enum {
  NVFP4_GATE_NONE = 0,
  NVFP4_GATE_CHANNEL = 1, /* gate [cols] */
  NVFP4_GATE_ROW = 2      /* gate [rows] */
};
typedef struct nvfp4_norm_params {
  int64_t rows, cols;
  int32_t stream_dtype; /* nvfp4_in_dtype of x, y, dy, dx                */
  int32_t gate_mode;    /* NVFP4_GATE_*                                  */
  float eps;            /* > 0                                           */
  float x_scale;        /* a, of the residual stream                     */
  float z_scale;        /* b, of the block's output                      */
} nvfp4_norm_params;

/* The norms after a block and before the next one in one pass:
 *   y = a x + b g (.) (z r_z w_post),   h = y r_y w_pre,
 *   r_v = (mean over the row of v^2 + eps)^(-1/2),
 * x the residual stream [rows, cols], z (bf16) the block's output, h (bf16)
 * the next block's input; w_post, w_pre, gate FP32.  y is rounded once when
 * stored, h comes from y before that rounding.  y may be x.
 * z NULL (with w_post NULL): y = a x, the first block's norm, y may be NULL
 * then; w_pre NULL (with h NULL): no norm follows.
 * cols % 8 == 0, cols <= 65536; all tensors contiguous and 16-byte aligned (a
 * row gate: 4-byte).  One launch.  Returns NVFP4_ERR_INVALID_ARG, _SHAPE,
 * _ALIGN, _ARCH, _CUDA. */
nvfp4_status nvfp4_residual_norm_fwd(const nvfp4_norm_params* p, const void* x, const void* z,
                                     const float* w_post, const float* gate, const float* w_pre,
                                     void* y, void* h, nvfp4_stream stream);

/* Its gradients from dy (NULL: zero) and dh (NULL exactly when w_pre is):
 * dx (the stream's type), dz bf16, and FP32 dw_post [cols], dgate (the gate's
 * shape), dw_pre [cols], written, not accumulated; an output is NULL exactly
 * when its input is.  Everything is recomputed from x and z: nothing of the
 * forward is kept.  dx may be dy, dz may be dh or z.  workspace: device,
 * 16-byte aligned, at least nvfp4_residual_norm_bwd_sizes gives.  Two
 * launches; sums are taken in a fixed order.  Statuses as the forward and
 * _WORKSPACE. */
nvfp4_status nvfp4_residual_norm_bwd_sizes(int64_t rows, int64_t cols, size_t* workspace_bytes);
nvfp4_status nvfp4_residual_norm_bwd(const nvfp4_norm_params* p, const void* dy, const void* dh,
                                     const void* x, const void* z, const float* w_post,
                                     const float* gate, const float* w_pre, void* dx, void* dz,
                                     float* dw_post, float* dgate, float* dw_pre,
                                     void* workspace, size_t workspace_bytes,
                                     nvfp4_stream stream);

#ifdef __cplusplus
}
#endif
#endif /* NVFP4_H */
