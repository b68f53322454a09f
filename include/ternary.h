/*
 * ternary.h - C ABI of the MI355X (gfx950) ternary-weight linear layer.
 *
 *     y[m,n] = sum_k x[m,k] * q[n,k] * s(n,k)          (y = x * (q (.) s)^T)
 *
 * Sources (page titles and sections):
 *   [trdm] trdm.cn, "三元量化模型接入vLLM：从逆向加载到Kernel优化的完整实战":
 *          §3.1 packing rule; §4.2 operand shapes; §4.4 2-D contiguous input.
 *   [nxbn] m.nxbn.cn/news/169761 (a 7B ternary checkpoint into vLLM):
 *          §2.2 code table and bit order; §3.2 per-channel scale broadcast
 *          over rows; §5.2 the layer's forward takes (x, weight, scale).
 *   [xxqk] m.xxqk.cn/news/593501 (Bonsai 2 27B into vLLM): §4.3 the layer is
 *          dequantise-then-matmul; §4.2/§5.2 checkpoints grouped by 64.
 *   [ch13] yangyitao.com vLLM book, "第13章 量化：精度与速度的工程平衡":
 *          §13.1.3 symmetric linear quantization; §13.1.4 its s/2 error
 *          bound; §13.3 scale granularity (per channel, per group; §13.3.3 group
 *          sizes 128, 32, 256); §13.8.2 group_size = -1 means one group per
 *          row.
 *
 * Format (fixed by [trdm §3.1] and [nxbn §2.2]):
 *   - each weight is a 2-bit code: 00 -> 0, 01 -> +1, 10 -> -1, 11 -> reserved,
 *     read as 0 by every function here and never written by ternary_pack;
 *   - four codes per byte, little-endian: weight 4j+i of a row lives in bits
 *     [2i+1:2i] of byte j of that row;
 *   - packed weights are [N, K/4] bytes, row-major (one row per output channel,
 *     K contiguous);
 *   - scales are IEEE binary16 bit patterns: [N] when group_size == -1 (one per
 *     output channel, [nxbn §3.2]) or [N, K/g] row-major when group_size == g
 *     (g consecutive K weights of a row share one: g = 128 in [trdm §3.1], 64
 *     in [xxqk §4.2], 32 and 256 in [ch13 §13.3.3]).
 *
 * Tiled layout (this library's, not the pages'; TERNARY_LAYOUT_TILED): the same
 * bytes as the row-major packing, permuted so that the matrix-core kernels read
 * one contiguous kilobyte per wave instruction.  Rows are padded to a multiple
 * of 16 and K to a multiple of 256 with code 00; with Ks = ceil(K / 256), byte
 * j of row n of the row-major packing (j < K/4) sits at
 *     ((n / 16) * Ks + j / 64) * 1024 + ((j % 64) / 16) * 256 + (n % 16) * 16 + j % 16
 * i.e. block (n/16, j/64) of 16 rows x 64 bytes is 1 KB, stored as four
 * [16 rows][16 bytes] quarters in K order.  ternary_tiled_bytes() gives the
 * size, ternary_tile()/ternary_untile() convert; every linear entry point that
 * takes a layout reads either.
 *
 * Conventions shared by every entry point:
 *   - All data pointers are DEVICE pointers, owned by the caller.  The library
 *     keeps no reference after a call returns and never allocates or frees
 *     caller memory.
 *   - The library owns one device workspace per (device, stream) for GEMM
 *     shapes whose K range it splits over several workgroups (fp32 partial
 *     tiles, added in a fixed order by a second kernel): shapes with few
 *     output tiles, few-token shapes with long K, and batches in which one
 *     problem's K is much longer than the others'.  The first call on a
 *     stream that needs a larger one allocates it (hipMalloc); the one it
 *     replaces stays allocated (a graph captured earlier may use it) until
 *     ternary_shutdown(), which frees them all.  Under stream capture nothing
 *     is allocated: a call that would need a larger workspace returns
 *     TERNARY_ERR_WORKSPACE, so warm a stream up (one call per shape) before
 *     capturing on it.  ternary_linear_batch_noalloc allocates nothing.
 *   - Work is enqueued asynchronously on `stream` (NULL = the default stream).
 *     Arguments are validated on the host before anything is launched; on any
 *     error a negative ternary_status is returned and nothing is enqueued.
 *     Faults during execution surface at the next synchronisation of the
 *     stream, as for any HIP kernel.
 *   - Every call is deterministic: the same inputs give the same bits.
 *   - No function throws; C++ exceptions never cross this boundary.
 */
#ifndef TERNARY_LINEAR_H
#define TERNARY_LINEAR_H

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    TERNARY_OK = 0,
    TERNARY_ERR_NULL = -1,   /* a required pointer is NULL                       */
    TERNARY_ERR_SHAPE = -2,  /* negative size, K % 4 != 0, K % group != 0, ...   */
    TERNARY_ERR_GROUP = -3,  /* group_size is not -1, 32, 64, 128 or 256         */
    TERNARY_ERR_DTYPE = -4,  /* activation dtype is not TERNARY_BF16/TERNARY_FP16*/
    TERNARY_ERR_ALIGN = -5,  /* a pointer is not aligned as documented           */
    TERNARY_ERR_ALIAS = -6,  /* the output overlaps an input                     */
    TERNARY_ERR_HIP = -7,    /* a HIP runtime call or kernel launch failed       */
    TERNARY_ERR_PATH = -8,   /* a forced kernel path cannot take this shape      */
    TERNARY_ERR_WORKSPACE = -9, /* stream under capture, its split-K workspace too
                                   small: run the same call once outside capture */
    TERNARY_ERR_SCRATCH = -10   /* ternary_linear_batch_noalloc: the call needs more
                                   split-K scratch than TERNARY_NOALLOC_SCRATCH_BYTES */
} ternary_status;

/* Weight layout of a linear call (see "Tiled layout" above). */
typedef enum { TERNARY_LAYOUT_ROWS = 0, TERNARY_LAYOUT_TILED = 1 } ternary_layout;

/* Activation / output element type (2 bytes per element; TERNARY_FP32, 4 bytes,
 * only where a function says so). */
typedef enum { TERNARY_BF16 = 0, TERNARY_FP16 = 1, TERNARY_FP32 = 2 } ternary_dtype;

/* Kernel path for ternary_linear_ex.  AUTO picks by M (see ternary_linear). */
typedef enum {
    TERNARY_PATH_AUTO = 0,
    TERNARY_PATH_GEMV = 1,     /* decode GEMV, requires 1 <= M <= ternary_gemv_max_m();
                                  at M == 1 the fp4 x fp8 kernel (a single call of
                                  fewer than 8192 channels and K > 8192: the
                                  16-bit one), at
                                  larger M the 16-bit one, each where it takes the
                                  shape, else the other                                */
    TERNARY_PATH_GEMM = 2,     /* prefill kernel (bf16/fp16 MFMA)                       */
    TERNARY_PATH_SIMPLE = 3,   /* plain one-output-per-thread kernel, any valid shape   */
    TERNARY_PATH_GEMV_F4 = 4,  /* decode GEMV on the scaled fp4 x fp8 matrix
                                  instruction (codes as fp4, x as exact fp8 pieces)     */
    TERNARY_PATH_GEMV_B16 = 5, /* decode GEMV on the bf16/fp16 matrix instruction
                                  (codes as 16-bit +-2 / 0)                            */
    TERNARY_PATH_GEMV_VALU = 6, /* decode GEMV on the vector ALU: each code adds +x, -x
                                  or nothing in fp32 ([nxbn §4.1]), lanes reduced by
                                  cross-lane exchange; M == 1, K % 256 == 0, per
                                  channel or groups of 64/128/256, row-major codes
                                  only.  Never chosen by AUTO (measured slower); kept
                                  for comparison                                        */
    TERNARY_PATH_FEW = 7,      /* few-token streaming GEMM: 1 <= M <= 32 (16 for groups
                                  of 128), K % 256 == 0, K <= 65536 (groups of 128:
                                  K >= 1024), per channel or groups of 128 / 256; x
                                  shared in LDS by the eight 16-channel blocks of a
                                  workgroup, codes streamed into registers             */
    TERNARY_PATH_GEMM_ZSKIP = 8 /* the pipelined GEMM skipping all-zero code blocks
                                  ([trdm §6]; a wave's channels x 64 K): the shapes
                                  TERNARY_PATH_GEMM takes on the pipelined kernel
                                  (K % 256 == 0, ...); the same bits as that path.
                                  Pays only on block-sparse codes; never chosen by
                                  AUTO                                                 */
} ternary_path;

/*
 * ternary_pack - encode ternary values as 2-bit codes ([trdm §3.1]).
 *   q             int8 [N, K], row-major, values in {-1, 0, +1}; 16-byte aligned.
 *   N, K          N >= 0, K >= 0, K % 4 == 0.
 *   packed        uint8 [N, K/4] output, 16-byte aligned, must not overlap q.
 *   invalid_count optional int32 (device).  Each value outside {-1, 0, +1} is
 *                 written as code 00 and counted; the count is ADDED to
 *                 *invalid_count (the caller zeroes it).  NULL skips counting.
 * N == 0 or K == 0 is a successful no-op.
 */
int ternary_pack(const int8_t *q, int64_t N, int64_t K, uint8_t *packed,
                 int32_t *invalid_count, hipStream_t stream);

/*
 * ternary_unpack - decode 2-bit codes to int8 {-1, 0, +1} ([trdm §3.1],
 * [nxbn §2.2]); code 11 decodes to 0.  Bit-exact inverse of ternary_pack for
 * bytes that hold no code 11.
 *   packed  uint8 [N, K/4], 16-byte aligned.
 *   q       int8 [N, K] output, 16-byte aligned, must not overlap packed.
 */
int ternary_unpack(const uint8_t *packed, int64_t N, int64_t K, int8_t *q, hipStream_t stream);

/*
 * ternary_tiled_bytes - size in bytes of the tiled layout of an [N, K] code
 * matrix: ceil(N/16) * 16 * ceil(K/256) * 64.  Returns TERNARY_ERR_SHAPE for
 * N < 0, K < 0, K % 4 != 0, N or K above 2^24, or more than 2^40 bytes (the
 * limits of ternary_tile / ternary_untile as well).
 */
int64_t ternary_tiled_bytes(int64_t N, int64_t K);

/*
 * ternary_tile - row-major packed codes -> tiled layout (a byte permutation;
 * padding bytes are written as 0).
 *   packed  uint8 [N, K/4], 16-byte aligned.
 *   tiled   uint8 [ternary_tiled_bytes(N, K)] output, 16-byte aligned, must not
 *           overlap packed.
 * N == 0 or K == 0 is a successful no-op.  ternary_untile is the inverse
 * (same arguments, tiled -> packed; padding bytes are not read).
 */
int ternary_tile(const uint8_t *packed, int64_t N, int64_t K, uint8_t *tiled,
                 hipStream_t stream);
int ternary_untile(const uint8_t *tiled, int64_t N, int64_t K, uint8_t *packed,
                   hipStream_t stream);

/*
 * ternary_quantize - codes and scales of 16-bit weights (the step before the
 * layer: its packed and scale inputs).
 *   w           [N, K] weights, dtype `dtype` (TERNARY_BF16 or TERNARY_FP16),
 *               row-major, 16-byte aligned.
 *   N, K        N >= 0, K > 0, K % 4 == 0, K % group_size == 0 when grouped;
 *               N == 0 is a successful no-op.
 *   group_size  -1 (one scale per row) or 32, 64, 128, 256.
 *   packed      uint8 [N, K/4] output, 16-byte aligned.
 *   scale       fp16 [N] or [N, K/group_size] output, 2-byte aligned.
 * No output may overlap w or the other output.  Rule: the symmetric linear
 * quantizer of [ch13 §13.1.3] with the code range {-1, 0, +1}: per group,
 * s = max |w| rounded to fp16 (nearest even), and q = round(w / s) with ties
 * to even, i.e. q = sign(w) where |w| > s/2 and 0 elsewhere; a group with
 * s == 0 gets q = 0.  Then |w - q*s| <= s/2 for every weight ([ch13 §13.1.4]).
 * w must be finite with every group's max |w| below 65520 (s finite in
 * fp16); results are unspecified otherwise.  Deterministic, bit-exact.
 */
int ternary_quantize(const void *w, int dtype, int64_t N, int64_t K, int64_t group_size,
                     uint8_t *packed, uint16_t *scale, hipStream_t stream);

/*
 * ternary_linear - y = x * (q (.) s)^T ([xxqk §4.3]; operand shapes [trdm §4.2]).
 *   x           [M, K] activations, dtype `dtype`, row-major contiguous
 *               ([trdm §4.4]: callers flatten leading dims to M), 16-byte aligned.
 *   dtype       TERNARY_BF16 or TERNARY_FP16; y has the same dtype.
 *   M, N, K     M >= 0, N >= 0, K > 0, K % 4 == 0; K % group_size == 0 when
 *               grouped.  M == 0 or N == 0 is a successful no-op.
 *   packed      uint8 [N, K/4] codes as above, 16-byte aligned.
 *   scale       fp16 bit patterns, [N] (group_size == -1) or [N, K/group_size]
 *               (grouped), 2-byte aligned.
 *   group_size  -1 (per output channel, [ch13 §13.8.2] convention) or the
 *               group size: 32, 64, 128 or 256.
 *   y           [M, N] output, 16-byte aligned, must not overlap any input.
 * Products are formed exactly and accumulated in fp32; the scale multiplies
 * each group's (or the row's) fp32 partial sum; y is rounded from fp32 to the
 * output dtype, round-to-nearest-even.  x and s must be finite (results for
 * non-finite inputs are unspecified) and |x| < 2^126.
 * Path choice: M <= ternary_gemv_max_m() runs the decode GEMV (the fp4 x fp8
 * kernel at M == 1 except for N < 8192 with K > 8192, the 16-bit one otherwise, each where
 * it takes the shape); 9 <= M <= 32 the few-token GEMM (TERNARY_PATH_FEW) where it takes
 * the shape (groups of 128: M <= 16); larger M and the rest the MFMA GEMM; shapes no fast kernel
 * takes (K % 128 != 0) run the plain kernel.  The GEMV gives each token 2
 * MFMA columns (per channel, groups of 128 or 256), 4 (groups of 64) or 8
 * (groups of 32) of 16, so it takes M <= 4 for groups of 64 and 32 (M <= 2
 * where the fp4 kernel's LDS cannot hold x), and K <= 65536.  Results of different paths agree within the bound
 * |y - y_ref| <= 1e-3 * sum_k |x_k| * s(n,k) + 1e-6, not bitwise.
 */
int ternary_linear(const void *x, int dtype, int64_t M, int64_t N, int64_t K,
                   const uint8_t *packed, const uint16_t *scale, int64_t group_size,
                   void *y, hipStream_t stream);

/* ternary_linear with an explicit kernel path (ternary_path); AUTO is the
 * default choice above.  A forced path that cannot take the shape returns
 * TERNARY_ERR_PATH without launching. */
int ternary_linear_ex(const void *x, int dtype, int64_t M, int64_t N, int64_t K,
                      const uint8_t *packed, const uint16_t *scale, int64_t group_size,
                      void *y, int path, hipStream_t stream);

/*
 * ternary_linear_tiled - ternary_linear_ex with the codes in the tiled layout:
 *   tiled  uint8 [ternary_tiled_bytes(N, K)], 16-byte aligned; every other
 *          argument as for ternary_linear_ex.
 * The same products, sums and rounding as the row-major call.  Paths: both
 * decode GEMVs, the pipelined GEMM and the plain kernel read the tiled
 * layout; the GEMM shapes only the 128 x 128 kernel takes (K % 256 != 0, group
 * size 32, an odd number of groups per row, scales not 4-byte aligned) run the
 * plain kernel under TERNARY_PATH_AUTO and return TERNARY_ERR_PATH when
 * TERNARY_PATH_GEMM is forced.  A forced path runs the same kernel, with the
 * same launch shape, on tiled as on row-major codes: the results are the
 * same bits.
 */
int ternary_linear_tiled(const void *x, int dtype, int64_t M, int64_t N, int64_t K,
                         const uint8_t *tiled, const uint16_t *scale, int64_t group_size,
                         void *y, int path, hipStream_t stream);

/* Most problems one ternary_linear_batch call takes. */
#define TERNARY_MAX_BATCH 8

/* One projection of a batched call: the arguments of ternary_linear. */
typedef struct {
    const void *x;          /* [M, K] activations, 16-byte aligned                  */
    const uint8_t *packed;  /* [N, K/4] codes, 16-byte aligned                      */
    const uint16_t *scale;  /* fp16 [N] or [N, K/group_size], 2-byte aligned        */
    void *y;                /* [M, N] output, 16-byte aligned                       */
    int64_t M, N, K;        /* as for ternary_linear                                */
    int64_t group_size;     /* -1, 32, 64, 128 or 256                               */
    int64_t layout;         /* TERNARY_LAYOUT_ROWS ([N, K/4] as above) or
                               TERNARY_LAYOUT_TILED (packed holds
                               ternary_tiled_bytes(N, K) bytes)                    */
} ternary_problem;

/*
 * ternary_linear_batch - several independent ternary_linear problems in as
 * few launches as possible, for the projections of one layer: the segments of
 * a fused QKV (or gate+up) weight, each with its own packed rows and scales
 * ([trdm §2.2]), or any set of projections that are ready together.
 *   problems  host array of `count` problems (1 <= count <= TERNARY_MAX_BATCH),
 *             read during the call only.
 *   dtype     activation/output dtype shared by all problems.
 * Every problem is validated as by ternary_linear (or ternary_linear_tiled);
 * an unknown layout returns TERNARY_ERR_SHAPE; in addition no output may
 * overlap any input or any other output of the batch (TERNARY_ERR_ALIAS).  On
 * any error nothing is launched.  Problems the automatic path sends to the
 * decode GEMV (see ternary_linear) run together in one launch per scale
 * mode (per channel, or each group size) and token count M; problems the
 * automatic path sends to the few-token GEMM run together in one launch per
 * scale mode (plus one launch adding the K slices of sliced problems);
 * the GEMM problems the pipelined kernel takes (K % 256 == 0; group sizes 64,
 * 128 or 256 with an even number of groups per row and 4-byte-aligned scales)
 * run together in one grouped GEMM launch per scale mode and tile shape
 * (longest K first); the others run as separate launches on the same stream.  Results are
 * deterministic (the same batch gives the same bits) and each satisfies the
 * bound of ternary_linear; they may differ from a single ternary_linear call on
 * the same problem in the last bits, because a batch may split a problem's K
 * range into a different number of partial sums.
 */
int ternary_linear_batch(const ternary_problem *problems, int count, int dtype,
                         hipStream_t stream);

/* The path ternary_linear_ex(..., TERNARY_PATH_AUTO, ...) takes for a shape
 * (a ternary_path value), or a negative status for invalid shapes.  A
 * group-128 scale array is assumed 4-byte aligned (else the few-token GEMM's
 * shapes take the GEMM). */
int ternary_select_path(int64_t M, int64_t N, int64_t K, int64_t group_size);

/* Largest M the decode GEMV accepts. */
int ternary_gemv_max_m(void);

/* Human-readable name of a ternary_status value (static storage). */
const char *ternary_status_string(int status);

/* Library ABI version (increments when a signature or a convention changes). */
int ternary_abi_version(void);

/*
 * ternary_shutdown - free the library's workspaces, those replaced by larger
 * ones included.  Waits for every device that holds one, then frees them;
 * later calls allocate again as needed.  A HIP graph captured before with a
 * split-K GEMM launch in it must not be replayed afterwards.  Returns
 * TERNARY_ERR_HIP if a synchronisation or free failed (the remaining
 * workspaces are still released).
 */
int ternary_shutdown(void);

/* Bytes of the static scratch array of ternary_linear_batch_noalloc. */
#define TERNARY_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

/*
 * ternary_linear_batch_noalloc - ternary_linear_batch for callers that cannot
 * allocate device memory: code under stream capture, tight serving loops,
 * harnesses that forbid hipMalloc.  Same arguments, validation, results (the
 * same bits) and launches as ternary_linear_batch, but the fp32 partial tiles
 * of a split-K GEMM and the K-slice sums of the few-token GEMM (one launch
 * after another, so they share it) go to a static device array of the library
 * (TERNARY_NOALLOC_SCRATCH_BYTES per GPU, held until the process ends) instead
 * of the per-stream workspace: the call never allocates or frees.  A batch
 * whose split-K partials need more returns TERNARY_ERR_SCRATCH and enqueues
 * nothing.  Every call on one GPU shares that GPU's array: calls that overlap
 * on a GPU (other streams, other host threads) race, and a graph captured with
 * it must not be replayed while another such call runs on the GPU.
 */
int ternary_linear_batch_noalloc(const ternary_problem *problems, int count, int dtype,
                                 hipStream_t stream);

/*
 * ---------------------------------------------------------------------------
 * 8-bit layers and experts.  The layers of a ternary model that stay at 8 bits
 * (ternary_fp8_linear), and mixtures of ternary experts, as one chain:
 *
 *   x   -> ternary_fp8_quantize -> ternary_fp8_linear (gate logits) -> ternary_route
 *   xq  -> ternary_linear_experts (gate | up) -> ternary_fp8_quantize (SwiGLU)
 *       -> ternary_linear_experts (down) -> ternary_combine
 *
 * An 8-bit value is an e4m3 code (OCP: 4 exponent bits, 3 fraction bits, largest
 * 448, 0x7f / 0xff NaN, no infinities); a scale is an fp32 number for each block of
 * 128 values along K, of one row (activations) or of 128 rows (weights): an
 * 8-bit matrix [M, Kp] (Kp a multiple of 128) has scales [M, Kp/128] or
 * [ceil(M/128), Kp/128], row-major, and stands for code * scale.
 *
 * The conventions above hold for these functions too; none of them uses a
 * library-owned workspace, so any of them may be captured, replayed and run
 * on several streams at once.
 * ---------------------------------------------------------------------------
 */

/* Values along K (and rows, for weights) that share one scale. */
#define TERNARY_FP8_BLOCK 128

/* Which values of ternary_fp8_quantize share a scale. */
typedef enum {
    TERNARY_BLOCK_ROW = 0,  /* 128 values of one row (activations)      */
    TERNARY_BLOCK_TILE = 1  /* 128 rows x 128 values of each (weights)  */
} ternary_block;

/* What ternary_fp8_quantize computes before it quantises. */
typedef enum {
    TERNARY_ACT_NONE = 0,
    TERNARY_ACT_SWIGLU = 1  /* silu(x[:, :K]) * x[:, K:2K], silu(g) = g / (1 + exp(-g)) */
} ternary_act;

/*
 * ternary_fp8_quantize - e4m3 codes and block scales of a matrix.
 *   x      [M, K] (TERNARY_ACT_SWIGLU: [M, 2K], the gate's K columns first), dtype
 *          `dtype` (TERNARY_BF16, TERNARY_FP16 or TERNARY_FP32), row r at element
 *          r * ldx; aligned to its elements' size.
 *   M, K   0 <= M, 0 < K, both up to 2^24; M == 0 is a successful no-op.
 *   ldx    elements between rows, at least the row's length.
 *   block  a ternary_block; act a ternary_act (TERNARY_ACT_SWIGLU with
 *          TERNARY_BLOCK_ROW only).
 *   q      uint8 [M, Kp] output, Kp = K rounded up to a multiple of 128 (the
 *          columns from K on are written as 0), 16-byte aligned.
 *   scale  fp32 output, [M, Kp/128] (rows) or [ceil(M/128), Kp/128] (tiles).
 * Rule: s = (largest |v| of the block) / 448 rounded to fp32, q = v / s rounded
 * to fp32 and then to the nearest e4m3 code, ties to even; v is x, or the
 * activation's fp32 result (not rounded in between).  A block with s == 0 gets
 * codes 0.  A NaN is written as NaN and left out of its block's largest; a block with an infinity has
 * scale infinity, its finite values the code 0 and its infinities NaN (so what it
 * stands for is NaN throughout).  No output may overlap x or the other output.
 */
int ternary_fp8_quantize(const void *x, int dtype, int64_t M, int64_t K, int64_t ldx, int block,
                         int act, uint8_t *q, float *scale, hipStream_t stream);

/*
 * ternary_fp8_linear - y = x * w^T of block-scaled 8-bit matrices.
 *   x, x_scale  e4m3 [M, K] and fp32 [M, K/128] (TERNARY_BLOCK_ROW).
 *   w, w_scale  e4m3 [N, K] and fp32 [ceil(N/128), K/128] (TERNARY_BLOCK_TILE).
 *   M, N, K     M >= 0, N >= 0, K > 0, K % 128 == 0, each up to 2^24, K up to 2^20;
 *               M == 0 or N == 0 is a successful no-op.
 *   y           [M, N] output, dtype `dtype` (TERNARY_BF16, TERNARY_FP16 or
 *               TERNARY_FP32), 16-byte aligned; must not overlap any input.
 * x and w 16-byte, the scales 4-byte aligned.  For each block of 128 along K
 * the products are exact and summed; x_scale * w_scale (an fp32
 * product) multiplies the block's sum and the blocks are added in fp32, in an
 * order that depends on M, N and K alone; y is rounded once, to nearest even.
 * Sums are fp32 for every dtype: each of a block's 128 additions is off by at most 2^-23 of
 * the block's sum of magnitudes (the matrix unit may cut what lies below instead of rounding).
 * A NaN code or scale gives NaN in every output that reads it.
 */
int ternary_fp8_linear(const uint8_t *x, const float *x_scale, const uint8_t *w,
                       const float *w_scale, int64_t M, int64_t N, int64_t K, void *y, int dtype,
                       hipStream_t stream);

/* What a router's logits become. */
typedef enum { TERNARY_SCORE_SOFTMAX = 0, TERNARY_SCORE_SIGMOID = 1 } ternary_score;

/* Limits of ternary_route (experts also of ternary_linear_experts, top_k of
 * ternary_combine). */
#define TERNARY_MAX_EXPERTS 512
#define TERNARY_MAX_TOP_K 32
#define TERNARY_MAX_EXPERT_GROUPS 64

/*
 * ternary_route - each token's experts, their weights, and the token slots
 * sorted by expert.
 *   logits      [T, E], dtype `dtype` (TERNARY_BF16, TERNARY_FP16, TERNARY_FP32),
 *               row-major, aligned to its elements' size.
 *   T, E        0 <= T <= 2^24, 1 <= E <= TERNARY_MAX_EXPERTS, T * top_k < 2^31.
 *   bias        fp32 [E] added to the scores for the choice only, or NULL.
 *   score       a ternary_score: p = softmax over the row, or 1 / (1 + exp(-l)).
 *   groups      experts fall into `groups` runs of E / groups (E % groups == 0, at
 *               most TERNARY_MAX_EXPERT_GROUPS); only experts of the `top_groups`
 *               best groups may be chosen, a group's worth being the sum of its
 *               two largest p + bias (its only one, if it has one).
 *   top_k       1 <= top_k <= min(TERNARY_MAX_TOP_K, top_groups * E / groups).
 *   renormalize nonzero: a token's weights are divided by their sum.
 *   scale       multiplies the weights at the end.
 *   ids, weights  int32 and fp32 [T, top_k] outputs: the experts with the largest
 *               p + bias, largest first, ties to the lower index, and their p
 *               (renormalised, scaled).
 *   order       int32 [T * top_k] output: the slots t * top_k + j that hold an expert,
 *               sorted by it (those of one expert ascending); -1 from
 *               offsets[E] on.
 *   offsets     int32 [E + 1] output: expert e's slots are order[offsets[e]] up to
 *               order[offsets[e + 1] - 1].
 *   slots       int32 [T, top_k] output: a slot's place in `order`, -1 if it
 *               holds no expert.
 *   workspace   device memory of ternary_route_workspace(T, E) bytes, 16-byte
 *               aligned (NULL where that is 0).  It is written before it is
 *               read and may be reused once the call's work is done.
 * An expert whose logit or bias is -inf or NaN in a row cannot be chosen there
 * and has p = 0; a logit of +inf counts as the largest finite fp32 number.  A slot for which no
 * expert is left (a padded token's row of -inf) gets id -1 and weight 0; a sum
 * of weights of 0 is not divided by.  Scores are computed in 64 bits, so that the choice
 * is the exact one but for scores that agree to about 1e-15.
 */
int ternary_route(const void *logits, int dtype, int64_t T, int64_t E, const float *bias,
                  int score, int groups, int top_groups, int top_k, int renormalize, float scale,
                  int32_t *ids, float *weights, int32_t *offsets, int32_t *order, int32_t *slots,
                  void *workspace, hipStream_t stream);

/* Bytes of ternary_route's workspace (0 for few tokens), or TERNARY_ERR_SHAPE. */
int64_t ternary_route_workspace(int64_t T, int64_t E);

/* Which row of x a sorted slot of ternary_linear_experts multiplies. */
typedef enum {
    TERNARY_ROWS_TOKENS = 0,  /* row order[r] / top_k: x holds the tokens      */
    TERNARY_ROWS_SORTED = 1   /* row r: x holds the sorted slots themselves   */
} ternary_rows;

/*
 * ternary_linear_experts - for each place r < offsets[E], of expert e,
 *     y[r, n] = sum_k x[row(r), k] * q_e[n, k] * s_e(n, k)
 * with 8-bit activations and the experts' weights as tiled ternary codes.
 *   x, x_scale  e4m3 [x_rows, Kp] and fp32 [x_rows, Kp/128], Kp = K rounded up to a
 *               multiple of 128 (what ternary_fp8_quantize writes).
 *   x_rows      rows of x: at least 1; with TERNARY_ROWS_SORTED at least R.
 *   tiled       uint8 [E, ternary_tiled_bytes(N, K)]: each expert's tiled codes.
 *   scale       fp16 [E, N] or [E, N, K/group_size].
 *   E, N, K     as for ternary_route and ternary_linear; K up to 2^20.
 *   group_size  -1 (per output channel), 128 or 256.
 *   offsets, order  of ternary_route (order is read with TERNARY_ROWS_TOKENS only,
 *               and may be NULL otherwise).
 *   R           places in `order` (T * top_k), up to 2^30.  Places past offsets[E] are
 *               left as they were in y.
 *   top_k       slots of a token, 1 .. TERNARY_MAX_TOP_K (TERNARY_ROWS_TOKENS).
 *   y           [R, N] output, dtype `dtype` (TERNARY_BF16, TERNARY_FP16 or
 *               TERNARY_FP32), 16-byte aligned; must not overlap any input.
 * x and tiled 16-byte, x_scale, offsets and order 4-byte, scale 2-byte aligned.  For each block
 * of 128 along K the products are exact and summed in fp32 (as by ternary_fp8_linear, for every
 * dtype); sums of blocks are multiplied by their scales and added in fp32, in an order that depends on
 * the sizes alone, and y is rounded once.  `offsets` must ascend from 0 to at most R and
 * `order` name rows of x: entries that do not are not followed (no memory outside the
 * arguments is touched), the outputs that they concern are unspecified.
 */
int ternary_linear_experts(const uint8_t *x, const float *x_scale, int64_t x_rows,
                           const uint8_t *tiled, const uint16_t *scale, int64_t E, int64_t N,
                           int64_t K, int64_t group_size, const int32_t *offsets,
                           const int32_t *order, int64_t R, int top_k, int rows, void *y,
                           int dtype, hipStream_t stream);

/*
 * ternary_combine - the weighted sum of a token's expert rows:
 *     out[t, n] = add[t, n] + sum_j weights[t, j] * y[slots[t, j], n]
 *   y        [R, N], dtype `dtype` (TERNARY_BF16, TERNARY_FP16, TERNARY_FP32).
 *   weights, slots  fp32 and int32 [T, top_k] (ternary_route); a slot outside
 *            [0, R) adds nothing (its row is not read).
 *   add      [T, N] of the same dtype (a shared expert's output, the residual), or
 *            NULL for none; may be `out` itself.
 *   out      [T, N] output of the same dtype; must not overlap the other inputs.
 * All pointers aligned to their elements' size.  Sums in fp32, add first, then j ascending, rounded once.
 * 0 <= T <= 2^24, 0 <= N <= 2^24, R < 2^31, 1 <= top_k <= TERNARY_MAX_TOP_K.
 */
int ternary_combine(const void *y, int dtype, int64_t R, int64_t N, const int32_t *slots,
                    const float *weights, int64_t T, int top_k, const void *add, void *out,
                    hipStream_t stream);

/*
 * ---------------------------------------------------------------------------
 * Training beside frozen ternary weights, and many adapters at once.  Slots sorted by given indices (another
 * router's experts, or each token's adapter), rows sent to their places and the gradients
 * of that exchange, and low-rank adapters beside a shared projection with their gradients:
 *
 *   ids -> ternary_sort_slots -> offsets, order, slots
 *   x   -> ternary_dispatch -> the experts -> ternary_combine, and back:
 *          ternary_combine_backward -> the experts' gradients -> ternary_dispatch_backward
 *   y = x W^T -> ternary_linear_adapters (add = y) -> ternary_linear_adapters_backward
 *
 * The conventions above hold; none of these uses a workspace of the library, so any of them
 * may be captured, replayed and run on several streams at once (each call with a workspace of its own).
 * `offsets` must ascend from 0 to at most the number of slots, `order` and `slots` be each other's inverse: entries that
 * name no row or place are not followed (no memory outside the arguments is touched), the outputs that
 * they concern are unspecified.
 * ---------------------------------------------------------------------------
 */

/* Largest rank of an adapter. */
#define TERNARY_MAX_RANK 128

/*
 * ternary_sort_slots - the token slots sorted by given indices.
 *   ids       int32 [T, top_k]: the expert (or adapter) of each slot; outside [0, E): none.  A token may name one
 *             more than once.
 *   T, E      0 <= T <= 2^24, 1 <= E <= TERNARY_MAX_EXPERTS, 1 <= top_k <= TERNARY_MAX_TOP_K,
 *             T * top_k < 2^31.
 *   ones      fp32 [T, top_k] output of 1 (weights for ternary_combine), or NULL.
 *   offsets, order, slots  outputs as of ternary_route: order holds the slots t * top_k + j by expert, those of one
 *             ascending, -1 from offsets[E] on; slots each slot's place, -1 if it has none.
 *   workspace device memory of ternary_sort_slots_workspace(T, top_k, E) bytes, 16-byte
 *             aligned (NULL where that is 0), written before it is read.
 * All pointers 4-byte aligned; no output may overlap ids or another.
 */
int ternary_sort_slots(const int32_t *ids, int64_t T, int top_k, int64_t E, float *ones, int32_t *offsets,
                       int32_t *order, int32_t *slots, void *workspace, hipStream_t stream);

/* Bytes of its workspace (0 for few slots), or TERNARY_ERR_SHAPE. */
int64_t ternary_sort_slots_workspace(int64_t T, int top_k, int64_t E);

/*
 * ternary_dispatch - each token's row at the places of its slots:
 *     out[slots[t, j], n] = weights[t, j] * x[t, n]
 *   x        [T, N], dtype `dtype` (TERNARY_BF16, TERNARY_FP16, TERNARY_FP32).
 *   slots    int32 [T, top_k]; a slot outside [0, R) is left out.
 *   weights  fp32 [T, top_k], or NULL: rows are copied.
 *   out      [R, N] of the same dtype; must not overlap an input.  Rows that no slot names are left as they were.
 * Pointers aligned to their elements' size.  One fp32 product, rounded once.  0 <= T, N <= 2^24, 0 <= R < 2^31,
 * T * top_k < 2^31, T * N and R * N up to 2^38 (for the two functions below as well).
 */
int ternary_dispatch(const void *x, int dtype, int64_t T, int64_t N, const int32_t *slots, const float *weights,
                     int top_k, int64_t R, void *out, hipStream_t stream);

/*
 * ternary_dispatch_backward - gradient of ternary_dispatch:
 *     dx[t, n] = add[t, n] + sum_j weights[t, j] * grad[slots[t, j], n]
 *     dweights[t, j] = sum_n x[t, n] * grad[slots[t, j], n]
 *   grad     [R, N], dtype `dtype`; rows that no slot names are not read.
 *   weights, x, dweights  those of the forward call and an fp32 [T, top_k] output, or NULL all three
 *            (an unweighted dispatch: weights of 1).  A slot without a place has dweights 0.
 *   add      [T, N] (another gradient of x), or NULL; may be dx itself.
 *   dx       [T, N] output; must not overlap the other inputs.
 * Sums in fp32: dx add first, then j ascending, rounded once; dweights in an order that depends on N alone.
 */
int ternary_dispatch_backward(const void *grad, int dtype, int64_t R, int64_t N, const int32_t *slots,
                              const float *weights, int64_t T, int top_k, const void *x, const void *add, void *dx,
                              float *dweights, hipStream_t stream);

/*
 * ternary_combine_backward - gradient of ternary_combine (that of its `add` is grad itself):
 *     dy[slots[t, j], n] = weights[t, j] * grad[t, n]
 *     dweights[t, j] = sum_n y[slots[t, j], n] * grad[t, n]
 *   grad     [T, N], y and dy [R, N], dtype `dtype`; rows of y that no slot names are not read, those of dy left as
 *            they were.  dweights fp32 [T, top_k], 0 for a slot without a place.
 * No output may overlap an input or the other output.
 */
int ternary_combine_backward(const void *grad, const void *y, int dtype, int64_t R, int64_t N, const int32_t *slots,
                             const float *weights, int64_t T, int top_k, void *dy, float *dweights, hipStream_t stream);

/*
 * ternary_linear_adapters - low-rank adapters beside a projection, each token with its own:
 *     y[t] = add[t] + scale[e] * (x[t] a_e^T) b_e^T,  e the adapter of token t
 *   x          [T, K], dtype `dtype` (TERNARY_BF16 or TERNARY_FP16), as are a, b, add and y.
 *   a, b       [E, rank, K] and [E, N, rank]; an adapter of a smaller rank is filled up with zeros.
 *   T, K, N    0 <= T <= 2^24, 1 <= K, N <= 2^24, T * K and T * N up to 2^38; T == 0 is a successful no-op.
 *   rank, E    1 <= rank <= TERNARY_MAX_RANK, 1 <= E <= TERNARY_MAX_EXPERTS, E * (K + N) up to 2^28.
 *   scale      fp32 [E], or NULL for 1.
 *   offsets, order, slots  of ternary_sort_slots with top_k = 1.
 *   add        [T, N] (the projection's output), or NULL for none; may be y itself.
 *   y          [T, N] output.  A token without an adapter gets add, or 0.
 *   hidden     fp32 [T, rank] output x[t] a_e^T for the gradient, 16-byte aligned, or NULL; rows of tokens without an
 *              adapter are left as they were.
 *   workspace  device memory of ternary_linear_adapters_workspace() bytes, 16-byte aligned (NULL where that is 0), written
 *              before it is read.
 * The other pointers aligned to their elements' size; no output may overlap an input (but add) or another.
 * Products are exact and their sums fp32, in an order that depends on the sizes alone; x a^T enters the second
 * product as two 16-bit numbers, within 2^-16 of it (bf16; fp16: 2^-22 of the row's largest); y is rounded once.
 * What one token holds (an infinity, a NaN) reaches that token's outputs only.
 */
int ternary_linear_adapters(const void *x, int dtype, int64_t T, int64_t K, int64_t N, int64_t rank, const void *a,
                            const void *b, int64_t E, const float *scale, const int32_t *offsets,
                            const int32_t *order, const int32_t *slots, const void *add, void *y, float *hidden,
                            void *workspace, hipStream_t stream);

/* Bytes of its workspace (0 for few tokens of small rank), or TERNARY_ERR_SHAPE. */
int64_t ternary_linear_adapters_workspace(int64_t T, int64_t K, int64_t N, int64_t rank, int64_t E);

/*
 * ternary_linear_adapters_backward - its gradients, from grad [T, N], that of y (which is add's own as well):
 *     dv[t] = scale[e] * grad[t] b_e,   dx[t] = add[t] + dv[t] a_e
 *     da[e] = sum dv[t]^T x[t],         db[e] = scale[e] * sum grad[t]^T hidden[t],  over the adapter's tokens
 *   hidden    fp32 [T, rank] as the forward call wrote it, 16-byte aligned.
 *   add       [T, K] (another gradient of x), or NULL; may be dx itself.
 *   dx        [T, K] output.  A token without an adapter gets add, or 0.
 *   da, db    [E, rank, K] and [E, N, rank] outputs, 16-byte aligned; 0 for an adapter without tokens (with T == 0: all).
 *   workspace device memory of ternary_linear_adapters_backward_workspace() bytes, 16-byte aligned.
 * dv and hidden enter their second products as two 16-bit numbers as above (fp16, in da and db: 2^-22 of the
 * largest of some of the adapter's tokens); every output is rounded once.  The rest as above.
 */
int ternary_linear_adapters_backward(const void *grad, const void *x, const float *hidden, int dtype, int64_t T,
                                     int64_t K, int64_t N, int64_t rank, const void *a, const void *b, int64_t E,
                                     const float *scale, const int32_t *offsets, const int32_t *order,
                                     const int32_t *slots, const void *add, void *dx, void *da, void *db,
                                     void *workspace, hipStream_t stream);

/* Bytes of its workspace, or TERNARY_ERR_SHAPE. */
int64_t ternary_linear_adapters_backward_workspace(int64_t T, int64_t K, int64_t N, int64_t rank, int64_t E);

#ifdef __cplusplus
}
#endif

#endif /* TERNARY_LINEAR_H */
