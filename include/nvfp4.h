/*
 * nvfp4.h -- C ABI of libnvfp4.so: NVFP4 quantization and block-scaled FP4 GEMMs for the
 * three training GEMMs of a linear layer, on NVIDIA B200 (sm_100a).
 *
 * Method (page title, section):
 *   [P1] "Pretraining Large Language Models with NVFP4" (gist.science summary), Resumen
 *        tecnico, section 2 "Metodologia Propuesta":
 *          - "Formato NVFP4": 4-bit E2M1 elements in blocks of 16, an E4M3 scale per block
 *            and an FP32 scale per tensor (two-level scaling); native on Blackwell tensor
 *            cores.
 *          - "Transformadas de Hadamard Aleatorias (RHT)": a 16x16 Hadamard transform with
 *            a fixed random sign vector on the inputs of the weight-gradient GEMM.
 *          - "Escalado Bidimensional (2D) y Redondeo Estocastico": weights scaled in 16x16
 *            blocks so the forward and backward GEMMs use the same quantized weights;
 *            stochastic rounding for gradients only.
 *   [P3] news.hamidun.com, "Como Funciona": 16x16 random Hadamard transforms on gradient
 *        inputs and stochastic rounding.
 *
 * The arithmetic each call performs (the pages fix the ingredients, not the formulas):
 *   amax   = max |y| over the tensor, y = x or its random Hadamard transform
 *   S_enc  = 2688 / amax (= 6 * 448 / amax, FP32 division); 1 if amax == 0; FLT_MAX if the
 *            quotient overflows
 *   sf     = E4M3(round-to-nearest-even, saturating)((b / 6) * S_enc), b = block max |y|
 *            (1x16 block, or the 16x16 tile for 2D weight scaling)
 *   r      = S_enc / float(sf), clamped to FLT_MAX; r = 0 when sf == 0
 *   code   = E2M1(y * r): round-to-nearest-even (RTN) or stochastic rounding (SR), sign
 *            kept, magnitudes saturate at 6
 *   SR     : round the magnitude up iff float(r16) < p * 65536, p = (|v| - lo) / (hi - lo);
 *            r16 = 16-bit lane (e & 7) of Philox-4x32-10 with key = seed and
 *            counter = (e >> 3, offset), e = element index r * cols + c of the quantized
 *            (logical) matrix
 *   RHT    : per 16 consecutive elements along the reduction axis, y = (1/4) H diag(s) x,
 *            H the Sylvester Hadamard matrix, s_i = -1 iff bit i of sign_mask is set,
 *            applied as FP32 butterflies of widths 1, 2, 4, 8
 *   GEMM   : D[m, n] = sum_k e2m1(A[m,k]) sf_A e2m1(B[n,k]) sf_B / (S_enc,A S_enc,B),
 *            FP32 accumulation
 *
 * Conventions for every call:
 *   - Ownership: the caller allocates every buffer (device memory unless stated) and keeps
 *     it alive until the work queued on `stream` has finished.  The library never
 *     allocates, frees or synchronizes; all GPU work is queued on `stream` (a cudaStream_t;
 *     NULL is the legacy default stream) of the current device.
 *   - Errors: invalid arguments return a status synchronously and queue no work.  Errors
 *     that depend on the data (a NaN or Inf in a quantizer input, a GEMM pipeline wait that
 *     ran out of time) are OR-ed as NVFP4_DEVSTAT_* bits into *dev_status (a device int,
 *     may be NULL), which the caller reads when it chooses; on non-finite input the codes
 *     and scales are zero and the amax is +Inf.
 *   - Alignment: every device pointer must be 16-byte aligned (TMA).
 *   - Devices: only compute capability 10.0 (B200) is accepted (NVFP4_ERR_DEVICE).
 *   - Determinism: results are a pure function of the inputs, flags, seed, offset and
 *     sign mask, bitwise reproducible from run to run.
 */
#ifndef NVFP4_H
#define NVFP4_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    NVFP4_OK = 0,
    NVFP4_ERR_NULL = 1,      /* a required pointer is NULL                                */
    NVFP4_ERR_SHAPE = 2,     /* a size violates the shape rules of the call              */
    NVFP4_ERR_ALIGN = 3,     /* a pointer or leading dimension is misaligned             */
    NVFP4_ERR_DEVICE = 4,    /* the current device is not an sm_100 GPU                  */
    NVFP4_ERR_CUDA = 5,      /* a CUDA runtime or driver call failed                     */
    NVFP4_ERR_NONFINITE = 6, /* (host-side helpers only) non-finite data                 */
    NVFP4_ERR_TIMEOUT = 7,   /* (host-side helpers only) a device wait timed out         */
    NVFP4_ERR_ARG = 8        /* an invalid flag combination or enum value                */
} nvfp4_status;

/* Bits OR-ed into *dev_status by the kernels. */
enum {
    NVFP4_DEVSTAT_NONFINITE = 1, /* a quantizer input (or its transform) held NaN/Inf     */
    NVFP4_DEVSTAT_TIMEOUT = 2,   /* a GEMM pipeline wait exceeded its time limit; the
                                    output of that GEMM is undefined                     */
    NVFP4_DEVSTAT_BOUNDS = 4,    /* (debug build only, see nvfp4_bounds_checked) a kernel
                                    computed a global access outside its buffer and
                                    skipped it; the outputs of that call are undefined   */
    NVFP4_DEVSTAT_INDEX = 8      /* a routing named an expert outside [-1, E); the pair was
                                    treated as having no expert                          */
};

/* Quantizer flags. */
enum {
    NVFP4_ROWWISE = 1,    /* produce out_row: x quantized along its columns (K = cols)   */
    NVFP4_COLWISE = 2,    /* produce out_col: x^T quantized along x's rows (K = rows)    */
    NVFP4_BLOCK2D = 4,    /* one scale per 16x16 tile (weights); RTN only                */
    NVFP4_SR = 8,         /* stochastic rounding (gradients)                             */
    NVFP4_AMAX_GIVEN = 16,/* skip the amax pass: read the tensor amax from the output
                             operand's `amax` (out_row's if present, else out_col's); the
                             data must then be finite                                    */
    NVFP4_MX = 32,        /* MXFP4 instead of NVFP4 (see below); not with NVFP4_BLOCK2D  */
    NVFP4_GATHER = 64     /* nvfp4_quantize_grouped only: x has a row per token          */
};

/* MXFP4, the comparison format of [P1 Formato NVFP4; Nuevo Formato NVFP4] (OCP MX):
 * E2M1 codes in blocks of 32 along K sharing one power-of-two scale X = 2^E, E =
 * floor(log2 b) - 2 for the block's largest magnitude b (clamped to [-127, 127]; -127 for a
 * zero block), stored as the E8M0 byte E + 127; elements E2M1(v / X) rounded to nearest even
 * (or stochastically with NVFP4_SR), saturating at 6; no tensor scale.  An MXFP4 operand has
 * the NVFP4 operand's layout: each 32-block's E8M0 byte fills both of its 16-element scale
 * slots, and `amax` holds the tensor amax only to flag non-finite data.  Multiply MXFP4
 * operands with nvfp4_gemm_mx. */

/* GEMM output types. */
enum { NVFP4_OUT_F32 = 0, NVFP4_OUT_BF16 = 1 };

/* A quantized operand, quantized along `cols` (its GEMM reduction axis K).
 *   codes  : rows * cols / 2 bytes, row-major, two E2M1 codes per byte, the even column in
 *            the low nibble.
 *   scales : nvfp4_scales_bytes(rows, cols) bytes of E4M3 block scales in the layout the
 *            tensor-core MMA reads: tiles of 128 rows x 4 blocks (512 bytes), tiles
 *            ordered by (row tile, block group) with the block groups of one row tile
 *            contiguous; inside a tile, the scale of (row r, block j) is at byte
 *            (r % 32) * 16 + ((r / 32) % 4) * 4 + (j % 4).  Rows beyond `rows` (padding to
 *            a multiple of 128) hold zeros.  nvfp4_scales_unswizzle() undoes the layout.
 *   amax   : one FP32, the amax the scales were derived from.
 * All three are device pointers. */
typedef struct {
    void* codes;
    void* scales;
    float* amax;
    int64_t rows;
    int64_t cols;
} nvfp4_operand;

/* Library version (major * 100 + minor). */
int nvfp4_version(void);

/* Human-readable name of a status. */
const char* nvfp4_status_string(nvfp4_status status);

/* Sizes in bytes of the codes and of the (padded) scale buffer of a rows x cols operand
 * quantized along cols.  Return 0 for invalid sizes. */
size_t nvfp4_codes_bytes(int64_t rows, int64_t cols);
size_t nvfp4_scales_bytes(int64_t rows, int64_t cols);

/* Device workspace needed by nvfp4_quantize / nvfp4_rht_quantize / nvfp4_quantize_row_rht
 * for a rows x cols input (the per-block partial maxima of the amax pass).  0 with
 * NVFP4_AMAX_GIVEN. */
size_t nvfp4_workspace_bytes(int64_t rows, int64_t cols, unsigned flags);

/* Device workspace needed by each nvfp4_linear_* call for T tokens, I in-features and O
 * out-features (the quantized operands plus the amax pass). */
size_t nvfp4_linear_workspace_bytes(int64_t T, int64_t I, int64_t O);

/* Host helper: the RHT sign mask drawn from a seed -- the low 16 bits of word 0 of
 * Philox-4x32-10 with key = seed and counter = (0, 0, 0, 0xFFFFFFFF).  [P1 RHT]: one random
 * sign vector, fixed for the whole of training. */
uint16_t nvfp4_sign_mask_from_seed(uint64_t seed);

/* Host helper: rewrite a scale buffer from the MMA layout described at nvfp4_operand into
 * plain row-major [rows x cols/16] bytes.  Both buffers are HOST memory. */
nvfp4_status nvfp4_scales_unswizzle(const void* swizzled, int64_t rows, int64_t cols,
                                    void* row_major);

/*
 * Quantize a bf16 matrix x (rows x cols, row stride ld elements, device) to NVFP4.
 * [P1 Formato NVFP4, Escalado 2D y Redondeo Estocastico].
 *   flags    : NVFP4_ROWWISE and/or NVFP4_COLWISE select the outputs; NVFP4_BLOCK2D gives
 *              one scale per 16x16 tile, so out_col's codes are exactly out_row's codes
 *              transposed; NVFP4_SR rounds stochastically; NVFP4_AMAX_GIVEN skips the
 *              amax pass.
 *   seed, offset : Philox key and stream for NVFP4_SR (ignored otherwise).
 *   out_row  : rows x cols operand (K = cols); required iff NVFP4_ROWWISE.
 *   out_col  : cols x rows operand (x^T, K = rows); required iff NVFP4_COLWISE.  Both
 *              outputs share one amax (both amax pointers are written).
 *   workspace: nvfp4_workspace_bytes(rows, cols, flags) device bytes (NULL if 0).
 * Shape rules: rows, cols >= 1 and multiples of 16; ld >= cols and a multiple of 8;
 * cols a multiple of 64 for out_row; rows a multiple of 64 for out_col.
 * Two passes over x: the amax, then the scales and codes.
 */
nvfp4_status nvfp4_quantize(const void* x_bf16, int64_t rows, int64_t cols, int64_t ld,
                            unsigned flags, uint64_t seed, uint64_t offset,
                            const nvfp4_operand* out_row, const nvfp4_operand* out_col,
                            void* workspace, int* dev_status, void* stream);

/*
 * Random-Hadamard-transform and quantize x^T along x's rows: the weight-gradient operands.
 * [P1 RHT; P3 Como Funciona].  Each 16 consecutive rows of every column of x are
 * transformed (y = (1/4) H diag(s) x), then quantized along the same axis in 1x16 blocks.
 * The amax is that of the transformed tensor.
 *   sign_mask: bit i set = sign -1 for element i of each 16-block.
 *   flags    : NVFP4_SR, NVFP4_AMAX_GIVEN and/or NVFP4_MX (NVFP4_COLWISE is implied; other
 *              bits are rejected).
 *   out_col  : cols x rows operand (K = rows).
 * Shape rules: rows a multiple of 64, cols a multiple of 16, ld >= cols, ld % 8 == 0.
 */
nvfp4_status nvfp4_rht_quantize(const void* x_bf16, int64_t rows, int64_t cols, int64_t ld,
                                uint16_t sign_mask, unsigned flags, uint64_t seed,
                                uint64_t offset, const nvfp4_operand* out_col,
                                void* workspace, int* dev_status, void* stream);

/*
 * Both quantizations a linear layer needs of one activation or output gradient x (T x C:
 * tokens x features), from one amax pass and one quantize pass over x.  [P1 Formato NVFP4;
 * RHT; Escalado 2D y Redondeo Estocastico]: x feeds the forward (or data-gradient) GEMM
 * quantized along its features, and the weight-gradient GEMM random-Hadamard-transformed and
 * quantized along its tokens.
 *   out_row  : rows x cols operand, exactly what nvfp4_quantize(x, NVFP4_ROWWISE | (flags &
 *              NVFP4_SR), seed, offset) writes (amax = max |x|).
 *   out_col  : cols x rows operand, exactly what nvfp4_rht_quantize(x, sign_mask, flags, seed,
 *              offset + 1) writes (amax = max |RHT(x)|): the two SR streams are offset and
 *              offset + 1, as for the data- and weight-gradient operands of one dY.
 *   flags    : NVFP4_SR and/or NVFP4_AMAX_GIVEN (both amaxes are then read from out_row->amax
 *              and out_col->amax); other bits are rejected with NVFP4_ERR_ARG.
 *   workspace: nvfp4_workspace_bytes(rows, cols, flags) device bytes (NULL if 0).
 * Shape rules: rows and cols multiples of 64, ld >= cols, ld % 8 == 0.  Each output is
 * zero-filled on its own when its amax is not finite (NVFP4_DEVSTAT_NONFINITE is set).
 */
nvfp4_status nvfp4_quantize_row_rht(const void* x_bf16, int64_t rows, int64_t cols, int64_t ld,
                                    uint16_t sign_mask, unsigned flags, uint64_t seed,
                                    uint64_t offset, const nvfp4_operand* out_row,
                                    const nvfp4_operand* out_col, void* workspace,
                                    int* dev_status, void* stream);

/*
 * nvfp4_gemm with bf16 output that also emits the two maxima the next quantization of D needs.
 * The recipe's tensor scales come from the amax of the quantized tensor [P1 Formato NVFP4],
 * and a layer's output D is the next layer's input (or, from dgrad, the previous layer's
 * output gradient), quantized row-wise and RHT'd column-wise [P1 RHT].
 *   amax_out : device, 2 FP32 (4-byte aligned), overwritten: amax_out[0] = max |D| and
 *              amax_out[1] = max |RHT(D)| (16x16 transform of every 16 consecutive rows of each
 *              column with sign_mask), both over D as stored in bf16 -- exactly the amax values
 *              nvfp4_quantize_row_rht(D, sign_mask) computes.  NaN or Inf in D makes the
 *              maximum +Inf or a NaN (the maxima are taken on the magnitude bit patterns), which
 *              the quantizer then treats as non-finite data: zero outputs and
 *              NVFP4_DEVSTAT_NONFINITE, as without the fused maxima.
 * Pass them to nvfp4_quantize_row_rht with NVFP4_AMAX_GIVEN (out_row->amax = &amax_out[0],
 * out_col->amax = &amax_out[1]) to skip its amax pass.  Other arguments as nvfp4_gemm.
 */
nvfp4_status nvfp4_gemm_amax(const nvfp4_operand* A, const nvfp4_operand* B, void* D_bf16,
                             int64_t ldd, uint16_t sign_mask, float* amax_out, int* dev_status,
                             void* stream);

/*
 * Self-test of the device-side bounded waits (no counterpart on the pages): queues one kernel
 * whose thread waits, with the GEMM's own wait routine, on an mbarrier that nothing completes.
 * After 50 ms the wait gives up, NVFP4_DEVSTAT_TIMEOUT is OR-ed into *dev_status (device,
 * 4-byte aligned) and the kernel returns; the context stays usable.  This is how the GEMM's
 * waits end if a copy or an MMA never signals, without hanging the GPU.
 */
nvfp4_status nvfp4_selftest_wait_timeout(int* dev_status, void* stream);

/*
 * Debug build (no counterpart on the pages).  The same sources compiled with
 * -DNVFP4_BOUNDS_CHECK give libnvfp4_checked.so, with this header's API unchanged: every
 * global load and store of the quantizers, the router, the expert plan and the combination is
 * checked against the extent of its buffer (the input's rows x ld values, the codes' rows x cols
 * / 2 bytes, the scales' padded size, the plan's arrays), and every TMA box the GEMM issues against the TMA start rules (non-negative coordinates, a
 * 16-byte aligned innermost start).  An access outside is skipped and NVFP4_DEVSTAT_BOUNDS is
 * OR-ed into *dev_status; the call's outputs are then undefined.  Such a build is slower and
 * meant for tests.
 *
 * nvfp4_bounds_checked returns 1 in that build and 0 in the normal one.
 *
 * nvfp4_selftest_bounds (checked build only; the normal one returns NVFP4_ERR_ARG and queues
 * nothing): queues one kernel whose thread stores one word through the checked-store routine
 * just past the end of a 16-byte buffer the routine is told about (the word itself lies inside
 * a larger array the library owns, so nothing outside the library's memory is named).  The
 * check refuses the store and sets NVFP4_DEVSTAT_BOUNDS in *dev_status (device, 4-byte
 * aligned); the context stays usable.
 */
int nvfp4_bounds_checked(void);
nvfp4_status nvfp4_selftest_bounds(int* dev_status, void* stream);

/*
 * nvfp4_gemm for two MXFP4 operands (quantized with NVFP4_MX): the same tensor-core GEMM
 * with E8M0 block scales and no tensor scales, D = A . B^T.  Arguments, shape rules and
 * errors as nvfp4_gemm.
 */
nvfp4_status nvfp4_gemm_mx(const nvfp4_operand* A, const nvfp4_operand* B, void* D, int d_dtype,
                           int64_t ldd, int* dev_status, void* stream);

/*
 * Block-scaled FP4 GEMM on the tcgen05 tensor cores: D = A . B^T.
 * [P1 Formato NVFP4: native NVFP4 support in Blackwell tensor cores].
 *   A : M x K operand, B : N x K operand (both quantized along K; A.cols == B.cols == K).
 *   D : device, M x N row-major with row stride ldd elements, FP32 or bf16 (d_dtype).
 *       D = FP32 accumulation of the block-scaled products, times 1 / (S_enc,A S_enc,B)
 *       computed from A.amax and B.amax on the device (0 if either amax is not finite).
 * Shape rules: K a multiple of 64; M, N multiples of 16; ldd >= N and ldd * element size
 * a multiple of 16 bytes.
 */
nvfp4_status nvfp4_gemm(const nvfp4_operand* A, const nvfp4_operand* B, void* D, int d_dtype,
                        int64_t ldd, int* dev_status, void* stream);

/*
 * The three training GEMMs of a linear layer y = x . W^T, each a self-contained call that
 * quantizes its bf16 inputs (row-major, contiguous) into `workspace`
 * (nvfp4_linear_workspace_bytes(T, I, O) device bytes) and multiplies them.
 * Shape rules: T, I, O multiples of 64.
 *
 * fprop: Y[T x O] = X[T x I] . W[O x I]^T; X 1x16 RTN, W 16x16 RTN.
 * dgrad: dX[T x I] = dY[T x O] . W; dY 1x16 SR (stream `offset`), W^T 16x16 RTN (the same
 *        quantized values as fprop's W [P1 Escalado 2D]).
 * wgrad: dW[O x I] = dY^T . X; dY^T RHT + SR (stream `offset + 1`), X^T RHT + RTN, both
 *        blocked along tokens [P1 RHT].
 * y_dtype / dx_dtype / dw_dtype: NVFP4_OUT_F32 or NVFP4_OUT_BF16.
 */
nvfp4_status nvfp4_linear_fprop(const void* X, const void* W, int64_t T, int64_t I, int64_t O,
                                void* Y, int y_dtype, void* workspace, int* dev_status,
                                void* stream);
nvfp4_status nvfp4_linear_dgrad(const void* dY, const void* W, int64_t T, int64_t I, int64_t O,
                                uint64_t seed, uint64_t offset, void* dX, int dx_dtype,
                                void* workspace, int* dev_status, void* stream);
nvfp4_status nvfp4_linear_wgrad(const void* dY, const void* X, int64_t T, int64_t I, int64_t O,
                                uint16_t sign_mask, uint64_t seed, uint64_t offset, void* dW,
                                int dw_dtype, void* workspace, int* dev_status, void* stream);

/*
 * nvfp4_linear_dgrad with bf16 output, also quantized for the previous layer's backward pass:
 * dX = dY . W and dX's two NVFP4 operands, the ones the previous layer's dgrad and wgrad read
 * (dX is that layer's output gradient) [P1 Escalado 2D y Redondeo Estocastico; P1 RHT]:
 *   dX_row : T x I along I, 1x16 SR on stream next_offset;
 *   dX_col : I x T along T, RHT + 1x16 SR on stream next_offset + 1;
 * bit for bit what nvfp4_linear_dgrad(..., NVFP4_OUT_BF16) followed by
 * nvfp4_quantize_row_rht(dX, sign_mask, NVFP4_SR, next_seed, next_offset) writes, including
 * each operand's amax.  The GEMM epilogue emits dX's two maxima (nvfp4_gemm_amax), so dX is
 * quantized without an amax pass.
 *   dX_bf16   : device, T x I bf16, row stride I.
 *   dX_row, dX_col : the caller's operands (shapes as above); checked before any work is
 *               queued, like every other argument.
 *   workspace : nvfp4_linear_workspace_bytes(T, I, O) device bytes.
 * Shape rules: T, I, O multiples of 64.
 */
nvfp4_status nvfp4_linear_dgrad_quantized(const void* dY, const void* W, int64_t T, int64_t I,
                                          int64_t O, uint64_t seed, uint64_t offset,
                                          void* dX_bf16, uint16_t sign_mask, uint64_t next_seed,
                                          uint64_t next_offset, const nvfp4_operand* dX_row,
                                          const nvfp4_operand* dX_col, void* workspace,
                                          int* dev_status, void* stream);

/*
 * nvfp4_quantize without a caller workspace, for callers that cannot allocate device memory
 * where they quantize (a host framework that owns all device memory through its own
 * fixed arena, or a latency-critical loop that must not enter cudaMalloc / cudaFree, which may
 * block or synchronize the device).  The pages have no counterpart to this call: it is a
 * deployment convenience of this library.
 *
 * Same arguments, rules and results as nvfp4_quantize, minus `workspace`: the partial maxima
 * of the amax pass live in a file-scope device array of NVFP4_NOALLOC_MAX_PARTIALS 32-bit slots
 * (8 KB per GPU that loads the library, held until the process exits).  The call allocates
 * nothing.  The first call on each device looks up the array's address and keeps it for the
 * life of the process; make that first call before any stream capture begins, and do not use
 * this entry point across a cudaDeviceReset (the kept address would belong to the destroyed
 * context).  Calls share the array: calls whose kernels overlap on the GPU (several streams or
 * host threads on one device) race and may give wrong results; calls queued on one stream are
 * ordered and safe.  A call whose amax pass would use more CTAs than the array has slots
 * returns NVFP4_ERR_SHAPE; the amax pass never launches more than 2048 CTAs, so no shape that
 * nvfp4_quantize accepts is rejected for this reason.  With NVFP4_AMAX_GIVEN there is no amax
 * pass and the array is not touched.
 */
#define NVFP4_NOALLOC_MAX_PARTIALS 2048
nvfp4_status nvfp4_quantize_noalloc(const void* x_bf16, int64_t rows, int64_t cols, int64_t ld,
                                    unsigned flags, uint64_t seed, uint64_t offset,
                                    const nvfp4_operand* out_row, const nvfp4_operand* out_col,
                                    int* dev_status, void* stream);

/*
 * ---- Mixture-of-experts layers ---------------------------------------------------------
 * A layer with E experts whose weights are E matrices W_e [O x I]; every token is multiplied by
 * those of its k experts.  The pages have no counterpart to these calls: they carry the recipe's
 * quantization and GEMMs of a linear layer over to a layer of experts.
 *
 *   nvfp4_route -> nvfp4_plan_experts -> nvfp4_experts_fprop (up, gathering the tokens) ->
 *   activation -> nvfp4_experts_fprop (down) -> nvfp4_combine
 *   and back: nvfp4_combine_backward -> nvfp4_experts_{dgrad,wgrad} (down) -> activation's
 *   gradient -> nvfp4_experts_{dgrad,wgrad} (up) -> nvfp4_combine without weights (the gradient
 *   of the gather), nvfp4_route_backward
 *
 * Expert order.  A pair is (token t, slot j), its index t * k + j.  An expert-ordered matrix has
 * `rows` rows; expert e owns the region offsets[e] .. offsets[e + 1], whose length is the number of
 * its pairs rounded up to a multiple of 128: one row per pair in the order of the pairs' indices,
 * then rows without a token, which count as zeros.  Rows behind offsets[E] are neither read nor
 * written by any call here.
 * All sizes that depend on the routing stay on the device: every call may be captured in a graph
 * and replayed for another routing.
 * The indices in a plan are checked where they are used (a token outside [0, tokens), a row beyond
 * `rows` count as absent), so that a plan of another routing gives wrong results but no access
 * outside the buffers.
 */
enum { NVFP4_SCORE_SOFTMAX = 0, NVFP4_SCORE_SIGMOID = 1 };

/* The expert-ordered rows of a routing of `tokens` tokens to k of `experts` experts each.  Device
 * pointers (4-byte aligned), written by nvfp4_plan_experts:
 *   offsets   : experts + 1 int32, the regions
 *   pair_row  : tokens * k int32, the row of every pair (-1: the pair has no expert)
 *   row_token : rows int32, the token of every row (-1: none)
 * Limits: tokens >= 1, 1 <= k <= 32, 1 <= experts <= 512, tokens * k < 2^31; rows a multiple of
 * 128, at least nvfp4_expert_rows(tokens, k, experts) and at most 8388480. */
typedef struct {
    int32_t* offsets;
    int32_t* pair_row;
    int32_t* row_token;
    int64_t tokens;
    int64_t k;
    int64_t experts;
    int64_t rows;
} nvfp4_expert_plan;

/* Rows that hold every routing of T tokens to k of E experts; 0 for sizes outside the limits. */
int64_t nvfp4_expert_rows(int64_t T, int64_t k, int64_t E);

/* Device workspace of nvfp4_plan_experts (0 for few pairs: no workspace is needed). */
size_t nvfp4_expert_plan_workspace_bytes(int64_t T, int64_t k, int64_t E);

/*
 * Experts and weights of every token from its router logits.
 *   logits  : T x E, FP32 or bf16 (dtype: NVFP4_OUT_F32 / NVFP4_OUT_BF16), row stride ld elements.
 *             -inf excludes an expert.  A row with NaN or +inf is routed nowhere (indices -1,
 *             weights 0) and sets NVFP4_DEVSTAT_NONFINITE.
 *   score   : NVFP4_SCORE_SOFTMAX over the E logits, or NVFP4_SCORE_SIGMOID of each.
 *   bias    : E FP32 added to the scores for the choice only (not to the weights), or NULL.  -inf
 *             excludes an expert; NaN and +inf are treated as in logits.
 *   groups, top_groups : with groups > 1 the experts form `groups` equal ranges, and only those in
 *             the top_groups ranges with the largest sum of their two best values (score + bias; of
 *             the one if only one is not excluded) are candidates.  groups <= 32.
 *   k       : experts per token, k <= E / groups * top_groups; chosen in falling order of score +
 *             bias.  Equal values go to the lower index.  With a bias or groups the choice is that of
 *             scores in FP64 (comparisons closer than FP32's error are decided there); with neither
 *             the logits themselves are compared, also where their scores are equal in FP64.
 *   experts : T x k int32 out; -1 where fewer than k experts can be chosen.
 *   weights : T x k FP32 out: scale * score, divided by the sum of the chosen scores with
 *             `renormalize`; 0 where the expert is -1.
 */
nvfp4_status nvfp4_route(const void* logits, int dtype, int64_t T, int64_t E, int64_t ld,
                         const float* bias, int score, int groups, int top_groups, int k,
                         int renormalize, float scale, int32_t* experts, float* weights,
                         int* dev_status, void* stream);

/*
 * Gradient of nvfp4_route's weights with respect to the logits (the choice itself has none).
 *   experts, dweights : T x k; pairs with expert -1 have no part.  An expert named twice counts
 *             twice.  Other indices outside [0, E) count as -1 and set NVFP4_DEVSTAT_INDEX.
 *   dlogits : T x E of the logits' type, row stride ldd, all written (zeros where no gradient
 *             arrives, and for rows without an expert).
 */
nvfp4_status nvfp4_route_backward(const void* logits, int dtype, int64_t T, int64_t E, int64_t ld,
                                  const int32_t* experts, const float* dweights, int score, int k,
                                  int renormalize, float scale, void* dlogits, int64_t ldd,
                                  int* dev_status, void* stream);

/*
 * The plan of a routing: fills plan->offsets, pair_row and row_token (all rows) from
 * experts (tokens x k).  Indices outside [-1, E) count as -1 and set NVFP4_DEVSTAT_INDEX; an
 * expert named twice by a token gets two rows.
 *   workspace : nvfp4_expert_plan_workspace_bytes(...) device bytes (NULL if 0).
 */
nvfp4_status nvfp4_plan_experts(const int32_t* experts, const nvfp4_expert_plan* plan,
                                void* workspace, int* dev_status, void* stream);

/*
 * Quantize an expert-ordered matrix (rows x cols) to NVFP4: what nvfp4_quantize(NVFP4_ROWWISE) and
 * nvfp4_rht_quantize give of it, in its regions; the amax is taken over them too.
 *   x       : bf16, row stride ld.  With NVFP4_GATHER a matrix with a row per token (tokens x
 *             cols): row r of the quantized matrix is x[row_token[r]].  Otherwise a matrix in
 *             expert order (rows x cols).  Rows of x that no pair takes are not looked at.
 *   flags   : NVFP4_ROWWISE (out_row, rows x cols) and/or NVFP4_COLWISE (out_col, cols x rows,
 *             random-Hadamard-transformed along the rows with sign_mask); NVFP4_SR,
 *             NVFP4_AMAX_GIVEN (each output's amax is read from it), NVFP4_GATHER.
 *   seed, offset : NVFP4_SR draws stream `offset` for out_row and `offset` + 1 for out_col, with the
 *             element indices of the rows x cols (cols x rows) matrix.
 *   workspace : nvfp4_workspace_bytes(rows, cols, flags) device bytes (NULL if 0).
 * Shape rules: cols a multiple of 64 (16 with NVFP4_COLWISE alone), ld >= cols, ld % 8 == 0.
 */
nvfp4_status nvfp4_quantize_grouped(const void* x_bf16, int64_t cols, int64_t ld,
                                    const nvfp4_expert_plan* plan, uint16_t sign_mask,
                                    unsigned flags, uint64_t seed, uint64_t offset,
                                    const nvfp4_operand* out_row, const nvfp4_operand* out_col,
                                    void* workspace, int* dev_status, void* stream);

/*
 * Every expert's rows times its matrix: D[r, :] = A[r, :] . B_e^T for the rows r of expert e.  Rows
 * behind the last region are not written; rows without a token are multiplied like the others and
 * give the zeros that nvfp4_quantize_grouped writes for them.
 *   A : rows x K operand in expert order.
 *   B : the E matrices B_e [N x K], stacked (an (E * N) x K operand; N a multiple of 128 if E > 1)
 *       or side by side (an N x (E * K) operand).  For a layer's weights W_e [O x I] stacked in one
 *       (E * O) x I matrix these are the row-wise output of nvfp4_quantize (forward) and its
 *       column-wise output (data gradient).
 *   D : device, rows x N, row stride ldd, FP32 or bf16.
 * Shape rules: K a multiple of 64, N of 16; ldd as in nvfp4_gemm.
 */
nvfp4_status nvfp4_gemm_grouped(const nvfp4_operand* A, const nvfp4_operand* B,
                                const nvfp4_expert_plan* plan, void* D, int d_dtype, int64_t ldd,
                                int* dev_status, void* stream);

/*
 * One product per expert along its rows: D_e = A[:, e's rows] . B[:, e's rows]^T, zeros for an
 * expert without pairs.
 *   A : M x rows operand, B : N x rows operand (column-wise outputs of nvfp4_quantize_grouped).
 *   D : device, (E * M) x N, row stride ldd, FP32 or bf16; D_e starts at row e * M.
 * Shape rules: M a multiple of 128, N of 16.
 */
nvfp4_status nvfp4_gemm_grouped_k(const nvfp4_operand* A, const nvfp4_operand* B,
                                  const nvfp4_expert_plan* plan, void* D, int d_dtype, int64_t ldd,
                                  int* dev_status, void* stream);

/* Device workspace of each nvfp4_experts_* call (rows: the plan's). */
size_t nvfp4_experts_workspace_bytes(int64_t T, int64_t k, int64_t E, int64_t rows, int64_t I,
                                     int64_t O);

/*
 * The three training GEMMs of a layer of experts, as nvfp4_linear_*, with the weights quantized
 * once by the caller: W is the (E * O) x I row-wise, Wt the I x (E * O) column-wise output of
 * nvfp4_quantize(NVFP4_BLOCK2D) of the stacked weights.
 *   fprop: Y[rows x O] = X . W_e^T; X 1x16 RTN, a row per token (gather != 0) or in expert order.
 *   dgrad: dX[rows x I] = dY . W_e; dY [rows x O] 1x16 SR (stream `offset`).
 *   wgrad: dW[(E * O) x I], dW_e = dY_e^T . X_e; dY RHT + SR (stream `offset` + 1), X RHT + RTN.
 * Shape rules: I a multiple of 64, O of 128, E * O < 2^31.
 */
nvfp4_status nvfp4_experts_fprop(const void* X, int64_t ldx, int gather, const nvfp4_operand* W,
                                 const nvfp4_expert_plan* plan, int64_t I, int64_t O, void* Y,
                                 int y_dtype, int64_t ldy, void* workspace, int* dev_status,
                                 void* stream);
nvfp4_status nvfp4_experts_dgrad(const void* dY, int64_t lddy, const nvfp4_operand* Wt,
                                 const nvfp4_expert_plan* plan, int64_t I, int64_t O, uint64_t seed,
                                 uint64_t offset, void* dX, int dx_dtype, int64_t lddx,
                                 void* workspace, int* dev_status, void* stream);
nvfp4_status nvfp4_experts_wgrad(const void* dY, int64_t lddy, const void* X, int64_t ldx, int gather,
                                 const nvfp4_expert_plan* plan, int64_t I, int64_t O,
                                 uint16_t sign_mask, uint64_t seed, uint64_t offset, void* dW,
                                 int dw_dtype, int64_t lddw, void* workspace, int* dev_status,
                                 void* stream);

/*
 * The rows of a layer of experts back to tokens: out[t] = sum_j weights[t, j] Y[pair_row[t, j]],
 * summed in FP32 in slot order (pairs without a row add nothing).  weights NULL: all 1, the
 * gradient of the gather.
 *   Y   : rows x cols bf16 in expert order, row stride ldy.
 *   out : tokens x cols FP32 or bf16, row stride ldo.
 * Shape rules: cols a multiple of 8; row strides multiples of 16 bytes.
 */
nvfp4_status nvfp4_combine(const void* Y_bf16, int64_t cols, int64_t ldy,
                           const nvfp4_expert_plan* plan, const float* weights, void* out,
                           int out_dtype, int64_t ldo, int* dev_status, void* stream);

/*
 * Gradients of nvfp4_combine: dY[pair_row[t, j]] = weights[t, j] dout[t] (zeros in the rows without a
 * token; rows behind the last region are not written) and dweights[t, j] = sum_c dout[t, c]
 * Y[pair_row[t, j], c] (0 for pairs without a row).  dout FP32 or bf16, Y and dY bf16.
 */
nvfp4_status nvfp4_combine_backward(const void* dout, int dout_dtype, int64_t ldo,
                                    const void* Y_bf16, int64_t cols, int64_t ldy,
                                    const nvfp4_expert_plan* plan, const float* weights,
                                    void* dY_bf16, int64_t lddy, float* dweights, int* dev_status,
                                    void* stream);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_H */
