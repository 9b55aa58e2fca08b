/*
 * iq.h -- C ABI of libiq, block-scaled low-precision quantization on MI355X.
 *
 * The method (Lorn blog, post "浅谈低精度浮点数", sections "FP8" and
 * "FP4 / MXFP4 / NVFP4"): a tensor x is represented as x^ = s * Q(x / s),
 * where s is a scale derived from an absolute maximum (per tensor, per row,
 * or per block along the contiguous dimension) and Q rounds onto a small
 * code grid.  One call reads x once and, in the same pass, derives the
 * scales, casts with saturating round-to-nearest-even, packs codes and
 * scales, dequantizes in registers and reduces error statistics.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Pointers named x, codes, scales, global_scale, stats, xhat, workspace,
 *   amax_in and amax_out are DEVICE pointers (HIP device memory of the current
 *   device), and so are all other operands that are not said to be host
 *   memory.  Descriptors are HOST pointers.  The caller allocates and
 *   owns every buffer; the library allocates nothing and never
 *   synchronizes.  Between calls it keeps only a cache of occupancy queries
 *   per kernel and device (host memory, guarded by a mutex), and the
 *   workspace tickets it leaves at zero.
 * - All work is enqueued on `stream` (0 = the null stream).  Functions
 *   return before the GPU finishes; outputs are valid after the caller
 *   synchronizes with the stream.
 * - Arguments are validated on the host before anything is enqueued.  On
 *   any error nothing is enqueued and no output is touched.
 * - x is row-major [rows, cols] with a row stride of ld_in >= cols elements.
 *   The base address must be 16-byte aligned and ld_in * sizeof(element) a
 *   multiple of 16.  codes, scales and xhat are dense row-major and 16-byte
 *   aligned; workspace is 256-byte aligned.
 * - rows == 0 or cols == 0 is legal: no codes or scales are written and the
 *   statistics (if requested) are written as zeros.
 *
 * Code and scale layouts (element (r, c); K = cols):
 *   INT8        codes  int8  [rows, K]   (two's complement, q in [-127, 127])
 *   FP8 E4M3/E5M2 codes uint8 [rows, K]  (OCP E4M3: max 448, NaN 0x7F;
 *                                         OCP E5M2: max 57344)
 *   MXFP4       codes  uint8 [rows, K/2]  E2M1 nibbles; scales uint8 E8M0 [rows, K/32]
 *   NVFP4       codes  uint8 [rows, K/2]  E2M1 nibbles; scales uint8 E4M3 [rows, K/16];
 *               global_scale float32 [1]
 *   INT4        codes  uint8 [rows, K/2]  two's-complement nibbles, q in [-7, 7];
 *               scales float16 bits [rows, K/128]
 *   INT4_ZP     codes  uint8 [rows, K/2]  unsigned nibbles w in [0, 15];
 *               scales float32 [rows, K/128]; shifts uint8 [rows, K/256]
 *               (4-bit sh, group 2t in bits 3:0); K a multiple of 256
 *   INT8 / FP8 scales: float32 [1] per tensor, float32 [rows] per row.
 *   4-bit codes: element 2t in bits 3:0 of byte t, element 2t+1 in bits 7:4
 *   (the order of the packed-word extract() of the Triton post, Puzzle 12).
 */
#ifndef IQ_H
#define IQ_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define IQ_ABI_VERSION 2

typedef enum {
    IQ_OK = 0,
    IQ_EINVAL = 1,       /* NULL required pointer, bad enum, bad shape, cols not a multiple of the block */
    IQ_EALIGN = 2,       /* a pointer or the row stride breaks the alignment rules above */
    IQ_EUNSUPPORTED = 3, /* legal but not supported: unknown flags, sizes beyond 2^31 chunks */
    IQ_EHIP = 4          /* the HIP runtime reported an error when launching */
} iq_status;

typedef enum {
    IQ_INT8 = 0,     /* symmetric, s = alpha / 127 ("FP8" section, INT8 quantizer) */
    IQ_FP8_E4M3 = 1, /* s = alpha / 448 */
    IQ_FP8_E5M2 = 2, /* s = alpha / 57344 */
    IQ_MXFP4 = 3,    /* E2M1 codes, one E8M0 scale per 32 elements ("MXFP4") */
    IQ_NVFP4 = 4,    /* E2M1 codes, one E4M3 scale per 16 + FP32 global scale ("NVFP4") */
    IQ_INT4 = 5,     /* symmetric, s = A / 7 per group of 128, FP16 scale ("INT4") */
    IQ_INT4_ZP = 6   /* asymmetric: unsigned codes, FP32 scale + 4-bit shift per group of 128
                        (Triton post, Puzzle 12); only through iq_quantize_zp / iq_dequantize_zp */
} iq_format;

typedef enum { IQ_F32 = 0, IQ_BF16 = 1 } iq_dtype;

typedef enum {
    IQ_PER_TENSOR = 0, /* INT8 / FP8 */
    IQ_PER_ROW = 1,    /* INT8 / FP8 */
    IQ_PER_BLOCK = 2   /* MXFP4 (32), NVFP4 (16), INT4 and INT4_ZP (128): the only legal choice for those */
} iq_gran;

/* Rule variants (iq_desc.flags); 0 selects the default readings. */
#define IQ_FLAG_MX_ROUND_NEAREST 0x1u /* MXFP4: E8M0 = 2^round(log2(A/6)) instead of 2^(floor(log2 A)-2) */
#define IQ_FLAG_MX_ROUND_UP 0x2u      /* MXFP4: E8M0 = 2^ceil(log2(A/6)) */
#define IQ_FLAG_NV_SCALE_RNE 0x4u     /* NVFP4: block scale to E4M3 by RNE instead of rounding up */

typedef struct {
    int32_t fmt;      /* iq_format */
    int32_t gran;     /* iq_gran */
    int32_t in_dtype; /* iq_dtype of x */
    int32_t reserved0;
    int64_t rows, cols;
    int64_t ld_in;    /* row stride of x, in elements */
    uint32_t flags;
    uint32_t reserved1;
} iq_desc;

/* Error statistics of one iq_quantize call, written to device memory.
 * n counts every element; sums, max_abs_err and n_zero_flush cover the
 * finite inputs.  d = x - x^ (exact in FP32).  MSE = sum_err2 / (n - n_nonfinite).
 *   n_saturated   elements with |x/s| above the grid's largest value
 *   n_zero_flush  finite x != 0 whose x^ is 0 */
typedef struct {
    uint64_t n, n_zero_flush, n_saturated, n_nonfinite;
    double sum_x2, sum_err2, sum_abs_err;
    float max_abs_err;
    uint32_t reserved;
} iq_stats;

/* Bytes of the codes / scales arrays for a descriptor (0 on an invalid one). */
size_t iq_codes_bytes(const iq_desc* d);
size_t iq_scales_bytes(const iq_desc* d);
/* Bytes of device workspace iq_quantize / iq_amax need (>= 256). */
size_t iq_workspace_bytes(const iq_desc* d);

/*
 * Quantize x (the whole hot path).  Sections "FP8" (x^ = s * round(x / s),
 * s = alpha / 127; FP8 with its own grid) and "FP4 / MXFP4 / NVFP4"
 * (MXFP4 x^ = s_mx * Q(x / s_mx); NVFP4 s_global = amax / (6 * 448),
 * s_block = (block_amax / 6) / s_global; INT4 s = A / 7).
 *   codes, scales    outputs, layouts above (required)
 *   global_scale     NVFP4 output s_global (required for NVFP4, else ignored)
 *   stats            optional output (NULL skips the statistics)
 *   xhat             optional dequantized output [rows, cols] of xhat_dtype
 *   workspace        iq_workspace_bytes(d) bytes of device scratch, zero-filled
 *                    before its first use (e.g. hipMemset once, or torch.zeros);
 *                    every call leaves it ready for the next one.  The
 *                    workgroups of a call count themselves on it to decide
 *                    which one folds the partial statistics, and the absmax
 *                    pre-pass leaves its per-workgroup maxima there for the
 *                    cast, so concurrent calls need separate workspaces
 */
iq_status iq_quantize(const iq_desc* d, const void* x, void* codes, void* scales,
                      float* global_scale, iq_stats* stats, void* xhat, int32_t xhat_dtype,
                      void* workspace, hipStream_t stream);

/*
 * iq_quantize for callers that cannot allocate device memory (code under
 * HIP graph capture, tight serving loops, harnesses that forbid allocation):
 * the same computation, arguments and results, with the library's own
 * workspace in place of the caller's.
 *   The workspace is one device array per GPU of 128 KiB (IQ_NOALLOC_SCRATCH_BYTES),
 *   zero-filled when the library loads and held until the process ends; the
 *   call rejects a descriptor whose workspace would not fit it
 *   (IQ_EUNSUPPORTED; every descriptor iq_quantize accepts fits).
 *   No hipMalloc, hipFree or other allocating call is made.  The first call
 *   on a device resolves the array's address on that device (make one call
 *   before capturing a graph); a failure to resolve it returns IQ_EHIP.
 *   Every call on a GPU shares that GPU's array, and each call leaves it
 *   ready for the next: calls that may overlap on one GPU (other streams,
 *   other host threads) race and must be serialized by the caller.
 */
#define IQ_NOALLOC_SCRATCH_BYTES (128u * 1024u)
iq_status iq_quantize_noalloc(const iq_desc* d, const void* x, void* codes, void* scales,
                              float* global_scale, iq_stats* stats, void* xhat, int32_t xhat_dtype,
                              hipStream_t stream);

/*
 * Dequantize: x^ = s * decode(q), bit-identical to the x^ of iq_quantize.
 * Sections "FP8" (x^ = s * round(x / s): the code's value times the scale)
 * and "FP4 / MXFP4 / NVFP4" (MXFP4: E2M1 value times 2^(E - 127); NVFP4:
 * E2M1 value times s_global times the E4M3 block scale; INT4: q times the
 * FP16 group scale).
 * d->in_dtype and d->ld_in are ignored; xhat is dense [rows, cols] of
 * xhat_dtype (BF16 output is the FP32 x^ rounded to nearest even).
 * No workspace.  Errors as for iq_quantize.
 */
iq_status iq_dequantize(const iq_desc* d, const void* codes, const void* scales,
                        const float* global_scale, void* xhat, int32_t xhat_dtype,
                        hipStream_t stream);

/*
 * Per-tensor absmax over the finite elements of x (the per-tensor "alpha"
 * of section "FP8", the global amax of NVFP4), written to amax_out (device
 * float32 [1]).  Only d->in_dtype, rows, cols and ld_in are used.  The
 * workspace rules are those of iq_quantize (zero-filled before first use).
 */
iq_status iq_amax(const iq_desc* d, const void* x, float* amax_out, void* workspace,
                  hipStream_t stream);

/*
 * Static (calibrated) scaling: iq_quantize with the per-tensor absmax taken
 * from *amax_in (device float32 [1], e.g. written by iq_amax over
 * calibration data) instead of measured, so x is read once.  The scale is
 * derived from it exactly as iq_quantize derives it from the measured one
 * (section "FP8": s = alpha / FMAX; "NVFP4": s_global = amax / (6 * 448)).
 *   Legal for INT8 / E4M3 / E5M2 per tensor and for NVFP4 (the global
 *   scale; block scales still come from each block).  Any other
 *   descriptor returns IQ_EINVAL.
 *   Elements beyond alpha saturate and are counted in n_saturated; NaN and
 *   +-Inf inputs are handled as in iq_quantize.
 *   A NaN, negative or infinite *amax_in is taken as 0 (every code +0,
 *   scale 0); -0 is taken as +0.
 *   The other arguments, layouts, workspace rules and errors are those of
 *   iq_quantize; amax_in must be 4-byte aligned (IQ_EALIGN otherwise).
 */
iq_status iq_quantize_static(const iq_desc* d, const void* x, const float* amax_in, void* codes,
                             void* scales, float* global_scale, iq_stats* stats, void* xhat,
                             int32_t xhat_dtype, void* workspace, hipStream_t stream);

/*
 * Asymmetric INT4, the format of the Triton post's Puzzle 12 ("Quantized
 * Matrix Mult"): unsigned 4-bit codes w, and per group of 128 along the row
 * an FP32 scale sc and a 4-bit shift sh, with x^ = sc * (w - sh).  The page
 * prints this decoder only; the encoder is the min-max one:
 *   lo = min(0, min x), hi = max(0, max x) over the group's finite elements;
 *   sc = (hi - lo) / 15 in FP32 (the largest float if that overflows);
 *   sh = round-half-even(-lo / sc), clamped to [0, 15];
 *   w  = clamp(round-half-even(x / sc) + sh, 0, 15).
 * sc == 0 gives w = sh = 0; NaN gives w = sh (x^ = 0), +-Inf the ends 15 / 0.
 * n_saturated counts x / sc above 15 - sh or below -sh.
 *   d->fmt must be IQ_INT4_ZP with IQ_PER_BLOCK and cols a multiple of 256
 *   (IQ_EINVAL otherwise); d->flags must be 0.
 *   codes   uint8 [rows, cols/2]: element 2t in bits 3:0 of byte t, i.e.
 *           eight per little-endian 32-bit word, element i in bits
 *           [4i, 4i+4) (the page's extract() order)
 *   scales  float32 [rows, cols/128], 4-byte aligned
 *   shifts  uint8 [rows, cols/256], group 2t in bits 3:0 of byte t (whole
 *           32-bit words of eight shifts per row when cols % 1024 == 0)
 * The other arguments, layouts, workspace rules and errors are those of
 * iq_quantize.  iq_quantize and iq_dequantize reject IQ_INT4_ZP.
 */
iq_status iq_quantize_zp(const iq_desc* d, const void* x, void* codes, float* scales, uint8_t* shifts,
                         iq_stats* stats, void* xhat, int32_t xhat_dtype, void* workspace,
                         hipStream_t stream);
/* x^ = sc * (w - sh) from codes, scales and shifts laid out as above;
 * otherwise as iq_dequantize. */
iq_status iq_dequantize_zp(const iq_desc* d, const void* codes, const float* scales,
                           const uint8_t* shifts, void* xhat, int32_t xhat_dtype, hipStream_t stream);
/* Bytes of the shifts array for an IQ_INT4_ZP descriptor (0 otherwise). */
size_t iq_shifts_bytes(const iq_desc* d);

/*
 * The consumer of Puzzle 12 (Triton post, "Quantized Matrix Mult"):
 *   z[j, k] = sum_l sc[j, l/128] * (w[j, l] - sh[j, l/128]) * y[l, k]
 * with the IQ_INT4_ZP weights of d (N0 = d->rows, K = d->cols; codes,
 * scales and shifts laid out as for iq_quantize_zp) and activations given
 * token-major: x is [n1, K] row-major BF16 with x[k, l] = y[l, k].
 *   z       output float32 [N0, n1] row-major, 4-byte aligned
 *   x_dtype must be IQ_BF16 (IQ_EUNSUPPORTED otherwise): the products
 *           (w - sh) * x are formed exactly on the BF16 matrix cores and
 *           summed in FP32; each group's sum is scaled by sc with one fma.
 * Accuracy: |z - exact| <= (K + 2) * 2^-24 * sum_l |sc (w - sh) y|.
 * d->in_dtype and d->ld_in are ignored; codes and x 16-byte aligned.
 * N0, n1 and K must fit 31 bits, and (N0/128)(n1/128) output tiles must
 * stay below 2^31 (IQ_EUNSUPPORTED).  n1 == 0 or N0 == 0 is
 * legal and writes nothing.  No workspace.
 * Grids too small to fill the GPU (from 33 tokens, below about one tile
 * per CU) split K in two halves: the call zeroes z with a kernel of its own,
 * then each half adds its FP32 sum atomically.  Two addends on a +0 start
 * give a + b rounded once in either order, so every call returns the same
 * bits; z must not be touched by other work until the call completes.
 */
iq_status iq_zp_gemm(const iq_desc* d, const void* codes, const float* scales, const uint8_t* shifts,
                     const void* x, int32_t x_dtype, int64_t n1, float* z, hipStream_t stream);

/*
 * FP4 GEMM over two MXFP4 operands (low-precision post, section "FP4 /
 * MXFP4 / NVFP4": an MXFP4 value is its E2M1 code times the block scale
 * 2^(E - 127), one E8M0 byte per 32 elements):
 *   z[j, t] = sum_k xw[j, k] * xa[t, k]
 * with the weights described by d (IQ_MXFP4, IQ_PER_BLOCK; N0 = d->rows,
 * K = d->cols) and n1 activation rows of the same K, both laid out as
 * iq_quantize writes MXFP4 (codes [rows, K/2], element 2t in the low
 * nibble; scales [rows, K/32] E8M0 bytes).
 *   z       output float32 [N0, n1] row-major, 4-byte aligned
 * The matrix cores form every product exactly (with its two block scales)
 * and sum in FP32: |z - exact| <= (K + 2) * 2^-24 * sum_k |xw xa|.  A scale
 * byte of 255 (E8M0 NaN; iq_quantize never writes it) makes every output of
 * its row or token NaN.
 * K must be a multiple of 128 (IQ_EINVAL); codes 16-byte aligned, scales
 * 4-byte aligned (IQ_EALIGN).  N0, n1 and K must fit 31 bits, and
 * (N0/128)(n1/128) output tiles must stay below 2^31 (IQ_EUNSUPPORTED).  n1 == 0 or N0 == 0 is legal and writes nothing.
 * d->in_dtype and d->ld_in are ignored.  No workspace; inputs are not
 * modified.
 */
iq_status iq_mx_gemm(const iq_desc* d, const void* codes_w, const void* scales_w, const void* codes_a,
                     const void* scales_a, int64_t n1, float* z, hipStream_t stream);

/*
 * MXFP4 weights against BF16 activations (low-precision post, section
 * "FP4 / MXFP4 / NVFP4": the weight values are E2M1 codes times the block
 * scale 2^(E - 127)):
 *   z[j, t] = sum_k xw[j, k] * x[t, k]
 * with the weights described by d (IQ_MXFP4, IQ_PER_BLOCK; N0 = d->rows,
 * K = d->cols; laid out as iq_quantize writes MXFP4) and x token-major
 * [n1, K] row-major.
 *   z       output float32 [N0, n1] row-major, 4-byte aligned
 *   x_dtype must be IQ_BF16 (IQ_EUNSUPPORTED otherwise).  Each weight is
 *           exact in BF16, so the BF16 matrix cores form exact products,
 *           summed in FP32: |z - exact| <= (K + 2) * 2^-24 * sum_k |xw x|.
 *           A scale byte of 255 (E8M0 NaN) makes its row's outputs NaN.
 * K must be a multiple of 128 (IQ_EINVAL); codes and x 16-byte aligned,
 * scales 4-byte aligned (IQ_EALIGN).  N0, n1 and K must fit 31 bits, and
 * (N0/128)(n1/128) output tiles must stay below 2^31 (IQ_EUNSUPPORTED).
 * n1 == 0 or N0 == 0 is legal and writes nothing.  d->in_dtype and d->ld_in
 * are ignored.  No workspace.  Grids too small to fill the GPU use 64-row
 * tiles; K is never split and z is written directly, once.
 */
iq_status iq_mxw_gemm(const iq_desc* d, const void* codes, const void* scales, const void* x, int32_t x_dtype,
                      int64_t n1, float* z, hipStream_t stream);

/* ---------------------------------------------------------------------------
 * The feed-forward half of a transformer layer, around the quantized
 * weights: layer norm, the gate and up projections with their activation,
 * and the products of a few tokens with packed 4-bit weights.  A model
 * trains with the BF16 forms, quantizes its weights with iq_quantize and
 * answers with the packed ones.
 * ------------------------------------------------------------------------- */

/*
 * Layer norm over the rows of x [rows, cols]:
 *   mean = sum x / cols, rstd = 1 / sqrt(sum (x - mean)^2 / cols + eps),
 *   y = (x - mean) * rstd * weight + bias.
 * Only d->in_dtype, rows, cols and ld_in are used.  x has row stride ld_in;
 * y is dense [rows, cols] of x's type.
 *   param_dtype  iq_dtype of weight and bias
 *   weight, bias [cols]; NULL stands for ones / zeros
 *   mean, rstd   float32 [rows]; NULL where they are not wanted
 * Any cols up to 2^26 (more: IQ_EUNSUPPORTED; of none, mean is 0 and rstd
 * 1 / sqrt(eps), and x and y may be NULL) and any alignment that the
 * element types need are accepted; BF16 rows that start on 16-byte words are
 * faster, in the backward pass nearly twice.  Statistics are held in FP32.  A NaN or an
 * infinity makes its whole row NaN.  eps must be finite and >= 0.
 */
iq_status iq_layer_norm(const iq_desc* d, const void* x, const void* weight, const void* bias,
                        int32_t param_dtype, float eps, void* y, float* mean, float* rstd, hipStream_t stream);

/*
 * Its backward pass.  With n = (x - mean) * rstd and a = dy * weight:
 *   dx      = rstd * (a - sum a / cols - n * sum (a n) / cols)
 *   dweight = sum over rows of dy * n,   dbias = sum over rows of dy
 * x as above; dy and dx dense [rows, cols] of x's type; mean and rstd as
 * iq_layer_norm wrote them; dweight and dbias [cols] of param_dtype.
 * dx, dweight and dbias may each be NULL; weight NULL stands for ones.
 * Row sums are added in FP32 in an order fixed by the shape, so every call
 * returns the same bits.  rows == 0 writes zero gradients.
 *   workspace  iq_layer_norm_workspace_bytes(d) bytes, 256-byte aligned,
 *              of any content; may be NULL where dweight and dbias are.
 */
iq_status iq_layer_norm_backward(const iq_desc* d, const void* x, const void* dy, const void* weight,
                                 int32_t param_dtype, const float* mean, const float* rstd, void* dx, void* dweight,
                                 void* dbias, void* workspace, hipStream_t stream);
size_t iq_layer_norm_workspace_bytes(const iq_desc* d);

typedef enum {
    IQ_ACT_SILU = 0,     /* g / (1 + e^-g) */
    IQ_ACT_GELU = 1,     /* g (1 + erf(g / sqrt 2)) / 2 */
    IQ_ACT_GELU_TANH = 2 /* g (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3))) / 2 */
} iq_act;

/* A gated block: `tokens` rows of x, `cols` input features, `features`
 * rows of each weight. */
typedef struct {
    int32_t act;      /* iq_act */
    int32_t dtype;    /* iq_dtype of every operand: IQ_BF16 */
    int64_t tokens, cols, features;
    int64_t ld_x;     /* row stride of x, in elements */
    uint32_t flags;   /* 0 */
    uint32_t reserved;
} iq_gated_desc;

/*
 * The gate and up projections, the activation and the product in one kernel:
 *   g = x w_gate^T, u = x w_up^T, h = act(g) * u.
 * x [tokens, cols] with row stride ld_x, w_gate and w_up dense
 * [features, cols], h dense [tokens, features], all BF16 and 16-byte
 * aligned; cols, features and ld_x multiples of 8 (IQ_EINVAL; IQ_EALIGN
 * for ld_x), cols and features at most 2^20, tokens below 2^31
 * (IQ_EUNSUPPORTED).  Sums are held in FP32 and g and u are not rounded
 * before h is.
 *   saved  NULL, or iq_gated_saved_bytes(d) bytes, 16-byte aligned, that
 *          receive what iq_gated_backward needs: g and u in FP32.  (Rounded
 *          to BF16 they would add an error of the gradients' own rounding.)
 */
iq_status iq_gated_forward(const iq_gated_desc* d, const void* x, const void* w_gate, const void* w_up, void* h,
                           void* saved, hipStream_t stream);

/*
 * Its backward pass, from dh dense [tokens, features]:
 *   dg = dh * u * act'(g), du = dh * act(g)     (FP32, rounded once to BF16)
 *   dx = dg w_gate + du w_up, dw_gate = dg^T x, dw_up = du^T x
 * dx dense [tokens, cols], dw_gate and dw_up dense [features, cols], BF16.
 * dx, and the pair dw_gate, dw_up, may be NULL.  x is read only for the
 * weights' gradients and w_gate, w_up only for dx.
 *   workspace  iq_gated_workspace_bytes(d) bytes, 256-byte aligned, of any
 *              content.
 * Sums are FP32 in an order fixed by the shape; those of few tiles and many
 * terms are added in parts that the workspace holds.  tokens == 0 writes zero
 * weight gradients.
 */
iq_status iq_gated_backward(const iq_gated_desc* d, const void* dh, const void* x, const void* w_gate,
                            const void* w_up, const void* saved, void* dx, void* dw_gate, void* dw_up,
                            void* workspace, hipStream_t stream);
size_t iq_gated_saved_bytes(const iq_gated_desc* d);
size_t iq_gated_workspace_bytes(const iq_gated_desc* d);

/*
 * A few tokens times packed 4-bit weights, the weights read once:
 *   z[t, j] = sum_k x[t, k] w[j, k]
 * with the weights of d (IQ_INT4, IQ_NVFP4 or IQ_MXFP4, IQ_PER_BLOCK; N0 =
 * d->rows, K = d->cols), laid out as iq_quantize writes them; K a multiple
 * of 32 (IQ_EINVAL).  global_scale is NVFP4's (ignored otherwise).
 *   x        BF16 token-major [n1, K], 16-byte aligned (x_dtype IQ_BF16,
 *            else IQ_EUNSUPPORTED), 1 to 64 tokens (more: IQ_EUNSUPPORTED;
 *            many tokens go through iq_dequantize and a matrix product)
 *   z        z_dtype [n1, N0] token-major, ready to be the next product's x
 * N0 up to 2^25 and K up to 2^22 (IQ_EUNSUPPORTED).
 * Weights enter the matrix cores exactly (NVFP4 without the global scale,
 * INT4 without the group scale, as 4 a + b with a in [-2, 1], b in [0, 3])
 * and are summed in FP32: before z's own rounding |z - exact| <=
 * (2 K + 8) 2^-24 sum_k |x| m, where m is |w|, for INT4 |w| plus six group
 * scales.  MXFP4 weights of 2^128 and more (the largest codes under scale
 * bytes 253 and 254) are infinite, as iq_dequantize gives them.  MXFP4 scale
 * bytes of 255 and NVFP4 ones of 0x7F or 0xFF are NaN
 * and make their row's outputs NaN.  An infinity in a token makes that
 * token's outputs infinite where the weight is not zero, or NaN for INT4,
 * whose two parts may pull either way.  Sums are made before INT4's group scale
 * and NVFP4's global scale, so activations beyond 2^100 may overflow there.
 * d->in_dtype and d->ld_in are ignored.  n1 == 0 or N0 == 0 is legal and
 * writes nothing, K == 0 writes zeros.  No workspace.
 */
iq_status iq_packed_gemv(const iq_desc* d, const void* codes, const void* scales, const float* global_scale,
                         const void* x, int32_t x_dtype, int64_t n1, void* z, int32_t z_dtype, hipStream_t stream);

/*
 * The gated block for a few tokens with both weights packed, one launch:
 *   h[t, j] = act(sum_k x[t, k] wg[j, k]) * sum_k x[t, k] wu[j, k]
 * Both weights share d; other rules as for iq_packed_gemv.  h is h_dtype
 * [n1, N0] token-major.
 */
iq_status iq_packed_gated(const iq_desc* d, int32_t act, const void* codes_gate, const void* scales_gate,
                          const float* global_gate, const void* codes_up, const void* scales_up,
                          const float* global_up, const void* x, int32_t x_dtype, int64_t n1, void* h,
                          int32_t h_dtype, hipStream_t stream);

/* ---------------------------------------------------------------------------
 * The attention half of a transformer layer around an 8-bit cache: rotary
 * positions, a paged cache of keys and values in INT8 or E4M3 with a scale for
 * each block of 32 tokens and head, and attention over it.
 * ------------------------------------------------------------------------- */

typedef enum {
    IQ_ROTARY_HALF = 0,       /* pair i: elements i and i + rot / 2 */
    IQ_ROTARY_INTERLEAVED = 1 /* pair i: elements 2 i and 2 i + 1 */
} iq_rotary_layout;

typedef enum {
    IQ_ROTARY_PLAIN = 0,
    IQ_ROTARY_LINEAR = 1, /* every angle over factor */
    IQ_ROTARY_BASE = 2,   /* base * factor^(rot / (rot - 2)): the slowest pair's angle over factor, the fastest's kept */
    IQ_ROTARY_PARTS = 3   /* pairs by their turns r over `context` positions: over factor up to `low`, kept from `high`
                             on, in between a mean of both with weight (r - low) / (high - low) for the kept angle */
} iq_rotary_scaling;

/*
 * The table that rotations read: turns per position of each of rot / 2 pairs,
 *   table[i] = base^(-2 i / rot) / (2 pi), scaled.
 * A HOST function: `table` is host memory, and the other calls take a copy of
 * it in device memory.  rot even and >= 0; base > 0, factor > 0 and, for
 * IQ_ROTARY_PARTS, context > 0 and high > low, all finite, and so the turns (IQ_EINVAL).
 */
iq_status iq_rotary_table(int32_t rot, double base, int32_t scaling, double factor, double context, double low,
                          double high, double* table);

/* Strides count elements; the elements of a head are contiguous.  Here and below nothing is asked of the stride of a
 * dimension of one element. */
typedef struct {
    int32_t dtype;                      /* iq_dtype of x and y */
    int32_t layout;                     /* iq_rotary_layout */
    int64_t tokens, heads, dim;
    int64_t ld_token, ld_head;          /* of x */
    int64_t ld_token_out, ld_head_out;  /* of y */
    int32_t rot;                        /* leading elements of a head that turn: even, 0 to dim */
    float amplitude;                    /* factor of what turns */
    uint32_t flags;                     /* 0 */
    uint32_t reserved;
} iq_rotary_desc;

/*
 * Rotary positions.  With the angle f = 2 pi positions[t] table[i] of token t
 * and pair i (a, b), A = amplitude:
 *   a' = A (a cos f - b sin f),  b' = A (b cos f + a sin f)
 * and elements from rot on as they are.  Angles are reduced in 64 bits, so
 * far positions keep their digits; products are FP32, rounded once.
 *   x, y       [tokens, heads, dim] of dtype, of any alignment that the type
 *              needs; faster where bases are 16-byte aligned, strides and dim
 *              multiples of 16 bytes, and rot of 32 (half) or 16 bytes.
 *              y may be x where both have the same strides; otherwise they
 *              must not overlap.  x may repeat itself (strides of 0), y not.
 *   positions  int32 [tokens], of either sign
 *   table      double [rot / 2], as iq_rotary_table writes it (device memory)
 * heads up to 4096, dim up to 1024, heads * dim up to 2^20, tokens below 2^24
 * (IQ_EUNSUPPORTED).
 */
iq_status iq_rotary(const iq_rotary_desc* d, const void* x, const int32_t* positions, const double* table, void* y,
                    hipStream_t stream);

/* Its backward pass: the transposed rotation, from dy (as x) to dx (as y):
 *   da = A (da' cos f + db' sin f),  db = A (db' cos f - da' sin f). */
iq_status iq_rotary_backward(const iq_rotary_desc* d, const void* dy, const int32_t* positions, const double* table,
                             void* dx, hipStream_t stream);

/*
 * The cache.  Memory is `pages` pages of `page` tokens for each of `heads`
 * key and value heads; the page table says which pages hold a sequence.
 *   codes   uint8 [pages, heads, page / 32, 2, 32 * dim], 16-byte aligned: for
 *           every block of 32 tokens the keys' codes (0), then the values' (1).
 *           Keys lie as [dim / 16, 32 tokens, 16], values as [dim, 32 places],
 *           token t of the block at place
 *             16 * bit 2 of t + 8 * bit 4 + 4 * bit 3 + (t mod 4),
 *           the orders in which the matrix cores take both
 *   scales  float32 [pages, heads, page / 32, 2], 8-byte aligned: key and value scale of each block;
 *           a value is its code's value (INT8, E4M3) times the scale
 *   page_table  int32 [batch, width]: token t of sequence b lies in page
 *           page_table[b][t / page].  Entries outside [0, pages) stand for absent pages:
 *           nothing is written there, and their tokens are not seen
 *   lengths int32 [batch]: tokens of each sequence, those of this call among them
 *   starts  int32 [batch + 1], ascending: the call's tokens of sequence b are rows starts[b] to
 *           starts[b + 1] - 1 of its dense operands, and the last of the sequence's
 *           lengths[b].  NULL: one token for each sequence (tokens == batch).
 *           Rows from starts[batch] on, and rows before a sequence's first
 *           token, are no sequence's: what they would write is left as it was
 *           (iq_cache_attention writes zeros for the latter)
 * These arrays are device memory and are read when the kernel runs; whatever
 * they hold, nothing outside the operands is read or written.
 */
typedef struct {
    int32_t fmt;          /* IQ_INT8 or IQ_FP8_E4M3 */
    int32_t heads;        /* key and value heads, 1 to 1024 */
    int32_t dim;          /* elements of a head: 64, 96, 128, 192 or 256 */
    int32_t page;         /* tokens of a page: a power of two, 32 to 4096 */
    int64_t pages;        /* pages of the memory, up to 2^31 - 1 */
    int64_t batch, width; /* of the page table: up to 2^20; width * page up to 2^30 */
    uint32_t flags;       /* 0 */
    uint32_t reserved;
} iq_cache_desc;

/* Bytes of the cache's memory (0 on an invalid descriptor); only fmt, heads, dim, page and pages are used. */
size_t iq_cache_codes_bytes(const iq_cache_desc* d);
size_t iq_cache_scales_bytes(const iq_cache_desc* d);

typedef struct {
    int32_t dtype;                  /* iq_dtype of k, v, q and q_out */
    int32_t layout;                 /* iq_rotary_layout */
    int64_t tokens;                 /* rows of k, v and q: below 2^24 */
    int64_t q_heads;                /* heads of q: up to 4096; 0 without q */
    int64_t ld_k_token, ld_k_head;  /* strides in elements */
    int64_t ld_v_token, ld_v_head;
    int64_t ld_q_token, ld_q_head;
    int32_t rot;                    /* elements of a key's and query's head that turn: even, 0 to dim */
    float amplitude;
    uint32_t flags;                 /* 0 */
    uint32_t reserved;
} iq_append_desc;

/*
 * Appends the call's tokens: keys are turned by their position in the sequence
 * (as iq_rotary, FP32, not rounded in between), keys and values quantized into
 * their pages, and queries, if there are any, turned by the same positions.
 *   k, v    [tokens, heads, dim] of dtype;  q [tokens, q_heads, dim] or NULL
 *   q_out   dense [tokens, q_heads, dim] of dtype; may be q where that is dense, otherwise they must not overlap
 *   table   double [rot / 2] (device memory; may be NULL where rot is 0)
 * A block whose first token comes with this call gets s = alpha / 127 or
 * alpha / 448 in FP32, alpha being the largest finite magnitude of its new
 * elements; codes are x / s rounded to nearest even.  A block that holds
 * tokens already keeps its scale if that is at least the new tokens' alpha /
 * 127 or 448; otherwise the scale doubles until it is, and the codes there are
 * divided by the same power of two and rounded to nearest even (E4M3 codes
 * lose nothing by it above E4M3's subnormal range; INT8 codes are off by less than
 * one new step however often it happens).  A scale of 0, all elements being 0, counts
 * as none.  The cache holds finite values only: NaN is stored as 0, an infinity as the largest
 * code of its sign (0 in a block whose scale is 0).  Codes of tokens that are not the sequence's are left as they were.
 * The pages that one call appends to must be distinct, within a sequence and among sequences; pages shared and only
 * read are fine.  (tokens / 32 + 2 batch) * heads * 2 + tokens up to 2^23 (IQ_EUNSUPPORTED).
 */
iq_status iq_cache_append(const iq_cache_desc* d, const iq_append_desc* a, const void* k, const void* v,
                          const int32_t* page_table, const int32_t* lengths, const int32_t* starts,
                          const double* table, const void* q, void* q_out, void* codes, float* scales,
                          hipStream_t stream);

/*
 * Reads back: rows starts[b] to starts[b + 1] - 1 of k and v receive the last
 * tokens of sequence b, as iq_cache_append takes them (keys turned), each the code's value times its
 * scale, rounded once to out_dtype.  k and v dense [tokens, heads, dim], 16-byte aligned, apart;
 * either may be NULL.  Tokens of absent pages are zeros.  Limits as for iq_cache_append.
 */
iq_status iq_cache_read(const iq_cache_desc* d, const void* codes, const float* scales, const int32_t* page_table,
                        const int32_t* lengths, const int32_t* starts, int64_t tokens, void* k, void* v,
                        int32_t out_dtype, hipStream_t stream);

typedef struct {
    int32_t dtype;              /* of q and o: IQ_BF16 */
    int32_t causal;             /* 1: a query sees tokens up to its own; 0: all of its sequence */
    int64_t tokens, q_heads;    /* q_heads a multiple of the cache's heads: query head h reads head
                                   h / (q_heads / heads) */
    int64_t ld_token, ld_head;  /* strides of q, in elements */
    int64_t window;             /* 0, or with causal 1 the number of tokens that a query sees, its own the last */
    float scale;                /* of the scores, finite and >= 0 */
    uint32_t flags;             /* 0 */
} iq_attention_desc;

/*
 * Attention of the call's tokens over the cache, their own keys and values
 * (appended before) among it:
 *   o = sum over seen t of softmax_t(scale q . k_t) v_t
 * for prompts, for pieces of prompts behind what the cache holds, and for
 * single tokens; the lengths of one call may differ as they like.
 *   q   [tokens, q_heads, dim] BF16, 16-byte aligned, strides multiples of 8 elements (IQ_EALIGN)
 *   o   dense [tokens, q_heads, dim] BF16, 16-byte aligned; may be q where that is dense, otherwise they must not
 *       overlap.  A query that sees nothing gets zeros
 *   workspace  iq_cache_attention_workspace_bytes(d, a) bytes, 256-byte aligned, of any content: up to 120 MB, as
 *       the GPU and not the call has it, where a sequence may have more than 64 pairs of a token and a query head for a key head
 * Which kernels run goes by shapes, the page table's width among them, since lengths are read on the GPU: results change by
 * roundings with it, and a table much wider than its sequences makes short calls slower (one token at 500 tokens 6.9 us,
 * and 12.9 with a table for 131072).
 * Codes enter the matrix cores exactly, as FP16, and so do queries, scaled by a power of
 * two for each row (elements below 2^-28 of their row's largest lose digits); probabilities times
 * their block's values scale are rounded to FP16 (half a step: 2^-11; of those below 2^-23 of the
 * largest such product that the query has seen 2^-34 of that); sums, maxima and the running output
 * are FP32, and probabilities below 2^-126 may count as 0.  Scores times log2(e) have to lie in FP32's range.
 * Tokens that a query does not see add nothing, whatever their codes and scales hold, but for NaN
 * codes of E4M3 (which iq_cache_append never writes) in tokens that the sequence holds: they may make
 * any of that sequence's outputs of their head NaN.  Scales of seen tokens have to be finite and >= 0.  A
 * NaN or an infinity in a query makes that query's output NaN where it sees anything.
 * The order of all sums is fixed by shapes, lengths and starts: calls repeat their bits.
 * tokens * q_heads up to 2^28 (IQ_EUNSUPPORTED).
 */
iq_status iq_cache_attention(const iq_cache_desc* d, const iq_attention_desc* a, const void* codes, const float* scales,
                             const int32_t* page_table, const int32_t* lengths, const int32_t* starts, const void* q,
                             void* o, void* workspace, hipStream_t stream);
size_t iq_cache_attention_workspace_bytes(const iq_cache_desc* d, const iq_attention_desc* a);

const char* iq_status_str(iq_status s);
int iq_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif
