/*
 * mx_mi355x.h - C ABI of the block-scaled (MX) operators and of the fused RMS norm on MI355X
 * (gfx950). Same library, status codes, error messages (gemm_last_error) and conventions as
 * gemm_mi355x.h: every tensor pointer is a caller-owned DEVICE pointer, launches are
 * asynchronous on `stream`, no entry point allocates device memory or synchronises, errors
 * are returned and never thrown.
 *
 * MX tensors (OCP Microscaling Formats v1.0). A (rows, k) matrix is held as element codes
 * and one scale per MX_BLOCK = 32 consecutive values of a row:
 *   value = element * 2^(scale - 127);   scale 255 makes the whole block NaN.
 * Element types: MX_E2M1 (4 bits, magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6) and MX_E4M3 (8 bits,
 * OCP "fn", largest 448). Storage, with nb = ceil(k / 32):
 *   codes   row-major, rows of nb * 32 codes: nb * 32 bytes (E4M3) or nb * 16 bytes (E2M1, two
 *           codes to a byte, the even element in the low half). The codes past k in the last
 *           block are zero.
 *   scales  bytes in (ceil(rows / 64), ceil(nb / 16), 64, 16) order: block b of row r is byte
 *           ((r / 64 * ceil(nb / 16) + b / 16) * 64 + r % 64) * 16 + b % 16. The scales of
 *           blocks past nb are not 255 (mx_quantize and rmsnorm_forward write 0); those of
 *           rows past `rows` are never read into a result and may hold anything.
 * A grouped tensor (G, rows, k) holds G such matrices one after the other.
 */
#ifndef MX_MI355X_H
#define MX_MI355X_H

#include "gemm_mi355x.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MX_BLOCK 32

typedef enum { MX_E2M1 = 0, MX_E4M3 = 1 } mx_format;

/* Bytes of the codes and of the scales of a (rows, k) MX matrix (0 for an empty one, -1 for a
 * negative size, an unknown format or a number past 63 bits). */
int64_t mx_code_bytes(int64_t rows, int64_t k, int32_t format);
int64_t mx_scale_bytes(int64_t rows, int64_t k);

/* Quantise x (rows, cols), row r at x + r * ldx elements, of type GEMM_DT_F16 / BF16 / F32.
 * transpose = 0: blocks run along a row and the result is a (rows, cols) MX matrix;
 * transpose = 1: blocks run along a column and the result is the (cols, rows) MX matrix of
 * x^T. Per block: scale = 127 + floor(log2 max|x|) - emax (emax 2 for E2M1, 8 for E4M3), kept
 * to [0, 254], 0 for a block of zeros; elements x / 2^(scale - 127) rounded to nearest, ties to
 * even, saturated. A block that holds a NaN or an infinity gets scale 255 and zero codes.
 * x needs the alignment of its element type only, and ldx >= cols when rows > 1. codes must be
 * 16-byte aligned. Empty matrices launch nothing. INVALID_ARG (NULL, negative size, unknown
 * type), UNSUPPORTED (rows or cols above 2^30, ldx above 2^48), ALIGNMENT, HIP. */
gemm_status mx_quantize(int32_t rows, int32_t cols, const void* x, int32_t x_type, int64_t ldx,
                        int32_t transpose, int32_t format, void* codes, void* scales, void* stream);

/* The values of an MX matrix as out (rows, k) of type GEMM_DT_F16 / BF16 / F32, row r at
 * out + r * ldo elements (ldo >= k when rows > 1), rounded to nearest even (exact for F32
 * down to its smallest subnormal). */
gemm_status mx_dequantize(int32_t rows, int32_t k, int32_t format, const void* codes, const void* scales,
                          void* out, int32_t out_type, int64_t ldo, void* stream);

/* Fused RMS norm over the rows of x (rows, cols):
 *   h    = x + residual, rounded to the type of x   (h = x without a residual)
 *   rstd = 1 / sqrt(mean(h^2) + eps)                (fp32, from the rounded h)
 *   y    = h * rstd * weight, rounded to fp32 (to half a step for magnitudes from 2^-90 on, smaller
 *          ones to 2^-130; whatever h * weight is), written rounded to the type of x and / or as an
 *          MX matrix (rows, cols) quantised from the unrounded value.
 * x, residual, h, y and weight share `type` (F16, BF16, F32); each matrix has its own leading
 * dimension. h_out may be NULL (required NULL without a residual: h is x) and may be x or
 * residual itself; y may not overlap x, residual or h. rstd (fp32[rows]) may be NULL. At least
 * one of y and q_codes is given unless rows = 0, which launches nothing; q_codes and q_scales come
 * together. 1 <= cols <= 2^24, rows <= 2^30. */
typedef struct {
  int32_t rows, cols;
  int32_t type;     /* gemm_dtype */
  int32_t q_format; /* mx_format, read when q_codes is given */
  float eps;        /* >= 0 */
  const void* x;
  const void* residual; /* or NULL */
  const void* weight;   /* (cols,), contiguous */
  void* h_out;          /* or NULL */
  void* y;              /* or NULL */
  void* q_codes;        /* or NULL; 16-byte aligned */
  void* q_scales;
  float* rstd; /* or NULL */
  int64_t ldx, ldr, ldh, ldy;
} rmsnorm_args;
gemm_status rmsnorm_forward(const rmsnorm_args* args, void* stream);

/* Gradients of that norm, in fp32. With n = h * rstd and p = dy * weight:
 *   dx = rstd * (p - n * mean(p * n)) + dres     dw = sum over rows of dy * n
 * dx (the gradient with respect to h, hence to x and to the residual) has the type of h; dres
 * (the gradient that reaches h past the norm) may be NULL; dw is fp32[cols]. dx may be dy or
 * dres itself. workspace: rmsnorm_backward_workspace(rows, cols) bytes of device memory, 16-byte
 * aligned, whose contents need no preparation. Sums run in a fixed order: results repeat bit for
 * bit. rows = 0 writes a zero dw. */
typedef struct {
  int32_t rows, cols;
  int32_t type; /* gemm_dtype of dy, h, weight, dres, dx */
  const void* dy;
  const void* h;
  const void* weight;
  const float* rstd;
  const void* dres; /* or NULL */
  void* dx;
  float* dw;
  void* workspace;
  int64_t workspace_bytes;
  int64_t lddy, ldh, lddres, lddx;
} rmsnorm_backward_args;
gemm_status rmsnorm_backward(const rmsnorm_backward_args* args, void* stream);
/* Bytes of workspace (-1 for a negative size, or one that rmsnorm_backward refuses as too large). */
int64_t rmsnorm_backward_workspace(int32_t rows, int32_t cols);

/* Product of MX operands with a fused epilogue:
 *   D       = A x B^T + C        PostAct = act(A x B^T + C)   (before D's rounding)
 * Sums are held in fp32. With an E4M3 operand the matrix instruction itself keeps the products of a
 * block of 32 only to 2^-13 of the block's largest (1 + 2^-13 is exact, 1 + 2^-14 gives 1), so an F32
 * output has fewer good bits than an fp32 product of the same values: of normal values, K = 4096, it is off
 * by 4e-6 (E4M3 x E2M1) or 1.5e-5 (E4M3 x E4M3) in the Frobenius norm, where fp32 sums are by 5e-8 and the
 * rounding to BF16 by 1.7e-3. E2M1 x E2M1 products are exact before the sum.
 * A (M, K), B (N, K) MX matrices of any of the two formats each; C, D, PostAct row-major (M, N)
 * of type F16 / BF16 / F32 with their own leading dimensions (in elements). Grouped (groups > 0):
 * B is (groups, N, K) and row r of A / C / D / PostAct belongs to group g with
 * cu_seqlens_m[g] <= r < cu_seqlens_m[g+1] (device int32[groups+1], 0 .. M, never decreasing;
 * an array that breaks this runs nothing and writes nothing).
 * At least one of d, post is present. N is a multiple of 8, every leading dimension one of 16
 * bytes, K at most 2^22, and every pointer is 16-byte aligned. K = 0 gives D = C (or 0). The activations
 * are those of gemm_run (ReLU of a NaN is 0). C may be D or PostAct itself (of its type and leading
 * dimension); D and PostAct are two matrices. tile: 0 lets the library choose; otherwise one of the
 * MX_TILE values. */
typedef enum {
  MX_TILE_AUTO = 0,
  MX_TILE_256 = 1,   /* 256x256 outputs a workgroup, operands staged through LDS         */
  MX_TILE_128 = 2,   /* 128x128, the same                                                */
  MX_TILE_32X64 = 3, /* 32 rows x 64 columns, the waves of a workgroup share out K       */
  MX_TILE_32 = 4,    /* 32x32, the same                                                  */
  MX_TILE_16X32 = 5, /* 16 rows x 32 columns, the same                                   */
  MX_TILE_16 = 6     /* 16x16, the same                                                  */
} mx_tile;
/* split: how many workgroups share out the K of a tile: 0 lets the library choose, 1 one. More
 * than one needs a dense plan, a tile other than MX_TILE_256 and the workspace at run time. */
typedef struct {
  int32_t M, N, K;
  int32_t groups; /* 0: dense */
  int32_t a_format, b_format; /* mx_format */
  int32_t c, d, post;         /* gemm_dtype (NONE: absent) */
  int32_t act;                /* gemm_act; NONE without post */
  int32_t tile;               /* mx_tile */
  int32_t split;
  int64_t ldc, ldd, ldp;
} mx_gemm_desc;
typedef struct {
  const void* a_codes;
  const void* a_scales;
  const void* b_codes;
  const void* b_scales;
  const void* C;
  void* D;
  void* PostAct;
  const int32_t* cu_seqlens_m; /* grouped plans */
  void* workspace;             /* mx_gemm_workspace bytes, 16-byte aligned, or NULL: K is not split */
  int64_t workspace_bytes;
} mx_gemm_args;
typedef struct mx_gemm_plan mx_gemm_plan;

/* Validate and build a plan (host memory only, no HIP call; may be used from several threads and
 * streams at once, by runs that overlap with a workspace each). Errors as gemm_create. */
gemm_status mx_gemm_create(const mx_gemm_desc* desc, mx_gemm_plan** out);
gemm_status mx_gemm_run(const mx_gemm_plan* plan, const mx_gemm_args* args, void* stream);
gemm_status mx_gemm_destroy(mx_gemm_plan* plan);
/* The tile (mx_tile) and the split the plan runs with on a device with num_cus compute units, given
 * its workspace. Either pointer may be NULL. */
gemm_status mx_gemm_plan_tile(const mx_gemm_plan* plan, int32_t num_cus, int32_t* tile, int32_t* split);
/* Bytes of workspace a run takes on such a device (0 for most shapes). Its contents need no
 * preparation, and runs that follow each other on a stream may share it. */
gemm_status mx_gemm_workspace(const mx_gemm_plan* plan, int32_t num_cus, int64_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* MX_MI355X_H */
