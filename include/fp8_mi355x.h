/*
 * fp8_mi355x.h - C ABI of the 8-bit operators with a scale per 128 values, and of activation
 * checkpoints in that format, on MI355X (gfx950). Same library, status codes, error messages
 * (gemm_last_error) and conventions as gemm_mi355x.h: every tensor pointer is a caller-owned DEVICE
 * pointer, launches are asynchronous on `stream`, no entry point allocates device memory or
 * synchronises, errors are returned and never thrown.
 *
 * FP8 matrices. A (rows, k) matrix is held as OCP e4m3 codes ("fn", largest 448) and one fp32 scale per
 * FP8_BLOCK = 128 consecutive values of a row (FP8_ROWS: activations and gradients) or per tile of 128
 * rows by 128 values (FP8_TILES: weights):   value = code * scale.  A NaN scale makes its block NaN.
 * Storage, with nb = ceil(k / 128) and nq = ceil(nb / 4):
 *   codes   row-major, rows of ceil(k / 16) * 16 bytes; the codes past k are zero.
 *   scales  FP8_ROWS: fp32 in (ceil(rows / 64), nq, 64, 4) order, block b of row r being element
 *           ((r / 64 * nq + b / 4) * 64 + r % 64) * 4 + b % 4; FP8_TILES: (ceil(rows / 128), nq * 4),
 *           tile (i, b) being element i * nq * 4 + b. The scales of blocks past nb lie below 2^63 in
 *           magnitude (the quantisers write 0; the product forms their products, which have to be finite);
 *           those of rows past `rows` are never read into a result and may hold anything.
 * A grouped matrix (G, rows, k) holds G such matrices one after the other.
 *
 * Quantisation of a block: r = 448 / max|x| (rounded to fp32), 2^126 at most, cut to 13 significant bits;
 * code = x * r rounded to nearest, ties to even; scale = 1 / r, rounded to fp32. (With 13 bits x * r is exact in fp32
 * for F16 and BF16 values, so that each code is the nearest one; the scale is at most 2^-12 larger than
 * max|x| / 448; F32 values within 2^-12 of the type's largest may come back as infinities.) A block that holds
 * a NaN or an infinity gets a NaN scale and zero codes. The codes 0x7F and 0xFF, which the quantisers never
 * write, are NaN.
 */
#ifndef FP8_MI355X_H
#define FP8_MI355X_H

#include "gemm_mi355x.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FP8_BLOCK 128

typedef enum { FP8_ROWS = 0, FP8_TILES = 1 } fp8_scaling;

/* Bytes of the codes and of the scales of a (rows, k) matrix (0 for an empty one, -1 for a negative
 * size, an unknown scaling or a number past 63 bits). */
int64_t fp8_code_bytes(int64_t rows, int64_t k);
int64_t fp8_scale_bytes(int64_t rows, int64_t k, int32_t scaling);

/* Quantise x (rows, cols), row r at x + r * ldx elements, of type GEMM_DT_F16 / BF16 / F32, in one pass over x:
 *   codes, scales      the (rows, cols) matrix of x: blocks along its rows (FP8_ROWS) or its tiles
 *   codes_t, scales_t  the (cols, rows) matrix of x^T: blocks along x's columns, or the same tiles
 * Either pair may be NULL, not both. Each is exact: codes and scales are the definition's, F32 values
 * included. x needs the alignment of its element type only, and ldx >= cols when rows > 1; codes are
 * 16-byte and scales 4-byte aligned. Empty matrices launch nothing. INVALID_ARG (NULL, negative size,
 * unknown type or scaling), UNSUPPORTED (rows or cols above 2^30, ldx above 2^48), ALIGNMENT, HIP. */
gemm_status fp8_quantize(int32_t rows, int32_t cols, const void* x, int32_t x_type, int64_t ldx,
                         int32_t scaling, void* codes, void* scales, void* codes_t, void* scales_t,
                         void* stream);

/* The values of an FP8 matrix as out (rows, k) of type GEMM_DT_F16 / BF16 / F32, row r at
 * out + r * ldo elements (ldo >= k when rows > 1), code * scale rounded to fp32 and then to the type. */
gemm_status fp8_dequantize(int32_t rows, int32_t k, int32_t scaling, const void* codes, const void* scales,
                           void* out, int32_t out_type, int64_t ldo, void* stream);

/* An activation between two products, keeping its input in 8 bits for the backward pass. Of x
 * (rows, cols), type F16 / BF16 / F32, in one pass:
 *   saved  x itself as an FP8 matrix (FP8_ROWS), exact as by fp8_quantize
 *   q      act(x) as an FP8 matrix (FP8_ROWS), the operand of the next product
 *   y      act(x) rounded to x's type
 * At least one of them; each pair of codes and scales comes together. act(x) is computed in fp32 from
 * the unrounded x; q is quantised from that fp32 value, its product with r rounded to fp32 before the
 * rounding to a code: F32 values near a border of two codes may get the other one, also where act(x) is x, and q then
 * differs from saved. The activations are those of gemm_run (ReLU of a NaN is 0); y may be x itself. */
typedef struct {
  int32_t rows, cols;
  int32_t type; /* gemm_dtype of x and y */
  int32_t act;  /* gemm_act */
  const void* x;
  void* saved_codes; /* or NULL; 16-byte aligned, as all codes */
  void* saved_scales;
  void* q_codes; /* or NULL */
  void* q_scales;
  void* y; /* or NULL */
  int64_t ldx, ldy;
} fp8_act_args;
gemm_status fp8_act_forward(const fp8_act_args* args, void* stream);

/* The backward pass from that checkpoint, in one pass over dy and the 8 bits. With x^ the value of `saved`
 * (FP8_ROWS) in fp32:
 *   dx = dy * act'(x^)   rounded to the type of dy (dx), as an FP8 matrix (q, for the product with the
 *                        weight) and as that of dx^T (qt, for the weight's gradient)
 *   y = act(x^)          rounded to `type` (y), and as the FP8 matrix of y^T (yt, for the gradient of
 *                        the weight behind the activation)
 * Each output may be NULL, not all of them; dy is needed for the first three and NULL without them
 * (act NONE then transposes a checkpoint: yt has its blocks along the other axis). act' of ReLU is 0 at 0; a NaN
 * block or code of `saved` makes its dx NaN (and y but for the ReLUs'). dx may be dy itself. All FP8 matrices are FP8_ROWS. */
typedef struct {
  int32_t rows, cols;
  int32_t type; /* gemm_dtype of dy, dx and y */
  int32_t act;  /* gemm_act */
  const void* dy;
  const void* saved_codes;
  const void* saved_scales;
  void* dx;
  void* q_codes;
  void* q_scales;
  void* qt_codes; /* (cols, rows) */
  void* qt_scales;
  void* y;
  void* yt_codes; /* (cols, rows) */
  void* yt_scales;
  int64_t lddy, lddx, ldy;
} fp8_act_backward_args;
gemm_status fp8_act_backward(const fp8_act_backward_args* args, void* stream);

/* Product of FP8 matrices with a fused epilogue:
 *   D       = A x B^T + C        PostAct = act(A x B^T + C)   (before D's rounding)
 *   (A x B^T)[m, n] = sum over blocks b of  sa[m, b] * sb[n, b] * sum over k in b of a[m, k] * b[n, k]
 * The matrix instruction sums the 128 products of a block, and the blocks are scaled and added in fp32. The
 * instruction keeps the products of 32 values only to 2^-13 of their largest, so an F32 output has
 * fewer good bits than an fp32 product of the same values. In fp32 sa * sb is formed first where B is FP8_TILES, the
 * block's sum times sb where it is FP8_ROWS: what of these lies below 2^-126 loses bits, and what passes fp32's range
 * gives infinities or, where a block's products sum to 0, NaN.
 * A (M, K) is FP8_ROWS; B (N, K) FP8_TILES (weights) or FP8_ROWS (the weight's gradient: dW = dY^T x X^T^T
 * of two matrices with blocks along the tokens). C, D, PostAct row-major (M, N) of type F16 / BF16 / F32
 * with their own leading dimensions (in elements). Grouped (groups > 0): B is (groups, N, K) and row r
 * of A / C / D / PostAct belongs to group g with cu_seqlens_m[g] <= r < cu_seqlens_m[g+1] (device
 * int32[groups+1], 0 .. M, never decreasing; an array that breaks this runs nothing and writes
 * nothing). The groups share out rows only: sums over a group's tokens, the gradients of the experts' weights, are
 * gemm_mi355x.h's variable-K products of 16-bit operands (blocks of 128 tokens run over the groups' borders). At
 * least one of d, post is present. N is a multiple of 8, every leading dimension one of 16 bytes, K at most 2^22, and
 * every pointer is 16-byte aligned. K = 0 gives D = C (or 0). The activations are those of gemm_run. C may be D or
 * PostAct itself (of its type and leading dimension); D and PostAct are two matrices. tile: 0 lets the library choose;
 * otherwise one of the FP8_TILE values. */
typedef enum {
  FP8_TILE_AUTO = 0,
  FP8_TILE_256 = 1,   /* 256x256 outputs a workgroup, operands staged through LDS       */
  FP8_TILE_128 = 2,   /* 128x128, the same                                              */
  FP8_TILE_64 = 3,    /* 64x64, the same, and the waves of a workgroup share out K      */
  FP8_TILE_32 = 4,    /* 32x32, the waves share out K and read their operands directly  */
  FP8_TILE_16X32 = 5, /* 16 rows x 32 columns, the same                                 */
  FP8_TILE_16 = 6     /* 16x16, the same                                                */
} fp8_tile;
/* split: how many workgroups share out the K of a tile: 0 lets the library choose, 1 one. More
 * than one needs a dense plan, a tile other than FP8_TILE_256 and the workspace at run time. */
typedef struct {
  int32_t M, N, K;
  int32_t groups;     /* 0: dense */
  int32_t b_scaling;  /* fp8_scaling */
  int32_t c, d, post; /* gemm_dtype (NONE: absent) */
  int32_t act;        /* gemm_act; NONE without post */
  int32_t tile;       /* fp8_tile */
  int32_t split;
  int64_t ldc, ldd, ldp;
} fp8_gemm_desc;
typedef struct {
  const void* a_codes;
  const void* a_scales;
  const void* b_codes;
  const void* b_scales;
  const void* C;
  void* D;
  void* PostAct;
  const int32_t* cu_seqlens_m; /* grouped plans */
  void* workspace;             /* fp8_gemm_workspace bytes, 16-byte aligned, or NULL: K is not split */
  int64_t workspace_bytes;
} fp8_gemm_args;
typedef struct fp8_gemm_plan fp8_gemm_plan;

/* Validate and build a plan (host memory only, no HIP call; may be used from several threads and
 * streams at once, by runs that overlap with a workspace each). Errors as gemm_create. */
gemm_status fp8_gemm_create(const fp8_gemm_desc* desc, fp8_gemm_plan** out);
gemm_status fp8_gemm_run(const fp8_gemm_plan* plan, const fp8_gemm_args* args, void* stream);
gemm_status fp8_gemm_destroy(fp8_gemm_plan* plan);
/* The tile (fp8_tile) and the split the plan runs with on a device with num_cus compute units, given
 * its workspace. Either pointer may be NULL. */
gemm_status fp8_gemm_plan_tile(const fp8_gemm_plan* plan, int32_t num_cus, int32_t* tile, int32_t* split);
/* Bytes of workspace a run takes on such a device (0 for most shapes). Its contents need no
 * preparation, and runs that follow each other on a stream may share it. */
gemm_status fp8_gemm_workspace(const fp8_gemm_plan* plan, int32_t num_cus, int64_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* FP8_MI355X_H */
