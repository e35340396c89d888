// FP8 quantiser and its inverse, and activations with their checkpoint in 8 bits (fp8_quantize, fp8_dequantize,
// fp8_act_forward, fp8_act_backward of the public header).
//
// All of them are bound by memory: every input is read once and every output written once. Two shapes:
//   rows   blocks along rows only. A thread takes 8 values, 16 lanes a block; the maximum crosses lanes by DPP.
//   tiles  anything with blocks along columns, or tiles. A workgroup takes 128 x 128 values, which hold whole
//          blocks of both directions, in registers.
//
// Measured (among other kernels, on inputs that are not in a cache; a copy moves 4.78 TB/s):
//   16 x 4096 bf16 along rows, and its inverse                 2.6 and 2.4 us, which are the launch
//   16768 x 4096 bf16, SiLU, saved and q                       62 us, 283 MB: 4.6 TB/s
//   8192 x 8192 bf16 by tiles, both ways                       56 to 62 us, 269 MB: 4.3 to 4.8 TB/s
//   5001 x 4104 f16 along rows and columns                     26 to 29 us, 82 MB; 19.2 from a cache
//   8192 x 8192 bf16 GELU backward, q, qt, yt                  98 to 103 us, 403 MB and 17 of scales: 4.1 TB/s (SiLU 93, the
//                                                              ReLUs 89; q alone 71)
//   8192 x 8192 inverse to bf16                                35 us, 201 MB: 5.7 TB/s
// q, qt and yt of a computed value round its product with the block's factor to fp32 before the rounding to a code, so that near a border
// of two codes the other one may be taken (also for an fp32 x or dy as it is: act NONE, ReLU); rounding to odd first, as for saved,
// takes 68 us for 60 of 16768 x 4096 bf16 SiLU with saved and q, 121 for 99 of the GELU backward pass, and in fp32 80 to 82 for 74
// and 133 for 118.
// What was measured and is not kept: workgroups that stay and load the next tile ahead (the compiler spills: 120 us for
// 56 by tiles); bounds of 4 or 6 workgroups a compute unit (backward 126 for 101, by tiles 80 for 56).
#include <algorithm>
#include <type_traits>

#include "../gemm_kernel.hpp"
#include "fp8_common.hpp"

namespace gep {
gemm_status fail(gemm_status st, const char* fmt, ...);
void clear_error();

namespace {

constexpr int kThreads = 256;
constexpr int kTile = kFp8Block;

__device__ __forceinline__ void act8(int act, float v[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    switch (act) {
      case ACT_RELU: v[e] = act_fn<ACT_RELU>(v[e]); break;
      case ACT_RELU_SQ: v[e] = act_fn<ACT_RELU_SQ>(v[e]); break;
      case ACT_GELU_TANH: v[e] = act_fn<ACT_GELU_TANH>(v[e]); break;
      case ACT_SILU: v[e] = act_fn<ACT_SILU>(v[e]); break;
      default: break;
    }
  }
}
// act(x) and its slope. Both smooth activations are x s with s = 1 / (1 + 2^-u), and their slope is s (1 + x (1 - s) z')
// with z = u log 2; 1 - s = 2^-u s keeps its digits for large z. Beyond |x| = 12 (GELU) and 80 (SiLU) x is kept to
// that, and 2^-u below infinity, so that all factors are finite: there s is 0 or 1 to within 2^-115. The slope at a NaN (of a block
// or of a code) is NaN, and so are the smooth ones' values: their clamps are v_minimum and v_maximum, which pass it on.
template <int ACT>
__device__ __forceinline__ void act_and_slope(float x, float& y, float& d) {
  if constexpr (ACT == ACT_RELU) {
    y = act_fn<ACT_RELU>(x);
    d = x > 0.f ? 1.f : (x <= 0.f ? 0.f : x);
  } else if constexpr (ACT == ACT_RELU_SQ) {
    y = act_fn<ACT_RELU_SQ>(x);
    d = 2.f * __builtin_elementwise_maximum(x, 0.f);
  } else if constexpr (ACT == ACT_GELU_TANH || ACT == ACT_SILU) {
    constexpr bool gelu = ACT == ACT_GELU_TANH;
    constexpr float top = gelu ? 12.f : 80.f, log2e = 1.4426950408889634f;
    const float up = __builtin_elementwise_maximum(x, -top), c = __builtin_elementwise_minimum(up, top), c2 = c * c;
    // -u, and z' = dz / dx with z = 2 sqrt(2 / pi) (x + 0.044715 x^3)
    const float u = gelu ? c * __builtin_fmaf(c2, -0.044715f * 1.5957691216057308f * log2e, -1.5957691216057308f * log2e) : c * -log2e;
    const float e = __builtin_amdgcn_exp2f(__builtin_elementwise_minimum(u, 120.f)), s = __builtin_amdgcn_rcpf(1.f + e);
    const float cz = gelu ? c * __builtin_fmaf(c2, 0.134145f * 1.5957691216057308f, 1.5957691216057308f) : c;
    d = s * __builtin_fmaf(cz, e * s, 1.f);
    y = up * s;
  } else {
    y = x;
    d = x == x ? 1.f : x;
  }
}

// One FP8 matrix (codes NULL: absent).
struct Mat {
  uint8_t* codes;
  float* scales;
};

// Quantise and store chunk ch (8 values) of row r, blocks along the row. In each of the 16 lanes of a block.
template <bool EXACT>
__device__ __forceinline__ void store_row_chunk(const Mat& m, const Fp8Geometry& g, int64_t r, int ch, const float v[8]) {
  const Fp8Factor f = fp8_block(row_max16(largest8(v)));
  const uint2 w = fp8_codes8<EXACT>(v, f.r);
  if (ch * 8 < g.kp) *(uint2*)(m.codes + r * g.kp + ch * 8) = w;
  if ((ch & 15) == 0) fp8_store_scale(m.scales + fp8_row_scale(r, ch >> 4, g.nq), ch >> 4, g, f.scale);
}

// ---- blocks along rows: x as it is (saved) and act(x) (q, y). Chunks are numbered row by row over rows
// [r0, r0 + rows), 16 to a block (below 2^31 in one launch).
template <typename T, bool WHOLE>
__global__ __launch_bounds__(kThreads) void rows_kernel(const T* x, int64_t ldx, int64_t r0, Fp8Geometry g, uint32_t n,
                                                        FastDiv fd_cpr, int act, Mat saved, Mat q, T* y, int64_t ldy) {
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= n) return;  // (n is a multiple of 16: blocks leave together)
  uint32_t rr, ch;
  fd_divmod(fd_cpr, i, rr, ch);
  const int64_t r = r0 + rr;
  const int c = (int)ch * 8;
  float v[8];
  load8<WHOLE>(x + r * ldx, c, g.k, v);
  if (saved.codes) store_row_chunk<sizeof(T) == 4>(saved, g, r, (int)ch, v);
  if (!q.codes && !y) return;
  act8(act, v);
  if (y) store_chunk<WHOLE>(y + r * ldy, c, g.k, pack<T>(v));
  if (q.codes) {
    if (c + 8 > g.k) {  // (act(0) = 0 for all of them; -0 past the end would be a code)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = c + e < g.k ? v[e] : 0.f;
    }
    store_row_chunk<false>(q, g, r, (int)ch, v);
  }
}

// ---- 128 x 128 values in registers: thread t holds rows 8 (t / 16) + [0, 8), columns 8 (t % 16) + [0, 8), so
// that 16 neighbouring lanes hold a block of a row, and the 8 codes of a thread in one column are neighbours in
// the transposed matrix.
struct TileShared {
  union {
    __attribute__((aligned(16))) uint32_t codes[kTile * kTile / 4];
    __attribute__((aligned(16))) float part[16 * kTile];  // before that: 16 partial maxima of each column
  };
  __attribute__((aligned(16))) float factor[kTile];
};

// The codes of the tile with the factors r[j] of the thread's columns, transposed through LDS into rows c0 ... of a
// matrix (cols, rows). Unit g (8 codes) of column c lies at unit g ^ (c / 8): 16 lanes that write one unit of columns 8
// apart reach distinct banks, and so do 8 that read a column.
template <bool EXACT>
__device__ __forceinline__ void write_transposed(const float (&v)[8][8], const float (&r)[8], int r0, int c0, int cols,
                                                 const Fp8Geometry& gt, uint8_t* codes, TileShared& s) {
  const int tid = threadIdx.x, g = tid >> 4, cl = tid & 15;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float w[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) w[p] = v[p][j];
    *(uint2*)(s.codes + (cl * 8 + j) * 32 + (g ^ cl) * 2) = fp8_codes8<EXACT>(w, r[j]);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int u = i * kThreads + tid, c = u >> 3, h = u & 7, x = c >> 3;
    uint4 w = *(const uint4*)(s.codes + c * 32 + ((2 * h) ^ (x & ~1)) * 2);
    if (x & 1) w = uint4{w.z, w.w, w.x, w.y};
    if (c0 + c < cols && r0 + h * 16 < gt.kp) *(uint4*)(codes + (int64_t)(c0 + c) * gt.kp + r0 + h * 16) = w;
  }
}

// Blocks along the columns of the tile.
template <bool EXACT>
__device__ __forceinline__ void store_columns(const Mat& m, const Fp8Geometry& gt, int r0, int c0, int cols, const float (&v)[8][8],
                                              TileShared& s) {
  const int tid = threadIdx.x, g = tid >> 4, cl = tid & 15;
  float a[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float w[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) w[p] = v[p][j];
    a[j] = largest8(w);
  }
  f32x4* part = (f32x4*)(s.part + g * kTile + cl * 8);
  part[0] = f32x4{a[0], a[1], a[2], a[3]};
  part[1] = f32x4{a[4], a[5], a[6], a[7]};
  __syncthreads();
  if (tid < kTile) {
    float top = s.part[tid];
#pragma unroll
    for (int i = 1; i < 16; ++i) top = larger(top, s.part[i * kTile + tid]);
    const Fp8Factor f = fp8_block(top);
    s.factor[tid] = f.r;
    const int b = r0 / kFp8Block;
    if (c0 + tid < cols) fp8_store_scale(m.scales + fp8_row_scale(c0 + tid, b, gt.nq), b, gt, f.scale);
  }
  __syncthreads();
  float r[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) r[j] = s.factor[cl * 8 + j];
  write_transposed<EXACT>(v, r, r0, c0, cols, gt, m.codes, s);
}

// Tile i of the matrix: along the rows, or (down) down the columns.
struct TileMap {
  uint32_t first;
  FastDiv fd;  // by the tiles of a row, or of a column
  int32_t down;
};
struct TileAt {
  int r0, c0;
};
__device__ __forceinline__ TileAt tile_at(const TileMap& m, uint32_t i) {
  uint32_t q, r;
  fd_divmod(m.fd, m.first + i, q, r);
  return m.down ? TileAt{(int)r * kTile, (int)q * kTile} : TileAt{(int)q * kTile, (int)r * kTile};
}

// A thread's rows of one matrix of the tile: the chunks of rows r + [0, 8) at column c. Rows past the end load the last
// one, so that no load has a branch.
template <typename T, bool WHOLE>
struct TileRows {
  Chunk<T> in[8];
  __device__ __forceinline__ void load(const T* x, int64_t ld, int r, int c, int rows, int cols) {
#pragma unroll
    for (int p = 0; p < 8; ++p) in[p] = load_chunk<WHOLE>(x + (int64_t)min(r + p, rows - 1) * ld, c, cols);
  }
  // Row p, zeros past the matrix (edge: the tile reaches there).
  __device__ __forceinline__ void values(int p, int r, int c, int rows, int cols, bool edge, float (&v)[8]) {
    if (edge) {
      settle<WHOLE>(in[p], c, cols);
      unpack(in[p], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = r + p < rows ? v[e] : 0.f;
    } else {
      unpack(in[p], v);
    }
  }
};

// ---- the quantiser of a whole matrix in both directions, or by tiles.
template <typename T, bool TILES, bool WHOLE>
__global__ __launch_bounds__(kThreads) void quantize_tiles_kernel(const T* x, int64_t ldx, int rows, int cols, TileMap map, Mat q, Mat qt) {
  constexpr bool kExact = sizeof(T) == 4;
  __shared__ TileShared s;
  const int tid = threadIdx.x, g = tid >> 4, cl = tid & 15;
  const Fp8Geometry geo = fp8_geometry(cols), geo_t = fp8_geometry(rows);
  const TileAt at = tile_at(map, blockIdx.x);
  const int r = at.r0 + g * 8, c = at.c0 + cl * 8;
  const bool edge = at.r0 + kTile > rows || at.c0 + kTile > cols;
  TileRows<T, WHOLE> in;
  in.load(x, ldx, r, c, rows, cols);
  float v[8][8];
#pragma unroll
  for (int p = 0; p < 8; ++p) in.values(p, r, c, rows, cols, edge, v[p]);
  if constexpr (TILES) {
    float a = largest8(v[0]);
#pragma unroll
    for (int p = 1; p < 8; ++p) a = larger(a, largest8(v[p]));
    a = row_max16(a);
    if (cl == 0) s.factor[g] = a;
    __syncthreads();
    a = s.factor[0];
#pragma unroll
    for (int j = 1; j < 16; ++j) a = larger(a, s.factor[j]);
    const Fp8Factor f = fp8_block(a);
    const int i = at.r0 / kTile, b = at.c0 / kTile;
    if (q.codes) {
#pragma unroll
      for (int p = 0; p < 8; ++p)
        if (r + p < rows && c < geo.kp) *(uint2*)(q.codes + (int64_t)(r + p) * geo.kp + c) = fp8_codes8<kExact>(v[p], f.r);
      if (tid == 0) fp8_store_scale(q.scales + fp8_tile_scale(i, b, geo.nq), b, geo, f.scale);
    }
    if (qt.codes) {
      if (tid == 0) fp8_store_scale(qt.scales + fp8_tile_scale(b, i, geo_t.nq), i, geo_t, f.scale);
      float all[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) all[j] = f.r;
      write_transposed<kExact>(v, all, at.r0, at.c0, cols, geo_t, qt.codes, s);
    }
  } else {
    if (q.codes) {
#pragma unroll
      for (int p = 0; p < 8; ++p)
        if (r + p < rows) store_row_chunk<kExact>(q, geo, r + p, c >> 3, v[p]);
    }
    if (qt.codes) store_columns<kExact>(qt, geo_t, at.r0, at.c0, cols, v, s);
  }
}

// ---- the backward pass of an activation from its checkpoint.
template <typename T>
struct BackArgs {
  int rows, cols;
  const T* dy;
  const uint8_t* codes;
  const float* scales;
  T *dx, *y;
  Mat q, qt, yt;
  int64_t lddy, lddx, ldy;
};
template <typename T, int ACT, bool WHOLE>
__global__ __launch_bounds__(kThreads) void act_backward_kernel(const BackArgs<T> a, TileMap map) {
  __shared__ TileShared sx, sy;
  const int tid = threadIdx.x, g = tid >> 4, cl = tid & 15;
  const Fp8Geometry geo = fp8_geometry(a.cols), geo_t = fp8_geometry(a.rows);
  const TileAt at = tile_at(map, blockIdx.x);
  const int r = at.r0 + g * 8, c = at.c0 + cl * 8;
  const bool edge = at.r0 + kTile > a.rows || at.c0 + kTile > a.cols;
  TileRows<T, WHOLE> in;
  uint2 w[8];
  float scale[8];
  if (a.dy) in.load(a.dy, a.lddy, r, c, a.rows, a.cols);
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int64_t row = min(r + p, a.rows - 1);
    w[p] = *(const uint2*)(a.codes + row * geo.kp + min(c, geo.kp - 8));
    scale[p] = a.scales[fp8_row_scale(row, at.c0 / kFp8Block, geo.nq)];
  }
  float v[8][8], y[8][8];
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    float x[8], d[8];
    fp8_values8(w[p], scale[p], x);
    if (a.dy) in.values(p, r, c, a.rows, a.cols, edge, v[p]);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      act_and_slope<ACT>(x[e], y[p][e], d[e]);
      if (a.dy) v[p][e] *= d[e];
    }
    if (edge) {  // (rows past the end are copies of the last one)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const bool inside = r + p < a.rows && c + e < a.cols;
        y[p][e] = inside ? y[p][e] : 0.f;
        v[p][e] = inside ? v[p][e] : 0.f;
      }
    }
    if (r + p < a.rows) {
      if (a.y) store_chunk<WHOLE>(a.y + (int64_t)(r + p) * a.ldy, c, a.cols, pack<T>(y[p]));
      if (a.dx) store_chunk<WHOLE>(a.dx + (int64_t)(r + p) * a.lddx, c, a.cols, pack<T>(v[p]));
      if (a.q.codes) store_row_chunk<false>(a.q, geo, r + p, c >> 3, v[p]);
    }
  }
  if (a.qt.codes) store_columns<false>(a.qt, geo_t, at.r0, at.c0, a.cols, v, sx);
  if (a.yt.codes) store_columns<false>(a.yt, geo_t, at.r0, at.c0, a.cols, y, sy);
}

// ---- values of the codes. A thread takes 8 codes and writes 8 values.
template <typename T, bool TILES>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(const uint8_t* codes, const float* scales, int64_t r0, Fp8Geometry g,
                                                              uint32_t n, FastDiv fd_cpr, T* out, int64_t ldo) {
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= n) return;
  uint32_t rr, ch;
  fd_divmod(fd_cpr, i, rr, ch);
  const int64_t r = r0 + rr;
  const int b = (int)ch >> 4;
  float v[8];
  fp8_values8(*(const uint2*)(codes + r * g.kp + ch * 8), scales[TILES ? fp8_tile_scale(r / kTile, b, g.nq) : fp8_row_scale(r, b, g.nq)], v);
  store_chunk<false>(out + r * ldo, (int)ch * 8, g.k, pack<T>(v));
}

gemm_status launched(const char* fn) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(GEMM_ERR_HIP, "%s launch: %s", fn, hipGetErrorString(e));
  return GEMM_OK;
}

// Launch `f(r0, n)` over ranges of rows whose chunks number below 2^31.
template <typename F>
void row_ranges(int32_t rows, uint32_t cpr, F&& f) {
  const int64_t per = std::max((int64_t)1, (int64_t)0x7FFFFF00 / cpr);
  for (int64_t r0 = 0; r0 < rows; r0 += per) f(r0, (uint32_t)(std::min((int64_t)rows - r0, per) * cpr));
}
// Launch `f(grid, map)` over the 128 x 128 tiles. Tiles follow each other along the rows, so that the lines of all matrices that the
// card works on at a time lie together (down the columns 8192 x 8192 in both directions takes 71 us for 60, by tiles 66 for 54, 8100 x
// 8192 87 for 66). But where rows of codes are no whole lines, two tiles side by side share a line of each row; workgroups go to the 8
// XCDs in turn, so down columns of a multiple of 8 tiles both are on one XCD, whose L2 puts the line together (5120 x 4104
// 19.1 us for 26.0, 8192 x 8200 78.5 for 81.4; with 41 tiles a column, 5200 x 4104, 26.0 either way). Over 292 sizes, types and
// scalings the rule is 0.4% slower than the better order in the mean, 16% at most (16384 x 4128); along the rows alone
// 3 and 37%.
template <typename F>
gemm_status tile_ranges(const char* fn, int32_t rows, int32_t cols, F&& f) {
  const int64_t ty = ((int64_t)rows + kTile - 1) / kTile, tx = ((int64_t)cols + kTile - 1) / kTile;
  if (ty * tx > 0x7FFFFF00) return fail(GEMM_ERR_UNSUPPORTED, "%s: more than 2^31 tiles", fn);
  TileMap m;
  m.down = fp8_geometry(cols).kp % 128 != 0 && ty % 8 == 0;  // (128 bytes a line, 8 XCDs)
  m.fd = make_fastdiv((uint32_t)(m.down ? ty : tx));
  constexpr int64_t most = 1 << 22;  // (a grid has below 2^32 threads)
  for (int64_t first = 0; first < ty * tx; first += most) {
    m.first = (uint32_t)first;
    f((uint32_t)std::min(ty * tx - first, most), m);
  }
  return launched(fn);
}

constexpr int32_t kMaxExtent = 1 << 30;

int element_bytes(int32_t type) { return type == GEMM_DT_F32 ? 4 : ((type == GEMM_DT_F16 || type == GEMM_DT_BF16) ? 2 : 0); }
gemm_status check_size(const char* fn, int32_t rows, int32_t cols, int32_t type) {
  if (rows < 0 || cols < 0) return fail(GEMM_ERR_INVALID_ARG, "%s: negative size", fn);
  if (rows > kMaxExtent || cols > kMaxExtent) return fail(GEMM_ERR_UNSUPPORTED, "%s: more than 2^30 rows or columns", fn);
  if (!element_bytes(type)) return fail(GEMM_ERR_INVALID_ARG, "%s: the type must be F16, BF16 or F32", fn);
  return GEMM_OK;
}
// A matrix argument (rows and cols not 0).
gemm_status check_matrix(const char* fn, const char* name, int32_t rows, int32_t cols, int32_t type, int64_t ld, const void* p) {
  if (ld < 0 || ld > ((int64_t)1 << 48)) return fail(GEMM_ERR_UNSUPPORTED, "%s: leading dimension of %s outside [0, 2^48]", fn, name);
  if (rows > 1 && ld < cols) return fail(GEMM_ERR_INVALID_ARG, "%s: leading dimension of %s below its columns", fn, name);
  if (!p) return fail(GEMM_ERR_INVALID_ARG, "%s: NULL %s", fn, name);
  if ((uintptr_t)p % element_bytes(type)) return fail(GEMM_ERR_ALIGNMENT, "%s: %s not aligned to its elements", fn, name);
  return GEMM_OK;
}
gemm_status check_fp8(const char* fn, const char* name, const void* codes, const void* scales) {
  if (!codes || !scales) return fail(GEMM_ERR_INVALID_ARG, "%s: codes and scales of %s come together", fn, name);
  if ((uintptr_t)codes & 15) return fail(GEMM_ERR_ALIGNMENT, "%s: codes of %s not 16-byte aligned", fn, name);
  if ((uintptr_t)scales & 3) return fail(GEMM_ERR_ALIGNMENT, "%s: scales of %s not 4-byte aligned", fn, name);
  return GEMM_OK;
}
template <typename T>
void run_rows(const T* x, int64_t ldx, int32_t rows, int32_t cols, int act, Mat saved, Mat q, T* y, int64_t ldy, hipStream_t s) {
  const Fp8Geometry g = fp8_geometry(cols);
  const uint32_t cpr = (uint32_t)g.nb * 16;
  row_ranges(rows, cpr, [&](int64_t r0, uint32_t n) {
    const unsigned grid = (n + kThreads - 1) / kThreads;
    if (cols % 8 == 0) rows_kernel<T, true><<<grid, kThreads, 0, s>>>(x, ldx, r0, g, n, make_fastdiv(cpr), act, saved, q, y, ldy);
    else rows_kernel<T, false><<<grid, kThreads, 0, s>>>(x, ldx, r0, g, n, make_fastdiv(cpr), act, saved, q, y, ldy);
  });
}

}  // namespace
}  // namespace gep

using namespace gep;

extern "C" {

gemm_status fp8_quantize(int32_t rows, int32_t cols, const void* x, int32_t x_type, int64_t ldx, int32_t scaling, void* codes,
                         void* scales, void* codes_t, void* scales_t, void* stream) {
  const char* fn = "fp8_quantize";
  gemm_status st = check_size(fn, rows, cols, x_type);
  if (st != GEMM_OK) return st;
  if (scaling != FP8_ROWS && scaling != FP8_TILES) return fail(GEMM_ERR_INVALID_ARG, "%s: unknown scaling %d", fn, scaling);
  if (rows == 0 || cols == 0) { clear_error(); return GEMM_OK; }
  if (!codes && !scales && !codes_t && !scales_t) return fail(GEMM_ERR_INVALID_ARG, "%s: no output", fn);
  st = check_matrix(fn, "x", rows, cols, x_type, ldx, x);
  if (st == GEMM_OK && (codes || scales)) st = check_fp8(fn, "x", codes, scales);
  if (st == GEMM_OK && (codes_t || scales_t)) st = check_fp8(fn, "x^T", codes_t, scales_t);
  if (st != GEMM_OK) return st;
  if (codes == codes_t) return fail(GEMM_ERR_INVALID_ARG, "%s: x and x^T are one matrix", fn);
  clear_error();
  hipStream_t s = (hipStream_t)stream;
  const Mat q{(uint8_t*)codes, (float*)scales}, qt{(uint8_t*)codes_t, (float*)scales_t};
  with_type(x_type, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    if (scaling == FP8_ROWS && !codes_t) {
      run_rows<T>((const T*)x, ldx, rows, cols, ACT_NONE, q, Mat{nullptr, nullptr}, nullptr, 0, s);
      st = launched(fn);
      return;
    }
    st = tile_ranges(fn, rows, cols, [&](uint32_t grid, const TileMap& m) {
      auto go = [&](auto by_tiles, auto whole) {
        quantize_tiles_kernel<T, decltype(by_tiles)::value, decltype(whole)::value><<<grid, kThreads, 0, s>>>((const T*)x, ldx, rows, cols, m, q, qt);
      };
      if (scaling == FP8_ROWS) cols % 8 == 0 ? go(std::false_type{}, std::true_type{}) : go(std::false_type{}, std::false_type{});
      else cols % 8 == 0 ? go(std::true_type{}, std::true_type{}) : go(std::true_type{}, std::false_type{});
    });
  });
  return st;
}

gemm_status fp8_dequantize(int32_t rows, int32_t k, int32_t scaling, const void* codes, const void* scales, void* out,
                           int32_t out_type, int64_t ldo, void* stream) {
  const char* fn = "fp8_dequantize";
  gemm_status st = check_size(fn, rows, k, out_type);
  if (st != GEMM_OK) return st;
  if (scaling != FP8_ROWS && scaling != FP8_TILES) return fail(GEMM_ERR_INVALID_ARG, "%s: unknown scaling %d", fn, scaling);
  if (rows == 0 || k == 0) { clear_error(); return GEMM_OK; }
  st = check_matrix(fn, "out", rows, k, out_type, ldo, out);
  if (st == GEMM_OK) st = check_fp8(fn, "the matrix", codes, scales);
  if (st != GEMM_OK) return st;
  clear_error();
  hipStream_t s = (hipStream_t)stream;
  const Fp8Geometry g = fp8_geometry(k);
  const uint32_t cpr = (uint32_t)g.kp / 8;
  const uint8_t* qc = (const uint8_t*)codes;
  const float* qs = (const float*)scales;
  with_type(out_type, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    row_ranges(rows, cpr, [&](int64_t r0, uint32_t n) {
      const unsigned grid = (n + kThreads - 1) / kThreads;
      if (scaling == FP8_ROWS) dequantize_kernel<T, false><<<grid, kThreads, 0, s>>>(qc, qs, r0, g, n, make_fastdiv(cpr), (T*)out, ldo);
      else dequantize_kernel<T, true><<<grid, kThreads, 0, s>>>(qc, qs, r0, g, n, make_fastdiv(cpr), (T*)out, ldo);
    });
  });
  return launched(fn);
}

gemm_status fp8_act_forward(const fp8_act_args* a, void* stream) {
  const char* fn = "fp8_act_forward";
  if (!a) return fail(GEMM_ERR_INVALID_ARG, "%s: NULL args", fn);
  gemm_status st = check_size(fn, a->rows, a->cols, a->type);
  if (st != GEMM_OK) return st;
  if (a->act < GEMM_ACT_NONE || a->act > GEMM_ACT_SILU) return fail(GEMM_ERR_INVALID_ARG, "%s: unknown activation %d", fn, a->act);
  if (a->rows == 0 || a->cols == 0) { clear_error(); return GEMM_OK; }
  const bool saved = a->saved_codes || a->saved_scales, q = a->q_codes || a->q_scales;
  if (!saved && !q && !a->y) return fail(GEMM_ERR_INVALID_ARG, "%s: no output", fn);
  st = check_matrix(fn, "x", a->rows, a->cols, a->type, a->ldx, a->x);
  if (st == GEMM_OK && a->y) st = check_matrix(fn, "y", a->rows, a->cols, a->type, a->ldy, a->y);
  if (st == GEMM_OK && saved) st = check_fp8(fn, "saved", a->saved_codes, a->saved_scales);
  if (st == GEMM_OK && q) st = check_fp8(fn, "q", a->q_codes, a->q_scales);
  if (st != GEMM_OK) return st;
  if (saved && a->saved_codes == a->q_codes) return fail(GEMM_ERR_INVALID_ARG, "%s: saved and q are one matrix", fn);
  if (a->y == a->x && a->rows > 1 && a->ldy != a->ldx) return fail(GEMM_ERR_INVALID_ARG, "%s: y in the place of x needs its leading dimension", fn);
  clear_error();
  with_type(a->type, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    run_rows<T>((const T*)a->x, a->ldx, a->rows, a->cols, a->act, Mat{(uint8_t*)a->saved_codes, (float*)a->saved_scales},
                Mat{(uint8_t*)a->q_codes, (float*)a->q_scales}, (T*)a->y, a->ldy, (hipStream_t)stream);
  });
  return launched(fn);
}

gemm_status fp8_act_backward(const fp8_act_backward_args* a, void* stream) {
  const char* fn = "fp8_act_backward";
  if (!a) return fail(GEMM_ERR_INVALID_ARG, "%s: NULL args", fn);
  gemm_status st = check_size(fn, a->rows, a->cols, a->type);
  if (st != GEMM_OK) return st;
  if (a->act < GEMM_ACT_NONE || a->act > GEMM_ACT_SILU) return fail(GEMM_ERR_INVALID_ARG, "%s: unknown activation %d", fn, a->act);
  if (a->rows == 0 || a->cols == 0) { clear_error(); return GEMM_OK; }
  const bool q = a->q_codes || a->q_scales, qt = a->qt_codes || a->qt_scales, yt = a->yt_codes || a->yt_scales;
  const bool grad = a->dx || q || qt;
  if (!grad && !a->y && !yt) return fail(GEMM_ERR_INVALID_ARG, "%s: no output", fn);
  if (grad != (a->dy != nullptr)) return fail(GEMM_ERR_INVALID_ARG, "%s: dy comes with dx, q or qt", fn);
  st = check_fp8(fn, "saved", a->saved_codes, a->saved_scales);
  if (st == GEMM_OK && grad) st = check_matrix(fn, "dy", a->rows, a->cols, a->type, a->lddy, a->dy);
  if (st == GEMM_OK && a->dx) st = check_matrix(fn, "dx", a->rows, a->cols, a->type, a->lddx, a->dx);
  if (st == GEMM_OK && a->y) st = check_matrix(fn, "y", a->rows, a->cols, a->type, a->ldy, a->y);
  if (st == GEMM_OK && q) st = check_fp8(fn, "q", a->q_codes, a->q_scales);
  if (st == GEMM_OK && qt) st = check_fp8(fn, "qt", a->qt_codes, a->qt_scales);
  if (st == GEMM_OK && yt) st = check_fp8(fn, "yt", a->yt_codes, a->yt_scales);
  if (st != GEMM_OK) return st;
  if (a->dx && a->dx == a->dy && a->rows > 1 && a->lddx != a->lddy)
    return fail(GEMM_ERR_INVALID_ARG, "%s: dx in the place of dy needs its leading dimension", fn);
  const void* outs[] = {a->dx, a->y, a->q_codes, a->qt_codes, a->yt_codes};
  for (int i = 0; i < 5; ++i) {
    if (outs[i] && outs[i] == a->saved_codes) return fail(GEMM_ERR_INVALID_ARG, "%s: an output in the place of the checkpoint", fn);
    for (int j = 0; j < i; ++j)
      if (outs[i] && outs[i] == outs[j]) return fail(GEMM_ERR_INVALID_ARG, "%s: two outputs are one matrix", fn);
  }
  if (a->y && a->y == a->dy) return fail(GEMM_ERR_INVALID_ARG, "%s: y in the place of dy", fn);
  clear_error();
  with_type(a->type, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    const BackArgs<T> b{a->rows, a->cols, (const T*)a->dy, (const uint8_t*)a->saved_codes, (const float*)a->saved_scales,
                        (T*)a->dx, (T*)a->y, Mat{(uint8_t*)a->q_codes, (float*)a->q_scales},
                        Mat{(uint8_t*)a->qt_codes, (float*)a->qt_scales}, Mat{(uint8_t*)a->yt_codes, (float*)a->yt_scales},
                        a->lddy, a->lddx, a->ldy};
    st = tile_ranges(fn, a->rows, a->cols, [&](uint32_t grid, const TileMap& m) {
      auto go = [&](auto act) {
        if (a->cols % 8 == 0) act_backward_kernel<T, decltype(act)::value, true><<<grid, kThreads, 0, (hipStream_t)stream>>>(b, m);
        else act_backward_kernel<T, decltype(act)::value, false><<<grid, kThreads, 0, (hipStream_t)stream>>>(b, m);
      };
      switch (a->act) {
        case GEMM_ACT_RELU: go(std::integral_constant<int, ACT_RELU>{}); break;
        case GEMM_ACT_RELU_SQ: go(std::integral_constant<int, ACT_RELU_SQ>{}); break;
        case GEMM_ACT_GELU_TANH: go(std::integral_constant<int, ACT_GELU_TANH>{}); break;
        case GEMM_ACT_SILU: go(std::integral_constant<int, ACT_SILU>{}); break;
        default: go(std::integral_constant<int, ACT_NONE>{}); break;
      }
    });
  });
  return st;
}

}  // extern "C"
