// Fused RMS norm with residual addition and MX output, and its gradients (rmsnorm_forward,
// rmsnorm_backward of the public header).
//
//   h = x + r (rounded),  rstd = (mean h^2 + eps)^(-1/2),  y = h rstd w
//   dx = rstd (p - n mean(p n)) + dres,  dw = sum_rows dy n,   n = h rstd, p = dy w
//
// Both are bound by memory. A row is held in registers from its single read to its last use:
// threads x CH chunks of 8 elements, chunk j of thread t at column (t + j threads) 8. Four
// adjacent lanes hold an MX block. Rows too long for registers take a kernel that reads them
// twice. All sums run in a fixed order. 16768 x 4096 bf16 with residual, h and e4m3 output: 80 us (483
// MB, 6.0 TB/s); gradients 8192 x 8192 bf16 with dres: 95 us (537 MB and 17 MB of column sums written and
// read, 6.0 TB/s; 91 and 5 us of it in the two kernels); one row of 4096: 3 us, the launch and two
// rounds of memory latency. (Times in these comments: calls in a graph, one after the other.)
#include <type_traits>

#include "mx_common.hpp"

namespace gep {
gemm_status fail(gemm_status st, const char* fmt, ...);
void clear_error();

namespace {

struct NormParams {
  const void *x, *r, *w;
  void *h, *y;
  uint8_t *codes, *scales;
  float* rstd;
  int64_t ldx, ldr, ldh, ldy;
  int32_t rows, cols, nb, nsb;
  int32_t row0;  // this launch's first row
  float eps;
  double inv_cols;
};

// v of another lane of the 16-lane row, by a DPP pattern.
template <int PATTERN>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), PATTERN, 0xF, 0xF, true));
}
template <int PATTERN>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, PATTERN, 0xF, 0xF, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), PATTERN, 0xF, 0xF, true);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
template <typename V>
__device__ __forceinline__ V wave_sum(V v) {
  v += dpp<0xB1>(v);   // lanes 1 0 3 2 of a quad
  v += dpp<0x4E>(v);   // lanes 2 3 0 1
  v += dpp<0x141>(v);  // mirrored half rows
  v += dpp<0x140>(v);  // mirrored rows
  v += __shfl_xor(v, 16);
  v += __shfl_xor(v, 32);
  return v;
}
// Sum over the threads of a row, in each of them. WAVE: a wave a row; else the workgroup (red: one
// value per wave).
template <bool WAVE, typename V>
__device__ __forceinline__ V row_sum(V v, V* red) {
  v = wave_sum(v);
  if constexpr (!WAVE) {
    __syncthreads();  // the last use of red is over
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0;
    for (int i = 0; i < (int)blockDim.x / 64; ++i) v += red[i];
  }
  return v;
}

// ---- y = h rstd w. A quantised value flips to its neighbour where an error carries y over the
// border between them, so y is the rounding of the exact product: squares are summed in 64 bits,
// rstd is held as hi + lo, h w is exact for 16-bit h and w (22 bits) or held as hi + lo too, and a y
// that falls on a border of the element type is moved to the side of it that the product lies on
// before it is quantised (y itself is stored as it is, the nearest fp32 number).
// (With fp32 sums and two fp32 products 56 of 69 million values flipped, and now none.) h w may leave
// fp32's range where h rstd w does not: chunks with a y that is not finite and rows of a very large or
// small rstd are computed again in 64 bits, as are those with a y on a border.
struct Rstd {
  float hi, lo;
  double r;
  bool far;  // outside [2^-32, 2^20] (inside, an h w below the normal range costs y 2^-130 at most)
};
__device__ __forceinline__ Rstd reciprocal_root(double mean_eps) {
  // (in 64 bits: squares of fp32 and bf16 values leave the fp32 range)
  const double r0 = __builtin_amdgcn_rsq(mean_eps);
  // One Newton step squares the relative error of the approximate root. (That is infinite for 0, and 0
  // or NaN for an infinite or NaN sum; those need no step.)
  const double r = __builtin_isfinite(r0) && r0 > 0 ? r0 + 0.5 * r0 * (1.0 - mean_eps * r0 * r0) : r0;
  Rstd s;
  s.r = r;
  s.hi = (float)r;
  s.lo = __builtin_isfinite(s.hi) ? (float)(r - (double)s.hi) : 0.f;
  s.far = !(s.hi >= 0x1p-32f && s.hi <= 0x1p20f);
  return s;
}
// Returns which y lie on a border beside their product: bit e, the product has the larger magnitude; bit 8 + e,
// the smaller.
template <typename T>
__device__ __forceinline__ uint32_t scale8(const float h[8], const float w[8], const Rstd& r, float y[8]) {
  uint32_t low = ~0u, move = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float hw = h[e] * w[e];
    float c = hw * r.lo;
    if constexpr (sizeof(T) == 4) c = fmaf(fmaf(h[e], w[e], -hw), r.hi, c);
    y[e] = fmaf(hw, r.hi, c);
    low = min(low, __float_as_uint(y[e]) << 13);
  }
  // Borders between values of at most four significant bits: the last 19 bits of y are zero there. So
  // they are in an infinity, and in the NaN that inf * hi + inf * lo gives.
  // (Branches of the whole wave, and a loop: rare code lies past the end of the common one and is short.
  // One row of 4096 bf16: 3.2 us; with eight copies of it in line 3.6.)
  if (__builtin_expect(__ballot((low == 0) | r.far) != 0, 0)) {
    bool again = r.far;
#pragma unroll
    for (int e = 0; e < 8; ++e) {  // (zeros, as those past the row's end, are right as they are)
      const uint32_t b = __float_as_uint(y[e]);
      again |= (b << 13) == 0 && (b << 1) != 0;
    }
    if (__ballot(again) == 0) return 0;
    float hr[8], wr[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) hr[e] = h[e], wr[e] = w[e];
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {  // element i is at place 0, and its result goes to place 7
      const double p = (double)hr[0] * (double)wr[0] * r.r;
      const float v = (float)p;
      const double rest = p - (double)v;
      const uint32_t b = __float_as_uint(v);
      const bool border = (b << 13) == 0 && (b << 1) != 0 && rest != 0 && __builtin_isfinite(rest);
      move = (move >> 1) | (border ? ((rest > 0) == (v > 0.f) ? 1u << 7 : 1u << 15) : 0u);
#pragma unroll
      for (int e = 0; e < 7; ++e) hr[e] = hr[e + 1], wr[e] = wr[e + 1], y[e] = y[e + 1];
      y[7] = v;
    }
  }
  return move;
}
// Sum of squares of a chunk.
__device__ __forceinline__ double squares(const float v[8]) {
  double s = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) s = fma((double)v[e], (double)v[e], s);
  return s;
}

// Output chunk `ch` of a row: y in its type and / or (FMT an mx_format, or kNoMx) quantised. move: by scale8.
constexpr int kNoMx = -1;
template <typename T, int FMT, bool WHOLE, int STREAM = 0>
__device__ __forceinline__ void norm_out(const NormParams& p, T* y_row, uint8_t* code_row, uint8_t* scale_row, int ch,
                                         float y[8], uint32_t move) {
  if (p.y) store_chunk<WHOLE, STREAM != 0>(y_row, ch * 8, p.cols, pack<T>(y));
  if constexpr (FMT != kNoMx) {
    if (__builtin_expect(__ballot(move != 0) != 0, 0)) {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = __uint_as_float(__float_as_uint(y[e]) + ((move >> e) & 1) - ((move >> (8 + e)) & 1));
    }
    if (ch < p.nb * 4) mx_store_chunk<FMT>(y, ch, p.nb, p.nsb, code_row, scale_row);
  }
}

// h is kept in its own type (its rounded value is exact there): half the registers of fp32 for
// 16-bit rows.
template <typename T, bool WAVE, int CH, int FMT, bool WHOLE, int STREAM>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void rmsnorm_kernel(const NormParams p) {
  __shared__ double red[WAVE ? 1 : 16];
  const int threads = WAVE ? 64 : blockDim.x;
  const int t = WAVE ? threadIdx.x & 63 : threadIdx.x;
  const int64_t row = p.row0 + (WAVE ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : (int64_t)blockIdx.x);
  if (WAVE && row >= p.rows) return;  // (a whole wave)
  const T* x = (const T*)p.x + row * p.ldx;
  Chunk<T> h[CH];
  double ss = 0;
#pragma unroll
  for (int j = 0; j < CH; ++j) h[j] = load_chunk<WHOLE, STREAM == 2>(x, (t + j * threads) * 8, p.cols);
  if (p.r) {
    const T* r = (const T*)p.r + row * p.ldr;
    Chunk<T> rc[CH];
#pragma unroll
    for (int j = 0; j < CH; ++j) rc[j] = load_chunk<WHOLE, STREAM == 2>(r, (t + j * threads) * 8, p.cols);
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = (t + j * threads) * 8;
      float a[8], b[8];
      settle<WHOLE>(h[j], c, p.cols);
      settle<WHOLE>(rc[j], c, p.cols);
      unpack(h[j], a);
      unpack(rc[j], b);
#pragma unroll
      for (int e = 0; e < 8; ++e) a[e] += b[e];
      h[j] = pack<T>(a);
      if (p.h) store_chunk<WHOLE, STREAM != 0>((T*)p.h + row * p.ldh, c, p.cols, h[j]);
      unpack(h[j], a);
      ss += squares(a);
    }
  } else {
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      float a[8];
      settle<WHOLE>(h[j], (t + j * threads) * 8, p.cols);
      unpack(h[j], a);
      ss += squares(a);
    }
  }
  const Rstd rstd = reciprocal_root(row_sum<WAVE>(ss, red) * p.inv_cols + (double)p.eps);
  if (p.rstd && t == 0) p.rstd[row] = rstd.hi;
  T* y_row = (T*)p.y + row * p.ldy;
  uint8_t *code_row = mx_code_row<FMT>(p.codes, row, p.nb), *scale_row = mx_scale_row(p.scales, row, p.nsb);
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    const int ch = t + j * threads;
    float a[8], w[8], y[8];
    forget(h[j]);
    unpack(h[j], a);
    load8<WHOLE>((const T*)p.w, ch * 8, p.cols, w);
    const uint32_t move = scale8<T>(a, w, rstd, y);
    norm_out<T, FMT, WHOLE, STREAM>(p, y_row, code_row, scale_row, ch, y, move);
  }
}

// Rows of any length: one workgroup a row, read twice (the second time from the caches).
template <typename T, int FMT>
__global__ __launch_bounds__(1024) void rmsnorm_long_kernel(const NormParams p) {
  __shared__ double red[16];
  const int64_t row = p.row0 + (int64_t)blockIdx.x;
  const T* x = (const T*)p.x + row * p.ldx;
  const T* r = p.r ? (const T*)p.r + row * p.ldr : nullptr;
  const int n = p.nb * 4;
  auto load_h = [&](int ch, float v[8]) {
    load8<false>(x, ch * 8, p.cols, v);
    if (r) {
      float q[8];
      load8<false>(r, ch * 8, p.cols, q);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += q[e];
      unpack(pack<T>(v), v);
    }
  };
  double ss = 0;
  for (int ch = threadIdx.x; ch < n; ch += 1024) {
    float v[8];
    load_h(ch, v);
    ss += squares(v);
  }
  const Rstd rstd = reciprocal_root(row_sum<false>(ss, red) * p.inv_cols + (double)p.eps);
  if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd.hi;
  for (int ch = threadIdx.x; ch < n; ch += 1024) {
    float v[8], w[8], y[8];
    load_h(ch, v);
    // (h may be x or the residual: every element is read again by the thread that replaces it)
    if (r && p.h) store_chunk<false>((T*)p.h + row * p.ldh, ch * 8, p.cols, pack<T>(v));
    load8<false>((const T*)p.w, ch * 8, p.cols, w);
    const uint32_t move = scale8<T>(v, w, rstd, y);
    norm_out<T, FMT, false>(p, (T*)p.y + row * p.ldy, mx_code_row<FMT>(p.codes, row, p.nb), mx_scale_row(p.scales, row, p.nsb), ch, y, move);
  }
}

// ---- gradients. A workgroup walks rows blockIdx.x, + gridDim.x, ... and keeps its columns' sums of
// dy n in registers; it writes them as row blockIdx.x of the partial sums, which a second
// kernel adds up in order.
struct NormGradParams {
  const void *dy, *h, *w, *dres;
  const float* rstd;
  void* dx;
  float* part;  // (gridDim.x, cols)
  int64_t lddy, ldh, lddres, lddx;
  int32_t rows, cols;
  float inv_cols;
};

template <typename T, bool WHOLE>
constexpr bool rows_ahead() {
  return WHOLE && sizeof(T) == 2;
}
template <typename T, bool WAVE, int CH, bool WHOLE, int STREAM>
__global__ __launch_bounds__(WAVE ? 64 : 1024) void rmsnorm_grad_kernel(const NormGradParams p) {
  __shared__ float red[WAVE ? 1 : 16];
  // The next row is on its way while this one meets at the barriers and is stored, where its registers
  // fit (fp32 rows, or chunks to be moved into place: 333 x 2050 fp32 9.5 us, ahead 14.6).
  constexpr bool kAhead = rows_ahead<T, WHOLE>();
  const int t = threadIdx.x, threads = blockDim.x;
  float dw[CH][8];
  Chunk<T> w[CH];
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    const int c = (t + j * threads) * 8;
    w[j] = load_chunk<WHOLE>((const T*)p.w, c, p.cols);
    settle<WHOLE>(w[j], c, p.cols);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[j][e] = 0.f;
  }
  struct Row {
    Chunk<T> h[CH], dy[CH], g[CH];
    float rstd;
  };
  auto load = [&](Row& r, int64_t row) {
    r.rstd = p.rstd[row];
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      r.h[j] = load_chunk<WHOLE, STREAM == 2>((const T*)p.h + row * p.ldh, (t + j * threads) * 8, p.cols);
      r.dy[j] = load_chunk<WHOLE, STREAM == 2>((const T*)p.dy + row * p.lddy, (t + j * threads) * 8, p.cols);
    }
    if (p.dres) {
#pragma unroll
      for (int j = 0; j < CH; ++j)
        r.g[j] = load_chunk<WHOLE, STREAM == 2>((const T*)p.dres + row * p.lddres, (t + j * threads) * 8, p.cols);
    }
  };
  Row next;
  if (kAhead && blockIdx.x < p.rows) load(next, blockIdx.x);
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    if (!kAhead) load(next, row);
    Chunk<T> hc[CH], dyc[CH], gc[CH];
#pragma unroll
    for (int j = 0; j < CH; ++j) hc[j] = next.h[j], dyc[j] = next.dy[j], gc[j] = next.g[j];
    const float rstd = next.rstd;
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = (t + j * threads) * 8;
      float n[8], dy[8], ww[8];
      settle<WHOLE>(hc[j], c, p.cols);
      settle<WHOLE>(dyc[j], c, p.cols);
      forget(w[j]);
      unpack(hc[j], n);
      unpack(dyc[j], dy);
      unpack(w[j], ww);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float dyn = dy[e] * (n[e] * rstd);
        dw[j][e] += dyn;
        dot = fmaf(dyn, ww[e], dot);
      }
    }
    if (kAhead && row + gridDim.x < p.rows) load(next, row + gridDim.x);
    const float m = row_sum<WAVE>(dot, red) * p.inv_cols;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = (t + j * threads) * 8;
      float n[8], dy[8], ww[8], g[8];
      forget(hc[j]);
      forget(dyc[j]);
      forget(w[j]);
      unpack(hc[j], n);
      unpack(dyc[j], dy);
      unpack(w[j], ww);
      if (p.dres) {
        settle<WHOLE>(gc[j], c, p.cols);
        unpack(gc[j], g);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] = fmaf(rstd, dy[e] * ww[e] - n[e] * rstd * m, g[e]);
      store_chunk<WHOLE, STREAM != 0>((T*)p.dx + row * p.lddx, c, p.cols, pack<T>(g));
    }
  }
  float* part = p.part + (int64_t)blockIdx.x * p.cols;
#pragma unroll
  for (int j = 0; j < CH; ++j) store_chunk<WHOLE>(part, (t + j * threads) * 8, p.cols, pack<float>(dw[j]));
}

// Rows of any length: each row is read twice and the column sums live in the workgroup's row of
// the partial sums.
template <typename T>
__global__ __launch_bounds__(1024) void rmsnorm_grad_long_kernel(const NormGradParams p) {
  __shared__ float red[16];
  float* part = p.part + (int64_t)blockIdx.x * p.cols;
  const int n8 = (p.cols + 7) / 8;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const float rstd = p.rstd[row];
    const T* h = (const T*)p.h + row * p.ldh;
    const T* dyp = (const T*)p.dy + row * p.lddy;
    float dot = 0.f;
    for (int ch = threadIdx.x; ch < n8; ch += 1024) {
      float n[8], dy[8], w[8], s[8];
      load8<false>(h, ch * 8, p.cols, n);
      load8<false>(dyp, ch * 8, p.cols, dy);
      load8<false>((const T*)p.w, ch * 8, p.cols, w);
      if (row == blockIdx.x) {
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] = 0.f;
      } else {
        load8<false>(part, ch * 8, p.cols, s);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float dyn = dy[e] * (n[e] * rstd);
        s[e] += dyn;
        dot = fmaf(dyn, w[e], dot);
      }
      store_chunk<false>(part, ch * 8, p.cols, pack<float>(s));
    }
    const float m = row_sum<false>(dot, red) * p.inv_cols;
    for (int ch = threadIdx.x; ch < n8; ch += 1024) {
      float n[8], dy[8], w[8], g[8];
      load8<false>(h, ch * 8, p.cols, n);
      load8<false>(dyp, ch * 8, p.cols, dy);
      load8<false>((const T*)p.w, ch * 8, p.cols, w);
      if (p.dres) {
        load8<false>((const T*)p.dres + row * p.lddres, ch * 8, p.cols, g);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] = fmaf(rstd, dy[e] * w[e] - n[e] * rstd * m, g[e]);
      store_chunk<false>((T*)p.dx + row * p.lddx, ch * 8, p.cols, pack<T>(g));
    }
  }
}

// dw = sum of `n` rows of partial sums: 32 columns (whole lines) a workgroup, 32 threads a column.
// (8192 x 8192 bf16, 512 rows of sums: both kernels 95.9 us; 16 columns 98.8, 64 columns 95.6; with fewer
// columns 64 are slower than 32: 8192 x 512 15.9 and 13.6.)
constexpr int kSumCols = 32, kSumRows = 32;
__global__ __launch_bounds__(kSumCols* kSumRows) void column_sum_kernel(const float* part, int n, int cols, float* dw) {
  __shared__ float s[kSumRows][kSumCols];
  const int c = blockIdx.x * kSumCols + threadIdx.x % kSumCols, g = threadIdx.x / kSumCols;
  float a = 0.f;
  if (c < cols) {
#pragma unroll 8
    for (int i = g; i < n; i += kSumRows) a += part[(int64_t)i * cols + c];
  }
  s[g][threadIdx.x % kSumCols] = a;
  __syncthreads();
  if (g == 0 && c < cols) {
    a = 0.f;
#pragma unroll 8
    for (int i = 0; i < kSumRows; ++i) a += s[i][threadIdx.x];
    dw[c] = a;
  }
}

int cdiv(int a, int b) { return (a + b - 1) / b; }

// Threads of a row and chunks of a thread: a wave up to 128 chunks (1024 columns), else two chunks
// a thread and as many waves as that takes, up to 16384 columns. (16768 x 4096 bf16 with residual
// and e4m3 output: 256 threads x 2 chunks 80 us, 512 x 1 93, 128 x 4 80.)
// With few rows one chunk a thread: the row's time is its latency (1 x 4096: 3.2 us, with two 3.7).
constexpr int kFewRows = 256;
template <typename F>
bool with_shape(int rows, int chunks, F&& f) {
  if (chunks <= 64) f(std::true_type{}, std::integral_constant<int, 1>{}, 64);
  else if (chunks <= 128) f(std::true_type{}, std::integral_constant<int, 2>{}, 64);
  else if (rows <= kFewRows && chunks <= 1024) f(std::false_type{}, std::integral_constant<int, 1>{}, cdiv(chunks, 64) * 64);
  else if (chunks <= 2048) f(std::false_type{}, std::integral_constant<int, 2>{}, cdiv(chunks, 128) * 64);
  else return false;
  return true;
}

// How a call's rows pass the caches (STREAM): 0 through them; past them, where it moves more bytes than
// they hold, 2 both ways or 1 only what it writes. 2 needs rows of whole lines: past the caches a line
// that two waves share is fetched twice (norm gradients 8192 x 5000 f16: 70 us with 1, 75 with 2, 82
// with 0; norm 16768 x 4096 bf16 to e4m3: 84 with 1, 80 with 2, 88 with 0). An fp32 chunk is two
// 16-byte accesses to one line: 0 (norm 16384 x 4096: 189 us, with 2 203).
int stream_mode(int64_t elements, int bytes, int64_t strides) {
  if (bytes != 2 || elements * bytes <= kCacheBytes) return 0;
  return strides % 64 ? 1 : 2;
}
// Call f with whether rows are whole chunks, and STREAM.
template <typename T, typename F>
void by_rows(int cols, int stream, F&& f) {
  using One = std::integral_constant<int, 1>;
  using Two = std::integral_constant<int, 2>;
  using Zero = std::integral_constant<int, 0>;
  if (cols % 8) f(std::false_type{}, Zero{});
  else if (sizeof(T) == 4 || stream == 0) f(std::true_type{}, Zero{});
  else if constexpr (sizeof(T) == 2) stream == 1 ? f(std::true_type{}, One{}) : f(std::true_type{}, Two{});
}

template <typename T, int FMT>
void launch_norm(NormParams p, int stream, hipStream_t s) {
  // (ranges of rows, a multiple of the four of a workgroup: a grid has below 2^32 threads)
  constexpr int kMostThreads = 1 << 30;
  auto ranges = [&](int threads, auto&& launch) {
    const int per = kMostThreads / threads;
    for (p.row0 = 0;; p.row0 += per) {
      launch(p.rows - p.row0 < per ? p.rows - p.row0 : per);
      if (p.rows - p.row0 <= per) break;
    }
  };
  const bool done = with_shape(p.rows, p.nb * 4, [&](auto wave, auto ch, int threads) {
    constexpr bool WAVE = decltype(wave)::value;
    constexpr int CH = decltype(ch)::value;
    ranges(WAVE ? 64 : 1024, [&](int rows) {
      const unsigned g = (unsigned)(WAVE ? cdiv(rows, 4) : rows), n = WAVE ? 256 : threads;
      by_rows<T>(p.cols, stream, [&](auto whole, auto past) {
        rmsnorm_kernel<T, WAVE, CH, FMT, decltype(whole)::value, decltype(past)::value><<<g, n, 0, s>>>(p);
      });
    });
  });
  if (!done) ranges(1024, [&](int rows) { rmsnorm_long_kernel<T, FMT><<<rows, 1024, 0, s>>>(p); });
}

// Rows of partial sums: the workgroups that run at once, with `waves` waves a compute unit, at most 16
// MB of sums up to 16384 columns. 8 waves where the next row is loaded ahead and rows are read through the
// caches (4096 x 4096 bf16 with dres 28.3 us, 16 waves 30.1; 8192 x 4096 without 37.5 and 39.4), else 16: past the
// caches that is 95.9 us at 8192 x 8192 bf16 with dres (8 waves 102), though 8 would be a little faster
// without dres (75.4 and 73.8) and in shorter rows (16768 x 4096 with dres 102 and 97).
int grad_parts(int rows, int cols, int waves) {
  int n = 256;
  with_shape(rows, cdiv(cols, 8), [&](auto, auto, int threads) { n = 256 * (waves * 64 > threads ? waves * 64 / threads : 1); });
  n = n < 2048 ? n : 2048;
  return rows < n ? rows : n;
}

template <typename T>
void launch_grad(const NormGradParams& p, int stream, int parts, hipStream_t s) {
  const bool done = with_shape(p.rows, cdiv(p.cols, 8), [&](auto wave, auto ch, int threads) {
    constexpr bool WAVE = decltype(wave)::value;
    constexpr int CH = decltype(ch)::value;
    by_rows<T>(p.cols, stream, [&](auto whole, auto past) {
      rmsnorm_grad_kernel<T, WAVE, CH, decltype(whole)::value, decltype(past)::value><<<parts, threads, 0, s>>>(p);
    });
  });
  if (!done) rmsnorm_grad_long_kernel<T><<<parts, 1024, 0, s>>>(p);
}

int type_bytes(int32_t t) { return t == GEMM_DT_F32 ? 4 : ((t == GEMM_DT_F16 || t == GEMM_DT_BF16) ? 2 : 0); }

constexpr int32_t kMaxExtent = 1 << 30, kMaxCols = 1 << 24;

gemm_status check_sizes(const char* fn, int32_t rows, int32_t cols, int32_t type) {
  if (rows < 0 || cols < 1) return fail(GEMM_ERR_INVALID_ARG, "%s: rows >= 0 and cols >= 1 expected", fn);
  if (rows > kMaxExtent || cols > kMaxCols) return fail(GEMM_ERR_UNSUPPORTED, "%s: more than 2^30 rows or 2^24 columns", fn);
  if (!type_bytes(type)) return fail(GEMM_ERR_INVALID_ARG, "%s: the type must be F16, BF16 or F32", fn);
  return GEMM_OK;
}
// A matrix argument (given): its leading dimension and alignment.
gemm_status check_arg(const char* fn, const char* name, const void* p, int64_t ld, int32_t rows, int32_t cols, int es) {
  if (!p) return fail(GEMM_ERR_INVALID_ARG, "%s: NULL %s", fn, name);
  if ((uintptr_t)p % es) return fail(GEMM_ERR_ALIGNMENT, "%s: %s not aligned to its elements", fn, name);
  if (ld < 0 || ld > ((int64_t)1 << 48)) return fail(GEMM_ERR_UNSUPPORTED, "%s: leading dimension of %s outside [0, 2^48]", fn, name);
  if (rows > 1 && ld < cols) return fail(GEMM_ERR_INVALID_ARG, "%s: leading dimension of %s below its columns", fn, name);
  return GEMM_OK;
}

#define CHECK(x)                       \
  do {                                 \
    const gemm_status st_ = (x);       \
    if (st_ != GEMM_OK) return st_;    \
  } while (0)

}  // namespace
}  // namespace gep

using namespace gep;

extern "C" {

gemm_status rmsnorm_forward(const rmsnorm_args* a, void* stream) {
  const char* fn = "rmsnorm_forward";
  if (!a) return fail(GEMM_ERR_INVALID_ARG, "%s: NULL args", fn);
  CHECK(check_sizes(fn, a->rows, a->cols, a->type));
  if (!(a->eps >= 0.f)) return fail(GEMM_ERR_INVALID_ARG, "%s: eps must be >= 0", fn);
  // (the address of an empty matrix is NULL)
  if (a->rows > 0 && !a->y && !a->q_codes) return fail(GEMM_ERR_INVALID_ARG, "%s: neither y nor q_codes given", fn);
  if ((a->q_codes != nullptr) != (a->q_scales != nullptr)) return fail(GEMM_ERR_INVALID_ARG, "%s: q_codes and q_scales come together", fn);
  if (a->h_out && !a->residual) return fail(GEMM_ERR_INVALID_ARG, "%s: h_out without a residual (h is x)", fn);
  if (a->q_codes && a->q_format != MX_E2M1 && a->q_format != MX_E4M3) return fail(GEMM_ERR_INVALID_ARG, "%s: unknown format %d", fn, a->q_format);
  const int es = type_bytes(a->type);
  if (a->rows > 0) {
    CHECK(check_arg(fn, "x", a->x, a->ldx, a->rows, a->cols, es));
    CHECK(check_arg(fn, "weight", a->weight, a->cols, a->rows, a->cols, es));
    if (a->residual) CHECK(check_arg(fn, "residual", a->residual, a->ldr, a->rows, a->cols, es));
    if (a->h_out) CHECK(check_arg(fn, "h_out", a->h_out, a->ldh, a->rows, a->cols, es));
    if (a->y) CHECK(check_arg(fn, "y", a->y, a->ldy, a->rows, a->cols, es));
    if ((uintptr_t)a->q_codes & 15) return fail(GEMM_ERR_ALIGNMENT, "%s: q_codes not 16-byte aligned", fn);
    if ((uintptr_t)a->rstd & 3) return fail(GEMM_ERR_ALIGNMENT, "%s: rstd not 4-byte aligned", fn);
    if (a->h_out == a->x && a->h_out && a->ldh != a->ldx) return fail(GEMM_ERR_INVALID_ARG, "%s: h_out in the place of x needs its leading dimension", fn);
    if (a->h_out == a->residual && a->h_out && a->ldh != a->ldr) return fail(GEMM_ERR_INVALID_ARG, "%s: h_out in the place of residual needs its leading dimension", fn);
    if (a->y && (a->y == a->x || a->y == a->residual || a->y == a->h_out)) return fail(GEMM_ERR_INVALID_ARG, "%s: y in the place of x, residual or h_out", fn);
  }
  clear_error();
  if (a->rows == 0) return GEMM_OK;
  NormParams p;
  p.x = a->x; p.r = a->residual; p.w = a->weight; p.h = a->h_out; p.y = a->y;
  p.codes = (uint8_t*)a->q_codes; p.scales = (uint8_t*)a->q_scales; p.rstd = a->rstd;
  p.ldx = a->ldx; p.ldr = a->ldr; p.ldh = a->ldh; p.ldy = a->ldy;
  p.rows = a->rows; p.cols = a->cols;
  p.nb = cdiv(a->cols, kMxBlock);
  p.nsb = cdiv(p.nb, kMxScaleBlocks);
  p.eps = a->eps;
  p.inv_cols = 1.0 / a->cols;
  const int tensors = 1 + (a->residual ? 1 : 0) + (a->h_out ? 1 : 0) + (a->y ? 1 : 0);
  const int stream_past = stream_mode((int64_t)a->rows * a->cols * tensors, es, a->cols | a->ldx | (a->residual ? a->ldr : 0));
  with_type(a->type, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    if (!a->q_codes) launch_norm<T, kNoMx>(p, stream_past, (hipStream_t)stream);
    else if (a->q_format == MX_E2M1) launch_norm<T, MX_E2M1>(p, stream_past, (hipStream_t)stream);
    else launch_norm<T, MX_E4M3>(p, stream_past, (hipStream_t)stream);
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(GEMM_ERR_HIP, "%s launch: %s", fn, hipGetErrorString(e));
  return GEMM_OK;
}

int64_t rmsnorm_backward_workspace(int32_t rows, int32_t cols) {
  if (rows < 0 || cols < 0 || rows > kMaxExtent || cols > kMaxCols) return -1;
  return (int64_t)grad_parts(rows, cols, 16) * cols * 4;
}

gemm_status rmsnorm_backward(const rmsnorm_backward_args* a, void* stream) {
  const char* fn = "rmsnorm_backward";
  if (!a) return fail(GEMM_ERR_INVALID_ARG, "%s: NULL args", fn);
  CHECK(check_sizes(fn, a->rows, a->cols, a->type));
  if (!a->dw) return fail(GEMM_ERR_INVALID_ARG, "%s: NULL dw", fn);
  if ((uintptr_t)a->dw & 3) return fail(GEMM_ERR_ALIGNMENT, "%s: dw not 4-byte aligned", fn);
  const int es = type_bytes(a->type);
  if (a->rows > 0) {
    CHECK(check_arg(fn, "dy", a->dy, a->lddy, a->rows, a->cols, es));
    CHECK(check_arg(fn, "h", a->h, a->ldh, a->rows, a->cols, es));
    CHECK(check_arg(fn, "weight", a->weight, a->cols, a->rows, a->cols, es));
    CHECK(check_arg(fn, "rstd", a->rstd, 1, 1, 1, 4));
    CHECK(check_arg(fn, "dx", a->dx, a->lddx, a->rows, a->cols, es));
    if (a->dres) CHECK(check_arg(fn, "dres", a->dres, a->lddres, a->rows, a->cols, es));
    const int64_t need = rmsnorm_backward_workspace(a->rows, a->cols);
    if (!a->workspace || a->workspace_bytes < need)
      return fail(GEMM_ERR_INVALID_ARG, "%s: workspace of %lld bytes expected", fn, (long long)need);
    if ((uintptr_t)a->workspace & 15) return fail(GEMM_ERR_ALIGNMENT, "%s: workspace not 16-byte aligned", fn);
    if (a->dx == a->dy && a->lddx != a->lddy) return fail(GEMM_ERR_INVALID_ARG, "%s: dx in the place of dy needs its leading dimension", fn);
    if (a->dx == a->dres && a->lddx != a->lddres) return fail(GEMM_ERR_INVALID_ARG, "%s: dx in the place of dres needs its leading dimension", fn);
  }
  clear_error();
  const int stream_past = stream_mode((int64_t)a->rows * a->cols * (a->dres ? 4 : 3), es,
                                      a->cols | a->lddy | a->ldh | (a->dres ? a->lddres : 0));
  const int parts = grad_parts(a->rows, a->cols, es == 2 && a->cols % 8 == 0 && stream_past != 2 ? 8 : 16);
  hipStream_t s = (hipStream_t)stream;
  NormGradParams p;
  p.dy = a->dy; p.h = a->h; p.w = a->weight; p.dres = a->dres; p.rstd = a->rstd; p.dx = a->dx;
  p.part = (float*)a->workspace;
  p.lddy = a->lddy; p.ldh = a->ldh; p.lddres = a->lddres; p.lddx = a->lddx;
  p.rows = a->rows; p.cols = a->cols;
  p.inv_cols = 1.f / (float)a->cols;
  if (parts > 0) with_type(a->type, [&](auto* t) { launch_grad<std::remove_pointer_t<decltype(t)>>(p, stream_past, parts, s); });
  column_sum_kernel<<<cdiv(a->cols, kSumCols), kSumCols * kSumRows, 0, s>>>(p.part, parts, a->cols, a->dw);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(GEMM_ERR_HIP, "%s launch: %s", fn, hipGetErrorString(e));
  return GEMM_OK;
}

}  // extern "C"
