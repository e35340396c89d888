// Fused RMS norm with residual addition and MX output, and its gradients (rmsnorm_forward,
// rmsnorm_backward of the public header).
//
//   h = x + r (rounded),  rstd = (mean h^2 + eps)^(-1/2),  y = h rstd w
//   dx = rstd (p - n mean(p n)) + dres,  dw = sum_rows dy n,   n = h rstd, p = dy w
//
// Both are bound by memory. A row is held in registers from its single read to its last use:
// TPR threads x CH chunks of 8 elements, chunk j of thread t at column (t + j TPR) 8. Four
// adjacent lanes hold an MX block. Rows too long for registers take a kernel that reads them
// twice. All sums are fp32, in a fixed order.
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
  int32_t rows, cols, nb, nsb, fmt;
  float eps, inv_cols;
};

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m);
  return v;
}
// Sum over the TPR threads that share a row, in each of them (red: one float per wave).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = wave_sum(v);
  if constexpr (TPR > 64) {
    __syncthreads();  // the last use of red is over
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 64; ++i) v += red[i];
  }
  return v;
}

// The type's rounding of h, so that the statistics see the stored values.
template <typename T>
__device__ __forceinline__ float round_to(float v) { return (float)(T)v; }

template <typename T, int FMT>
__device__ __forceinline__ void norm_store(const NormParams& p, int64_t row, int ch, const float y[8]) {
  if (p.y) store8_tail((T*)p.y + row * p.ldy, ch * 8, p.cols, y);
  if (p.codes && ch < p.nb * 4) mx_store_chunk<FMT>(y, row, ch, p.nb, p.nsb, p.codes, p.scales);
}
template <typename T>
__device__ __forceinline__ void norm_out(const NormParams& p, int64_t row, int ch, const float y[8]) {
  if (p.fmt == MX_E2M1) norm_store<T, MX_E2M1>(p, row, ch, y);
  else norm_store<T, MX_E4M3>(p, row, ch, y);
}

template <typename T, int TPR, int CH>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void rmsnorm_kernel(const NormParams p) {
  constexpr int kRows = TPR < 256 ? 256 / TPR : 1;  // rows of a workgroup
  __shared__ float red[TPR > 64 ? TPR / 64 : 1];
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
  if (TPR == 64 && row >= p.rows) return;  // (a whole wave)
  const T* x = (const T*)p.x + row * p.ldx;
  float h[CH][8];
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < CH; ++j) load8_tail(x, (t + j * TPR) * 8, p.cols, h[j]);
  if (p.r) {
    const T* r = (const T*)p.r + row * p.ldr;
    float rv[CH][8];
#pragma unroll
    for (int j = 0; j < CH; ++j) load8_tail(r, (t + j * TPR) * 8, p.cols, rv[j]);
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) h[j][e] = round_to<T>(h[j][e] + rv[j][e]);
    if (p.h) {
#pragma unroll
      for (int j = 0; j < CH; ++j) store8_tail((T*)p.h + row * p.ldh, (t + j * TPR) * 8, p.cols, h[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < CH; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(h[j][e], h[j][e], ss);
  const float rstd = 1.f / sqrtf(row_sum<TPR>(ss, red) * p.inv_cols + p.eps);
  if (p.rstd && t == 0) p.rstd[row] = rstd;
  if (!p.y && !p.codes) return;
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    const int ch = t + j * TPR;
    float w[8], y[8];
    load8_tail((const T*)p.w, ch * 8, p.cols, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = h[j][e] * rstd * w[e];
    norm_out<T>(p, row, ch, y);
  }
}

// Rows of any length: one workgroup a row, read twice (the second time from the caches).
template <typename T>
__global__ __launch_bounds__(1024) void rmsnorm_long_kernel(const NormParams p) {
  __shared__ float red[16];
  const int64_t row = blockIdx.x;
  const T* x = (const T*)p.x + row * p.ldx;
  const T* r = p.r ? (const T*)p.r + row * p.ldr : nullptr;
  const int n = p.nb * 4;
  auto load_h = [&](int ch, float v[8]) {
    load8_tail(x, ch * 8, p.cols, v);
    if (r) {
      float q[8];
      load8_tail(r, ch * 8, p.cols, q);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = round_to<T>(v[e] + q[e]);
    }
  };
  float ss = 0.f;
  for (int ch = threadIdx.x; ch < n; ch += 1024) {
    float v[8];
    load_h(ch, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(v[e], v[e], ss);
  }
  const float rstd = 1.f / sqrtf(row_sum<1024>(ss, red) * p.inv_cols + p.eps);
  if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
  for (int ch = threadIdx.x; ch < n; ch += 1024) {
    float v[8], w[8], y[8];
    load_h(ch, v);
    // (h may be x or the residual: every element is read again by the thread that replaces it)
    if (r && p.h) store8_tail((T*)p.h + row * p.ldh, ch * 8, p.cols, v);
    load8_tail((const T*)p.w, ch * 8, p.cols, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = v[e] * rstd * w[e];
    norm_out<T>(p, row, ch, y);
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

template <typename T, int TPR, int CH>
__global__ __launch_bounds__(TPR) void rmsnorm_grad_kernel(const NormGradParams p) {
  __shared__ float red[TPR > 64 ? TPR / 64 : 1];
  const int t = threadIdx.x;
  float dw[CH][8], w[CH][8];
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    load8_tail((const T*)p.w, (t + j * TPR) * 8, p.cols, w[j]);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[j][e] = 0.f;
  }
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const float rstd = p.rstd[row];
    float n[CH][8], dy[CH][8];
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      load8_tail((const T*)p.h + row * p.ldh, (t + j * TPR) * 8, p.cols, n[j]);
      load8_tail((const T*)p.dy + row * p.lddy, (t + j * TPR) * 8, p.cols, dy[j]);
    }
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        n[j][e] *= rstd;
        const float dyn = dy[j][e] * n[j][e];
        dw[j][e] += dyn;
        dot = fmaf(dyn, w[j][e], dot);
      }
    const float m = row_sum<TPR>(dot, red) * p.inv_cols;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = (t + j * TPR) * 8;
      float g[8];
      if (p.dres) {
        load8_tail((const T*)p.dres + row * p.lddres, c, p.cols, g);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] = fmaf(rstd, dy[j][e] * w[j][e] - n[j][e] * m, g[e]);
      store8_tail((T*)p.dx + row * p.lddx, c, p.cols, g);
    }
  }
  float* part = p.part + (int64_t)blockIdx.x * p.cols;
#pragma unroll
  for (int j = 0; j < CH; ++j) store8_tail(part, (t + j * TPR) * 8, p.cols, dw[j]);
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
      load8_tail(h, ch * 8, p.cols, n);
      load8_tail(dyp, ch * 8, p.cols, dy);
      load8_tail((const T*)p.w, ch * 8, p.cols, w);
      if (row == blockIdx.x) {
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] = 0.f;
      } else {
        load8_tail(part, ch * 8, p.cols, s);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float dyn = dy[e] * (n[e] * rstd);
        s[e] += dyn;
        dot = fmaf(dyn, w[e], dot);
      }
      store8_tail(part, ch * 8, p.cols, s);
    }
    const float m = row_sum<1024>(dot, red) * p.inv_cols;
    for (int ch = threadIdx.x; ch < n8; ch += 1024) {
      float n[8], dy[8], w[8], g[8];
      load8_tail(h, ch * 8, p.cols, n);
      load8_tail(dyp, ch * 8, p.cols, dy);
      load8_tail((const T*)p.w, ch * 8, p.cols, w);
      if (p.dres) {
        load8_tail((const T*)p.dres + row * p.lddres, ch * 8, p.cols, g);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] = fmaf(rstd, dy[e] * w[e] - n[e] * rstd * m, g[e]);
      store8_tail((T*)p.dx + row * p.lddx, ch * 8, p.cols, g);
    }
  }
}

// dw = sum of `n` rows of partial sums: 64 columns a workgroup, 16 threads a row strip.
constexpr int kSumCols = 64, kSumRows = 16;
__global__ __launch_bounds__(kSumCols* kSumRows) void column_sum_kernel(const float* part, int n, int cols, float* dw) {
  __shared__ float s[kSumRows][kSumCols];
  const int c = blockIdx.x * kSumCols + threadIdx.x % kSumCols, g = threadIdx.x / kSumCols;
  float a = 0.f;
  if (c < cols) {
#pragma unroll 4
    for (int i = g; i < n; i += kSumRows) a += part[(int64_t)i * cols + c];
  }
  s[g][threadIdx.x % kSumCols] = a;
  __syncthreads();
  if (g == 0 && c < cols) {
    a = 0.f;
#pragma unroll
    for (int i = 0; i < kSumRows; ++i) a += s[i][threadIdx.x];
    dw[c] = a;
  }
}

int cdiv(int a, int b) { return (a + b - 1) / b; }

template <typename T>
void launch_norm(const NormParams& p, hipStream_t s) {
  // Threads of a row: a wave up to 4096 columns when there are rows enough to fill the card
  // with waves, else a workgroup.
  const int ch = p.nb * 4;
  auto go = [&](auto tpr, auto n) {
    constexpr int TPR = decltype(tpr)::value, CH = decltype(n)::value;
    constexpr int rows = TPR < 256 ? 256 / TPR : 1;
    rmsnorm_kernel<T, TPR, CH><<<cdiv(p.rows, rows), TPR < 256 ? 256 : TPR, 0, s>>>(p);
  };
#define GO(TPR, CH) go(std::integral_constant<int, TPR>{}, std::integral_constant<int, CH>{})
  if (ch <= 64) GO(64, 1);
  else if (ch <= 128 && p.rows >= 1024) GO(64, 2);
  else if (ch <= 256 && p.rows >= 1024) GO(64, 4);
  else if (ch <= 512 && p.rows >= 1024) GO(64, 8);
  else if (ch <= 256) GO(256, 1);
  else if (ch <= 512) GO(256, 2);
  else if (ch <= 1024) GO(256, 4);
  else if (ch <= 2048) GO(1024, 2);
  else if (ch <= 4096) GO(1024, 4);
  else rmsnorm_long_kernel<T><<<p.rows, 1024, 0, s>>>(p);
#undef GO
}

// Rows of partial sums: enough workgroups to fill the card, at most 16 MB of sums up to 16384
// columns.
int grad_parts(int rows, int cols) {
  int n = cols > 0 ? (1 << 22) / cols : 2048;
  n = n < 256 ? 256 : (n > 2048 ? 2048 : n);
  return rows < n ? rows : n;
}

template <typename T>
void launch_grad(const NormGradParams& p, int parts, hipStream_t s) {
  const int ch = cdiv(p.cols, 8);
#define GO(TPR, CH) rmsnorm_grad_kernel<T, TPR, CH><<<parts, TPR, 0, s>>>(p)
  if (ch <= 64) GO(64, 1);
  else if (ch <= 128) GO(64, 2);
  else if (ch <= 256) GO(256, 1);
  else if (ch <= 512) GO(256, 2);
  else if (ch <= 1024) GO(256, 4);
  else if (ch <= 2048) GO(1024, 2);
  else if (ch <= 4096) GO(1024, 4);
  else rmsnorm_grad_long_kernel<T><<<parts, 1024, 0, s>>>(p);
#undef GO
}

int type_bytes(int32_t t) { return t == GEMM_DT_F32 ? 4 : ((t == GEMM_DT_F16 || t == GEMM_DT_BF16) ? 2 : 0); }

constexpr int32_t kMaxExtent = 1 << 30;

gemm_status check_sizes(const char* fn, int32_t rows, int32_t cols, int32_t type) {
  if (rows < 0 || cols < 1) return fail(GEMM_ERR_INVALID_ARG, "%s: rows >= 0 and cols >= 1 expected", fn);
  if (rows > kMaxExtent || cols > kMaxExtent) return fail(GEMM_ERR_UNSUPPORTED, "%s: more than 2^30 rows or columns", fn);
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
  if (!a->y && !a->q_codes) return fail(GEMM_ERR_INVALID_ARG, "%s: neither y nor q_codes given", fn);
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
  p.fmt = a->q_codes ? a->q_format : MX_E4M3;
  p.eps = a->eps;
  p.inv_cols = 1.f / (float)a->cols;
  with_type(a->type, [&](auto* t) { launch_norm<std::remove_pointer_t<decltype(t)>>(p, (hipStream_t)stream); });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(GEMM_ERR_HIP, "%s launch: %s", fn, hipGetErrorString(e));
  return GEMM_OK;
}

int64_t rmsnorm_backward_workspace(int32_t rows, int32_t cols) {
  if (rows < 0 || cols < 0) return -1;
  return (int64_t)grad_parts(rows, cols) * cols * 4;
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
  const int parts = grad_parts(a->rows, a->cols);
  hipStream_t s = (hipStream_t)stream;
  NormGradParams p;
  p.dy = a->dy; p.h = a->h; p.w = a->weight; p.dres = a->dres; p.rstd = a->rstd; p.dx = a->dx;
  p.part = (float*)a->workspace;
  p.lddy = a->lddy; p.ldh = a->ldh; p.lddres = a->lddres; p.lddx = a->lddx;
  p.rows = a->rows; p.cols = a->cols;
  p.inv_cols = 1.f / (float)a->cols;
  if (parts > 0) with_type(a->type, [&](auto* t) { launch_grad<std::remove_pointer_t<decltype(t)>>(p, parts, s); });
  column_sum_kernel<<<cdiv(a->cols, kSumCols), kSumCols * kSumRows, 0, s>>>(p.part, parts, a->cols, a->dw);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(GEMM_ERR_HIP, "%s launch: %s", fn, hipGetErrorString(e));
  return GEMM_OK;
}

}  // extern "C"
