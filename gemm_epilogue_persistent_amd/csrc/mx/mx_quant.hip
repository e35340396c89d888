// MX quantiser and its inverse (mx_quantize, mx_dequantize of the public header).
//
// Both are bound by memory: the input is read once, codes and scales (8.25 or 4.25 bits a value)
// are written once, and a value costs about ten vector instructions. 8192 x 8192 bf16 to e2m1: 33 us
// (172 MB, 5.2 TB/s); back to bf16 26 us (6.6 TB/s, part of it from the last-level cache). A torch copy of 4
// GiB reaches 4.7 TB/s.
#include <type_traits>

#include "mx_common.hpp"

namespace gep {
gemm_status fail(gemm_status st, const char* fmt, ...);
void clear_error();

namespace {

constexpr int kThreads = 256;

// ---- blocks along a row. A thread takes a chunk of 8 values (16 or 32 bytes), the four lanes of
// a quad a block: the maximum crosses lanes by DPP, loads and stores are contiguous over the
// wave. Chunks are numbered row by row over rows [r0, r0 + rows) (below 2^31 in one launch).
template <typename T, int FMT, bool WHOLE>
__global__ __launch_bounds__(kThreads) void quantize_rows_kernel(const T* x, int64_t ldx, int64_t r0, int cols, int nb,
                                                                 int nsb, uint32_t n, FastDiv fd_cpr, uint8_t* codes,
                                                                 uint8_t* scales) {
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= n) return;  // (n is a multiple of 4: quads leave together)
  uint32_t rr, ch;
  fd_divmod(fd_cpr, i, rr, ch);
  const int64_t r = r0 + rr;
  float v[8];
  load8<WHOLE>(x + r * ldx, (int)ch * 8, cols, v);
  mx_store_chunk<FMT>(v, (int)ch, nb, nsb, mx_code_row<FMT>(codes, r, nb), mx_scale_row(scales, r, nsb));
}

// ---- blocks along a column. A workgroup takes kTB blocks of 32 rows by kRowDw dwords of columns:
// the rows are read 16 bytes a lane into LDS; then each thread holds one dword column (two
// 16-bit columns or one fp32 column) of one block in registers, kTB neighbouring lanes the kTB
// blocks of a column, so that they write kTB x 32 (E4M3) or 16 (E2M1) contiguous bytes of an
// output row. Each block starts 64 / kTB dwords further in LDS, so the 64 / kTB dword columns x kTB
// blocks that a wave reads are distinct modulo 64 dwords. (Not modulo 32: two blocks' columns meet there, and
// each read is counted with two conflict cycles, 0.33 M of the 0.99 M LDS cycles of the first call below.) 5001
// x 4104 f16 to e4m3: 14.7 us in a graph of such calls (62 MB, 4.2 TB/s), 16 us with other kernels between them;
// 4096 x 4096 bf16 10.3 and 12.8 us: its 1024 workgroups all run at once, so that the card first only reads
// and then only writes.
template <typename T, int FMT, int kTB, int kRowDw>
__global__ __launch_bounds__(kTB* kRowDw) void quantize_cols_kernel(const T* x, int64_t ldx, int rows, int cols, int nb,
                                                                 int nsb, uint32_t first, uint32_t tiles, FastDiv fd_ty,
                                                                 uint8_t* codes, uint8_t* scales) {
  constexpr int kVec = 16 / (int)sizeof(T);     // elements of a 16-byte load
  constexpr int kCols = kRowDw * 4 / (int)sizeof(T);   // columns of a tile
  constexpr int kTR = kTB * kMxBlock, kSkewDw = 64 / kTB;
  constexpr int kTileDw = kTR * kRowDw + kTB * kSkewDw;
  constexpr int kLR = kRowDw / 4;                // lanes of a row
  constexpr int kRP = kTB * kRowDw / kLR;       // rows of a pass
  constexpr int kPer = 4 / (int)sizeof(T);      // columns of a dword
  __shared__ __attribute__((aligned(16))) uint32_t tile[kTileDw];
  const int tid = threadIdx.x;
  // Workgroups go to the eight XCDs in turn; each XCD takes a run of tiles down the rows, so that
  // the lines of the output that two tiles share are put together in one L2. This launch has tiles
  // first, ..., first + tiles - 1.
  const uint32_t per = (tiles + 7) >> 3, i = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if (i >= tiles) return;
  uint32_t bx, by;
  fd_divmod(fd_ty, first + i, bx, by);
  const int r0 = (int)by * kTR, c0 = (int)bx * kCols;
  uint4 in[kTR / kRP];
  const int lc = c0 + (tid % kLR) * kVec;
#pragma unroll
  for (int q = 0; q < kTR / kRP; ++q) {
    const int r = r0 + q * kRP + tid / kLR;
    in[q] = uint4{0, 0, 0, 0};
    if (r < rows) {
      const T* p = x + (int64_t)r * ldx + lc;
      if (lc + kVec <= cols) {
        __builtin_memcpy(&in[q], (const void*)p, 16);
      } else {
        T e[kVec] = {};
#pragma unroll
        for (int k = 0; k < kVec; ++k)
          if (lc + k < cols) e[k] = p[k];
        __builtin_memcpy(&in[q], e, 16);
      }
    }
  }
#pragma unroll
  for (int q = 0; q < kTR / kRP; ++q) {
    const int r = q * kRP + tid / kLR;
    *(uint4*)(tile + r * kRowDw + (r / kMxBlock) * kSkewDw + (tid % kLR) * 4) = in[q];
  }
  __syncthreads();
  const int blk = tid % kTB, dc = tid / kTB;  // block of the tile, dword column
  const int b = (int)by * kTB + blk;
  const uint32_t* col = tile + blk * (kMxBlock * kRowDw + kSkewDw) + dc;
  uint32_t w[kMxBlock];
#pragma unroll
  for (int i = 0; i < kMxBlock; ++i) w[i] = col[i * kRowDw];
  if (b >= nb) return;
#pragma unroll
  for (int h = 0; h < kPer; ++h) {
    const int c = c0 + dc * kPer + h;
    if (c >= cols) break;
    float v[kMxBlock];
    uint32_t am = 0;
#pragma unroll
    for (int i = 0; i < kMxBlock; ++i) {
      if constexpr (sizeof(T) == 4) {
        v[i] = __uint_as_float(w[i]);
      } else {
        T e[2];
        __builtin_memcpy(e, &w[i], 4);
        v[i] = (float)e[h];
      }
      am = max(am, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    }
    float inv;
    const uint32_t s = mx_scale<FMT>(am, inv);
    uint32_t o[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint2 p = mx_codes8<FMT>(v + 8 * j, inv, s == 255u);
      if constexpr (FMT == MX_E4M3) {
        o[2 * j] = p.x;
        o[2 * j + 1] = p.y;
      } else {
        o[j] = p.x;
      }
    }
    if constexpr (FMT == MX_E4M3) {
      uint4* dst = (uint4*)(codes + ((int64_t)c * nb + b) * 32);
      dst[0] = uint4{o[0], o[1], o[2], o[3]};
      dst[1] = uint4{o[4], o[5], o[6], o[7]};
    } else {
      *(uint4*)(codes + ((int64_t)c * nb + b) * 16) = uint4{o[0], o[1], o[2], o[3]};
    }
    uint8_t* scale_row = mx_scale_row(scales, c, nsb);
    scale_row[mx_scale_offset(b)] = (uint8_t)s;
    if (b == nb - 1)
      for (int q = nb; q < nsb * kMxScaleBlocks; ++q) scale_row[mx_scale_offset(q)] = 0;
  }
}

// ---- values of the codes. A thread takes 8 codes (8 or 4 bytes) and writes 8 values. (Stores past
// the caches make the call itself shorter, 4096 x 4096 e4m3 6.7 us instead of 9.3, but the next reader
// pays for it: with a copy of the values 21.5 and 20.2.)
template <typename T, int FMT>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(const uint8_t* codes, const uint8_t* scales, int64_t r0,
                                                              int k, int nb, int nsb, uint32_t n, FastDiv fd_cpr, T* out,
                                                              int64_t ldo) {
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= n) return;
  uint32_t rr, ch;
  fd_divmod(fd_cpr, i, rr, ch);
  const int64_t r = r0 + rr;
  const int s = mx_scale_row(const_cast<uint8_t*>(scales), r, nsb)[mx_scale_offset((int)ch >> 2)];
  float v[8];
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  f32x2 p[4];
  if constexpr (FMT == MX_E4M3) {
    const uint2 w = *(const uint2*)(codes + (r * nb * 4 + ch) * 8);
    p[0] = __builtin_amdgcn_cvt_pk_f32_fp8(w.x, false);
    p[1] = __builtin_amdgcn_cvt_pk_f32_fp8(w.x, true);
    p[2] = __builtin_amdgcn_cvt_pk_f32_fp8(w.y, false);
    p[3] = __builtin_amdgcn_cvt_pk_f32_fp8(w.y, true);
  } else {
    const uint32_t w = *(const uint32_t*)(codes + (r * nb * 4 + ch) * 4);
#if defined(__HIP_DEVICE_COMPILE__)
    p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 0);
    p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 1);
    p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 2);
    p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 3);
#endif
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    v[e] = s == 255 ? __uint_as_float(0x7FC00000u) : __builtin_ldexpf(p[e >> 1][e & 1], s - 127);
  store_chunk<false>(out + r * ldo, (int)ch * 8, k, pack<T>(v));
}

// Launch `f(r0, n)` over ranges of rows whose chunks number below 2^31.
template <typename F>
void row_ranges(int32_t rows, uint32_t cpr, F&& f) {
  const int64_t per = max((int64_t)1, (int64_t)0x7FFFFF00 / cpr);
  for (int64_t r0 = 0; r0 < rows; r0 += per) f(r0, (uint32_t)(min((int64_t)rows - r0, per) * cpr));
}

using E2M1 = std::integral_constant<int, MX_E2M1>;
using E4M3 = std::integral_constant<int, MX_E4M3>;

constexpr int32_t kMaxExtent = 1 << 30;

gemm_status check_matrix(const char* fn, int32_t rows, int32_t cols, int32_t type, int64_t ld, const char* name,
                         const void* p) {
  if (rows < 0 || cols < 0) return fail(GEMM_ERR_INVALID_ARG, "%s: negative size", fn);
  if (rows > kMaxExtent || cols > kMaxExtent) return fail(GEMM_ERR_UNSUPPORTED, "%s: more than 2^30 rows or columns", fn);
  const int es = type == GEMM_DT_F32 ? 4 : ((type == GEMM_DT_F16 || type == GEMM_DT_BF16) ? 2 : 0);
  if (!es) return fail(GEMM_ERR_INVALID_ARG, "%s: %s must be F16, BF16 or F32", fn, name);
  if (rows > 1 && ld < cols) return fail(GEMM_ERR_INVALID_ARG, "%s: leading dimension of %s below its columns", fn, name);
  if (ld < 0 || ld > ((int64_t)1 << 48)) return fail(GEMM_ERR_UNSUPPORTED, "%s: leading dimension of %s outside [0, 2^48]", fn, name);
  if (rows == 0 || cols == 0) return GEMM_OK;
  if (!p) return fail(GEMM_ERR_INVALID_ARG, "%s: NULL %s", fn, name);
  if ((uintptr_t)p % es) return fail(GEMM_ERR_ALIGNMENT, "%s: %s not aligned to its elements", fn, name);
  return GEMM_OK;
}
gemm_status check_mx(const char* fn, int32_t format, const void* codes, const void* scales, bool empty) {
  if (format != MX_E2M1 && format != MX_E4M3) return fail(GEMM_ERR_INVALID_ARG, "%s: unknown format %d", fn, format);
  if (empty) return GEMM_OK;
  if (!codes || !scales) return fail(GEMM_ERR_INVALID_ARG, "%s: NULL codes or scales", fn);
  if ((uintptr_t)codes & 15) return fail(GEMM_ERR_ALIGNMENT, "%s: codes not 16-byte aligned", fn);
  return GEMM_OK;
}

}  // namespace
}  // namespace gep

using namespace gep;

extern "C" {

gemm_status mx_quantize(int32_t rows, int32_t cols, const void* x, int32_t x_type, int64_t ldx, int32_t transpose,
                        int32_t format, void* codes, void* scales, void* stream) {
  const bool empty = rows == 0 || cols == 0;
  gemm_status st = check_matrix("mx_quantize", rows, cols, x_type, ldx, "x", x);
  if (st == GEMM_OK) st = check_mx("mx_quantize", format, codes, scales, empty);
  if (st != GEMM_OK) return st;
  if (transpose != 0 && transpose != 1) return fail(GEMM_ERR_INVALID_ARG, "mx_quantize: transpose must be 0 or 1");
  clear_error();
  if (empty) return GEMM_OK;
  hipStream_t s = (hipStream_t)stream;
  const int nb = ((transpose ? rows : cols) + kMxBlock - 1) / kMxBlock;
  const int nsb = (nb + kMxScaleBlocks - 1) / kMxScaleBlocks;
  uint8_t *qc = (uint8_t*)codes, *qs = (uint8_t*)scales;
  with_type(x_type, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    if (transpose) {
      // 16-bit: 256 rows x 64 columns, the longest runs of the output (5001 x 4104 f16 to e4m3 14.7 us;
      // 128 x 128 15.3, 64 x 128 15.7); fp32: 128 x 64, the longest of the input (8192 x 8192 to e2m1
      // 69 us; 256 x 32 77).
      constexpr int kTB = sizeof(T) == 2 ? 8 : 4, kRowDw = sizeof(T) == 2 ? 32 : 64, tc = kRowDw * 4 / (int)sizeof(T);
      const int64_t ty = (nb + kTB - 1) / kTB, tx = ((int64_t)cols + tc - 1) / tc;
      if (ty * tx > 0x7FFFFF00) { st = fail(GEMM_ERR_UNSUPPORTED, "mx_quantize: more than 2^31 tiles"); return; }
      const FastDiv fd = make_fastdiv((uint32_t)ty);
      constexpr int64_t most = 1 << 23;  // tiles of a launch (a grid has below 2^32 threads)
      for (int64_t first = 0; first < ty * tx; first += most) {
        const uint32_t tiles = (uint32_t)min(ty * tx - first, most), grid = (tiles + 7) / 8 * 8;
        auto go = [&](auto fmt) {
          quantize_cols_kernel<T, decltype(fmt)::value, kTB, kRowDw><<<grid, kTB * kRowDw, 0, s>>>(
              (const T*)x, ldx, rows, cols, nb, nsb, (uint32_t)first, tiles, fd, qc, qs);
        };
        format == MX_E2M1 ? go(E2M1{}) : go(E4M3{});
      }
    } else {
      const uint32_t cpr = (uint32_t)nb * 4;
      row_ranges(rows, cpr, [&](int64_t r0, uint32_t n) {
        const unsigned g = (n + kThreads - 1) / kThreads;
        auto go = [&](auto fmt, auto whole) {
          quantize_rows_kernel<T, decltype(fmt)::value, decltype(whole)::value><<<g, kThreads, 0, s>>>(
              (const T*)x, ldx, r0, cols, nb, nsb, n, make_fastdiv(cpr), qc, qs);
        };
        if (cols % 8 == 0) format == MX_E2M1 ? go(E2M1{}, std::true_type{}) : go(E4M3{}, std::true_type{});
        else format == MX_E2M1 ? go(E2M1{}, std::false_type{}) : go(E4M3{}, std::false_type{});
      });
    }
  });
  if (st != GEMM_OK) return st;
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(GEMM_ERR_HIP, "mx_quantize launch: %s", hipGetErrorString(e));
  return GEMM_OK;
}

gemm_status mx_dequantize(int32_t rows, int32_t k, int32_t format, const void* codes, const void* scales, void* out,
                          int32_t out_type, int64_t ldo, void* stream) {
  const bool empty = rows == 0 || k == 0;
  gemm_status st = check_matrix("mx_dequantize", rows, k, out_type, ldo, "out", out);
  if (st == GEMM_OK) st = check_mx("mx_dequantize", format, codes, scales, empty);
  if (st != GEMM_OK) return st;
  clear_error();
  if (empty) return GEMM_OK;
  hipStream_t s = (hipStream_t)stream;
  const int nb = (k + kMxBlock - 1) / kMxBlock, nsb = (nb + kMxScaleBlocks - 1) / kMxScaleBlocks;
  const uint32_t cpr = (uint32_t)nb * 4;
  const uint8_t *qc = (const uint8_t*)codes, *qs = (const uint8_t*)scales;
  with_type(out_type, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    row_ranges(rows, cpr, [&](int64_t r0, uint32_t n) {
      const unsigned g = (n + kThreads - 1) / kThreads;
      if (format == MX_E2M1) dequantize_kernel<T, MX_E2M1><<<g, kThreads, 0, s>>>(qc, qs, r0, k, nb, nsb, n, make_fastdiv(cpr), (T*)out, ldo);
      else dequantize_kernel<T, MX_E4M3><<<g, kThreads, 0, s>>>(qc, qs, r0, k, nb, nsb, n, make_fastdiv(cpr), (T*)out, ldo);
    });
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(GEMM_ERR_HIP, "mx_dequantize launch: %s", hipGetErrorString(e));
  return GEMM_OK;
}

}  // extern "C"
