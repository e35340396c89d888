// Shared device helpers of the MX (block-scaled) quantiser and the fused RMS norm: 8-element
// chunks of any float type at element alignment, and the rounding of one block of 32.
//
// MX block (OCP Microscaling v1.0): scale byte s = 127 + floor(log2 max|x|) - emax in [0, 254],
// element = x / 2^(s - 127) rounded to nearest even, saturated. floor(log2) of a positive fp32 is
// its exponent field minus 127, and a subnormal's is below every s >= 0, so with the field f of
// max|x|: s = max(0, f - emax). The division is an exact product with 2^(127 - s) (a
// quotient that leaves the fp32 normal range is far below half of the smallest element).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../../include/mx_mi355x.h"
#include "../params.hpp"

namespace gep {

constexpr int kMxBlock = 32;
constexpr int kMxScaleRows = 64, kMxScaleBlocks = 16;  // one scale tile, 1 KB

// Byte offset of the scale of block b of row r; nsb = ceil(blocks per row / 16).
__host__ __device__ __forceinline__ int64_t mx_scale_at(int64_t r, int b, int nsb) {
  return ((r / kMxScaleRows * nsb + b / kMxScaleBlocks) * kMxScaleRows + r % kMxScaleRows) * kMxScaleBlocks +
         b % kMxScaleBlocks;
}

struct __attribute__((packed, aligned(2))) U16x8 { uint32_t w[4]; };  // 8 16-bit elements, any even address
struct __attribute__((packed, aligned(4))) F32x8 { float w[8]; };

// T: _Float16, __bf16 or float. Eight consecutive elements to and from fp32, at the alignment
// of the element only: one (16-bit) or two (fp32) 16-byte accesses. Rows of an odd number of
// elements start at any multiple of the element size; gfx950 takes such addresses.
template <typename T>
__device__ __forceinline__ float to_f32(T v) { return (float)v; }

template <typename T>
__device__ __forceinline__ void load8(const T* p, float v[8]) {
  if constexpr (sizeof(T) == 4) {
    const F32x8 x = *(const F32x8*)p;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = x.w[e];
  } else {
    const U16x8 x = *(const U16x8*)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      T h[2];
      __builtin_memcpy(h, &x.w[i], 4);
      v[2 * i] = (float)h[0];
      v[2 * i + 1] = (float)h[1];
    }
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float v[8]) {
  if constexpr (sizeof(T) == 4) {
    F32x8 x;
#pragma unroll
    for (int e = 0; e < 8; ++e) x.w[e] = v[e];
    *(F32x8*)p = x;
  } else {
    U16x8 x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      T h[2] = {(T)v[2 * i], (T)v[2 * i + 1]};
      __builtin_memcpy(&x.w[i], h, 4);
    }
    *(U16x8*)p = x;
  }
}

// Elements [c, c + 8) of a row of n elements; those past the end read as zero / are not written.
template <typename T>
__device__ __forceinline__ void load8_tail(const T* row, int c, int n, float v[8]) {
  if (c + 8 <= n) {
    load8(row + c, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = c + e < n ? (float)row[c + e] : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void store8_tail(T* row, int c, int n, const float v[8]) {
  if (c + 8 <= n) {
    store8(row + c, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < n) row[c + e] = (T)v[e];
  }
}

// Largest magnitude of 8 values as fp32 bits without the sign (a NaN's bits are the largest).
__device__ __forceinline__ uint32_t amax_bits(const float v[8]) {
  uint32_t a = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) a = max(a, __float_as_uint(v[e]) & 0x7FFFFFFFu);
  return a;
}
// Maximum over the four lanes of a quad (lanes 4q .. 4q + 3), in each of them.
__device__ __forceinline__ uint32_t quad_max(uint32_t a) {
  a = max(a, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a, 0xB1, 0xF, 0xF, true));  // lanes 1 0 3 2
  return max(a, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a, 0x4E, 0xF, 0xF, true));  // lanes 2 3 0 1
}

// The block's scale byte, and the factor 2^(127 - s) its values are multiplied with (0 for a
// block with a NaN or an infinity, whose codes are zero under scale 255).
template <int FMT>
__device__ __forceinline__ uint32_t mx_scale(uint32_t amax, float& inv) {
  constexpr int emax = FMT == MX_E2M1 ? 2 : 8;
  const int f = (int)(amax >> 23);
  const int s = max(0, f - emax);
  inv = __uint_as_float((uint32_t)(254 - s) << 23);
  if (f == 255) {
    inv = 0.f;
    return 255u;
  }
  return (uint32_t)s;
}

// Eight scaled values as codes: 8 bytes of E4M3 or 4 bytes of E2M1. (v * 0 of a NaN or an
// infinity would be NaN: such blocks pass bad = true.) v_cvt_pk_fp8_f32 does not saturate by
// itself; the fp4 conversion does.
template <int FMT>
__device__ __forceinline__ uint2 mx_codes8(const float v[8], float inv, bool bad) {
  float c[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) c[e] = bad ? 0.f : v[e] * inv;
  uint2 w = {0u, 0u};
  if constexpr (FMT == MX_E4M3) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = __builtin_amdgcn_fmed3f(c[e], -448.f, 448.f);
    int x = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], 0, false);
    x = __builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], x, true);
    int y = __builtin_amdgcn_cvt_pk_fp8_f32(c[4], c[5], 0, false);
    y = __builtin_amdgcn_cvt_pk_fp8_f32(c[6], c[7], y, true);
    w.x = (uint32_t)x;
    w.y = (uint32_t)y;
  } else {
#if defined(__HIP_DEVICE_COMPILE__)
    w.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w.x, c[0], c[1], 1.f, 0);
    w.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w.x, c[2], c[3], 1.f, 1);
    w.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w.x, c[4], c[5], 1.f, 2);
    w.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w.x, c[6], c[7], 1.f, 3);
#endif
  }
  return w;
}

// Quantise and store chunk `ch` (8 values, in the lanes of one quad the 32 of a block) of row r:
// its codes, the block's scale (by the quad's first lane) and, after the row's last block, zero
// scales up to a whole tile. nb blocks per row, nsb = ceil(nb / 16).
template <int FMT>
__device__ __forceinline__ void mx_store_chunk(const float v[8], int64_t r, int ch, int nb, int nsb, uint8_t* codes,
                                               uint8_t* scales) {
  const uint32_t am = quad_max(amax_bits(v));
  float inv;
  const uint32_t s = mx_scale<FMT>(am, inv);
  const uint2 w = mx_codes8<FMT>(v, inv, s == 255u);
  if constexpr (FMT == MX_E4M3) *(uint2*)(codes + (r * nb * 4 + ch) * 8) = w;
  else *(uint32_t*)(codes + (r * nb * 4 + ch) * 4) = w.x;
  const int b = ch >> 2;
  if ((ch & 3) == 0) {
    scales[mx_scale_at(r, b, nsb)] = (uint8_t)s;
    if (b == nb - 1)
      for (int q = nb; q < nsb * kMxScaleBlocks; ++q) scales[mx_scale_at(r, q, nsb)] = 0;
  }
}

// Call f with a null pointer of the element type that a gemm_dtype names (F16, BF16 or F32).
template <typename F>
static inline bool with_type(int32_t dt, F&& f) {
  switch (dt) {
    case GEMM_DT_F16: f((_Float16*)nullptr); return true;
    case GEMM_DT_BF16: f((__bf16*)nullptr); return true;
    case GEMM_DT_F32: f((float*)nullptr); return true;
    default: return false;
  }
}

}  // namespace gep
