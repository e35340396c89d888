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

// ---- chunks of 8 elements of a row of n elements of T (_Float16, __bf16 or float), at the
// alignment of the element: rows of an odd length start anywhere, and gfx950 takes 16-byte
// accesses at such addresses.
typedef uint32_t Words __attribute__((ext_vector_type(4)));
typedef uint32_t Words2 __attribute__((ext_vector_type(4), aligned(2)));

// The registers of a loaded chunk.
template <typename T>
struct Chunk {
  static constexpr int kW = (int)sizeof(T) * 2;
  uint32_t w[kW];
};

// Load elements [c, c + 8) of a row. The load itself has no branch, so that a thread's loads go out
// together: a chunk that reaches past the end loads the row's last 8 elements instead, and settle
// moves them into place. WHOLE: n is a multiple of 8 and not 0. STREAM: not to be kept in the caches
// (operands of a call that moves more than they hold).
template <bool WHOLE, bool STREAM = false, typename T>
__device__ __forceinline__ Chunk<T> load_chunk(const T* row, int c, int n) {
  Chunk<T> k;
  if (WHOLE || n >= 8) {  // (the same in every thread)
    const T* p = row + (c + 8 <= n ? c : n - 8);
#pragma unroll
    for (int i = 0; i < Chunk<T>::kW; i += 4) {
      Words x;
      if constexpr (STREAM) x = __builtin_nontemporal_load((const Words2*)p + i / 4);
      else x = *((const Words2*)p + i / 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) k.w[i + e] = x[e];
    }
  } else {
    T e[8] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < n) e[i] = row[c + i];
    __builtin_memcpy(k.w, e, sizeof(e));
  }
  return k;
}

// The chunk as fp32.
template <typename T>
__device__ __forceinline__ void unpack(const Chunk<T>& k, float v[8]) {
  T e[8];
  __builtin_memcpy(e, k.w, sizeof(e));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (float)e[i];
}
// After load_chunk(row, c, n): a chunk that reaches past the end gets its elements into place, zeros
// behind them. To be called once per loaded chunk, before unpack.
template <bool WHOLE, typename T>
__device__ __forceinline__ void settle(Chunk<T>& k, int c, int n) {
  if constexpr (WHOLE) {
#pragma unroll
    for (int i = 0; i < Chunk<T>::kW; ++i) k.w[i] = c < n ? k.w[i] : 0u;
  } else if (c + 8 > n && n >= 8) {
    const int s = c + 8 - n;  // places to move down
    T v[8];
    __builtin_memcpy(v, k.w, sizeof(v));
#pragma unroll
    for (int st = 4; st > 0; st >>= 1)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = (s & st) ? (e + st < 8 ? v[e + st] : (T)0.f) : v[e];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = s >= 8 ? (T)0.f : v[e];
    __builtin_memcpy(k.w, v, sizeof(v));
  }
}
// The chunk's registers as values the compiler knows nothing about: what is unpacked from them
// after this is unpacked again, not kept in fp32 (twice the registers) from before.
template <typename T>
__device__ __forceinline__ void forget(Chunk<T>& k) {
#pragma unroll
  for (int i = 0; i < Chunk<T>::kW; ++i) asm volatile("" : "+v"(k.w[i]));
}
template <bool WHOLE, typename T>
__device__ __forceinline__ void load8(const T* row, int c, int n, float v[8]) {
  Chunk<T> k = load_chunk<WHOLE>(row, c, n);
  settle<WHOLE>(k, c, n);
  unpack(k, v);
}
// Eight values rounded to T.
template <typename T>
__device__ __forceinline__ Chunk<T> pack(const float v[8]) {
  Chunk<T> k;
  T e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = (T)v[i];
  __builtin_memcpy(k.w, e, sizeof(e));
  return k;
}
// Store a chunk of unshifted elements; those past the end of the row are not written.
template <bool WHOLE, bool STREAM = false, typename T>
__device__ __forceinline__ void store_chunk(T* row, int c, int n, const Chunk<T>& k) {
  if (c + 8 <= n) {
#pragma unroll
    for (int i = 0; i < Chunk<T>::kW; i += 4) {
      const Words x = {k.w[i], k.w[i + 1], k.w[i + 2], k.w[i + 3]};
      if constexpr (STREAM) __builtin_nontemporal_store(x, (Words2*)(row + c) + i / 4);
      else *((Words2*)(row + c) + i / 4) = x;
    }
  } else if (!WHOLE && c < n) {
    T e[8];
    __builtin_memcpy(e, k.w, sizeof(e));
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < n) row[c + i] = e[i];
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

// The codes of row r, and the scale of its block 0 (block b: (b / 16) * 1024 + b % 16 bytes further).
template <int FMT>
__device__ __forceinline__ uint8_t* mx_code_row(uint8_t* codes, int64_t r, int nb) {
  return codes + r * nb * (FMT == MX_E4M3 ? 32 : 16);
}
__device__ __forceinline__ uint8_t* mx_scale_row(uint8_t* scales, int64_t r, int nsb) {
  return scales + ((r / kMxScaleRows) * nsb * kMxScaleRows + r % kMxScaleRows) * kMxScaleBlocks;
}
__device__ __forceinline__ int mx_scale_offset(int b) {
  return (b / kMxScaleBlocks) * (kMxScaleRows * kMxScaleBlocks) + b % kMxScaleBlocks;
}

// Quantise and store chunk `ch` of a row (8 values, in the lanes of one quad the 32 of a block): its
// codes, the block's scale (by the quad's first lane) and, after the row's last block, zero scales up
// to a whole tile. nb blocks a row, nsb = ceil(nb / 16).
template <int FMT>
__device__ __forceinline__ void mx_store_chunk(const float v[8], int ch, int nb, int nsb, uint8_t* code_row,
                                               uint8_t* scale_row) {
  const uint32_t am = quad_max(amax_bits(v));
  float inv;
  const uint32_t s = mx_scale<FMT>(am, inv);
  const uint2 w = mx_codes8<FMT>(v, inv, s == 255u);
  if constexpr (FMT == MX_E4M3) *(uint2*)(code_row + ch * 8) = w;
  else *(uint32_t*)(code_row + ch * 4) = w.x;
  const int b = ch >> 2;
  if ((ch & 3) == 0) {
    scale_row[mx_scale_offset(b)] = (uint8_t)s;
    if (b == nb - 1)
      for (int q = nb; q < nsb * kMxScaleBlocks; ++q) scale_row[mx_scale_offset(q)] = 0;
  }
}

// A call that moves more bytes than the card's last-level cache holds may read and write past the
// caches: what it would leave there would be replaced before its next use. (Norm gradients 8192 x 8192 bf16
// and a copy of dx behind them: 157 us through the caches, 142 past them. Smaller ones gain nothing: 2048 x
// 4096, 67 MB, and the copy 24.9 and 25.2.)
constexpr int64_t kCacheBytes = 256 << 20;

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
