// Shared device helpers of the 8-bit operators with a scale per 128 values: the factor of a block and the
// rounding of its values.
//
// Of a block's largest magnitude a: r = 448 / a in fp32, 2^126 at most, cut to 13 significant bits; a code is x r
// rounded to nearest even, and scale = 1 / r in fp32. Why 13 bits: an F16 value has 11 and a BF16 value 8, so x r is
// exact in fp32 and the conversion to a code is its only rounding. (With r in full, or with the quotient by
// a / 448, fp32 rounds the product onto a border between two codes for 1 in 2^20 of random values and for
// percents of 16-bit ones, whose quotients x / a are simple fractions; a repair costs about ten vector
// instructions a value, where the plain form takes three. Measured with r in full and the repair: 16768 x 4096
// bf16 along rows 42 to 49 us for 39 to 41, 8192 x 8192 by tiles both ways 56.5 for 54.0, 5001 x 4104 f16 both
// ways 25.7 for 21.6, 16768 x 4096 SiLU with saved and q 67.8 for 59.9.) fp32 values take the repair: see fp8_scaled.
#pragma once
#include "../../../include/fp8_mi355x.h"
#include "../mx/mx_common.hpp"

namespace gep {

constexpr int kFp8Block = 128;

// The block's factor r (0 for one with a NaN or an infinity, whose codes are zero) and its scale, from its largest
// magnitude (NaN if there is one).
struct Fp8Factor {
  float r, scale;
};
__device__ __forceinline__ float fp8_factor(float amax) {
  const float r = fminf(448.f / amax, 0x1p126f);  // (correctly rounded; 448 / 0 is infinite)
  return __uint_as_float(__float_as_uint(r) & 0xFFFFF800u);
}
// 1 / r of a normal r of 13 bits, correctly rounded: one step from a reciprocal within one unit.
__device__ __forceinline__ float fp8_inverse(float r) {
  const float y = __builtin_amdgcn_rcpf(r);
  return __builtin_fmaf(__builtin_fmaf(-r, y, 1.f), y, y);
}
__device__ __forceinline__ Fp8Factor fp8_block(float amax) {
  if (!(amax < __builtin_inff())) return Fp8Factor{0.f, __uint_as_float(0x7FC00000u)};
  const float r = fp8_factor(amax);
  return Fp8Factor{r, fp8_inverse(r)};
}

// x r for the conversion to a code. EXACT (fp32 x): rounded to odd, the exact product cut to fp32 with its last
// bit set where something was cut, so that it lies on a border between two codes only if the product does.
template <bool EXACT>
__device__ __forceinline__ float fp8_scaled(float x, float r) {
  const float q = x * r;
  if constexpr (!EXACT) return q;
  const float e = __builtin_fmaf(x, r, -q);  // what q lacks, exactly
  const uint32_t m = __float_as_uint(q);
  const uint32_t cut = (m + (uint32_t)((int)(m ^ __float_as_uint(e)) >> 31)) | 1u;  // (e against q: q was rounded up)
  return e != 0.f ? __uint_as_float(cut) : q;
}

// Eight values of a block with factor r as codes. (v_cvt_pk_fp8_f32 does not saturate by itself, and need not: r times the
// largest value passes 448 by half an fp32 step at most, which rounds to 448.)
template <bool EXACT>
__device__ __forceinline__ uint2 fp8_codes8(const float v[8], float r) {
  float c[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) c[e] = fp8_scaled<EXACT>(v[e], r);
  int x = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], 0, false);
  x = __builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], x, true);
  int y = __builtin_amdgcn_cvt_pk_fp8_f32(c[4], c[5], 0, false);
  y = __builtin_amdgcn_cvt_pk_fp8_f32(c[6], c[7], y, true);
  return r == 0.f ? uint2{0u, 0u} : uint2{(uint32_t)x, (uint32_t)y};  // (a NaN or an infinity times 0)
}
// Eight codes as the values that they stand for under one scale.
__device__ __forceinline__ void fp8_values8(uint2 w, float scale, float v[8]) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 p[4] = {__builtin_amdgcn_cvt_pk_f32_fp8(w.x, false), __builtin_amdgcn_cvt_pk_f32_fp8(w.x, true),
                      __builtin_amdgcn_cvt_pk_f32_fp8(w.y, false), __builtin_amdgcn_cvt_pk_f32_fp8(w.y, true)};
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = p[e >> 1][e & 1] * scale;
}

// The larger magnitude, NaN if either is one (v_maximum3_f32 takes three operands and their magnitudes).
__device__ __forceinline__ float larger(float a, float b) { return __builtin_elementwise_maximum(__builtin_fabsf(a), __builtin_fabsf(b)); }
__device__ __forceinline__ float largest8(const float v[8]) {
  float a = larger(v[0], v[1]);
#pragma unroll
  for (int e = 2; e < 8; e += 2) a = larger(larger(a, v[e]), v[e + 1]);
  return a;
}
// Largest magnitude over 16 neighbouring lanes (a block, 8 values a lane), in each of them.
template <int CTRL>
__device__ __forceinline__ float lanes(float a) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(a), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float row_max16(float a) {
  a = larger(a, lanes<0xB1>(a));   // lanes 1 0 3 2
  a = larger(a, lanes<0x4E>(a));   // lanes 2 3 0 1
  a = larger(a, lanes<0x141>(a));  // within 8: i <-> 7 - i
  return larger(a, lanes<0x140>(a));  // within 16: i <-> 15 - i
}

// ---- storage. nb blocks a row, nq = ceil(nb / 4), kp bytes of codes a row.
struct Fp8Geometry {
  int k, kp, nb, nq;
};
__host__ __device__ __forceinline__ Fp8Geometry fp8_geometry(int k) {
  const int nb = (int)(((int64_t)k + kFp8Block - 1) / kFp8Block);
  return Fp8Geometry{k, (int)(((int64_t)k + 15) / 16 * 16), nb, (nb + 3) / 4};
}
// Element of the scale of block b of row r.
__device__ __forceinline__ int64_t fp8_row_scale(int64_t r, int b, int nq) {
  return (((r >> 6) * nq + (b >> 2)) * 64 + (r & 63)) * 4 + (b & 3);
}
__device__ __forceinline__ int64_t fp8_tile_scale(int64_t i, int b, int nq) { return i * nq * 4 + b; }

// Store one block's scale at p (element of block b); the last block's writer fills the row up to a whole quad.
// (A quad's four scales of a row are neighbours in either layout.)
__device__ __forceinline__ void fp8_store_scale(float* p, int b, const Fp8Geometry& g, float scale) {
  *p = scale;
  if (b == g.nb - 1)
    for (int q = 1; q < g.nq * 4 - b; ++q) p[q] = 0.f;
}

}  // namespace gep
