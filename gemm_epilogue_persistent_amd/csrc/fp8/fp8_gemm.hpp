// Products of 8-bit operands with an fp32 scale per 128 values (fp8_gemm_* of the public header):
//   D = A x B^T + C,  PostAct = act(A x B^T + C)
//   (A x B^T)[m, n] = sum over blocks b of sa[m, b] sb[n, b] (sum over k in b of a[m, k] b[n, k])
//
// v_mfma_f32_16x16x128_f8f6f4 sums exactly one block: its result starts from zero, and one fp32 FMA a value adds it
// to the accumulator with the scale sa sb. A lane holds 4 consecutive columns of one row, so that with a scale per
// 128 x 128 tile of B the product sa sb is one number for all of a lane's values in a row block (4 FMAs a matrix
// instruction of 32 cycles), and with a scale per row of B the column's scale is a second factor (4 more
// multiplications). The FMAs run kLag matrix instructions behind, so that none waits for a result.
//
// The kernels are those of the MX product (MxRing, MxDirect) with these parts in the place of the scale operands of
// the matrix instruction; four scales of a row are 16 bytes, as 16 MX scales are, and take the same way. For 64 to some
// hundred rows there is one more, Fp8Staged.
//
// Measured: 8192^3 with B's scales by tiles 425 to 490 us, 2.2 to 2.6 PFLOP/s (by card, bursts and long runs), matrix pipes 63%
// busy at 1.95 GHz; MxRing with e4m3 operands, without the FMAs, 368 to 386, a library product with one scale 363.
// (The pipes and the FMAs alone, from registers, reach 3.7 to 3.9 PFLOP/s, without FMAs 4.0 to 4.3: the clock falls
// under their load.) By rows 524 to 557: with 8 vector instructions a matrix instruction the FMAs are the bound. 16768 x 4096 x 4096 over 8
// experts with SiLU 302 to 323: four rounds of 65, of which SiLU is 3.5, and a last partial round of 42 in 128x128 quarters.
// Measured at 8192^3 and not kept: a ring of four A fragments (436 to 454 where this took 425 to 442), all transfers behind the
// barrier, the two waves of a SIMD taking turns (451), FMAs one instruction behind (2% slower) or three, other
// priorities. 128x128 tiles for the experts: 338 for 302.
#pragma once
#include "../mx/mx_gemm.hpp"
#include "fp8_common.hpp"

namespace gep {

using Fp8Frag = MxFrag<MX_E4M3>;
__device__ __forceinline__ f32x4 fp8_mma(const Fp8Frag& b, const Fp8Frag& a) {
  // (zero scale operands make the compiler emit the unscaled instruction)
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_regs<MX_E4M3>(b), mx_regs<MX_E4M3>(a), f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0,
                                                          0, 0, 0, 0);
}

// BROWS: B has a scale per 128 values of a row, else per 128 x 128 tile.
template <int BM, int BN, int NW, int NS, bool VM, int EPI, bool BROWS>
struct Fp8Ring : MxRing<BM, BN, NW, NS, MX_E4M3, MX_E4M3, VM, EPI> {
  using R = MxRing<BM, BN, NW, NS, MX_E4M3, MX_E4M3, VM, EPI>;
  using At = typename R::At;
  using Stages = typename R::Stages;
  static constexpr int kMI = R::kMI, kNI = R::kNI, kN = R::kN, kRA = R::kRA;
  static constexpr int kLag = 2;   // matrix instructions between a result and its FMAs
  static constexpr int kTmp = 4;   // results held
  static_assert(kLag < kTmp && kLag <= kNI && kN % kTmp == 0 && kMI % 2 == 0, "indices that do not depend on the step");

  struct Src : R::Src {
    uint32_t s_step;  // bytes between the scales of a row's quads of steps
  };
  using Lane = typename R::Lane;
  struct Frags {
    Fp8Frag a[kRA];
    Fp8Frag b[R::kDB ? 2 : 1][kNI];
    f32x4 t[kTmp];               // results on their way into the accumulators
    float sa[kRA];               // of the rows of the A fragments
    float s[2];                  // factor of the row block (sa sb, or sa alone): row block r in r % 2
    float sb[2];                 // tiles: of this step and the next
    f32x4 sc[BROWS ? kNI : 1];   // rows: of a column block's 4 columns of this lane
  };

  static __device__ __forceinline__ void scale_source(Src& s, const MxParams& mp, const MxTileInfo& ti, int q0, int wave, int lane) {
    R::scale_source(s, mp, ti, q0, wave, lane);
    s.s_step = 1024;
    if constexpr (!BROWS) {
      if (wave >= BM / 64) {  // row i of the tile's B rows: its 128 x 128 tile's row of scales (n0 is a multiple of 128)
        const int64_t so = ((int64_t)(ti.n0 >> 7) * mp.nsb + q0) * 16;
        s.s = make_rsrc(mp.sb + (int64_t)ti.g * mp.sb_bytes + so, mp.sb_bytes - so);
        const int i = (wave - BM / 64) * 64 + lane;
        s.s_off = ti.n0 + i < mp.k.N ? (uint32_t)((i >> 7) * mp.nsb * 16) : kOOB;
        s.s_step = 16;
      }
    }
  }
  static __device__ __forceinline__ void dma_scales(const Src& s, int quad, GEP_LDS char* smem, int stage, int wave) {
    if constexpr ((BM + BN) / 64 < NW)
      if (wave >= (BM + BN) / 64) return;
#if defined(__HIP_DEVICE_COMPILE__)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(s.s, (GEP_LDS void*)(smem + R::kSOff + stage * R::kSBytes + wave * 1024), 16,
                                             quad < s.nsb ? s.s_off + quad * s.s_step : kOOB, 0, 0, 0);
#endif
  }
  static __device__ __forceinline__ Lane lane_offsets(int lane, int wm0, int wn0) {
    Lane o = R::lane_offsets(lane, wm0, wn0);
    o.sa = R::kSOff + (wm0 + (lane & 15)) * 16;
    o.sb = R::kSOff + (BM + wn0 + (BROWS ? 4 * (lane >> 4) : 0)) * 16;
    return o;
  }
  template <int T>
  static __device__ __forceinline__ float read_scale(const GEP_LDS char* p) { return *(const GEP_LDS float*)(p + T * 4); }
  template <int T>
  static __device__ __forceinline__ void read_a(Frags& f, const GEP_LDS char* smem, const At& x, int r) {
    f.a[r % kRA] = R::template read<MX_E4M3, R::kRowA>(smem, x.a, x.a2, r);
    f.sa[r % kRA] = read_scale<T>(smem + x.sa + r * 256);
  }
  template <int T>
  static __device__ __forceinline__ void read_b(Frags& f, const GEP_LDS char* smem, const At& x, int c) {
    f.b[R::bset(T)][c] = R::template read<MX_E4M3, R::kRowB>(smem, x.b, x.b2, c);
  }
  template <int T>
  static __device__ __forceinline__ void read_columns(Frags& f, const GEP_LDS char* smem, const At& x, int c) {
#pragma unroll
    for (int e = 0; e < 4; ++e) f.sc[BROWS ? c : 0][e] = read_scale<T>(smem + x.sb + (c * 16 + e) * 16);
  }
  // The next step's scales of column block c are read once this step's last FMAs with them are done, kLag behind
  // its last matrix instruction: at position p of this step for the next, or of the next step for itself.
  static constexpr int next_columns(int p) { return BROWS && p - R::kLastP - kLag >= 0 ? p - R::kLastP - kLag : -1; }
  static constexpr int own_columns(int p) { return BROWS && p < kLag ? kNI - kLag + p : -1; }

  static __device__ __forceinline__ void first_reads(Frags& f, const GEP_LDS char* smem, const Lane& o) {
    const At x = R::template at<0>(o, 0, 0);
#pragma unroll
    for (int r = 0; r < kRA - 1; ++r) read_a<0>(f, smem, x, r);
#pragma unroll
    for (int c = 0; c < kNI; ++c) read_b<0>(f, smem, x, c);
#pragma unroll
    for (int i = 0; i < kTmp; ++i) f.t[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    f.s[0] = f.s[1] = 0.f;
    f.sb[0] = f.sb[1] = 0.f;
    if constexpr (BROWS) {
#pragma unroll
      for (int c = 0; c < kNI; ++c) {
        if (c < kNI - kLag) read_columns<0>(f, smem, x, c);
        else f.sc[c] = f32x4{0.f, 0.f, 0.f, 0.f};  // (read by the first step; its first FMAs add nothing)
      }
    } else {
      f.sb[0] = read_scale<0>(smem + x.sb);
    }
  }
  // The FMAs of position P.
  template <int P>
  static __device__ __forceinline__ void add(f32x4 (&acc)[kMI][kNI], const Frags& f) {
    constexpr int r = P / kNI, c = P % kNI;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float t = BROWS ? f.t[P % kTmp][e] * f.sc[BROWS ? c : 0][e] : f.t[P % kTmp][e];
      acc[r][c][e] = __builtin_fmaf(t, f.s[r & 1], acc[r][c][e]);
    }
  }
  static __device__ __forceinline__ void drain(f32x4 (&acc)[kMI][kNI], Frags& f) {
    add<kN - 2>(acc, f);
    add<kN - 1>(acc, f);
    static_assert(kLag == 2);
  }

  static constexpr int reads(int, int p) {  // LDS reads after position p
    return 3 * (R::a_after(p) >= 0) + 3 * (R::na_after(p) >= 0) + 2 * (R::nb_after(p) >= 0) +
           2 * ((next_columns(p) >= 0) + (own_columns(p) >= 0)) + (!BROWS && p == R::kBarP);
  }
  template <int T, int P, int E>
  static __device__ __forceinline__ void sched() {
    if constexpr (P < E) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x002, (BROWS ? 8 : 4) + (P % kNI == 0), 0);
      if constexpr (reads(T, P) > 0) __builtin_amdgcn_sched_group_barrier(0x100, reads(T, P), 0);
      if constexpr (R::transfers(T, P) > 0) __builtin_amdgcn_sched_group_barrier(0x020, R::transfers(T, P), 0);
      sched<T, P + 1, E>();
    }
  }
  // Positions [P, E) of step T of quad q (x: this step's addresses, y: the next one's).
  template <bool MM, int T, int P, int E>
  static __device__ __forceinline__ void positions(f32x4 (&acc)[kMI][kNI], Frags& f, GEP_LDS char* smem, const At& x,
                                                   const At& y, const Src& s, int q, const Stages& st, int wave) {
    if constexpr (P < E) {
      constexpr int NT = (T + 1) & 3;
      if constexpr (MM) {
        constexpr int r = P / kNI, c = P % kNI;
        f.t[P % kTmp] = fp8_mma(f.b[R::bset(T)][c], f.a[r % kRA]);
        if constexpr (c == 0) f.s[r & 1] = BROWS ? f.sa[r % kRA] : f.sa[r % kRA] * f.sb[T & 1];
        add<(P + kN - kLag) % kN>(acc, f);
        if constexpr (R::a_after(P) >= 0) read_a<T>(f, smem, x, R::a_after(P));
        if constexpr (R::na_after(P) >= 0) read_a<NT>(f, smem, y, R::na_after(P));
        if constexpr (R::nb_after(P) >= 0) read_b<NT>(f, smem, y, R::nb_after(P));
        if constexpr (own_columns(P) >= 0) read_columns<T>(f, smem, x, own_columns(P));
        if constexpr (next_columns(P) >= 0) read_columns<NT>(f, smem, y, next_columns(P));
        if constexpr (!BROWS && P == R::kBarP) f.sb[NT & 1] = read_scale<NT>(smem + y.sb);
      }
      constexpr int h = R::head_at(T, P), u = R::tail_at(T, P);
      const int n = q * 4 + T;  // this stage's number
      if constexpr (h >= 0) R::template transfer<h, true>(s, n + NS - 1, smem + st.prev, wave);
      if constexpr (P == R::kScaleP && T == 0) dma_scales(s, q + 1, smem, (q + 1) & 1, wave);
      if constexpr (u >= 0) R::template transfer<u, false>(s, n + NS, smem + st.cur, wave);
      positions<MM, T, P + 1, E>(acc, f, smem, x, y, s, q, st, wave);
    }
  }

  static __device__ __forceinline__ void run(const MxParams& mp) { R::template run_as<Fp8Ring>(mp); }
};

template <int MB, int NB, int NW, int D, bool VM, bool BROWS>
struct Fp8Direct : MxDirect<MB, NB, NW, D, MX_E4M3, MX_E4M3, VM> {
  using R = MxDirect<MB, NB, NW, D, MX_E4M3, MX_E4M3, VM>;
  using Src = typename R::Src;
  using Buf = typename R::Buf;
  static constexpr int kSB = BROWS ? 4 * NB : 1;  // 16-byte loads of B's scales: 4 columns a column block, or the tile's
  struct Scales {
    f32x4 a[MB], b[kSB];
  };
  using Now = Scales;
  static __device__ __forceinline__ void scale_source(Src& s, const MxParams& mp, int g, int m0, int n0, int row_end, int lane) {
    R::scale_source(s, mp, g, m0, n0, row_end, lane);
    if constexpr (BROWS) {
#pragma unroll
      for (int j = 0; j < NB; ++j) {  // columns 4 (lane / 16) + [0, 4): their scales are 64 bytes
        const int c = j * 16 + 4 * (lane >> 4), q = (n0 & 63) + c;
        s.sbo[j] = n0 + c < mp.k.N ? (uint32_t)((q >> 6) * mp.nsb * 1024 + (q & 63) * 16) : kOOB;
      }
    } else {
      const int64_t so = (int64_t)(n0 >> 7) * mp.nsb * 16;  // (the workgroup's columns lie in one tile)
      s.sb = make_rsrc(mp.sb + (int64_t)g * mp.sb_bytes + so, mp.sb_bytes - so);
    }
  }
  static __device__ __forceinline__ f32x4 load(__amdgpu_buffer_rsrc_t rs, uint32_t off) {
    return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0));
  }
  static __device__ __forceinline__ void fetch_scales(Scales& q, const Src& s, int tile) {
    if constexpr (BROWS) {
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) q.b[4 * j + e] = load(s.sb, tile < s.nsb ? s.sbo[j] + tile * 1024 + e * 16 : kOOB);
    } else {
      q.b[0] = load(s.sb, tile < s.nsb ? tile * 16 : kOOB);
    }
#pragma unroll
    for (int i = 0; i < MB; ++i) q.a[i] = load(s.sa, tile < s.nsb ? s.sao[i] + tile * 1024 : kOOB);
  }
  static __device__ __forceinline__ void take(Now& now, const Scales& sc, int) { now = sc; }
  template <int T>
  static __device__ __forceinline__ void multiply(f32x4 (&acc)[MB][NB], const Buf& b, const Now& now) {
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const float s = BROWS ? now.a[i][T] : now.a[i][T] * now.b[0][T];
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const f32x4 t = fp8_mma(b.b[j], b.a[i]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[i][j][e] = __builtin_fmaf(BROWS ? t[e] * now.b[BROWS ? 4 * j + e : 0][T] : t[e], s, acc[i][j][e]);
      }
    }
  }
  static __device__ __forceinline__ void run(const MxParams& mp) { R::template run_as<Fp8Direct>(mp); }
};

// 64 x 64 outputs a workgroup of four waves that share out K, as in MxDirect, but each wave's operands come through LDS in
// a ring of its own, two steps ahead: whole lines of 128 bytes (fragments read from memory directly take 64 bytes of
// each of 16 rows at a time), and no barrier. Wave w takes step w of every quad of steps. 85 KB a microsecond and compute
// unit, where direct kernels move 33 and 128x128 tiles 55 to 65 between their barriers. 256 x 4096 x 4096 11.6 us (direct
// 64x64 tiles 20.4, 32x64 25.6, 128x128 over four workgroups 21.7), 64 x 8192 x 8192 17.0 for 67 MB (25.5 and 23.0), 512 x
// 4096 x 4096 21.0 (38, 45, 25.6). Whole quads for each wave, with their scales in registers: 12.7, and 7.2 instead of 6.0 at
// 512 x 1024 x 1024, where two waves had none.
template <bool VM, bool BROWS>
struct Fp8Staged : MxDirect<4, 4, 4, 1, MX_E4M3, MX_E4M3, VM> {
  using R = MxDirect<4, 4, 4, 1, MX_E4M3, MX_E4M3, VM>;
  static constexpr int kWaves = 4, kPart = 64 * 128, kScales = 2 * kPart, kStage = kScales + 2048, kRing = 2 * kStage;
  static constexpr int kLag = 2;
  static constexpr int kPer = 18;  // transfers of a stage: A, B, and the scales of their rows
  static_assert(R::kPlane * 4 <= kRing, "the waves' sums lie in their rings");
  struct Src {
    __amdgpu_buffer_rsrc_t a, b, sa, sb;
    uint32_t ao[8], bo[8];  // this lane's chunk of row 8 q + lane / 8 (kOOB past the operand)
    int ka[2], kb[2];       // bytes of a row past that chunk, for even and odd q
    uint32_t sao, sbo;      // the scales of row `lane`
    int sb_step;            // bytes from a row's quad of B's scales to the next
    int t1;                 // quads up to here
  };
  static __device__ __forceinline__ void move(__amdgpu_buffer_rsrc_t rs, uint32_t off, GEP_LDS char* lds) {
#if defined(__HIP_DEVICE_COMPILE__)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (GEP_LDS void*)lds, 16, off, 0, 0, 0);
#endif
  }
  static __device__ __forceinline__ void transfer(const Src& s, int quad, int wave, GEP_LDS char* lds) {
    const int kb = (quad * 4 + wave) * 128;
#pragma unroll
    for (int q = 0; q < 8; ++q) move(s.b, kb < s.kb[q & 1] ? s.bo[q] + kb : kOOB, lds + kPart + q * 1024);
#pragma unroll
    for (int q = 0; q < 8; ++q) move(s.a, kb < s.ka[q & 1] ? s.ao[q] + kb : kOOB, lds + q * 1024);
    // (past the last quad: zeros, as its codes)
    move(s.sa, quad < s.t1 ? s.sao + quad * 1024 : kOOB, lds + kScales);
    move(s.sb, quad < s.t1 ? s.sbo + quad * s.sb_step : kOOB, lds + kScales + 1024);
  }
  static __device__ __forceinline__ Fp8Frag fragment(const GEP_LDS char* lds, int at, int r) {
    return Fp8Frag{*(const GEP_LDS i32x4*)(lds + at + r * 2048), *(const GEP_LDS i32x4*)(lds + (at ^ 64) + r * 2048)};
  }
  // The step whose stage is `lds`, and the transfers of the step two behind it.
  static __device__ __forceinline__ void step(f32x4 (&acc)[4][4], const Src& s, int quad, int wave, GEP_LDS char* lds, int at, int lane) {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kPer) : "memory");  // (outstanding: the next step's)
    __builtin_amdgcn_sched_barrier(0);
    Fp8Frag a[4], b[4];
    float sa[4];
    f32x4 sb[BROWS ? 4 : 1];
    const GEP_LDS char* sp = lds + kScales + wave * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      b[i] = fragment(lds + kPart, at, i);
      a[i] = fragment(lds, at, i);
      sa[i] = *(const GEP_LDS float*)(sp + (i * 16 + (lane & 15)) * 16);
      if constexpr (BROWS) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sb[i][e] = *(const GEP_LDS float*)(sp + 1024 + (i * 16 + 4 * (lane >> 4) + e) * 16);
      }
    }
    if constexpr (!BROWS) sb[0][0] = *(const GEP_LDS float*)(sp + 1024);
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the stage is free
    __builtin_amdgcn_sched_barrier(0);
    transfer(s, quad + 2, wave, lds);
    if constexpr (!BROWS) {
#pragma unroll
      for (int i = 0; i < 4; ++i) sa[i] *= sb[0][0];
    }
    f32x4 t[4];
#pragma unroll
    for (int q = 0; q < 16 + kLag; ++q) {  // the FMAs two matrix instructions behind
      if (q < 16) t[q & 3] = fp8_mma(b[q & 3], a[q >> 2]);
      if (q < kLag) continue;
      const int i = (q - kLag) >> 2, j = (q - kLag) & 3;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v = t[(q - kLag) & 3][e];
        acc[i][j][e] = __builtin_fmaf(BROWS ? v * sb[BROWS ? j : 0][e] : v, sa[i], acc[i][j][e]);
      }
    }
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x002, BROWS ? 8 : 4, 0);
    }
  }
  static __device__ __forceinline__ void run(const MxParams& mp) {
    const KParams& p = mp.k;
    __shared__ __attribute__((aligned(1024))) char smem[kWaves * kRing];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    typename R::Place pl;
    if (!R::place(pl, mp, lane)) return;
    Src s;
    const int64_t ao = (int64_t)pl.m0 * p.lda, bo = (int64_t)pl.n0 * p.ldb;
    s.a = make_rsrc((const char*)p.A + ao, p.a_bytes - ao);
    s.b = make_rsrc((const char*)p.B + (int64_t)pl.g * p.b_bytes + bo, p.b_bytes - bo);
    // (chunk c of row r lies at chunk c ^ kswz(r), a key that repeats every 16 rows)
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int row = q * 8 + (lane >> 3), c = (lane & 7) ^ kswz(row);
      s.ao[q] = pl.m0 + row < pl.row_end ? (uint32_t)(row * (int)p.lda + c * 16) : kOOB;
      s.bo[q] = pl.n0 + row < p.N ? (uint32_t)(row * (int)p.ldb + c * 16) : kOOB;
      if (q < 2) {
        s.ka[q] = min((int)p.lda, pl.t1 * 512) - c * 16;
        s.kb[q] = min((int)p.ldb, pl.t1 * 512) - c * 16;
      }
    }
    {
      const int64_t so = (int64_t)(pl.m0 >> 6) * mp.nsb * 1024;
      const int q = (pl.m0 & 63) + lane;
      s.sa = make_rsrc(mp.sa + so, mp.sa_bytes - so);
      s.sao = pl.m0 + lane < pl.row_end ? (uint32_t)((q >> 6) * mp.nsb * 1024 + (q & 63) * 16) : kOOB;
    }
    const int64_t so = BROWS ? (int64_t)(pl.n0 >> 6) * mp.nsb * 1024 : (int64_t)(pl.n0 >> 7) * mp.nsb * 16;
    s.sb = make_rsrc(mp.sb + (int64_t)pl.g * mp.sb_bytes + so, mp.sb_bytes - so);
    s.sbo = !BROWS ? 0 : (pl.n0 + lane < p.N ? (uint32_t)lane * 16 : kOOB);
    s.sb_step = BROWS ? 1024 : 16;
    s.t1 = pl.t1;
    const int at = (lane & 15) * 128 + (((lane >> 4) ^ kswz(lane & 15)) << 4);
    f32x4 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    GEP_LDS char* ring = (GEP_LDS char*)smem + wave * kRing;
    if (pl.t0 < pl.t1) {
      transfer(s, pl.t0, wave, ring);
      transfer(s, pl.t0 + 1, wave, ring + kStage);
      for (int quad = pl.t0; quad < pl.t1; quad += 2) {
        step(acc, s, quad, wave, ring, at, lane);
        step(acc, s, quad + 1, wave, ring + kStage, at, lane);
      }
    }
    dma_barrier();  // transfers past K have landed: the sums take the rings' place
    R::join(mp, pl, acc, (float*)smem);
  }
};

template <int BM, int NW, int WG, bool VM, int EPI, bool BROWS>
__global__ __launch_bounds__(NW * 64, WG) void fp8_ring_kernel(const MxParams p) {
  Fp8Ring<BM, BM, NW, mx_stages<BM, MX_E4M3, MX_E4M3, WG>(), VM, EPI, BROWS>::run(p);
}
template <int BM, int NW, int WG, bool VM, bool BROWS>
void fp8_launch_ring(const MxParams& p, dim3 grid, hipStream_t s) {
  if constexpr (BM == 256) fp8_ring_kernel<BM, NW, WG, VM, 0, BROWS><<<grid, NW * 64, 0, s>>>(p);
  else if (mx_epilogue_kind(p) == 1) fp8_ring_kernel<BM, NW, WG, VM, 1, BROWS><<<grid, NW * 64, 0, s>>>(p);
  else fp8_ring_kernel<BM, NW, WG, VM, 2, BROWS><<<grid, NW * 64, 0, s>>>(p);
}
template <int MB, int NB, int NW, int D, bool VM, bool BROWS>
__global__ __launch_bounds__(NW * 64) void fp8_direct_kernel(const MxParams p) {
  Fp8Direct<MB, NB, NW, D, VM, BROWS>::run(p);
}

// (Bounds of 512 threads for its 256: the compiler then keeps to 256 registers, and results out of the accumulation ones.)
template <bool VM, bool BROWS>
__global__ __launch_bounds__(512) void fp8_staged_kernel(const MxParams p) {
  Fp8Staged<VM, BROWS>::run(p);
}

// The kernels (launch configuration by mx_plan.cpp; the tiles are numbered as the MX product's).
template <bool BROWS, bool VM>
hipError_t fp8_launch(int32_t tile, const MxParams& p, dim3 grid, hipStream_t s);

#define GEP_FP8_LAUNCH(BROWS, VM)                                                                     \
  template <>                                                                                         \
  hipError_t fp8_launch<BROWS, VM>(int32_t tile, const MxParams& p, dim3 grid, hipStream_t s) {       \
    switch (tile) {                                                                                   \
      case MX_TILE_256: fp8_launch_ring<256, 8, 1, VM, BROWS>(p, grid, s); break;                     \
      case MX_TILE_128:                                                                               \
        if (p.k.P <= p.cus) fp8_launch_ring<128, 4, 1, VM, BROWS>(p, grid, s);                        \
        else fp8_launch_ring<128, 4, 2, VM, BROWS>(p, grid, s);                                       \
        break;                                                                                        \
      case FP8_TILE_64: fp8_staged_kernel<VM, BROWS><<<grid, 256, 0, s>>>(p); break;                  \
      case MX_TILE_32: fp8_direct_kernel<2, 2, 4, 2, VM, BROWS><<<grid, 256, 0, s>>>(p); break;       \
      case MX_TILE_16X32: fp8_direct_kernel<1, 2, 8, 2, VM, BROWS><<<grid, 512, 0, s>>>(p); break;    \
      case MX_TILE_16: fp8_direct_kernel<1, 1, 4, 2, VM, BROWS><<<grid, 256, 0, s>>>(p); break;       \
      default: return hipErrorInvalidValue;                                                           \
    }                                                                                                 \
    return hipGetLastError();                                                                         \
  }

}  // namespace gep
