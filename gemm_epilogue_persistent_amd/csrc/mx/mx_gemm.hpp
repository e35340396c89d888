// Products of MX operands with a fused epilogue for gfx950 (mx_gemm_* of the public header):
//   D = A x B^T + C,  PostAct = act(A x B^T + C)
//
// v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 16 x 128 by 128 x 16 blocks in either element
// type per operand and applies one scale byte per 32 values of K to each of them, so the scales
// cost no vector arithmetic: A[m, k] = a 2^(sa - 127), and each block of 32 contributes
// 2^(sa + sb - 254) sum a b to the fp32 accumulator. Lane l holds row l % 16 of a fragment:
// E2M1 its 32 codes of K block l / 16 (16 bytes), E4M3 the 16-byte chunks l / 16 and l / 16 + 4
// of the row's 128 bytes; the scale it supplies is that of row l % 16, K block l / 16 (the same
// for both types; checked on the hardware element by element).
//
// Two kernels:
//   MxRing   large problems. 256x256 or 256x128 outputs per workgroup of 8 waves, 128x128 of 4: both
//            operands go through LDS (global -> LDS transfers, two stages), persistent tile loop.
//   MxDirect few rows. 16x16 to 64x64 outputs per workgroup, whose waves share out K and read
//            their fragments from global memory themselves; one join in LDS at the end.
#pragma once
#include "../gemm_kernel.hpp"
#include "mx_common.hpp"

namespace gep {

// Kernel arguments. k: sizes, output pointers and strides, raster constants; lda / ldb are the
// operands' row pitches in bytes.
struct MxParams {
  KParams k;
  const uint8_t *sa, *sb;  // scales
  int64_t sa_bytes, sb_bytes;  // their extents (sb: of one group)
  int32_t nsb;             // scale tiles along K (512 values each)
  int32_t steps;           // MFMA steps of 128 along K
  // K shared out over `split` workgroups a tile (dense; 1: not), `per` scale tiles each: slice s
  // writes its fp32 sums as matrix s of `sums`, (split, M, N), and mx_join_kernel adds them up
  int32_t split, per;
  float* sums;
};

template <int FMT>
struct MxFmt {
  static constexpr bool k8 = FMT == MX_E4M3;
  static constexpr int kCode = k8 ? 0 : 4;       // format field of the instruction
  static constexpr int kStepBytes = k8 ? 128 : 64;  // bytes of a row per 128 values
  static constexpr int kBlockBytes = k8 ? 32 : 16;
};

// The fragment registers of one 16 x 128 block (E2M1 uses the first four).
template <int FMT>
struct MxFrag {
  i32x4 lo, hi;
};
template <>
struct MxFrag<MX_E2M1> {
  i32x4 lo;
};
template <int FMT>
__device__ __forceinline__ i32x8 mx_regs(const MxFrag<FMT>& f) {
  if constexpr (FMT == MX_E4M3) return __builtin_shufflevector(f.lo, f.hi, 0, 1, 2, 3, 4, 5, 6, 7);
  else return __builtin_shufflevector(f.lo, f.lo, 0, 1, 2, 3, -1, -1, -1, -1);
}
// B first, A second: a lane then holds 4 consecutive columns of one row (as in gemm_kernel.hpp).
// OS: which byte of the scale registers applies.
template <int FA, int FB, int OS = 0>
__device__ __forceinline__ f32x4 mx_mma(const MxFrag<FB>& b, const MxFrag<FA>& a, f32x4 c, int sb, int sa) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_regs<FB>(b), mx_regs<FA>(a), c, MxFmt<FB>::kCode,
                                                          MxFmt<FA>::kCode, OS, sb, OS, sa);
}

// ---- outputs: 8 consecutive columns of a row
__device__ __forceinline__ void mx_load8(int dt, const char* p, float v[8]) {
  if (dt == DT_F32) {
    const f32x4 a = *(const f32x4*)p, b = *(const f32x4*)(p + 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = a[e], v[4 + e] = b[e];
  } else {
    const uint4 x = *(const uint4*)p;
    unpack4_16(dt, uint2{x.x, x.y}, v);
    unpack4_16(dt, uint2{x.z, x.w}, v + 4);
  }
}
__device__ __forceinline__ void mx_store8(int dt, char* p, const float v[8]) {
  if (dt == DT_F32) {
    *(f32x4*)p = f32x4{v[0], v[1], v[2], v[3]};
    *(f32x4*)(p + 16) = f32x4{v[4], v[5], v[6], v[7]};
  } else {
    const uint2 a = pack4_16(dt, v), b = pack4_16(dt, v + 4);
    *(uint4*)p = uint4{a.x, a.y, b.x, b.y};
  }
}
__device__ __forceinline__ void mx_act8(int act, float v[8]) {
  switch (act) {
    case ACT_RELU:
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = act_fn<ACT_RELU>(v[e]);
      break;
    case ACT_RELU_SQ:
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = act_fn<ACT_RELU_SQ>(v[e]);
      break;
    case ACT_GELU_TANH:
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = act_fn<ACT_GELU_TANH>(v[e]);
      break;
    case ACT_SILU:
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = act_fn<ACT_SILU>(v[e]);
      break;
    default: break;
  }
}
// C, D and PostAct of row m, columns [n, n + 8) from the product v.
__device__ __forceinline__ void mx_finish8(const KParams& p, int64_t m, int n, float v[8]) {
  if (p.c_dt != DT_NONE) {
    float c[8];
    mx_load8(p.c_dt, (const char*)p.C + (m * p.ldc + n) * dt_bytes(p.c_dt), c);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += c[e];
  }
  if (p.d_dt != DT_NONE) mx_store8(p.d_dt, (char*)p.D + (m * p.ldd + n) * dt_bytes(p.d_dt), v);
  if (p.p_dt != DT_NONE) {
    mx_act8(p.act, v);
    mx_store8(p.p_dt, (char*)p.Post + (m * p.ldp + n) * dt_bytes(p.p_dt), v);
  }
}

// The same for a slice of K: its sums, to be added up later.
__device__ __forceinline__ void mx_slice8(const MxParams& p, int slice, int64_t m, int n, const float v[8]) {
  mx_store8(DT_F32, (char*)(p.sums + ((int64_t)slice * p.k.M + m) * p.k.N + n), v);
}

// One output tile of a grouped or dense problem.
struct MxTileInfo {
  int g, m0, n0, row_end, slice;
};

// ------------------------------------------------------------------------------------
// MxRing
// ------------------------------------------------------------------------------------
// A stage holds 128 bytes of K per row: one step (128 values) of an E4M3 operand, a pair of
// steps (256 values) of an E2M1 one; each operand has two stages. The scales of four steps (16
// bytes a row, in storage order) go through a two-stage ring of their own. The loop runs quads of
// four steps; steps past K read zero codes.
//
// A step is kMI x kNI MFMAs, row by row. kRA A fragments are held in a ring (block row r in r %
// kRA; r is read after row r - kRA's last MFMA) and the kNI B fragments of the step, with kDB
// those of the next step too. The barrier comes when every wave has read its last fragment of
// the stage; after it the next step's first fragments are read and the first half of the
// transfers into the freed stage goes out; the second half follows at the head of the next step.
// (No barrier in the middle of a pair when both operands are E2M1: neither stage changes.)
template <int BM, int BN, int NW, int FA, int FB, bool VM>
struct MxRing {
  static constexpr int kThreads = NW * 64;
  static constexpr bool kSplit = BM == 128 && !VM;  // may run slices of K
  static constexpr int kWN = 64, kWavesN = BN / kWN, kWavesM = NW / kWavesN, kWM = BM / kWavesM;
  static constexpr int kMI = kWM / 16, kNI = kWN / 16;
  static constexpr int kABytes = BM * kRowBytes, kBBytes = BN * kRowBytes;
  static constexpr int kBOff = 2 * kABytes, kSOff = kBOff + 2 * kBBytes, kSBytes = (BM + BN) * 16;
  static constexpr int kLdsBytes = kSOff + 2 * kSBytes;
  static constexpr int kVarlenLds = VM ? (kMaxVarlenGroups + 1 + kThreads + 1) * 4 : 0;
  static constexpr int kInstrA = BM / 8 / NW, kInstrB = BN / 8 / NW;  // transfers (8 rows each) of a stage
  static_assert((BM + BN) / 64 <= NW, "at most one scale transfer (64 rows) a wave");
  static_assert(kMI >= 4 && kMI % 2 == 0 && kNI == 4, "the fragment schedule below");
  static_assert(kInstrA % 2 == 0 && kInstrB % 2 == 0 && kInstrA <= 4 && kInstrB <= 4, "half a stage at a time");
  static constexpr int kHalfA = kInstrA / 2, kHalf = kInstrA / 2 + kInstrB / 2;  // transfers of half a stage: A's, then B's
  static constexpr int kN = kMI * kNI, kLastP = kN - kNI;
  static constexpr bool kDeep = FA == MX_E2M1 && FB == MX_E2M1;
  static constexpr int kRA = kDeep ? 4 : 2;
  static constexpr bool kDB = kDeep;
  // Two E2M1 operands: lane group g takes the K blocks c = {0, 6, 2, 4}[g] and c + 1 of the eight
  // of a pair of steps, one in each step (A and B alike, so the same products meet). Its two
  // scales are then neighbours. A ds_read_b128 serves 16 lanes at a time: rows 0-3 and 12-15 of
  // one lane group with rows 4-11 of its neighbour, and so on; under kswz their chunks lie in
  // distinct banks when the neighbours' blocks differ by 1, 6 or 7 (by 4: every read twice as
  // long, counted).
  static constexpr bool kPairScales = kDeep;
  // the barrier's position: past the last read of the step's own fragments (and, without kDB,
  // where the next step's fragments find free registers)
  static constexpr int kBarP = !kDB ? kLastP : ((kMI - kRA) * kNI > kNI ? (kMI - kRA) * kNI : kNI);
  static constexpr int kPrioP = (kBarP / 2 + 3) / 4 * 4;
  static constexpr int kTailStep = (kN - kBarP) / kHalf;  // between the transfers after the barrier
  using A = MxFmt<FA>;
  using B = MxFmt<FB>;

  struct Loader {  // this lane's share of one operand's transfers
    uint32_t off[4];
    int32_t klim;  // bytes of a row past this lane's chunk
  };
  template <int N>
  static __device__ __forceinline__ void init(Loader& l, int wave, int lane, int rows_valid, int ld, int row_bytes) {
    const int c = (lane & 7) ^ kswz(wave * 8 + (lane >> 3));  // (the key repeats every 16 rows)
#pragma unroll
    for (int q = 0; q < N; ++q) {
      const int row = (q * NW + wave) * 8 + (lane >> 3);
      l.off[q] = row < rows_valid ? (uint32_t)(row * ld + c * 16) : kOOB;
    }
    l.klim = row_bytes - c * 16;
  }
  // Transfers [Q0, Q1) of the stage at `lds`: bytes [kb, kb + 128) of the rows. (kb is added to
  // the lane's offset: the range check, which turns kOOB into zeros, is stated for that sum. An
  // offset is below 2^31, so kOOB + kb does not wrap.)
  template <int Q0, int Q1>
  static __device__ __forceinline__ void dma(const Loader& l, __amdgpu_buffer_rsrc_t rs, int kb, GEP_LDS char* lds,
                                             int wave) {
    if constexpr (Q0 < Q1) {
#if defined(__HIP_DEVICE_COMPILE__)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (GEP_LDS void*)(lds + (Q0 * NW + wave) * 1024), 16,
                                               kb < l.klim ? l.off[Q0] + kb : kOOB, 0, 0, 0);
#endif
      dma<Q0 + 1, Q1>(l, rs, kb, lds, wave);
    }
  }

  struct Src {
    __amdgpu_buffer_rsrc_t a, b, s;
    Loader la, lb;
    uint32_t s_off;  // this lane's row in the wave's scale transfer
    int32_t nsb;
  };
  static __device__ __forceinline__ void dma_scales(const Src& s, int quad, GEP_LDS char* smem, int stage, int wave) {
    if constexpr ((BM + BN) / 64 < NW)
      if (wave >= (BM + BN) / 64) return;
#if defined(__HIP_DEVICE_COMPILE__)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(s.s, (GEP_LDS void*)(smem + kSOff + stage * kSBytes + wave * 1024), 16,
                                             quad < s.nsb ? s.s_off + quad * 1024 : kOOB, 0, 0, 0);
#endif
  }

  // Lane offsets (A: from the start of the ring; B and scales likewise).
  struct Lane {
    int a0, a1;  // E4M3: the two chunks; E2M1: steps 0 and 1 of a pair
    int b0, b1;
    int sa, sb;  // scale bytes, of the current scale stage
  };
  static __device__ __forceinline__ Lane lane_offsets(int lane, int wm0, int wn0) {
    Lane o;
    const int ra = wm0 + (lane & 15), rb = wn0 + (lane & 15), g = lane >> 4;
    // first K block (E2M1) or chunk (E4M3) of lane group g, and how far the other one is
    const int c = kPairScales ? (0x4260 >> (4 * g)) & 7 : g, far = kPairScales ? 16 : 64;
    o.a0 = ra * kRowBytes + ((c ^ kswz(ra)) << 4);
    o.b0 = kBOff + rb * kRowBytes + ((c ^ kswz(rb)) << 4);
    o.a1 = o.a0 ^ far;
    o.b1 = o.b0 ^ far;
    o.sa = kSOff + ra * 16 + c;
    o.sb = kSOff + (BM + rb) * 16 + c;
    return o;
  }
  // Stage of an operand in step T of a quad.
  template <int F>
  static constexpr int stage(int t) { return F == MX_E4M3 ? (t & 1) : ((t >> 1) & 1); }
  template <int F, int T>
  static __device__ __forceinline__ MxFrag<F> read(const GEP_LDS char* smem, int stage_bytes, int r, int o0, int o1) {
    const GEP_LDS char* p = smem + stage<F>(T) * stage_bytes + r * 16 * kRowBytes;
    MxFrag<F> f;
    if constexpr (F == MX_E4M3) {
      f.lo = *(const GEP_LDS i32x4*)(p + o0);
      f.hi = *(const GEP_LDS i32x4*)(p + o1);
    } else {
      f.lo = *(const GEP_LDS i32x4*)(p + ((T & 1) ? o1 : o0));
    }
    return f;
  }
  // kPairScales: the lane's two scales of a pair of steps in one read, every other step.
  template <int T>
  static __device__ __forceinline__ void read_scale(int& v, const GEP_LDS char* smem, int o, int r) {
    if constexpr (kPairScales) {
      if constexpr (T % 2 == 0) v = *(const GEP_LDS uint16_t*)(smem + o + r * 256 + T * 4);
    } else {
      v = *(const GEP_LDS uint8_t*)(smem + o + r * 256 + T * 4);
    }
  }

  struct Frags {
    MxFrag<FA> a[kRA];
    MxFrag<FB> b[kDB ? 2 : 1][kNI];
    int sa[kPairScales ? kMI : kRA], sb[kDB ? 2 : 1][kNI];
  };
  static constexpr int sset(int t) { return !kDB ? 0 : (kPairScales ? (t >> 1) & 1 : t & 1); }
  static constexpr int bset(int t) { return kDB ? t & 1 : 0; }
  template <int T>
  static __device__ __forceinline__ void read_a(Frags& f, const GEP_LDS char* smem, const Lane& o, int r, int so) {
    f.a[r % kRA] = read<FA, T>(smem, kABytes, r, o.a0, o.a1);
    read_scale<T>(f.sa[kPairScales ? r : r % kRA], smem, o.sa + so, r);
  }
  template <int T>
  static __device__ __forceinline__ void read_b(Frags& f, const GEP_LDS char* smem, const Lane& o, int c, int so) {
    f.b[bset(T)][c] = read<FB, T>(smem, kBBytes, c, o.b0, o.b1);
    read_scale<T>(f.sb[sset(T)][c], smem, o.sb + so, c);
  }

  static constexpr bool bar(int t) { return A::k8 || B::k8 || (t & 1); }
  // What is read after position p: the A fragment of this step's row a_after (the rows past the ring's
  // first kRA - 1), of the next step's row na_after, the next step's B fragment nb_after (-1: none).
  static constexpr int a_after(int p) {
    for (int r = kRA - 1; r < kMI; ++r)
      if ((r == kRA - 1 ? 0 : (r - kRA + 1) * kNI - 1) == p) return r;
    return -1;
  }
  static constexpr int na_after(int p) {
    for (int r = 0; r < kRA - 1; ++r) {
      const int free = (kMI - kRA + r + 1) * kNI - 1;
      if ((free > kBarP ? free : kBarP) == p) return r;
    }
    return -1;
  }
  static constexpr int nb_after(int p) {
    for (int c = 0; c < kNI; ++c)
      if ((kDB ? kBarP + 2 * c : kLastP + c) == p) return c;
    return -1;
  }
  static_assert(kDB || kRA == 2, "a deeper ring reads the next step's rows before the last");
  static constexpr int reads(int t, int p) {  // LDS reads after position p of step t
    const int own = !kPairScales || t % 2 == 0, next = !kPairScales || t % 2 == 1;  // with a scale?
    return ((A::k8 ? 2 : 1) + own) * (a_after(p) >= 0) + ((A::k8 ? 2 : 1) + next) * (na_after(p) >= 0) +
           ((B::k8 ? 2 : 1) + next) * (nb_after(p) >= 0);
  }
  // Transfers after position p of step t: the second half of the next stage at the head (every other
  // position; behind them the next quad's scales), the first half of the one after it behind the
  // barrier. head_at / tail_at: which transfer of its half goes out after position p (A's first), or -1.
  static constexpr int head_at(int p) { return p % 2 == 0 && p / 2 < kHalf ? p / 2 : -1; }
  static constexpr int tail_at(int p) {
    return p >= kBarP && (p - kBarP) % kTailStep == 0 && (p - kBarP) / kTailStep < kHalf ? (p - kBarP) / kTailStep : -1;
  }
  static constexpr bool in_step(bool is_a, bool tail, int t) {  // an E2M1 stage covers two steps
    return (is_a ? A::k8 : B::k8) || (t & 1) == (tail ? 1 : 0);
  }
  static constexpr int kScaleP = 2 * kHalf;
  static constexpr int transfers(int t, int p) {
    int n = p == kScaleP && t == 0;
    if (head_at(p) >= 0) n += in_step(head_at(p) < kHalfA, false, t);
    if (tail_at(p) >= 0) n += in_step(tail_at(p) < kHalfA, true, t);
    return n;
  }
  static_assert(kScaleP < kN, "the scales' transfer is issued inside the step");
  // Transfer u of the first (SECOND = false) or second half of the stage `slot` (a step of an E4M3
  // operand, a pair of an E2M1 one; 128 bytes of a row each) that is held in stage st.
  template <int U, bool SECOND>
  static __device__ __forceinline__ void transfer(const Src& s, int slot, GEP_LDS char* smem, int st, int wave) {
    if constexpr (U < kHalfA) {
      constexpr int q = U + (SECOND ? kInstrA / 2 : 0);
      dma<q, q + 1>(s.la, s.a, slot * 128, smem + st * kABytes, wave);
    } else {
      constexpr int q = U - kHalfA + (SECOND ? kInstrB / 2 : 0);
      dma<q, q + 1>(s.lb, s.b, slot * 128, smem + kBOff + st * kBBytes, wave);
    }
  }
  template <int T, int P, int E>
  static __device__ __forceinline__ void sched() {
    if constexpr (P < E) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if constexpr (reads(T, P) > 0) __builtin_amdgcn_sched_group_barrier(0x100, reads(T, P), 0);
      if constexpr (transfers(T, P) > 0) __builtin_amdgcn_sched_group_barrier(0x020, transfers(T, P), 0);
      sched<T, P + 1, E>();
    }
  }

  // Positions [P, E) of step T of quad q (so: its scale stage's offset; so_next: the next step's).
  template <bool MM, int T, int P, int E>
  static __device__ __forceinline__ void positions(f32x4 (&acc)[kMI][kNI], Frags& f, GEP_LDS char* smem, const Lane& o,
                                                   const Src& s, int q, int so, int so_next, int wave) {
    if constexpr (P < E) {
      constexpr int NT = (T + 1) & 3;
      if constexpr (MM) {
        constexpr int r = P / kNI, c = P % kNI;
        acc[r][c] = mx_mma<FA, FB, kPairScales ? T % 2 : 0>(f.b[bset(T)][c], f.a[r % kRA], acc[r][c], f.sb[sset(T)][c],
                                                            f.sa[kPairScales ? r : r % kRA]);
        if constexpr (a_after(P) >= 0) read_a<T>(f, smem, o, a_after(P), so);
        if constexpr (na_after(P) >= 0) read_a<NT>(f, smem, o, na_after(P), so_next);
        if constexpr (nb_after(P) >= 0) read_b<NT>(f, smem, o, nb_after(P), so_next);
      }
      const int step = q * 4 + T;
      constexpr int h = head_at(P), u = tail_at(P);
      if constexpr (h >= 0 && in_step(h < kHalfA, false, T)) {
        constexpr bool k8 = h < kHalfA ? A::k8 : B::k8;
        transfer<h, true>(s, (k8 ? step : step >> 1) + 1, smem, (h < kHalfA ? stage<FA>(T) : stage<FB>(T)) ^ 1, wave);
      }
      if constexpr (P == kScaleP && T == 0) dma_scales(s, q + 1, smem, (q + 1) & 1, wave);
      if constexpr (u >= 0 && in_step(u < kHalfA, true, T)) {
        constexpr bool k8 = u < kHalfA ? A::k8 : B::k8;
        transfer<u, false>(s, (k8 ? step : step >> 1) + 2, smem, u < kHalfA ? stage<FA>(T) : stage<FB>(T), wave);
      }
      positions<MM, T, P + 1, E>(acc, f, smem, o, s, q, so, so_next, wave);
    }
  }
  template <bool MM, int T>
  static __device__ __forceinline__ void step(f32x4 (&acc)[kMI][kNI], Frags& f, GEP_LDS char* smem, const Lane& lo,
                                              const Src& s, int q, int wave) {
    const int so = (q & 1) * kSBytes, so_next = T == 3 ? ((q + 1) & 1) * kSBytes : so;
    // opaque offsets: stage and block-row offsets then fold into the reads' immediates
    Lane o = lo;
    asm volatile("" : "+v"(o.a0), "+v"(o.a1), "+v"(o.b0), "+v"(o.b1), "+v"(o.sa), "+v"(o.sb));
    if constexpr (MM) {
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_setprio(1);
      __builtin_amdgcn_sched_barrier(0);
      positions<true, T, 0, kPrioP>(acc, f, smem, o, s, q, so, so_next, wave);
      sched<T, 0, kPrioP>();
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_setprio(0);
      __builtin_amdgcn_sched_barrier(0);
      positions<true, T, kPrioP, kBarP>(acc, f, smem, o, s, q, so, so_next, wave);
      sched<T, kPrioP, kBarP>();
      if constexpr (bar(T)) dma_barrier();
      positions<true, T, kBarP, kN>(acc, f, smem, o, s, q, so, so_next, wave);
      sched<T, kBarP, kN>();
      __builtin_amdgcn_sched_barrier(0);
    } else {
      positions<false, T, 0, kBarP>(acc, f, smem, o, s, q, so, so_next, wave);
      if constexpr (bar(T)) dma_barrier();
      positions<false, T, kBarP, kN>(acc, f, smem, o, s, q, so, so_next, wave);
    }
  }
  template <bool MM>
  static __device__ __forceinline__ void mainloop(f32x4 (&acc)[kMI][kNI], Frags& f, GEP_LDS char* smem, const Lane& o,
                                                  const Src& s, int steps, int wave) {
    for (int q = 0; q * 4 < steps; ++q) {
      step<MM, 0>(acc, f, smem, o, s, q, wave);
      step<MM, 1>(acc, f, smem, o, s, q, wave);
      if (q * 4 + 2 < steps) {
        step<MM, 2>(acc, f, smem, o, s, q, wave);
        step<MM, 3>(acc, f, smem, o, s, q, wave);
      }
    }
  }

  // ---- epilogue. It runs while the next tile's first transfers are under way (they fill stage 0),
  // through 4 KB a wave of A's stage 1. One 16-bit output without C: the values are final in the
  // accumulators, so they are converted there and pass through LDS as 16-bit rows (32 rows a
  // pass). Otherwise fp32 rows (16 a pass). Either way a lane then holds 8 consecutive columns, and C,
  // D and PostAct are accessed 16 bytes or more at a time, 128 bytes a row. Chunks are XOR-swizzled
  // by the row as in gemm_kernel.hpp's 16x16 epilogues.
  static constexpr int kRegion = 4096;
  static_assert(kRegion * NW <= kABytes, "the epilogue's buffers lie in a stage of A");
  static __device__ __forceinline__ int ebuf(int r, int c8, int hf) {
    return r * 256 + hf * 128 + ((c8 ^ ((r & 3) | ((r >> 1) & 4))) << 4);
  }
  static __device__ __forceinline__ int ebuf16(int r, int c) { return r * 128 + ((c ^ ((r >> 1) & 7)) << 4); }

  // Stores of the 16-bit path; the count lets the wait for the transfers issued before them leave
  // the stores in flight. (So every one is issued: rows and columns past the output go to an
  // offset that the range check drops.)
  static constexpr int kStores16 = kWM / 8;
  static constexpr int64_t kMaxLd16 = 1 << 22;  // its offsets inside a tile are 32-bit

  template <int DT>
  static __device__ __forceinline__ void epilogue16(const KParams& p, const MxTileInfo& ti, const f32x4 (&acc)[kMI][kNI],
                                                    GEP_LDS char* buf, int lane, int wm0, int wn0) {
    const bool post = p.p_dt != DT_NONE;
    const int64_t ld = post ? p.ldp : p.ldd;
    const int row0 = ti.m0 + wm0, col0 = ti.n0 + wn0;
    const __amdgpu_buffer_rsrc_t out =
        make_rsrc((post ? (char*)p.Post : (char*)p.D) + ((int64_t)row0 * ld + col0) * 2, 0x7FFFFFFF);
    const int q = lane >> 4, rl = lane >> 3, c = lane & 7;
    const bool col_ok = col0 + 8 * c < p.N;
#pragma unroll
    for (int pass = 0; pass < kMI / 2; ++pass) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = i * 16 + (lane & 15);
#pragma unroll
        for (int j = 0; j < kNI; j += 2) {
          const f32x4 &x = acc[pass * 2 + i][j], &y = acc[pass * 2 + i][j + 1];
          float v[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
          if (post) mx_act8(p.act, v);
          const uint2 lo = pack4_16(DT, v), hi = pack4_16(DT, v + 4);
          *(GEP_LDS i32x2*)(buf + ebuf16(r, 2 * j + (q >> 1)) + 8 * (q & 1)) = i32x2{(int)lo.x, (int)lo.y};
          *(GEP_LDS i32x2*)(buf + ebuf16(r, 2 * j + 2 + (q >> 1)) + 8 * (q & 1)) = i32x2{(int)hi.x, (int)hi.y};
        }
      }
      asm volatile("" ::: "memory");  // (LDS operations of a wave complete in order)
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const int r = it * 8 + rl;
        const i32x4 x = *(const GEP_LDS i32x4*)(buf + ebuf16(r, c));
        const bool ok = col_ok && row0 + pass * 32 + r < ti.row_end;
        __builtin_amdgcn_raw_buffer_store_b128(x, out, ok ? (uint32_t)((pass * 32 + r) * (int)ld * 2 + c * 16) : kOOB, 0, 0);
      }
      asm volatile("" ::: "memory");
    }
  }

  // Returns whether exactly kStores16 stores are the last vector memory operations issued.
  static __device__ __forceinline__ bool epilogue(const MxParams& mp, const MxTileInfo& ti, const f32x4 (&acc)[kMI][kNI],
                                                  GEP_LDS char* buf, int lane, int wm0, int wn0) {
    const KParams& p = mp.k;
    const bool slice = kSplit && mp.split > 1;
    asm volatile("" : "+v"(lane));
    if (!slice && p.c_dt == DT_NONE && (p.d_dt == DT_NONE) != (p.p_dt == DT_NONE)) {
      const int dt = p.d_dt != DT_NONE ? p.d_dt : p.p_dt;
      if ((p.d_dt != DT_NONE ? p.ldd : p.ldp) < kMaxLd16 && dt != DT_F32) {
        if (dt == DT_BF16) epilogue16<DT_BF16>(p, ti, acc, buf, lane, wm0, wn0);
        else epilogue16<DT_F16>(p, ti, acc, buf, lane, wm0, wn0);
        return true;
      }
    }
    const int row0 = ti.m0 + wm0, col0 = ti.n0 + wn0;
    const int rl = lane >> 3, n = col0 + 8 * (lane & 7);
#pragma unroll
    for (int pass = 0; pass < kMI; ++pass) {
#pragma unroll
      for (int j = 0; j < kNI; ++j)
        *(f32x4 GEP_LDS*)(buf + ebuf(lane & 15, 2 * j + (lane >> 5), (lane >> 4) & 1)) = acc[pass][j];
      asm volatile("" ::: "memory");
#pragma unroll
      for (int it = 0; it < 2; ++it) {
        const int r = it * 8 + rl;
        const int64_t m = row0 + pass * 16 + r;
        const f32x4 x0 = *(const f32x4 GEP_LDS*)(buf + ebuf(r, lane & 7, 0));
        const f32x4 x1 = *(const f32x4 GEP_LDS*)(buf + ebuf(r, lane & 7, 1));
        float v[8] = {x0[0], x0[1], x0[2], x0[3], x1[0], x1[1], x1[2], x1[3]};
        if (m < ti.row_end && n < p.N) {
          if (slice) mx_slice8(mp, ti.slice, m, n, v);
          else mx_finish8(p, m, n, v);
        }
      }
      asm volatile("" ::: "memory");
    }
    return false;
  }
  // All transfers issued before the last kStores16 operations have landed; then the workgroup meets.
  static __device__ __forceinline__ void dma_barrier_stores() {
    __builtin_amdgcn_sched_barrier(0);
    static_assert(kStores16 == 16 || kStores16 == 8, "the literal counts below");
    if constexpr (kStores16 == 16) asm volatile("s_waitcnt vmcnt(16) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    else asm volatile("s_waitcnt vmcnt(8) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  }

  static __device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }

  // Item u of this launch -> output tile. The map has tiles of BM x BN; in a split tail's launch
  // (p.tail == 2, the 128x128 kernels) of 256x256, and item u is quarter u & 3 of map tile t_lo + u / 4:
  // its rows (u & 1) and columns (u >> 1 & 1), possibly wholly outside the output.
  static __device__ __forceinline__ MxTileInfo decode(const MxParams& mp, int u, const int32_t* gstart, int t_lo) {
    const KParams& p = mp.k;
    const bool quarter = BM == 128 && p.tail == 2;
    const int MT = quarter ? 2 * BM : BM, NT = quarter ? 2 * BN : BN;
    MxTileInfo ti;
    ti.slice = kSplit && mp.split > 1 ? u / p.T : 0;  // slices of K: all tiles of the first, then the second, ...
    const int t = quarter ? t_lo + (u >> 2) : u - ti.slice * p.T;
    uint32_t mb, nb;
    int row_base = 0;
    if constexpr (VM) {
      int lo = 0, hi = p.L - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (gstart[mid] <= t) lo = mid; else hi = mid - 1;
      }
      row_base = p.cu_seqlens[lo];
      ti.row_end = p.cu_seqlens[lo + 1];
      ti.g = lo;
      raster(p, (uint32_t)(t - gstart[lo]), (uint32_t)((ti.row_end - row_base + MT - 1) / MT), (uint32_t)p.tn, p.fd_Gtn, mb, nb);
    } else {
      ti.g = 0;
      ti.row_end = p.M;
      raster(p, (uint32_t)t, (uint32_t)p.tm, (uint32_t)p.tn, p.fd_Gtn, mb, nb);
    }
    ti.g = uni(ti.g);
    ti.slice = uni(ti.slice);
    ti.m0 = uni(row_base + (int)mb * MT + (quarter ? (u & 1) * BM : 0));
    ti.n0 = uni((int)nb * NT + (quarter ? ((u >> 1) & 1) * BN : 0));
    ti.row_end = uni(ti.row_end);
    return ti;
  }

  static __device__ __forceinline__ void run(const MxParams& mp) {
    const KParams& p = mp.k;
    __shared__ __attribute__((aligned(1024))) char smem_raw[kLdsBytes + kVarlenLds];
    GEP_LDS char* smem = (GEP_LDS char*)smem_raw;
    const int tid = threadIdx.x, lane_id = tid & 63;
    const int wave = uni(tid >> 6);
    // 8 waves: w and w + 4 share a SIMD and take the two row halves of a column block
    const int wm0 = (wave / kWavesN) * kWM, wn0 = (wave % kWavesN) * kWN;

    int T = p.T;
    [[maybe_unused]] int32_t* gstart = nullptr;
    [[maybe_unused]] const int MT = BM == 128 && p.tail == 2 ? 2 * BM : BM;
    if constexpr (VM) {
      // tile offsets of the groups; an array that does not run 0 .. M without decreasing gives
      // no tiles (see gemm_kernel.hpp: the flag shares the one LDS array)
      gstart = (int32_t*)(smem_raw + kLdsBytes);
      int32_t* part = gstart + kMaxVarlenGroups + 1;
      volatile int32_t* s_bad = part + kThreads;
      if (tid == 0) *s_bad = 0;
      __syncthreads();
      constexpr int kPer = kMaxVarlenGroups / kThreads;
      int32_t local[kPer], sum = 0;
      int bad = 0;
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        const int g = tid * kPer + q;
        int32_t tiles = 0;
        if (g < p.L) {
          const int c0 = p.cu_seqlens[g], c1 = p.cu_seqlens[g + 1];
          bad |= c1 < c0 || (g == 0 && c0 != 0) || (g == p.L - 1 && c1 != p.M);
          tiles = c1 > c0 ? (int)(((int64_t)c1 - c0 + MT - 1) / MT) * p.tn : 0;
        }
        local[q] = sum;
        sum += tiles;
      }
      if (bad) *s_bad = 1;
      part[tid] = sum;
      __syncthreads();
      bad = uni(*s_bad);
      for (int off = 1; off < kThreads; off <<= 1) {
        const int32_t add = tid >= off ? part[tid - off] : 0;
        __syncthreads();
        part[tid] += add;
        __syncthreads();
      }
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        const int g = tid * kPer + q;
        if (g < p.L) gstart[g] = part[tid] - sum + local[q];
      }
      T = uni(bad ? 0 : part[kThreads - 1]);
      __syncthreads();
    }
    const int P = p.P;
    const bool xq = p.xcd_remap && (P & 7) == 0;
    const int bid = blockIdx.x;
    const int qx = xq ? bid & 7 : 0, qj = xq ? bid >> 3 : bid, Q = xq ? P >> 3 : P;
    int b0 = qx * Q + qj;
    // Split tail: when the last round of map tiles is partial and at most half full, the first
    // launch (tail 1) stops before it and a second one (tail 2) takes it in quarters. Both decide
    // from T. The second one's XCDs take a run of quarters each.
    int t_lo = 0, U = kSplit && mp.split > 1 ? T * mp.split : T;
    if (p.tail != 0) {
      const int rem = T % p.P_big;
      const bool split = T > p.P_big && rem > 0 && 2 * rem <= p.P_big;
      U = p.tail == 1 ? (split ? T - rem : T) : (split ? 4 * rem : 0);
      t_lo = T - rem;
      if (p.tail == 2 && xq && U <= P) {
        const int run = (U + 7) >> 3;
        b0 = qj < run ? qx * run + qj : U;
      }
    }

    MxTileInfo ti;
    Src s;
    int steps;
    // The tile's operands, and its first transfers: stage 0 and the first scales.
    auto begin_tile = [&](int t) {
      ti = decode(mp, t, gstart, t_lo);
      int lane = lane_id;
      asm volatile("" : "+v"(lane));  // (lane offsets are not kept across the main loop)
      const int q0 = kSplit ? ti.slice * mp.per : 0;  // the slice's first scale tile, four steps each
      const int ka = q0 * 4 * A::kStepBytes, kb = q0 * 4 * B::kStepBytes;
      steps = kSplit && mp.split > 1 ? min(mp.per * 4, mp.steps - q0 * 4) : mp.steps;
      init<kInstrA>(s.la, wave, lane, ti.row_end - ti.m0, (int)p.lda, (int)p.lda - ka);
      init<kInstrB>(s.lb, wave, lane, p.N - ti.n0, (int)p.ldb, (int)p.ldb - kb);
      const int64_t ao = (int64_t)ti.m0 * p.lda + ka, bo = (int64_t)ti.n0 * p.ldb + kb;
      s.a = make_rsrc((const char*)p.A + ao, p.a_bytes - ao);
      s.b = make_rsrc((const char*)p.B + (int64_t)ti.g * p.b_bytes + bo, p.b_bytes - bo);
      s.nsb = mp.nsb - q0;
      const bool is_a = wave < BM / 64;  // (waves past (BM + BN) / 64 move no scales)
      const int first = is_a ? ti.m0 : ti.n0;  // row of the tile's first scale
      const int i = (is_a ? wave : wave - BM / 64) * 64 + lane;  // row of the tile
      const int64_t so = ((int64_t)(first >> 6) * mp.nsb + q0) * 1024;
      s.s = make_rsrc(is_a ? mp.sa + so : mp.sb + (int64_t)ti.g * mp.sb_bytes + so,
                      (is_a ? mp.sa_bytes : mp.sb_bytes) - so);
      const int rr = (first & 63) + i;
      s.s_off = first + i < (is_a ? ti.row_end : p.N) ? (uint32_t)((rr >> 6) * mp.nsb * 1024 + (rr & 63) * 16) : kOOB;
      dma<0, kInstrA>(s.la, s.a, 0, smem, wave);
      dma<0, kInstrB>(s.lb, s.b, 0, smem + kBOff, wave);
      dma_scales(s, 0, smem, 0, wave);
    };

    if (b0 < U) begin_tile(b0);
    bool stores = false;  // the wave's last operations are the stores of epilogue16
    for (int t = b0; t < U;) {
      f32x4 acc[kMI][kNI];
#pragma unroll
      for (int i = 0; i < kMI; ++i)
#pragma unroll
        for (int j = 0; j < kNI; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
      // a wave whose rows or columns all lie past the output only moves data
      const bool idle = ti.m0 + wm0 >= ti.row_end || ti.n0 + wn0 >= p.N;
      // stage 0 has landed; the previous tile's epilogue buffers (stage 1) are free
      if (stores) dma_barrier_stores();
      else dma_barrier();
      dma<0, kInstrA / 2>(s.la, s.a, 128, smem + kABytes, wave);
      dma<0, kInstrB / 2>(s.lb, s.b, 128, smem + kBOff + kBBytes, wave);
      int lane = lane_id;
      asm volatile("" : "+v"(lane));
      const Lane o = lane_offsets(lane, wm0, wn0);
      Frags f;
      if (idle) {
        __builtin_amdgcn_s_setprio(0);
        mainloop<false>(acc, f, smem, o, s, steps, wave);
      } else {
#pragma unroll
        for (int r = 0; r < kRA - 1; ++r) read_a<0>(f, smem, o, r, 0);
#pragma unroll
        for (int c = 0; c < kNI; ++c) read_b<0>(f, smem, o, c, 0);
        mainloop<true>(acc, f, smem, o, s, steps, wave);
      }
      dma_barrier();  // transfers past K have landed and every wave has left the ring
      const MxTileInfo done = ti;
      t += P;
      if (t < U) begin_tile(t);
      asm volatile("" ::: "memory");  // (its transfers are issued before the epilogue's stores)
      __builtin_amdgcn_sched_barrier(0);
      stores = false;
      if (!idle) stores = epilogue(mp, done, acc, smem + kABytes + wave * kRegion, lane_id, wm0, wn0);
    }
  }
};

// ------------------------------------------------------------------------------------
// MxDirect
// ------------------------------------------------------------------------------------
// 16 MB x 16 NB outputs per workgroup of NW waves; wave w takes the scale tiles (512 values of
// K) w, w + NW, ... and reads its fragments straight from global memory, D steps ahead. With one
// row of activations the operand B is read once from HBM in 64-byte runs of 16 rows, and nothing
// waits on a barrier. The waves' partial sums meet in LDS in a fixed order.
template <int MB, int NB, int NW, int D, int FA, int FB, bool VM>
struct MxDirect {
  static constexpr int kBM = 16 * MB, kBN = 16 * NB;
  static constexpr int kPitch = kBN + 4;  // floats of a row of partial sums
  static constexpr int kPlane = kBM * kPitch;

  struct Buf {
    MxFrag<FA> a[MB];
    MxFrag<FB> b[NB];
  };
  struct Src {
    __amdgpu_buffer_rsrc_t a, b, sa, sb;
    uint32_t ao[MB], bo[NB], sao[MB], sbo[NB];  // this lane's rows (kOOB past the operand)
    int ka, kb;   // bytes of a row past the lane's first chunk
    int nsb;
  };
  template <int F>
  static __device__ __forceinline__ MxFrag<F> load(__amdgpu_buffer_rsrc_t rs, uint32_t off, int klim, int step) {
    MxFrag<F> f;
    const int kb = step * MxFmt<F>::kStepBytes;
    f.lo = __builtin_amdgcn_raw_buffer_load_b128(rs, kb < klim ? off + kb : kOOB, 0, 0);
    if constexpr (F == MX_E4M3) f.hi = __builtin_amdgcn_raw_buffer_load_b128(rs, kb + 64 < klim ? off + kb + 64 : kOOB, 0, 0);
    return f;
  }
  static __device__ __forceinline__ void fetch(Buf& b, const Src& s, int step) {
#pragma unroll
    for (int j = 0; j < NB; ++j) b.b[j] = load<FB>(s.b, s.bo[j], s.kb, step);
#pragma unroll
    for (int i = 0; i < MB; ++i) b.a[i] = load<FA>(s.a, s.ao[i], s.ka, step);
  }
  struct Scales {
    i32x4 a[MB], b[NB];
  };
  static __device__ __forceinline__ void fetch_scales(Scales& q, const Src& s, int tile) {
#pragma unroll
    for (int j = 0; j < NB; ++j) q.b[j] = __builtin_amdgcn_raw_buffer_load_b128(s.sb, tile < s.nsb ? s.sbo[j] + tile * 1024 : kOOB, 0, 0);
#pragma unroll
    for (int i = 0; i < MB; ++i) q.a[i] = __builtin_amdgcn_raw_buffer_load_b128(s.sa, tile < s.nsb ? s.sao[i] + tile * 1024 : kOOB, 0, 0);
  }
  // Byte t of the result: the lane's scale (byte l / 16 of word t) of step t.
  static __device__ __forceinline__ int gather_scale(const i32x4& w, uint32_t sel) {
    const uint32_t lo = __builtin_amdgcn_perm((uint32_t)w[1], (uint32_t)w[0], sel);
    const uint32_t hi = __builtin_amdgcn_perm((uint32_t)w[3], (uint32_t)w[2], sel);
    return (int)(lo | (hi << 16));
  }

  template <int T>
  static __device__ __forceinline__ void step(f32x4 (&acc)[MB][NB], Buf (&buf)[D], const Src& s, const int (&sa)[MB],
                                              const int (&sb)[NB], int tile) {
    Buf& b = buf[T % D];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = mx_mma<FA, FB, T>(b.b[j], b.a[i], acc[i][j], sb[j], sa[i]);
    // the step D further on, in this tile of scales or in the wave's next
    fetch(b, s, T + D < 4 ? tile * 4 + T + D : (tile + NW) * 4 + T + D - 4);
  }

  static __device__ __forceinline__ void run(const MxParams& mp) {
    const KParams& p = mp.k;
    __shared__ __attribute__((aligned(16))) float sums[NW * kPlane];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int g = 0, m0 = blockIdx.y * kBM, row_end = p.M;
    // this workgroup's scale tiles [t0, t1)
    const int slice = VM ? 0 : blockIdx.z, t0 = VM ? 0 : slice * mp.per, t1 = VM ? mp.nsb : min(mp.nsb, t0 + mp.per);
    const int n0 = blockIdx.x * kBN;
    if constexpr (VM) {
      // the group of row block blockIdx.y: 64 groups a pass, one a lane; the whole array is
      // checked (0 .. M, never decreasing)
      int base = 0, found = 0, bad = 0;
      const int want = blockIdx.y;
      for (int g0 = 0; g0 < p.L; g0 += 64) {
        const int gi = g0 + lane;
        int c0 = 0, c1 = 0;
        if (gi < p.L) {
          c0 = p.cu_seqlens[gi];
          c1 = p.cu_seqlens[gi + 1];
          bad |= c1 < c0 || (gi == 0 && c0 != 0) || (gi == p.L - 1 && c1 != p.M);
        }
        const int tiles = c1 > c0 ? (int)(((int64_t)c1 - c0 + kBM - 1) / kBM) : 0;
        int incl = tiles;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
          const int u = __shfl_up(incl, off);
          if (lane >= off) incl += u;
        }
        const int first = base + incl - tiles;
        const uint64_t hit = __ballot(want >= first && want < first + tiles);
        if (hit) {
          const int src = __ffsll((unsigned long long)hit) - 1;
          g = g0 + src;
          m0 = __shfl(c0, src) + (want - __shfl(first, src)) * kBM;
          row_end = __shfl(c1, src);
          found = 1;
        }
        base += __shfl(incl, 63);
      }
      if (__ballot(bad) || !found) return;  // (the same in every wave)
      g = __builtin_amdgcn_readfirstlane(g);
      m0 = __builtin_amdgcn_readfirstlane(m0);
      row_end = __builtin_amdgcn_readfirstlane(row_end);
    }
    const int r = lane & 15, kg = lane >> 4;
    Src s;
    const int64_t ao = (int64_t)m0 * p.lda, bo = (int64_t)n0 * p.ldb;
    s.a = make_rsrc((const char*)p.A + ao, p.a_bytes - ao);
    s.b = make_rsrc((const char*)p.B + (int64_t)g * p.b_bytes + bo, p.b_bytes - bo);
    const int64_t sao = (int64_t)(m0 >> 6) * mp.nsb * 1024, sbo = (int64_t)(n0 >> 6) * mp.nsb * 1024;
    s.sa = make_rsrc(mp.sa + sao, mp.sa_bytes - sao);
    s.sb = make_rsrc(mp.sb + (int64_t)g * mp.sb_bytes + sbo, mp.sb_bytes - sbo);
    s.nsb = t1;
    s.ka = min((int)p.lda, t1 * 4 * MxFmt<FA>::kStepBytes) - kg * 16;
    s.kb = min((int)p.ldb, t1 * 4 * MxFmt<FB>::kStepBytes) - kg * 16;
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const int row = i * 16 + r, q = (m0 & 63) + row;
      s.ao[i] = m0 + row < row_end ? (uint32_t)(row * (int)p.lda + kg * 16) : kOOB;
      s.sao[i] = m0 + row < row_end ? (uint32_t)((q >> 6) * mp.nsb * 1024 + (q & 63) * 16) : kOOB;
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int row = j * 16 + r, q = (n0 & 63) + row;
      s.bo[j] = n0 + row < p.N ? (uint32_t)(row * (int)p.ldb + kg * 16) : kOOB;
      s.sbo[j] = n0 + row < p.N ? (uint32_t)((q >> 6) * mp.nsb * 1024 + (q & 63) * 16) : kOOB;
    }
    f32x4 acc[MB][NB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    if (t0 + wave < t1) {
      const uint32_t sel = (uint32_t)kg | ((uint32_t)(4 + kg) << 8) | 0x0C0C0000u;  // (0x0C: a zero byte)
      Scales sc;
      fetch_scales(sc, s, t0 + wave);
      Buf buf[D];
#pragma unroll
      for (int t = 0; t < D; ++t) fetch(buf[t], s, (t0 + wave) * 4 + t);
      for (int tile = t0 + wave; tile < t1; tile += NW) {
        int sa[MB], sb[NB];
#pragma unroll
        for (int i = 0; i < MB; ++i) sa[i] = gather_scale(sc.a[i], sel);
#pragma unroll
        for (int j = 0; j < NB; ++j) sb[j] = gather_scale(sc.b[j], sel);
        fetch_scales(sc, s, tile + NW);
        step<0>(acc, buf, s, sa, sb, tile);
        step<1>(acc, buf, s, sa, sb, tile);
        step<2>(acc, buf, s, sa, sb, tile);
        step<3>(acc, buf, s, sa, sb, tile);
      }
    }
    // lane l of block (i, j) holds row l % 16, columns 4 (l / 16) + [0, 4)
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
        *(f32x4*)(sums + wave * kPlane + (i * 16 + r) * kPitch + j * 16 + kg * 4) = acc[i][j];
    __syncthreads();
    for (int u = tid; u < kBM * kBN / 8; u += NW * 64) {
      const int row = u / (kBN / 8), col = u % (kBN / 8) * 8;
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float* q = sums + w * kPlane + row * kPitch + col;
        const f32x4 x = *(const f32x4*)q, y = *(const f32x4*)(q + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += x[e], v[4 + e] += y[e];
      }
      if (m0 + row < row_end && n0 + col < p.N) {
        if (!VM && mp.split > 1) mx_slice8(mp, slice, m0 + row, n0 + col, v);
        else mx_finish8(p, m0 + row, n0 + col, v);
      }
    }
  }
};

template <int BM, int BN, int NW, int FA, int FB, bool VM>
__global__ __launch_bounds__(NW * 64, (NW == 8 ? 1 : 2)) void mx_ring_kernel(const MxParams p) {
  MxRing<BM, BN, NW, FA, FB, VM>::run(p);
}
template <int MB, int NB, int NW, int D, int FA, int FB, bool VM>
__global__ __launch_bounds__(NW * 64) void mx_direct_kernel(const MxParams p) {
  MxDirect<MB, NB, NW, D, FA, FB, VM>::run(p);
}

// The kernels (launch configuration by mx_plan.cpp).
template <int FA, int FB, bool VM>
hipError_t mx_launch(int32_t tile, const MxParams& p, dim3 grid, hipStream_t s);

#define GEP_MX_LAUNCH(FA, FB, VM)                                                                    \
  template <>                                                                                        \
  hipError_t mx_launch<FA, FB, VM>(int32_t tile, const MxParams& p, dim3 grid, hipStream_t s) {      \
    switch (tile) {                                                                                  \
      case MX_TILE_256: mx_ring_kernel<256, 256, 8, FA, FB, VM><<<grid, 512, 0, s>>>(p); break;      \
      case MX_TILE_128: mx_ring_kernel<128, 128, 4, FA, FB, VM><<<grid, 256, 0, s>>>(p); break;      \
      case MX_TILE_32X64: mx_direct_kernel<2, 4, 4, 2, FA, FB, VM><<<grid, 256, 0, s>>>(p); break;   \
      case MX_TILE_32: mx_direct_kernel<2, 2, 4, 2, FA, FB, VM><<<grid, 256, 0, s>>>(p); break;      \
      case MX_TILE_16X32: mx_direct_kernel<1, 2, 8, 2, FA, FB, VM><<<grid, 512, 0, s>>>(p); break;   \
      case MX_TILE_16: mx_direct_kernel<1, 1, 8, 2, FA, FB, VM><<<grid, 512, 0, s>>>(p); break;      \
      default: return hipErrorInvalidValue;                                                          \
    }                                                                                                \
    return hipGetLastError();                                                                        \
  }

}  // namespace gep
