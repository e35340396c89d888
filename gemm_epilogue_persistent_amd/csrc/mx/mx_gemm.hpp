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
//   MxRing   large problems. 256x256 outputs per workgroup of 8 waves, 128x128 of 4: both operands go
//            through LDS (global -> LDS transfers, two to four stages), persistent tile loop.
//   MxDirect few rows. 16x16 to 32x64 outputs per workgroup, whose waves share out K and read
//            their fragments from global memory themselves; one join in LDS at the end.
// MxRing 8192^3 e2m1 x e2m1: 246 us, 4.47 PFLOP/s (in short bursts 233, in long runs 254); the matrix pipes
// are busy 62% of the cycles, and the chip holds 1.79 GHz of its 2.4 under that load. LDS is busy 37% of the
// cycles; 18% of those are conflicts of the scale bytes' reads (see Lane). 16768 x 4096 x 4096 e4m3 x e2m1 over
// 8 experts: 237 to 241 us, 2.35 PFLOP/s, 59% busy at 2.04 GHz; a library product of e4m3 8192^3 reaches 2.66.
// MxDirect 1 x 8192 x 8192 e4m3 x e2m1: 8.0 us in a graph, 8.4 between other kernels, for 35.7 MB, of which 2.5
// us are the launch. 256x128 tiles were measured and are not kept: as fast as 128x128 at 4096 x 2048 x 4096 e4m3,
// one round either way, and 28 us for 22 at 2048 x 2048 x 4096.
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
  int32_t cus;  // compute units of the device
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

// The group that holds tile `want` when every group has ceil(rows / bm) * per tiles: its index, rows
// [begin, end) and first tile. 64 groups a pass, one a lane; every lane gets the result. The whole
// offset array is checked (0 .. M, never decreasing): if it is not such, or `want` is in no group, index
// is -1 and first the number of tiles (0 for a bad array).
struct MxGroup {
  int index, begin, end, first;
};
__device__ __forceinline__ MxGroup mx_find_group(const KParams& p, int want, int bm, int per, int lane) {
  MxGroup r{-1, 0, 0, 0};
  int base = 0, bad = 0, first_hit = 0;
  for (int g0 = 0; g0 < p.L; g0 += 64) {
    const int gi = g0 + lane;
    int c0 = 0, c1 = 0;
    if (gi < p.L) {
      c0 = p.cu_seqlens[gi];
      c1 = p.cu_seqlens[gi + 1];
      bad |= c1 < c0 || (gi == 0 && c0 != 0) || (gi == p.L - 1 && c1 != p.M);
    }
    const int tiles = c1 > c0 ? (int)(((int64_t)c1 - c0 + bm - 1) / bm) * per : 0;
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
      r.index = g0 + src;
      r.begin = __shfl(c0, src);
      r.end = __shfl(c1, src);
      first_hit = __shfl(first, src);
    }
    base += __shfl(incl, 63);
  }
  if (__ballot(bad)) return MxGroup{-1, 0, 0, 0};
  r.first = r.index >= 0 ? first_hit : base;
  r.index = __builtin_amdgcn_readfirstlane(r.index);
  r.begin = __builtin_amdgcn_readfirstlane(r.begin);
  r.end = __builtin_amdgcn_readfirstlane(r.end);
  r.first = __builtin_amdgcn_readfirstlane(r.first);
  return r;
}

// Which epilogue of MxRing: 0 any types, and slices of K; 1 one 16-bit output without C; else 16-bit rows,
// 2 + (C) + 2 (both outputs). (16-bit offsets inside a tile are 32-bit: 256 rows of less than 2^22.)
constexpr int64_t kMaxLd16 = 1 << 22;
__host__ __device__ __forceinline__ int mx_epilogue_kind(const MxParams& mp) {
  const KParams& p = mp.k;
  if (mp.split > 1) return 0;
  auto fits = [](int dt, int64_t ld) { return dt == DT_NONE || (dt != DT_F32 && ld < kMaxLd16); };
  if (!fits(p.c_dt, p.ldc) || !fits(p.d_dt, p.ldd) || !fits(p.p_dt, p.ldp)) return 0;
  const int c = p.c_dt != DT_NONE, both = p.d_dt != DT_NONE && p.p_dt != DT_NONE;
  return !c && !both ? 1 : 2 + c + 2 * both;
}

// ------------------------------------------------------------------------------------
// MxRing
// ------------------------------------------------------------------------------------
// A stage holds kSPS steps (of 128 values of K) of both operands: two steps of two E2M1 operands
// (128 bytes a row), else one (128 bytes a row of E4M3, 64 of E2M1). NS stages lie in LDS: one is
// being multiplied, the next has landed or is landing, the others are on their way. The scales of
// four steps (a quad; 16 bytes a row, in storage order) go through a two-stage ring of their own.
// Steps past K read zero codes.
//
// A step is kMI x kNI MFMAs, row by row. kRA A fragments are held in a ring (block row r in r %
// kRA; r is read after row r - kRA's last MFMA) and the kNI B fragments of the step, with kDB
// those of the next step too. The barrier comes when every wave has read its last fragment of
// the stage; it also waits for the transfers of the next stage (those of later stages, issued
// after them, may be outstanding). After it the next step's first fragments are read and the first
// half of the transfers into the freed stage goes out; the second half follows at the head of the
// next step.
//
// The parts that depend on how operands are scaled are the class's that derives from this one (Self; MxRing itself
// for MX operands): Src, Lane, Frags, scale_source, dma_scales, lane_offsets, first_reads, positions, sched, drain.
//
// EPI: the epilogues of the kernel, all kinds (0), kind 1 (1) or the others (2). Kind 1 has a kernel of
// its own where the larger code costs it something: in 128x128 tiles (4096 x 2048 x 4096 e4m3, 4%) and in
// 256x256 tiles of two E2M1 operands (8192^3, 1%), but not in those with an E4M3 operand (16384 x 4096 x
// 4096, 1% faster in one kernel than in two).
template <int BM, int BN, int NW, int NS, int FA, int FB, bool VM, int EPI>
struct MxRing {
  static constexpr int kThreads = NW * 64;
  static constexpr bool kSplit = BM == 128 && !VM && EPI != 1;  // may run slices of K
  static constexpr int kWN = 64, kWavesN = BN / kWN, kWavesM = NW / kWavesN, kWM = BM / kWavesM;
  static constexpr int kMI = kWM / 16, kNI = kWN / 16;
  using A = MxFmt<FA>;
  using B = MxFmt<FB>;
  static constexpr bool kDeep = FA == MX_E2M1 && FB == MX_E2M1;
  static constexpr int kSPS = kDeep ? 2 : 1;
  static constexpr int kRowA = A::kStepBytes * kSPS, kRowB = B::kStepBytes * kSPS;  // bytes of a row in a stage
  static constexpr int kABytes = BM * kRowA, kBBytes = BN * kRowB, kStage = kABytes + kBBytes;
  static constexpr int kSOff = NS * kStage, kSBytes = (BM + BN) * 16;
  static constexpr int kLdsBytes = kSOff + 2 * kSBytes;
  static constexpr int kInstrA = kABytes / 1024 / NW, kInstrB = kBBytes / 1024 / NW;  // a wave's transfers of a stage
  static constexpr int kPer = kInstrA + kInstrB;
  static constexpr int kHalfA = kInstrA / 2, kHalf = kHalfA + kInstrB / 2;  // half a stage: A's transfers, then B's
  static_assert((BM + BN) / 64 <= NW, "at most one scale transfer (64 rows) a wave");
  static_assert(kMI >= 4 && kMI % 2 == 0 && kNI == 4, "the fragment schedule below");
  static_assert(kInstrA % 2 == 0 && kInstrB % 2 == 0 && kInstrA <= 4 && kInstrB <= 4, "half a stage at a time");
  static_assert(NS >= 2 && NS <= (kSPS == 2 ? 3 : 4), "a quad's scales must have landed by its predecessor's last barrier");
  static constexpr int kStores16 = kWM / 8;  // stores of the 16-bit epilogue (see there)
  static constexpr int kAhead = (NS - 2) * kPer;  // transfers that may be outstanding at a barrier
  static constexpr int kN = kMI * kNI, kLastP = kN - kNI;
  // (What the registers hold next to the accumulators. With two stages an earlier barrier leaves the
  // transfers less time: E4M3 x E4M3, 128x128 tiles, 8192^3, 6% slower.)
  static constexpr int kRA = kDeep || (BM == 128 && NS > 2) ? 4 : 2;
  static constexpr bool kDB = FB == MX_E2M1 || (BM == 128 && NS > 2);
  // The barrier's position: past the last read of the step's own fragments, and past the head's
  // transfers if they belong to the same stage; without kDB, where the next step's fragments find
  // free registers.
  static constexpr int kFreeP = (kMI - kRA) * kNI, kHeadEnd = kSPS == 1 ? 2 * kHalf : kNI;
  static constexpr int kBarP = !kDB ? kLastP : (kFreeP > kHeadEnd ? kFreeP : kHeadEnd);
  // Two E2M1 operands: lane group g takes the K blocks c = {0, 6, 2, 4}[g] and c + 1 of the eight
  // of a pair of steps, one in each step (A and B alike, so the same products meet). Its two
  // scales are then neighbours and read as one.
  static constexpr bool kPairScales = kDeep;
  static constexpr int kPrioP = (kBarP / 2 + 3) / 4 * 4;
  static constexpr int kTailStep = (kN - kBarP) / kHalf;  // between the transfers after the barrier

  // 16-byte chunk c of row r of a stage lies at chunk c ^ key(r). A ds_read_b128 serves 16 lanes
  // at a time, rows 0-3 and 12-15 of one lane group with rows 4-11 of its neighbour, and so on.
  // Under these keys their chunks lie in distinct banks when those of neighbouring groups differ
  // by 1, 6 or 7 (rows of 128 bytes; by 4: every read twice as long, counted), or by 1 (64 bytes).
  template <int ROW>
  static __device__ __forceinline__ int key(int r) { return ROW == 128 ? kswz(r) : ((r >> 3) & 1) * 2; }

  template <int N>
  struct Loader {  // this lane's share of one operand's transfers
    uint32_t off[N];
    int32_t klim;  // bytes of a row past this lane's chunk
  };
  template <int ROW, int N>
  static __device__ __forceinline__ void init(Loader<N>& l, int wave, int lane, int rows_valid, int ld, int row_bytes) {
    constexpr int cpr = ROW / 16, rpi = 64 / cpr;  // chunks of a row, rows of a transfer
    const int c = (lane % cpr) ^ key<ROW>(wave * rpi + lane / cpr);  // (the key repeats every 16 rows)
#pragma unroll
    for (int q = 0; q < N; ++q) {
      const int row = (q * NW + wave) * rpi + lane / cpr;
      l.off[q] = row < rows_valid ? (uint32_t)(row * ld + c * 16) : kOOB;
    }
    l.klim = row_bytes - c * 16;
  }
  // Transfers [Q0, Q1) of one operand's part (at `lds`) of a stage: the rows' bytes from kb on. (kb is
  // added to the lane's offset: the range check, which turns kOOB into zeros, is stated for that
  // sum. An offset is below 2^31, so kOOB + kb does not wrap.)
  template <int Q0, int Q1, int N>
  static __device__ __forceinline__ void dma(const Loader<N>& l, __amdgpu_buffer_rsrc_t rs, int kb, GEP_LDS char* lds,
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
    Loader<kInstrA> la;
    Loader<kInstrB> lb;
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
  // Transfer U of the first (SECOND = false) or second half of the K range's stage number `n`, to `lds`.
  template <int U, bool SECOND>
  static __device__ __forceinline__ void transfer(const Src& s, int n, GEP_LDS char* lds, int wave) {
    if constexpr (U < kHalfA) {
      constexpr int q = U + (SECOND ? kInstrA / 2 : 0);
      dma<q, q + 1>(s.la, s.a, n * kRowA, lds, wave);
    } else {
      constexpr int q = U - kHalfA + (SECOND ? kInstrB / 2 : 0);
      dma<q, q + 1>(s.lb, s.b, n * kRowB, lds + kABytes, wave);
    }
  }

  // Wait until at most kAhead of this wave's vector memory operations are outstanding (and `more` x
  // kStores16 besides; 0, 1 or 2, the same in every lane) and its LDS operations are done; then the
  // workgroup meets. (The branches are inside the asm: as one of the compiler's it would cut the step
  // into blocks and the accumulators would move between them.)
  static __device__ __forceinline__ void ring_barrier() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kAhead) : "memory");
    __builtin_amdgcn_sched_barrier(0);
  }
  static __device__ __forceinline__ void ring_barrier(int more) {
    static_assert(kAhead + 2 * kStores16 < 64, "a six-bit counter");
    __builtin_amdgcn_sched_barrier(0);
    asm volatile(
        "s_cmp_lt_u32 %3, 1\n\ts_cbranch_scc0 1f\n\ts_waitcnt vmcnt(%0)\n1:\n\t"
        "s_cmp_lt_u32 %3, 2\n\ts_cbranch_scc0 2f\n\ts_waitcnt vmcnt(%1)\n2:\n\t"
        "s_waitcnt vmcnt(%2) lgkmcnt(0)\n\ts_barrier" ::"n"(kAhead),
        "n"(kAhead + kStores16), "n"(kAhead + 2 * kStores16), "s"(more)
        : "memory", "scc");
    __builtin_amdgcn_sched_barrier(0);
  }

  // Lane offsets of the fragments in a stage, and of the scale bytes from kSOff on. (The keys are the
  // fragments'. A scale is a byte or two of a row of 16 bytes, so 16 rows of a read meet in pairs in 32
  // banks: two conflict cycles a read, 18 to 20% of the LDS cycles.)
  struct Lane {
    int a, b, sa, sb;
  };
  static __device__ __forceinline__ Lane lane_offsets(int lane, int wm0, int wn0) {
    Lane o;
    const int ra = wm0 + (lane & 15), rb = wn0 + (lane & 15), g = lane >> 4;
    const int c = kPairScales ? (0x4260 >> (4 * g)) & 7 : g;  // the lane group's first chunk and K block
    o.a = ra * kRowA + ((c ^ key<kRowA>(ra)) << 4);
    o.b = kABytes + rb * kRowB + ((c ^ key<kRowB>(rb)) << 4);
    o.sa = kSOff + ra * 16 + c;
    o.sb = kSOff + (BM + rb) * 16 + c;
    return o;
  }
  // The fragment of block row r whose first chunk of row block 0 is at p (E4M3: p2 the second one).
  template <int F, int ROW>
  static __device__ __forceinline__ MxFrag<F> read(const GEP_LDS char* smem, int p, int p2, int r) {
    MxFrag<F> f;
    f.lo = *(const GEP_LDS i32x4*)(smem + p + r * 16 * ROW);
    if constexpr (F == MX_E4M3) f.hi = *(const GEP_LDS i32x4*)(smem + p2 + r * 16 * ROW);
    return f;
  }

  struct Frags {
    MxFrag<FA> a[kRA];
    MxFrag<FB> b[kDB ? 2 : 1][kNI];
    int sa[kPairScales ? kMI : kRA], sb[kDB ? 2 : 1][kNI];
  };
  static constexpr int bset(int t) { return kDB ? t & 1 : 0; }
  static constexpr int sset(int t) { return !kDB ? 0 : (kPairScales ? (t >> 1) & 1 : t & 1); }
  static constexpr int sa_at(int r) { return kPairScales ? r : r % kRA; }
  struct At {  // addresses of one step's fragments and scales
    int a, a2, b, b2, sa, sb;
  };
  template <int T>
  static __device__ __forceinline__ At at(const Lane& o, int stage, int scale_stage) {
    constexpr int flip = kSPS == 2 && (T & 1) ? 16 : 0;  // the second step's chunk
    At x{(o.a ^ flip) + stage, (o.a ^ 64) + stage, (o.b ^ flip) + stage, (o.b ^ 64) + stage, o.sa + scale_stage, o.sb + scale_stage};
    // opaque: block-row offsets then fold into the reads' immediates
    asm volatile("" : "+v"(x.a), "+v"(x.b), "+v"(x.sa), "+v"(x.sb));
    if constexpr (A::k8) asm volatile("" : "+v"(x.a2));
    if constexpr (B::k8) asm volatile("" : "+v"(x.b2));
    return x;
  }
  template <int T>
  static __device__ __forceinline__ void read_scale(int& v, const GEP_LDS char* p) {
    if constexpr (!kPairScales) v = *(const GEP_LDS uint8_t*)(p + T * 4);
    else if constexpr (T % 2 == 0) v = *(const GEP_LDS uint16_t*)(p + T * 4);
  }
  template <int T>
  static __device__ __forceinline__ void read_a(Frags& f, const GEP_LDS char* smem, const At& x, int r) {
    f.a[r % kRA] = read<FA, kRowA>(smem, x.a, x.a2, r);
    read_scale<T>(f.sa[sa_at(r)], smem + x.sa + r * 256);
  }
  template <int T>
  static __device__ __forceinline__ void read_b(Frags& f, const GEP_LDS char* smem, const At& x, int c) {
    f.b[bset(T)][c] = read<FB, kRowB>(smem, x.b, x.b2, c);
    read_scale<T>(f.sb[sset(T)][c], smem + x.sb + c * 256);
  }

  // What is read after position p: the A fragment of this step's row a_after (the rows past the ring's
  // first kRA - 1), of the next step's row na_after, the next step's B fragment nb_after (-1: none).
  static constexpr int a_after(int p) {
    for (int r = kRA - 1; r < kMI; ++r)
      if ((r == kRA - 1 ? 0 : (r - kRA + 1) * kNI - 1) == p) return r;
    return -1;
  }
  static constexpr int na_after(int p) {
    for (int r = 0; r < kRA - 1; ++r) {
      const int free = (kMI - kRA + r + 1) * kNI - 1, first = kBarP + (kDB ? 2 * r + 1 : 0);
      if ((free > first ? free : first) == p) return r;
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
  // Transfers after position p of step t: the second half of the stage NS - 1 ahead at the head of a
  // stage's first step (every other position; behind them the next quad's scales), the first half of
  // the one NS ahead behind the barrier, in its last. head_at / tail_at: which transfer of its half
  // goes out after position p (A's first), or -1.
  static constexpr bool first_step(int t) { return t % kSPS == 0; }
  static constexpr bool last_step(int t) { return t % kSPS == kSPS - 1; }
  static constexpr int head_at(int t, int p) { return first_step(t) && p % 2 == 0 && p / 2 < kHalf ? p / 2 : -1; }
  static constexpr int tail_at(int t, int p) {
    return last_step(t) && p >= kBarP && (p - kBarP) % kTailStep == 0 && (p - kBarP) / kTailStep < kHalf ? (p - kBarP) / kTailStep : -1;
  }
  static constexpr int kScaleP = 2 * kHalf;
  static_assert((kSPS == 2 || 2 * (kHalf - 1) < kBarP) && kScaleP < kN, "the head's transfers come before the stage's barrier");
  static constexpr int transfers(int t, int p) { return (p == kScaleP && t == 0) + (head_at(t, p) >= 0) + (tail_at(t, p) >= 0); }

  template <int T, int P, int E>
  static __device__ __forceinline__ void sched() {
    if constexpr (P < E) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if constexpr (reads(T, P) > 0) __builtin_amdgcn_sched_group_barrier(0x100, reads(T, P), 0);
      if constexpr (transfers(T, P) > 0) __builtin_amdgcn_sched_group_barrier(0x020, transfers(T, P), 0);
      sched<T, P + 1, E>();
    }
  }

  // The offsets of the previous, this and the next stage.
  struct Stages {
    int prev, cur, next;
    __device__ __forceinline__ void advance() {
      prev = cur;
      cur = next;
      next = next + kStage == kSOff ? 0 : next + kStage;
      asm volatile("" : "+s"(next));  // (known, the compiler would keep addresses of all stages)
    }
  };

  // Positions [P, E) of step T of quad q (x: this step's addresses, y: the next one's).
  template <bool MM, int T, int P, int E>
  static __device__ __forceinline__ void positions(f32x4 (&acc)[kMI][kNI], Frags& f, GEP_LDS char* smem, const At& x,
                                                   const At& y, const Src& s, int q, const Stages& st, int wave) {
    if constexpr (P < E) {
      constexpr int NT = (T + 1) & 3;
      if constexpr (MM) {
        constexpr int r = P / kNI, c = P % kNI;
        acc[r][c] = mx_mma<FA, FB, kPairScales ? T % 2 : 0>(f.b[bset(T)][c], f.a[r % kRA], acc[r][c], f.sb[sset(T)][c], f.sa[sa_at(r)]);
        if constexpr (a_after(P) >= 0) read_a<T>(f, smem, x, a_after(P));
        if constexpr (na_after(P) >= 0) read_a<NT>(f, smem, y, na_after(P));
        if constexpr (nb_after(P) >= 0) read_b<NT>(f, smem, y, nb_after(P));
      }
      constexpr int h = head_at(T, P), u = tail_at(T, P);
      const int n = (q * 4 + T) / kSPS;  // this stage's number
      if constexpr (h >= 0) transfer<h, true>(s, n + NS - 1, smem + st.prev, wave);
      if constexpr (P == kScaleP && T == 0) dma_scales(s, q + 1, smem, (q + 1) & 1, wave);
      if constexpr (u >= 0) transfer<u, false>(s, n + NS, smem + st.cur, wave);
      positions<MM, T, P + 1, E>(acc, f, smem, x, y, s, q, st, wave);
    }
  }

  // The first step's fragments, before the main loop; what is left to add behind it.
  static __device__ __forceinline__ void first_reads(Frags& f, const GEP_LDS char* smem, const Lane& o) {
    const At x = at<0>(o, 0, 0);
#pragma unroll
    for (int r = 0; r < kRA - 1; ++r) read_a<0>(f, smem, x, r);
#pragma unroll
    for (int c = 0; c < kNI; ++c) read_b<0>(f, smem, x, c);
  }
  static __device__ __forceinline__ void drain(f32x4 (&)[kMI][kNI], Frags&) {}

  // stores: the stores x kStores16 stores of the previous tile's epilogue lie between this tile's transfers
  // of stage NS - 2 and NS - 1, and need not be waited for before those.
  template <class Self, bool MM, int T>
  static __device__ __forceinline__ void step(f32x4 (&acc)[kMI][kNI], typename Self::Frags& f, GEP_LDS char* smem,
                                              const typename Self::Lane& lo, const typename Self::Src& s, int q, Stages& st,
                                              int stores, int wave) {
    const int so = (q & 1) * kSBytes, so_next = T == 3 ? ((q + 1) & 1) * kSBytes : so;
    const At x = at<T>(lo, st.cur, so), y = at<(T + 1) & 3>(lo, last_step(T) ? st.next : st.cur, so_next);
    if constexpr (MM) {
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_setprio(1);
      __builtin_amdgcn_sched_barrier(0);
      Self::template positions<true, T, 0, kPrioP>(acc, f, smem, x, y, s, q, st, wave);
      Self::template sched<T, 0, kPrioP>();
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_setprio(0);
      __builtin_amdgcn_sched_barrier(0);
    }
    Self::template positions<MM, T, MM ? kPrioP : 0, kBarP>(acc, f, smem, x, y, s, q, st, wave);
    if constexpr (MM) Self::template sched<T, kPrioP, kBarP>();
    if constexpr (last_step(T)) {
      if constexpr (T / kSPS <= NS - 3) ring_barrier(stores);
      else ring_barrier();
    }
    Self::template positions<MM, T, kBarP, kN>(acc, f, smem, x, y, s, q, st, wave);
    if constexpr (MM) {
      Self::template sched<T, kBarP, kN>();
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (last_step(T)) st.advance();
  }
  template <class Self, bool MM>
  static __device__ __forceinline__ void mainloop(f32x4 (&acc)[kMI][kNI], typename Self::Frags& f, GEP_LDS char* smem,
                                                  const typename Self::Lane& o, const typename Self::Src& s, int steps,
                                                  int stores, int wave) {
    Stages st{(NS - 1) * kStage, 0, kStage};
    int q = 0;
    for (; q * 4 + 2 < steps; ++q) {
      step<Self, MM, 0>(acc, f, smem, o, s, q, st, stores, wave);
      step<Self, MM, 1>(acc, f, smem, o, s, q, st, stores, wave);
      step<Self, MM, 2>(acc, f, smem, o, s, q, st, stores, wave);
      step<Self, MM, 3>(acc, f, smem, o, s, q, st, stores, wave);
      stores = 0;
    }
    if (q * 4 < steps) {
      step<Self, MM, 0>(acc, f, smem, o, s, q, st, stores, wave);
      step<Self, MM, 1>(acc, f, smem, o, s, q, st, stores, wave);
    }
  }

  // ---- epilogue. It runs while the next tile's first transfers are under way (all stages but the
  // last), through 4 KB a wave of the last stage. One 16-bit output without C: the values are final in the
  // accumulators, so they are converted there and pass through LDS as 16-bit rows (32 rows a
  // pass); a 16-bit C is then loaded four or eight rows a lane ahead, the first of them before the next
  // tile's transfers (16384 x 4096 x 4096 e4m3 x e2m1 with C 218 us, each row's load waited for in its
  // turn 237, without C 196; 8192 x 8192 x 2048 e2m1 with C 102 and 124, without 81). Either way a lane then holds 8
  // consecutive columns, and C, D and PostAct are accessed 16 bytes or more at a time, 128 bytes a
  // row. Chunks are XOR-swizzled by the row as in gemm_kernel.hpp's 16x16 epilogues.
  static constexpr int kRegion = 4096;
  static_assert(kRegion * NW <= kStage, "the epilogue's buffers lie in one stage");
  static __device__ __forceinline__ int ebuf(int r, int c8, int hf) {
    return r * 256 + hf * 128 + ((c8 ^ ((r & 3) | ((r >> 1) & 4))) << 4);
  }
  static __device__ __forceinline__ int ebuf16(int r, int c) { return r * 128 + ((c ^ ((r >> 1) & 7)) << 4); }

  // Stores of the 16-bit path; the count lets the wait for the transfers issued before them leave
  // the stores in flight. (So every one is issued: rows and columns past the output go to an
  // offset that the range check drops.)
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

  // 16-bit rows of C, D and PostAct with C or both outputs. Row i * 8 + lane / 8 of the wave's is item i of
  // a lane; kRing items of C are under way (256x256: what the registers hold; eight spill 24 to 40).
  static constexpr int kItems = 2 * kMI, kRing = BM == 256 ? 4 : 8;
  struct CRing {
    i32x4 v[kRing];
  };
  struct Rows16 {  // one of the matrices, at the wave's first row and column
    __amdgpu_buffer_rsrc_t rs;
    int ld;
  };
  static __device__ __forceinline__ Rows16 rows16(const void* base, int64_t ld, const MxTileInfo& ti, int wm0, int wn0) {
    return Rows16{make_rsrc((const char*)base + ((int64_t)(ti.m0 + wm0) * ld + ti.n0 + wn0) * 2, 0x7FFFFFFF), (int)ld};
  }
  // Byte offset of item i, or past the range where the output has no such row or column.
  static __device__ __forceinline__ uint32_t item_offset(const Rows16& m, const KParams& p, const MxTileInfo& ti, int i,
                                                         int lane, int wm0, int wn0) {
    const int r = i * 8 + (lane >> 3), c = 8 * (lane & 7);
    return ti.m0 + wm0 + r < ti.row_end && ti.n0 + wn0 + c < p.N ? (uint32_t)((r * m.ld + c) * 2) : kOOB;
  }
  static __device__ __forceinline__ void load_c(CRing& ring, const KParams& p, const MxTileInfo& ti, int lane, int wm0, int wn0) {
    const Rows16 c = rows16(p.C, p.ldc, ti, wm0, wn0);
#pragma unroll
    for (int i = 0; i < kRing; ++i)
      ring.v[i] = __builtin_amdgcn_raw_buffer_load_b128(c.rs, item_offset(c, p, ti, i, lane, wm0, wn0), 0, 0);
  }
  template <bool HASC, bool BOTH>
  static __device__ __forceinline__ void epilogue_rows(const KParams& p, const MxTileInfo& ti, const f32x4 (&acc)[kMI][kNI],
                                                       CRing& ring, GEP_LDS char* buf, int lane, int wm0, int wn0) {
    const bool post = p.p_dt != DT_NONE;
    const Rows16 cm = rows16(p.C, p.ldc, ti, wm0, wn0);
    const Rows16 d = BOTH || !post ? rows16(p.D, p.ldd, ti, wm0, wn0) : rows16(p.Post, p.ldp, ti, wm0, wn0);
    const Rows16 q = BOTH ? rows16(p.Post, p.ldp, ti, wm0, wn0) : d;
    const int d_dt = BOTH || !post ? p.d_dt : p.p_dt;
    auto store = [&](const Rows16& m, int dt, int i, const float (&v)[8]) {
      const uint2 lo = pack4_16(dt, v), hi = pack4_16(dt, v + 4);
      __builtin_amdgcn_raw_buffer_store_b128(i32x4{(int)lo.x, (int)lo.y, (int)hi.x, (int)hi.y}, m.rs,
                                             item_offset(m, p, ti, i, lane, wm0, wn0), 0, 0);
    };
#pragma unroll
    for (int pass = 0; pass < kMI; ++pass) {
#pragma unroll
      for (int j = 0; j < kNI; ++j)
        *(f32x4 GEP_LDS*)(buf + ebuf(lane & 15, 2 * j + (lane >> 5), (lane >> 4) & 1)) = acc[pass][j];
      asm volatile("" ::: "memory");
#pragma unroll
      for (int it = 0; it < 2; ++it) {
        const int i = pass * 2 + it, r = it * 8 + (lane >> 3);
        const f32x4 x0 = *(const f32x4 GEP_LDS*)(buf + ebuf(r, lane & 7, 0));
        const f32x4 x1 = *(const f32x4 GEP_LDS*)(buf + ebuf(r, lane & 7, 1));
        float v[8] = {x0[0], x0[1], x0[2], x0[3], x1[0], x1[1], x1[2], x1[3]};
        if constexpr (HASC) {
          const i32x4 x = ring.v[i % kRing];
          float c[8];
          unpack4_16(p.c_dt, uint2{(uint32_t)x[0], (uint32_t)x[1]}, c);
          unpack4_16(p.c_dt, uint2{(uint32_t)x[2], (uint32_t)x[3]}, c + 4);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] += c[e];
          if (i + kRing < kItems)
            ring.v[i % kRing] = __builtin_amdgcn_raw_buffer_load_b128(cm.rs, item_offset(cm, p, ti, i + kRing, lane, wm0, wn0), 0, 0);
        }
        if constexpr (BOTH) store(d, d_dt, i, v);
        if (post) mx_act8(p.act, v);
        if constexpr (BOTH) store(q, p.p_dt, i, v);
        else store(d, d_dt, i, v);
      }
      asm volatile("" ::: "memory");
    }
  }

  // Returns how often kStores16 stores are the last vector memory operations issued.
  static __device__ __forceinline__ int epilogue(const MxParams& mp, int kind, const MxTileInfo& ti, const f32x4 (&acc)[kMI][kNI],
                                                 CRing& ring, GEP_LDS char* buf, int lane, int wm0, int wn0) {
    const KParams& p = mp.k;
    const bool slice = kSplit && mp.split > 1;
    asm volatile("" : "+v"(lane));
    if constexpr (EPI != 2) {
      if (kind == 1) {
        if ((p.d_dt != DT_NONE ? p.d_dt : p.p_dt) == DT_BF16) epilogue16<DT_BF16>(p, ti, acc, buf, lane, wm0, wn0);
        else epilogue16<DT_F16>(p, ti, acc, buf, lane, wm0, wn0);
        return 1;
      }
    }
    if constexpr (EPI == 1) return 0;
    switch (kind) {
      case 3: epilogue_rows<true, false>(p, ti, acc, ring, buf, lane, wm0, wn0); return 1;
      case 4: epilogue_rows<false, true>(p, ti, acc, ring, buf, lane, wm0, wn0); return 2;
      case 5: epilogue_rows<true, true>(p, ti, acc, ring, buf, lane, wm0, wn0); return 2;
      default: break;
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
    return 0;
  }
  static __device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }

  // Item u of this launch -> output tile. The map has tiles of BM x BN; in a split tail's launch
  // (p.tail == 2, the 128x128 kernels) of 256x256, and item u is quarter u & 3 of map tile t_lo + u / 4:
  // its rows (u & 1) and columns (u >> 1 & 1), possibly wholly outside the output.
  static __device__ __forceinline__ MxTileInfo decode(const MxParams& mp, int u, int t_lo, int lane) {
    const KParams& p = mp.k;
    const bool quarter = BM == 128 && p.tail == 2;
    const int MT = quarter ? 2 * BM : BM, NT = quarter ? 2 * BN : BN;
    MxTileInfo ti;
    ti.slice = kSplit && mp.split > 1 ? u / p.T : 0;  // slices of K: all tiles of the first, then the second, ...
    const int t = quarter ? t_lo + (u >> 2) : u - ti.slice * p.T;
    uint32_t mb, nb;
    int row_base = 0;
    if constexpr (VM) {
      const MxGroup g = mx_find_group(p, t, MT, p.tn, lane);
      row_base = g.begin;
      ti.row_end = g.end;
      ti.g = g.index;
      raster(p, (uint32_t)(t - g.first), (uint32_t)((ti.row_end - row_base + MT - 1) / MT), (uint32_t)p.tn, p.fd_Gtn, mb, nb);
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

  // Where this lane's scales come from: row i of the tile's A rows, then of its B rows, a wave 64 of them.
  static __device__ __forceinline__ void scale_source(Src& s, const MxParams& mp, const MxTileInfo& ti, int q0, int wave, int lane) {
    const KParams& p = mp.k;
    s.nsb = mp.nsb - q0;
    const bool is_a = wave < BM / 64;  // (waves past (BM + BN) / 64 move no scales)
    const int first = is_a ? ti.m0 : ti.n0;  // row of the tile's first scale
    const int i = (is_a ? wave : wave - BM / 64) * 64 + lane;  // row of the tile
    const int64_t so = ((int64_t)(first >> 6) * mp.nsb + q0) * 1024;
    s.s = make_rsrc(is_a ? mp.sa + so : mp.sb + (int64_t)ti.g * mp.sb_bytes + so,
                    (is_a ? mp.sa_bytes : mp.sb_bytes) - so);
    const int rr = (first & 63) + i;
    s.s_off = first + i < (is_a ? ti.row_end : p.N) ? (uint32_t)((rr >> 6) * mp.nsb * 1024 + (rr & 63) * 16) : kOOB;
  }

  static __device__ __forceinline__ void run(const MxParams& mp) { run_as<MxRing>(mp); }
  template <class Self>
  static __device__ __forceinline__ void run_as(const MxParams& mp) {
    const KParams& p = mp.k;
    __shared__ __attribute__((aligned(1024))) char smem_raw[kLdsBytes];
    GEP_LDS char* smem = (GEP_LDS char*)smem_raw;
    const int tid = threadIdx.x, lane_id = tid & 63;
    const int wave = uni(tid >> 6);
    // 8 waves: w and w + 4 share a SIMD and take the two row halves of a column block
    const int wm0 = (wave / kWavesN) * kWM, wn0 = (wave % kWavesN) * kWN;

    int T = p.T;
    // (an array that does not run 0 .. M without decreasing gives no tiles)
    if constexpr (VM) T = mx_find_group(p, -1, BM == 128 && p.tail == 2 ? 2 * BM : BM, p.tn, lane_id).first;
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
    typename Self::Src s;
    int steps;
    // The tile's operands, and its first transfers: the first scales and all stages but the last.
    auto begin_tile = [&](int t) {
      int lane = lane_id;
      asm volatile("" : "+v"(lane));  // (lane offsets are not kept across the main loop)
      ti = decode(mp, t, t_lo, lane);
      const int q0 = kSplit ? ti.slice * mp.per : 0;  // the slice's first scale tile, four steps each
      const int ka = q0 * 4 * A::kStepBytes, kb = q0 * 4 * B::kStepBytes;
      steps = kSplit && mp.split > 1 ? min(mp.per * 4, mp.steps - q0 * 4) : mp.steps;
      init<kRowA>(s.la, wave, lane, ti.row_end - ti.m0, (int)p.lda, (int)p.lda - ka);
      init<kRowB>(s.lb, wave, lane, p.N - ti.n0, (int)p.ldb, (int)p.ldb - kb);
      const int64_t ao = (int64_t)ti.m0 * p.lda + ka, bo = (int64_t)ti.n0 * p.ldb + kb;
      s.a = make_rsrc((const char*)p.A + ao, p.a_bytes - ao);
      s.b = make_rsrc((const char*)p.B + (int64_t)ti.g * p.b_bytes + bo, p.b_bytes - bo);
      Self::scale_source(s, mp, ti, q0, wave, lane);
      Self::dma_scales(s, 0, smem, 0, wave);
#pragma unroll
      for (int i = 0; i < NS - 1; ++i) {
        dma<0, kInstrA>(s.la, s.a, i * kRowA, smem + i * kStage, wave);
        dma<0, kInstrB>(s.lb, s.b, i * kRowB, smem + i * kStage + kABytes, wave);
      }
    };

    if (b0 < U) begin_tile(b0);
    int stores = 0;  // how often kStores16 stores are the wave's last operations
    const int kind = EPI == 1 ? 1 : uni(mx_epilogue_kind(mp));
    for (int t = b0; t < U;) {
      f32x4 acc[kMI][kNI];
#pragma unroll
      for (int i = 0; i < kMI; ++i)
#pragma unroll
        for (int j = 0; j < kNI; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
      // a wave whose rows or columns all lie past the output only moves data
      const bool idle = ti.m0 + wm0 >= ti.row_end || ti.n0 + wn0 >= p.N;
      // the first step has landed; the previous tile's epilogue buffers (the last stage) are free
      ring_barrier(stores);
      dma<0, kInstrA / 2>(s.la, s.a, (NS - 1) * kRowA, smem + (NS - 1) * kStage, wave);
      dma<0, kInstrB / 2>(s.lb, s.b, (NS - 1) * kRowB, smem + (NS - 1) * kStage + kABytes, wave);
      int lane = lane_id;
      asm volatile("" : "+v"(lane));
      const typename Self::Lane o = Self::lane_offsets(lane, wm0, wn0);
      typename Self::Frags f;
      if (idle) {
        __builtin_amdgcn_s_setprio(0);
        mainloop<Self, false>(acc, f, smem, o, s, steps, stores, wave);
      } else {
        Self::first_reads(f, smem, o);
        mainloop<Self, true>(acc, f, smem, o, s, steps, stores, wave);
        Self::drain(acc, f);
      }
      dma_barrier();  // transfers past K have landed and every wave has left the ring
      const MxTileInfo done = ti;
      CRing ring;
      if ((kind == 3 || kind == 5) && !idle) load_c(ring, p, done, lane, wm0, wn0);
      t += P;
      if (t < U) begin_tile(t);
      asm volatile("" ::: "memory");  // (its transfers are issued before the epilogue's stores)
      __builtin_amdgcn_sched_barrier(0);
      stores = 0;
      if (!idle) stores = uni(epilogue(mp, kind, done, acc, ring, smem + (NS - 1) * kStage + wave * kRegion, lane_id, wm0, wn0));
    }
  }
};

// ------------------------------------------------------------------------------------
// MxDirect
// ------------------------------------------------------------------------------------
// 16 MB x 16 NB outputs per workgroup of NW waves; wave w takes the scale tiles (512 values of
// K) w, w + NW, ... and reads its fragments straight from global memory, D steps ahead. With one
// row of activations the operand B is read once from HBM in 64-byte runs of 16 rows, and nothing
// waits on a barrier. The waves' partial sums meet in LDS in a fixed order. What depends on how operands are scaled is
// the class's that derives from this one (Self): Scales, Now, scale_source, fetch_scales, take, step.
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

  // The scales of the four steps that are multiplied.
  struct Now {
    int a[MB], b[NB];
  };
  static __device__ __forceinline__ void take(Now& now, const Scales& sc, int kg) {
    const uint32_t sel = (uint32_t)kg | ((uint32_t)(4 + kg) << 8) | 0x0C0C0000u;  // (0x0C: a zero byte)
#pragma unroll
    for (int i = 0; i < MB; ++i) now.a[i] = gather_scale(sc.a[i], sel);
#pragma unroll
    for (int j = 0; j < NB; ++j) now.b[j] = gather_scale(sc.b[j], sel);
  }
  // This lane's scales: row r of each fragment.
  static __device__ __forceinline__ void scale_source(Src& s, const MxParams& mp, int g, int m0, int n0, int row_end, int lane) {
    const int r = lane & 15;
    const int64_t sao = (int64_t)(m0 >> 6) * mp.nsb * 1024, sbo = (int64_t)(n0 >> 6) * mp.nsb * 1024;
    s.sa = make_rsrc(mp.sa + sao, mp.sa_bytes - sao);
    s.sb = make_rsrc(mp.sb + (int64_t)g * mp.sb_bytes + sbo, mp.sb_bytes - sbo);
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const int q = (m0 & 63) + i * 16 + r;
      s.sao[i] = m0 + i * 16 + r < row_end ? (uint32_t)((q >> 6) * mp.nsb * 1024 + (q & 63) * 16) : kOOB;
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int q = (n0 & 63) + j * 16 + r;
      s.sbo[j] = n0 + j * 16 + r < mp.k.N ? (uint32_t)((q >> 6) * mp.nsb * 1024 + (q & 63) * 16) : kOOB;
    }
  }
  template <int T>
  static __device__ __forceinline__ void multiply(f32x4 (&acc)[MB][NB], const Buf& b, const Now& now) {
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = mx_mma<FA, FB, T>(b.b[j], b.a[i], acc[i][j], now.b[j], now.a[i]);
  }

  template <class Self, int T>
  static __device__ __forceinline__ void step(f32x4 (&acc)[MB][NB], Buf (&buf)[D], const Src& s, const typename Self::Now& now,
                                              int tile) {
    Buf& b = buf[T % D];
    Self::template multiply<T>(acc, b, now);
    // the step D further on, in this tile of scales or in the wave's next
    fetch(b, s, T + D < 4 ? tile * 4 + T + D : (tile + NW) * 4 + T + D - 4);
  }

  static __device__ __forceinline__ void run(const MxParams& mp) { run_as<MxDirect>(mp); }
  // The workgroup's tile and scale tiles [t0, t1). False: there is no such tile (the same in every wave).
  struct Place {
    int g, m0, n0, row_end, slice, t0, t1;
  };
  static __device__ __forceinline__ bool place(Place& at, const MxParams& mp, int lane) {
    const KParams& p = mp.k;
    const int slice = VM ? 0 : blockIdx.z, t0 = VM ? 0 : slice * mp.per;
    at = Place{0, (int)blockIdx.y * kBM, (int)blockIdx.x * kBN, p.M, slice, t0, VM ? mp.nsb : min(mp.nsb, t0 + mp.per)};
    if constexpr (VM) {
      const MxGroup found = mx_find_group(p, (int)blockIdx.y, kBM, 1, lane);
      if (found.index < 0) return false;
      at.g = found.index;
      at.m0 = found.begin + ((int)blockIdx.y - found.first) * kBM;
      at.row_end = found.end;
    }
    return true;
  }
  // Adds up the waves' sums in LDS, in order, and finishes the tile.
  static __device__ __forceinline__ void join(const MxParams& mp, const Place& at, const f32x4 (&acc)[MB][NB], float* sums) {
    const KParams& p = mp.k;
    const int tid = threadIdx.x, r = tid & 15, kg = (tid & 63) >> 4, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
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
      if (at.m0 + row < at.row_end && at.n0 + col < p.N) {
        if (!VM && mp.split > 1) mx_slice8(mp, at.slice, at.m0 + row, at.n0 + col, v);
        else mx_finish8(p, at.m0 + row, at.n0 + col, v);
      }
    }
  }

  template <class Self>
  static __device__ __forceinline__ void run_as(const MxParams& mp) {
    const KParams& p = mp.k;
    __shared__ __attribute__((aligned(16))) float sums[NW * kPlane];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Place at;
    if (!place(at, mp, lane)) return;
    const int m0 = at.m0, n0 = at.n0, row_end = at.row_end, t0 = at.t0, t1 = at.t1;
    const int r = lane & 15, kg = lane >> 4;
    Src s;
    const int64_t ao = (int64_t)m0 * p.lda, bo = (int64_t)n0 * p.ldb;
    s.a = make_rsrc((const char*)p.A + ao, p.a_bytes - ao);
    s.b = make_rsrc((const char*)p.B + (int64_t)at.g * p.b_bytes + bo, p.b_bytes - bo);
    Self::scale_source(s, mp, at.g, m0, n0, row_end, lane);
    s.nsb = t1;
    s.ka = min((int)p.lda, t1 * 4 * MxFmt<FA>::kStepBytes) - kg * 16;
    s.kb = min((int)p.ldb, t1 * 4 * MxFmt<FB>::kStepBytes) - kg * 16;
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const int row = i * 16 + r;
      s.ao[i] = m0 + row < row_end ? (uint32_t)(row * (int)p.lda + kg * 16) : kOOB;
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int row = j * 16 + r;
      s.bo[j] = n0 + row < p.N ? (uint32_t)(row * (int)p.ldb + kg * 16) : kOOB;
    }
    f32x4 acc[MB][NB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    if (t0 + wave < t1) {
      typename Self::Scales sc;
      Self::fetch_scales(sc, s, t0 + wave);
      Buf buf[D];
#pragma unroll
      for (int t = 0; t < D; ++t) fetch(buf[t], s, (t0 + wave) * 4 + t);
      for (int tile = t0 + wave; tile < t1; tile += NW) {
        typename Self::Now now;
        Self::take(now, sc, kg);
        Self::fetch_scales(sc, s, tile + NW);
        step<Self, 0>(acc, buf, s, now, tile);
        step<Self, 1>(acc, buf, s, now, tile);
        step<Self, 2>(acc, buf, s, now, tile);
        step<Self, 3>(acc, buf, s, now, tile);
      }
    }
    join(mp, at, acc, sums);
  }
};

// Stages in LDS: as many as fit, at most four (two E2M1 operands: three). WG: workgroups a compute unit.
template <int BM, int FA, int FB, int WG>
constexpr int mx_stages() {
  constexpr bool deep = FA == MX_E2M1 && FB == MX_E2M1;
  const int stage = BM * (MxFmt<FA>::kStepBytes + MxFmt<FB>::kStepBytes) * (deep ? 2 : 1);
  const int n = (163840 / WG - 2 * 2 * BM * 16) / stage, most = deep ? 3 : 4;
  return n > most ? most : n;
}
// 128x128 tiles run two workgroups a compute unit, or with no more workgroups than compute units
// one with all of LDS: 512 x 4096 x 16384 (128 tiles) e4m3 x e4m3 56 us with four stages, 78 with
// two; 8192^3 (many tiles) 15% slower with one workgroup than with two, 475 us.
template <int BM, int NW, int WG, int FA, int FB, bool VM, int EPI>
__global__ __launch_bounds__(NW * 64, WG) void mx_ring_kernel(const MxParams p) {
  MxRing<BM, BM, NW, mx_stages<BM, FA, FB, WG>(), FA, FB, VM, EPI>::run(p);
}
template <int BM, int NW, int WG, int FA, int FB, bool VM>
void mx_launch_ring(const MxParams& p, dim3 grid, hipStream_t s) {
  if constexpr (BM == 256 && (FA == MX_E4M3 || FB == MX_E4M3)) mx_ring_kernel<BM, NW, WG, FA, FB, VM, 0><<<grid, NW * 64, 0, s>>>(p);
  else if (mx_epilogue_kind(p) == 1) mx_ring_kernel<BM, NW, WG, FA, FB, VM, 1><<<grid, NW * 64, 0, s>>>(p);
  else mx_ring_kernel<BM, NW, WG, FA, FB, VM, 2><<<grid, NW * 64, 0, s>>>(p);
}
// Direct kernels: fragments two steps ahead. (Four steps, or twice the waves, are slower everywhere:
// 1 x 8192 x 8192 e4m3 x e2m1 in 16x32 tiles 8.0 us, four steps or 16 waves 10% more; in 16x16 tiles 9.0 on
// four waves, on eight 8% more, on 16 29%.)
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
      case MX_TILE_256: mx_launch_ring<256, 8, 1, FA, FB, VM>(p, grid, s); break;                    \
      case MX_TILE_128:                                                                              \
        if (p.k.P <= p.cus) mx_launch_ring<128, 4, 1, FA, FB, VM>(p, grid, s);                       \
        else mx_launch_ring<128, 4, 2, FA, FB, VM>(p, grid, s);                                      \
        break;                                                                                       \
      case MX_TILE_32X64: mx_direct_kernel<2, 4, 4, 2, FA, FB, VM><<<grid, 256, 0, s>>>(p); break;   \
      case MX_TILE_32: mx_direct_kernel<2, 2, 4, 2, FA, FB, VM><<<grid, 256, 0, s>>>(p); break;      \
      case MX_TILE_16X32: mx_direct_kernel<1, 2, 8, 2, FA, FB, VM><<<grid, 512, 0, s>>>(p); break;   \
      case MX_TILE_16: mx_direct_kernel<1, 1, 4, 2, FA, FB, VM><<<grid, 256, 0, s>>>(p); break;      \
      default: return hipErrorInvalidValue;                                                          \
    }                                                                                                \
    return hipGetLastError();                                                                        \
  }

}  // namespace gep
