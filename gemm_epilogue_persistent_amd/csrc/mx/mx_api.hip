// mx_gemm_run and fp8_gemm_run (C ABI): the launch of a product of block-scaled operands.
#include <atomic>
#include <utility>

#include "../fp8/fp8_gemm.hpp"
#include "mx_gemm.hpp"
#include "mx_plan.hpp"

namespace gep {
gemm_status fail(gemm_status st, const char* fmt, ...);
void clear_error();

#define GEP_MX_DECLARE(FA, FB)                                                              \
  template <> hipError_t mx_launch<FA, FB, false>(int32_t, const MxParams&, dim3, hipStream_t); \
  template <> hipError_t mx_launch<FA, FB, true>(int32_t, const MxParams&, dim3, hipStream_t);
GEP_MX_DECLARE(MX_E2M1, MX_E2M1)
GEP_MX_DECLARE(MX_E2M1, MX_E4M3)
GEP_MX_DECLARE(MX_E4M3, MX_E2M1)
GEP_MX_DECLARE(MX_E4M3, MX_E4M3)

template <> hipError_t fp8_launch<false, false>(int32_t, const MxParams&, dim3, hipStream_t);
template <> hipError_t fp8_launch<false, true>(int32_t, const MxParams&, dim3, hipStream_t);
template <> hipError_t fp8_launch<true, false>(int32_t, const MxParams&, dim3, hipStream_t);
template <> hipError_t fp8_launch<true, true>(int32_t, const MxParams&, dim3, hipStream_t);

template <bool VM>
static hipError_t launch(const mx_gemm_plan& plan, int32_t tile, const MxParams& p, dim3 g, hipStream_t s) {
  const mx_gemm_desc& d = plan.d;
  if (plan.b_scaling == FP8_ROWS) return fp8_launch<true, VM>(tile, p, g, s);
  if (plan.b_scaling == FP8_TILES) return fp8_launch<false, VM>(tile, p, g, s);
  if (d.a_format == MX_E2M1)
    return d.b_format == MX_E2M1 ? mx_launch<MX_E2M1, MX_E2M1, VM>(tile, p, g, s) : mx_launch<MX_E2M1, MX_E4M3, VM>(tile, p, g, s);
  return d.b_format == MX_E2M1 ? mx_launch<MX_E4M3, MX_E2M1, VM>(tile, p, g, s) : mx_launch<MX_E4M3, MX_E4M3, VM>(tile, p, g, s);
}

constexpr int32_t kRasterG = 8;

// Adds up the slices of K, in order, and finishes 8 columns a thread.
__global__ __launch_bounds__(256) void mx_join_kernel(const MxParams p, uint32_t n, FastDiv fd_cols8) {
  const uint32_t i = blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  uint32_t m, c;
  fd_divmod(fd_cols8, i, m, c);
  const float* q = p.sums + (int64_t)m * p.k.N + c * 8;
  const int64_t plane = (int64_t)p.k.M * p.k.N;
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = 0.f;
#pragma unroll 4
  for (int s = 0; s < p.split; ++s) {
    const f32x4 a = *(const f32x4*)(q + s * plane), b = *(const f32x4*)(q + s * plane + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += a[e], v[4 + e] += b[e];
  }
  mx_finish8(p.k, m, (int)c * 8, v);
}

// Compute units of the current device, looked up once per device.
gemm_status compute_units(int32_t* cus) {
  static std::atomic<int32_t> cache[64];
  int dev = 0, n = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return fail(GEMM_ERR_HIP, "hipGetDevice: %s", hipGetErrorString(e));
  const bool cached = dev >= 0 && dev < 64;
  if (cached && (n = cache[dev].load(std::memory_order_relaxed)) > 0) {
    *cus = n;
    return GEMM_OK;
  }
  e = hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev);
  if (e != hipSuccess || n <= 0) return fail(GEMM_ERR_HIP, "hipDeviceGetAttribute: %s", hipGetErrorString(e));
  if (cached) cache[dev].store(n, std::memory_order_relaxed);
  *cus = n;
  return GEMM_OK;
}

gemm_status block_gemm_run(const char* fn, const mx_gemm_plan* plan, const mx_gemm_args* a, void* stream) {
  if (!plan || !a) return fail(GEMM_ERR_INVALID_ARG, "%s: NULL plan or args", fn);
  const mx_gemm_desc& d = plan->d;
  if (d.M == 0 || d.N == 0) { clear_error(); return GEMM_OK; }
  if (d.K > 0 && (!a->a_codes || !a->a_scales || ((!a->b_codes || !a->b_scales))))
    return fail(GEMM_ERR_INVALID_ARG, "%s: A and B are required", fn);
  if ((d.c != GEMM_DT_NONE) != (a->C != nullptr)) return fail(GEMM_ERR_INVALID_ARG, "%s: C must be given iff the plan has a C type", fn);
  if ((d.d != GEMM_DT_NONE) != (a->D != nullptr)) return fail(GEMM_ERR_INVALID_ARG, "%s: D must be given iff the plan has a D type", fn);
  if ((d.post != GEMM_DT_NONE) != (a->PostAct != nullptr)) return fail(GEMM_ERR_INVALID_ARG, "%s: PostAct must be given iff the plan has a PostAct type", fn);
  if ((d.groups > 0) != (a->cu_seqlens_m != nullptr)) return fail(GEMM_ERR_INVALID_ARG, "%s: cu_seqlens_m must be given iff the plan is grouped", fn);
  for (const void* p : {a->a_codes, a->a_scales, a->b_codes, a->b_scales, a->C, (const void*)a->D, (const void*)a->PostAct})
    if ((uintptr_t)p & 15) return fail(GEMM_ERR_ALIGNMENT, "%s: pointers must be 16-byte aligned", fn);
  if ((uintptr_t)a->cu_seqlens_m & 3) return fail(GEMM_ERR_ALIGNMENT, "%s: cu_seqlens_m not 4-byte aligned", fn);
  for (const auto& o : {std::pair<const void*, std::pair<int32_t, int64_t>>{a->D, {d.d, d.ldd}}, {a->PostAct, {d.post, d.ldp}}})
    if (a->C && a->C == o.first && (d.c != o.second.first || (d.M > 1 && d.ldc != o.second.second)))
      return fail(GEMM_ERR_INVALID_ARG, "%s: C in the place of an output needs its type and leading dimension", fn);
  if (a->D && a->D == a->PostAct) return fail(GEMM_ERR_INVALID_ARG, "%s: D and PostAct are one matrix", fn);
  int32_t cus = 0;
  const gemm_status st = compute_units(&cus);
  if (st != GEMM_OK) return st;

  MxChoice choice = mx_choice(*plan, cus, true);
  if (choice.split > 1) {
    const int64_t need = mx_workspace_bytes(*plan, choice);
    if (!a->workspace) choice = mx_choice(*plan, cus, false);
    else if (a->workspace_bytes < need) return fail(GEMM_ERR_INVALID_ARG, "%s: workspace of %lld bytes expected", fn, (long long)need);
    else if ((uintptr_t)a->workspace & 15) return fail(GEMM_ERR_ALIGNMENT, "%s: workspace not 16-byte aligned", fn);
  }
  const int32_t tile = choice.tile;
  int32_t bm, bn;
  mx_tile_extent(*plan, tile, &bm, &bn);
  MxParams p{};
  KParams& k = p.k;
  k.A = a->a_codes; k.B = a->b_codes; k.C = a->C; k.D = a->D; k.Post = a->PostAct;
  k.lda = plan->lda; k.ldb = plan->ldb; k.ldc = d.ldc; k.ldd = d.ldd; k.ldp = d.ldp;
  k.a_bytes = plan->a_bytes; k.b_bytes = plan->b_bytes;
  k.M = d.M; k.N = d.N; k.K = d.K; k.L = d.groups;
  k.cu_seqlens = a->cu_seqlens_m;
  k.c_dt = d.c; k.d_dt = d.d; k.p_dt = d.post; k.act = d.act;
  p.sa = (const uint8_t*)a->a_scales; p.sb = (const uint8_t*)a->b_scales;
  p.sa_bytes = plan->sa_bytes; p.sb_bytes = plan->sb_bytes;
  p.nsb = (d.K + 511) / 512;
  p.steps = (d.K + 127) / 128;
  p.cus = cus;
  p.split = choice.split;
  p.per = choice.per;
  p.sums = (float*)a->workspace;
  if (p.split > 1 && (int64_t)d.M * (d.N / 8) > 0x7FFFFF00) return fail(GEMM_ERR_UNSUPPORTED, "%s: too many outputs to share out K", fn);
  const int64_t tm = mx_row_blocks(*plan, bm), tn = (d.N + bn - 1) / bn;
  dim3 grid;
  int32_t tail_grid = 0;  // workgroups of the split tail's launch
  if (tile == MX_TILE_256 || tile == MX_TILE_128) {
    k.tm = (int32_t)tm;
    k.tn = (int32_t)tn;
    k.T = (int32_t)(tm * tn);  // (grouped: the kernel counts its tiles itself)
    const int32_t cap = tile == MX_TILE_128 ? 2 * cus : cus;
    k.P = k.T * p.split < cap ? k.T * p.split : cap;
    k.log2G = 3;
    k.xcd_remap = 1;
    k.fd_Gtn = make_fastdiv((uint32_t)(kRasterG * tn));
    for (int w = 1; w < kRasterG; ++w) k.fd_tail[w] = make_fastdiv((uint32_t)w);
    grid = dim3((unsigned)k.P);
    if (tile == MX_TILE_256 && k.T > k.P) {
      // (a grouped plan's tile count is known on the device only; its second launch exits at
      // once when there is no such tail)
      const int32_t rem = k.T % k.P;
      if (d.groups) tail_grid = 2 * cus;
      else if (rem > 0 && 2 * rem <= k.P) tail_grid = 4 * rem < 2 * cus ? 4 * rem : 2 * cus;
      if (tail_grid > 0) {
        k.tail = 1;
        k.P_big = k.P;
      }
    }
  } else {
    if (!mx_direct_fits(*plan, tile)) return fail(GEMM_ERR_UNSUPPORTED, "%s: too many rows or columns for the tile asked for", fn);
    grid = dim3((unsigned)tn, (unsigned)tm, (unsigned)p.split);
  }
  hipStream_t s = (hipStream_t)stream;
  auto run = [&](int32_t t, dim3 g) { return d.groups ? launch<true>(*plan, t, p, g, s) : launch<false>(*plan, t, p, g, s); };
  hipError_t e = run(tile, grid);
  if (e == hipSuccess && tail_grid > 0) {
    k.tail = 2;
    k.P = tail_grid;
    e = run(MX_TILE_128, dim3((unsigned)tail_grid));
  }
  if (e == hipSuccess && p.split > 1) {
    const uint32_t n = (uint32_t)((int64_t)d.M * (d.N / 8));
    mx_join_kernel<<<(n + 255) / 256, 256, 0, s>>>(p, n, make_fastdiv((uint32_t)d.N / 8));
    e = hipGetLastError();
  }
  if (e != hipSuccess) return fail(GEMM_ERR_HIP, "%s launch: %s", fn, hipGetErrorString(e));
  clear_error();
  return GEMM_OK;
}

}  // namespace gep

using namespace gep;

extern "C" gemm_status mx_gemm_run(const mx_gemm_plan* plan, const mx_gemm_args* a, void* stream) {
  return block_gemm_run("mx_gemm_run", plan, a, stream);
}

extern "C" gemm_status fp8_gemm_run(const fp8_gemm_plan* plan, const fp8_gemm_args* a, void* stream) {
  if (!a) return fail(GEMM_ERR_INVALID_ARG, "fp8_gemm_run: NULL plan or args");
  const mx_gemm_args m{a->a_codes, a->a_scales, a->b_codes, a->b_scales, a->C, a->D, a->PostAct, a->cu_seqlens_m, a->workspace, a->workspace_bytes};
  return block_gemm_run("fp8_gemm_run", plan, &m, stream);
}
