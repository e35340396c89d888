// Host side of the MX product's C ABI: validation of a description and the choice of the
// kernel. No HIP call is made here.
#include "mx_plan.hpp"

#include <initializer_list>
#include <new>

namespace gep {

gemm_status fail(gemm_status st, const char* fmt, ...);
void clear_error();

namespace {
int out_bytes(int32_t dt) {
  switch (dt) {
    case GEMM_DT_F16:
    case GEMM_DT_BF16: return 2;
    case GEMM_DT_F32: return 4;
    default: return 0;
  }
}
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

gemm_status check_out(const char* name, int32_t dt, int64_t ld, int32_t M, int32_t N) {
  if (dt == GEMM_DT_NONE) return GEMM_OK;
  const int es = out_bytes(dt);
  if (!es) return fail(GEMM_ERR_UNSUPPORTED, "mx_gemm_create: %s must be F16, BF16 or F32", name);
  if (ld < 0) return fail(GEMM_ERR_INVALID_ARG, "mx_gemm_create: negative leading dimension of %s", name);
  if (ld > ((int64_t)1 << 48)) return fail(GEMM_ERR_UNSUPPORTED, "mx_gemm_create: leading dimension of %s beyond 2^48", name);
  if (M > 1 && ld < N) return fail(GEMM_ERR_INVALID_ARG, "mx_gemm_create: leading dimension of %s below N", name);
  if (ld * es % 16) return fail(GEMM_ERR_ALIGNMENT, "mx_gemm_create: leading dimension of %s is not a multiple of 16 bytes", name);
  return GEMM_OK;
}
}  // namespace

void mx_tile_extent(int32_t tile, int32_t* bm, int32_t* bn) {
  switch (tile) {
    case MX_TILE_256: *bm = *bn = 256; break;
    case MX_TILE_128: *bm = *bn = 128; break;
    case MX_TILE_32X64: *bm = 32; *bn = 64; break;
    case MX_TILE_32: *bm = *bn = 32; break;
    case MX_TILE_16X32: *bm = 16; *bn = 32; break;
    default: *bm = *bn = 16; break;
  }
}

int64_t mx_row_blocks(const mx_gemm_plan& p, int32_t bm) {
  const int64_t m = p.d.M;
  if (!p.d.groups) return cdiv(m, bm);
  // every group adds at most one partial block, and a group without rows none
  return m / bm + (m < p.d.groups ? m : p.d.groups);
}

MxChoice mx_choose(const mx_gemm_plan& p, int32_t cus, bool workspace) {
  MxChoice c{p.d.tile, 1, 0};
  const int32_t nsb = (int32_t)cdiv(p.d.K, 512);
  const int64_t rows = p.d.groups ? cdiv(p.d.M, p.d.groups) : p.d.M;
  if (c.tile == MX_TILE_AUTO) {
    if (rows <= 16) c.tile = MX_TILE_16;
    else if (rows <= 32) c.tile = MX_TILE_16X32;
    else if (rows <= 64) c.tile = MX_TILE_32;
    else if (mx_row_blocks(p, 256) * cdiv(p.d.N, 256) >= cus) c.tile = MX_TILE_256;
    else if (mx_row_blocks(p, 128) * cdiv(p.d.N, 128) >= cus / 2) c.tile = MX_TILE_128;
    else c.tile = MX_TILE_32X64;
  }
  if (!p.d.groups && workspace && c.tile != MX_TILE_256 && p.d.split > 1) c.split = p.d.split;
  if (c.split > nsb) c.split = nsb > 1 ? nsb : 1;
  c.per = nsb > 0 ? (int32_t)cdiv(nsb, c.split) : 1;
  c.split = nsb > 0 ? (int32_t)cdiv(nsb, c.per) : 1;
  return c;
}

int64_t mx_workspace_bytes(const mx_gemm_plan& p, const MxChoice& c) {
  return c.split > 1 ? (int64_t)c.split * p.d.M * p.d.N * 4 : 0;
}

}  // namespace gep

using namespace gep;

extern "C" {

int64_t mx_code_bytes(int64_t rows, int64_t k, int32_t format) {
  if (rows < 0 || k < 0 || (format != MX_E2M1 && format != MX_E4M3)) return -1;
  return rows * ((k + MX_BLOCK - 1) / MX_BLOCK) * (format == MX_E2M1 ? 16 : 32);
}

int64_t mx_scale_bytes(int64_t rows, int64_t k) {
  if (rows < 0 || k < 0) return -1;
  const int64_t nb = (k + MX_BLOCK - 1) / MX_BLOCK;
  return cdiv(rows, 64) * cdiv(nb, 16) * 64 * 16;
}

gemm_status mx_gemm_create(const mx_gemm_desc* d, mx_gemm_plan** out) {
  if (!out) return fail(GEMM_ERR_INVALID_ARG, "mx_gemm_create: NULL out");
  *out = nullptr;
  if (!d) return fail(GEMM_ERR_INVALID_ARG, "mx_gemm_create: NULL desc");
  if (d->M < 0 || d->N < 0 || d->K < 0) return fail(GEMM_ERR_INVALID_ARG, "mx_gemm_create: negative size");
  if (d->groups < 0) return fail(GEMM_ERR_INVALID_ARG, "mx_gemm_create: negative group count");
  if (d->groups > kMaxVarlenGroups) return fail(GEMM_ERR_UNSUPPORTED, "mx_gemm_create: more than %d groups", kMaxVarlenGroups);
  for (int32_t f : {d->a_format, d->b_format})
    if (f != MX_E2M1 && f != MX_E4M3) return fail(GEMM_ERR_INVALID_ARG, "mx_gemm_create: unknown format %d", f);
  for (int32_t t : {d->c, d->d, d->post})
    if (t < GEMM_DT_NONE || t > GEMM_DT_E5M2) return fail(GEMM_ERR_INVALID_ARG, "mx_gemm_create: unknown type %d", t);
  if (d->d == GEMM_DT_NONE && d->post == GEMM_DT_NONE) return fail(GEMM_ERR_INVALID_ARG, "mx_gemm_create: neither D nor PostAct");
  if (d->act < GEMM_ACT_NONE || d->act > GEMM_ACT_SILU) return fail(GEMM_ERR_INVALID_ARG, "mx_gemm_create: unknown activation %d", d->act);
  if (d->act != GEMM_ACT_NONE && d->post == GEMM_DT_NONE) return fail(GEMM_ERR_INVALID_ARG, "mx_gemm_create: an activation without PostAct");
  if (d->tile < MX_TILE_AUTO || d->tile > MX_TILE_16) return fail(GEMM_ERR_INVALID_ARG, "mx_gemm_create: unknown tile %d", d->tile);
  if (d->split < 0 || d->split > 64) return fail(GEMM_ERR_INVALID_ARG, "mx_gemm_create: split must lie in [0, 64]");
  if (d->split > 1 && (d->groups || d->tile == MX_TILE_256))
    return fail(GEMM_ERR_UNSUPPORTED, "mx_gemm_create: a grouped plan and MX_TILE_256 do not split K");
  if (d->N % 8) return fail(GEMM_ERR_ALIGNMENT, "mx_gemm_create: N = %d is not a multiple of 8", d->N);
  // (256 rows of codes stay below 2^31 bytes: the kernels' offsets inside a tile are 32-bit)
  if (d->K > (1 << 22)) return fail(GEMM_ERR_UNSUPPORTED, "mx_gemm_create: K above 2^22");
  gemm_status st = check_out("C", d->c, d->ldc, d->M, d->N);
  if (st == GEMM_OK) st = check_out("D", d->d, d->ldd, d->M, d->N);
  if (st == GEMM_OK) st = check_out("PostAct", d->post, d->ldp, d->M, d->N);
  if (st != GEMM_OK) return st;
  mx_gemm_plan* p = new (std::nothrow) mx_gemm_plan;
  if (!p) return fail(GEMM_ERR_NO_MEMORY, "mx_gemm_create: out of memory");
  p->d = *d;
  p->lda = (int32_t)mx_code_bytes(1, d->K, d->a_format);
  p->ldb = (int32_t)mx_code_bytes(1, d->K, d->b_format);
  p->a_bytes = mx_code_bytes(d->M, d->K, d->a_format);
  p->b_bytes = mx_code_bytes(d->N, d->K, d->b_format);
  p->sa_bytes = mx_scale_bytes(d->M, d->K);
  p->sb_bytes = mx_scale_bytes(d->N, d->K);
  int32_t bm, bn;
  mx_tile_extent(MX_TILE_128, &bm, &bn);
  if (mx_row_blocks(*p, bm) * cdiv(d->N, bn) > 0xFFFFFF) {
    delete p;
    return fail(GEMM_ERR_UNSUPPORTED, "mx_gemm_create: too many output tiles");
  }
  clear_error();
  *out = p;
  return GEMM_OK;
}

gemm_status mx_gemm_destroy(mx_gemm_plan* plan) {
  delete plan;
  clear_error();
  return GEMM_OK;
}

gemm_status mx_gemm_plan_tile(const mx_gemm_plan* plan, int32_t num_cus, int32_t* tile, int32_t* split) {
  if (!plan || num_cus < 1) return fail(GEMM_ERR_INVALID_ARG, "mx_gemm_plan_tile: NULL plan or no compute units");
  const MxChoice c = mx_choose(*plan, num_cus, true);
  if (tile) *tile = c.tile;
  if (split) *split = c.split;
  clear_error();
  return GEMM_OK;
}

gemm_status mx_gemm_workspace(const mx_gemm_plan* plan, int32_t num_cus, int64_t* bytes) {
  if (!plan || !bytes || num_cus < 1) return fail(GEMM_ERR_INVALID_ARG, "mx_gemm_workspace: NULL argument or no compute units");
  *bytes = mx_workspace_bytes(*plan, mx_choose(*plan, num_cus, true));
  clear_error();
  return GEMM_OK;
}

}  // extern "C"
