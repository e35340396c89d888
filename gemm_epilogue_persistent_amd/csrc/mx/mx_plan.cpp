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
int64_t blocks_of(int64_t a, int64_t b) { return a / b + (a % b != 0); }  // (cdiv of any size)

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

// Which kernel: the one with the least estimated time, over the tiles and, for a dense plan with a
// workspace, over 1 to 16 workgroups a tile's K. The estimates (microseconds) are fits to
// measurements of all of them at 30 shapes from 1x1024x1024 to 8192x512x4096 in the three usual
// pairs of formats:
//   direct kernels: 2.7 to 3.4 us, and a step of 128 along K moves the tile's rows of both operands at 33
//     KB a microsecond and compute unit, whether one workgroup runs there or several, each for 1.6
//     us at least (32x64: 2.2) (128x4096x4096 e4m3 x e2m1 in 32x64 tiles 10.7 measured, 11.2 estimated)
//   128x128: 7 us, and 74 KB a microsecond alone on a compute unit, 56 for two workgroups
//     (512x4096x4096 18.3, 17.4; 16384x4096x4096 230, 234)
//   256x256: 6 us, a round 5 us and 1.36 a step with an e4m3 operand, 0.85 without (4096^3 53.2, 54.5;
//     16384x4096x4096 196, 200), the quarters of a last round 4 us and 1.3 times their share of one
//   a split adds 3 us and the sums' way to memory and back at 4.2 MB a microsecond
//     (1024x1024x8192 in 128x128 tiles over four workgroups 22.3, 23.2; over one 29.4)
// so 16-row tiles serve few rows (1x8192x8192 8.0; in 32x64 tiles 13.8), 32x64 up to 128 or 256 rows,
// 128x128 up to one round of 256x256 tiles, and deep products with few tiles are split
// (128x512x8192: 8.3 in 32x32 tiles over four workgroups, 13.8 over one).
static double estimate(const mx_gemm_plan& p, int32_t cus, int32_t tile, int32_t split) {
  int32_t bm, bn;
  mx_tile_extent(tile, &bm, &bn);
  // (grouped: half a partial row block for each group)
  const double blocks = p.d.groups ? (double)p.d.M / bm + 0.5 * (p.d.M < p.d.groups ? p.d.M : p.d.groups) : (double)mx_row_blocks(p, bm);
  const double wgs = blocks * (double)cdiv(p.d.N, bn) * split;
  const int64_t nsb = cdiv(p.d.K, 512);
  const double steps = split > 1 ? 4.0 * (double)cdiv(nsb, split) : (double)cdiv(p.d.K, 128);
  const double rows_a = p.d.M < bm ? p.d.M : bm, rows_b = p.d.N < bn ? p.d.N : bn;
  const double kb = (rows_a * (p.d.a_format == MX_E4M3 ? 128 : 64) + rows_b * (p.d.b_format == MX_E4M3 ? 128 : 64)) / 1024;
  double t;
  if (tile == MX_TILE_256) {
    // (a last round of at most half the card runs in 128x128 quarters)
    const double step = p.d.a_format == MX_E2M1 && p.d.b_format == MX_E2M1 ? 0.85 : 1.36;
    const double full = (double)((int64_t)wgs / cus), rest = wgs / cus - full;
    const bool quarters = full > 0 && rest > 0 && rest <= 0.5;
    t = 6 + (full + (quarters ? rest * 1.3 : rest > 0)) * (steps * step + 5) + (quarters ? 4 : 0);
  } else if (tile == MX_TILE_128) {
    t = 7 + (wgs <= cus ? steps * kb / 74 : (double)cdiv((int64_t)wgs, 2 * (int64_t)cus) * (steps * 2 * kb / 56 + 1) - 1);
  } else {
    const double load = wgs / cus, one = steps * kb / 33;
    const double start = tile == MX_TILE_16 ? 2.7 : tile == MX_TILE_16X32 ? 2.8 : tile == MX_TILE_32 ? 3.0 : 3.4;
    const double least = tile == MX_TILE_32X64 ? 2.2 : 1.6;
    t = start + (one > least ? one : least) * (load > 1 ? load : 1);
  }
  if (split > 1) t += 3 + (double)split * p.d.M * p.d.N * 8 / 4.2e6;
  return t;
}

MxChoice mx_choose(const mx_gemm_plan& p, int32_t cus, bool workspace) {
  const int32_t nsb = (int32_t)cdiv(p.d.K, 512);
  const bool may_split = !p.d.groups && workspace;
  int32_t best_tile = p.d.tile, best_split = 1;
  double best = 1e300;
  for (int32_t tile = MX_TILE_256; tile <= MX_TILE_16; ++tile) {
    if (p.d.tile != MX_TILE_AUTO && p.d.tile != tile) continue;
    int32_t bm, bn;
    mx_tile_extent(tile, &bm, &bn);
    if (p.d.tile == MX_TILE_AUTO && !mx_direct_fits(p, tile)) continue;
    for (int32_t split = 1; split <= 64; ++split) {
      const bool wanted = p.d.split > 0 ? split == p.d.split : (split & (split - 1)) == 0 && split <= 16;
      if (!wanted && split > 1) continue;
      if (split > 1 && (!may_split || tile == MX_TILE_256 || split > nsb)) continue;
      if (p.d.split == 1 && split > 1) continue;
      const double t = estimate(p, cus, tile, split) - (p.d.split > 1 && split == p.d.split ? 1e9 : 0);
      if (t < best) {
        best = t;
        best_tile = tile;
        best_split = split;
      }
    }
  }
  MxChoice c{best_tile, p.d.split > 1 && may_split && best_tile != MX_TILE_256 ? p.d.split : best_split, 0};
  if (c.split > nsb) c.split = nsb > 1 ? nsb : 1;
  c.per = nsb > 0 ? (int32_t)cdiv(nsb, c.split) : 1;
  c.split = nsb > 0 ? (int32_t)cdiv(nsb, c.per) : 1;
  return c;
}

MxChoice mx_choice(const mx_gemm_plan& p, int32_t cus, bool workspace) {
  if (cus > 0xFFFF) return mx_choose(p, cus, workspace);
  std::atomic<uint64_t>& slot = p.chosen[workspace];
  const uint64_t v = slot.load(std::memory_order_relaxed);
  if (v >> 48 == (uint64_t)cus) return MxChoice{(int32_t)(v >> 40 & 0xFF), (int32_t)(v >> 32 & 0xFF), (int32_t)(uint32_t)v};
  const MxChoice c = mx_choose(p, cus, workspace);
  slot.store((uint64_t)cus << 48 | (uint64_t)c.tile << 40 | (uint64_t)c.split << 32 | (uint32_t)c.per, std::memory_order_relaxed);
  return c;
}

bool mx_direct_fits(const mx_gemm_plan& p, int32_t tile) {
  if (tile == MX_TILE_256 || tile == MX_TILE_128) return true;
  int32_t bm, bn;
  mx_tile_extent(tile, &bm, &bn);
  return mx_row_blocks(p, bm) <= 65535 && cdiv(p.d.N, bn) < (1 << 23);
}

int64_t mx_workspace_bytes(const mx_gemm_plan& p, const MxChoice& c) {
  return c.split > 1 ? (int64_t)c.split * p.d.M * p.d.N * 4 : 0;
}

}  // namespace gep

using namespace gep;

extern "C" {

int64_t mx_code_bytes(int64_t rows, int64_t k, int32_t format) {
  if (rows < 0 || k < 0 || (format != MX_E2M1 && format != MX_E4M3)) return -1;
  if (rows == 0) return 0;
  int64_t row, all;
  if (__builtin_mul_overflow(blocks_of(k, MX_BLOCK), (int64_t)(format == MX_E2M1 ? 16 : 32), &row) ||
      __builtin_mul_overflow(rows, row, &all))
    return -1;
  return all;
}

int64_t mx_scale_bytes(int64_t rows, int64_t k) {
  if (rows < 0 || k < 0) return -1;
  int64_t tiles, all;
  if (__builtin_mul_overflow(blocks_of(rows, 64), blocks_of(blocks_of(k, MX_BLOCK), 16), &tiles) ||
      __builtin_mul_overflow(tiles, (int64_t)(64 * 16), &all))
    return -1;
  return all;
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
  const MxChoice c = mx_choice(*plan, num_cus, true);
  if (tile) *tile = c.tile;
  if (split) *split = c.split;
  clear_error();
  return GEMM_OK;
}

gemm_status mx_gemm_workspace(const mx_gemm_plan* plan, int32_t num_cus, int64_t* bytes) {
  if (!plan || !bytes || num_cus < 1) return fail(GEMM_ERR_INVALID_ARG, "mx_gemm_workspace: NULL argument or no compute units");
  *bytes = mx_workspace_bytes(*plan, mx_choice(*plan, num_cus, true));
  clear_error();
  return GEMM_OK;
}

}  // extern "C"
