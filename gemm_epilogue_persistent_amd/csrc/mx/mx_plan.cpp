// Host side of the C ABI of the MX and FP8 products: validation of a description and the choice of the
// kernel. No HIP call is made here.
#include "mx_plan.hpp"

#include <cmath>
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

gemm_status check_out(const char* fn, const char* name, int32_t dt, int64_t ld, int32_t M, int32_t N) {
  if (dt == GEMM_DT_NONE) return GEMM_OK;
  const int es = out_bytes(dt);
  if (!es) return fail(GEMM_ERR_UNSUPPORTED, "%s: %s must be F16, BF16 or F32", fn, name);
  if (ld < 0) return fail(GEMM_ERR_INVALID_ARG, "%s: negative leading dimension of %s", fn, name);
  if (ld > ((int64_t)1 << 48)) return fail(GEMM_ERR_UNSUPPORTED, "%s: leading dimension of %s beyond 2^48", fn, name);
  if (M > 1 && ld < N) return fail(GEMM_ERR_INVALID_ARG, "%s: leading dimension of %s below N", fn, name);
  if (ld * es % 16) return fail(GEMM_ERR_ALIGNMENT, "%s: leading dimension of %s is not a multiple of 16 bytes", fn, name);
  return GEMM_OK;
}
}  // namespace

void mx_tile_extent(const mx_gemm_plan& p, int32_t tile, int32_t* bm, int32_t* bn) {
  switch (tile) {
    case MX_TILE_256: *bm = *bn = 256; break;
    case MX_TILE_128: *bm = *bn = 128; break;
    case MX_TILE_32X64: *bm = p.b_scaling >= 0 ? 64 : 32; *bn = 64; break;
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
  mx_tile_extent(p, tile, &bm, &bn);
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

// The same of FP8 products, whose kernels have more vector arithmetic (256x256, 128x128, 32x32 and less) or are their own
// (64x64). Dense: fits to 108 shapes each with B's scales by tiles and (in brackets) by rows from 1x1024x1024 to 4096x8192x8192;
// the choice is 1% slower than the best kernel in the mean, 18% at most.
//   256x256: 6 us, a round 5 us and 1.66 (2.07) a step (4096^3 63.5 measured, 64.1 estimated; 2048x8192x8192 115.9, 117)
//   128x128: 7 us, and 55 (43) KB a microsecond alone on a compute unit, 65 (55) for two workgroups (256x4096x4096 over
//     one 25.8, 25.6, over four 21.8, 22.7; 2048x4096x4096 38.3, 38.5), and B at 7 MB a microsecond at most
//     (64x8192x8192 over four 23.1, 23.6)
//   64x64: 2.8 (2.3) us, a round 1.8 (2.6) and 0.55 (0.72) a quad of steps, up to 0.35 (0.22) more with the card
//     full; B at 6 (5.6) MB a microsecond at most (256x4096x4096 11.6, 11.7; 64x8192x8192 17.0, 16.5; 512x4096x4096 21.0,
//     20.6). Direct 32x64 tiles, which MX products have in their place, were nowhere the fastest (256x4096x4096 25.6, 128 rows
//     14.8 and 10.5, 64x8192x8192 25.5 and 17.0)
//   16x16, 16x32, 32x32: 2.7 to 3 us, B's bytes, from memory, at 25, 19.5 and 18.5 KB a microsecond, A's, from a cache,
//     at 50, 100 and 95 (16x16 and 16x32: 1x8192x8192 13.3, 13.3 and 16.1, 16.0; 16x8192x8192 18.1, 18.1 and 16.4, 17.2)
// Grouped: the groups that have rows are those of a choice at random, with as many each, and their B come from HBM; fits to 60
// shapes of 8 to 8192 rows over 8 and 64 groups (2% slower than the best in the mean, 21% at most). A workgroup looks its
// group up first, 1.8 us a round in 64x64 tiles and as much before the first of a direct kernel; B at 4.5 MB a microsecond
// in 128x128 and 64x64 tiles, 6.1 in direct ones, 3.6 in 256x256 (512 rows over 64 experts of 4096x4096: 246, 230, 207 in
// 32x32, 269; 8192 rows 305, 471, 1067, 295).
static double estimate_fp8(const mx_gemm_plan& p, int32_t cus, int32_t tile, int32_t split) {
  int32_t bm, bn;
  mx_tile_extent(p, tile, &bm, &bn);
  const bool grouped = p.d.groups > 0, rows = p.b_scaling == FP8_ROWS;
  const double groups = grouped ? p.d.groups * (1 - std::exp(-(double)p.d.M / p.d.groups)) : 1, m = p.d.M / (groups > 0 ? groups : 1);
  double blocks = grouped ? (double)p.d.M / bm + 0.5 * groups : (double)mx_row_blocks(p, bm);
  if (blocks < groups) blocks = groups;
  const double wgs = blocks * (double)cdiv(p.d.N, bn) * split, load = wgs / cus, full = load < 1 ? load : 1;
  const int64_t nsb = cdiv(p.d.K, 512);
  const double steps = split > 1 ? 4.0 * (double)cdiv(nsb, split) : (double)cdiv(p.d.K, 128);
  const double kb_a = (m < bm ? m : bm) / 8, kb_b = (double)(p.d.N < bn ? p.d.N : bn) / 8;  // KB of a step
  const double bytes_b = groups * p.d.N * p.d.K;
  double start, work, rate;  // us before the first step and behind it, us of the work, B's bytes a us at most
  if (tile == FP8_TILE_256) {
    // (a last round of at most half the card runs in 128x128 quarters)
    const double rounds = (double)(int64_t)load, rest = load - rounds;
    const bool quarters = rounds > 0 && rest > 0 && rest <= 0.5;
    start = 6;
    work = (rounds + (quarters ? rest * 1.3 : rest > 0)) * (steps * (rows ? 2.07 : 1.66) + 5) + (quarters ? 4 : 0);
    rate = grouped ? 3.6e6 : 1e9;
  } else if (tile == FP8_TILE_128) {
    start = grouped ? 9.3 : 7;
    work = load <= 1 ? steps * (kb_a + kb_b) / (rows ? 43 : 55)
                     : (double)cdiv((int64_t)wgs, 2 * (int64_t)cus) * (steps * 2 * (kb_a + kb_b) / (rows ? 55 : 65) + 1) - 1;
    rate = grouped ? 4.55e6 : 7e6;
  } else if (tile == FP8_TILE_64) {
    const double rounds = load <= 2 ? (double)cdiv((int64_t)wgs, cus) : load, fill = full * (kb_a + kb_b) / 16;
    const double quad = rows ? 0.72 + 0.22 * fill : 0.55 + 0.35 * fill;
    start = grouped ? 4.2 : (rows ? 2.3 : 2.8);
    work = rounds * (steps / 4 * quad + (grouped ? 3.6 : (rows ? 2.6 : 1.8)));
    rate = grouped ? 4.5e6 : (rows ? 5.6e6 : 6e6);
  } else {
    const int i = tile == FP8_TILE_16 ? 0 : (tile == FP8_TILE_16X32 ? 1 : 2);
    const double first[] = {2.7, 2.8, 3.0}, kb_us_a[] = {50, 100, 95};
    const double kb_us_b[] = {25, 19.5, 18.5}, grouped_b[] = {19.2, 17.6, 18.2}, each[] = {0.15, 0.4, 0.23};
    double one = steps * (kb_b / (grouped ? grouped_b : kb_us_b)[i] + kb_a / kb_us_a[i]);
    if (grouped) one += each[i];
    else if (one < 1.6) one = 1.6;
    start = first[i] + (grouped ? 1.9 : 0);
    work = one * (load > 1 ? load : 1);
    rate = grouped ? 6.1e6 : 1e9;
  }
  double t = start + (work > bytes_b / rate ? work : bytes_b / rate);
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
    mx_tile_extent(p, tile, &bm, &bn);
    if (p.d.tile == MX_TILE_AUTO && !mx_direct_fits(p, tile)) continue;
    for (int32_t split = 1; split <= 64; ++split) {
      const bool wanted = p.d.split > 0 ? split == p.d.split : (split & (split - 1)) == 0 && split <= 16;
      if (!wanted && split > 1) continue;
      if (split > 1 && (!may_split || tile == MX_TILE_256 || split > nsb)) continue;
      if (p.d.split == 1 && split > 1) continue;
      const double t = (p.b_scaling >= 0 ? estimate_fp8 : estimate)(p, cus, tile, split) - (p.d.split > 1 && split == p.d.split ? 1e9 : 0);
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
  mx_tile_extent(p, tile, &bm, &bn);
  return mx_row_blocks(p, bm) <= 65535 && cdiv(p.d.N, bn) < (1 << 23);
}

int64_t mx_workspace_bytes(const mx_gemm_plan& p, const MxChoice& c) {
  return c.split > 1 ? (int64_t)c.split * p.d.M * p.d.N * 4 : 0;
}

gemm_status block_gemm_init(const char* fn, const mx_gemm_desc& d, int32_t b_scaling, mx_gemm_plan* p) {
  if (d.M < 0 || d.N < 0 || d.K < 0) return fail(GEMM_ERR_INVALID_ARG, "%s: negative size", fn);
  if (d.groups < 0) return fail(GEMM_ERR_INVALID_ARG, "%s: negative group count", fn);
  if (d.groups > kMaxVarlenGroups) return fail(GEMM_ERR_UNSUPPORTED, "%s: more than %d groups", fn, kMaxVarlenGroups);
  for (int32_t f : {d.a_format, d.b_format})
    if (f != MX_E2M1 && f != MX_E4M3) return fail(GEMM_ERR_INVALID_ARG, "%s: unknown format %d", fn, f);
  for (int32_t t : {d.c, d.d, d.post})
    if (t < GEMM_DT_NONE || t > GEMM_DT_E5M2) return fail(GEMM_ERR_INVALID_ARG, "%s: unknown type %d", fn, t);
  if (d.d == GEMM_DT_NONE && d.post == GEMM_DT_NONE) return fail(GEMM_ERR_INVALID_ARG, "%s: neither D nor PostAct", fn);
  if (d.act < GEMM_ACT_NONE || d.act > GEMM_ACT_SILU) return fail(GEMM_ERR_INVALID_ARG, "%s: unknown activation %d", fn, d.act);
  if (d.act != GEMM_ACT_NONE && d.post == GEMM_DT_NONE) return fail(GEMM_ERR_INVALID_ARG, "%s: an activation without PostAct", fn);
  if (d.tile < MX_TILE_AUTO || d.tile > MX_TILE_16) return fail(GEMM_ERR_INVALID_ARG, "%s: unknown tile %d", fn, d.tile);
  if (d.split < 0 || d.split > 64) return fail(GEMM_ERR_INVALID_ARG, "%s: split must lie in [0, 64]", fn);
  if (d.split > 1 && (d.groups || d.tile == MX_TILE_256))
    return fail(GEMM_ERR_UNSUPPORTED, "%s: a grouped plan and the 256x256 tile do not split K", fn);
  if (d.N % 8) return fail(GEMM_ERR_ALIGNMENT, "%s: N = %d is not a multiple of 8", fn, d.N);
  // (256 rows of codes stay below 2^31 bytes: the kernels' offsets inside a tile are 32-bit)
  if (d.K > (1 << 22)) return fail(GEMM_ERR_UNSUPPORTED, "%s: K above 2^22", fn);
  gemm_status st = check_out(fn, "C", d.c, d.ldc, d.M, d.N);
  if (st == GEMM_OK) st = check_out(fn, "D", d.d, d.ldd, d.M, d.N);
  if (st == GEMM_OK) st = check_out(fn, "PostAct", d.post, d.ldp, d.M, d.N);
  if (st != GEMM_OK) return st;
  p->d = d;
  p->b_scaling = b_scaling;
  const bool fp8 = b_scaling >= 0;
  auto codes = [&](int64_t rows, int32_t format) { return fp8 ? fp8_code_bytes(rows, d.K) : mx_code_bytes(rows, d.K, format); };
  p->lda = (int32_t)codes(1, d.a_format);
  p->ldb = (int32_t)codes(1, d.b_format);
  p->a_bytes = codes(d.M, d.a_format);
  p->b_bytes = codes(d.N, d.b_format);
  p->sa_bytes = fp8 ? fp8_scale_bytes(d.M, d.K, FP8_ROWS) : mx_scale_bytes(d.M, d.K);
  p->sb_bytes = fp8 ? fp8_scale_bytes(d.N, d.K, b_scaling) : mx_scale_bytes(d.N, d.K);
  int32_t bm, bn;
  mx_tile_extent(*p, MX_TILE_128, &bm, &bn);
  if (mx_row_blocks(*p, bm) * cdiv(d.N, bn) > 0xFFFFFF) return fail(GEMM_ERR_UNSUPPORTED, "%s: too many output tiles", fn);
  clear_error();
  return GEMM_OK;
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
  const char* fn = "mx_gemm_create";
  if (!out) return fail(GEMM_ERR_INVALID_ARG, "%s: NULL out", fn);
  *out = nullptr;
  if (!d) return fail(GEMM_ERR_INVALID_ARG, "%s: NULL desc", fn);
  mx_gemm_plan* p = new (std::nothrow) mx_gemm_plan;
  if (!p) return fail(GEMM_ERR_NO_MEMORY, "%s: out of memory", fn);
  const gemm_status st = block_gemm_init(fn, *d, -1, p);
  if (st != GEMM_OK) {
    delete p;
    return st;
  }
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

// ---- FP8 products

static_assert((int)FP8_TILE_AUTO == (int)MX_TILE_AUTO && (int)FP8_TILE_256 == (int)MX_TILE_256 && (int)FP8_TILE_128 == (int)MX_TILE_128 &&
                  (int)FP8_TILE_64 == (int)MX_TILE_32X64 && (int)FP8_TILE_32 == (int)MX_TILE_32 &&
                  (int)FP8_TILE_16X32 == (int)MX_TILE_16X32 && (int)FP8_TILE_16 == (int)MX_TILE_16,
              "one numbering of the tiles");

int64_t fp8_code_bytes(int64_t rows, int64_t k) {
  if (rows < 0 || k < 0) return -1;
  int64_t row, all;
  if (__builtin_mul_overflow(blocks_of(k, 16), (int64_t)16, &row) || __builtin_mul_overflow(rows, row, &all)) return rows == 0 ? 0 : -1;
  return all;
}

int64_t fp8_scale_bytes(int64_t rows, int64_t k, int32_t scaling) {
  if (rows < 0 || k < 0 || (scaling != FP8_ROWS && scaling != FP8_TILES)) return -1;
  int64_t quads, all;
  const int64_t units = scaling == FP8_ROWS ? blocks_of(rows, 64) : blocks_of(rows, FP8_BLOCK);
  if (__builtin_mul_overflow(units, blocks_of(blocks_of(k, FP8_BLOCK), 4), &quads) ||
      __builtin_mul_overflow(quads, (int64_t)(scaling == FP8_ROWS ? 64 * 16 : 16), &all))
    return -1;
  return all;
}

gemm_status fp8_gemm_create(const fp8_gemm_desc* d, fp8_gemm_plan** out) {
  const char* fn = "fp8_gemm_create";
  if (!out) return fail(GEMM_ERR_INVALID_ARG, "%s: NULL out", fn);
  *out = nullptr;
  if (!d) return fail(GEMM_ERR_INVALID_ARG, "%s: NULL desc", fn);
  if (d->b_scaling != FP8_ROWS && d->b_scaling != FP8_TILES) return fail(GEMM_ERR_INVALID_ARG, "%s: unknown scaling %d", fn, d->b_scaling);
  fp8_gemm_plan* p = new (std::nothrow) fp8_gemm_plan;
  if (!p) return fail(GEMM_ERR_NO_MEMORY, "%s: out of memory", fn);
  const mx_gemm_desc m{d->M, d->N, d->K, d->groups, MX_E4M3, MX_E4M3, d->c, d->d, d->post, d->act, d->tile, d->split, d->ldc, d->ldd, d->ldp};
  const gemm_status st = block_gemm_init(fn, m, d->b_scaling, p);
  if (st != GEMM_OK) {
    delete p;
    return st;
  }
  *out = p;
  return GEMM_OK;
}

gemm_status fp8_gemm_destroy(fp8_gemm_plan* plan) {
  delete plan;
  clear_error();
  return GEMM_OK;
}

gemm_status fp8_gemm_plan_tile(const fp8_gemm_plan* plan, int32_t num_cus, int32_t* tile, int32_t* split) {
  if (!plan || num_cus < 1) return fail(GEMM_ERR_INVALID_ARG, "fp8_gemm_plan_tile: NULL plan or no compute units");
  return mx_gemm_plan_tile(plan, num_cus, tile, split);
}

gemm_status fp8_gemm_workspace(const fp8_gemm_plan* plan, int32_t num_cus, int64_t* bytes) {
  if (!plan || !bytes || num_cus < 1) return fail(GEMM_ERR_INVALID_ARG, "fp8_gemm_workspace: NULL argument or no compute units");
  return mx_gemm_workspace(plan, num_cus, bytes);
}

}  // extern "C"
