// Host-side plan of a product of block-scaled operands: MX, or FP8 with a scale per 128 values.
#pragma once
#include <stdint.h>

#include <atomic>

#include "../../../include/fp8_mi355x.h"
#include "../../../include/mx_mi355x.h"
#include "../params.hpp"

struct mx_gemm_plan {
  mx_gemm_desc d;               // (FP8: both formats MX_E4M3)
  int32_t b_scaling = -1;       // FP8 operands: the fp8_scaling of B; -1: MX operands
  int64_t a_bytes, b_bytes;    // codes (B: of one group)
  int64_t sa_bytes, sb_bytes;  // scales
  int32_t lda, ldb;            // bytes of a row of codes
  // The choice made last, with and without a workspace: compute units, tile, split and per in 16, 8, 8
  // and 32 bits (0: none yet). Choosing takes 1.2 us, a fifth of a short run.
  mutable std::atomic<uint64_t> chosen[2] = {{0}, {0}};
};

// (An FP8 plan is the same thing under its own entry points.)
struct fp8_gemm_plan : mx_gemm_plan {};

namespace gep {
// Validate `d` for the entry point `fn` and fill in `p`.
gemm_status block_gemm_init(const char* fn, const mx_gemm_desc& d, int32_t b_scaling, mx_gemm_plan* p);
// Launch a plan's product for the entry point `fn`.
gemm_status block_gemm_run(const char* fn, const mx_gemm_plan* plan, const mx_gemm_args* a, void* stream);

// How a plan runs on `cus` compute units: the tile (an mx_tile, never AUTO), over how many
// workgroups a tile's K is shared out, and the scale tiles (512 values of K) of each.
struct MxChoice {
  int32_t tile, split, per;
};
MxChoice mx_choose(const mx_gemm_plan& p, int32_t cus, bool workspace);
// The same, kept in the plan for the next run.
MxChoice mx_choice(const mx_gemm_plan& p, int32_t cus, bool workspace);
// (Tile 3 is 32x64 of an MX plan and 64x64 of an FP8 one; the others are alike.)
void mx_tile_extent(const mx_gemm_plan& p, int32_t tile, int32_t* bm, int32_t* bn);
// Upper bound of the row blocks of a tile of bm rows over all groups (exact for a dense plan).
int64_t mx_row_blocks(const mx_gemm_plan& p, int32_t bm);
// Whether the grid of a direct kernel (tiles of at most 64 rows) can be launched: row blocks in 16 bits,
// columns of up to 512 threads in 32. True for the other tiles.
bool mx_direct_fits(const mx_gemm_plan& p, int32_t tile);
int64_t mx_workspace_bytes(const mx_gemm_plan& p, const MxChoice& c);
}  // namespace gep
