// Host-side plan of an MX product.
#pragma once
#include <stdint.h>

#include <atomic>

#include "../../../include/mx_mi355x.h"
#include "../params.hpp"

struct mx_gemm_plan {
  mx_gemm_desc d;
  int64_t a_bytes, b_bytes;    // codes (B: of one group)
  int64_t sa_bytes, sb_bytes;  // scales
  int32_t lda, ldb;            // bytes of a row of codes
  // The choice made last, with and without a workspace: compute units, tile, split and per in 16, 8, 8
  // and 32 bits (0: none yet). Choosing takes 1.2 us, a fifth of a short run.
  mutable std::atomic<uint64_t> chosen[2] = {{0}, {0}};
};

namespace gep {
// How a plan runs on `cus` compute units: the tile (an mx_tile, never AUTO), over how many
// workgroups a tile's K is shared out, and the scale tiles (512 values of K) of each.
struct MxChoice {
  int32_t tile, split, per;
};
MxChoice mx_choose(const mx_gemm_plan& p, int32_t cus, bool workspace);
// The same, kept in the plan for the next run.
MxChoice mx_choice(const mx_gemm_plan& p, int32_t cus, bool workspace);
void mx_tile_extent(int32_t tile, int32_t* bm, int32_t* bn);
// Upper bound of the row blocks of a tile of bm rows over all groups (exact for a dense plan).
int64_t mx_row_blocks(const mx_gemm_plan& p, int32_t bm);
// Whether the grid of a direct kernel (tiles of at most 32 rows) can be launched: row blocks in 16 bits,
// columns of up to 512 threads in 32. True for the other tiles.
bool mx_direct_fits(const mx_gemm_plan& p, int32_t tile);
int64_t mx_workspace_bytes(const mx_gemm_plan& p, const MxChoice& c);
}  // namespace gep
