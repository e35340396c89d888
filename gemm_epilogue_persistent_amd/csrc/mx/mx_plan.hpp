// Host-side plan of an MX product.
#pragma once
#include <stdint.h>

#include "../../../include/mx_mi355x.h"
#include "../params.hpp"

struct mx_gemm_plan {
  mx_gemm_desc d;
  int64_t a_bytes, b_bytes;    // codes (B: of one group)
  int64_t sa_bytes, sb_bytes;  // scales
  int32_t lda, ldb;            // bytes of a row of codes
};

namespace gep {
// The tile a plan runs with `cus` compute units (an mx_tile, never AUTO), and its rows and columns.
int32_t mx_choose_tile(const mx_gemm_plan& p, int32_t cus);
void mx_tile_extent(int32_t tile, int32_t* bm, int32_t* bn);
// Upper bound of the row blocks of a tile of bm rows over all groups (exact for a dense plan).
int64_t mx_row_blocks(const mx_gemm_plan& p, int32_t bm);
}  // namespace gep
