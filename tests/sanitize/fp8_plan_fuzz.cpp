// Host-only fuzz of the FP8 product's plans and of the storage sizes for a sanitizer build: seeded random
// descriptors, most near the validation boundaries, and sizes up to the largest int64. Every call must
// return without undefined behaviour or invalid memory use; valid plans must report a tile, a split and a
// workspace that agree. Exit status 0 on success.
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <initializer_list>

#include "../../include/fp8_mi355x.h"

static uint64_t rs = 0xA0761D6478BD642Full;
static uint64_t next() {  // splitmix64
  uint64_t z = (rs += 0x9E3779B97F4A7C15ull);
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return z ^ (z >> 31);
}
static int64_t pick(const int64_t* v, int n) { return v[next() % n]; }

int main() {
  const int64_t sizes[] = {0, 1, 7, 8, 16, 100, 512, 513, 4096, 8192, 65536, 1 << 20, 1 << 22, (1 << 22) + 1, 1 << 30, 0x7FFFFFF8, 0x7FFFFFFF, -1, -0x7FFFFFFF - 1};
  const int64_t lds[] = {0, 8, 16, 64, 260, 8192, 1 << 24, (int64_t)1 << 31, (int64_t)1 << 48, ((int64_t)1 << 48) + 8, INT64_MAX, INT64_MIN, -8};
  const int ns = (int)(sizeof(sizes) / sizeof(sizes[0])), nl = (int)(sizeof(lds) / sizeof(lds[0]));
  int ok = 0, rejected = 0;
  for (int it = 0; it < 100000; ++it) {
    fp8_gemm_desc d;
    memset(&d, 0, sizeof(d));
    d.M = (int32_t)(next() % 20000);
    d.N = (int32_t)(8 * (next() % 1200));
    d.K = (int32_t)(next() % 20000);
    d.groups = next() % 3 ? 0 : (int32_t)(next() % 1025);
    d.b_scaling = (int32_t)(next() % 2);
    d.c = next() % 2 ? GEMM_DT_NONE : GEMM_DT_BF16;
    d.d = GEMM_DT_F32;
    d.post = next() % 2 ? GEMM_DT_NONE : GEMM_DT_F16;
    d.act = d.post ? (int32_t)(next() % 5) : 0;
    d.tile = next() % 2 ? 0 : (int32_t)(next() % 7);
    d.split = next() % 2 ? 0 : (int32_t)(next() % 65);
    d.ldc = d.ldd = d.ldp = d.N + 8 * (int64_t)(next() % 3);
    for (uint64_t n = next() % 3; n > 0; --n) {
      switch (next() % 10) {
        case 0: d.M = (int32_t)pick(sizes, ns); break;
        case 1: d.N = (int32_t)pick(sizes, ns); d.ldc = d.ldd = d.ldp = d.N; break;
        case 2: d.K = (int32_t)pick(sizes, ns); break;
        case 3: d.groups = (int32_t)pick(sizes, ns); break;
        case 4: d.ldc = pick(lds, nl); break;
        case 5: d.ldd = pick(lds, nl); break;
        case 6: d.ldp = pick(lds, nl); break;
        case 7: d.b_scaling = (int32_t)(next() % 4) - 1; d.d = (int32_t)(next() % 8) - 1; break;
        case 8: d.tile = (int32_t)(next() % 9) - 1; break;
        default: d.split = (int32_t)pick(sizes, ns); break;
      }
    }
    fp8_gemm_plan* p = nullptr;
    if (fp8_gemm_create(&d, &p) == GEMM_OK) {
      ++ok;
      for (int32_t cus : {1, 256, 65535, 65536, 0x7FFFFFFF}) {
        int32_t tile = 0, split = 0;
        int64_t bytes = -1;
        if (fp8_gemm_plan_tile(p, cus, &tile, &split) != GEMM_OK || fp8_gemm_workspace(p, cus, &bytes) != GEMM_OK) return 2;
        if (tile < FP8_TILE_256 || tile > FP8_TILE_16 || split < 1 || split > 64 || (d.tile && tile != d.tile)) return 3;
        if (split > 1 && (d.groups || tile == FP8_TILE_256 || (int64_t)(split - 1) * 512 >= d.K)) return 4;
        if (bytes != (split > 1 ? (int64_t)split * d.M * d.N * 4 : 0)) return 5;
      }
      if (fp8_gemm_destroy(p) != GEMM_OK) return 6;
    } else {
      ++rejected;
      if (p != nullptr || gemm_last_error()[0] == 0) return 7;
    }
  }
  if (fp8_gemm_create(nullptr, nullptr) == GEMM_OK) return 8;
  const int64_t wide[] = {0, 1, 15, 16, 17, 64, 128, 129, 512, (int64_t)1 << 31, (int64_t)1 << 40, INT64_MAX - 127, INT64_MAX, -1, INT64_MIN};
  const int nw = (int)(sizeof(wide) / sizeof(wide[0]));
  for (int i = 0; i < nw; ++i)
    for (int j = 0; j < nw; ++j)
      for (int32_t f = -1; f < 3; ++f) {
        const int64_t r = wide[i], k = wide[j], c = fp8_code_bytes(r, k), s = fp8_scale_bytes(r, k, f);
        const bool bad = r < 0 || k < 0, unknown = f != FP8_ROWS && f != FP8_TILES;
        // the sizes as 128-bit products, or -1 where 63 bits do not hold them
        const __int128 most = INT64_MAX, kp = bad ? 0 : ((__int128)k + 15) / 16 * 16, nq = bad ? 0 : (((__int128)k + 127) / 128 + 3) / 4;
        const __int128 rows = bad ? 0 : r, units = f == FP8_ROWS ? (rows + 63) / 64 : (rows + 127) / 128, each = f == FP8_ROWS ? 1024 : 16;
        const bool fits = units == 0 || nq == 0 || units <= most / each / nq;
        const bool codes = rows == 0 || kp == 0 || rows <= most / kp;
        if (c != (bad || !codes ? -1 : (int64_t)(rows * kp))) return 9;
        if (s != (bad || unknown || !fits ? -1 : (int64_t)(units * nq * each))) return 10;
      }
  printf("fp8 plans accepted %d, rejected %d\n", ok, rejected);
  return ok > 0 && rejected > 0 ? 0 : 11;
}
