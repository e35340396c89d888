// Host-only fuzz of the MX product's plans and of the storage sizes for a sanitizer build: seeded random
// descriptors, most near the validation boundaries, and sizes up to the largest int64. Every call must
// return without undefined behaviour or invalid memory use; valid plans must report a tile, a split and a
// workspace that agree. Exit status 0 on success.
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <initializer_list>

#include "../../include/mx_mi355x.h"

static uint64_t rs = 0xD1B54A32D192ED03ull;
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
    // a valid descriptor, then (most of the time) a field or two perturbed
    mx_gemm_desc d;
    memset(&d, 0, sizeof(d));
    d.M = (int32_t)(next() % 20000);
    d.N = (int32_t)(8 * (next() % 1200));
    d.K = (int32_t)(next() % 20000);
    d.groups = next() % 3 ? 0 : (int32_t)(next() % 1025);
    d.a_format = (int32_t)(next() % 2);
    d.b_format = (int32_t)(next() % 2);
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
        case 7: d.a_format = (int32_t)(next() % 4) - 1; d.d = (int32_t)(next() % 8) - 1; break;
        case 8: d.tile = (int32_t)(next() % 9) - 1; break;
        default: d.split = (int32_t)pick(sizes, ns); break;
      }
    }
    mx_gemm_plan* p = nullptr;
    if (mx_gemm_create(&d, &p) == GEMM_OK) {
      ++ok;
      for (int32_t cus : {1, 256, 65535, 65536, 0x7FFFFFFF}) {
        int32_t tile = 0, split = 0;
        int64_t bytes = -1;
        if (mx_gemm_plan_tile(p, cus, &tile, &split) != GEMM_OK || mx_gemm_workspace(p, cus, &bytes) != GEMM_OK) return 2;
        if (tile < MX_TILE_256 || tile > MX_TILE_16 || split < 1 || split > 64 || (d.tile && tile != d.tile)) return 3;
        if (split > 1 && (d.groups || tile == MX_TILE_256 || (int64_t)(split - 1) * 512 >= d.K)) return 4;
        if (bytes != (split > 1 ? (int64_t)split * d.M * d.N * 4 : 0)) return 5;
      }
      if (mx_gemm_destroy(p) != GEMM_OK) return 6;
    } else {
      ++rejected;
      if (p != nullptr || gemm_last_error()[0] == 0) return 7;
    }
  }
  if (mx_gemm_create(nullptr, nullptr) == GEMM_OK) return 8;
  const int64_t wide[] = {0, 1, 31, 32, 33, 64, 512, (int64_t)1 << 31, (int64_t)1 << 40, INT64_MAX - 31, INT64_MAX, -1, INT64_MIN};
  const int nw = (int)(sizeof(wide) / sizeof(wide[0]));
  for (int i = 0; i < nw; ++i)
    for (int j = 0; j < nw; ++j)
      for (int32_t f = -1; f < 3; ++f) {
        const int64_t r = wide[i], k = wide[j], c = mx_code_bytes(r, k, f), s = mx_scale_bytes(r, k);
        const bool bad = r < 0 || k < 0;
        // the sizes as 128-bit products, or -1 where 63 bits do not hold them
        const __int128 nb = bad ? 0 : ((__int128)k + 31) / 32, most = INT64_MAX;
        const __int128 wc = (__int128)(bad ? 0 : r) * nb * (f == MX_E2M1 ? 16 : 32);
        const __int128 rows = bad ? 0 : ((__int128)r + 63) / 64, tiles = (nb + 15) / 16;
        const bool fits = rows == 0 || tiles == 0 || rows <= most / 1024 / tiles;
        if (c != (bad || (f != MX_E2M1 && f != MX_E4M3) || wc > most ? -1 : (int64_t)wc)) return 9;
        if (s != (bad || !fits ? -1 : (int64_t)(rows * tiles * 1024))) return 10;
      }
  printf("mx plans accepted %d, rejected %d\n", ok, rejected);
  return ok > 0 && rejected > 0 ? 0 : 11;
}
