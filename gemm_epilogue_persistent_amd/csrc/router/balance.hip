// Per-expert counts, balance loss and its gradient (router_balance, router_balance_backward of the public header).
//
// The logits are read once in each direction. G neighbouring lanes hold a token's logits, 8 (or 16, 32) a lane, so that a
// row is one coalesced load and its sums stay in registers; a workgroup takes a run of tokens of one sequence.
//
// Three kernels: sums of a workgroup, their join, the gradient. Bound by the launches and by the latency of what follows
// on each other: 16 tokens over 8 experts 3.7 us (one workgroup, no join) and 2.1; 8 x 4096 tokens over 256 experts bf16
// with sigmoids 9.2 to 10.3, 6.2 to 6.6 and 9.6 to 11.4 us, of which memory needs 3.5, 0 and 7 and the about 21 vector instructions a value
// 5 in each direction; 8192 tokens over 2048 experts 14, 10 and 17 for 34 MB in and 34 out. Forward workgroups
// of 512 threads are no faster than of 1024; backward, up to 2048 workgroups in all instead of 1024 save 2 us in 31.
#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "../../../include/router_mi355x.h"
#include "../mx/mx_common.hpp"

namespace gep {
gemm_status fail(gemm_status st, const char* fmt, ...);
void clear_error();

namespace {

constexpr int kThreads = 256;
constexpr int kMaxExperts = 2048;
__device__ __forceinline__ uint32_t lesser(uint32_t a, uint32_t b) { return a < b ? a : b; }

// ---- exchange over the G lanes of a row (G a power of two; fixed order, the same result in every lane)
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xF, 0xF, true));
}
template <int G, typename F>
__device__ __forceinline__ float reduce(float v, F&& f) {
  if constexpr (G >= 2) v = f(v, dpp<0xB1>(v));   // lanes 1 0 3 2
  if constexpr (G >= 4) v = f(v, dpp<0x4E>(v));   // lanes 2 3 0 1
  if constexpr (G >= 8) v = f(v, dpp<0x141>(v));  // within 8: i <-> 7 - i
  if constexpr (G >= 16) v = f(v, dpp<0x140>(v));  // within 16: i <-> 15 - i
  if constexpr (G >= 32) v = f(v, __shfl_xor(v, 16));
  if constexpr (G >= 64) v = f(v, __shfl_xor(v, 32));
  return v;
}
template <int G>
__device__ __forceinline__ float row_sum(float v) { return reduce<G>(v, [](float a, float b) { return a + b; }); }
template <int G>
__device__ __forceinline__ float row_max(float v) { return reduce<G>(v, [](float a, float b) { return fmaxf(a, b); }); }
// Whether v holds in any lane of the row.
template <int G>
__device__ __forceinline__ bool row_any(bool v) {
  const uint64_t all = __ballot(v);
  if constexpr (G == 64) return all != 0;
  else return (all >> (threadIdx.x & (64 - G)) & (((uint64_t)1 << G) - 1)) != 0;
}

// e^x of x <= 0 to about an fp32 step: what the roundings of x log2 e and of log2 e itself leave is put back, so that the error does
// not grow with x (1.2e-7 of the value down to -87, 0 below; without log2 e's own rest 1.2e-6 at -80). NaN for NaN.
__device__ __forceinline__ float exp_neg(float x) {
  constexpr float log2e = 1.44269502162933349609375f, rest = 1.925962989e-8f;  // (log2 e in two numbers)
  const float c = __builtin_elementwise_maximum(x, -104.f);  // (e^-104 is below fp32)
  const float t = c * log2e, lo = __builtin_fmaf(c, rest, __builtin_fmaf(c, log2e, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(e * lo, 0.693147182464599609375f, e);
}
template <int G, int N>
__device__ __forceinline__ float row_top(const float (&x)[N][8]) {
  float top = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, x[i][e]);
  return row_max<G>(top);
}

// The scores of a row from its logits x, -inf past the last expert: p = u inv (8 N a lane), 0 where p is below fp32's normal
// numbers. miss: 1 - s(x) (sigmoid). A row of -inf alone has inv = 0; a NaN, and an infinity under a softmax, make the sum and inv NaN.
template <int G, int N, int SCORES>
__device__ __forceinline__ float row_scores(const float (&x)[N][8], float (&u)[N][8], float (&miss)[N][8]) {
  float sum = 0.f;
  if constexpr (SCORES == ROUTER_SOFTMAX) {
    const float m = fmaxf(row_top<G, N>(x), -3.402823466e38f);  // (-inf less -inf is no number)
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) u[i][e] = exp_neg(x[i][e] - m), sum += u[i][e];
    sum = row_sum<G>(sum);
  } else {
    // s(x) = a q or q with a = e^-|x|, q = 1 / (1 + a); 1 - s(x) is the other one
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float a = exp_neg(-fabsf(x[i][e])), q = __builtin_amdgcn_rcpf(1.f + a), aq = a * q;
        u[i][e] = x[i][e] < 0.f ? aq : q;
        miss[i][e] = x[i][e] < 0.f ? q : aq;
        sum += u[i][e];
      }
    sum = row_sum<G>(sum);
    // e^x ends at 2^-126 = e^-87.3, p only where s(x) / sum does: a row whose sum is below 1 and that has a logit further down
    // takes s(x) = e^x (1 - s(x)) times e^-top, which the quotient cancels. (Looking for one where all sums are below 1: 8 x 4096
    // tokens over 256 experts bf16, forward 16.6 to 17.5 us, backward 13.2 to 13.5.)
    if (sum < 1.f) {
      float low = 0.f;  // (of the finite ones)
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) low = fminf(low, x[i][e] > -__builtin_inff() ? x[i][e] : 0.f);
      if (row_any<G>(low < -87.f)) {
        const float m = row_top<G, N>(x);
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) u[i][e] = exp_neg(x[i][e] - m) * miss[i][e], sum += u[i][e];
        sum = row_sum<G>(sum);
      }
    }
  }
  return sum == 0.f ? 0.f : 1.f / sum;
}

// WHOLE: the experts fill the lanes.
template <typename T, int G, int N, bool WHOLE>
struct Rows {
  Chunk<T> c[N];
  // Lane l of the row's group takes chunks l, l + G, ...
  __device__ __forceinline__ void load(const T* row, int experts, int lane) {
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = load_chunk<WHOLE>(row, (i * G + lane) * 8, experts);
  }
  __device__ __forceinline__ void values(int experts, int lane, float (&x)[N][8]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = (i * G + lane) * 8;
      if (!WHOLE) settle<false>(c[i], at, experts);
      unpack(c[i], x[i]);
      if (WHOLE) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i][e] = at + e < experts ? x[i][e] : -__builtin_inff();
    }
  }
};

struct Forward {
  int batch, tokens, experts, k, scores, index_bytes;
  float coef;
  const void* logits;
  const void* chosen;
  const uint8_t* mask;
  int32_t *counts, *valid, *cu_seqlens;
  float *probs, *loss;
  int64_t ld, ldb;
  int per, wgs;  // tokens of a workgroup, workgroups of a sequence
  // partial results of workgroup i of sequence b: part (b * wgs + i); and what the join shares
  float* part_p;
  int32_t *part_c, *part_n;
  float* part_loss;
  uint32_t* ticket;
};

// Expert e of sequence b is joined; its share of sum_e c_e P_e / n.
__device__ __forceinline__ float finish_expert(const Forward& a, int b, int e, float p, int32_t c, int32_t n) {
  const float mean = n > 0 ? p / (float)n : 0.f;
  a.probs[(int64_t)b * a.experts + e] = mean;
  a.counts[(int64_t)b * a.experts + e] = c;
  return n > 0 ? (float)c / (float)n * mean : 0.f;
}
__device__ __forceinline__ float loss_factor(const Forward& a) { return a.coef * (float)a.experts / ((float)a.batch * (float)a.k); }

// Sum over the workgroup in a fixed order, in every thread. buf: a float for each wave.
template <int TH>
__device__ __forceinline__ float block_sum(float v, float* buf) {
  v = row_sum<64>(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
  __syncthreads();
  v = buf[0];
#pragma unroll
  for (int w = 1; w < TH / 64; ++w) v += buf[w];
  return v;
}
// cu[i + 1] = sum of the first i + 1 totals (total(e): a function); one workgroup.
template <int TH, typename F>
__device__ __forceinline__ void offsets(int32_t* cu, int experts, F&& total, int32_t* buf) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int32_t base = 0;
  if (tid == 0) cu[0] = 0;
  for (int e0 = 0; e0 < experts; e0 += TH) {
    const int e = e0 + tid;
    int32_t v = e < experts ? total(e) : 0;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int32_t u = __shfl_up(v, off);
      if (lane >= off) v += u;
    }
    __syncthreads();
    if (lane == 63) buf[wave] = v;
    __syncthreads();
    int32_t before = base;
#pragma unroll
    for (int w = 0; w < TH / 64; ++w) {
      before += w < wave ? buf[w] : 0;
      base += buf[w];
    }
    if (e < experts) cu[e + 1] = before + v;
  }
}

// The tokens of one workgroup of TH threads. ONE: they are all there are, and the results are finished here.
template <typename T, int G, int N, int SCORES, bool WHOLE, bool ONE, int TH>
__global__ __launch_bounds__(TH) void balance_kernel(const Forward a) {
  constexpr int kCols = 8 * G * N, kWaves = TH / 64, kGroups = TH / G, kAhead = N == 1 ? 4 : (N == 2 ? 2 : 1);
  __shared__ float psum[kWaves][kCols];
  __shared__ int32_t hist[kCols];
  __shared__ int32_t tokens_seen;
  __shared__ float red[kWaves];
  const int tid = threadIdx.x, lane = tid & (G - 1), group = tid / G, wave = tid >> 6;
  const int b = blockIdx.y, wg = blockIdx.x;
  const uint32_t t0 = (uint32_t)wg * a.per, t1 = lesser((uint32_t)a.tokens, t0 + a.per);  // (a token's number may pass the last one)
  const uint8_t* mask = a.mask ? a.mask + (int64_t)b * a.tokens : nullptr;
  const T* logits = (const T*)a.logits + b * a.ldb;
  Rows<T, G, N, WHOLE> rows[kAhead];
  bool use[kAhead];
  auto fetch = [&](uint32_t t) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const uint32_t tt = t + u * kGroups, at = lesser(tt, t1 - 1);
      use[u] = tt < t1 && (!mask || mask[at]);
      rows[u].load(logits + at * a.ld, a.experts, lane);
    }
  };
  fetch(t0 + group);  // (under way while the choices are counted)
  if (!ONE && tid == 0 && b == 0 && wg == 0) *a.ticket = 0;  // (for the join, the next launch)
  for (int e = tid; e < kCols; e += TH) hist[e] = 0;
  if (tid == 0) tokens_seen = 0;
  __syncthreads();
  const int64_t id0 = ((int64_t)b * a.tokens + t0) * a.k;
  const uint32_t ids = (t1 - t0) * (uint32_t)a.k;
  for (uint32_t i = tid; i < ids; i += 4 * TH) {  // (four loads under way)
    int64_t e[4];
    bool counts[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t at = lesser(i + u * TH, ids - 1);
      e[u] = a.index_bytes == 8 ? ((const int64_t*)a.chosen)[id0 + at] : (int64_t)((const int32_t*)a.chosen)[id0 + at];
      counts[u] = i + u * TH < ids && (!mask || mask[t0 + at / (uint32_t)a.k]);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (counts[u] && e[u] >= 0 && e[u] < a.experts) atomicAdd(&hist[(int)e[u]], 1);
  }
  float acc[N][8];
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[i][e] = 0.f;
  int seen = 0;
  for (uint32_t t = t0 + group;;) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (!use[u]) continue;
      float x[N][8], s[N][8], miss[N][8];
      rows[u].values(a.experts, lane, x);
      const float inv = row_scores<G, N, SCORES>(x, s, miss);
      ++seen;
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[i][e] = __builtin_fmaf(s[i][e], inv, acc[i][e]);
    }
    t += kGroups * kAhead;
    if (t >= t1) break;
    fetch(t);
  }
  if (lane == 0 && seen) atomicAdd(&tokens_seen, seen);
  // over the row groups of the wave, then over the waves
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
      for (int off = G; off < 64; off <<= 1) acc[i][e] += __shfl_xor(acc[i][e], off);
  if ((tid & 63) < G) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) psum[wave][(i * G + lane) * 8 + e] = acc[i][e];
  }
  __syncthreads();
  const int32_t n = tokens_seen;
  float mine = 0.f;
  for (int e = tid; e < a.experts; e += TH) {
    float p = psum[0][e];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) p += psum[w][e];
    if constexpr (ONE) {
      mine += finish_expert(a, b, e, p, hist[e], n);
    } else {
      const int64_t at = ((int64_t)b * a.wgs + wg) * a.experts + e;
      a.part_p[at] = p;
      a.part_c[at] = hist[e];
    }
  }
  if constexpr (ONE) {
    const float all = block_sum<TH>(mine, red);
    if (tid == 0) {
      a.valid[0] = n;
      *a.loss = all * loss_factor(a);
    }
    if (a.cu_seqlens) offsets<TH>(a.cu_seqlens, a.experts, [&](int e) { return hist[e]; }, (int32_t*)red);
  } else if (tid == 0) {
    a.part_n[(int64_t)b * a.wgs + wg] = n;
  }
}

// Joins the workgroups' sums of one sequence for 64 experts, a share of them in each wave of TH threads; the last workgroup of all
// adds up the loss, in order, and the offsets.
template <int TH>
__global__ __launch_bounds__(TH) void balance_join_kernel(const Forward a) {
  constexpr int kWaves = TH / 64;
  __shared__ float psum[kWaves][64];
  __shared__ int32_t csum[kWaves][64], nsum[kWaves];
  __shared__ float red[kWaves];
  __shared__ uint32_t last;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, b = blockIdx.y;
  const int e = blockIdx.x * 64 + lane;
  const int64_t first = (int64_t)b * a.wgs;
  int32_t n = 0;
  for (int i = tid; i < a.wgs; i += TH) n += a.part_n[first + i];
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) n += __shfl_xor(n, off);
  float p = 0.f;
  int32_t c = 0;
  if (e < a.experts) {
#pragma unroll 8
    for (int i = wave; i < a.wgs; i += kWaves) {
      p += a.part_p[(first + i) * a.experts + e];
      c += a.part_c[(first + i) * a.experts + e];
    }
  }
  psum[wave][lane] = p;
  csum[wave][lane] = c;
  if (lane == 0) nsum[wave] = n;
  __syncthreads();
  if (wave == 0) {
    n = nsum[0], p = psum[0][lane], c = csum[0][lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) n += nsum[w], p += psum[w][lane], c += csum[w][lane];
    float mine = e < a.experts ? finish_expert(a, b, e, p, c, n) : 0.f;
    mine = row_sum<64>(mine);
    if (lane == 0) {
      if (blockIdx.x == 0) a.valid[b] = n;
      a.part_loss[(int64_t)b * gridDim.x + blockIdx.x] = mine;
    }
  }
  if (wave == 0) {  // (all stores are its own; a fence of every wave costs 0.5 us each)
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent");
    if (lane == 0) last = atomicAdd(a.ticket, 1u) == gridDim.x * gridDim.y - 1;
  }
  __syncthreads();
  if (!last) return;
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  // (the fences order the others' stores before these loads; eight are under way at a time)
  float v = 0.f;
#pragma unroll 8
  for (uint32_t i = tid; i < gridDim.x * gridDim.y; i += TH) v += a.part_loss[i];
  v = block_sum<TH>(v, red);
  if (tid == 0) *a.loss = v * loss_factor(a);
  if (!a.cu_seqlens) return;
  // An expert's count over all sequences: one thread's, or several threads' where they are idle and have eight sequences each
  // (65535 sequences over 8 experts: offsets 2140 us from one thread each, 80 from 32; 64 experts 2230 and 590).
  const int shares = min(TH / a.experts, (a.batch + 7) / 8);
  int32_t* part = &csum[0][0];
  if (shares > 1) {
    const int step = shares * a.experts;
    int32_t s = 0;
    if (tid < step) {
#pragma unroll 8
      for (int64_t i = tid; i < (int64_t)a.batch * a.experts; i += step) s += a.counts[i];
    }
    part[tid] = s;
    __syncthreads();
  }
  offsets<TH>(a.cu_seqlens, a.experts, [&](int x) {
    int32_t s = 0;
    if (shares > 1) {
#pragma unroll 8
      for (int i = 0; i < shares; ++i) s += part[i * a.experts + x];
    } else {
#pragma unroll 8
      for (int y = 0; y < a.batch; ++y) s += a.counts[(int64_t)y * a.experts + x];
    }
    return s;
  }, (int32_t*)red);
}

// No tokens: zeros.
__global__ __launch_bounds__(kThreads) void balance_zero_kernel(const Forward a) {
  const int64_t n = (int64_t)a.batch * a.experts;
  const int64_t i0 = (int64_t)blockIdx.x * kThreads + threadIdx.x, step = (int64_t)gridDim.x * kThreads;
  for (int64_t i = i0; i < n; i += step) a.counts[i] = 0, a.probs[i] = 0.f;
  for (int64_t i = i0; i < a.batch; i += step) a.valid[i] = 0;
  if (a.cu_seqlens)
    for (int64_t i = i0; i <= a.experts; i += step) a.cu_seqlens[i] = 0;
  if (i0 == 0) *a.loss = 0.f;
}

struct Backward {
  int batch, tokens, experts, scores;
  float factor;  // coef * experts / (batch * k)
  const void* logits;
  const uint8_t* mask;
  const int32_t *counts, *valid;
  const float* grad;
  void* dlogits;
  int64_t ld, ldb, ldd, lddb;
  int per;
};
template <typename T, int G, int N, int SCORES, bool WHOLE>
__global__ __launch_bounds__(kThreads) void balance_backward_kernel(const Backward a) {
  constexpr int kGroups = kThreads / G, kAhead = N == 1 ? 4 : (N == 2 ? 2 : 1);
  const int tid = threadIdx.x, lane = tid & (G - 1), group = tid / G, b = blockIdx.y;
  const uint32_t t0 = blockIdx.x * (uint32_t)a.per, t1 = lesser((uint32_t)a.tokens, t0 + a.per);
  const uint8_t* mask = a.mask ? a.mask + (int64_t)b * a.tokens : nullptr;
  const T* logits = (const T*)a.logits + b * a.ldb;
  T* out = (T*)a.dlogits + b * a.lddb;
  Rows<T, G, N, WHOLE> rows[kAhead];
  bool use[kAhead];
  auto fetch = [&](uint32_t t) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const uint32_t at = lesser(t + u * kGroups, t1 - 1);
      use[u] = !mask || mask[at];
      rows[u].load(logits + at * a.ld, a.experts, lane);
    }
  };
  fetch(t0 + group);  // (under way while the weights are formed)
  const float n = (float)a.valid[b];
  const float factor = n > 0.f ? (a.grad ? *a.grad : 1.f) * (a.factor / n / n) : 0.f;
  // the counts less the smallest one, exact integers
  int32_t c[N][8], least = 0x7FFFFFFF;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int at = (i * G + lane) * 8 + e;
      c[i][e] = WHOLE || at < a.experts ? a.counts[(int64_t)b * a.experts + at] : 0x7FFFFFFF;
      least = min(least, c[i][e]);
    }
#pragma unroll
  for (int off = 1; off < G; off <<= 1) least = min(least, __shfl_xor(least, off));
  float w[N][8];
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) w[i][e] = WHOLE || (i * G + lane) * 8 + e < a.experts ? (float)(c[i][e] - least) * factor : 0.f;
  for (uint32_t t = t0 + group; t < t1;) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const uint32_t tt = t + u * kGroups;
      if (tt >= t1) continue;
      float d[N][8];
      if (use[u]) {
        float x[N][8], s[N][8], miss[N][8];
        rows[u].values(a.experts, lane, x);
        const float inv = row_scores<G, N, SCORES>(x, s, miss);
        float mean = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) mean = __builtin_fmaf(s[i][e], w[i][e], mean);
        mean = row_sum<G>(mean) * inv;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            d[i][e] = (s[i][e] * inv) * (w[i][e] - mean);
            if (SCORES == ROUTER_SIGMOID) d[i][e] *= miss[i][e];
          }
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) d[i][e] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < N; ++i) store_chunk<WHOLE>(out + tt * a.ldd, (i * G + lane) * 8, a.experts, pack<T>(d[i]));
    }
    t += kGroups * kAhead;
    if (t < t1) fetch(t);
  }
}

// Call f(G, N) with the lanes of a row and the chunks of a lane.
template <typename F>
void with_rows(int experts, F&& f) {
  using std::integral_constant;
  auto go = [&](auto g, auto n) { f(g, n); };
  const int chunks = (experts + 7) / 8;
  integral_constant<int, 1> one;
  if (chunks <= 1) go(one, one);
  else if (chunks <= 2) go(integral_constant<int, 2>{}, one);
  else if (chunks <= 4) go(integral_constant<int, 4>{}, one);
  else if (chunks <= 8) go(integral_constant<int, 8>{}, one);
  else if (chunks <= 16) go(integral_constant<int, 16>{}, one);
  else if (chunks <= 32) go(integral_constant<int, 32>{}, one);
  else if (chunks <= 64) go(integral_constant<int, 64>{}, one);
  else if (chunks <= 128) go(integral_constant<int, 64>{}, integral_constant<int, 2>{});
  else go(integral_constant<int, 64>{}, integral_constant<int, 4>{});
}
template <typename F>
void with_case(int scores, bool whole, F&& f) {
  std::integral_constant<int, ROUTER_SOFTMAX> softmax;
  std::integral_constant<int, ROUTER_SIGMOID> sigmoid;
  if (scores == ROUTER_SOFTMAX) whole ? f(softmax, std::true_type{}) : f(softmax, std::false_type{});
  else whole ? f(sigmoid, std::true_type{}) : f(sigmoid, std::false_type{});
}
int lanes_of(int experts) {
  int g = 1;
  while (g < 64 && g * 8 < experts) g *= 2;
  return g;
}

// How the tokens of a sequence are shared out: about `most` workgroups in all, of whole passes of `threads`.
struct Share {
  int per, wgs;
};
Share share(int32_t batch, int32_t tokens, int32_t experts, int32_t threads, int32_t most) {
  const int64_t pass = threads / lanes_of(experts);
  const int64_t want = std::max((int64_t)1, (int64_t)most / std::max(batch, 1));
  int64_t per = ((int64_t)tokens + want - 1) / want;
  per = (per + pass - 1) / pass * pass;
  per = std::max(per, pass);
  return Share{(int)std::min(per, (int64_t)0x7FFFFFFF), (int)(((int64_t)tokens + per - 1) / per)};
}
// Forward: as many threads a workgroup as the registers of a lane allow, since every workgroup leaves sums of all
// experts behind; backward: many small ones.
int forward_threads(int32_t experts) { return experts <= 512 ? 1024 : 256; }
// One workgroup's: 256 where they take their tokens at once, four a group of lanes.
int one_threads(int32_t tokens, int32_t experts) {
  return tokens <= 4 * kThreads / lanes_of(experts) ? kThreads : forward_threads(experts);
}
// Tokens that one workgroup takes instead of several and their join, a group of lanes: four, which are under way at once. (Over 8 to 512
// experts, fp32 and bf16, softmax and sigmoids: with two a group 6.0 to 8.5 us for 9.0 to 11.3, with four 7.5 to 10.6 for 8.8 to
// 11.4; with five a softmax takes as long either way or 8% less, sigmoids 3 to 13% longer; with six 1 to 27% longer.)
constexpr int kOne = 4;
Share forward_share(int32_t batch, int32_t tokens, int32_t experts) {
  if (batch == 1 && tokens <= kOne * forward_threads(experts) / lanes_of(experts))  // (one workgroup, and no join)
    return share(batch, tokens, experts, one_threads(tokens, experts), 1);
  return share(batch, tokens, experts, forward_threads(experts), 256);
}
Share backward_share(int32_t batch, int32_t tokens, int32_t experts) { return share(batch, tokens, experts, kThreads, 2048); }

// Of more sums than these the join takes 512 threads, else 256. (Forward passes over 8 to 2048 experts: of 8 to 64 sums 256 threads are
// 1 to 10% faster, 4096 tokens over 64 experts 9.4 us for 10.3; of 128 512 threads by 0 to 7%, 2048 over 512 10.9 for 11.6; of 256 by 8 to
// 17%, 8192 over 512 13.1 for 15.0.)
constexpr int kManySums = 64;

int64_t round16(int64_t v) { return (v + 15) / 16 * 16; }
struct Layout {
  int64_t p, c, n, loss, ticket, bytes;
};
Layout layout(int32_t batch, int32_t wgs, int32_t experts) {
  Layout l;
  const int64_t parts = (int64_t)batch * wgs;
  l.p = 0;
  l.c = l.p + round16(parts * experts * 4);
  l.n = l.c + round16(parts * experts * 4);
  l.loss = l.n + round16(parts * 4);
  l.ticket = l.loss + round16((int64_t)batch * ((experts + 63) / 64) * 4);
  l.bytes = l.ticket + 16;
  return l;
}

gemm_status check_sizes(const char* fn, int32_t batch, int32_t tokens, int32_t experts, int32_t k, int32_t type, int32_t scores) {
  if (batch < 0 || tokens < 0) return fail(GEMM_ERR_INVALID_ARG, "%s: negative size", fn);
  if (experts < 1 || k < 1 || k > experts) return fail(GEMM_ERR_INVALID_ARG, "%s: 1 <= k <= experts expected", fn);
  if (experts > kMaxExperts) return fail(GEMM_ERR_UNSUPPORTED, "%s: more than %d experts", fn, kMaxExperts);
  if (batch > 65535) return fail(GEMM_ERR_UNSUPPORTED, "%s: more than 65535 sequences", fn);
  if ((int64_t)batch * tokens > 0x7FFFFFFF / k) return fail(GEMM_ERR_UNSUPPORTED, "%s: 2^31 choices or more", fn);
  if (type != GEMM_DT_F16 && type != GEMM_DT_BF16 && type != GEMM_DT_F32) return fail(GEMM_ERR_INVALID_ARG, "%s: the logits must be F16, BF16 or F32", fn);
  if (scores != ROUTER_SOFTMAX && scores != ROUTER_SIGMOID) return fail(GEMM_ERR_INVALID_ARG, "%s: unknown scores %d", fn, scores);
  return GEMM_OK;
}
gemm_status check_logits(const char* fn, const char* name, int32_t batch, int32_t tokens, int32_t experts, int32_t type, const void* p,
                         int64_t ld, int64_t ldb) {
  const int64_t most = (int64_t)1 << 48;
  if (ld < 0 || ld > most || ldb < 0 || ldb > most) return fail(GEMM_ERR_UNSUPPORTED, "%s: strides of %s outside [0, 2^48]", fn, name);
  if (tokens > 1 && ld < experts) return fail(GEMM_ERR_INVALID_ARG, "%s: rows of %s overlap", fn, name);
  const __int128 l = ld, b = ldb;
  const bool apart = b >= (tokens - 1) * l + experts, alternate = ldb >= experts && l >= (batch - 1) * b + experts;
  if (batch > 1 && tokens > 0 && !apart && !(alternate && tokens > 1)) return fail(GEMM_ERR_INVALID_ARG, "%s: sequences of %s overlap", fn, name);
  if (!p) return fail(GEMM_ERR_INVALID_ARG, "%s: NULL %s", fn, name);
  if ((uintptr_t)p % (type == GEMM_DT_F32 ? 4 : 2)) return fail(GEMM_ERR_ALIGNMENT, "%s: %s not aligned to its elements", fn, name);
  return GEMM_OK;
}
gemm_status launched(const char* fn) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(GEMM_ERR_HIP, "%s launch: %s", fn, hipGetErrorString(e));
  return GEMM_OK;
}

}  // namespace
}  // namespace gep

using namespace gep;

extern "C" {

int64_t router_balance_workspace(int32_t batch, int32_t tokens, int32_t experts) {
  if (batch < 0 || tokens < 0 || experts < 1 || experts > kMaxExperts || batch > 65535 || (int64_t)batch * tokens > 0x7FFFFFFF) return -1;
  return layout(batch, forward_share(batch, tokens, experts).wgs, experts).bytes;
}

gemm_status router_balance(const router_balance_args* a, void* stream) {
  const char* fn = "router_balance";
  if (!a) return fail(GEMM_ERR_INVALID_ARG, "%s: NULL args", fn);
  gemm_status st = check_sizes(fn, a->batch, a->tokens, a->experts, a->k, a->type, a->scores);
  if (st != GEMM_OK) return st;
  if (a->index_bytes != 4 && a->index_bytes != 8) return fail(GEMM_ERR_INVALID_ARG, "%s: indices of 4 or 8 bytes expected", fn);
  const bool empty = a->batch == 0 || a->tokens == 0;
  if (!empty) {
    st = check_logits(fn, "logits", a->batch, a->tokens, a->experts, a->type, a->logits, a->logits_ld, a->logits_batch);
    if (st != GEMM_OK) return st;
    if (!a->chosen) return fail(GEMM_ERR_INVALID_ARG, "%s: NULL chosen", fn);
    if ((uintptr_t)a->chosen % a->index_bytes) return fail(GEMM_ERR_ALIGNMENT, "%s: chosen not aligned to its elements", fn);
  }
  if (!a->loss || (a->batch > 0 && (!a->counts || !a->valid || !a->probs))) return fail(GEMM_ERR_INVALID_ARG, "%s: NULL counts, valid, probs or loss", fn);
  for (const void* p : {(const void*)a->counts, (const void*)a->valid, (const void*)a->cu_seqlens, (const void*)a->probs, (const void*)a->loss})
    if ((uintptr_t)p & 3) return fail(GEMM_ERR_ALIGNMENT, "%s: outputs not 4-byte aligned", fn);
  const Share sh = forward_share(a->batch, a->tokens, a->experts);
  const Layout l = layout(a->batch, sh.wgs, a->experts);
  if (!a->workspace || a->workspace_bytes < l.bytes) return fail(GEMM_ERR_INVALID_ARG, "%s: workspace of %lld bytes expected", fn, (long long)l.bytes);
  if ((uintptr_t)a->workspace & 15) return fail(GEMM_ERR_ALIGNMENT, "%s: workspace not 16-byte aligned", fn);
  clear_error();
  char* w = (char*)a->workspace;
  Forward f{a->batch, a->tokens, a->experts, a->k, a->scores, a->index_bytes, a->coef, a->logits, a->chosen, a->mask,
            a->counts, a->valid, a->cu_seqlens, a->probs, a->loss, a->logits_ld, a->logits_batch, sh.per, sh.wgs,
            (float*)(w + l.p), (int32_t*)(w + l.c), (int32_t*)(w + l.n), (float*)(w + l.loss), (uint32_t*)(w + l.ticket)};
  hipStream_t s = (hipStream_t)stream;
  if (empty) {
    balance_zero_kernel<<<256, kThreads, 0, s>>>(f);
    return launched(fn);
  }
  const bool one = a->batch == 1 && sh.wgs == 1;
  with_type(a->type, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    with_rows(a->experts, [&](auto g, auto n) {
      constexpr int G = decltype(g)::value, N = decltype(n)::value, TH = N == 1 ? 1024 : 256;
      const dim3 grid((unsigned)sh.wgs, (unsigned)a->batch);
      auto go = [&](auto scores, auto whole) {
        constexpr int S = decltype(scores)::value;
        constexpr bool W = decltype(whole)::value;
        if (one && one_threads(a->tokens, a->experts) == kThreads) balance_kernel<T, G, N, S, W, true, kThreads><<<grid, kThreads, 0, s>>>(f);
        else if (one) balance_kernel<T, G, N, S, W, true, TH><<<grid, TH, 0, s>>>(f);
        else balance_kernel<T, G, N, S, W, false, TH><<<grid, TH, 0, s>>>(f);
      };
      with_case(a->scores, a->experts == 8 * G * N, go);
    });
  });
  if (!one) {
    const dim3 grid((unsigned)(a->experts + 63) / 64, (unsigned)a->batch);
    if (sh.wgs > kManySums) balance_join_kernel<512><<<grid, 512, 0, s>>>(f);
    else balance_join_kernel<256><<<grid, 256, 0, s>>>(f);
  }
  return launched(fn);
}

gemm_status router_balance_backward(const router_balance_backward_args* a, void* stream) {
  const char* fn = "router_balance_backward";
  if (!a) return fail(GEMM_ERR_INVALID_ARG, "%s: NULL args", fn);
  gemm_status st = check_sizes(fn, a->batch, a->tokens, a->experts, a->k, a->type, a->scores);
  if (st != GEMM_OK) return st;
  if (a->batch == 0 || a->tokens == 0) { clear_error(); return GEMM_OK; }
  st = check_logits(fn, "logits", a->batch, a->tokens, a->experts, a->type, a->logits, a->logits_ld, a->logits_batch);
  if (st == GEMM_OK) st = check_logits(fn, "dlogits", a->batch, a->tokens, a->experts, a->type, a->dlogits, a->dlogits_ld, a->dlogits_batch);
  if (st != GEMM_OK) return st;
  if (!a->counts || !a->valid) return fail(GEMM_ERR_INVALID_ARG, "%s: NULL counts or valid", fn);
  for (const void* p : {(const void*)a->counts, (const void*)a->valid, (const void*)a->grad})
    if ((uintptr_t)p & 3) return fail(GEMM_ERR_ALIGNMENT, "%s: counts, valid or grad not 4-byte aligned", fn);
  if (a->dlogits == a->logits && ((a->tokens > 1 && a->dlogits_ld != a->logits_ld) || (a->batch > 1 && a->dlogits_batch != a->logits_batch)))
    return fail(GEMM_ERR_INVALID_ARG, "%s: dlogits in the place of the logits needs their strides", fn);
  clear_error();
  const Share sh = backward_share(a->batch, a->tokens, a->experts);
  const Backward f{a->batch, a->tokens, a->experts, a->scores, a->coef * (float)a->experts / ((float)a->batch * (float)a->k),
                   a->logits, a->mask, a->counts, a->valid, a->grad, a->dlogits, a->logits_ld, a->logits_batch,
                   a->dlogits_ld, a->dlogits_batch, sh.per};
  with_type(a->type, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    with_rows(a->experts, [&](auto g, auto n) {
      constexpr int G = decltype(g)::value, N = decltype(n)::value;
      const dim3 grid((unsigned)sh.wgs, (unsigned)a->batch);
      with_case(a->scores, a->experts == 8 * G * N, [&](auto scores, auto whole) {
        balance_backward_kernel<T, G, N, decltype(scores)::value, decltype(whole)::value><<<grid, kThreads, 0, (hipStream_t)stream>>>(f);
      });
    });
  });
  return launched(fn);
}

}  // extern "C"
