// layer_norm.cuh -- layer norm over the hidden states of the sequence shards,
// forward and backward.
//
// Rows are tokens of the sequence-sharded hidden states [P][B][Nl][C]; token
// r*Nl + n of sample b is row (r*B + b)*Nl + n, and tokens at or past N are
// padding.  With xh = (x - mean) * rstd, rstd = 1 / sqrt(var + eps):
//   forward    y  = xh * w + b
//   backward   g  = dy * w,  dx = rstd * (g - mean(g) - xh * mean(g * xh)),
//              dw = sum over rows of dy * xh,  db = sum over rows of dy
// w and b are one row for all tokens, or one row per sample (the modulation
// of a diffusion transformer block).  All arithmetic is fp32 on bf16 inputs;
// every output is rounded once.
//
// Both passes are bound by memory: the forward moves 4 bytes an element, the
// backward 6.  At the rate of the memory an SM has 22 (33) instructions for an
// element, so what is done once per thread and row must be spread over many
// elements: a team of warps takes a row, each thread V vectors of 8 columns (up
// to 6 forward, 4 backward, where both gradient sums of every column stay in
// registers).  One vector a thread and a block a row was bound by instructions:
// 547 us forward and 644 us backward at 75,600 x 5,120, against 248 and 422.
// The parameters lie in shared memory in fp32.  Each thread copies its own
// columns of the next three rows into shared memory (cp.async, which needs no
// synchronisation), so that some 100 KB an SM are in flight.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>

#include "permute.cuh"
#include "sm100.cuh"

namespace sp {

struct LnParams {
  const uint4 *x;          // [P][B][Nl][C] bf16
  const uint4 *dy;         // backward
  uint4 *y;                // forward: y; backward: dx
  const void *weight, *bias;  // [C] or [B][C], or null
  float *mean, *rstd;      // [P][B][Nl], or null (forward)
  const float *mean_in, *rstd_in;  // backward
  float *partial;          // backward: [groups][blocks][2][C]
  void *dweight, *dbias;   // backward, or null
  int32_t C8;              // C / 8
  int32_t P, B, Nl, N;
  FastDiv div_n, div_nl;
  int32_t per_sample;      // w and b are [B][C]
  int32_t linear;          // B or P is 1: row i of the valid ones is row i of memory
  int32_t param_f32;       // fp32 parameters (and their gradients), else bf16
  float eps, c, inv_c;     // c: hidden elements
};

constexpr int kLnFwdVec = 6, kLnBwdVec = 4;  // vectors of a thread at most
constexpr int kLnStages = 4;                 // rows of a team's ring
// Warps of a block at most and blocks of an SM, by registers: 128 a thread (64
// with few vectors) forward; 80, 128, 168 or 200 backward, where more warps with
// fewer registers were slower (5,120 columns, four vectors a thread: 420 us with
// 10 warps' registers, 467 with 12 warps'; two vectors and 20 warps 530).
__host__ __device__ constexpr int ln_max_warps(int V, bool backward) {
  return !backward || V == 2 ? 16 : V == 4 ? 10 : 12;
}
__host__ __device__ constexpr int ln_blocks_per_sm(int V, bool backward) {
  return V <= (backward ? 1 : 2) ? 2 : 1;
}

__device__ __forceinline__ void ln_unpack(const uint4 &v, float *f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// Parameters 8c .. 8c + 7 of parameter row `row`.
__device__ __forceinline__ void ln_param8(const void *base, int f32, int64_t row, int C8, int c,
                                          float *f) {
  const int64_t i = row * C8 + c;
  if (f32) {
    const float4 *p = static_cast<const float4 *>(base) + 2 * i;
    const float4 a = __ldg(p), b = __ldg(p + 1);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  } else {
    ln_unpack(__ldg(static_cast<const uint4 *>(base) + i), f);
  }
}

// Rows of one group of a pass, in the order of the logical sequence (so that
// sums do not depend on P): i-th valid row of all samples, or of sample `g`
// when every sample has its own parameters.
__device__ __forceinline__ int64_t ln_row(const LnParams &p, uint32_t g, uint32_t i) {
  if (p.linear) return static_cast<int64_t>(p.per_sample ? g * p.N : 0u) + i;
  const uint32_t b = p.per_sample ? g : fdiv(i, p.div_n);
  const uint32_t t = p.per_sample ? i : i - b * static_cast<uint32_t>(p.N);
  const uint32_t r = fdiv(t, p.div_nl);
  return static_cast<int64_t>(r * p.B + b) * p.Nl + (t - r * p.Nl);
}

// Sums of M values over a team of tn threads, in a fixed order; every thread gets
// them.  kSub: tn is at most 32, a power of two; else whole warps (through the
// team's 12 slots of M rows of `red`, zero past the last warp, which the team's
// previous sums do not use).
constexpr int kLnTeamSlots = 12, kLnRed = 8 * kLnTeamSlots;  // (teams of several warps: 8 at most)

template <int M, bool kSub>
__device__ __forceinline__ void team_sums(float (&v)[M], float (*red)[kLnRed], int team, int tn) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
    if (!kSub || d < tn) {
#pragma unroll
      for (int m = 0; m < M; ++m) v[m] += __shfl_xor_sync(0xffffffffu, v[m], d);
    }
  if (kSub || tn == 32) return;
  const int base = team * kLnTeamSlots;
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int m = 0; m < M; ++m) red[m][base + ((threadIdx.x - team * tn) >> 5)] = v[m];
  }
  asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(tn) : "memory");
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const float4 *t = reinterpret_cast<const float4 *>(&red[m][base]);
    const float4 a = t[0], b = t[1], c = t[2];
    v[m] = ((a.x + a.y) + (a.z + a.w)) + (((b.x + b.y) + (b.z + b.w)) + ((c.x + c.y) + (c.z + c.w)));
  }
}

__device__ __forceinline__ void clear_red(float *red) {
  for (int k = threadIdx.x; k < 4 * kLnRed; k += blockDim.x) red[k] = 0.f;
}

// Parameter row `row` into shared memory in fp32; `none` where there is none.
__device__ __forceinline__ void ln_stage_params(const LnParams &p, const void *src, float none,
                                                int64_t row, float4 *dst) {
  for (int c = threadIdx.x; c < p.C8; c += blockDim.x) {
    float t[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = none;
    if (src != nullptr) ln_param8(src, p.param_f32, row, p.C8, c, t);
    // the halves of a vector apart, so that consecutive lanes read
    // consecutive 16-byte words
    dst[c] = make_float4(t[0], t[1], t[2], t[3]);
    dst[p.C8 + c] = make_float4(t[4], t[5], t[6], t[7]);
  }
}

// Columns as four pairs of fp32.
__device__ __forceinline__ void ln_unpack2(const uint4 &v, uint64_t *f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = f2_pack_bits(w[i] << 16, w[i] & 0xffff0000u);
}
__device__ __forceinline__ uint4 ln_pack2(const uint64_t *f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    f2_unpack(f[i], lo, hi);
    w[i] = pack_bf16x2(lo, hi);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void ln_load_params(const float4 *src, int C8, int c, uint64_t *f) {
  const ulonglong2 a = reinterpret_cast<const ulonglong2 *>(src)[c];
  const ulonglong2 b = reinterpret_cast<const ulonglong2 *>(src)[C8 + c];
  f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
}
__device__ __forceinline__ float f2_sum(uint64_t v) {
  float lo, hi;
  f2_unpack(v, lo, hi);
  return lo + hi;
}

// Zeroes rows past N of y (and of the statistics), shared among all blocks.
__device__ __forceinline__ void ln_zero_padding(const LnParams &p, bool stats) {
  const int64_t pad = static_cast<int64_t>(p.P) * p.Nl - p.N;
  const int64_t nblk = static_cast<int64_t>(gridDim.x) * gridDim.y;
  for (int64_t j = static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x; j < pad * p.B;
       j += nblk) {
    const int b = static_cast<int>(j / pad);
    const int t = static_cast<int>(p.N + (j - b * pad));
    const int r = t / p.Nl;
    const int64_t row = (static_cast<int64_t>(r) * p.B + b) * p.Nl + (t - r * p.Nl);
    for (int c = threadIdx.x; c < p.C8; c += blockDim.x)
      p.y[row * p.C8 + c] = make_uint4(0u, 0u, 0u, 0u);
    if (stats && threadIdx.x == 0) {
      if (p.mean != nullptr) p.mean[row] = 0.f;
      if (p.rstd != nullptr) p.rstd[row] = 0.f;
    }
  }
}

// Forward.  The variance is summed around the mean in a second sweep over the
// registers, so that a large mean costs no digits.  Team i takes rows i,
// i + teams, ... of group blockIdx.y.
template <int V>
__global__ void __launch_bounds__(32 * ln_max_warps(V, false), ln_blocks_per_sm(V, false))
layer_norm_kernel(const LnParams p, int tn) {
  constexpr int K = kLnStages;
  constexpr bool kSub = V == 1;
  __shared__ __align__(16) float red[4][kLnRed];
  extern __shared__ __align__(16) uint8_t ln_smem[];
  float4 *const sw = reinterpret_cast<float4 *>(ln_smem), *const sb = sw + 2 * p.C8;
  const int team = threadIdx.x / tn, tt = threadIdx.x - team * tn;
  const uint32_t sub = kSub ? (threadIdx.x & 31) / tn : 0;  // team of the warp
  const uint32_t g = blockIdx.y;
  const uint32_t nrows = p.per_sample ? p.N : p.B * p.N;  // below 2^31
  const uint32_t block_teams = blockDim.x / tn, teams = gridDim.x * block_teams;
  const uint32_t ring = smem_u32(sb + 2 * p.C8) + threadIdx.x * 16;
  const uint32_t vec = blockDim.x * 16, line = V * vec;  // bytes between vectors, rows
  auto fetch = [&](int s, uint32_t i) {
    if (i < nrows) {
      const uint4 *x = p.x + ln_row(p, g, i) * p.C8;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (tt + v * tn < p.C8) cp_async16(ring + s * line + v * vec, x + tt + v * tn, 16);
    }
    cp_async_commit();
  };
  uint32_t i = blockIdx.x * block_teams + team;
#pragma unroll
  for (int s = 0; s < K - 1; ++s) fetch(s, i + s * teams);
  ln_stage_params(p, p.weight, 1.f, p.per_sample ? g : 0, sw);
  ln_stage_params(p, p.bias, 0.f, p.per_sample ? g : 0, sb);
  clear_red(red[0]);
  __syncthreads();
  int s = 0, ph = 0;
  for (; i - sub < nrows; i += teams, ph ^= 2) {  // (the same steps in all lanes)
    cp_async_wait_group<K - 2>();
    const bool row_in = !kSub || i < nrows;
    uint64_t f[V][4];
    uint64_t acc = f2_pack(0.f, 0.f), acc2 = acc;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      ln_unpack2(row_in && tt + v * tn < p.C8 ? ld_shared_v4(ring + s * line + v * vec)
                                              : make_uint4(0u, 0u, 0u, 0u), f[v]);
      acc = f2_add(acc, f2_add(f[v][0], f[v][1]));
      acc2 = f2_add(acc2, f2_add(f[v][2], f[v][3]));
    }
    // the stage read in the last step takes the row K - 1 steps ahead
    fetch(s == 0 ? K - 1 : s - 1, i + (K - 1) * teams);
    s = s + 1 == K ? 0 : s + 1;
    float sum[1] = {f2_sum(f2_add(acc, acc2))};
    team_sums<1, kSub>(sum, red + ph, team, tn);
    // (a quotient: times the rounded 1 / C the mean of a constant row is off,
    // and its xh = (x - mean) / sqrt(eps) with it: 0.06 for 1,000 in 328 columns)
    const float mean = sum[0] / p.c;
    const uint64_t nmean2 = f2_pack(-mean, -mean);
    acc = acc2 = f2_pack(0.f, 0.f);
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int e = 0; e < 4; ++e) f[v][e] = f2_add(f[v][e], nmean2);
      if (tt + v * tn < p.C8) {
        acc = f2_fma(f[v][0], f[v][0], f2_fma(f[v][1], f[v][1], acc));
        acc2 = f2_fma(f[v][2], f[v][2], f2_fma(f[v][3], f[v][3], acc2));
      }
    }
    sum[0] = f2_sum(f2_add(acc, acc2));
    team_sums<1, kSub>(sum, red + ph + 1, team, tn);
    if (!row_in) continue;
    const float rstd = 1.0f / sqrtf(sum[0] * p.inv_c + p.eps);
    const uint64_t rstd2 = f2_pack(rstd, rstd);
    const int64_t row = ln_row(p, g, i);
    if (tt == 0) {
      if (p.mean != nullptr) p.mean[row] = mean;
      if (p.rstd != nullptr) p.rstd[row] = rstd;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = tt + v * tn;
      if (c < p.C8) {
        uint64_t w[4], b[4];
        ln_load_params(sw, p.C8, c, w);
        ln_load_params(sb, p.C8, c, b);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[v][e] = f2_fma(f2_mul(f[v][e], rstd2), w[e], b[e]);
        p.y[row * p.C8 + c] = ln_pack2(f[v]);
      }
    }
  }
  ln_zero_padding(p, true);
}

// Backward.  Each team keeps the gradient sums of its rows; a block's teams are
// added in order, and the sums leave as one partial row per block, which
// layer_norm_grad_kernel adds in block order: the result depends on no race.
template <int V, bool kGrad>
__global__ void __launch_bounds__(32 * ln_max_warps(V, true), ln_blocks_per_sm(V, true))
layer_norm_backward_kernel(const LnParams p, int tn) {
  constexpr int K = kLnStages;
  constexpr bool kSub = V == 1;
  __shared__ __align__(16) float red[4][kLnRed];
  extern __shared__ __align__(16) uint8_t ln_smem[];
  // (the kernel that adds the partial rows may take its place meanwhile)
  asm volatile("griddepcontrol.launch_dependents;");
  float4 *const sw = reinterpret_cast<float4 *>(ln_smem);
  const int team = threadIdx.x / tn, tt = threadIdx.x - team * tn;
  const uint32_t sub = kSub ? (threadIdx.x & 31) / tn : 0;  // team of the warp
  const uint32_t g = blockIdx.y;
  const uint32_t nrows = p.per_sample ? p.N : p.B * p.N;  // below 2^31
  const uint32_t block_teams = blockDim.x / tn, teams = gridDim.x * block_teams;
  const uint32_t ring = smem_u32(sw + 2 * p.C8) + threadIdx.x * 16;
  const uint32_t vec = blockDim.x * 16, line = 2 * V * vec;
  auto fetch = [&](int s, uint32_t i) {
    if (i < nrows) {
      const int64_t off = ln_row(p, g, i) * p.C8;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = tt + v * tn;
        if (c < p.C8) {
          cp_async16(ring + s * line + 2 * v * vec, p.x + off + c, 16);
          cp_async16(ring + s * line + (2 * v + 1) * vec, p.dy + off + c, 16);
        }
      }
    }
    cp_async_commit();
  };
  uint32_t i = blockIdx.x * block_teams + team;
#pragma unroll
  for (int s = 0; s < K - 1; ++s) fetch(s, i + s * teams);
  int64_t row = 0;
  float rstd = 0.f, mean = 0.f;  // of the next row
  auto stats = [&](uint32_t j) {
    mean = rstd = 0.f;
    if (j < nrows) {
      row = ln_row(p, g, j);
      mean = __ldg(p.mean_in + row);
      rstd = __ldg(p.rstd_in + row);
    }
  };
  stats(i);
  ln_stage_params(p, p.weight, 1.f, p.per_sample ? g : 0, sw);
  clear_red(red[0]);
  __syncthreads();
  const uint64_t zero2 = f2_pack(0.f, 0.f);
  uint64_t dw[V][4], db[V][4];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int e = 0; e < 4; ++e) dw[v][e] = db[v][e] = zero2;
  int s = 0, ph = 0;
  for (; i - sub < nrows; i += teams, ph ^= 2) {  // (the same steps in all lanes)
    cp_async_wait_group<K - 2>();
    const bool row_in = !kSub || i < nrows;
    // xh = (x - mean) rstd, in this order in both sweeps: x rstd - mean rstd
    // would be off by the product's rounding, |mean| rstd 2^-24 (0.4 in a constant
    // row of 9,984), where x - mean is exact
    const float rs = rstd;
    const uint64_t rstd2 = f2_pack(rs, rs), nmean2 = f2_pack(-mean, -mean);
    uint4 *dx = p.y + row * p.C8;
    // g stays in registers for the second sweep, or dy packed when V = 4
    // (kept, its 16 registers spilled)
    constexpr bool kKeep = V < 4;
    uint4 xp[V], dk[kKeep ? 1 : V];
    uint64_t gk[kKeep ? V : 1][4];
    uint64_t a1 = zero2, a2 = zero2;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = tt + v * tn;
      const bool in = row_in && c < p.C8;
      // past the row, where only a last vector can be, x - mean is 0 as dy is: 0
      // times -mean rstd is NaN where that product is past fp32 (a row of 1e36)
      const uint64_t center2 = v < V - 1 || in ? nmean2 : zero2;
      uint4 dp = make_uint4(0u, 0u, 0u, 0u);
      xp[v] = dp;
      if (in) {
        xp[v] = ld_shared_v4(ring + s * line + 2 * v * vec);
        dp = ld_shared_v4(ring + s * line + (2 * v + 1) * vec);
      }
      uint64_t x[4], d[4], w[4];
      ln_unpack2(xp[v], x);
      ln_unpack2(dp, d);
      if (!kKeep) dk[kKeep ? 0 : v] = dp;
      ln_load_params(sw, p.C8, in ? c : 0, w);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint64_t xh = f2_mul(f2_add(x[e], center2), rstd2);
        const uint64_t gv = f2_mul(d[e], w[e]);   // (0 past the row)
        if (kKeep) gk[kKeep ? v : 0][e] = gv;
        a1 = f2_add(a1, gv);
        a2 = f2_fma(gv, xh, a2);
        if (kGrad) {
          dw[v][e] = f2_fma(d[e], xh, dw[v][e]);
          db[v][e] = f2_add(db[v][e], d[e]);
        }
      }
    }
    fetch(s == 0 ? K - 1 : s - 1, i + (K - 1) * teams);
    s = s + 1 == K ? 0 : s + 1;
    stats(i + teams);  // in flight across the reduction
    float sums[2] = {f2_sum(a1), f2_sum(a2)};
    team_sums<2, kSub>(sums, red + ph, team, tn);
    if (!row_in) continue;
    // dx = rstd (g - s1 - xh s2) = g rstd + ((x - mean) a + b)
    const float s1 = sums[0] * p.inv_c, s2 = sums[1] * p.inv_c;
    const float a = -rs * rs * s2, bb = -rs * s1;
    const uint64_t aa2 = f2_pack(a, a), bb2 = f2_pack(bb, bb);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = tt + v * tn;
      if (c < p.C8) {
        uint64_t x[4], gv[4];
        ln_unpack2(xp[v], x);
        if (!kKeep) {
          uint64_t w[4];
          ln_unpack2(dk[kKeep ? 0 : v], gv);
          ln_load_params(sw, p.C8, c, w);
#pragma unroll
          for (int e = 0; e < 4; ++e) gv[e] = f2_mul(gv[e], w[e]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[e] = f2_fma(kKeep ? gk[kKeep ? v : 0][e] : gv[e], rstd2,
                        f2_fma(f2_add(x[e], nmean2), aa2, bb2));
        dx[c] = ln_pack2(x);
      }
    }
  }
  if (kGrad) {
    // the warps' teams, then the block's warps (or larger teams) in order,
    // through the ring: [dw, db][half][C8] float4
    cp_async_wait_group<0>();
    if (kSub)
      for (int d = tn; d < 32; d <<= 1)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          dw[0][e] = f2_add(dw[0][e], __shfl_xor_sync(0xffffffffu, dw[0][e], d));
          db[0][e] = f2_add(db[0][e], __shfl_xor_sync(0xffffffffu, db[0][e], d));
        }
    const int turns = blockDim.x / max(tn, 32), turn = kSub ? threadIdx.x >> 5 : team;
    ulonglong2 *acc = reinterpret_cast<ulonglong2 *>(sw + 2 * p.C8);
    for (int k = 0; k < turns; ++k) {
      __syncthreads();
      if (turn != k || sub != 0) continue;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = tt + v * tn;
        if (c >= p.C8) continue;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const uint64_t *a = (h < 2 ? dw[v] : db[v]) + 2 * (h & 1);
          ulonglong2 t = make_ulonglong2(a[0], a[1]);
          ulonglong2 *slot = acc + h * p.C8 + c;
          if (k > 0) {
            const ulonglong2 o = *slot;
            t = make_ulonglong2(f2_add(o.x, t.x), f2_add(o.y, t.y));
          }
          *slot = t;
        }
      }
    }
    __syncthreads();
    float4 *out = reinterpret_cast<float4 *>(p.partial) +
                  (static_cast<int64_t>(g) * gridDim.x + blockIdx.x) * 4 * p.C8;
    const float4 *sums = sw + 2 * p.C8;
    for (int c = threadIdx.x; c < p.C8; c += blockDim.x)
#pragma unroll
      for (int h = 0; h < 4; ++h) out[(h >> 1) * 2 * p.C8 + 2 * c + (h & 1)] = sums[h * p.C8 + c];
  }
  ln_zero_padding(p, false);
}

// Sums the blocks' partial rows [groups][blocks][2][C] in a fixed order: thread
// (x, y) adds columns 4x .. 4x + 3 of partial rows y, y + 32, ..., then the 32
// sums of a column are added in order.  blockIdx.y is the group, blockIdx.z 0
// for dw, 1 for db; 8 x 32 threads.
constexpr int kLnGradRows = 32;
__global__ void __launch_bounds__(256) layer_norm_grad_kernel(const LnParams p, int blocks) {
  __shared__ float4 red[kLnGradRows][8];
  const int x = threadIdx.x & 7, y = threadIdx.x >> 3;
  const int64_t C4 = 2ll * p.C8;  // float4 of a row
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 8 + x;
  const int64_t g = blockIdx.y;
  const int which = blockIdx.z;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (col < C4) {
    const float4 *src = reinterpret_cast<const float4 *>(p.partial) + (g * blocks * 2 + which) * C4 + col;
#pragma unroll 8
    for (int k = y; k < blocks; k += kLnGradRows) {
      const float4 v = src[static_cast<int64_t>(k) * 2 * C4];
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
  }
  red[y][x] = s;
  __syncthreads();
  if (y == 0 && col < C4) {
#pragma unroll
    for (int k = 1; k < kLnGradRows; ++k) {
      const float4 v = red[k][x];
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    void *out = which ? p.dbias : p.dweight;
    if (p.param_f32)
      static_cast<float4 *>(out)[g * C4 + col] = s;
    else
      static_cast<uint2 *>(out)[g * C4 + col] =
          make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
  }
}

}  // namespace sp
