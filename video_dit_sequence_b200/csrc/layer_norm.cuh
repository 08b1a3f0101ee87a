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
// backward 6.  So each element is read once and kept in registers as it came
// (packed bf16) for the statistics and the result.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>

namespace sp {

constexpr int kLnMaxHidden = 8192;

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
  int64_t rows;            // P * B * Nl
  int32_t per_sample;      // w and b are [B][C]
  int32_t param_f32;       // fp32 parameters (and their gradients), else bf16
  float eps, inv_c;
};

// The input rows are read once: past L1, so that the parameters stay there.
__device__ __forceinline__ uint4 ln_load(const uint4 *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void ln_unpack(const uint4 &v, float *f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 ln_pack(const float *f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
  return make_uint4(w[0], w[1], w[2], w[3]);
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

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

constexpr int kLnFwdWarps = 4;

// One warp per row; lane l holds vectors l, l + 32, ... (V of them at most)
// of 8 elements.  The variance is summed around the mean in a second sweep
// over the registers, so that a large mean costs no digits.
template <int V>
__global__ void __launch_bounds__(32 * kLnFwdWarps) layer_norm_kernel(const LnParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kLnFwdWarps + (threadIdx.x >> 5);
  if (row >= p.rows) return;
  const int64_t slot = row / p.Nl;
  const int n = static_cast<int>(row - slot * p.Nl);
  const int r = static_cast<int>(slot / p.B), b = static_cast<int>(slot - static_cast<int64_t>(r) * p.B);
  uint4 *y = p.y + row * p.C8;
  if (static_cast<int64_t>(r) * p.Nl + n >= p.N) {  // padding: zeros, and statistics of 0
    for (int c = lane; c < p.C8; c += 32) y[c] = make_uint4(0u, 0u, 0u, 0u);
    if (lane == 0) {
      if (p.mean != nullptr) p.mean[row] = 0.f;
      if (p.rstd != nullptr) p.rstd[row] = 0.f;
    }
    return;
  }
  const uint4 *x = p.x + row * p.C8;
  uint4 v[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = lane + 32 * i;
    v[i] = c < p.C8 ? ln_load(x + c) : make_uint4(0u, 0u, 0u, 0u);
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float f[8];
    ln_unpack(v[i], f);
    s += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
  }
  const float mean = warp_sum(s) * p.inv_c;
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (lane + 32 * i < p.C8) {
      float f[8];
      ln_unpack(v[i], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = f[e] - mean;
        q = fmaf(d, d, q);
      }
    }
  }
  const float rstd = 1.0f / sqrtf(warp_sum(q) * p.inv_c + p.eps);
  if (lane == 0) {
    if (p.mean != nullptr) p.mean[row] = mean;
    if (p.rstd != nullptr) p.rstd[row] = rstd;
  }
  const int64_t prow = p.per_sample ? b : 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = lane + 32 * i;
    if (c < p.C8) {
      float f[8], t[8];
      ln_unpack(v[i], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = (f[e] - mean) * rstd;
      if (p.weight != nullptr) {
        ln_param8(p.weight, p.param_f32, prow, p.C8, c, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= t[e];
      }
      if (p.bias != nullptr) {
        ln_param8(p.bias, p.param_f32, prow, p.C8, c, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] += t[e];
      }
      y[c] = ln_pack(f);
    }
  }
}

// Rows of one group of the backward pass, in the order of the logical
// sequence (so that sums do not depend on P): i-th valid row of all samples,
// or of sample `g` when every sample has its own parameters.
__device__ __forceinline__ int64_t ln_row(const LnParams &p, int g, int64_t i) {
  int b = g;
  int t;
  if (p.per_sample) {
    t = static_cast<int>(i);
  } else {
    b = static_cast<int>(i / p.N);
    t = static_cast<int>(i - static_cast<int64_t>(b) * p.N);
  }
  const int r = t / p.Nl;
  return (static_cast<int64_t>(r) * p.B + b) * p.Nl + (t - r * p.Nl);
}

// Backward: a block takes rows blockIdx.x, blockIdx.x + gridDim.x, ... of
// group blockIdx.y; thread t holds V vectors of 8 columns (t, t + blockDim.x)
// of every row, with their weights and their two gradient sums in registers,
// so that the rows are read once for dx and for the parameters' gradients.
// The sums leave as one partial row per block, which layer_norm_grad_kernel
// adds in block order: the result depends on no race.
template <int V, bool kGrad>
__global__ void __launch_bounds__(512) layer_norm_backward_kernel(const LnParams p) {
  __shared__ float2 red[2][16];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nwarps = blockDim.x >> 5;
  const int g = blockIdx.y;
  const int64_t nrows = p.per_sample ? p.N : static_cast<int64_t>(p.B) * p.N;
  float w[V][8], dw[V][8], db[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = tid + v * blockDim.x;
#pragma unroll
    for (int e = 0; e < 8; ++e) w[v][e] = 1.f, dw[v][e] = 0.f, db[v][e] = 0.f;
    if (p.weight != nullptr && c < p.C8)
      ln_param8(p.weight, p.param_f32, p.per_sample ? g : 0, p.C8, c, w[v]);
  }
  uint4 xv[V], dv[V];
  float mean = 0.f, rstd = 0.f;
  auto load = [&](int64_t row) {
    const uint4 *x = p.x + row * p.C8, *dy = p.dy + row * p.C8;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = tid + v * blockDim.x;
      xv[v] = c < p.C8 ? ln_load(x + c) : make_uint4(0u, 0u, 0u, 0u);
      dv[v] = c < p.C8 ? ln_load(dy + c) : make_uint4(0u, 0u, 0u, 0u);
    }
    mean = __ldg(p.mean_in + row);
    rstd = __ldg(p.rstd_in + row);
  };
  int64_t i = blockIdx.x;
  int64_t row = 0;
  if (i < nrows) load(row = ln_row(p, g, i));
  for (int ph = 0; i < nrows; i += gridDim.x, ph ^= 1) {
    float gv[V][8], xh[V][8];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float d[8];
      ln_unpack(xv[v], xh[v]);
      ln_unpack(dv[v], d);
      const bool in = tid + v * static_cast<int>(blockDim.x) < p.C8;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        xh[v][e] = in ? (xh[v][e] - mean) * rstd : 0.f;
        if (kGrad) {
          dw[v][e] = fmaf(d[e], xh[v][e], dw[v][e]);
          db[v][e] += d[e];
        }
        gv[v][e] = d[e] * w[v][e];
        s1 += gv[v][e];
        s2 = fmaf(gv[v][e], xh[v][e], s2);
      }
    }
    const float rs = rstd;
    uint4 *dx = p.y + row * p.C8;
    // the next row's loads are in flight across the reduction
    if (i + gridDim.x < nrows) load(row = ln_row(p, g, i + gridDim.x));
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
    if (lane == 0) red[ph][warp] = make_float2(s1, s2);
    __syncthreads();  // one barrier a row: the next row uses the other half of red
    s1 = 0.f;
    s2 = 0.f;
    for (int k = 0; k < nwarps; ++k) {
      const float2 t = red[ph][k];
      s1 += t.x;
      s2 += t.y;
    }
    s1 *= p.inv_c;
    s2 *= p.inv_c;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = tid + v * blockDim.x;
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = rs * (gv[v][e] - s1 - xh[v][e] * s2);
      if (c < p.C8) dx[c] = ln_pack(f);
    }
  }
  if (kGrad) {
    float4 *out = reinterpret_cast<float4 *>(
        p.partial + (static_cast<int64_t>(g) * gridDim.x + blockIdx.x) * 16 * p.C8);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = tid + v * blockDim.x;
      if (c < p.C8) {
        out[2 * c] = make_float4(dw[v][0], dw[v][1], dw[v][2], dw[v][3]);
        out[2 * c + 1] = make_float4(dw[v][4], dw[v][5], dw[v][6], dw[v][7]);
        out[2 * (p.C8 + c)] = make_float4(db[v][0], db[v][1], db[v][2], db[v][3]);
        out[2 * (p.C8 + c) + 1] = make_float4(db[v][4], db[v][5], db[v][6], db[v][7]);
      }
    }
  }
  // padding rows of dx are zero (all samples', shared among all blocks)
  const int64_t pad = static_cast<int64_t>(p.P) * p.Nl - p.N;
  const int64_t nblk = static_cast<int64_t>(gridDim.x) * gridDim.y;
  for (int64_t j = static_cast<int64_t>(g) * gridDim.x + blockIdx.x; j < pad * p.B; j += nblk) {
    const int b = static_cast<int>(j / pad);
    const int t = static_cast<int>(p.N + (j - b * pad));
    const int r = t / p.Nl;
    uint4 *dx = p.y + ((static_cast<int64_t>(r) * p.B + b) * p.Nl + (t - r * p.Nl)) * p.C8;
    for (int c = tid; c < p.C8; c += blockDim.x) dx[c] = make_uint4(0u, 0u, 0u, 0u);
  }
}

constexpr int kLnGradCols = 32, kLnGradRows = 16;

// Sums the blocks' partial rows [groups][blocks][2][C] in block order: thread
// (x, y) adds column x of partial rows y, y + 16, ..., then the 16 sums of a
// column are added in order.  blockIdx.y is the group, blockIdx.z 0 for dw, 1 for db.
__global__ void __launch_bounds__(kLnGradCols *kLnGradRows)
layer_norm_grad_kernel(const LnParams p, int blocks) {
  __shared__ float red[kLnGradRows][kLnGradCols + 1];
  const int x = threadIdx.x % kLnGradCols, y = threadIdx.x / kLnGradCols;
  const int64_t C = 8ll * p.C8;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * kLnGradCols + x;
  const int64_t g = blockIdx.y;
  const int which = blockIdx.z;
  float s = 0.f;
  if (col < C)
    for (int k = y; k < blocks; k += kLnGradRows)
      s += p.partial[((g * blocks + k) * 2 + which) * C + col];
  red[y][x] = s;
  __syncthreads();
  if (y == 0 && col < C) {
#pragma unroll
    for (int k = 1; k < kLnGradRows; ++k) s += red[k][x];
    void *out = which ? p.dbias : p.dweight;
    if (p.param_f32)
      static_cast<float *>(out)[g * C + col] = s;
    else
      static_cast<__nv_bfloat16 *>(out)[g * C + col] = __float2bfloat16_rn(s);
  }
}

}  // namespace sp
