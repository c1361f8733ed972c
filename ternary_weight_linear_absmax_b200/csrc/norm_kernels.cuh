// Layer norm (forward to floats or to the contraction's int8 tokens, backward)
// and the 8-bit activation checkpoints that the backward passes read.
//
//   μ = mean x, d = x − μ, σ² = mean d², r = 1/√(σ² + ε), x̂ = d·r, y = x̂·w + b
//   dx = r·(g − mean g − x̂·mean(g·x̂)) with g = w·dy,  dw = Σ_m dy·x̂,  db = Σ_m dy
//
// The two row sums of the forward are taken in 64 bits and μ, r rounded once to
// fp32; d, x̂ and y are one fp32 operation each, in the order written. So
// the int8 tokens made from y are decided by the same fp32 values whatever
// the order of the sums.
//
// Checkpoint: groups of 64 columns, one fp32 scale each. With m = max|v| over
// the group and top = 127 (signed) or 255 (unsigned): codes Round(v·(top/m)),
// scale m/top; a group whose m is below 2^-100 holds zeros. A code is off by at
// most half a step, m/(2·top).
#pragma once

#include "bl_device.cuh"

namespace bl {

constexpr int kNormThreads = 256;
constexpr float kCkptTiny = 7.888609052210118e-31f;  // 2^-100

// Eight consecutive elements as fp32.
template <typename T>
__device__ __forceinline__ void norm_load8(const T* p, float (&v)[8]) {
  if constexpr (sizeof(T) == 1) {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
    const int8_t* b = reinterpret_cast<const int8_t*>(&u);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (float)b[j];
  } else if constexpr (sizeof(T) == 2) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
    const __nv_bfloat16* b = reinterpret_cast<const __nv_bfloat16*>(&u);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __bfloat162float(b[j]);
  } else {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}

template <typename T>
__device__ __forceinline__ void norm_store8(T* p, const float (&v)[8]) {
  if constexpr (sizeof(T) == 2) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

__device__ __forceinline__ float warp_sum_f(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the block in a fixed order, returned to every thread. `red` holds
// one value per warp; the barrier in front lets it be used again.
__device__ __forceinline__ double block_sum_d(double v, double* red) {
  v = warp_sum_d(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  double t = 0.0;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) t += red[w];
  return t;
}
__device__ __forceinline__ float block_sum_f(float v, float* red) {
  v = warp_sum_f(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.f;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) t += red[w];
  return t;
}
__device__ __forceinline__ float block_max_f(float v, float* red) {
  v = warp_max(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.f;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) t = fmaxf(t, red[w]);
  return t;
}

// Checkpoint codes of eight columns of a group held by eight neighbouring
// lanes (all 32 lanes of the warp take part; lanes without columns pass
// zeros). Unsigned codes (top 255) take v ≥ 0. Returns the scale.
template <bool SIGNED>
__device__ __forceinline__ float ckpt_codes8(const float (&v)[8], uint32_t& w0, uint32_t& w1) {
  constexpr float top = SIGNED ? 127.0f : 255.0f;
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[j]));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const bool live = m >= kCkptTiny;
  const float inv = live ? __fdiv_rn(top, m) : 0.f;
  uint32_t b[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)  // the sum's low byte is the rounded integer (ties to even)
    b[j] = __float_as_uint(__fadd_rn(__fmul_rn(v[j], inv), 12582912.0f));
  w0 = pack4_low_bytes(b[0], b[1], b[2], b[3]);
  w1 = pack4_low_bytes(b[4], b[5], b[6], b[7]);
  return live ? __fdiv_rn(m, top) : 0.f;
}

// ---------------------------------------------------------------------------
// Forward, one CTA per row, eight columns per thread and step.
struct NormParams {
  const void* X;
  const float* weight;  // [K]
  const float* bias;    // [K] or null
  int64_t M, K;
  float eps, q_eps;
  void* Y;              // floats: [M, K]
  float* mean;          // [M] or null
  float* rstd;          // [M] or null
  int8_t* Aq;           // tokens: [M, K]
  float* gamma;         // [M]
  int32_t* rowsum;      // [M] or null
  int8_t* xq;           // checkpoint of x̂ [M, K] or null
  float* xs;            // [M, K/64]
};

__device__ __forceinline__ void norm_affine8(const float (&x)[8], float mean, float rstd,
                                             const float* weight, const float* bias, int64_t c,
                                             float (&xhat)[8], float (&y)[8]) {
  float w[8];
  norm_load8(weight + c, w);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    xhat[j] = __fmul_rn(__fsub_rn(x[j], mean), rstd);
    y[j] = __fmul_rn(xhat[j], w[j]);
  }
  if (bias != nullptr) {
    norm_load8(bias + c, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = __fadd_rn(y[j], w[j]);
  }
}

// OUT: fp32/bf16 rows, or int8_t for the tokens.
template <typename T, typename OUT>
__global__ void __launch_bounds__(kNormThreads) layernorm_kernel(const NormParams p) {
  __shared__ double redd[kNormThreads / 32];
  __shared__ float redf[kNormThreads / 32];
  const int64_t m = blockIdx.x, units = p.K / 8;
  const T* row = reinterpret_cast<const T*>(p.X) + m * p.K;
  float x[8];
  double s = 0.0;
  for (int64_t u = threadIdx.x; u < units; u += kNormThreads) {
    norm_load8(row + 8 * u, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) s += (double)x[j];
  }
  const float mean = (float)(block_sum_d(s, redd) / (double)p.K);
  s = 0.0;
  for (int64_t u = threadIdx.x; u < units; u += kNormThreads) {
    norm_load8(row + 8 * u, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const double d = (double)__fsub_rn(x[j], mean);
      s = fma(d, d, s);
    }
  }
  const float rstd = (float)(1.0 / sqrt(block_sum_d(s, redd) / (double)p.K + (double)p.eps));
  if (threadIdx.x == 0) {
    if (p.mean != nullptr) p.mean[m] = mean;
    if (p.rstd != nullptr) p.rstd[m] = rstd;
  }
  float xhat[8], y[8];
  if constexpr (sizeof(OUT) > 1) {
    for (int64_t u = threadIdx.x; u < units; u += kNormThreads) {
      norm_load8(row + 8 * u, x);
      norm_affine8(x, mean, rstd, p.weight, p.bias, 8 * u, xhat, y);
      norm_store8(reinterpret_cast<OUT*>(p.Y) + m * p.K + 8 * u, y);
    }
  } else {
    float mx = 0.f;
    const int64_t rounds = (units + kNormThreads - 1) / kNormThreads;
    for (int64_t i = 0; i < rounds; ++i) {  // whole warps: a checkpoint group is eight lanes
      const int64_t u = i * kNormThreads + threadIdx.x;
#pragma unroll
      for (int j = 0; j < 8; ++j) xhat[j] = 0.f;
      if (u < units) {
        norm_load8(row + 8 * u, x);
        norm_affine8(x, mean, rstd, p.weight, p.bias, 8 * u, xhat, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) mx = fmaxf(mx, fabsf(y[j]));
      }
      if (p.xq != nullptr) {
        uint32_t w0, w1;
        const float sc = ckpt_codes8<true>(xhat, w0, w1);
        if (u < units) {
          *reinterpret_cast<uint2*>(p.xq + m * p.K + 8 * u) = make_uint2(w0, w1);
          if ((u & 7) == 0) p.xs[(m * p.K + 8 * u) / 64] = sc;
        }
      }
    }
    mx = block_max_f(mx, redf);
    const float scale = __fdiv_rn(127.0f, __fadd_rn(mx, p.q_eps));
    int sum = 0;
    for (int64_t u = threadIdx.x; u < units; u += kNormThreads) {
      norm_load8(row + 8 * u, x);
      norm_affine8(x, mean, rstd, p.weight, p.bias, 8 * u, xhat, y);
      uint32_t b[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) b[j] = quant_i8_bits(y[j], scale);
      const uint32_t w0 = pack4_low_bytes(b[0], b[1], b[2], b[3]);
      const uint32_t w1 = pack4_low_bytes(b[4], b[5], b[6], b[7]);
      sum = dp4a(w1, 0x01010101u, dp4a(w0, 0x01010101u, sum));
      *reinterpret_cast<uint2*>(p.Aq + m * p.K + 8 * u) = make_uint2(w0, w1);
    }
    __shared__ int redi[kNormThreads / 32];
    sum = warp_sum_i(sum);
    if ((threadIdx.x & 31) == 0) redi[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
      p.gamma[m] = mx;
      if (p.rowsum != nullptr) {
        int t = 0;
        for (int w = 0; w < kNormThreads / 32; ++w) t += redi[w];
        p.rowsum[m] = t;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Backward. Each CTA takes every gridDim.x-th row and writes its share of dw
// and db into its own row of `part` (2·K floats); norm_colsum_kernel adds the
// rows in a fixed order, so the result does not depend on timing.
constexpr int kNormGradParts = 296;

struct NormGradParams {
  const void* dY;      // [M, K]
  const void* X;       // [M, K] input, or int8 checkpoint of x̂
  const float* xs;     // checkpoint scales [M, K/64]
  const float* mean;   // [M] (input form)
  const float* rstd;   // [M]
  const float* weight; // [K]
  int64_t M, K;
  void* dX;            // [M, K]
  float* part;         // [grid, 2, K]
};

// x̂ of eight columns: from the input, or from the checkpoint (TX = int8_t).
template <typename TX>
__device__ __forceinline__ void norm_xhat8(const NormGradParams& p, int64_t m, int64_t c,
                                           float mean, float rstd, float (&xh)[8]) {
  norm_load8(reinterpret_cast<const TX*>(p.X) + m * p.K + c, xh);
  if constexpr (sizeof(TX) == 1) {
    const float s = __ldg(p.xs + (m * p.K + c) / 64);
#pragma unroll
    for (int j = 0; j < 8; ++j) xh[j] = __fmul_rn(xh[j], s);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) xh[j] = __fmul_rn(__fsub_rn(xh[j], mean), rstd);
  }
}

template <typename TD, typename TX, typename TO>
__global__ void __launch_bounds__(kNormThreads) layernorm_grad_kernel(const NormGradParams p) {
  __shared__ float red[kNormThreads / 32];
  const int64_t units = p.K / 8;
  float* pw = p.part + (int64_t)blockIdx.x * 2 * p.K;
  float* pb = pw + p.K;
  for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x) {
    const bool first = m == blockIdx.x;
    const float rstd = __ldg(p.rstd + m), mean = sizeof(TX) == 1 ? 0.f : __ldg(p.mean + m);
    const TD* dyr = reinterpret_cast<const TD*>(p.dY) + m * p.K;
    float dy[8], xh[8], w[8];
    float a = 0.f, b = 0.f;
    for (int64_t u = threadIdx.x; u < units; u += kNormThreads) {
      const int64_t c = 8 * u;
      norm_load8(dyr + c, dy);
      norm_xhat8<TX>(p, m, c, mean, rstd, xh);
      norm_load8(p.weight + c, w);
      float aw[8], ab[8];
      if (!first) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          aw[j] = pw[c + j];
          ab[j] = pb[c + j];
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float gj = dy[j] * w[j];
        a += gj;
        b = fmaf(gj, xh[j], b);
        pw[c + j] = first ? dy[j] * xh[j] : fmaf(dy[j], xh[j], aw[j]);
        pb[c + j] = first ? dy[j] : ab[j] + dy[j];
      }
    }
    a = block_sum_f(a, red) / (float)p.K;
    b = block_sum_f(b, red) / (float)p.K;
    for (int64_t u = threadIdx.x; u < units; u += kNormThreads) {
      const int64_t c = 8 * u;
      norm_load8(dyr + c, dy);
      norm_xhat8<TX>(p, m, c, mean, rstd, xh);
      norm_load8(p.weight + c, w);
      float dx[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) dx[j] = rstd * (fmaf(-xh[j], b, dy[j] * w[j] - a));
      norm_store8(reinterpret_cast<TO*>(p.dX) + m * p.K + c, dx);
    }
  }
}

__global__ void __launch_bounds__(256)
norm_colsum_kernel(const float* __restrict__ part, int parts, int64_t K, float* __restrict__ dw,
                   float* __restrict__ db) {
  const int64_t c = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;  // 0 .. 2K
  if (c >= 2 * K) return;
  float s = 0.f;
  for (int i = 0; i < parts; ++i) s += part[(int64_t)i * 2 * K + c];
  if (c < K)
    dw[c] = s;
  else if (db != nullptr)
    db[c - K] = s;
}

// ---------------------------------------------------------------------------
// ReLU² of the FFN's hidden layer in training: from the up-projection's INT32
// accumulators, the requantised tokens of the down-projection (the arithmetic
// of relu2_requant_kernel) and an 8-bit checkpoint of p = max(h, 0). One CTA
// per token.
__global__ void __launch_bounds__(kNormThreads)
relu2_requant_q8_kernel(const int32_t* __restrict__ acc, int64_t H,
                        const float* __restrict__ gammaX, const float* __restrict__ g_up, float eps,
                        int8_t* __restrict__ Rq, float* __restrict__ gammaR,
                        int32_t* __restrict__ rowsum, uint8_t* __restrict__ Pq,
                        float* __restrict__ ps) {
  __shared__ float redf[kNormThreads / 32];
  __shared__ int redi[kNormThreads / 32];
  const int64_t m = blockIdx.x, units = H / 8;
  const int4* a4 = reinterpret_cast<const int4*>(acc + m * H);
  const float sc = __fdiv_rn(__fmul_rn(gammaX[m], *g_up), 127.0f);
  auto load_p = [&](int64_t u, float (&v)[8]) {
    const int4 a = __ldg(a4 + 2 * u), b = __ldg(a4 + 2 * u + 1);
    const int e[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = fmaxf(__fmul_rn((float)e[j], sc), 0.0f);
  };
  float v[8], mx = 0.f;
  const int64_t rounds = (units + kNormThreads - 1) / kNormThreads;
  for (int64_t i = 0; i < rounds; ++i) {
    const int64_t u = i * kNormThreads + threadIdx.x;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.f;
    if (u < units) load_p(u, v);
    uint32_t w0, w1;
    const float s = ckpt_codes8<false>(v, w0, w1);
    if (u < units) {
      *reinterpret_cast<uint2*>(Pq + m * H + 8 * u) = make_uint2(w0, w1);
      if ((u & 7) == 0) ps[(m * H + 8 * u) / 64] = s;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) mx = fmaxf(mx, __fmul_rn(v[j], v[j]));
  }
  mx = block_max_f(mx, redf);
  const float s = __fdiv_rn(127.0f, __fadd_rn(mx, eps));
  int sum = 0;
  for (int64_t u = threadIdx.x; u < units; u += kNormThreads) {
    load_p(u, v);
    uint32_t b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) b[j] = quant_i8_bits(__fmul_rn(v[j], v[j]), s);
    const uint32_t w0 = pack4_low_bytes(b[0], b[1], b[2], b[3]);
    const uint32_t w1 = pack4_low_bytes(b[4], b[5], b[6], b[7]);
    sum = dp4a(w1, 0x01010101u, dp4a(w0, 0x01010101u, sum));
    *reinterpret_cast<uint2*>(Rq + m * H + 8 * u) = make_uint2(w0, w1);
  }
  sum = warp_sum_i(sum);
  if ((threadIdx.x & 31) == 0) redi[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    gammaR[m] = mx;
    if (rowsum != nullptr) {
      int t = 0;
      for (int w = 0; w < kNormThreads / 32; ++w) t += redi[w];
      rowsum[m] = t;
    }
  }
}

// dH = 2·p̂·dR, p̂ = scale·code: eight columns per thread.
template <typename TD, typename TO>
__global__ void __launch_bounds__(kNormThreads)
relu2_grad_q8_kernel(const TD* __restrict__ dR, const uint8_t* __restrict__ Pq,
                     const float* __restrict__ ps, int64_t units, TO* __restrict__ dH) {
  for (int64_t u = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; u < units;
       u += (int64_t)gridDim.x * blockDim.x) {
    float d[8];
    norm_load8(dR + 8 * u, d);
    const uint2 q = __ldg(reinterpret_cast<const uint2*>(Pq + 8 * u));
    const float s = 2.0f * __ldg(ps + u / 8);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      d[j] *= s * (float)(((j < 4 ? q.x : q.y) >> (8 * (j & 3))) & 255u);
    norm_store8(dH + 8 * u, d);
  }
}

}  // namespace bl
