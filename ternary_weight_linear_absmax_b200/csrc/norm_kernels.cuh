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
// Threads of a row kernel's CTA, at 64 (128) registers each.
__host__ __device__ constexpr int norm_threads(int nu) { return nu <= 2 ? 1024 : 512; }
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

__device__ __forceinline__ void norm_load4(const float* p, float (&v)[4]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
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

// A unit of eight columns as a thread takes it: four and, 32 further on, four
// more of a group of 64, which eight neighbouring threads share. So a warp's
// accesses fill whole sectors whatever the type. `c` is the unit's first column.
__device__ __forceinline__ int64_t unit_column(int64_t u) { return (u >> 3) * 64 + (u & 7) * 4; }
template <typename T>
__device__ __forceinline__ void load_unit(const T* row, int64_t c, float (&v)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (sizeof(T) == 4) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(row + c + 32 * h));
      v[4 * h] = a.x; v[4 * h + 1] = a.y; v[4 * h + 2] = a.z; v[4 * h + 3] = a.w;
    } else {
      const uint2 a = __ldg(reinterpret_cast<const uint2*>(row + c + 32 * h));
      v[4 * h] = __uint_as_float(a.x << 16);
      v[4 * h + 1] = __uint_as_float(a.x & 0xFFFF0000u);
      v[4 * h + 2] = __uint_as_float(a.y << 16);
      v[4 * h + 3] = __uint_as_float(a.y & 0xFFFF0000u);
    }
  }
}
template <typename T>
__device__ __forceinline__ void store_unit(T* row, int64_t c, const float (&v)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(row + c + 32 * h) =
          make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
    } else {
      const __nv_bfloat162 a = __floats2bfloat162_rn(v[4 * h], v[4 * h + 1]);
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[4 * h + 2], v[4 * h + 3]);
      *reinterpret_cast<uint2*>(row + c + 32 * h) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
  }
}
// Eight bytes of a unit, four per word.
__device__ __forceinline__ void store_unit_bytes(void* row, int64_t c, uint32_t w0, uint32_t w1) {
  uint8_t* p = reinterpret_cast<uint8_t*>(row) + c;
  *reinterpret_cast<uint32_t*>(p) = w0;
  *reinterpret_cast<uint32_t*>(p + 32) = w1;
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

// Maximum for a checkpoint group. x̂ may be NaN (SIGNED), and so is the maximum
// then; max(h, 0) never is.
template <bool SIGNED>
__device__ __forceinline__ float ckpt_max(float a, float b) {
  if constexpr (!SIGNED) return fmaxf(a, b);
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}
// What a code counts; a NaN in the group is kept in its scale.
template <bool SIGNED>
__device__ __forceinline__ float ckpt_scale(float m, bool live) {
  const float s = live ? __fdiv_rn(m, SIGNED ? 127.0f : 255.0f) : 0.f;
  return SIGNED && m != m ? m : s;
}

// Checkpoint codes of eight columns of a group held by eight neighbouring
// lanes (all 32 lanes of the warp take part; lanes without columns pass
// zeros). Unsigned codes (top 255) take v ≥ 0. Returns the scale.
template <bool SIGNED>
__device__ __forceinline__ float ckpt_codes8(const float (&v)[8], uint32_t& w0, uint32_t& w1) {
  constexpr float top = SIGNED ? 127.0f : 255.0f;
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = ckpt_max<SIGNED>(m, fabsf(v[j]));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) m = ckpt_max<SIGNED>(m, __shfl_xor_sync(0xffffffffu, m, o));
  const bool live = m >= kCkptTiny;
  const float inv = live ? __fdiv_rn(top, m) : 0.f;
  uint32_t b[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)  // the sum's low byte is the rounded integer (ties to even)
    b[j] = __float_as_uint(__fadd_rn(__fmul_rn(v[j], inv), 12582912.0f));
  w0 = pack4_low_bytes(b[0], b[1], b[2], b[3]);
  w1 = pack4_low_bytes(b[4], b[5], b[6], b[7]);
  return ckpt_scale<SIGNED>(m, live);
}

// Checkpoint codes of NU units (at most eight) per thread, eight neighbouring
// lanes to a group of each unit. The divisions of all the units' groups are
// done at once: lane i of a group takes unit i's maximum. Returns unit i's scale
// in lane i of its group.
template <bool SIGNED, int NU>
__device__ __forceinline__ float ckpt_codes(const float (&v)[NU][8], uint32_t (&w)[NU][2]) {
  constexpr float top = SIGNED ? 127.0f : 255.0f;
  const int l = threadIdx.x & 7;
  float mine = 0.f;
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = ckpt_max<SIGNED>(m, fabsf(v[i][j]));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = ckpt_max<SIGNED>(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (l == i) mine = m;
  }
  const bool live = mine >= kCkptTiny;
  const float inv_mine = live ? __fdiv_rn(top, mine) : 0.f;
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const float inv = __shfl_sync(0xffffffffu, inv_mine, (threadIdx.x & 24) + i);
    uint32_t b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)  // the sum's low byte is the rounded integer (ties to even)
      b[j] = __float_as_uint(__fadd_rn(__fmul_rn(v[i][j], inv), 12582912.0f));
    w[i][0] = pack4_low_bytes(b[0], b[1], b[2], b[3]);
    w[i][1] = pack4_low_bytes(b[4], b[5], b[6], b[7]);
  }
  return ckpt_scale<SIGNED>(mine, live);
}

// quant_i8_bits for values that the scale keeps within the int8 range: with a
// finite s = 127/(max + eps), |v·s| < 127.5, so nothing is clipped, and what is
// left of the clip gives a NaN the same code.
__device__ __forceinline__ uint32_t token_bits(float v, float s) {
  return __float_as_uint(__fadd_rn(fmaxf(__fmul_rn(v, s), -128.0f), 12582912.0f));
}
// s is infinite where max + eps is below 3.8e-37. What quant_i8_bits then makes
// of v is an end of the range (0·s is a NaN); with a scale of 1 token_bits keeps it.
__device__ __forceinline__ bool token_scale_overflows(float s) { return s > 3.402823466e38f; }
__device__ __forceinline__ void token_ends(float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = v[j] > 0.0f ? 127.0f : -128.0f;
}

// ---------------------------------------------------------------------------
// Forward.
struct NormParams {
  const void* X;
  const float* weight;  // [K]
  const float* bias;    // [K] or null
  int64_t M, K;
  double inv_k;         // 1/K
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

// y of a unit from x̂; y may be x̂.
__device__ __forceinline__ void norm_affine_unit(const float (&xhat)[8], const float* weight,
                                                 const float* bias, int64_t c, float (&y)[8]) {
  float w[8];
  load_unit(weight, c, w);
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = __fmul_rn(xhat[j], w[j]);
  if (bias != nullptr) {
    load_unit(bias, c, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = __fadd_rn(y[j], w[j]);
  }
}

// Threads that share a row. A CTA holds blockDim.x / T such groups; with T = 32
// a group is a warp and needs no barrier; there are at most 15 larger ones.
struct RowGroup {
  int T, id, tid, warps;  // threads, which group, thread in it, its warps
  __device__ __forceinline__ explicit RowGroup(int t)
      : T(t), id((int)threadIdx.x / t), tid((int)threadIdx.x % t), warps(t >> 5) {}
  // First of the thread's units when each warp of the group takes 32·nu units in
  // a row; the others follow 32 apart, at distances known to the compiler.
  __device__ __forceinline__ int first_unit(int nu) const {
    return (tid >> 5) * 32 * nu + (tid & 31);
  }
  __device__ __forceinline__ void sync() const {
    if (T == 32)
      __syncwarp();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(T) : "memory");  // 0 is the CTA's
  }
};

// Values of the group's warps, combined in a fixed order and returned to all.
// `buf` is one of several buffers of 32 values per CTA, not used again before
// another of the group's barriers.
template <typename T, typename Op>
__device__ __forceinline__ T group_reduce(const RowGroup& g, T v, T* buf, Op op) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  if (g.T == 32) return v;
  T* mine = buf + (g.id * g.T >> 5);
  if ((threadIdx.x & 31) == 0) mine[g.tid >> 5] = v;
  g.sync();
  v = mine[0];
  for (int w = 1; w < g.warps; ++w) v = op(v, mine[w]);
  return v;
}

// 1/√v in 64 bits, rounded once to fp32: the fp32 estimate (2^-22) and two
// Newton steps, each of which squares the error.
__device__ __forceinline__ float rsqrt_once(double v) {
  if (!(v > 1e-30 && v < 1e30)) return (float)(1.0 / sqrt(v));
  double r = (double)rsqrtf((float)v);
#pragma unroll
  for (int i = 0; i < 2; ++i) r = fma(0.5 * r, fma(-v * r, r, 1.0), r);
  return (float)r;
}

// A unit as loaded.
template <typename T>
struct RawUnit {
  uint2 a[sizeof(T)];
  __device__ __forceinline__ void load(const T* row, int64_t c) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 q = __ldg(reinterpret_cast<const uint4*>(row + c + 32 * h));
        a[2 * h] = make_uint2(q.x, q.y);
        a[2 * h + 1] = make_uint2(q.z, q.w);
      }
    } else {
      a[0] = __ldg(reinterpret_cast<const uint2*>(row + c));
      a[1] = __ldg(reinterpret_cast<const uint2*>(row + c + 32));
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) {
      if constexpr (sizeof(T) == 4) {
        v[2 * i] = __uint_as_float(a[i].x);
        v[2 * i + 1] = __uint_as_float(a[i].y);
      } else {
        v[4 * i] = __uint_as_float(a[i].x << 16);
        v[4 * i + 1] = __uint_as_float(a[i].x & 0xFFFF0000u);
        v[4 * i + 2] = __uint_as_float(a[i].y << 16);
        v[4 * i + 3] = __uint_as_float(a[i].y & 0xFFFF0000u);
      }
    }
  }
};

// One row per group of T threads at a time, NU units of eight columns per
// thread, the row in registers between the passes and the next one on its way.
// FULL: the units are T·NU, every thread has all of its own. OUT: fp32/bf16
// rows, or int8_t for the tokens.
//
// 2048 x 4096 bf16 to bf16 takes 11.3 us (3.0 TB/s, 46 % of the copy rate), bound
// by the latency of the 64-bit sums that a row's threads exchange: four units a
// thread and 128 threads a row beat two units (12.5 us, twice the warps but twice
// the exchanges), one (18 us) and a warp per row with sixteen (26-35 us, too few
// warps); reading the row again instead of keeping it, 14.5 us.
template <typename T, typename OUT, int NU, bool FULL>
__global__ void __launch_bounds__(norm_threads(NU)) layernorm_kernel(const NormParams p, int group) {
  __shared__ double redd[2][32];
  __shared__ float redf[32];
  __shared__ int redi[32];
  const RowGroup g(group);
  const int units = (int)(p.K / 8), groups = (int)blockDim.x / group;
  const int64_t step = (int64_t)gridDim.x * groups;
  auto add = [](auto a, auto b) { return a + b; };
  const int u0 = g.first_unit(NU);
  auto has = [&](int i) { return FULL || u0 + 32 * i < units; };
  RawUnit<T> raw[NU];
  auto load = [&](int64_t m) {
    if (m >= p.M) return;
    const T* row = reinterpret_cast<const T*>(p.X) + m * p.K;
#pragma unroll
    for (int i = 0; i < NU; ++i)
      if (has(i)) raw[i].load(row, unit_column(u0 + 32 * i));
  };
  int64_t m = (int64_t)blockIdx.x * groups + g.id;
  load(m);
  // The barriers in between keep a buffer from being written for the next row
  // while a warp still reads it.
  for (; m < p.M; m += step) {
    float v[NU][8];
    double s[4] = {0.0, 0.0, 0.0, 0.0};  // four chains: a 64-bit addition takes long
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      if (has(i)) {
        raw[i].get(v[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j & 3] += (double)v[i][j];
      }
    }
    load(m + step);
    const float mean = (float)(group_reduce(g, (s[0] + s[1]) + (s[2] + s[3]), redd[0], add) * p.inv_k);
    s[0] = s[1] = s[2] = s[3] = 0.0;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      if (has(i)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[i][j] = __fsub_rn(v[i][j], mean);
          const double d = (double)v[i][j];
          s[j & 3] = fma(d, d, s[j & 3]);
        }
      }
    }
    const float rstd = rsqrt_once(
        fma(group_reduce(g, (s[0] + s[1]) + (s[2] + s[3]), redd[1], add), p.inv_k, (double)p.eps));
    if (g.tid == 0) {
      if (p.mean != nullptr) p.mean[m] = mean;
      if (p.rstd != nullptr) p.rstd[m] = rstd;
    }
    // d becomes x̂, zeros past the row.
#pragma unroll
    for (int i = 0; i < NU; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = has(i) ? __fmul_rn(v[i][j], rstd) : 0.f;
    }
    if constexpr (sizeof(OUT) > 1) {
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        if (has(i)) {
          const int64_t c = unit_column(u0 + 32 * i);
          norm_affine_unit(v[i], p.weight, p.bias, c, v[i]);
          store_unit(reinterpret_cast<OUT*>(p.Y) + m * p.K, c, v[i]);
        }
      }
    } else {
      float mx = 0.f;
      if (p.xq != nullptr) {
        uint32_t w[NU][2];
        const float sc = ckpt_codes<true, NU>(v, w);
#pragma unroll
        for (int i = 0; i < NU; ++i) {
          const int u = u0 + 32 * i;
          if (has(i)) {
            store_unit_bytes(p.xq + m * p.K, unit_column(u), w[i][0], w[i][1]);
            if ((u & 7) == i) p.xs[(m * p.K + 8 * u) / 64] = sc;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        if (has(i)) {
          norm_affine_unit(v[i], p.weight, p.bias, unit_column(u0 + 32 * i), v[i]);
#pragma unroll
          for (int j = 0; j < 8; ++j) mx = fmaxf(mx, fabsf(v[i][j]));
        }
      }
      mx = group_reduce(g, mx, redf, [](float a, float b) { return fmaxf(a, b); });
      float scale = __fdiv_rn(127.0f, __fadd_rn(mx, p.q_eps));
      if (token_scale_overflows(scale)) {
        scale = 1.0f;
#pragma unroll
        for (int i = 0; i < NU; ++i) token_ends(v[i]);
      }
      int sum = 0;
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        if (has(i)) {
          uint32_t b[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) b[j] = token_bits(v[i][j], scale);
          const uint32_t w0 = pack4_low_bytes(b[0], b[1], b[2], b[3]);
          const uint32_t w1 = pack4_low_bytes(b[4], b[5], b[6], b[7]);
          sum = dp4a(w1, 0x01010101u, dp4a(w0, 0x01010101u, sum));
          store_unit_bytes(p.Aq + m * p.K, unit_column(u0 + 32 * i), w0, w1);
        }
      }
      if (p.rowsum != nullptr) sum = group_reduce(g, sum, redi, add);
      if (g.tid == 0) {
        p.gamma[m] = mx;
        if (p.rowsum != nullptr) p.rowsum[m] = sum;
      }
    }
  }
}

// Rows longer than a CTA's registers hold: every pass reads the row again.
template <typename T, typename OUT>
__global__ void __launch_bounds__(kNormThreads) layernorm_long_kernel(const NormParams p) {
  __shared__ double redd[kNormThreads / 32];
  __shared__ float redf[kNormThreads / 32];
  const int64_t m = blockIdx.x, units = p.K / 8;
  const T* row = reinterpret_cast<const T*>(p.X) + m * p.K;
  float x[8];
  double s = 0.0;
  for (int64_t u = threadIdx.x; u < units; u += kNormThreads) {
    load_unit(row, unit_column(u), x);
#pragma unroll
    for (int j = 0; j < 8; ++j) s += (double)x[j];
  }
  const float mean = (float)(block_sum_d(s, redd) * p.inv_k);
  s = 0.0;
  for (int64_t u = threadIdx.x; u < units; u += kNormThreads) {
    load_unit(row, unit_column(u), x);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const double d = (double)__fsub_rn(x[j], mean);
      s = fma(d, d, s);
    }
  }
  const float rstd = rsqrt_once(fma(block_sum_d(s, redd), p.inv_k, (double)p.eps));
  if (threadIdx.x == 0) {
    if (p.mean != nullptr) p.mean[m] = mean;
    if (p.rstd != nullptr) p.rstd[m] = rstd;
  }
  float y[8];
  if constexpr (sizeof(OUT) > 1) {
    for (int64_t u = threadIdx.x; u < units; u += kNormThreads) {
      load_unit(row, unit_column(u), x);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = __fmul_rn(__fsub_rn(x[j], mean), rstd);
      norm_affine_unit(x, p.weight, p.bias, unit_column(u), y);
      store_unit(reinterpret_cast<OUT*>(p.Y) + m * p.K, unit_column(u), y);
    }
  } else {
    float mx = 0.f;
    const int64_t rounds = (units + kNormThreads - 1) / kNormThreads;
    for (int64_t i = 0; i < rounds; ++i) {  // whole warps: a checkpoint group is eight lanes
      const int64_t u = i * kNormThreads + threadIdx.x;
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = 0.f;
      if (u < units) {
        load_unit(row, unit_column(u), x);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __fmul_rn(__fsub_rn(x[j], mean), rstd);
        norm_affine_unit(x, p.weight, p.bias, unit_column(u), y);
#pragma unroll
        for (int j = 0; j < 8; ++j) mx = fmaxf(mx, fabsf(y[j]));
      }
      if (p.xq != nullptr) {
        uint32_t w0, w1;
        const float sc = ckpt_codes8<true>(x, w0, w1);
        if (u < units) {
          store_unit_bytes(p.xq + m * p.K, unit_column(u), w0, w1);
          if ((u & 7) == 0) p.xs[(m * p.K + 8 * u) / 64] = sc;
        }
      }
    }
    mx = block_max_f(mx, redf);
    float scale = __fdiv_rn(127.0f, __fadd_rn(mx, p.q_eps));
    const bool ends = token_scale_overflows(scale);
    if (ends) scale = 1.0f;
    int sum = 0;
    for (int64_t u = threadIdx.x; u < units; u += kNormThreads) {
      load_unit(row, unit_column(u), x);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = __fmul_rn(__fsub_rn(x[j], mean), rstd);
      norm_affine_unit(x, p.weight, p.bias, unit_column(u), y);
      if (ends) token_ends(y);
      uint32_t b[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) b[j] = token_bits(y[j], scale);
      const uint32_t w0 = pack4_low_bytes(b[0], b[1], b[2], b[3]);
      const uint32_t w1 = pack4_low_bytes(b[4], b[5], b[6], b[7]);
      sum = dp4a(w1, 0x01010101u, dp4a(w0, 0x01010101u, sum));
      store_unit_bytes(p.Aq + m * p.K, unit_column(u), w0, w1);
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
constexpr int kNormGradParts = 148;

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

// Four signed bytes as floats: byte ^ 0x80 in the low bits of 2^23.
__device__ __forceinline__ void bytes_to_float(uint32_t w, float* v) {
  w ^= 0x80808080u;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    v[j] = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7540 | j)) - 8388736.0f;
}

template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}

// Four elements from shared memory as fp32.
template <typename T>
__device__ __forceinline__ void lds4(uint32_t a, float (&v)[4]) {
  if constexpr (sizeof(T) == 4) {
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "r"(a));
  } else if constexpr (sizeof(T) == 2) {
    uint32_t x, y;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(x), "=r"(y) : "r"(a));
    v[0] = __uint_as_float(x << 16);
    v[1] = __uint_as_float(x & 0xFFFF0000u);
    v[2] = __uint_as_float(y << 16);
    v[3] = __uint_as_float(y & 0xFFFF0000u);
  } else {
    uint32_t w;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(a));
    bytes_to_float(w, v);
  }
}
template <typename T>
__device__ __forceinline__ void store4(T* p, const float (&v)[4]) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
}

// Sums of a and b over the warp, returned to all lanes. The first step leaves
// a's halves to the lower lanes and b's to the upper ones, so that one value per
// lane is left to add up.
__device__ __forceinline__ void pair_sum(float& a, float& b) {
  const bool up = (threadIdx.x & 16) != 0;
  float v = (up ? b : a) + __shfl_xor_sync(0xffffffffu, up ? a : b, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  a = __shfl_sync(0xffffffffu, v, 0);
  b = __shfl_sync(0xffffffffu, v, 16);
}

// Threads of a CTA at most: 12·NU registers hold dw, db and w, 8·NU the row.
template <int NU>
constexpr int kNormGradThreads = 512;

// Bytes of one row in a ring stage, for one group of T threads: pieces of four
// elements, neighbouring threads on neighbouring pieces (whole sectors).
template <typename TD, typename TX, int NU>
__host__ __device__ constexpr int norm_stage_bytes(int T) {
  return NU * T * 4 * (int)(sizeof(TD) + sizeof(TX));
}

// One row per group of T threads at a time, NU units of four columns per
// thread. A thread copies its own columns of the coming rows into its part of
// the ring (cp.async: nobody else reads them, so no barrier guards the ring),
// and keeps their shares of dw and db in registers; the two row sums are the
// only thing that the group exchanges. The CTA's groups add up their shares in
// shared memory at the end.
//
// Bound by HBM: 8191 x 2560 in fp32 takes 43.3 us with the column sums, 5.8 TB/s,
// 90 % of the copy rate. What it took: pieces of four columns, so that
// neighbouring threads' copies fill whole sectors (eight fp32 columns per thread
// moved every sector twice: 70 us); the row kept between its two uses (read
// again from the ring: 77 us); 512 threads at 128 registers (1024 at 64 spilled
// 60 bytes: 98 us); units at distances known to the compiler (46 us without).
template <typename TD, typename TX, typename TO, int NU, bool FULL>
__global__ void __launch_bounds__(kNormGradThreads<NU>)
layernorm_grad_kernel(const NormGradParams p, int group, int stages) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float2 red[2][32];
  const RowGroup g(group);
  const int groups = (int)blockDim.x / group, T = group, units = (int)(p.K / 4);
  constexpr int BD = 4 * sizeof(TD), BX = 4 * sizeof(TX);  // bytes of a piece
  const int stage_bytes = norm_stage_bytes<TD, TX, NU>(T);
  const uint32_t ring = smem_u32(smem) + g.id * stages * stage_bytes;
  const int u0 = g.first_unit(NU);
  auto has = [&](int i) { return FULL || u0 + 32 * i < units; };
  const uint32_t mine_d = ring + BD * u0, mine_x = ring + NU * T * BD + BX * u0;
  const int64_t step = (int64_t)gridDim.x * groups;
  int64_t next = (int64_t)g.id * gridDim.x + blockIdx.x;  // the next row to request
  const int64_t first = next;
  int q = 0;
  auto request = [&]() {
    if (next < p.M) {
      const TD* d = reinterpret_cast<const TD*>(p.dY) + next * p.K + 4 * u0;
      const TX* x = reinterpret_cast<const TX*>(p.X) + next * p.K + 4 * u0;
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        if (has(i)) {
          cp_async<BD>(mine_d + q * stage_bytes + 32 * i * BD, d + 128 * i);
          cp_async<BX>(mine_x + q * stage_bytes + 32 * i * BX, x + 128 * i);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    next += step;
    q = q + 1 == stages ? 0 : q + 1;
  };
  for (int s = 0; s < stages - 1; ++s) request();

  float dw[NU][4], db[NU][4], w[NU][4];
#pragma unroll
  for (int i = 0; i < NU; ++i) {
#pragma unroll
    for (int j = 0; j < 4; ++j) dw[i][j] = db[i][j] = w[i][j] = 0.f;
    if (NU < 8 && has(i)) norm_load4(p.weight + 4 * u0 + 128 * i, w[i]);
  }
  auto get = [&](int stage, int i, float mean, float rstd, float xs, float (&dy)[4], float (&xh)[4]) {
    lds4<TD>(mine_d + stage * stage_bytes + 32 * i * BD, dy);
    lds4<TX>(mine_x + stage * stage_bytes + 32 * i * BX, xh);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      xh[j] = sizeof(TX) == 1 ? __fmul_rn(xh[j], xs) : __fmul_rn(__fsub_rn(xh[j], mean), rstd);
  };

  int stage = 0, buf = 0;
  const float inv_k = 1.0f / (float)p.K;
  // The next row's scalars are on the way while a row is worked on.
  float rstd_n = 0.f, mean_n = 0.f, xs_n[NU];
  auto scalars = [&](int64_t m) {
    if (m >= p.M) return;
    rstd_n = __ldg(p.rstd + m);
    if constexpr (sizeof(TX) > 1) mean_n = __ldg(p.mean + m);
#pragma unroll
    for (int i = 0; i < NU; ++i)
      if (sizeof(TX) == 1 && has(i)) xs_n[i] = __ldg(p.xs + m * (units / 16) + u0 / 16 + 2 * i);
  };
#pragma unroll
  for (int i = 0; i < NU; ++i) xs_n[i] = 0.f;
  scalars(first);
  for (int64_t m = first; m < p.M; m += step) {
    const float rstd = rstd_n, mean = mean_n;
    float xs[NU];
#pragma unroll
    for (int i = 0; i < NU; ++i) xs[i] = xs_n[i];
    scalars(m + step);
    // The stage read last is this thread's own, and read.
    request();
    if (stages == 4)
      asm volatile("cp.async.wait_group 3;" ::: "memory");
    else if (stages == 3)
      asm volatile("cp.async.wait_group 2;" ::: "memory");
    else
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    float dy[NU][4], xh[NU][4];
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      if (has(i)) {
        get(stage, i, mean, rstd, xs[i], dy[i], xh[i]);
        if (NU == 8) norm_load4(p.weight + 4 * u0 + 128 * i, w[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          dw[i][j] = fmaf(dy[i][j], xh[i][j], dw[i][j]);
          db[i][j] += dy[i][j];
          const float gj = dy[i][j] * w[i][j];
          a += gj;
          b = fmaf(gj, xh[i][j], b);
        }
      }
    }
    pair_sum(a, b);
    if (T > 32) {
      float2* mine = red[buf] + (g.id * T >> 5);
      if ((threadIdx.x & 31) == 0) mine[g.tid >> 5] = make_float2(a, b);
      g.sync();  // one barrier per row: the buffers alternate
      const int l = threadIdx.x & 31;
      const float2 v = l < g.warps ? mine[l] : make_float2(0.f, 0.f);
      a = v.x;
      b = v.y;
      pair_sum(a, b);
      buf ^= 1;
    }
    a *= inv_k;
    b *= inv_k;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      if (has(i)) {
        if (NU == 8) {  // read again rather than kept
          get(stage, i, mean, rstd, xs[i], dy[i], xh[i]);
          norm_load4(p.weight + 4 * u0 + 128 * i, w[i]);
        }
        float dx[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) dx[j] = rstd * fmaf(-xh[i][j], b, fmaf(dy[i][j], w[i][j], -a));
        store4(reinterpret_cast<TO*>(p.dX) + m * p.K + 4 * u0 + 128 * i, dx);
      }
    }
    stage = stage + 1 == stages ? 0 : stage + 1;
  }
  // The groups' shares, [group][2][K] in what was the ring.
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  float* share = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    if (has(i)) {
      store4(share + (int64_t)g.id * 2 * p.K + 4 * u0 + 128 * i, dw[i]);
      store4(share + (int64_t)g.id * 2 * p.K + p.K + 4 * u0 + 128 * i, db[i]);
    }
  }
  __syncthreads();
  float* out = p.part + (int64_t)blockIdx.x * 2 * p.K;
  for (int c = 4 * (int)threadIdx.x; c < 2 * p.K; c += 4 * (int)blockDim.x) {
    float4 s = *reinterpret_cast<const float4*>(share + c);
    for (int k = 1; k < groups; ++k) {
      const float4 v = *reinterpret_cast<const float4*>(share + (int64_t)k * 2 * p.K + c);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    *reinterpret_cast<float4*>(out + c) = s;
  }
}

// Rows longer than a CTA's registers hold: the shares of dw and db live in the
// workspace, and every pass reads the row again.
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
__global__ void __launch_bounds__(kNormThreads) layernorm_grad_long_kernel(const NormGradParams p) {
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

// dw and db from the CTAs' shares: 32 columns per CTA, 32 threads per column
// take every 32nd share each, and add up in order.
__global__ void __launch_bounds__(1024)
norm_colsum_kernel(const float* __restrict__ part, int parts, int64_t K, float* __restrict__ dw,
                   float* __restrict__ db) {
  __shared__ float red[32][33];
  const int lane = threadIdx.x & 31, k = threadIdx.x >> 5;
  const int64_t c = blockIdx.x * (int64_t)32;  // of 0 .. 2K, a multiple of 64
  pdl_wait_prior_grid();
  float v[(kNormGradParts + 31) / 32];
#pragma unroll
  for (int i = 0; i < (kNormGradParts + 31) / 32; ++i)
    v[i] = k + 32 * i < parts ? __ldg(part + (int64_t)(k + 32 * i) * 2 * K + c + lane) : 0.f;
  float s = v[0];
#pragma unroll
  for (int i = 1; i < (kNormGradParts + 31) / 32; ++i) s += v[i];
  red[k][lane] = s;
  __syncthreads();
  s = warp_sum_f(red[lane][k]);  // warp k has column k now
  if (lane != 0) return;
  if (c + k < K)
    dw[c + k] = s;
  else if (db != nullptr)
    db[c + k - K] = s;
}

// ---------------------------------------------------------------------------
// ReLU² of the FFN's hidden layer in training: from the up-projection's INT32
// accumulators, the requantised tokens of the down-projection (the arithmetic
// of relu2_requant_kernel) and an 8-bit checkpoint of p = max(h, 0). One row
// per group of T threads, in registers between the checkpoint and the tokens.
// FULL as in layernorm_kernel.
struct Relu2Params {
  const int32_t* acc;   // [M, H]
  const float* gammaX;  // [M]
  const float* g_up;    // 1
  int64_t M, H;
  float eps;
  int8_t* Rq;           // [M, H]
  float* gammaR;        // [M]
  int32_t* rowsum;      // [M] or null
  uint8_t* Pq;          // [M, H] or null
  float* ps;            // [M, H/64]
};

template <int NU, bool FULL>
__global__ void __launch_bounds__(512, 2) relu2_requant_q8_kernel(const Relu2Params p, int group) {
  __shared__ float redf[32];
  __shared__ int redi[32];
  const RowGroup g(group);
  const int units = (int)(p.H / 8), groups = (int)blockDim.x / group;
  const int64_t m = (int64_t)blockIdx.x * groups + g.id;
  if (m >= p.M) return;  // whole groups
  const int u0 = g.first_unit(NU);
  auto has = [&](int i) { return FULL || u0 + 32 * i < units; };
  const int32_t* row = p.acc + m * p.H;
  int4 raw[NU][2];
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    if (has(i)) {
      const int64_t c = unit_column(u0 + 32 * i);
      raw[i][0] = __ldg(reinterpret_cast<const int4*>(row + c));
      raw[i][1] = __ldg(reinterpret_cast<const int4*>(row + c + 32));
    }
  }
  const float sc = __fdiv_rn(__fmul_rn(__ldg(p.gammaX + m), __ldg(p.g_up)), 127.0f);
  float v[NU][8], mx = 0.f;
#pragma unroll
  for (int i = 0; i < NU; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    if (has(i)) {
      const int e[8] = {raw[i][0].x, raw[i][0].y, raw[i][0].z, raw[i][0].w,
                        raw[i][1].x, raw[i][1].y, raw[i][1].z, raw[i][1].w};
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = fmaxf(__fmul_rn((float)e[j], sc), 0.0f);
    }
  }
  if (p.Pq != nullptr) {
    uint32_t w[NU][2];
    const float sc8 = ckpt_codes<false, NU>(v, w);
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const int u = u0 + 32 * i;
      if (has(i)) {
        store_unit_bytes(p.Pq + m * p.H, unit_column(u), w[i][0], w[i][1]);
        if ((u & 7) == i) p.ps[(m * p.H + 8 * u) / 64] = sc8;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NU; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[i][j] = __fmul_rn(v[i][j], v[i][j]);
      mx = fmaxf(mx, v[i][j]);
    }
  }
  mx = group_reduce(g, mx, redf, [](float a, float b) { return fmaxf(a, b); });
  float s = __fdiv_rn(127.0f, __fadd_rn(mx, p.eps));
  if (token_scale_overflows(s)) {
    s = 1.0f;
#pragma unroll
    for (int i = 0; i < NU; ++i) token_ends(v[i]);
  }
  int sum = 0;
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    if (has(i)) {
      uint32_t b[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) b[j] = token_bits(v[i][j], s);
      const uint32_t w0 = pack4_low_bytes(b[0], b[1], b[2], b[3]);
      const uint32_t w1 = pack4_low_bytes(b[4], b[5], b[6], b[7]);
      sum = dp4a(w1, 0x01010101u, dp4a(w0, 0x01010101u, sum));
      store_unit_bytes(p.Rq + m * p.H, unit_column(u0 + 32 * i), w0, w1);
    }
  }
  sum = group_reduce(g, sum, redi, [](int a, int b) { return a + b; });
  if (g.tid == 0) {
    p.gammaR[m] = mx;
    if (p.rowsum != nullptr) p.rowsum[m] = sum;
  }
}

// Many rows (relu2_shape), or rows longer than registers hold: the second pass
// reads them again, through L2. At 32 registers an SM holds eight such CTAs: 2048 x 11008
// takes 33 us (4.2 TB/s of its 137 MB, bound by issue, 76 % full) against 47 with
// the row kept in registers, and 58 us with the gradient after it, 79 % of the copy
// rate for both.
template <bool KEEP>
__global__ void __launch_bounds__(kNormThreads, 8) relu2_requant_q8_long_kernel(const Relu2Params p) {
  __shared__ float redf[kNormThreads / 32];
  __shared__ int redi[kNormThreads / 32];
  const int64_t m = blockIdx.x, units = p.H / 8;
  const int4* a4 = reinterpret_cast<const int4*>(p.acc + m * p.H);
  const float sc = __fdiv_rn(__fmul_rn(p.gammaX[m], *p.g_up), 127.0f);
  auto load_p = [&](int64_t u, float (&v)[8]) {
    const int4 a = __ldg(a4 + unit_column(u) / 4), b = __ldg(a4 + unit_column(u) / 4 + 8);
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
    if constexpr (KEEP) {
      uint32_t w0, w1;
      const float s = ckpt_codes8<false>(v, w0, w1);
      if (u < units) {
        store_unit_bytes(p.Pq + m * p.H, unit_column(u), w0, w1);
        if ((u & 7) == 0) p.ps[(m * p.H + 8 * u) / 64] = s;
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) mx = fmaxf(mx, __fmul_rn(v[j], v[j]));
  }
  mx = block_max_f(mx, redf);
  float s = __fdiv_rn(127.0f, __fadd_rn(mx, p.eps));
  const bool ends = token_scale_overflows(s);
  if (ends) s = 1.0f;
  int sum = 0;
  for (int64_t u = threadIdx.x; u < units; u += kNormThreads) {
    load_p(u, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(v[j], v[j]);
    if (ends) token_ends(v);
    uint32_t b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) b[j] = token_bits(v[j], s);
    const uint32_t w0 = pack4_low_bytes(b[0], b[1], b[2], b[3]);
    const uint32_t w1 = pack4_low_bytes(b[4], b[5], b[6], b[7]);
    sum = dp4a(w1, 0x01010101u, dp4a(w0, 0x01010101u, sum));
    store_unit_bytes(p.Rq + m * p.H, unit_column(u), w0, w1);
  }
  sum = warp_sum_i(sum);
  if ((threadIdx.x & 31) == 0) redi[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    p.gammaR[m] = mx;
    if (p.rowsum != nullptr) {
      int t = 0;
      for (int w = 0; w < kNormThreads / 32; ++w) t += redi[w];
      p.rowsum[m] = t;
    }
  }
}

// dH = 2·p̂·dR, p̂ = scale·code: units of eight columns, four of them under way
// per thread. Bound by HBM: 2048 x 11008 from fp32 to bf16, 159 MB, in 24 us.
template <typename TD, typename TO>
__global__ void __launch_bounds__(kNormThreads)
relu2_grad_q8_kernel(const TD* __restrict__ dR, const uint8_t* __restrict__ Pq,
                     const float* __restrict__ ps, int64_t units, TO* __restrict__ dH) {
  constexpr int B = 4;
  const int64_t step = (int64_t)gridDim.x * kNormThreads;
  for (int64_t u0 = blockIdx.x * (int64_t)kNormThreads + threadIdx.x; u0 < units; u0 += B * step) {
    RawUnit<TD> raw[B];
    uint32_t q[B][2];
    float s[B];
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int64_t u = u0 + b * step, c = unit_column(u);
      if (u < units) {
        raw[b].load(dR, c);
        q[b][0] = __ldg(reinterpret_cast<const uint32_t*>(Pq + c));
        q[b][1] = __ldg(reinterpret_cast<const uint32_t*>(Pq + c + 32));
        s[b] = __ldg(ps + u / 8);
      }
    }
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int64_t u = u0 + b * step;
      if (u < units) {
        float d[8];
        raw[b].get(d);
        const float s2 = 2.0f * s[b];
#pragma unroll
        for (int j = 0; j < 8; ++j)  // the code in the low bits of 2^23
          d[j] *= s2 * (__uint_as_float(__byte_perm(q[b][j >> 2], 0x4B000000u, 0x7540 | (j & 3))) - 8388608.0f);
        store_unit(dH, unit_column(u), d);
      }
    }
  }
}

}  // namespace bl
