// 4-bit weights with group scales: quantiser, packing, unpacking and the
// few-token product Y = X·Wᵀ, for the matrices of a model that are not
// ternarised (the language-model head, the first and last projections).
//
//   w[n, k] = s[n, k/G] · (q[n, k] − z[n, k/G]),  q ∈ [0, 15], G ∈ {32, 64, 128},
//   s bf16, z = 8 (symmetric) or stored, 0..15.
//
// Layout. A warp-level bf16 MMA (m16n8k16) takes 16 weight rows × 16 columns
// as its A operand: lane 4g + t holds rows g and g + 8. The packed matrix is
// cut into blocks of 16 rows × 128 columns, 1024 bytes each, K blocks of a row
// block one after the other. Word (h, g, t, u) of a block (u fastest) holds
// row 16·rb + 8·h + g, columns 128·kb + 32·u + 8·t + (0..7), column 2·p + e of
// those at bit 4·p + 16·e. So lane 4g + t reads 16 contiguous bytes per row
// half (a warp reads 512 contiguous bytes), its four words lie in the four
// 32-column groups of the block, and (word >> 4p) & 0x000F000F is the pair of
// codes of two neighbouring columns in the two halves of a register.
// Scales and zero points are [rb, kb, g, 128/G, h]: a lane's are contiguous.
// Rows past N and columns past K hold scale 0.
#pragma once

#include "bl_device.cuh"

namespace bl {

struct W4Params {
  const void* X;                  // [M, K] fp32/bf16
  const uint8_t* W4;              // packed blocks
  const __nv_bfloat16* scales;    // [rb, kb, 8, V, 2]
  const uint8_t* zeros;           // same shape, or null: 8
  void* Y;                        // [M, N] fp32/bf16
  int64_t M, N, K;
  int y_bf16;
};

__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                               uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The pair p of codes of a packed word as bf16 (q − z)/128, exact: 0x3F80 | q
// is the bf16 1 + q/128 (7 mantissa bits), `one_z` holds 1 + z/128 twice. The
// sums stay 128 times smaller until the result is written, so that no product
// overflows whose scaled sum does not.
constexpr float kW4Unit = 128.0f;
__device__ __forceinline__ uint32_t w4_pair(uint32_t word, int p, __nv_bfloat162 one_z) {
  const uint32_t v = ((word >> (4 * p)) & 0x000F000Fu) | 0x3F803F80u;
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), one_z);
  return *reinterpret_cast<const uint32_t*>(&d);
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Eight consecutive activations as bf16 pairs. A bf16 row is taken as it is;
// an fp32 value is the exact sum of three bf16 pieces, each the leading 8 bits
// of what the ones before left (cut, not rounded: 3 × 8 bits hold the 24-bit
// significand, and no piece overflows), one per MMA column, so the products
// stay exact and the sum is an fp32 sum.
template <typename T>
__device__ __forceinline__ uint4 w4_load_x(const T* p, int piece) {
  if constexpr (sizeof(T) == 2) {
    return __ldg(reinterpret_cast<const uint4*>(p));
  } else {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      for (int i = 0; i < piece; ++i)
        v[j] = __fsub_rn(v[j], __uint_as_float(__float_as_uint(v[j]) & 0xFFFF0000u));
    auto top2 = [](float lo, float hi) {
      return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
    };
    return make_uint4(top2(v[0], v[1]), top2(v[2], v[3]), top2(v[4], v[5]), top2(v[6], v[7]));
  }
}

constexpr int kW4Warps = 8;
constexpr int kW4Threads = 32 * kW4Warps;

// One CTA per 16-row block and group of tokens; its warps take every eighth
// 128-column block and their sums meet in shared memory.
template <typename T, int G>
__global__ void __launch_bounds__(kW4Threads) w4_linear_kernel(const W4Params p) {
  constexpr int V = 128 / G;                    // groups per block
  constexpr int P = sizeof(T) == 2 ? 1 : 3;     // MMA columns per token
  constexpr int TOK = 8 / P;                    // tokens per pass
  __shared__ float part[kW4Warps][16][8];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int64_t rb = blockIdx.x;
  const int64_t KB = (p.K + 127) / 128;
  for (int64_t m0 = (int64_t)blockIdx.y * TOK; m0 < p.M; m0 += (int64_t)gridDim.y * TOK) {
    const int64_t tok = m0 + g / P;
    const bool col = g < TOK * P && tok < p.M;
    const T* xrow = reinterpret_cast<const T*>(p.X) + tok * p.K;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int64_t kb = warp; kb < KB; kb += kW4Warps) {
      const int64_t blk = rb * KB + kb;
      const uint4* wp = reinterpret_cast<const uint4*>(p.W4 + blk * 1024) + lane;
      const uint4 wlo = __ldg(wp), whi = __ldg(wp + 32);
      const uint32_t lo[4] = {wlo.x, wlo.y, wlo.z, wlo.w}, hi[4] = {whi.x, whi.y, whi.z, whi.w};
      const int64_t so = (blk * 8 + g) * (2 * V);
      float part_acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int v = u / (4 / V);
        __nv_bfloat162 z0 = __float2bfloat162_rn(1.0f + 8.0f / kW4Unit), z1 = z0;
        if (p.zeros != nullptr) {
          z0 = __float2bfloat162_rn(1.0f + (float)__ldg(p.zeros + so + 2 * v) / kW4Unit);
          z1 = __float2bfloat162_rn(1.0f + (float)__ldg(p.zeros + so + 2 * v + 1) / kW4Unit);
        }
        const int64_t k = kb * 128 + 32 * u + 8 * t;
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (col && k < p.K) x = w4_load_x(xrow + k, g % P);
        mma_bf16_16816(part_acc, w4_pair(lo[u], 0, z0), w4_pair(hi[u], 0, z1), w4_pair(lo[u], 1, z0),
                       w4_pair(hi[u], 1, z1), x.x, x.y);
        mma_bf16_16816(part_acc, w4_pair(lo[u], 2, z0), w4_pair(hi[u], 2, z1), w4_pair(lo[u], 3, z0),
                       w4_pair(hi[u], 3, z1), x.z, x.w);
        if ((u + 1) % (4 / V) == 0) {
          const float s0 = __bfloat162float(p.scales[so + 2 * v]);
          const float s1 = __bfloat162float(p.scales[so + 2 * v + 1]);
          acc[0] = fmaf(s0, part_acc[0], acc[0]);
          acc[1] = fmaf(s0, part_acc[1], acc[1]);
          acc[2] = fmaf(s1, part_acc[2], acc[2]);
          acc[3] = fmaf(s1, part_acc[3], acc[3]);
          part_acc[0] = part_acc[1] = part_acc[2] = part_acc[3] = 0.f;
        }
      }
    }
    part[warp][g][2 * t] = acc[0];
    part[warp][g][2 * t + 1] = acc[1];
    part[warp][g + 8][2 * t] = acc[2];
    part[warp][g + 8][2 * t + 1] = acc[3];
    __syncthreads();
    if (tid < 16 * TOK) {
      const int r = tid & 15, c = tid >> 4;
      float y = 0.f;
      for (int pc = P - 1; pc >= 0; --pc)
        for (int w = 0; w < kW4Warps; ++w) y += part[w][r][c * P + pc];
      y *= kW4Unit;
      const int64_t n = rb * 16 + r, m = m0 + c;
      if (n < p.N && m < p.M) {
        if (p.y_bf16)
          reinterpret_cast<__nv_bfloat16*>(p.Y)[m * p.N + n] = __float2bfloat16_rn(y);
        else
          reinterpret_cast<float*>(p.Y)[m * p.N + n] = y;
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Quantising, packing and unpacking. Sixteen lanes take the 128 columns of one
// row in a block, eight columns each (lane 4u + t): a warp reads 256 or 512
// contiguous bytes per row and a group's lanes are neighbours.

// Round(w ÷ s) to the nearest integer, ties to even, as for the exact
// quotient: w is near k·s, both k·s (4 + 8 bits) and the residual w − k·s
// are exact in fp32, so the residual against s/2 settles what the rounding
// of the fp32 quotient may have moved onto or over a border.
__device__ __forceinline__ float w4_round_quotient(float w, float s) {
  float k = rintf(__fdiv_rn(w, s));
  const float r = fmaf(-k, s, w), h = 0.5f * s, dir = copysignf(1.0f, r);
  if (fabsf(r) > h || (fabsf(r) == h && fmodf(k, 2.0f) != 0.0f)) k += dir;
  return k;
}

template <typename T>
__device__ __forceinline__ void w4_load8(const T* p, float (&v)[8]) {
  if constexpr (sizeof(T) == 2) {
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

// Word of eight codes in column order.
__device__ __forceinline__ uint32_t w4_word(const uint32_t (&q)[8]) {
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) w |= q[j] << (4 * (j >> 1) + 16 * (j & 1));
  return w;
}

// Where the eight columns 8·l of row r (0..15) of block (rb, kb) are packed.
__device__ __forceinline__ int64_t w4_word_index(int64_t blk, int r, int l) {
  return blk * 256 + ((r * 4 + (l & 3)) * 4 + (l >> 2));
}
__device__ __forceinline__ int64_t w4_group_index(int64_t blk, int r, int v, int V) {
  return ((blk * 8 + (r & 7)) * V + v) * 2 + (r >> 3);
}

template <typename T>
__global__ void __launch_bounds__(256)
w4_quant_kernel(const T* __restrict__ W, int64_t N, int64_t K, int G, uint32_t* __restrict__ W4,
                __nv_bfloat16* __restrict__ scales, uint8_t* __restrict__ zeros) {
  const int64_t KB = (K + 127) / 128, total = (N + 15) / 16 * KB * 16;  // (row block, kb, row)
  const int l = threadIdx.x & 15, V = 128 / G, gl = G / 8;
  const int64_t step = (int64_t)gridDim.x * (blockDim.x >> 4);
  const int64_t rounds = (total + step - 1) / step;
  for (int64_t i = 0; i < rounds; ++i) {  // every lane takes every round: the shuffles need whole warps
    const int64_t id = (int64_t)blockIdx.x * (blockDim.x >> 4) + (threadIdx.x >> 4) + i * step;
    const int r = (int)(id & 15);
    const int64_t blk = id >> 4, rb = blk / KB, kb = blk - rb * KB;
    const int64_t n = rb * 16 + r, k = kb * 128 + 8 * l;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (id < total && n < N && k < K) w4_load8(W + n * K + k, v);
    float hi = 0.f, lo = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      hi = fmaxf(hi, v[j]);
      lo = fminf(lo, v[j]);
    }
    for (int o = 1; o < gl; o <<= 1) {
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    }
    if (id >= total) continue;
    const float raw = zeros != nullptr ? __fdiv_rn(__fsub_rn(hi, lo), 15.0f)
                                       : __fdiv_rn(fmaxf(hi, -lo), 7.0f);
    const __nv_bfloat16 sb = __float2bfloat16_rn(raw);
    const float s = __bfloat162float(sb);
    float z = 8.0f;
    if (zeros != nullptr) z = s > 0.f ? fminf(w4_round_quotient(-lo, s), 15.0f) : 0.0f;
    uint32_t q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float c = s > 0.f ? w4_round_quotient(v[j], s) + z : z;
      q[j] = (uint32_t)fminf(fmaxf(c, 0.0f), 15.0f);
    }
    W4[w4_word_index(blk, r, l)] = w4_word(q);
    if (l % gl == 0) {
      scales[w4_group_index(blk, r, l / gl, V)] = sb;
      if (zeros != nullptr) zeros[w4_group_index(blk, r, l / gl, V)] = (uint8_t)z;
    }
  }
}

// Codes [N, K/2] (two per byte, the lower column in the low half), scales and
// zero points [N, ceil(K/G)] in row order → the packed layout.
__global__ void __launch_bounds__(256)
w4_pack_kernel(const uint32_t* __restrict__ codes, const __nv_bfloat16* __restrict__ s_in,
               const uint8_t* __restrict__ z_in, int64_t N, int64_t K, int G,
               uint32_t* __restrict__ W4, __nv_bfloat16* __restrict__ scales,
               uint8_t* __restrict__ zeros) {
  const int64_t KB = (K + 127) / 128, total = (N + 15) / 16 * KB * 256, groups = (K + G - 1) / G;
  const int V = 128 / G, gl = G / 8;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int l = (int)(i & 15), r = (int)((i >> 4) & 15);
    const int64_t blk = i >> 8, rb = blk / KB, kb = blk - rb * KB;
    const int64_t n = rb * 16 + r, k = kb * 128 + 8 * l;
    const bool in = n < N && k < K;
    const uint32_t c = in ? __ldg(codes + (n * K + k) / 8) : 0u;
    uint32_t q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = (c >> (4 * j)) & 15u;
    W4[w4_word_index(blk, r, l)] = w4_word(q);
    if (l % gl == 0) {
      const int64_t o = w4_group_index(blk, r, l / gl, V), src = n * groups + k / G;
      scales[o] = in ? s_in[src] : __float2bfloat16_rn(0.0f);
      if (zeros != nullptr) zeros[o] = in ? (uint8_t)(z_in[src] & 15) : (uint8_t)0;
    }
  }
}

// The matrix the packed weights stand for: fl32(s·(q − z)) (exact: 8 + 5 bits),
// rounded once more for a bf16 output.
__global__ void __launch_bounds__(256)
w4_unpack_kernel(const uint32_t* __restrict__ W4, const __nv_bfloat16* __restrict__ scales,
                 const uint8_t* __restrict__ zeros, int64_t N, int64_t K, int G, void* W,
                 int w_bf16) {
  const int64_t KB = (K + 127) / 128, total = (N + 15) / 16 * KB * 256;
  const int V = 128 / G, gl = G / 8;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int l = (int)(i & 15), r = (int)((i >> 4) & 15);
    const int64_t blk = i >> 8, rb = blk / KB, kb = blk - rb * KB;
    const int64_t n = rb * 16 + r, k = kb * 128 + 8 * l;
    if (n >= N || k >= K) continue;
    const uint32_t w = __ldg(W4 + w4_word_index(blk, r, l));
    const int64_t o = w4_group_index(blk, r, l / gl, V);
    const float s = __bfloat162float(scales[o]);
    const int z = zeros != nullptr ? zeros[o] : 8;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[j] = __fmul_rn(s, (float)((int)((w >> (4 * (j >> 1) + 16 * (j & 1))) & 15u) - z));
    if (w_bf16) {
      *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(W) + n * K + k) =
          make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                     pack_bf16x2(v[6], v[7]));
    } else {
      float4* out = reinterpret_cast<float4*>(reinterpret_cast<float*>(W) + n * K + k);
      out[0] = make_float4(v[0], v[1], v[2], v[3]);
      out[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
}

}  // namespace bl
