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
  int split;                      // warps per row block: 1, 2, 4, 8 or 16
  int depth;                      // blocks in flight per warp: 2, 4 or 8
  uint32_t ones;                  // kW4Ones
};

__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                               uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The pair q of codes of a packed word as bf16 (q − z)/128, exact: 0x3F80 | q
// is the bf16 1 + q/128 (7 mantissa bits), `one_z` holds 1 + z/128 twice. The
// sums stay 128 times smaller until the result is written, so that no product
// overflows whose scaled sum does not. `ones` is 0x3F803F80 in a register that
// the compiler does not see through: with both constants known it takes two
// logic operations per pair instead of one.
constexpr float kW4Unit = 128.0f;
constexpr uint32_t kW4Ones = 0x3F803F80u;
__device__ __forceinline__ uint32_t w4_pair(uint32_t word, int q, uint32_t ones, uint32_t one_z) {
  uint32_t v;
  asm("lop3.b32 %0, %1, 0x000F000F, %2, 0xEA;" : "=r"(v) : "r"(word >> (4 * q)), "r"(ones));
  uint32_t d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(v), "r"(one_z));
  return d;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Eight consecutive activations. A bf16 row is taken as it is; an fp32 value
// is the exact sum of three bf16 pieces, each the leading 8 bits of what the
// ones before left (cut, not rounded: 3 × 8 bits hold the 24-bit significand,
// and no piece overflows), one per MMA column, so the products stay exact and
// the sum is an fp32 sum.
template <typename T>
struct W4Eight {
  float v[8];
  __device__ __forceinline__ void load(const T* p) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.f;
  }
  // The next piece, as bf16 pairs; what it leaves stays for the one after.
  __device__ __forceinline__ uint4 piece() {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = __byte_perm(__float_as_uint(v[2 * j]), __float_as_uint(v[2 * j + 1]), 0x7632);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[j] = __fsub_rn(v[j], __uint_as_float(__float_as_uint(v[j]) & 0xFFFF0000u));
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct W4Eight<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void clear() { v = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ uint4 piece() { return v; }
};

constexpr int kW4Warps = 16;
constexpr int kW4Threads = 32 * kW4Warps;
constexpr size_t kW4SmemCap = 226 * 1024;

// Shared memory: the sums [2][warp][16 rows][8·NT],
// each warp's ring of blocks (codes, scales, zero points), the activations.
template <int NT>
__host__ __device__ constexpr size_t w4_part_bytes() {
  return (size_t)2 * kW4Warps * 16 * 8 * NT * 4;
}
template <int V>
__host__ __device__ constexpr int w4_stage_bytes() {
  return 1024 + 48 * V;
}
template <int V, int NT>
__host__ __device__ constexpr size_t w4_fixed_bytes(int depth) {
  return w4_part_bytes<NT>() + (size_t)kW4Warps * depth * w4_stage_bytes<V>();
}
// One MMA column of activations: KB blocks of 256 bytes and 64 more, so that
// two columns (the eight lanes of a 16-byte read) fall on different banks.
__host__ __device__ inline size_t w4_x_stride(int64_t K) { return (size_t)((K + 127) / 128) * 256 + 64; }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
// The load where `on` holds, `v` as it was elsewhere.
__device__ __forceinline__ void lds128_if(uint4& v, uint32_t a, bool on) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
               "@p ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
               : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w) : "r"(a), "r"((int)on));
}
__device__ __forceinline__ uint32_t lds_u32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Y = X·Wᵀ for up to 8·NT MMA columns (tokens, or three pieces of an fp32
// token) per grid row. Each CTA owns a slab of 16-row blocks. Groups of
// `split` warps take a row block each, its 128-column blocks in turn, `depth`
// blocks in flight per warp; the warps' sums meet in shared memory, in a
// fixed order. XS: the activations lie in shared memory (each CTA reads them
// once), else they are read through L2 (long rows).
template <typename T, int V, int NT, bool XS>
__global__ void __launch_bounds__(kW4Threads) w4_linear_kernel(const W4Params p) {
  constexpr int P = sizeof(T) == 2 ? 1 : 3;     // MMA columns per token
  constexpr int COLS = 8 * NT, TOK = COLS / P;  // tokens per pass
  constexpr int ST = w4_stage_bytes<V>();
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int S = p.split, D = p.depth, G = kW4Warps / S;
  const int group = warp / S, ks = warp - group * S;
  float* part = reinterpret_cast<float*>(smem);
  uint8_t* ring = smem + w4_part_bytes<NT>() + warp * (D * ST);
  uint8_t* xs = smem + w4_fixed_bytes<V, NT>(D);
  // Blocks are counted in 32 bits: 2^31 of them are 2 TB.
  const int RB = (int)((p.N + 15) / 16), KB = (int)((p.K + 127) / 128);
  const int rb0 = (int)((int64_t)RB * blockIdx.x / gridDim.x);
  const int rb1 = (int)((int64_t)RB * (blockIdx.x + 1) / gridDim.x);
  const int64_t m0 = (int64_t)blockIdx.y * TOK;
  const int toks = (int)min((int64_t)TOK, p.M - m0), cols = toks * P;
  const T* X = reinterpret_cast<const T*>(p.X) + m0 * p.K;
  const int xstride = (int)w4_x_stride(p.K);

  pdl_launch_dependents();
  // Requests run ahead of the compute loop over the same blocks: 1024 bytes of
  // codes, two pieces per lane, and 32·V bytes of scales and 16·V of zero
  // points by the first lanes. The first ones go out before the wait for the
  // previous kernel, which does not write the weights.
  const uint8_t* w_src = p.W4 + 16 * lane;
  const bool is_scale = lane < 2 * V, has_aux = is_scale || (lane < 3 * V && p.zeros != nullptr);
  const uint8_t* aux_src = is_scale ? reinterpret_cast<const uint8_t*>(p.scales) + 16 * lane
                                    : p.zeros + 16 * (lane - 2 * V);
  const uint32_t aux_step = is_scale ? 32 * V : 16 * V;
  const uint32_t ring_s = smem_u32(ring), ring_end = ring_s + D * ST;
  uint32_t q_dst = ring_s + 16 * lane;
  int q_rb = ks < KB ? rb0 + group : rb1, q_kb = ks;
  auto request = [&]() {
    if (q_rb < rb1) {
      const uint32_t blk = (uint32_t)q_rb * KB + q_kb;
      const uint8_t* w = w_src + (uint64_t)blk * 1024u;
      cp_async16(q_dst, w);
      cp_async16(q_dst + 512, w + 512);
      if (has_aux) cp_async16(q_dst + 1024, aux_src + (uint64_t)blk * aux_step);
      q_kb += S;
      if (q_kb >= KB) {
        q_kb = ks;
        q_rb += G;
      }
      q_dst += ST;
      if (q_dst >= ring_end) q_dst -= D * ST;
    }
    cp_async_commit();
  };
  for (int d = 0; d < D - 1; ++d) request();
  pdl_wait_prior_grid();

  if constexpr (XS) {
    const int units = KB * 16;  // 8 columns of K each
    constexpr int B = P == 1 ? 4 : 2;
    for (int c = 0; c < toks; c += B) {  // a few tokens' loads in flight together
      for (int u = tid; u < units; u += kW4Threads) {
        W4Eight<T> e[B];
#pragma unroll
        for (int b = 0; b < B; ++b) {
          e[b].clear();
          if (c + b < toks && 8 * u < p.K) e[b].load(X + (int64_t)(c + b) * p.K + 8 * u);
        }
#pragma unroll
        for (int b = 0; b < B; ++b) {
          if (c + b < toks) {
#pragma unroll
            for (int i = 0; i < P; ++i)
              *reinterpret_cast<uint4*>(xs + ((c + b) * P + i) * xstride + 16 * u) = e[b].piece();
          }
        }
      }
    }
    __syncthreads();
  }

  // Activations of the lane's MMA columns 8n + g; columns past the tokens stay 0.
  uint32_t xaddr[NT];
  bool live[NT];
  uint4 x[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    live[n] = 8 * n + g < cols;
    xaddr[n] = smem_u32(xs + (8 * n + g) * xstride + 16 * t);
#pragma unroll
    for (int u = 0; u < 4; ++u) x[n][u] = make_uint4(0u, 0u, 0u, 0u);
  }

  const uint32_t ones = p.ones;
  uint32_t src = ring_s;
  int buf = 0;
  for (int rb = rb0 + group; rb < rb1; rb += G) {
    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
    for (int kb = ks; kb < KB; kb += S) {
      __syncwarp();  // the stage read last is free: every lane is past its reads
      request();
      if (D == 8)
        cp_async_wait<7>();
      else if (D == 4)
        cp_async_wait<3>();
      else
        cp_async_wait<1>();
      __syncwarp();
      const uint4 wlo = lds128(src + 16 * lane), whi = lds128(src + 512 + 16 * lane);
      const uint32_t lo[4] = {wlo.x, wlo.y, wlo.z, wlo.w}, hi[4] = {whi.x, whi.y, whi.z, whi.w};
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if constexpr (XS) {
#pragma unroll
          for (int u = 0; u < 4; ++u) lds128_if(x[n][u], xaddr[n] + kb * 256 + 64 * u, live[n]);
        } else {
          const int c = 8 * n + g;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int64_t k = (int64_t)kb * 128 + 32 * u + 8 * t;
            W4Eight<T> e;
            e.clear();
            if (live[n] && k < p.K) e.load(X + (int64_t)(c / P) * p.K + k);
            x[n][u] = e.piece();
            for (int i = 0; i < c % P; ++i) x[n][u] = e.piece();
          }
        }
      }
      float pa[NT][4];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        // bf16 1 + z/128 twice, for rows g and g + 8: z in the mantissa
        uint32_t z = 0x0808u;
        if (p.zeros != nullptr) z = lds_u16(src + 1024 + 32 * V + (g * V + v) * 2);
        z |= 0x3F8080u;
        const uint32_t z0 = __byte_perm(z, 0u, 0x2020), z1 = __byte_perm(z, 0u, 0x2121);
#pragma unroll
        for (int n = 0; n < NT; ++n) pa[n][0] = pa[n][1] = pa[n][2] = pa[n][3] = 0.f;
#pragma unroll
        for (int u = v * (4 / V); u < (v + 1) * (4 / V); ++u) {
          uint32_t a[8];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            a[2 * q] = w4_pair(lo[u], q, ones, z0);
            a[2 * q + 1] = w4_pair(hi[u], q, ones, z1);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_bf16_16816(pa[n], a[0], a[1], a[2], a[3], x[n][u].x, x[n][u].y);
            mma_bf16_16816(pa[n], a[4], a[5], a[6], a[7], x[n][u].z, x[n][u].w);
          }
        }
        const uint32_t s = lds_u32(src + 1024 + (g * V + v) * 4);
        const float s0 = __uint_as_float(s << 16), s1 = __uint_as_float(s & 0xFFFF0000u);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          acc[n][0] = fmaf(s0, pa[n][0], acc[n][0]);
          acc[n][1] = fmaf(s0, pa[n][1], acc[n][1]);
          acc[n][2] = fmaf(s1, pa[n][2], acc[n][2]);
          acc[n][3] = fmaf(s1, pa[n][3], acc[n][3]);
        }
      }
      src += ST;
      if (src >= ring_end) src -= D * ST;
    }
    // The group's sums of this row block. Two buffers: a warp overwrites one
    // only after the barrier of the row block between, when every warp of the
    // group has read it.
    float* mine = part + ((buf * kW4Warps + warp) * 16 + g) * COLS + 2 * t;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      *reinterpret_cast<float2*>(mine + 8 * n) = make_float2(acc[n][0], acc[n][1]);
      *reinterpret_cast<float2*>(mine + 8 * n + 8 * COLS) = make_float2(acc[n][2], acc[n][3]);
    }
    if (S == 1)
      __syncwarp();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * S) : "memory");
    const float* sums = part + (buf * kW4Warps + group * S) * 16 * COLS;
    for (int j = ks * 32 + lane; j < 16 * toks; j += 32 * S) {
      const int r = j & 15, c = j >> 4;
      float y = 0.f;
#pragma unroll
      for (int pc = P - 1; pc >= 0; --pc)
        for (int w = 0; w < S; ++w) y += sums[(w * 16 + r) * COLS + c * P + pc];
      y *= kW4Unit;
      const int64_t row = (int64_t)rb * 16 + r, o = (m0 + c) * p.N + row;
      if (row < p.N) {
        if (p.y_bf16)
          reinterpret_cast<__nv_bfloat16*>(p.Y)[o] = __float2bfloat16_rn(y);
        else
          reinterpret_cast<float*>(p.Y)[o] = y;
      }
    }
    if (S == 1) __syncwarp();
    buf ^= 1;
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
