// 4-bit weights with group scales: quantiser, packing, unpacking and the
// few-token product Y = X·Wᵀ, for the matrices of a model that are not
// ternarised (the language-model head, the first and last projections).
//
//   w[n, k] = s[n, k/G] · (q[n, k] − z[n, k/G]),  q ∈ [0, 15], G ∈ {32, 64, 128},
//   s bf16, z = 8 (symmetric) or stored, 0..15.
//
// Layout. A warp-level int8 MMA (m16n8k32) takes 16 weight rows × 32 columns
// as its A operand: lane 4g + t holds rows g and g + 8. The packed matrix is
// cut into blocks of 16 rows × 128 columns, 1024 bytes each, K blocks of a row
// block one after the other. Word (h, g, t, u) of a block (u fastest) holds
// row 16·rb + 8·h + g, columns 128·kb + 32·u + 8·t + (0..7), column 2·p + e of
// those at bit 4·p + 16·e. So lane 4g + t reads 16 contiguous bytes per row
// half (a warp reads 512 contiguous bytes), its four words lie in the four
// 32-column groups of the block, and word & 0x0F0F0F0F, (word >> 4) &
// 0x0F0F0F0F are its codes of columns (0, 4, 1, 5) and (2, 6, 3, 7) as bytes.
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
  int slab_rows, slab_more;       // row blocks per slab; the first slab_more have one more
  const uint8_t* digits;          // records of w4_digits_kernel [pass][kb][record], or null
};

// d = A·B + c.
__device__ __forceinline__ void mma_s8_16832(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                               uint32_t a3, uint32_t b0, uint32_t b1, const int (&c)[4]) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %11, %12, %13};"
      : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(c[0]), "r"(c[1]), "r"(c[2]), "r"(c[3]));
}

__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                               const float (&c)[4]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]),
        "f"(c[3]));
}

template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
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
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A float at `addr` of this CTA's shared memory, read from CTA `rank` of the cluster.
__device__ __forceinline__ float cluster_lds_f32(uint32_t addr, uint32_t rank) {
  uint32_t a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

constexpr int kW4Warps = 16;
constexpr int kW4Threads = 32 * kW4Warps;
constexpr size_t kW4SmemCap = 226 * 1024;
constexpr size_t kW4OutCap = 32 * 1024;       // sums of a slab
constexpr int kW4MaxCluster = 8;

// MMA column tiles of a pass and its tokens. Integer passes (NT > 0): an
// activation is three 8-bit digits, each in an MMA column of its own. With one or
// two tiles the columns are packed (token c/3, digit c mod 3); otherwise three
// tiles take the three digits of eight tokens, so that a lane holds a token's
// digits itself. bf16 passes (−NT tiles): a column is a token.
template <int NT>
struct W4Pass {
  static constexpr bool kFloat = NT < 0, kPlanar = NT >= 3;
  static constexpr int kTiles = kFloat ? -NT : NT;
  static constexpr int kTok = kFloat ? -8 * NT : kPlanar ? 8 * (NT / 3) : 8 * NT / 3;
  static constexpr int kSums = kPlanar ? 8 * (NT / 3) : 8 * kTiles;  // sums per weight row
  static constexpr int kParts = kFloat || kPlanar ? 1 : 3;           // of them per token
};

// Shared memory of a CTA, in bytes from its start.
struct W4Smem {
  uint32_t part;   // float [warp][2][16][sums]: a run's first and last shares
  uint32_t ring;   // [warp][stage]: codes, scales, zero points
  uint32_t out;    // float [row block][token][16], in a cluster
  uint32_t x;      // records of the CTA's K blocks
  uint32_t total;
};
// The activations of 128 columns: the digits' MMA columns, 128 bytes each, the
// sums of the groups (float [group][sum]) and what a digit, or 1 in fixed point,
// counts (float [sum]). A packed column has its digit's sum, |Σd| ≤ 2^14; a pair of
// three-tile tokens has four values, their fixed-point sums in multiples of 2^16 and the
// rests of those (|.| ≤ 2^15): all exact. A column's eight 16-byte pieces are
// swapped in pairs in odd columns, so that two columns (the eight lanes of a
// 16-byte read) fall on different banks. bf16 passes: the activations as they
// are, 256 bytes a token, its four-piece groups swapped in pairs in odd tokens.
template <int V, int NT>
struct W4Record {
  uint32_t dsum, cf, bytes;
  __host__ __device__ __forceinline__ explicit W4Record(int toks) {
    dsum = cf = bytes = 256 * toks;
    if (W4Pass<NT>::kFloat) return;
    dsum = 3 * toks * 128;
    cf = dsum + (W4Pass<NT>::kPlanar ? 2 : 1) * V * W4Pass<NT>::kSums * 4;
    bytes = cf + W4Pass<NT>::kSums * 4;
  }
};
template <int V>
__host__ __device__ constexpr int w4_stage_bytes() {
  return 1024 + 48 * V;
}
// Ring stages per warp: three where the scales make a stage longer, so that the
// longest rows fit for every group size, and for passes of 16 bf16 tokens. Those
// gain nothing from a fourth at any row length: 9, 16 and 32 tokens, K from 1024 to
// 11008, N = 4096 and 11008 take 0 to 5 % longer with it where it changes nothing
// else, and rows of 4096 and 8192 need twice the CTAs (16 tokens, 4096 -> 11008 15.9
// against 13.2 us, 8192 -> 4096 25.5 against 13.9). One token is where it pays
// (2048 -> 128256, groups of 64, 28.3 against 29.8 us; groups of 128 26.9 against 27.9).
// The launcher takes three for fp32 passes of more than five tokens, too, where
// those fit in one CTA or a pair and four do not (16 tokens, 2560 -> 6912 in groups of
// 64 13.9 us in pairs, 10.9 in single CTAs). In clusters of four it does not: their
// grid runs in two waves (16 tokens, 11008 -> 4096 47 us, 37 in clusters of eight).
template <int V, int NT>
__host__ __device__ constexpr int w4_stages() {
  return V == 4 || NT == -2 ? 3 : 4;
}
// KB: blocks of K of this CTA, at most; slab: row blocks, at most.
template <int V, int NT>
__host__ __device__ inline W4Smem w4_smem(int KB, int slab, int toks, int ranks, int stages) {
  using C = W4Pass<NT>;
  W4Smem s;
  s.part = 0;
  s.ring = s.part + 2 * kW4Warps * 16 * C::kSums * 4;
  s.out = s.ring + kW4Warps * stages * w4_stage_bytes<V>();
  s.x = s.out + (ranks > 1 ? slab * toks * 64 : 0);
  s.total = s.x + KB * W4Record<V, NT>(toks).bytes;
  return s;
}

// One warp's request of a block into a ring stage: two 16-byte pieces of codes
// per lane, one of scales or zero points where `aux`; nothing with `left` ≤ 0.
__device__ __forceinline__ void w4_request(uint32_t dst, const uint8_t* w, const uint8_t* aux, int left,
                                           int has_aux) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.gt.s32 p, %3, 0;\n\t"
      "setp.ne.and.s32 q, %4, 0, p;\n\t"
      "@p cp.async.cg.shared.global [%0], [%1], 16;\n\t"
      "@p cp.async.cg.shared.global [%0 + 512], [%1 + 512], 16;\n\t"
      "@q cp.async.cg.shared.global [%0 + 1024], [%2], 16;\n\t"
      "cp.async.commit_group;\n\t}" ::"r"(dst),
      "l"(w), "l"(aux), "r"(left), "r"(has_aux)
      : "memory");
}

// The warp whose run holds item i of `items` (runs as in the kernel).
__device__ __forceinline__ int w4_warp_of(int i, int items) {
  int w = i * kW4Warps / items;
  while (w + 1 < kW4Warps && items * (w + 1) / kW4Warps <= i) ++w;
  return w;
}

// Sum of token c, row r of a row block over the shares of warps w_lo..w_hi (the
// first in `slot_lo`, the others in their slot 0), lowest digit first.
template <int NT>
__device__ __forceinline__ float w4_gather(const float* part, int w_lo, int w_hi, int slot_lo, int r,
                                           int c) {
  constexpr int SUMS = W4Pass<NT>::kSums, P = W4Pass<NT>::kParts;
  float y = 0.f;
#pragma unroll
  for (int pc = P - 1; pc >= 0; --pc) {
    y += part[(slot_lo * 16 + r) * SUMS + c * P + pc];
    for (int w = w_lo + 1; w <= w_hi; ++w) y += part[(w * 32 + r) * SUMS + c * P + pc];
  }
  return y;
}

// Output j of a row block: row j mod 16 of token j/16 of the pass.
__device__ __forceinline__ void w4_store(const W4Params& p, int rb, int64_t m0, int j, float y) {
  const int64_t row = (int64_t)rb * 16 + (j & 15), at = (m0 + (j >> 4)) * p.N + row;
  if (row < p.N) {
    if (p.y_bf16)
      reinterpret_cast<__nv_bfloat16*>(p.Y)[at] = __float2bfloat16_rn(y);
    else
      reinterpret_cast<float*>(p.Y)[at] = y;
  }
}

// Eight activations of token m, columns 8·l .. 8·l + 7 of a 128-column block, into
// the block's record, as digits; the sixteen lanes of a block (half a warp) call
// together. f is the largest power of two with max|x|·f ≤ 127·2^16; x·f is
// rounded to a 24-bit integer d2·2^16 + d1·2^8 + d0 with digits in [−128, 127]
// (adding 0x808080 and flipping the same bits carries between them), and
// digit i counts 2^(8i)/f. The rounding, half of 1/f, is at most 1.21e-7 (2^-22.99)
// of the block's largest value: about what aligning to it in an fp32 sum loses.
template <int V, int NT>
__device__ __forceinline__ void w4_digits(const float (&v)[8], uint8_t* rec, const W4Record<V, NT>& R,
                                          int m, bool write) {
  constexpr bool PL = W4Pass<NT>::kPlanar;
  constexpr int SUMS = W4Pass<NT>::kSums, GL = 16 / V;  // GL lanes per group
  const int l = threadIdx.x & 15;
  uint32_t top = 0;  // largest magnitude, as bits: an infinity or NaN stays on top
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[j]) & 0x7FFFFFFFu);
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  // f = 2^e, at most 2^125: a block below 1e-31 keeps fewer bits
  const float f0 = __fdiv_rn(127.0f * 65536.0f, fmaxf(__uint_as_float(top), 1e-31f));
  const uint32_t fb = __float_as_uint(f0) & 0xFF800000u;
  const float f = __uint_as_float(fb);
  // 1/f, its exponent mirrored; an infinity or NaN makes the token's results NaN
  const float unit = __uint_as_float(top < 0x7F800000u ? 0x7F000000u - fb : 0x7FFFFFFFu);
  int fixed = 0;
  uint32_t outer = 0, middle = 0;
  uint32_t w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int n = __float2int_rn(__fmul_rn(v[j], f));
    const uint32_t b = (uint32_t)n + 0x808080u;  // its bytes are the digits + 128
    if (PL) fixed += n;
    if (NT == 1) {
      outer += b & 0x00FF00FFu;
      middle += (b >> 8) & 0xFFu;
    }
    w[j] = b ^ 0x808080u;
  }
  auto digit = [&](int d) {  // byte d of the eight words
    const uint32_t sel = d | ((4 + d) << 4);
    const uint32_t a04 = __byte_perm(w[0], w[4], sel), a15 = __byte_perm(w[1], w[5], sel);
    const uint32_t a26 = __byte_perm(w[2], w[6], sel), a37 = __byte_perm(w[3], w[7], sel);
    return make_uint2(__byte_perm(a04, a15, 0x5410), __byte_perm(a26, a37, 0x5410));
  };
  auto put = [&](int d, uint2 q) {
    const int xc = m * 3 + 2 - d;  // the highest digit first
    // [t][u][8 bytes], t = l mod 4, u = l / 4
    const uint32_t off = (((l & 3) * 2 + (l >> 3)) ^ (xc & 1)) * 16 + ((l >> 2) & 1) * 8;
    *reinterpret_cast<uint2*>(rec + xc * 128 + off) = q;
  };
  float* s = reinterpret_cast<float*>(rec + R.dsum);
  if constexpr (NT == 1) {
    // The digits' sums over a group, of bytes (≤ 2^15, so two fit side by side in a
    // word), before the digits are put together: with 64 registers that is 3 to 5 %
    // of a call of long rows faster than what follows for five tokens.
#pragma unroll
    for (int o = 1; o < GL; o <<= 1) {
      outer += __shfl_xor_sync(0xffffffffu, outer, o);
      middle += __shfl_xor_sync(0xffffffffu, middle, o);
    }
    if (!write) return;
#pragma unroll
    for (int d = 0; d < 3; ++d) put(d, digit(d));
    if (l % GL == 0) {
      constexpr int kBias = 128 * 8 * GL;
      s += (l / GL) * SUMS + 3 * m;
      s[0] = (float)((int)(outer >> 16) - kBias);
      s[1] = (float)((int)middle - kBias);
      s[2] = (float)((int)(outer & 0xFFFFu) - kBias);
    }
  } else {
    int sum[3];
#pragma unroll
    for (int d = 0; d < 3; ++d) {
      const uint2 q = digit(d);
      if (!PL) sum[d] = dp4a(q.y, 0x01010101u, dp4a(q.x, 0x01010101u, 0));
      if (write) put(d, q);
    }
    if constexpr (PL) {  // the token's sum, |fixed| ≤ 128·2^23
#pragma unroll
      for (int o = 1; o < GL; o <<= 1) fixed += __shfl_xor_sync(0xffffffffu, fixed, o);
      if (write && l % GL == 0) {
        s += ((l / GL) * SUMS + (m & ~1)) * 2 + (m & 1);
        const int high = (fixed + 32768) >> 16;
        s[0] = (float)high;
        s[2] = (float)(fixed - high * 65536);
      }
    } else {
      // The digits' sums. The first step leaves the two upper ones (≤ 2^14 each, side
      // by side in one word) to the group's lower lanes and the lowest one to
      // the upper lanes, so that one value per lane is left to add up.
      const bool up = (l & (GL / 2)) != 0;
      const int upper = sum[2] * 65536 + sum[1];
      int v1 = (up ? sum[0] : upper) + __shfl_xor_sync(0xffffffffu, up ? upper : sum[0], GL / 2);
#pragma unroll
      for (int o = 1; o < GL / 2; o <<= 1) v1 += __shfl_xor_sync(0xffffffffu, v1, o);
      if (write && l % (GL / 2) == 0) {
        s += (l / GL) * SUMS + 3 * m;
        if (up) {
          s[2] = (float)v1;
        } else {
          const int s1 = (int16_t)(v1 & 0xFFFF);
          s[0] = (float)((v1 - s1) >> 16);
          s[1] = (float)s1;
        }
      }
    }
    if (!write) return;
  }
  if (l == 0) {
    float* c = reinterpret_cast<float*>(rec + R.cf) + (PL ? m : 3 * m);
    if (!PL) {
      c[0] = __fmul_rn(unit, 65536.0f);
      c[1] = __fmul_rn(unit, 256.0f);
    }
    c[PL ? 0 : 2] = unit;
  }
}

// Eight activations as loaded, zeros where `in` is false. bf16 values stay as they
// are until they are needed: four registers instead of eight.
template <typename T>
struct W4Values {
  static constexpr int kWords = 2 * sizeof(T);
  uint32_t a[kWords];
  __device__ __forceinline__ void load(const T* p, bool in) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) a[i] = 0u;
    if (!in) return;
#pragma unroll
    for (int i = 0; i < kWords; i += 4) {
      if constexpr (sizeof(T) == 2) {  // volatile: the compiler would convert at once
        asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(a[i]), "=r"(a[i + 1]), "=r"(a[i + 2]), "=r"(a[i + 3]) : "l"(p));
      } else {
        const uint4 q = __ldg(reinterpret_cast<const uint4*>(p) + i / 4);
        a[i] = q.x; a[i + 1] = q.y; a[i + 2] = q.z; a[i + 3] = q.w;
      }
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[j] = sizeof(T) == 4 ? __uint_as_float(a[j % kWords])
                            : __uint_as_float(j & 1 ? a[j / 2] & 0xFFFF0000u : a[j / 2] << 16);
  }
};

// A CTA's own activations into shared memory, B blocks' loads in flight
// together.
template <typename T, int V, int NT, int B>
__device__ __forceinline__ void w4_stage_x(uint8_t* x, const W4Record<V, NT>& R, const T* X, int64_t K,
                                           int kb0, int KB, int toks) {
  const int units = KB * 16, total = units * toks;
  for (int i0 = threadIdx.x; i0 - (int)(threadIdx.x & 31) < total; i0 += B * kW4Threads) {
    W4Values<T> v[B];
    int tok[B], unit_of[B];
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int i = i0 + b * kW4Threads;
      tok[b] = toks == 1 ? 0 : i / units;
      unit_of[b] = i - tok[b] * units;
      const int64_t k = ((int64_t)kb0 * 16 + unit_of[b]) * 8;
      v[b].load(X + (int64_t)tok[b] * K + k, i < total && k < K);
    }
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int i = i0 + b * kW4Threads;
      if (i - (int)(threadIdx.x & 31) >= total) break;  // the same for the warp
      float x8[8];
      v[b].get(x8);
      w4_digits<V, NT>(x8, x + (unit_of[b] >> 4) * R.bytes, R, tok[b], i < total);
    }
  }
}

// bf16 activations into shared memory as they are, zeros past column K.
template <int V, int NT>
__device__ __forceinline__ void w4_copy_x(uint32_t x, const W4Record<V, NT>& R, const __nv_bfloat16* X,
                                          int64_t K, int kb0, int KB, int toks) {
  const int c = threadIdx.x & 15;
  for (int kb = threadIdx.x >> 4; kb < KB; kb += kW4Threads / 16) {
    const int64_t k = (int64_t)(kb0 + kb) * 128 + 8 * c;
    const int bytes = k < K ? 16 : 0;
    const __nv_bfloat16* src = X + (bytes ? k : 0);
    const uint32_t even = x + kb * R.bytes + 16 * c, odd = x + kb * R.bytes + 16 * (c ^ 4) + 256;
    auto copy = [&](uint32_t dst) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
      src += K;
    };
    int m = 0;
#pragma unroll 4
    for (; m + 1 < toks; m += 2) {
      copy(even + 256 * m);
      copy(odd + 256 * m);
    }
    if (m < toks) copy(even + 256 * m);
  }
}

// The records of all tokens and blocks in global memory, [pass][kb][record]:
// with more than a few tokens, making them again in every CTA would take longer
// than the product. One warp per two blocks of a token (blockIdx.y and on).
template <typename T, int V, int NT>
__global__ void __launch_bounds__(256)
w4_digits_kernel(const T* __restrict__ X, int64_t M, int64_t K, uint8_t* __restrict__ out) {
  constexpr int TOK = W4Pass<NT>::kTok;
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const int KB = (int)((K + 127) / 128), img = (int)min((int64_t)TOK, M);
  const W4Record<V, NT> R(img);
  const int kb = (int)(blockIdx.x * 16 + (threadIdx.x >> 4)), l = threadIdx.x & 15;
  for (int64_t m = blockIdx.y; m < M; m += gridDim.y) {
    const int64_t k = (int64_t)kb * 128 + 8 * l;
    W4Values<T> raw;
    raw.load(X + m * K + k, k < K);
    float v[8];
    raw.get(v);
    uint8_t* rec = out + ((m / TOK) * KB + kb) * (int64_t)R.bytes;
    w4_digits<V, NT>(v, rec, R, (int)(m % TOK), kb < KB);
  }
}

// Two codes in the low bits of their halves, as bf16, less 128 + z.
__device__ __forceinline__ uint32_t w4_centre(uint32_t w, uint32_t z) {
  const uint32_t q = (w & 0x000F000Fu) | 0x43004300u;
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&q),
                                   *reinterpret_cast<const __nv_bfloat162*>(&z));
  return *reinterpret_cast<const uint32_t*>(&d);
}

// Y = X·Wᵀ for up to W4Pass<NT>::kTok tokens per grid row.
//
// The product is one of integers: the codes as bytes against the activations'
// digits, Σ q·d − z·Σ d exact for a group and digit, then in fp32 times s and
// what the digit counts. What bounds a decode product here is the
// issue of instructions, not the tensor pipe (m16n8k16 of bf16 and m16n8k32 of
// int8 both take 8 cycles of it per sub-partition): as bytes, eight codes take
// three logic operations and half an MMA, as exact bf16 values (q − z)
// eleven and one. For 3 x 2048 -> 128256 that is 38.7 us against 31.9, and 6.5 to 6.9
// against 6.4 for 1 x 2560 -> 6912. Above five tokens, where the digits take three
// times the MMAs and a token's sums more fp32 work than the codes, bf16
// activations go through bf16 MMAs as they are: products are exact, a group's
// sum is the MMA's fp32 one. 16 x 4096 -> 11008 takes 13.4 us so, 19.9 in digits.
// The border at five is the head's; where a CTA has few row blocks making the
// digits costs more than the codes: 5 x 4096 -> 4096 in groups of 32 takes 12.1 us,
// 7.4 as bf16, and 2 x 11008 -> 4096 12.7 and 11.3.
//
// Each CTA owns a slab of 16-row blocks, contiguous in memory; its 16 warps
// take equal, contiguous runs of the slab's 1 KB blocks, so the load is even
// whatever the shape. The sums of a row block that a run holds whole are
// complete; the first and the last, which it may share with its neighbours,
// meet in shared memory at the end, in the order of the warps. The CTAs of a
// cluster share a slab: each takes a range of K, so that its activations fit
// in shared memory, and the slab's sums meet there, in the order of the CTAs.
//
// Measured (one B200, calls in a graph): 1 x 2560 -> 6912 6.5 us and
// 4 x 512 -> 256 5.5 us, where a dependent launch, one trip for the activations
// and one for the weights are what is left; 3 x 2048 -> 128256 32 us, 4.3 TB/s, 67 %
// of the copy rate, the issue slots 64 % full; 16 x 4096 -> 11008 with zero points
// and groups of 64 13.4 us from bf16, no unit above 45 %: the one CTA of an SM
// waits for all its activations before the first MMA (19.9 us from fp32 with the
// launch that makes the digits, 24 MMAs per 1 KB block).
template <typename T, int V, int NT, int D>
__global__ void __launch_bounds__(kW4Threads, NT == 1 ? 2 : 1) w4_linear_kernel(const W4Params p) {
  using C = W4Pass<NT>;
  constexpr int SUMS = C::kSums, TOK = C::kTok, ST = w4_stage_bytes<V>();
  constexpr int NA = SUMS / 8, TILES = C::kTiles;  // accumulator tiles
  extern __shared__ __align__(128) uint8_t w4_mem[];
  const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int ranks = (int)cluster_size(), rank = (int)cluster_rank();
  // Blocks are counted in 32 bits: 2^31 of them are 2 TB.
  const int KBt = (int)((p.K + 127) / 128);
  const int slab = (int)blockIdx.x >> (31 - __clz(ranks));  // ranks is a power of two
  const int rb0 = slab * p.slab_rows + min(slab, p.slab_more);
  const int nrb = p.slab_rows + (slab < p.slab_more ? 1 : 0);
  const int kb0 = KBt * rank / ranks, KB = KBt * (rank + 1) / ranks - kb0;
  const int items = nrb * KB;
  const int it0 = items * warp / kW4Warps, it1 = items * (warp + 1) / kW4Warps;
  const int64_t m0 = (int64_t)blockIdx.y * TOK;
  const int toks = (int)min((int64_t)TOK, p.M - m0);
  const W4Smem L = w4_smem<V, NT>((KBt + ranks - 1) / ranks, p.slab_rows + (p.slab_more > 0 ? 1 : 0),
                                  (int)min((int64_t)TOK, p.M), ranks, D);
  float* part = reinterpret_cast<float*>(w4_mem + L.part);
  float* out = reinterpret_cast<float*>(w4_mem + L.out);

  pdl_launch_dependents();
  // Requests run ahead of the compute loop: 1024 bytes of codes, two pieces
  // per lane, and 32·V bytes of scales and 16·V of zero points by the first
  // lanes. The first ones go out before the wait for the previous kernel,
  // which does not write the weights.
  const bool is_scale = lane < 2 * V;
  const int has_aux = is_scale || (lane < 3 * V && p.zeros != nullptr);
  const uint32_t aux_step = is_scale ? 32 * V : 16 * V;
  const uint8_t* w_src = p.W4 + 16 * lane;
  const uint8_t* aux_src = is_scale ? reinterpret_cast<const uint8_t*>(p.scales) + 16 * lane
                                    : p.zeros + 16 * (lane - 2 * V);
  const uint32_t ring = smem_u32(w4_mem) + L.ring + warp * (D * ST);
  int q_kb = it0 % KB, left = it1 - it0;  // every CTA has a block of K: clusters are for long rows
  uint32_t q_blk = (uint32_t)(rb0 + it0 / KB) * KBt + kb0 + q_kb;
  auto request = [&](uint32_t dst) {
    w4_request(dst + 16 * lane, w_src + (uint64_t)q_blk * 1024u, aux_src + (uint64_t)q_blk * aux_step,
               left, has_aux);
    --left;
    ++q_blk;
    if (++q_kb == KB) {  // on to the next row block, past the other CTAs' blocks
      q_kb = 0;
      q_blk += KBt - KB;
    }
  };
#pragma unroll
  for (int d = 0; d < D - 1; ++d) request(ring + d * ST);
  pdl_wait_prior_grid();

  const int img = (int)min((int64_t)TOK, p.M);
  const W4Record<V, NT> R(img);
  uint8_t* x = w4_mem + L.x;
  if constexpr (C::kPlanar) {
    const uint8_t* rec = p.digits + ((int64_t)blockIdx.y * KBt + kb0) * R.bytes;
    for (uint32_t i = 16 * tid; i < KB * R.bytes; i += 16 * kW4Threads) cp_async16(smem_u32(x) + i, rec + i);
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if constexpr (C::kFloat) {
    const auto* X = reinterpret_cast<const __nv_bfloat16*>(p.X) + m0 * p.K;
    w4_copy_x<V, NT>(smem_u32(x), R, X, p.K, kb0, KB, toks);
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    const T* X = reinterpret_cast<const T*>(p.X) + m0 * p.K;
    if (KB * 16 * toks <= kW4Threads)
      w4_stage_x<T, V, NT, 1>(x, R, X, p.K, kb0, KB, toks);
    else
      w4_stage_x<T, V, NT, 4>(x, R, X, p.K, kb0, KB, toks);
  }
  if (it0 == it1)  // fewer blocks than warps: an empty run adds nothing
    for (int j = lane; j < 16 * SUMS; j += 32) part[warp * 32 * SUMS + j] = 0.f;
  __syncthreads();

  // Digits of the lane's MMA columns 8n + g. Columns past the tokens repeat
  // another's: what they sum to is never read.
  uint32_t xaddr[TILES], xother[TILES];  // the two pieces of a lane's 32 bytes (bf16: even and odd ones)
#pragma unroll
  for (int n = 0; n < TILES; ++n) {
    int xc;
    if constexpr (C::kFloat) {
      xc = (8 * n + g) % toks;
      xaddr[n] = smem_u32(x) + xc * 256 + 16 * t + 64 * (xc & 1);
      xother[n] = smem_u32(x) + xc * 256 + 16 * t + 64 - 64 * (xc & 1);
      continue;
    }
    if constexpr (C::kPlanar)
      xc = (8 * (n / 3) + g) % toks * 3 + n % 3;
    else
      xc = (8 * n + g) % (3 * toks);
    xaddr[n] = smem_u32(x) + xc * 128 + 16 * ((2 * t) ^ (xc & 1));
    xother[n] = xaddr[n] ^ 16u;
  }
  uint32_t sums = smem_u32(x) + R.dsum + (C::kPlanar ? 16 : 8) * t;
  // From the sums to what they count.
  const uint32_t CF = C::kPlanar ? 2 * V * SUMS * 4 - 8 * t : V * SUMS * 4;
  const bool zs = p.zeros != nullptr;
  // The bits of 1.5·2^23 in four registers, out of the compiler's sight: it would
  // set them anew for every group.
  int magic[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) asm volatile("mov.b32 %0, 0x4B400000;" : "=r"(magic[e]));

  uint32_t src = ring, last = ring + (D - 1) * ST;  // the next stage, the one before it
  int rb = it0 / KB, kb = it0 - rb * KB, slot = 0, at_kb = 0;
  for (int it = it0; it < it1;) {
    const int begin = kb, end = min(KB, kb + (it1 - it));  // this run's part of row block rb
    float acc[NA][4];
#pragma unroll
    for (int n = 0; n < NA; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
    if (begin != at_kb) {  // the addresses move on with the blocks
      const uint32_t move = (begin - at_kb) * R.bytes;
#pragma unroll
      for (int n = 0; n < TILES; ++n) {
        xaddr[n] += move;
        xother[n] += move;
      }
      sums += move;
    }
    for (; kb < end; ++kb) {
      // D − 1 blocks are under way; the oldest is next. Past the barrier every
      // lane sees it and is done with the stage before it, which is filled anew.
      cp_async_wait<D - 2>();
      __syncwarp();
      request(last);
      const uint4 wlo = lds128(src + 16 * lane), whi = lds128(src + 16 * lane + 512);
      const uint32_t lo[4] = {wlo.x, wlo.y, wlo.z, wlo.w}, hi[4] = {whi.x, whi.y, whi.z, whi.w};
      float s0[V], s1[V], z0[V], z1[V];
      uint32_t zz[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const uint32_t s = lds_u32(src + 1024 + (g * V + v) * 4);
        s0[v] = __uint_as_float(s << 16);
        s1[v] = __uint_as_float(s & 0xFFFF0000u);
        uint32_t z = 0x0808u;
        if (zs) z = lds_u16(src + 1024 + 32 * V + (g * V + v) * 2);
        zz[v] = z;
        // 2^23 + z has z in its low bits
        z0[v] = 8388608.0f - __uint_as_float(0x4B000000u | (z & 0xFFu));
        z1[v] = 8388608.0f - __uint_as_float(0x4B000000u | (z >> 8));
      }
      if constexpr (C::kFloat) {
        // (q − z) as exact bf16: the bits of 128 + q less 128 + z. Two MMAs of 16
        // columns per word: pairs (0, 1) and (2, 3) of the lane's eight.
        constexpr float zero[4] = {0.f, 0.f, 0.f, 0.f};
        float d[NA][4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          constexpr int L = 4 / V;  // words of a group
          const int v = u / L;
          const uint32_t b0 = __byte_perm(zz[v], 0x43u, 0x4040), b1 = __byte_perm(zz[v], 0x43u, 0x4141);
          uint32_t a[2][4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            a[q >> 1][(q & 1) * 2] = w4_centre(lo[u] >> (4 * q), b0);
            a[q >> 1][(q & 1) * 2 + 1] = w4_centre(hi[u] >> (4 * q), b1);
          }
#pragma unroll
          for (int n = 0; n < NA; ++n) {
            const uint4 b = lds128(((u & 1) ? xother[n] : xaddr[n]) + 128 * (u >> 1));
            if (u % L == 0)
              mma_bf16_16816(d[n], a[0], b.x, b.y, zero);
            else
              mma_bf16_16816(d[n], a[0], b.x, b.y, d[n]);
            mma_bf16_16816(d[n], a[1], b.z, b.w, d[n]);
            if (u % L == L - 1) {
              acc[n][0] = fmaf(d[n][0], s0[v], acc[n][0]);
              acc[n][1] = fmaf(d[n][1], s0[v], acc[n][1]);
              acc[n][2] = fmaf(d[n][2], s1[v], acc[n][2]);
              acc[n][3] = fmaf(d[n][3], s1[v], acc[n][3]);
            }
          }
        }
      } else {
        uint32_t a[4][4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          a[u][0] = lo[u] & 0x0F0F0F0Fu;
          a[u][1] = hi[u] & 0x0F0F0F0Fu;
          a[u][2] = (lo[u] >> 4) & 0x0F0F0F0Fu;
          a[u][3] = (hi[u] >> 4) & 0x0F0F0F0Fu;
        }
#pragma unroll
        for (int n = 0; n < NA; ++n) {
          constexpr int ND = C::kPlanar ? 3 : 1;  // tiles of this accumulator: digits, or one
          // The sums start at the bits of the float 1.5·2^23: what they end as, read
          // as a float, less 1.5·2^23 is the sum (|sum| < 2^18).
          int d[ND][V][4];
#pragma unroll
          for (int j = 0; j < ND; ++j) {
            const int tile = n * ND + j;
            const uint4 x0 = lds128(xaddr[tile]), x1 = lds128(xother[tile]);
            const uint32_t b[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
            for (int v = 0; v < V; ++v) {
#pragma unroll
              for (int u = v * (4 / V); u < (v + 1) * (4 / V); ++u) {
                if (u == v * (4 / V))
                  mma_s8_16832(d[j][v], a[u][0], a[u][1], a[u][2], a[u][3], b[2 * u], b[2 * u + 1], magic);
                else
                  mma_s8_16832(d[j][v], a[u][0], a[u][1], a[u][2], a[u][3], b[2 * u], b[2 * u + 1], d[j][v]);
              }
            }
          }
          const uint2 cq = lds64(sums + CF + 32 * n);
          const float c0 = __uint_as_float(cq.x), c1 = __uint_as_float(cq.y);
#pragma unroll
          for (int v = 0; v < V; ++v) {
            // Less z times the activations' sum, within the group and its digit: an
            // exact integer below 2^19. What is scaled and added up is then
            // Σ (q − z)·d, and nothing of the size of z·Σ|x| is ever rounded. Three
            // tiles: the highest digit is less z times the sum's multiple of
            // 2^16, the two others join it, each sum exact below 2^24, and the sum's
            // rest goes last: off by 2^-24 of the group's result, or by nothing.
            float t0, t1, r0 = 0.f, r1 = 0.f;
            if constexpr (C::kPlanar) {
              const uint4 q = lds128(sums + (2 * v * SUMS + 16 * n) * 4);
              t0 = __uint_as_float(q.x);
              t1 = __uint_as_float(q.y);
              r0 = __uint_as_float(q.z);
              r1 = __uint_as_float(q.w);
            } else {
              const uint2 q = lds64(sums + (v * SUMS + 8 * n) * 4);
              t0 = __uint_as_float(q.x);
              t1 = __uint_as_float(q.y);
            }
            float y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float z = e < 2 ? z0[v] : z1[v];
              y[e] = fmaf(z, e & 1 ? t1 : t0, __int_as_float(d[0][v][e]) - 12582912.0f);
#pragma unroll
              for (int j = 1; j < ND; ++j) y[e] = fmaf(y[e], 256.0f, __int_as_float(d[j][v][e]) - 12582912.0f);
              if constexpr (C::kPlanar) y[e] = fmaf(z, e & 1 ? r1 : r0, y[e]);
            }
            acc[n][0] = fmaf(y[0], s0[v] * c0, acc[n][0]);
            acc[n][1] = fmaf(y[1], s0[v] * c1, acc[n][1]);
            acc[n][2] = fmaf(y[2], s1[v] * c0, acc[n][2]);
            acc[n][3] = fmaf(y[3], s1[v] * c1, acc[n][3]);
          }
        }
      }
#pragma unroll
      for (int n = 0; n < TILES; ++n) {
        xaddr[n] += R.bytes;
        xother[n] += R.bytes;
      }
      sums += R.bytes;
      last = src;
      src = src == ring + (D - 1) * ST ? ring : src + ST;
    }
    it += end - begin;
    at_kb = end;
    // The share of row block rb: slot 0 for the run's first, 1 for a later one.
    float* mine = part + ((warp * 2 + slot) * 16 + g) * SUMS + 2 * t;
#pragma unroll
    for (int n = 0; n < NA; ++n) {
      *reinterpret_cast<float2*>(mine + 8 * n) = make_float2(acc[n][0], acc[n][1]);
      *reinterpret_cast<float2*>(mine + 8 * n + 8 * SUMS) = make_float2(acc[n][2], acc[n][3]);
    }
    if (begin == 0 && end == KB) {  // whole
      __syncwarp();
      for (int j = lane; j < 16 * toks; j += 32) {
        const float y = w4_gather<NT>(part, warp, warp, warp * 2 + slot, j & 15, j >> 4);
        if (ranks > 1)
          out[rb * toks * 16 + j] = y;
        else
          w4_store(p, rb0 + rb, m0, j, y);
      }
      __syncwarp();
    }
    slot = 1;
    kb = 0;
    ++rb;
  }
  __syncthreads();
  // Row blocks that several runs share.
  for (int r = warp; r < nrb; r += kW4Warps) {
    const int w_lo = w4_warp_of(r * KB, items), w_hi = w4_warp_of(r * KB + KB - 1, items);
    if (w_lo == w_hi) continue;
    // the first of them may have begun in an earlier row block
    const int slot_lo = w_lo * 2 + (items * w_lo / kW4Warps < r * KB ? 1 : 0);
    for (int j = lane; j < 16 * toks; j += 32) {
      const float y = w4_gather<NT>(part, w_lo, w_hi, slot_lo, j & 15, j >> 4);
      if (ranks > 1)
        out[r * toks * 16 + j] = y;
      else
        w4_store(p, rb0 + r, m0, j, y);
    }
  }
  if (ranks > 1) {
    __syncwarp();
    cluster_barrier();
    for (int r = warp * ranks + rank; r < nrb; r += kW4Warps * ranks) {
      for (int j = lane; j < 16 * toks; j += 32) {
        const uint32_t o = smem_u32(out + r * toks * 16 + j);
        float y = 0.f;
        for (int k = 0; k < ranks; ++k) y += cluster_lds_f32(o, k);
        w4_store(p, rb0 + r, m0, j, y);
      }
    }
    __syncwarp();
    cluster_barrier();  // the others may still read this CTA's sums
  }
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// ---------------------------------------------------------------------------
// Quantising, packing and unpacking. Sixteen lanes take the 128 columns of one
// row in a block, eight columns each (lane 4u + t): a warp reads 256 or 512
// contiguous bytes per row and a group's lanes are neighbours.

// Round(w ÷ s) to the nearest integer, ties to even, as for the exact
// quotient, |w| < 16·s. The product with a rounded 1/s is near enough to be off
// by one at most; the residual r = w − k·s is exact in fp32 (k·s has 5 + 8
// bits), so 2·|r| − s says whether k is the nearest: positive, it is off by
// one, zero, it is one side of a tie. Read as an integer plus the parity of k
// (the low bit of the sum with 1.5·2^23) it is positive exactly when k has to
// move towards r. s below 2^-60 comes scaled.
struct W4Rounder {
  float s, inv, up;
  __device__ __forceinline__ explicit W4Rounder(float scale) {
    // exact, and 1/s stays finite; a scale of 0 makes every value 0
    // (or NaN: whatever the codes, it reads back as NaN)
    up = scale > 0.f ? (scale < 0x1p-60f ? 0x1p80f : 1.0f) : 0.f;
    s = scale > 0.f ? scale * up : 0.f;
    inv = s > 0.f ? __fdividef(1.0f, s) : 0.f;
  }
  __device__ __forceinline__ float operator()(float w) const {
    w *= up;
    const float b = __fadd_rn(__fmul_rn(w, inv), 12582912.0f);
    const float k = b - 12582912.0f, r = fmaf(-k, s, w);
    const int c = __float_as_int(fmaf(2.0f, fabsf(r), -s)) + (int)(__float_as_uint(b) & 1u);
    const float moved = k + copysignf(1.0f, r);
    return c > 0 ? moved : k;
  }
};

// Extremes that a NaN in a group passes on to its scale.
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float m;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
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

// Word of eight codes given as floats 0..15: the bits of 2^23 + q are
// 0x4B000000 + q, and the shifted constants add up to one that is taken off.
__device__ __forceinline__ uint32_t w4_word(const float (&q)[8]) {
  uint32_t w = 0, off = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int sh = 4 * (j >> 1) + 16 * (j & 1);
    w += __float_as_uint(q[j] + 8388608.0f) << sh;
    off += 0x4B000000u << sh;
  }
  return w - off;
}

// Where the eight columns 8·l of row r (0..15) of block (rb, kb) are packed.
__device__ __forceinline__ int64_t w4_word_index(int64_t blk, int r, int l) {
  return blk * 256 + ((r * 4 + (l & 3)) * 4 + (l >> 2));
}
__device__ __forceinline__ int64_t w4_group_index(int64_t blk, int r, int v, int V) {
  return ((blk * 8 + (r & 7)) * V + v) * 2 + (r >> 3);
}

// One CTA per row block (blockIdx.x): sixteen lanes per row, K blocks
// blockIdx.y, + gridDim.y, ..., two of them under way at a time. Bound by issue
// (82 % full): 6912 x 2560 bf16 in groups of 128 takes 19.5 us (2.3 TB/s, 35 % of the
// copy rate), 4001 x 4160 fp32 with zero points in groups of 32 20.7 us (3.7 TB/s).
template <typename T, int G, bool ZP>
__global__ void __launch_bounds__(256)
w4_quant_kernel(const T* __restrict__ W, int64_t N, int64_t K, uint32_t* __restrict__ W4,
                __nv_bfloat16* __restrict__ scales, uint8_t* __restrict__ zeros) {
  const int KB = (int)((K + 127) / 128), l = threadIdx.x & 15, r = threadIdx.x >> 4;
  constexpr int V = 128 / G, gl = G / 8;
  const int64_t rb = blockIdx.x, n = rb * 16 + r;
  const T* row = W + n * K + 8 * l;
  constexpr int B = 2;
  for (int kb0 = blockIdx.y; kb0 < KB; kb0 += B * gridDim.y) {
    float v[B][8];
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int64_t k = (int64_t)(kb0 + b * (int)gridDim.y) * 128;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[b][j] = 0.f;
      if (n < N && k + 8 * l < K) w4_load8(row + k, v[b]);
    }
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int kb = kb0 + b * (int)gridDim.y;
      if (kb >= KB) break;  // the same for the CTA
      const int64_t blk = rb * KB + kb;
      float hi = 0.f, lo = 0.f;  // without zero points: hi of the magnitudes
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        hi = max_nan(hi, ZP ? v[b][j] : fabsf(v[b][j]));
        if (ZP) lo = min_nan(lo, v[b][j]);
      }
#pragma unroll
      for (int o = 1; o < gl; o <<= 1) {
        hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        if (ZP) lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      }
      const float raw = ZP ? __fdiv_rn(__fsub_rn(hi, lo), 15.0f) : __fdiv_rn(hi, 7.0f);
      const __nv_bfloat16 sb = __float2bfloat16_rn(raw);
      const W4Rounder round(__bfloat162float(sb));
      const float z = ZP ? fminf(round(-lo), 15.0f) : 8.0f;
      float q[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) q[j] = fminf(fmaxf(round(v[b][j]) + z, 0.0f), 15.0f);
      W4[w4_word_index(blk, r, l)] = w4_word(q);
      if (l % gl == 0) {
        scales[w4_group_index(blk, r, l / gl, V)] = sb;
        if (ZP) zeros[w4_group_index(blk, r, l / gl, V)] = (uint8_t)z;
      }
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
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = (float)((c >> (4 * j)) & 15u);
    W4[w4_word_index(blk, r, l)] = w4_word(q);
    if (l % gl == 0) {
      const int64_t o = w4_group_index(blk, r, l / gl, V), src = n * groups + k / G;
      scales[o] = in ? s_in[src] : __float2bfloat16_rn(0.0f);
      if (zeros != nullptr) zeros[o] = in ? (uint8_t)(z_in[src] & 15) : (uint8_t)0;
    }
  }
}

// The matrix the packed weights stand for: fl32(s·(q − z)) (exact: 8 + 5 bits),
// rounded once more for a bf16 output. CTAs as in the quantiser. Bound by HBM:
// 6912 x 2560 to fp32 takes 15.4 us (5.2 TB/s, 80 % of the copy rate), to bf16 11.8. `wide`: W is
// 32-byte aligned, and eight fp32 values go out in one store (whole sectors).
template <int G>
__global__ void __launch_bounds__(256)
w4_unpack_kernel(const uint32_t* __restrict__ W4, const __nv_bfloat16* __restrict__ scales,
                 const uint8_t* __restrict__ zeros, int64_t N, int64_t K, void* W, int w_bf16,
                 int wide) {
  const int KB = (int)((K + 127) / 128), l = threadIdx.x & 15, r = threadIdx.x >> 4;
  constexpr int V = 128 / G, gl = G / 8;
  const int64_t rb = blockIdx.x, n = rb * 16 + r;
  if (n >= N) return;
  constexpr int B = 4;
  for (int kb0 = blockIdx.y; kb0 < KB; kb0 += B * gridDim.y) {
    uint32_t w[B];
    float s[B], z[B];
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int kb = kb0 + b * (int)gridDim.y;
      w[b] = 0u;
      s[b] = z[b] = 0.f;
      if (kb * (int64_t)128 + 8 * l < K) {
        const int64_t blk = rb * KB + kb, o = w4_group_index(blk, r, l / gl, V);
        w[b] = __ldg(W4 + w4_word_index(blk, r, l));
        s[b] = __bfloat162float(scales[o]);
        // 2^23 + z
        z[b] = __uint_as_float(0x4B000000u | (zeros != nullptr ? __ldg(zeros + o) : 8u));
      }
    }
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int64_t k = (int64_t)(kb0 + b * (int)gridDim.y) * 128 + 8 * l;
      if (k >= K) break;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t q = (w[b] >> (4 * (j >> 1) + 16 * (j & 1))) & 15u;
        v[j] = __fmul_rn(s[b], __uint_as_float(0x4B000000u | q) - z[b]);
      }
      if (w_bf16) {
        *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(W) + n * K + k) =
            make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                       pack_bf16x2(v[6], v[7]));
      } else {
        float* out = reinterpret_cast<float*>(W) + n * K + k;
        if (wide) {
          asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(out), "f"(v[0]),
                       "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                       : "memory");
        } else {
          reinterpret_cast<float4*>(out)[0] = make_float4(v[0], v[1], v[2], v[3]);
          reinterpret_cast<float4*>(out)[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
      }
    }
  }
}

}  // namespace bl
