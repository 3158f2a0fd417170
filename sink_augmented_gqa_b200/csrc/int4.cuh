// INT4 KV cache: rows stored as 4-bit codes with one bf16 scale per block of
// 32 elements, 4.5 bits an element, and the kernels that write such rows and
// read quantised rows back.
//
// A block of 32 bf16 values x with m its element of largest magnitude (the
// positive one of two opposite ones) is kept as
//   s = -m / 8 rounded to 5 significant bits (nearest, ties to even), bf16
//   u = min(15, floor(x / s + 8.5)),  0 <= u <= 15
// and stands for s (u - 8). The scale carries the sign that sends m to the
// code 0, the one end of the range that has a step more: with the step
// |m| / 8 instead of |m| / 7 the error of the other elements is an eighth
// smaller, and only elements beyond 7.5 / 8 of m with the opposite sign are
// clipped (by less than a step). s has 5 significant bits and u - 8 at most
// 3, so every stored value is exactly a bf16 number: all readers see the
// same rows (decode multiplies codes and scales apart, the read-back returns
// bf16), and rows read back and appended again give the same codes, because
// the element coded 0 stands for -8 s, whose eighth is s.
// A block whose largest magnitude is under 2^-120 is kept as zeros (scale 0,
// codes 8); a block with an infinity or a NaN reads back as 32 NaNs (scale
// NaN, codes 8).
//
// Codes lie in [B][n_kv][cap][d / 2] bytes, element 2 i of a row in the low
// half of byte i and element 2 i + 1 in the high half; scales in
// [B][n_kv][cap][d / 32] bf16.
#pragma once

#include "fp8.cuh"
#include "ptx.cuh"
#include "rope.cuh"

namespace sa {

constexpr int kI4Block = 32;

// Quantises 8 consecutive elements per lane (bf16 pairs in v); the four lanes
// of an aligned group of four hold one block. Returns the 8 codes as a word,
// element i in bits 4i.., and the block's scale bits (the same on all four).
// Every lane of the warp takes part.
__device__ __forceinline__ uint32_t i4_quantise8(uint4 v, uint16_t& scale) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  // 16-bit keys (magnitude << 1 | positive): their maximum is m, infinities
  // and NaNs above every number
  uint32_t key = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    key = __vmaxu2(key, ((w[i] << 1) & 0xFFFEFFFEu) | ((~w[i] >> 15) & 0x00010001u));
  key = __vmaxu2(key, __shfl_xor_sync(0xffffffffu, key, 1));
  key = __vmaxu2(key, __shfl_xor_sync(0xffffffffu, key, 2));
  key = max(key & 0xFFFFu, key >> 16);
  const uint32_t mag = key >> 1;
  if (mag >= 0x7F80u) {
    scale = 0x7FC0u;
    return 0x88888888u;
  }
  if (mag < 0x0380u) {   // 2^-120
    scale = 0;
    return 0x88888888u;
  }
  // |m| / 8 (three off the exponent, exact), then the 7 fraction bits rounded to 4
  uint32_t sb = mag - (3u << 7);
  sb = (sb + 3u + ((sb >> 3) & 1u)) & ~7u;
  sb |= (key & 1u) << 15;
  scale = (uint16_t)sb;
  // floor(x / s + 8.5) by the reciprocal: x and s have 8 and 5 significant
  // bits, so x / s + 8.5 is an integer or at least 2^-9 away from one (checked
  // over all pairs), while fma(x, 1/s, .) is off by under 2^-18; with 2^-11
  // added, rounding x / s + 8 to the nearest integer gives that floor.
  const float r = __fdividef(1.0f, __uint_as_float(sb << 16));
  constexpr float MAGIC = 12582912.0f;   // 1.5 * 2^23: its sum's low bits are the rounded integer
  uint32_t word = 0;
#pragma unroll
  for (int i = 7; i >= 0; --i) {
    const float x = (i & 1) ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
    const float y = fminf(fmaf(x, r, 8.0f + 0x1p-11f), 15.0f) + MAGIC;
    word = (word << 4) + __float_as_uint(y);
  }
  // each term carried MAGIC's own bits 0x4B400000, at shifts 0, 4, .., 28
  constexpr uint32_t EXTRA = [] {
    uint32_t e = 0;
    for (int i = 0; i < 8; ++i) e = (e << 4) + 0x4B400000u;
    return e;
  }();
  return word - EXTRA;
}

// 8 codes (a word, element i in bits 4i..) and their block's scale to bf16
// pairs in order. 0x4300 | u is the bf16 number 128 + u; both packed
// operations after it are exact (see above).
__device__ __forceinline__ uint4 i4_dequantise8(uint32_t w, uint16_t scale) {
  const __nv_bfloat162 s2 = __halves2bfloat162(__ushort_as_bfloat16(scale), __ushort_as_bfloat16(scale));
  const __nv_bfloat162 c2 = __float2bfloat162_rn(-136.0f);
  uint32_t p[4];   // elements (i, i + 4)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t b = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
    const __nv_bfloat162 y = __hmul2(__hadd2(*reinterpret_cast<const __nv_bfloat162*>(&b), c2), s2);
    p[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
  return make_uint4(__byte_perm(p[0], p[1], 0x5410), __byte_perm(p[2], p[3], 0x5410),
                    __byte_perm(p[0], p[1], 0x7632), __byte_perm(p[2], p[3], 0x7632));
}

// A run of rows [T] of every (sequence, KV head) as bf16, and the cache rows
// they go to or come from: position index t is row (row0 + t), less cap once
// it passes the end of a ring.
struct RowsParams {
  const void* ck;   // codes, or bf16 rows
  const void* cv;
  const void* cks;  // scales: bf16 [..][d / 32] (INT4), fp32 (FP8)
  const void* cvs;
  const __nv_bfloat16* k;   // bf16 rows [B][T][n_kv][d]: the source of an append,
  const __nv_bfloat16* v;   // the destination of a read
  long long ks0, ks1, ks2, vs0, vs1, vs2;
  int T, n_kv, cap;
  int row0;
  int blocks_t;     // blocks of rows per (sequence, KV head)
};

// One thread per (row, 8 elements), K and V together; a block takes rows of
// one (sequence, KV head), so its codes and scales are one contiguous run
// and each row's 16-byte pieces are adjacent lanes.
template <int D>
struct RowsCfg {
  static constexpr int CH = D / 8;             // 8-element chunks of a row
  static constexpr int RB = 256 / CH;          // rows per block
  static constexpr int NB = D / kI4Block;
};

// Appends T bf16 rows to an INT4 cache.
template <int D>
__global__ void __launch_bounds__(256) kv_append_i4_kernel(const RowsParams p) {
  using C = RowsCfg<D>;
  const int bg = blockIdx.x / p.blocks_t;
  const int ch = threadIdx.x % C::CH, rb = threadIdx.x / C::CH;
  const int t = (blockIdx.x - bg * p.blocks_t) * C::RB + rb;
  const int b = bg / p.n_kv, g = bg - b * p.n_kv;
  const bool live = rb < C::RB && t < p.T;
  uint4 kw = make_uint4(0, 0, 0, 0), vw = kw;
  if (live) {
    kw = *reinterpret_cast<const uint4*>(p.k + b * p.ks0 + t * p.ks1 + g * p.ks2 + 8 * ch);
    vw = *reinterpret_cast<const uint4*>(p.v + b * p.vs0 + t * p.vs1 + g * p.vs2 + 8 * ch);
  }
  uint16_t sk, sv;
  const uint32_t ck = i4_quantise8(kw, sk), cv = i4_quantise8(vw, sv);
  if (!live) return;
  long long row = (long long)p.row0 + t;
  if (row >= p.cap) row -= p.cap;
  const long long at = (long long)bg * p.cap + row;
  reinterpret_cast<uint32_t*>(const_cast<void*>(p.ck))[at * C::CH + ch] = ck;
  reinterpret_cast<uint32_t*>(const_cast<void*>(p.cv))[at * C::CH + ch] = cv;
  if ((ch & 3) == 0) {
    reinterpret_cast<uint16_t*>(const_cast<void*>(p.cks))[at * C::NB + ch / 4] = sk;
    reinterpret_cast<uint16_t*>(const_cast<void*>(p.cvs))[at * C::NB + ch / 4] = sv;
  }
}

enum : int { ROWS_BF16 = 0, ROWS_FP8 = 1, ROWS_INT4 = 2 };

// code * scale rounded to bf16 once: the fp32 product towards zero, its last
// bit set where it was not exact (round to odd; 24 bits >= 8 + 2, so rounding
// that to bf16 makes no false tie). The remainder is exact while it is no
// subnormal; scales under 2^-90 go through fp64.
__device__ __forceinline__ float f8_product(float code, float scale) {
  const float p = __fmul_rz(code, scale);
  return __fmaf_rn(code, scale, -p) != 0.f ? __uint_as_float(__float_as_uint(p) | 1u) : p;
}

// Elements 8 ch.. of cache row `at` as bf16 pairs.
template <int D, int KIND>
__device__ __forceinline__ uint4 load_row8(const void* rows, const void* scales, long long at, int ch) {
  using C = RowsCfg<D>;
  if constexpr (KIND == ROWS_BF16) {
    return *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(rows) + at * D + 8 * ch);
  } else if constexpr (KIND == ROWS_INT4) {
    return i4_dequantise8(static_cast<const uint32_t*>(rows)[at * C::CH + ch],
                          static_cast<const uint16_t*>(scales)[at * C::NB + ch / 4]);
  } else {
    const uint2 c = static_cast<const uint2*>(rows)[at * C::CH + ch];
    const float s = static_cast<const float*>(scales)[at];
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t h = f16x2_from_e4m3x2((uint16_t)((i < 2 ? c.x : c.y) >> (16 * (i & 1))));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      if (s >= 0x1p-90f) {
        r[i] = pack_bf16(f8_product(f.x, s), f8_product(f.y, s));
      } else {
        r[i] = bf16_bits_from_f64((double)f.x * (double)s) | bf16_bits_from_f64((double)f.y * (double)s) << 16;
      }
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
  }
}

// Reads T positions of a cache back as bf16 rows.
template <int D, int KIND>
__global__ void __launch_bounds__(256) kv_read_kernel(const RowsParams p) {
  using C = RowsCfg<D>;
  const int bg = blockIdx.x / p.blocks_t;
  const int ch = threadIdx.x % C::CH, rb = threadIdx.x / C::CH;
  const int t = (blockIdx.x - bg * p.blocks_t) * C::RB + rb;
  if (rb >= C::RB || t >= p.T) return;
  const int b = bg / p.n_kv, g = bg - b * p.n_kv;
  long long row = (long long)p.row0 + t;
  if (row >= p.cap) row -= p.cap;
  const long long at = (long long)bg * p.cap + row;
  const uint4 kw = load_row8<D, KIND>(p.ck, p.cks, at, ch), vw = load_row8<D, KIND>(p.cv, p.cvs, at, ch);
  *reinterpret_cast<uint4*>(const_cast<__nv_bfloat16*>(p.k) + b * p.ks0 + t * p.ks1 + g * p.ks2 + 8 * ch) = kw;
  *reinterpret_cast<uint4*>(const_cast<__nv_bfloat16*>(p.v) + b * p.vs0 + t * p.vs1 + g * p.vs2 + 8 * ch) = vw;
}

}  // namespace sa
