// The launch before the attention kernel of a prefill on an FP8 or INT4 cache.
// The call's K rows are rotated, K and V rows quantised into the cache, and
// the bf16 rows that they and the cached ones before them stand for written to
// the workspace, which the attention kernel then reads like a bf16 cache; the
// queries are staged, rotated, in the output buffer where that kernel wants
// them so. Bound by the workspace's writes (4 d bytes a position and KV head: 86
// MB for 512 rows behind 16,384 of 2 sequences); in one launch, because for a chunk of
// some hundred rows each further one costs as much as its work: three launches
// (rotate, quantise, read back) took 18.5 us for 777 rows of 3 sequences on an
// FP8 cache, 25 us for 512 rows behind 16,384 of 2 sequences on an INT4 cache;
// this one takes 10 and 21.
#pragma once

#include "fp8.cuh"
#include "int4.cuh"
#include "rope.cuh"

namespace sa {

struct QuantStageParams {
  void* ck;
  void* cv;
  void* cks;
  void* cvs;
  int B, n_kv, n_q, cap;
  int row_old, row_new;   // cache rows of the first position attended and of the call's first
  int prefix, T;          // cached rows before the call's, and the call's
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  long long ks0, ks1, ks2, vs0, vs1, vs2;
  int rope;
  const float* cos_t;     // table rows of the call's first position
  const float* sin_t;
  __nv_bfloat16* wk;      // workspace [B][n_kv][prefix + T][d]
  __nv_bfloat16* wv;
  const __nv_bfloat16* q;
  long long qs0, qs1, qs2;
  __nv_bfloat16* qo;
  long long os0, os1, os2;
  int blocks_new, blocks_old;   // per (sequence, KV head)
  int n_new, n_old;             // in all; blocks behind them stage queries
};

template <int D, bool F8>
__global__ void __launch_bounds__(256) quant_stage_kernel(const QuantStageParams p) {
  using C = RowsCfg<D>;
  constexpr int HALF = D / 2, PC = D / 16, NR = 4;
  __shared__ __align__(16) __nv_bfloat16 rot[C::RB * D];
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x;
  const int rb = tid / C::CH, ch = tid - rb * C::CH;
  const long long w_rows = (long long)p.prefix + p.T;
  int blk = blockIdx.x;
  if (blk < p.n_new) {
    // ------------------------------------------------------------ the call's rows
    const int bg = blk / p.blocks_new, t0 = (blk - bg * p.blocks_new) * C::RB;
    const int b = bg / p.n_kv, g = bg - b * p.n_kv;
    const __nv_bfloat16* v = p.v + b * p.vs0 + g * p.vs2;
    const int t = t0 + rb;
    const bool live = rb < C::RB && t < p.T;
    uint4 vw = make_uint4(0, 0, 0, 0);
    if (!F8 && live) vw = *reinterpret_cast<const uint4*>(v + t * p.vs1 + 8 * ch);
    if (tid < C::RB * PC) {
      const int r = tid / PC, c = tid - r * PC;
      if (t0 + r < p.T) {
        const __nv_bfloat16* src = p.k + b * p.ks0 + (t0 + r) * p.ks1 + g * p.ks2 + 8 * c;
        uint4 x1 = *reinterpret_cast<const uint4*>(src), x2 = *reinterpret_cast<const uint4*>(src + HALF);
        if (p.rope) {
          const long long at = (long long)(t0 + r) * HALF + 8 * c;
          rotate8(x1, x2, p.cos_t + at, p.sin_t + at);
        }
        *reinterpret_cast<uint4*>(rot + r * D + 8 * c) = x1;
        *reinterpret_cast<uint4*>(rot + r * D + HALF + 8 * c) = x2;
      }
    }
    __syncthreads();
    if constexpr (F8) {
      const int lane = tid & 31;
      for (int r = tid >> 5; r < C::RB && t0 + r < p.T; r += 8) {
        float xk[2][2], xv[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int c = 2 * lane + 64 * i;
          uint32_t a = 0, e = 0;
          if (c < D) {
            a = *reinterpret_cast<const uint32_t*>(rot + r * D + c);
            e = *reinterpret_cast<const uint32_t*>(v + (t0 + r) * p.vs1 + c);
          }
          xk[i][0] = bf16_lo(a);
          xk[i][1] = bf16_hi(a);
          xv[i][0] = bf16_lo(e);
          xv[i][1] = bf16_hi(e);
        }
        long long row = (long long)p.row_new + t0 + r;
        if (row >= p.cap) row -= p.cap;
        const long long at = (long long)bg * p.cap + row, w = bg * w_rows + p.prefix + t0 + r;
        uint16_t ck[2], cv[2];
        const float sk = quantize_row_warp<2>(xk, D, static_cast<uint8_t*>(p.ck) + at * D, lane, ck);
        const float sv = quantize_row_warp<2>(xv, D, static_cast<uint8_t*>(p.cv) + at * D, lane, cv);
        if (lane == 0) {
          static_cast<float*>(p.cks)[at] = sk;
          static_cast<float*>(p.cvs)[at] = sv;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int c = 2 * lane + 64 * i;
          if (c < D) {
            *reinterpret_cast<uint32_t*>(p.wk + w * D + c) = f8_pair_bf16(ck[i], sk);
            *reinterpret_cast<uint32_t*>(p.wv + w * D + c) = f8_pair_bf16(cv[i], sv);
          }
        }
      }
    } else {
      uint4 kw = make_uint4(0, 0, 0, 0);
      if (live) kw = *reinterpret_cast<const uint4*>(rot + rb * D + 8 * ch);
      uint16_t sk, sv;
      const uint32_t ck = i4_quantise8(kw, sk), cv = i4_quantise8(vw, sv);
      if (live) {
        long long row = (long long)p.row_new + t;
        if (row >= p.cap) row -= p.cap;
        const long long at = (long long)bg * p.cap + row, w = bg * w_rows + p.prefix + t;
        static_cast<uint32_t*>(p.ck)[at * C::CH + ch] = ck;
        static_cast<uint32_t*>(p.cv)[at * C::CH + ch] = cv;
        if ((ch & 3) == 0) {
          static_cast<uint16_t*>(p.cks)[at * C::NB + ch / 4] = sk;
          static_cast<uint16_t*>(p.cvs)[at * C::NB + ch / 4] = sv;
        }
        *reinterpret_cast<uint4*>(p.wk + w * D + 8 * ch) = i4_dequantise8(ck, sk);
        *reinterpret_cast<uint4*>(p.wv + w * D + 8 * ch) = i4_dequantise8(cv, sv);
      }
    }
    return;
  }
  blk -= p.n_new;
  if (blk < p.n_old) {
    // ------------------------------------------------------------ the cached rows
    constexpr int KIND = F8 ? ROWS_FP8 : ROWS_INT4;
    const int bg = blk / p.blocks_old, t0 = (blk - bg * p.blocks_old) * (C::RB * NR) + rb;
    if (rb >= C::RB) return;
    StoredRow8<KIND> kr[NR], vr[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int t = t0 + i * C::RB;
      long long row = (long long)p.row_old + t;
      if (row >= p.cap) row -= p.cap;
      const long long at = (long long)bg * p.cap + row;
      if (t < p.prefix) {
        kr[i] = load_row8<D, KIND>(p.ck, p.cks, at, ch);
        vr[i] = load_row8<D, KIND>(p.cv, p.cvs, at, ch);
      }
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int t = t0 + i * C::RB;
      if (t < p.prefix) {
        const long long w = (bg * w_rows + t) * D + 8 * ch;
        *reinterpret_cast<uint4*>(p.wk + w) = row8_bf16<KIND>(kr[i]);
        *reinterpret_cast<uint4*>(p.wv + w) = row8_bf16<KIND>(vr[i]);
      }
    }
    return;
  }
  // ------------------------------------------------------------ the queries
  const long long n = (long long)p.B * p.T * p.n_q * PC;
  const bool narrow = n <= 0xffffffffLL;
  const long long step = (long long)(gridDim.x - p.n_new - p.n_old) * 256;
  for (long long idx = (long long)(blk - p.n_old) * 256 + tid; idx < n; idx += step) {
    int b, t, h, c;
    split_row_chunk(idx, narrow, PC, p.n_q, p.T, b, t, h, c);
    const __nv_bfloat16* src = p.q + b * p.qs0 + t * p.qs1 + h * p.qs2 + 8 * c;
    __nv_bfloat16* dst = p.qo + b * p.os0 + t * p.os1 + h * p.os2 + 8 * c;
    uint4 x1 = *reinterpret_cast<const uint4*>(src), x2 = *reinterpret_cast<const uint4*>(src + HALF);
    const long long at = (long long)t * HALF + 8 * c;
    rotate8(x1, x2, p.cos_t + at, p.sin_t + at);
    *reinterpret_cast<uint4*>(dst) = x1;
    *reinterpret_cast<uint4*>(dst + HALF) = x2;
  }
}

}  // namespace sa
