// What the two products of few tokens share (lora_few.hip, lora_few_back.hip):
// a wave's 16·MT tokens x 128 outputs on the matrix cores, with the packed
// weights turned into operands between the MFMAs, and the meeting of a
// workgroup's four waves.
#pragma once

#include "gemm_types.h"
#include "lora_common.h"
#include "lora_stage.h"

namespace awq {
namespace {

constexpr int kFewWaves = 4;
constexpr int kFewCols = 128;     // outputs per workgroup

typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

// Per wave: 16·MT tokens x 64 channels (rows of 8 chunks of 16 bytes, chunk c of
// row i at c ^ (i / 2) % 8).
template <int MT>
using FewX = uint4[kFewWaves][16 * MT * 8];

// The copies of a stage of the activations, and its reads. Rows past T are zero,
// or, in a 16-row block past T, the last block's: they are never stored.
struct FewRows {
  __amdgpu_buffer_rsrc_t rs;
  uint32_t off[2];     // copy i takes rows 8i .. + 7: the swizzle repeats every 16
  uint32_t at[2];      // the lane's operand of block h
  int step, last;
};
template <int MT>
__device__ __forceinline__ FewRows few_rows(const uint16_t* X, int64_t t0, int64_t T,
                                                int64_t ld) {
  FewRows f;
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const int rows = int(T - t0 < 16 * MT ? T - t0 : 16 * MT);
  f.rs = rows_rsrc(X + t0 * ld, rows, ld);
  f.last = (rows - 1) / 16;
  f.step = int(16 * ld * 2);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = 8 * i + (lane >> 3);
    f.off[i] = uint32_t((row * ld + ((lane & 7) ^ (row >> 1)) * 8) * 2);
    f.at[i] = uint32_t(lr * 8 + ((4 * i + lg) ^ (lr >> 1)));
  }
  return f;
}
template <int MT>
__device__ __forceinline__ void few_copy_rows(const FewRows& f, uint4* stage, int k) {
#pragma unroll
  for (int i = 0; i < 2 * MT; ++i)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(f.rs, AWQ_LORA_LDS(stage + 64 * i), 16, f.off[i & 1],
                                             (i / 2 < f.last ? i / 2 : f.last) * f.step + 2 * k,
                                             0, 0);
}

// A pair before its rounding: two float32 numbers, or (fp16) what it is.
template <bool F16>
__device__ __forceinline__ uint32_t few_round(uint32_t lo, uint32_t hi) {
  if constexpr (F16) return lo;
  else return pack2<false>(__builtin_bit_cast(float, lo), __builtin_bit_cast(float, hi));
}

// The accumulators stay in AGPRs through inline asm: 128 of them among the
// vector registers make the allocator spill at two waves per SIMD. The
// compiler puts no wait states around asm: FIRST (the operand was just
// written) waits for two, and few_settle for the reads at the end.
template <bool FIRST>
__device__ __forceinline__ void mfma_few(floatx4& c, const bf16x8_t& a, const bf16x8_t& b) {
  if constexpr (FIRST)
    asm volatile("s_nop 1\n\tv_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
  else asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}
template <bool FIRST>
__device__ __forceinline__ void mfma_few(floatx4& c, const f16x8_t& a, const f16x8_t& b) {
  if constexpr (FIRST)
    asm volatile("s_nop 1\n\tv_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
  else asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}
template <int MT>
__device__ __forceinline__ void few_settle(floatx4 (&acc)[8][MT]) {
  asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
#pragma unroll
  for (int r = 0; r < 8; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) asm volatile("" : "+a"(acc[r][m]));
}

// Operand R's MFMAs, 4 / MT pairs of operand R + 1 before each: a matrix
// instruction takes as long as four vector instructions, which go on beside
// it. A pair is rounded a step after it is made (the wait between the two
// would be a cycle lost). W::pair<R, E>(lo, hi) makes word W::word(E) of operand
// R; it is called for R = 0, E = 0, 1, .. in order.
template <bool F16, int MT, int R, int M, class W, class V>
__device__ __forceinline__ void few_mfmas(W& w, const V (&xv)[MT], const V& b,
                                          uint32_t (&nb)[4], uint32_t (&f)[2],
                                          floatx4 (&acc)[MT]) {
  if constexpr (M < MT) {
    if constexpr (R < 7) {
      constexpr int kE = 4 / MT;
      uint32_t g[2];
      w.template pair<R + 1, M * kE>(g[0], g[1]);
      if constexpr (M > 0) nb[W::word(M * kE - 1)] = few_round<F16>(f[0], f[1]);
      if constexpr (kE == 2) {
        w.template pair<R + 1, M * kE + 1>(f[0], f[1]);
        nb[W::word(M * kE)] = few_round<F16>(g[0], g[1]);
      } else {
        f[0] = g[0];
        f[1] = g[1];
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    mfma_few<M == 0>(acc[M], xv[M], b);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (R < 7 && M == MT - 1) nb[W::word(3)] = few_round<F16>(f[0], f[1]);
    few_mfmas<F16, MT, R, M + 1>(w, xv, b, nb, f, acc);
  }
}
template <bool F16, int MT, int R, class W, class V>
__device__ __forceinline__ void few_operands(W& w, const V (&xv)[MT], uint32_t (&b)[4],
                                             floatx4 (&acc)[8][MT]) {
  if constexpr (R < 8) {
    uint32_t nb[4] = {}, f[2] = {};
    few_mfmas<F16, MT, R, 0>(w, xv, __builtin_bit_cast(V, make_uint4(b[0], b[1], b[2], b[3])), nb,
                             f, acc[R]);
    few_operands<F16, MT, R + 1>(w, xv, nb, acc);
  }
}
// A block of 32 rows of the contraction.
template <bool F16, int MT, class W, class V>
__device__ __forceinline__ void few_block(W& w, const V (&xv)[MT], floatx4 (&acc)[8][MT]) {
  uint32_t b[4], f[4][2];
  w.template pair<0, 0>(f[0][0], f[0][1]);
  w.template pair<0, 1>(f[1][0], f[1][1]);
  w.template pair<0, 2>(f[2][0], f[2][1]);
  w.template pair<0, 3>(f[3][0], f[3][1]);
#pragma unroll
  for (int e = 0; e < 4; ++e) b[W::word(e)] = few_round<F16>(f[e][0], f[e][1]);
  few_operands<F16, MT, 0>(w, xv, b, acc);
}

}  // namespace
}  // namespace awq

// The waves meet in LDS, a quarter of the operands (2u, 2u + 1) at a time: in
// step i wave w adds quarter (w + i) % 4, so all four work and an output's
// order depends on nothing but its column. store(u, m, x) gets the totals of
// operands 2u and 2u + 1 and of the 16 tokens m. (A macro: as a function the
// compiler joins the quarters' branches through a pointer to the accumulators,
// and they end up in memory.)
#define AWQ_FEW_MEET(acc, sx, wave, lane, MT, store)                                         \
  {                                                                                          \
    floatx4* const red_ = reinterpret_cast<floatx4*>(&sx) + lane;                            \
    __syncthreads();                                                                         \
    _Pragma("unroll") for (int i_ = 0; i_ < 4; ++i_) {                                       \
      _Pragma("unroll") for (int u_ = 0; u_ < 4; ++u_) {                                     \
        if (((wave + i_) & 3) != u_) continue;                                               \
        _Pragma("unroll") for (int m_ = 0; m_ < MT; ++m_) {                                  \
          floatx4 x_[2];                                                                     \
          _Pragma("unroll") for (int r_ = 0; r_ < 2; ++r_) {                                 \
            floatx4* const at_ = red_ + ((2 * u_ + r_) * MT + m_) * 64;                      \
            x_[r_] = acc[2 * u_ + r_][m_];                                                   \
            if (i_) x_[r_] += *at_;                                                          \
            if (i_ < 3) *at_ = x_[r_];                                                       \
          }                                                                                  \
          if (i_ == 3) store(u_, m_, x_);                                                    \
        }                                                                                    \
      }                                                                                      \
      if (i_ < 3) __syncthreads();                                                           \
    }                                                                                        \
  }
