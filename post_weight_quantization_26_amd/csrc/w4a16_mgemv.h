// The W4A16 / W3A16 decode on the matrix cores (w4a16.hip; beside low-rank
// adapters, lora_few.hip).
#pragma once

#include "device_common.h"
#include "gemm_types.h"

namespace awq {
namespace {

// ---------------------------------------------------------------------------
// decode on the matrix cores: exact integer codes against the activations
// ---------------------------------------------------------------------------
//
// Per group g of k rows, Σ_k x·ŵ = scale·Σ_k x·(q − z). The codes enter the
// MFMA as B = 1 + q/16, built from the bits: q goes into the top four
// mantissa bits of a 16-bit float of exponent 0 (bf16 0x3F80 | q << 3, fp16
// 0x3C00 | q << 6). Every x·B has at most 16 significant bits, so the
// v_mfma_f32_16x16x32 products are exact and P'[t][n] = Σ_k x[t][k]·B[k][n]
// is an ordinary float32 sum. One more MFMA against a column of ones gives
// S[t] = Σ_k x[t][k], and Σ_k x·(q − z) = 16·P' − (16 + z)·S. After each
// 32-row k-block a lane adds scale·(P' − ((16 + z)/16)·S) to its float32
// totals (scaled by 16 once at the end). Token rows past T read row 0 and
// are never stored.
//
// Operand layout (16x16x32): lane l holds 8 consecutive k (k = 8·(l/16) + e)
// of row l % 16 of A and of column l % 16 of B, and receives D[4·(l/16) + v]
// [l % 16] for v = 0..3. The contraction only needs A and B to agree on which
// k each (lane group, element) holds, so a lane loads k rows 8·(l/16) + e of
// its qweight words and each nibble position r of a word feeds its own MFMA:
// MFMA (c, r) covers output channels 8·(wc + c) + r over the 16 lanes' word
// columns wc. A is read straight from X (16 bytes per lane and k-block).
//
// Workgroup (cb, kc): 4 waves, 256 outputs (a lane owns 16: two adjacent
// 4-bit word columns, one 8-byte load per k row, or half of a 3-bit group of
// 32), k rows kc·4·kpw ..;
// wave w takes kpw of them (a multiple of 32), and the waves' totals meet in
// LDS in a fixed order before one float32 partial per (kc, t, n) is stored.
constexpr int kMgWaves = 4;
constexpr int kMgCols = 32;       // word columns per workgroup
constexpr int kMgMfma = 16;       // (c, r): 2 word columns x 8 nibbles per lane

// B = 1 + q/16 for nibble r of two qweight words (two consecutive k rows),
// packed as a pair of 16-bit floats (lo word in the low half). v_perm puts
// byte r/2 of each word at bits 0-7 and 16-23; one shift moves the nibble to
// the top four mantissa bits and one and-or masks it and sets the exponent.
// The other bytes perm and the shift bring along fall outside the mask.
template <bool F16, int R>
__device__ __forceinline__ uint32_t code_pair(uint32_t w_lo, uint32_t w_hi) {
  constexpr uint32_t b = R >> 1;
  const uint32_t x = __builtin_amdgcn_perm(w_hi, w_lo, 0x0C000C00u | ((4u + b) << 16) | b);
  // nibble at bits 0-3 (R even) or 4-7 (R odd) of each half -> mantissa top
  constexpr int kTop = F16 ? 6 : 3;          // lowest bit of the top 4 mantissa bits
  constexpr int kShift = kTop - 4 * (R & 1);
  const uint32_t y = kShift >= 0 ? (x << kShift) : (x >> -kShift);
  constexpr uint32_t kMask = F16 ? 0x03C003C0u : 0x00780078u;
  constexpr uint32_t kOne = F16 ? 0x3C003C00u : 0x3F803F80u;
  return (y & kMask) | kOne;
}

// The 3-bit layout keeps a 32-row group's codes in 3 words; the two lanes
// that share a group each load 2 of them (words 0-1 or 1-2) and funnel-shift
// their 64 bits right by 0 or 16, so that both hold their 16 codes at bits
// 3r .. 3r+2 of a 48-bit value (lo, hi): codes 0-9 in lo, 11-15 in hi, and
// code 10 across the two. B = 1 + q/16 for code R of two consecutive k rows,
// as code_pair: v_perm takes a 2-byte window holding the code from each
// row's word, one shift puts it at the mantissa bits of q/16 and one and-or
// masks it and sets the exponent (the bits the shift carries across the
// halves fall outside the mask).
template <bool F16, int R>
__device__ __forceinline__ uint32_t code3_pair(uint32_t lo_a, uint32_t hi_a, uint32_t lo_b,
                                               uint32_t hi_b, uint32_t one) {
  constexpr int kLow = F16 ? 6 : 3;          // lowest mantissa bit of q/16
  constexpr int b = R < 10 ? 3 * R : R > 10 ? 3 * R - 32 : 0;
  uint32_t wa, wb;
  if constexpr (R < 10) {
    wa = lo_a;
    wb = lo_b;
  } else if constexpr (R > 10) {
    wa = hi_a;
    wb = hi_b;
  } else {
    wa = __builtin_amdgcn_alignbit(hi_a, lo_a, 30);
    wb = __builtin_amdgcn_alignbit(hi_b, lo_b, 30);
  }
  constexpr uint32_t B0 = (b >> 3) < 2 ? uint32_t(b >> 3) : 2u;
  constexpr int kShift = b - 8 * int(B0) - kLow;
  const uint32_t x =
      __builtin_amdgcn_perm(wb, wa, B0 | ((B0 + 1u) << 8) | ((B0 + 4u) << 16) | ((B0 + 5u) << 24));
  const uint32_t y = kShift >= 0 ? (x >> kShift) : (x << -kShift);
  constexpr uint32_t kMask = (7u << kLow) | (7u << (16 + kLow));
  return (y & kMask) | one;
}

// Code r of a lane's aligned 48-bit value (lo, hi), as an integer.
template <int R>
__device__ __forceinline__ uint32_t code3_at(uint32_t lo, uint32_t hi) {
  if constexpr (R < 10) return (lo >> (3 * R)) & 7u;
  else if constexpr (R > 10) return (hi >> (3 * R - 32)) & 7u;
  else return __builtin_amdgcn_alignbit(hi, lo, 30) & 7u;
}

// Registers of one wave: totals per MFMA (c, r); four k-block slots (codes,
// activations, and the group parameters when the block opens a group: raw
// fp16 scale pairs and packed zero points), of which three are live at a
// time (two blocks are prefetched ahead); and the open group's scales and
// decoded zero points.
constexpr int kMgSlots = 4;

template <bool F16>
struct MgState {
  floatx4 tot[kMgMfma];
  floatx4 pacc[kMgMfma], sacc;  // the open group's MFMA sums P' and S
  uint2 w[kMgSlots][8];
  uint4 a[kMgSlots];
  uint4 ps0[kMgSlots], ps1[kMgSlots];
  uint2 pz[kMgSlots];
  uint4 s0, s1;
  float zf[kMgMfma];
};

// Block j (0..3) of a 128-row super-block starting at kb, for groups of G
// rows (a 128-row super-block holds whole groups, so j's place in its group
// is known here): at a group's first block take its parameters from the
// block's slot; prefetch block j + 2 into slot (j + 2) % 4 (with its group's
// parameters if it opens one); then S = Σ x and, per (c, r), P' = Σ x·B
// from zero, folded at once: tot += scale·(P' − ((16 + z)/16)·S). That is
// scale·(16·P' − (16 + z)·S) / 16 with the same rounding; the factor 16 is
// applied once at the end.
template <bool F16, int BITS, int G, int TV, int J, class LoadData, class LoadPar>
__device__ __forceinline__ void mg_block(MgState<F16>& st, int kb, const LoadData& load_data,
                                         const LoadPar& load_par, uint32_t one) {
  typedef typename Operand<F16>::type V;
  constexpr int BPG = G / 32;
  constexpr bool kFirst = J % BPG == 0;
  constexpr bool kAheadOpens = (J + 2) % BPG == 0;
  constexpr int B = J & 3, BA = (J + 2) & 3;
  // 3 bits: this lane's funnel shift (0 or 16, by the parity of its group
  // half)
  const uint32_t sh3 = (threadIdx.x & 1u) << 4;
  if constexpr (kFirst) {
    st.s0 = st.ps0[B];
    st.s1 = st.ps1[B];
    if constexpr (BITS == 4) {
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        st.zf[r] = float(16u + ((st.pz[B].x >> (4 * r)) & 0xFu)) * 0.0625f;
        st.zf[8 + r] = float(16u + ((st.pz[B].y >> (4 * r)) & 0xFu)) * 0.0625f;
      }
    } else {
      const uint32_t zl = __builtin_amdgcn_alignbit(st.pz[B].y, st.pz[B].x, sh3);
      const uint32_t zh = st.pz[B].y >> sh3;
#define AWQ_MG_Z3(R) st.zf[R] = float(16u + code3_at<R>(zl, zh)) * 0.0625f;
      AWQ_MG_Z3(0) AWQ_MG_Z3(1) AWQ_MG_Z3(2) AWQ_MG_Z3(3) AWQ_MG_Z3(4) AWQ_MG_Z3(5)
      AWQ_MG_Z3(6) AWQ_MG_Z3(7) AWQ_MG_Z3(8) AWQ_MG_Z3(9) AWQ_MG_Z3(10) AWQ_MG_Z3(11)
      AWQ_MG_Z3(12) AWQ_MG_Z3(13) AWQ_MG_Z3(14) AWQ_MG_Z3(15)
#undef AWQ_MG_Z3
    }
  }
  load_data(kb + 32 * (J + 2), st.w[BA], st.a[BA]);
  if constexpr (kAheadOpens) load_par(kb + 32 * (J + 2), st.ps0[BA], st.ps1[BA], st.pz[BA]);

  const V a = __builtin_bit_cast(V, st.a[B]);
  const floatx4 zero = {0.f, 0.f, 0.f, 0.f};
  V ones;
#pragma unroll
  for (int e = 0; e < 8; ++e) ones[e] = 1;
  // At T = 1 the MFMAs accumulate a group's blocks (P' and S over up to 128
  // rows) and the fold runs once per group; with more token rows the extra
  // 64 registers would spill, so every block folds.
  constexpr bool kAccFirst = TV == 1 ? kFirst : true;
  constexpr bool kAccLast = TV == 1 ? J % BPG == BPG - 1 : true;
  const floatx4 sx = mfma_16x16x32(a, ones, kAccFirst ? zero : st.sacc);
  if constexpr (!kAccLast) st.sacc = sx;
  const uint32_t sw[8] = {st.s0.x, st.s0.y, st.s0.z, st.s0.w, st.s1.x, st.s1.y, st.s1.z, st.s1.w};
  if constexpr (BITS == 3) {
    uint32_t lo[8], hi[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      lo[e] = __builtin_amdgcn_alignbit(st.w[B][e].y, st.w[B][e].x, sh3);
      hi[e] = st.w[B][e].y >> sh3;
    }
#define AWQ_MG_CODE3(R)                                                                     \
  {                                                                                         \
    const V b = __builtin_bit_cast(                                                         \
        V, make_uint4(code3_pair<F16, R>(lo[0], hi[0], lo[1], hi[1], one),                  \
                      code3_pair<F16, R>(lo[2], hi[2], lo[3], hi[3], one),                  \
                      code3_pair<F16, R>(lo[4], hi[4], lo[5], hi[5], one),                  \
                      code3_pair<F16, R>(lo[6], hi[6], lo[7], hi[7], one)));                \
    const floatx4 p = mfma_16x16x32(a, b, kAccFirst ? zero : st.pacc[R]);                          \
    if constexpr (kAccLast) {                                                               \
      const float sc = f16_to_f32(uint16_t((sw[R >> 1] >> (16 * (R & 1))) & 0xFFFFu));      \
      for (int v = 0; v < TV; ++v)                                                          \
        st.tot[R][v] = __builtin_fmaf(sc, __builtin_fmaf(-st.zf[R], sx[v], p[v]), st.tot[R][v]); \
    } else {                                                                                \
      st.pacc[R] = p;                                                                       \
    }                                                                                       \
  }
    AWQ_MG_CODE3(0) AWQ_MG_CODE3(1) AWQ_MG_CODE3(2) AWQ_MG_CODE3(3)
    AWQ_MG_CODE3(4) AWQ_MG_CODE3(5) AWQ_MG_CODE3(6) AWQ_MG_CODE3(7)
    AWQ_MG_CODE3(8) AWQ_MG_CODE3(9) AWQ_MG_CODE3(10) AWQ_MG_CODE3(11)
    AWQ_MG_CODE3(12) AWQ_MG_CODE3(13) AWQ_MG_CODE3(14) AWQ_MG_CODE3(15)
#undef AWQ_MG_CODE3
  } else {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = c ? st.w[B][e].y : st.w[B][e].x;
#define AWQ_MG_CODE(R)                                                                      \
  {                                                                                         \
    constexpr int m = c * 8 + R;                                                            \
    const V b = __builtin_bit_cast(                                                         \
        V, make_uint4(code_pair<F16, R>(w[0], w[1]), code_pair<F16, R>(w[2], w[3]),         \
                      code_pair<F16, R>(w[4], w[5]), code_pair<F16, R>(w[6], w[7])));       \
    const floatx4 p = mfma_16x16x32(a, b, kAccFirst ? zero : st.pacc[m]);                          \
    if constexpr (kAccLast) {                                                               \
      const float sc = f16_to_f32(uint16_t((sw[m >> 1] >> (16 * (m & 1))) & 0xFFFFu));      \
      for (int v = 0; v < TV; ++v)                                                          \
        st.tot[m][v] = __builtin_fmaf(sc, __builtin_fmaf(-st.zf[m], sx[v], p[v]), st.tot[m][v]); \
    } else {                                                                                \
      st.pacc[m] = p;                                                                       \
    }                                                                                       \
  }
    if (c == 0) {
      constexpr int c = 0;
      AWQ_MG_CODE(0) AWQ_MG_CODE(1) AWQ_MG_CODE(2) AWQ_MG_CODE(3)
      AWQ_MG_CODE(4) AWQ_MG_CODE(5) AWQ_MG_CODE(6) AWQ_MG_CODE(7)
    } else {
      constexpr int c = 1;
      AWQ_MG_CODE(0) AWQ_MG_CODE(1) AWQ_MG_CODE(2) AWQ_MG_CODE(3)
      AWQ_MG_CODE(4) AWQ_MG_CODE(5) AWQ_MG_CODE(6) AWQ_MG_CODE(7)
    }
#undef AWQ_MG_CODE
  }
  }
}

// Workgroup `id` of a grid of gx column blocks x gy chunks.
typedef float MgRed[16][kMgCols * 8 + 4];
template <bool F16, int BITS, int G, int TV>
__device__ __forceinline__ void mgemv_workgroup(
    const uint16_t* __restrict__ X, int64_t T, int64_t N, int64_t K,
    const int32_t* __restrict__ qweight, const int32_t* __restrict__ qzeros,
    const uint16_t* __restrict__ scales, int kpw, float* __restrict__ partial, int id, int gx,
    int gy, MgRed* red) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  const int jj = lane & 15, lg = lane >> 4;
  // Words per k row, and the lane's 16 output rows n0 .. n0 + 15: 4 bits, two
  // adjacent word columns (one 8-byte load per k row); 3 bits, half of a
  // 32-row group, words 0-1 (even jj) or 1-2 (odd jj) of its 3 (two 4-byte
  // loads). Lanes past N (N a multiple of 16, or of 32 for 3 bits: whole
  // lanes, whole lane pairs) and token rows past T read column 0 / row 0
  // instead: every load stays in bounds and needs no branch, and an MFMA
  // output column depends only on its own B column (an output row on its own
  // A row), so those lanes' results, which are never stored, do not reach the
  // others.
  const int64_t RS = BITS == 4 ? N / 8 : N / 32 * 3;
  // Workgroups are dealt to the 8 XCDs in turn, and each XCD has its own L2.
  // XCD i takes a contiguous run of (column block, chunk) indices, column
  // blocks fastest, so neighbouring column blocks, whose qweight row
  // segments can share cache lines (3 bits: 96 bytes per row and block),
  // meet in one L2.
  int bx, by;
  {
    const int W = gx * gy;
    const int q = W / 8, r = W % 8, xi = id % 8;
    const int L = xi * q + (xi < r ? xi : r) + id / 8;
    bx = L % gx;
    by = L / gx;
  }
  const int64_t n0 = int64_t(bx) * (kMgCols * 8) + 16 * jj;
  const bool live = n0 < N;
  const int64_t nl0 = live ? n0 : 0;
  const int64_t wq = !live ? 0 : BITS == 4 ? n0 / 8 : 3 * (n0 / 32) + (jj & 1);
  // This wave's k rows: kpw (a multiple of 128) from its place in the grid,
  // cut at K (a multiple of 128); waves past K have none.
  const int kw0 = (by * kMgWaves + wave) * kpw;
  const int kw1 = kw0 + kpw < int(K) ? kw0 + kpw : int(K);
  const uint16_t* xrow = X + int64_t(jj < T ? jj : 0) * K + 8 * lg;
  const int32_t* qlane = qweight + int64_t(8 * lg) * RS + wq;
  auto load2 = [](const int32_t* p) {
    if constexpr (BITS == 4) return *reinterpret_cast<const uint2*>(p);
    else return make_uint2(uint32_t(p[0]), uint32_t(p[1]));
  };

  MgState<F16> st;
#pragma unroll
  for (int m = 0; m < kMgMfma; ++m) st.tot[m] = floatx4{0.f, 0.f, 0.f, 0.f};

  // The exponent bits of B = 1 + q/16, held in a register so that the 3-bit
  // operand's mask and or fuse into one instruction.
  uint32_t one = F16 ? 0x3C003C00u : 0x3F803F80u;
  asm volatile("" : "+v"(one));
  if (kw0 < kw1) {
    // k-blocks past the wave's last re-read its last block (a harmless
    // in-bounds prefetch)
    auto load_data = [&](int kb, uint2 (&w)[8], uint4& a) {
      const int kc = kb < kw1 ? kb : kw1 - 32;
      const int32_t* q = qlane + int64_t(kc) * RS;
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = load2(q + e * RS);
      a = *reinterpret_cast<const uint4*>(xrow + kc);
    };
    auto load_par = [&](int kb, uint4& s0, uint4& s1, uint2& z) {
      const int64_t g = (kb < kw1 ? kb : kw1 - 32) / G;
      s0 = *reinterpret_cast<const uint4*>(scales + g * N + nl0);
      s1 = *reinterpret_cast<const uint4*>(scales + g * N + nl0 + 8);
      z = load2(qzeros + g * RS + wq);
    };
    load_data(kw0, st.w[0], st.a[0]);
    load_par(kw0, st.ps0[0], st.ps1[0], st.pz[0]);
    load_data(kw0 + 32, st.w[1], st.a[1]);
    if (G == 32) load_par(kw0 + 32, st.ps0[1], st.ps1[1], st.pz[1]);
    for (int kb = kw0; kb < kw1; kb += 128) {
      mg_block<F16, BITS, G, TV, 0>(st, kb, load_data, load_par, one);
      __builtin_amdgcn_sched_barrier(0);
      mg_block<F16, BITS, G, TV, 1>(st, kb, load_data, load_par, one);
      __builtin_amdgcn_sched_barrier(0);
      mg_block<F16, BITS, G, TV, 2>(st, kb, load_data, load_par, one);
      __builtin_amdgcn_sched_barrier(0);
      mg_block<F16, BITS, G, TV, 3>(st, kb, load_data, load_par, one);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
#pragma unroll
  for (int m = 0; m < kMgMfma; ++m)
#pragma unroll
    for (int v = 0; v < TV; ++v) st.tot[m][v] *= 16.f;

  // totals -> LDS [wave][t][n_local], n_local = 16·jj + m (rows 4·lg + v
  // for v < TV: with TV < 4, T <= TV and only lane group 0's rows are read)
#pragma unroll
  for (int m = 0; m < kMgMfma; ++m)
#pragma unroll
    for (int v = 0; v < TV; ++v) red[wave][4 * lg + v][16 * jj + m] = st.tot[m][v];
  __syncthreads();
  const int nl = threadIdx.x;
  const int64_t n = int64_t(bx) * kMgCols * 8 + nl;
  if (n < N) {
    for (int t = 0; t < T; ++t) {
      const float s = ((red[0][t][nl] + red[1][t][nl]) + red[2][t][nl]) + red[3][t][nl];
      partial[(int64_t(by) * T + t) * N + n] = s;
    }
  }
}

}  // namespace
}  // namespace awq
