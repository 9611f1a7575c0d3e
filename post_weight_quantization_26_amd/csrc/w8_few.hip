// 8-bit products of few tokens (decode): Y[t][n] = xs_t·w_n·Σ_k x[t][k]·q[n][k],
// and the gated pair act(G)·U of two layers.
//
// Bound by HBM: the codes q (N·K bytes, twice that for a pair) are read once
// per 16·TB tokens, straight into the matrix cores' operand registers. A
// workgroup owns 16·RB output channels and 16·TB tokens; its waves take
// consecutive parts of K, so that one launch has enough of them at any N, and
// meet in LDS. Every lane of a row's four reads 32 consecutive bytes of a
// 128-byte block (the contraction's order is free as long as both operands
// share it), so a wave's loads cover whole lines. Integer sums are exact, in
// any order.
#include "w8_common.h"

namespace awq {
namespace {

// Waves of a workgroup at most: their sums fit 64 KiB of LDS.
constexpr int few_waves(int rb, int tb) { return 64 / (rb * tb) < 16 ? 64 / (rb * tb) : 16; }
#ifndef FEW_U
#define FEW_U 4
#endif
constexpr int few_units(int rb, int tb) { return FEW_U / (rb + tb) < 1 ? 1 : FEW_U / (rb + tb); }

template <bool F16, int RB, int TB, bool GATED, int ACT>
__global__ __launch_bounds__(few_waves(RB, TB) * 64) void w8_few_kernel(const W8Product p) {
  static_assert(!GATED || RB % 2 == 0, "a pair takes blocks of both layers");
  constexpr int NB = GATED ? RB / 2 : RB;   // blocks of 16 output channels
  extern __shared__ int few_sums[];         // [waves][RB·TB][256]
  // (a scalar: the matrix instructions ignore the execution mask, so what skips
  // them has to be a branch)
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const int r = lane & 15, q = lane >> 4;
  const int64_t n0 = int64_t(blockIdx.x) * (16 * NB), t0 = int64_t(blockIdx.y) * (16 * TB);
  const int64_t K = p.K;
  // rows past the last are the last one's again; their sums are not stored
  const int8_t* w[RB];
  const int8_t* x[TB];
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    const int64_t n = n0 + (b % NB) * 16 + r;
    w[b] = (b < NB ? p.w.q : p.u.q) + (n < p.N ? n : p.N - 1) * K + q * 32;
  }
#pragma unroll
  for (int b = 0; b < TB; ++b) {
    const int64_t t = t0 + b * 16 + r;
    x[b] = p.x + (t < p.T ? t : p.T - 1) * K + q * 32;
  }
  intx4 acc[RB][TB] = {};
  const int units = int(K >> 7);
  const int u1 = units * (wave + 1) / waves;   // units < 1024
  int u = units * wave / waves;
  // U blocks of 128 bytes at a time, the next ones loaded before these are used
  constexpr int U = few_units(RB, TB);
  struct Batch {
    intx4 a[U][RB][2], b[U][TB][2];
  };
  auto load = [&](Batch& d, int at_unit) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (at_unit + i >= u1) break;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t at = int64_t(at_unit + i) * 128 + h * 16;
#pragma unroll
        for (int j = 0; j < RB; ++j) d.a[i][j][h] = *reinterpret_cast<const intx4*>(w[j] + at);
#pragma unroll
        for (int j = 0; j < TB; ++j) d.b[i][j][h] = *reinterpret_cast<const intx4*>(x[j] + at);
      }
    }
  };
  auto use = [&](const Batch& d, int at_unit) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (at_unit + i >= u1) break;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < RB; ++j)
#pragma unroll
          for (int k = 0; k < TB; ++k) acc[j][k] = mfma_16x16x64(d.a[i][j][h], d.b[i][k][h], acc[j][k]);
    }
  };
  Batch d0, d1;
  load(d0, u);
  for (; u < u1; u += 2 * U) {
    load(d1, u + U);
    use(d0, u);
    load(d0, u + 2 * U);
    use(d1, u + U);
  }

  // element (row 4q + v, token r) of a block at 16·r + 4q + v: a token's 16
  // channels are consecutive
#pragma unroll
  for (int j = 0; j < RB; ++j)
#pragma unroll
    for (int k = 0; k < TB; ++k)
      *reinterpret_cast<intx4*>(few_sums + ((wave * RB + j) * TB + k) * 256 + 16 * r + 4 * q) =
          acc[j][k];
  __syncthreads();
  for (int i = threadIdx.x; i < NB * TB * 256; i += blockDim.x) {
    const int e = i & 255, blk = i >> 8, j = blk / TB, k = blk % TB;
    const int64_t n = n0 + j * 16 + (e & 15), t = t0 + k * 16 + (e >> 4);
    int s = 0, su = 0;
    for (int v = 0; v < waves; ++v) {
      s += few_sums[((v * RB + j) * TB + k) * 256 + e];
      if (GATED) su += few_sums[((v * RB + NB + j) * TB + k) * 256 + e];
    }
    if (n >= p.N || t >= p.T) continue;
    const float xs = p.xs[t];
    float y = scaled(s, xs, p.w.steps[n]);
    const int64_t o = t * p.N + n;
    if constexpr (GATED) {
      const float uu = scaled(su, xs, p.u.steps[n]);
      if (p.G) {
        p.G[o] = round16<F16>(y);
        p.U[o] = round16<F16>(uu);
      }
      y = act_of<ACT>(y) * uu;
    } else if (p.bias) {
      y += widen16<F16>(p.bias[n]);
    }
    p.Y[o] = round16<F16>(y);
  }
}

template <bool F16, int RB, int TB, bool GATED, int ACT>
hipError_t launch_few(const W8Product& p, hipStream_t st) {
  constexpr int NB = GATED ? RB / 2 : RB;
  const int64_t blocks = (p.N + 16 * NB - 1) / (16 * NB), tiles = (p.T + 16 * TB - 1) / (16 * TB);
  const int64_t units = p.K / 128;
  // 8 waves per CU or more where K has a block of 128 for each; the waves'
  // sums fit 64 KiB
  static int tgt = getenv("FEW_W") ? atoi(getenv("FEW_W")) : 2048;
  int64_t waves = (tgt + blocks * tiles - 1) / (blocks * tiles);
  if (waves < 4) waves = 4;
  if (waves > few_waves(RB, TB)) waves = few_waves(RB, TB);
  if (waves > units) waves = units;
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(tiles));
  w8_few_kernel<F16, RB, TB, GATED, ACT>
      <<<grid, unsigned(waves * 64), size_t(waves) * RB * TB * 1024, st>>>(p);
  return hipGetLastError();
}

template <bool F16, bool GATED, int ACT>
hipError_t launch_few_t(const W8Product& p, hipStream_t st) {
  static int rb = getenv("FEW_RB") ? atoi(getenv("FEW_RB")) : 1;
  if constexpr (!GATED) if (p.T <= 16 && rb == 1) return launch_few<F16, 1, 1, GATED, ACT>(p, st);
  if (p.T <= 16) return launch_few<F16, 2, 1, GATED, ACT>(p, st);
  if (p.T <= 32) return launch_few<F16, 2, 2, GATED, ACT>(p, st);
  return launch_few<F16, 4, 4, GATED, ACT>(p, st);
}

template <bool F16>
hipError_t launch_few_f(const W8Product& p, hipStream_t st) {
  if (!p.u.q) return launch_few_t<F16, false, kSilu>(p, st);
  if (p.act == kSilu) return launch_few_t<F16, true, kSilu>(p, st);
  return launch_few_t<F16, true, kGelu>(p, st);
}

}  // namespace

hipError_t launch_w8_few(const W8Product& p, hipStream_t st) {
  return p.f16 ? launch_few_f<true>(p, st) : launch_few_f<false>(p, st);
}

}  // namespace awq
