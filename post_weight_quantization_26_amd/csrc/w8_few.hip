// 8-bit products of up to 16 tokens (decode): Y[t][n] = xs_t·w_n·Σ_k x[t][k]·q[n][k],
// and the gated pair act(G)·U of two layers.
//
// Bound by HBM: the codes q (N·K bytes, twice that for a pair) are read once,
// straight into the matrix cores' operand registers. A workgroup owns 16 output
// channels (of either layer); its waves take consecutive parts of K, so that one
// launch has enough of them at any N, and meet in LDS. Every lane of a row's four
// reads 32 consecutive bytes of a 128-byte block (the contraction's order is free
// as long as both operands share it), so a wave's loads cover whole lines. Integer
// sums are exact, in any order. One token: 4096x11008 10.6 us, 28672x8192 37 us
// (part of it from the cache behind L2), a pair of these 82 us (5.7 TB/s).
#include "w8_common.h"

namespace awq {
namespace {

constexpr int kFewWaves = 16;   // of a workgroup, at most
// 128-byte blocks of K loaded at once, twice (64 registers): more was slower (85
// instead of 37 us for a token of 28672x8192 with twice as many).
constexpr int few_units(int rb) { return 4 / (rb + 1); }

template <bool F16, int RB, bool GATED, int ACT>
__global__ __launch_bounds__(kFewWaves * 64) void w8_few_kernel(const W8Product p) {
  static_assert(!GATED || RB % 2 == 0, "a pair takes blocks of both layers");
  constexpr int NB = GATED ? RB / 2 : RB;   // blocks of 16 output channels
  extern __shared__ int few_sums[];         // [waves][RB][256]
  // (a scalar: the matrix instructions ignore the execution mask, so what skips
  // them has to be a branch)
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const int r = lane & 15, q = lane >> 4;
  const int64_t n0 = int64_t(blockIdx.x) * (16 * NB), K = p.K;
  // rows past the last are the last one's again; their sums are not stored
  const int8_t* w[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    const int64_t n = n0 + (b % NB) * 16 + r;
    w[b] = (b < NB ? p.w.q : p.u.q) + (n < p.N ? n : p.N - 1) * K + q * 32;
  }
  const int8_t* x = p.x + (r < p.T ? r : p.T - 1) * K + q * 32;
  intx4 acc[RB] = {};
  const int units = int(K >> 7);
  const int u1 = units * (wave + 1) / waves;   // units < 1024
  int u = units * wave / waves;
  // U blocks of 128 bytes at a time, the next ones loaded before these are used
  constexpr int U = few_units(RB);
  struct Batch {
    intx4 a[U][RB][2], b[U][2];
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
        d.b[i][h] = *reinterpret_cast<const intx4*>(x + at);
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
        for (int j = 0; j < RB; ++j) acc[j] = mfma_16x16x64(d.a[i][j][h], d.b[i][h], acc[j]);
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
    *reinterpret_cast<intx4*>(few_sums + (wave * RB + j) * 256 + 16 * r + 4 * q) = acc[j];
  __syncthreads();
  for (int i = threadIdx.x; i < NB * 256; i += blockDim.x) {
    const int e = i & 255, j = i >> 8, t = e >> 4;
    const int64_t n = n0 + j * 16 + (e & 15);
    int s = 0, su = 0;
    for (int v = 0; v < waves; ++v) {
      s += few_sums[(v * RB + j) * 256 + e];
      if (GATED) su += few_sums[(v * RB + NB + j) * 256 + e];
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

template <bool F16, int RB, bool GATED, int ACT>
hipError_t launch_few(const W8Product& p, hipStream_t st) {
  constexpr int NB = GATED ? RB / 2 : RB;
  if (p.T > 16) return hipErrorInvalidValue;
  const int64_t blocks = (p.N + 16 * NB - 1) / (16 * NB), units = p.K / 128;
  // 8 waves per CU or more, each with a block of 128 of K
  int64_t waves = (2048 + blocks - 1) / blocks;
  if (waves < 4) waves = 4;
  if (waves > kFewWaves) waves = kFewWaves;
  if (waves > units) waves = units;
  w8_few_kernel<F16, RB, GATED, ACT>
      <<<unsigned(blocks), unsigned(waves * 64), size_t(waves) * RB * 1024, st>>>(p);
  return hipGetLastError();
}

template <bool F16>
hipError_t launch_few_f(const W8Product& p, hipStream_t st) {
  if (!p.u.q) return launch_few<F16, 1, false, kSilu>(p, st);
  if (p.act == kSilu) return launch_few<F16, 2, true, kSilu>(p, st);
  return launch_few<F16, 2, true, kGelu>(p, st);
}

}  // namespace

hipError_t launch_w8_few(const W8Product& p, hipStream_t st) {
  return p.f16 ? launch_few_f<true>(p, st) : launch_few_f<false>(p, st);
}

}  // namespace awq
