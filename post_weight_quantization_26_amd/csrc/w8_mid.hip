// 8-bit products of a few hundred tokens (w8_mid.h): tiles of 128 or 256 channels
// (a pair: half of them of either layer) x 32 to 128 tokens, and where these are
// still too few, the contraction in runs whose exact integer sums a second launch
// adds.
#include "w8_mid.h"

namespace awq {
namespace {

template <bool F16, bool GATED, int ACT, int RA, int TR, bool RUNS>
__global__ __launch_bounds__(256) void w8_mid_kernel(const W8Product p, int tiles_n, int tiles_t) {
  constexpr int BC = GATED ? RA / 2 : RA;
  int tn, tt;
  if (!mid_tile_of(blockIdx.x, tiles_n, tiles_t, tn, tt)) return;
  const int64_t n0 = int64_t(tn) * BC, t0 = int64_t(tt) * TR, K = p.K;
  const int64_t rows_n = p.N - n0 < BC ? p.N - n0 : BC, rows_t = p.T - t0 < TR ? p.T - t0 : TR;
  const MidTile m = mid_setup<GATED, RA, TR>(
      p.w.q + n0 * K, GATED ? p.u.q + n0 * K : nullptr, rows_n, p.x + t0 * K, rows_t, K);
  const int steps = int(K >> 7), run = blockIdx.y;
  const int begin = RUNS ? int(int64_t(steps) * run / p.runs) : 0;
  const int end = RUNS ? int(int64_t(steps) * (run + 1) / p.runs) : steps;
  intx4 acc[RA / 32][TR / 32] = {};
  mid_loop<i8x16_t, GATED, RA, TR>(m, begin, end, acc);

  const int lane = threadIdx.x & 63;
  constexpr int NI = GATED ? RA / 64 : RA / 32;
  const Outputs out = outputs_at(p, t0, n0);
  // every step and bias before the first store (w8_gemm.hip)
  Channels<GATED> ch[RUNS ? 1 : NI];
  float xs[TR / 32];
  if constexpr (!RUNS) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
      ch[i] = channels<F16, GATED>(p, n0 + (m.wave >> 1) * (BC / 2) + i * 16 + 4 * (lane >> 4));
#pragma unroll
    for (int j = 0; j < TR / 32; ++j) {
      const int64_t t = t0 + (m.wave & 1) * (TR / 2) + j * 16 + (lane & 15);
      xs[j] = p.xs[t < p.T ? t : p.T - 1];
    }
  }
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int64_t n = n0 + (m.wave >> 1) * (BC / 2) + i * 16 + 4 * (lane >> 4);
    if (n >= p.N) continue;
#pragma unroll
    for (int j = 0; j < TR / 32; ++j) {
      const int64_t t = t0 + (m.wave & 1) * (TR / 2) + j * 16 + (lane & 15);
      if (t >= p.T) continue;
      if constexpr (RUNS) {
        int* o = p.partial + ((int64_t(run) * (GATED ? 2 : 1)) * p.T + t) * p.ldp + n;
        *reinterpret_cast<intx4*>(o) = acc[i][j];
        if constexpr (GATED) *reinterpret_cast<intx4*>(o + p.T * p.ldp) = acc[i + NI][j];
      } else {
        finish4<F16, GATED, ACT>(out, ch[i], xs[j], p.bias,
                                 uint32_t(t - t0) * uint32_t(p.N) + uint32_t(n - n0),
                                 p.N % 4 == 0, p.N - n, acc[i][j], acc[GATED ? i + NI : i][j]);
      }
    }
  }
}

// Adds the runs' sums: 4 channels of a token a thread.
template <bool F16, bool GATED, int ACT>
__global__ __launch_bounds__(256) void w8_mid_sum_kernel(const W8Product p) {
  const uint32_t quads = uint32_t(p.ldp / 4);
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= p.T * quads) return;
  const int64_t t = i / quads, n = (i - t * quads) * 4;
  const int* o = p.partial + t * p.ldp + n;
  const int64_t step = p.T * p.ldp;
  intx4 s = {}, su = {};
  for (int r = 0; r < p.runs; ++r) {
    s += *reinterpret_cast<const intx4*>(o);
    if constexpr (GATED) su += *reinterpret_cast<const intx4*>(o + step);
    o += GATED ? 2 * step : step;
  }
  const Channels<GATED> ch = channels<F16, GATED>(p, n);
  finish4<F16, GATED, ACT>(outputs_at(p, t, n), ch, p.xs[t], p.bias, 0, p.N % 4 == 0, p.N - n, s, su);
}

template <bool F16, bool GATED, int ACT, int RA, int TR>
hipError_t launch_mid(const W8Product& p, hipStream_t st) {
  constexpr int BC = GATED ? RA / 2 : RA;
  const int tiles_n = int((p.N + BC - 1) / BC), tiles_t = int((p.T + TR - 1) / TR);
  const dim3 grid(unsigned(mid_blocks(tiles_n, tiles_t)), unsigned(p.runs));
  if (p.runs == 1) {
    w8_mid_kernel<F16, GATED, ACT, RA, TR, false><<<grid, 256, 0, st>>>(p, tiles_n, tiles_t);
    return hipGetLastError();
  }
  if constexpr (RA == 128)
    w8_mid_kernel<F16, GATED, ACT, RA, TR, true><<<grid, 256, 0, st>>>(p, tiles_n, tiles_t);
  else return hipErrorInvalidValue;   // runs are cut of tiles of 128 rows only
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  w8_mid_sum_kernel<F16, GATED, ACT>
      <<<unsigned((p.T * (p.ldp / 4) + 255) / 256), 256, 0, st>>>(p);
  return hipGetLastError();
}

template <bool F16, bool GATED, int ACT>
hipError_t launch_mid_t(const W8Product& p, hipStream_t st) {
  if (p.tile_n == 256) return launch_mid<F16, GATED, ACT, 256, 128>(p, st);
  if (p.tile_t == 32) return launch_mid<F16, GATED, ACT, 128, 32>(p, st);
  if (p.tile_t == 64) return launch_mid<F16, GATED, ACT, 128, 64>(p, st);
  return launch_mid<F16, GATED, ACT, 128, 128>(p, st);
}

template <bool F16>
hipError_t launch_mid_f(const W8Product& p, hipStream_t st) {
  if (!p.u.q) return launch_mid_t<F16, false, kSilu>(p, st);
  if (p.act == kSilu) return launch_mid_t<F16, true, kSilu>(p, st);
  return launch_mid_t<F16, true, kGelu>(p, st);
}

}  // namespace

hipError_t launch_w8_mid(const W8Product& p, hipStream_t st) {
  return p.f16 ? launch_mid_f<true>(p, st) : launch_mid_f<false>(p, st);
}

}  // namespace awq
