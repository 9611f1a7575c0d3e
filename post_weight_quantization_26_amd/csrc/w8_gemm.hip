// 8-bit products of many tokens: the 256x256 main loop of w8_ring.h with
// v_mfma_i32_16x16x64_i8, whose operands have the size of 16 bits' 16x16x32 at
// twice the multiplications. The main loop's A rows are output channels, so a
// lane holds 4 consecutive outputs of a token and the epilogue (steps, bias or
// activation and product, rounding) stays in registers. A gated pair's tile
// takes 128 channels of either layer, in turns of 64, so that both sums of an
// output meet in one lane.
//
// Bound by the matrix cores.
#include "w8_cut.h"

namespace awq {
namespace {

template <bool F16, bool GATED, int ACT, bool CUT>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(1, 1)))
void w8_gemm_kernel(const W8Product p, int tiles_t, int tiles_n) {
  constexpr int BC = GATED ? BM / 2 : BM;   // output channels of a tile
  const W8Unit unit = w8_unit<CUT>(p.cut, tiles_t, tiles_n);
  const int64_t t0 = int64_t(unit.tt) * BN, n0 = int64_t(unit.tn) * BC;
  int kt0 = 0, kt1 = int(p.K / 128);
  if constexpr (CUT) w8_run(p.cut, unit, kt1, kt0, kt1);
  const int64_t k0 = int64_t(kt0) * 128;
  const int64_t rows_t = p.T - t0 < BN ? p.T - t0 : BN;
  RingCtx c;
  c.wave = uniform(int(threadIdx.x >> 6));
  c.b.set(RingKind::kRows, p.x + t0 * p.K + k0, int(rows_t), int(p.K), c.wave * 64, 128, kt1 - kt0);
  if constexpr (GATED) {
    const PairRows rows = pair_rows(n0, c.wave, p.N);
    c.a.set(RingKind::kRows, (c.wave & 1 ? p.u.q : p.w.q) + rows.first * p.K + k0, rows.valid,
            int(p.K), 0, 128, kt1 - kt0);
  } else {
    const int64_t rows = p.N - n0 < BM ? p.N - n0 : BM;
    c.a.set(RingKind::kRows, p.w.q + n0 * p.K + k0, int(rows), int(p.K), c.wave * 64, 128,
            kt1 - kt0);
  }
  floatx4 acc[8][8];
  ring_mainloop<i8x16_t>(c, acc);

  const int lane = threadIdx.x & 63;
  const int wm = c.wave >> 1, wn = c.wave & 1;
  constexpr int NI = GATED ? 4 : 8, COLS = BC / 2;
  const int64_t tw = t0 + wn * 128, nw = n0 + wm * COLS;   // the wave's first
  const int left_t = int(rows_t) - wn * 128, left_n = int(p.N - nw < COLS ? p.N - nw : COLS);
  // every step and bias first: the compiler does not move a load over a store, and
  // one load's latency for each of the 64 blocks took 20 us
  Channels<GATED> ch[NI];
  float xs[8];
#pragma unroll
  for (int i = 0; i < NI; ++i) ch[i] = channels<F16, GATED>(p, nw + i * 16 + 4 * (lane >> 4));
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int64_t t = tw + j * 16 + (lane & 15);
    xs[j] = p.xs[t < p.T ? t : p.T - 1];
  }
  const WaveTile<COLS> tile(c.wave);
  const int64_t first = tw * p.N + nw;
  const bool bias = p.bias;
  // a pair's passes: G and U, if they are kept, then H; none for a run of a cut tile
  // (one way out: with a branch around the passes the compiler spilled)
#pragma unroll 1
  for (int pass = CUT && unit.slot >= 0 ? 3 : GATED && p.G ? 0 : 2; pass < 3; ++pass) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const intx4 s = __builtin_bit_cast(intx4, from_agpr(acc[i][j]));
        float y[4];
        if constexpr (GATED) {
          const intx4 su = __builtin_bit_cast(intx4, from_agpr(acc[i + 4][j]));
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            if (pass != 1) y[v] = scaled(s[v], xs[j], ch[i].w[v]);
            if (pass == 2) y[v] = act_of<ACT>(y[v]) * scaled(su[v], xs[j], ch[i].u[v]);
            if (pass == 1) y[v] = scaled(su[v], xs[j], ch[i].u[v]);
          }
        } else {
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            y[v] = scaled(s[v], xs[j], ch[i].w[v]);
            if (bias) y[v] += ch[i].bias[v];
          }
        }
        tile.template put<F16>(j * 16 + (lane & 15), i * 16 + 4 * (lane >> 4), y);
      }
    uint16_t* out = GATED && pass == 0 ? p.G : GATED && pass == 1 ? p.U : p.Y;
    tile.store(out + first, uint32_t(p.N), left_t, left_n);
  }
  if (CUT && unit.slot >= 0) w8_store_run(p.cut, unit, c.wave, acc);
}

// Workgroup (cut tile, wave, block row i) adds the runs of 16 channels x 128 tokens.
template <bool F16, bool GATED, int ACT>
__global__ __launch_bounds__(256) void w8_gemm_sum_kernel(const W8Product p, int tiles_t,
                                                          int tiles_n) {
  constexpr int BC = GATED ? BM / 2 : BM;
  const int cut = int(blockIdx.x), wave = int(blockIdx.y), i = int(blockIdx.z);
  const int lane = threadIdx.x & 63, tile = p.cut.full + cut;
  int tt, tn;
  w8_tile(tile, tiles_t, tiles_n, tt, tn);
  const int64_t t0 = int64_t(tt) * BN + (wave & 1) * 128 + (lane & 15);
  const int64_t n = int64_t(tn) * BC + (wave >> 1) * (BC / 2) + i * 16 +
                    4 * (lane >> 4);
  if (n >= p.N) return;
  const Channels<GATED> ch = channels<F16, GATED>(p, n);
#pragma unroll
  for (int j = threadIdx.x >> 6; j < 8; j += 4) {
    const int64_t t = t0 + j * 16;
    if (t >= p.T) continue;
    const intx4 s = w8_sum_runs<intx4>(p.cut, cut, wave, i, j);
    intx4 su = s;
    if constexpr (GATED) su = w8_sum_runs<intx4>(p.cut, cut, wave, i + 4, j);
    finish4<F16, GATED, ACT>(outputs_at(p, t, n), ch, p.xs[t], p.bias, 0, p.N % 4 == 0, p.N - n, s,
                             su);
  }
}

template <bool F16, bool GATED, int ACT>
hipError_t launch_gemm(const W8Product& p, hipStream_t st) {
  constexpr int BC = GATED ? BM / 2 : BM;
  const int tiles_t = int((p.T + BN - 1) / BN), tiles_n = int((p.N + BC - 1) / BC);
  if (!p.cut.runs) {
    w8_gemm_kernel<F16, GATED, ACT, false>
        <<<unsigned(tiles_t * tiles_n), NT, 0, st>>>(p, tiles_t, tiles_n);
    return hipGetLastError();
  }
  const int cut = tiles_t * tiles_n - p.cut.full;
  w8_gemm_kernel<F16, GATED, ACT, true>
      <<<unsigned(p.cut.full + cut * p.cut.runs), NT, 0, st>>>(p, tiles_t, tiles_n);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  w8_gemm_sum_kernel<F16, GATED, ACT>
      <<<dim3(unsigned(cut), 4, GATED ? 4 : 8), 256, 0, st>>>(p, tiles_t, tiles_n);
  return hipGetLastError();
}

template <bool F16>
hipError_t launch_gemm_f(const W8Product& p, hipStream_t st) {
  if (!p.u.q) return launch_gemm<F16, false, kSilu>(p, st);
  if (p.act == kSilu) return launch_gemm<F16, true, kSilu>(p, st);
  return launch_gemm<F16, true, kGelu>(p, st);
}

}  // namespace

hipError_t launch_w8_gemm(const W8Product& p, hipStream_t st) {
  return p.f16 ? launch_gemm_f<true>(p, st) : launch_gemm_f<false>(p, st);
}

}  // namespace awq
