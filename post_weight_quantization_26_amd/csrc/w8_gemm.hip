// 8-bit products of many tokens: the 256x256 main loop of gemm_core.h with
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
  W8Unit unit;
  if (!w8_unit<CUT>(p.cut, tiles_t, tiles_n, unit)) return;
  const int64_t t0 = int64_t(unit.tt) * BN, n0 = int64_t(unit.tn) * BC;
  const int64_t ld = p.K / 2;               // codes in pairs
  int64_t k0 = 0, k1 = ld;
  if constexpr (CUT) w8_run(p.cut, unit, int(ld / BK64), k0, k1);
  const uint16_t* x = reinterpret_cast<const uint16_t*>(p.x) + t0 * ld + k0;
  const int64_t rows_t = p.T - t0 < BN ? p.T - t0 : BN;
  GemmCtx64 c;
  if constexpr (GATED) {
    // wave w copies A rows 64w .. + 63: 64 channels from n0 + 64·(w / 2) of the
    // first layer (even w) or of the second
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t first = n0 + 64 * (w >> 1), last = p.N - 1;
    const int64_t left = p.N - first;
    const int64_t rows = left < 0 ? 0 : left < 64 ? left : 64;
    const uint16_t* q = reinterpret_cast<const uint16_t*>(w & 1 ? p.u.q : p.w.q) +
                        (first < p.N ? first : last) * ld + k0;
    w8_setup(c, q, rows, x, rows_t, ld, k1 - k0);
#pragma unroll
    for (int j = 0; j < 2; ++j) c.vbaseA[j] -= w * 64 * int(ld) * 2;
  } else {
    const int64_t rows = p.N - n0 < BM ? p.N - n0 : BM;
    w8_setup(c, reinterpret_cast<const uint16_t*>(p.w.q) + n0 * ld + k0, rows, x, rows_t, ld,
             k1 - k0);
  }
  floatx4 acc[8][8];
  gemm_mainloop16_of<i8x16_t>(c, acc);

  if (CUT && unit.slot >= 0) {
    w8_store_run(p.cut, unit, c.wave, acc);
    return;
  }
  const int lane = threadIdx.x & 63;
  const int wm = c.wave >> 1, wn = c.wave & 1;
  constexpr int NI = GATED ? 4 : 8;
  const bool whole = p.N % 4 == 0;          // every row of Y is 8-byte aligned
  const Outputs out = outputs_at(p, t0, n0);
  const int left_t = int(rows_t), left_n = int(p.N - n0 < BC ? p.N - n0 : BC);
  const uint32_t N = uint32_t(p.N);
  // every step and bias first: the compiler does not move a load over a store, and
  // one load's latency for each of the 64 blocks took 20 us
  Channels<GATED> ch[NI];
  float xs[8];
#pragma unroll
  for (int i = 0; i < NI; ++i)
    ch[i] = channels<F16, GATED>(p, n0 + wm * (BC / 2) + i * 16 + 4 * (lane >> 4));
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int t = wn * 128 + j * 16 + (lane & 15);
    xs[j] = p.xs[t0 + (t < left_t ? t : left_t - 1)];
  }
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int n = wm * (BC / 2) + i * 16 + 4 * (lane >> 4);
    if (n >= left_n) continue;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int t = wn * 128 + j * 16 + (lane & 15);
      if (t < left_t)
        finish4<F16, GATED, ACT>(out, ch[i], xs[j], p.bias, uint32_t(t) * N + uint32_t(n), whole,
                                 left_n - n, __builtin_bit_cast(intx4, from_agpr(acc[i][j])),
                                 __builtin_bit_cast(intx4, from_agpr(acc[GATED ? i + 4 : i][j])));
    }
  }
}

// Workgroup (cut tile, wave, block row i) adds the runs of 16 channels x 128 tokens.
template <bool F16, bool GATED, int ACT>
__global__ __launch_bounds__(256) void w8_gemm_sum_kernel(const W8Product p, int tiles_t) {
  constexpr int BC = GATED ? BM / 2 : BM;
  const int cut = int(blockIdx.x), wave = int(blockIdx.y), i = int(blockIdx.z);
  const int lane = threadIdx.x & 63, tile = p.cut.full + cut;
  const int64_t t0 = int64_t(tile % tiles_t) * BN + (wave & 1) * 128 + (lane & 15);
  const int64_t n = int64_t(tile / tiles_t) * BC + (wave >> 1) * (BC / 2) + i * 16 +
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
        <<<unsigned(gemm_blocks(tiles_t, tiles_n)), NT, 0, st>>>(p, tiles_t, tiles_n);
    return hipGetLastError();
  }
  const int cut = tiles_t * tiles_n - p.cut.full;
  w8_gemm_kernel<F16, GATED, ACT, true>
      <<<unsigned(p.cut.full + cut * p.cut.runs), NT, 0, st>>>(p, tiles_t, tiles_n);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  w8_gemm_sum_kernel<F16, GATED, ACT>
      <<<dim3(unsigned(cut), 4, GATED ? 4 : 8), 256, 0, st>>>(p, tiles_t);
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
