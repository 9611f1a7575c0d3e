// Gradient of the 8-bit products with respect to their input (taken as the
// values that its 8-bit rows stand for):
//
//   plain   dx[t][k] = Σ_n (dy[t][n]·w_n)·q[n][k]
//   gated   dg = dh·u·act'(g), du = dh·act(g);
//           dx[t][k] = Σ_n (dg·wg_n)·qg[n][k] + Σ_n (du·wu_n)·qu[n][k]
//
// One fp16 product: the steps join the gradient in the operand A (one rounding),
// the codes are exact fp16 numbers. A pair's two sums are one contraction of
// twice the length. fp16 for bf16 gradients too: it keeps 3 bits more, and a
// power of two per row takes the place of bf16's range. The rounding is 2^-11 of a term,
// as large as fp16's of an output (dX's mean error 2.9e-4 instead of 2.1e-4); a second
// operand of what the first one leaves would keep float32's terms at twice the matrix
// work, most of the time of large calls. Launch 1 forms A; then
//  * many tokens: launch 2 writes the codes' transpose as the fp16 operand of [K, C]
//    and launch 3 is the 256x256 main loop of w8_ring.h;
//  * fewer: w8_back_few.hip takes the codes as they are.
#include "w8_cut.h"
#include "w8_back.h"

namespace awq {
namespace {

__device__ __forceinline__ uint32_t finite_abs(float v) {
  const uint32_t u = __float_as_uint(v) & 0x7FFFFFFFu;
  return u < 0x7F800000u ? u : 0;
}

// The power of two of a row whose largest finite |a| has these bits: 2^e takes it
// to [2^13, 2^14), where |code|·a stays far from the fp16 and float32 limits.
// Returns e, with 2^e and 2^-e normal numbers; 0 for a row of zeros.
__device__ __forceinline__ int row_exponent(uint32_t largest) {
  if (!largest) return 0;
  const int e = int(largest >> 23) - 127 - 13;
  return e < -126 ? -126 : e;   // at most 254 - 140
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(uint32_t(127 + e) << 23); }

// dg·wg and du·wu (or dy·w alone) of one output.
template <bool GATED, int ACT>
__device__ __forceinline__ void back_values(float d, float g, float u, float w, float wu, float& a,
                                            float& b, float& dg, float& du) {
  if constexpr (GATED) {
    float ac;
    const float slope = act_slope<ACT>(g, ac);
    dg = (d * u) * slope;
    du = d * ac;
    a = dg * w;
    b = du * wu;
  } else {
    a = d * w;
    b = 0.f;
  }
}

__device__ __forceinline__ uint32_t block_max(uint32_t m) {
  __shared__ uint32_t red[16];
  m = wave_max(m);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  uint32_t r = 0;
  for (int i = 0; i < int(blockDim.x >> 6); ++i) r = r > red[i] ? r : red[i];
  return r;
}

// A's element (t, c), c over the layers' Np each: panels of 64 c of every token (a
// tile's k-tile is 32 KiB in one piece, where rows of 44 KB take a page for two:
// gradient of 4096 tokens of a pair of 11008, its product 634 -> 576 us), or, for
// few tokens, the order of that kernel's operand: blocks of 32 c x 16 tokens, a
// lane's 8 consecutive c together.
__device__ __forceinline__ int64_t operand_at(const W8Back& p, int64_t t, int64_t c) {
  if (!p.few) return ((c >> 6) * p.T + t) * 64 + (c & 63);
  const int64_t tb = (p.T + 15) >> 4;
  return (((c >> 5) * tb + (t >> 4)) * 64 + ((c >> 3) & 3) * 16 + (t & 15)) * 8 + (c & 7);
}

// A row of A, its values held in registers between the maximum and the rounding:
// dY, G and U are read once. N a multiple of 8, at most 8·V·blockDim. Bound by HBM.
template <bool F16, bool GATED, int ACT, int V>
__global__ __launch_bounds__(1024) void w8_grad_rows_kernel(const W8Back p) {
  const int64_t t = blockIdx.x;
  const int n8 = int(p.N >> 3);
  const int64_t row = t * p.N;
  uint4 rd[V], rg[V], ru[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int j = threadIdx.x + i * blockDim.x;
    if (j >= n8) continue;
    rd[i] = *reinterpret_cast<const uint4*>(p.dY + row + j * 8);
    if constexpr (GATED) {
      rg[i] = *reinterpret_cast<const uint4*>(p.G + row + j * 8);
      ru[i] = *reinterpret_cast<const uint4*>(p.U + row + j * 8);
    }
  }
  auto half = [](const uint4& v, int e) {
    const uint32_t w = e < 2 ? v.x : e < 4 ? v.y : e < 6 ? v.z : v.w;
    return widen16<F16>(uint16_t(e & 1 ? w >> 16 : w));
  };
  float a[V][8], b[GATED ? V : 1][8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int j = threadIdx.x + i * blockDim.x;
    if (j >= n8) continue;
    float w[8], wu[8];
    load8<0>(p.w.steps, j * 8, w);
    if constexpr (GATED) load8<0>(p.u.steps, j * 8, wu);
    uint32_t hg[4], hu[4];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float dg, du, bb;
      back_values<GATED, ACT>(half(rd[i], e), GATED ? half(rg[i], e) : 0.f,
                              GATED ? half(ru[i], e) : 0.f, w[e], GATED ? wu[e] : 0.f, a[i][e], bb,
                              dg, du);
      const uint32_t ma = finite_abs(a[i][e]);
      m = m > ma ? m : ma;
      if constexpr (GATED) {
        b[i][e] = bb;
        const uint32_t mb = finite_abs(bb);
        m = m > mb ? m : mb;
        const uint32_t g16 = round16<F16>(dg), u16 = round16<F16>(du);
        hg[e >> 1] = e & 1 ? hg[e >> 1] | g16 << 16 : g16;
        hu[e >> 1] = e & 1 ? hu[e >> 1] | u16 << 16 : u16;
      }
    }
    if constexpr (GATED) {
      *reinterpret_cast<uint4*>(p.dG + row + j * 8) = make_uint4(hg[0], hg[1], hg[2], hg[3]);
      *reinterpret_cast<uint4*>(p.dU + row + j * 8) = make_uint4(hu[0], hu[1], hu[2], hu[3]);
    }
  }
  const int e = row_exponent(block_max(m));
  const float down = pow2(-e);
  if (threadIdx.x == 0) p.E[t] = pow2(e);
  auto store = [&](const float (&v)[8], int64_t c) {
    float s[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) s[k] = v[k] * down;
    store8<2>(p.A, operand_at(p, t, c), s);
  };
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int j = threadIdx.x + i * blockDim.x;
    if (j >= n8) continue;
    store(a[i], j * 8);
    if constexpr (GATED) store(b[i], p.Np + j * 8);
  }
  // from N to Np: zeros
  const int pad = int((p.Np - p.N) >> 3);
  const float zero[8] = {};
  if (int(threadIdx.x) < pad) {
    store8<2>(p.A, operand_at(p, t, p.N + threadIdx.x * 8), zero);
    if constexpr (GATED) store8<2>(p.A, operand_at(p, t, p.Np + p.N + threadIdx.x * 8), zero);
  }
}

// The same for any N, element by element in two passes (a pair's gradient of 4096 tokens
// of 4096 inputs: 757 us for 11007 outputs, 650 for 11008).
template <bool F16, bool GATED, int ACT>
__global__ __launch_bounds__(256) void w8_grad_rows_any_kernel(const W8Back p) {
  const int64_t t = blockIdx.x;
  const int64_t row = t * p.N;
  auto values = [&](int64_t n, float& a, float& b, float& dg, float& du) {
    back_values<GATED, ACT>(widen16<F16>(p.dY[row + n]), GATED ? widen16<F16>(p.G[row + n]) : 0.f,
                            GATED ? widen16<F16>(p.U[row + n]) : 0.f, p.w.steps[n],
                            GATED ? p.u.steps[n] : 0.f, a, b, dg, du);
  };
  uint32_t m = 0;
  for (int64_t n = threadIdx.x; n < p.N; n += 256) {
    float a, b, dg, du;
    values(n, a, b, dg, du);
    const uint32_t ma = finite_abs(a), mb = finite_abs(b);
    m = m > ma ? m : ma;
    m = m > mb ? m : mb;
  }
  const int e = row_exponent(block_max(m));
  const float down = pow2(-e);
  if (threadIdx.x == 0) p.E[t] = pow2(e);
  for (int64_t n = threadIdx.x; n < p.Np; n += 256) {
    float a = 0.f, b = 0.f, dg, du;
    if (n < p.N) {
      values(n, a, b, dg, du);
      if constexpr (GATED) {
        p.dG[row + n] = round16<F16>(dg);
        p.dU[row + n] = round16<F16>(du);
      }
    }
    p.A[operand_at(p, t, n)] = round16<true>(a * down);
    if constexpr (GATED) p.A[operand_at(p, t, p.Np + n)] = round16<true>(b * down);
  }
}

// B in panels: 64 x 64 codes through LDS, as fp16 numbers, 8 KiB in one piece. grid
// (Np / 64, K / 64, layers).
__global__ __launch_bounds__(256) void w8_transpose_kernel(const W8Back p) {
  __shared__ uint32_t tile[64][17];   // [n][k / 4]
  const int64_t n0 = int64_t(blockIdx.x) * 64, k0 = int64_t(blockIdx.y) * 64;
  const int8_t* q = blockIdx.z ? p.u.q : p.w.q;
  const int r = threadIdx.x >> 2, c = threadIdx.x & 3;
  uint4 v = make_uint4(0, 0, 0, 0);
  if (n0 + r < p.N) v = *reinterpret_cast<const uint4*>(q + (n0 + r) * p.K + k0 + c * 16);
  tile[r][c * 4] = v.x;
  tile[r][c * 4 + 1] = v.y;
  tile[r][c * 4 + 2] = v.z;
  tile[r][c * 4 + 3] = v.w;
  __syncthreads();
  // row k of B: 16 consecutive n a thread
  const int k = threadIdx.x >> 2, nn = (threadIdx.x & 3) * 16;
  uint32_t h[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    h[i] = codes_to_f16(tile[nn + 2 * i][k >> 2], tile[nn + 2 * i + 1][k >> 2],
                        byte_pair(0) + 0x00010001u * (k & 3));
  const int64_t panel = int64_t(blockIdx.z) * (p.Np >> 6) + blockIdx.x;
  uint4* o = reinterpret_cast<uint4*>(p.B + (panel * p.K + k0 + k) * 64 + nn);
  o[0] = make_uint4(h[0], h[1], h[2], h[3]);
  o[1] = make_uint4(h[4], h[5], h[6], h[7]);
}

// Channels k .. k + 3 of a token.
template <bool F16>
__device__ __forceinline__ void store_dx(const W8Back& p, int64_t t, int64_t k, float e,
                                         floatx4 s) {
  const float y[4] = {s[0] * e, s[1] * e, s[2] * e, s[3] * e};
  store4<F16>(p.dX + t * p.K + k, true, 4, y);
}

// dX = E·(A·Bᵀ): the main loop's A rows are the channels k, so a lane holds 4
// consecutive ones of a token. Bound by the matrix cores.
template <bool F16, bool CUT>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(1, 1)))
void w8_back_gemm_kernel(const W8Back p, int steps, int tiles_t, int tiles_k) {
  const W8Unit unit = w8_unit<CUT>(p.cut, tiles_t, tiles_k);
  const int64_t t0 = int64_t(unit.tt) * BN, o0 = int64_t(unit.tn) * BM;
  const int64_t rows_o = p.K - o0 < BM ? p.K - o0 : BM;
  const int64_t rows_t = p.T - t0 < BN ? p.T - t0 : BN;
  int k0 = 0, k1 = steps;
  if constexpr (CUT) w8_run(p.cut, unit, steps, k0, k1);
  const int64_t panel_a = p.K * 64, panel_b = p.T * 64;
  RingCtx c;
  c.wave = uniform(int(threadIdx.x >> 6));
  c.a.set(RingKind::kPanels, p.B + k0 * panel_a + o0 * 64, int(rows_o), 128, c.wave * 64,
          panel_a * 2, k1 - k0);
  c.b.set(RingKind::kPanels, p.A + k0 * panel_b + t0 * 64, int(rows_t), 128, c.wave * 64,
          panel_b * 2, k1 - k0);
  floatx4 acc[8][8];
  ring_mainloop<f16x8_t>(c, acc);
  if (CUT && unit.slot >= 0) {
    w8_store_run(p.cut, unit, c.wave, acc);
    return;
  }
  const int lane = threadIdx.x & 63;
  const int wm = c.wave >> 1, wn = c.wave & 1;
  const int64_t tw = t0 + wn * 128, ow = o0 + wm * 128;
  const int left_t = int(rows_t) - wn * 128;
  if (left_t <= 0 || ow >= p.K) return;   // K is a multiple of 128
  const WaveTile<128> tile(c.wave);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int t = j * 16 + (lane & 15);
    const float e = p.E[tw + (t < left_t ? t : left_t - 1)];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const floatx4 s = from_agpr(acc[i][j]);
      const float y[4] = {s[0] * e, s[1] * e, s[2] * e, s[3] * e};
      tile.template put<F16>(t, i * 16 + 4 * (lane >> 4), y);
    }
  }
  tile.store(p.dX + tw * p.K + ow, uint32_t(p.K), left_t, 128);
}

// Workgroup (cut tile, wave, block row i) adds the runs of 16 channels x 128 tokens.
template <bool F16>
__global__ __launch_bounds__(256) void w8_back_gemm_sum_kernel(const W8Back p, int tiles_t,
                                                               int tiles_k) {
  const int cut = int(blockIdx.x), wave = int(blockIdx.y), i = int(blockIdx.z);
  const int lane = threadIdx.x & 63, tile = p.cut.full + cut;
  int tt, tk;
  w8_tile(tile, tiles_t, tiles_k, tt, tk);
  const int64_t t0 = int64_t(tt) * BN + (wave & 1) * 128 + (lane & 15);
  const int64_t k = int64_t(tk) * BM + (wave >> 1) * 128 + i * 16 + 4 * (lane >> 4);
  if (k >= p.K) return;
#pragma unroll
  for (int j = threadIdx.x >> 6; j < 8; j += 4) {
    const int64_t t = t0 + j * 16;
    if (t < p.T)
      store_dx<F16>(p, t, k, p.E[t], w8_sum_runs<floatx4>(p.cut, cut, wave, i, j));
  }
}

template <bool F16, bool GATED, int ACT>
hipError_t launch_rows(const W8Back& p, hipStream_t st) {
  const unsigned rows = unsigned(p.T);
  // steps are 16-byte aligned where a row of 8 values takes them at once
  const bool vec = p.N % 8 == 0 && p.N <= 32768 && p.vec;
  if (!vec) w8_grad_rows_any_kernel<F16, GATED, ACT><<<rows, 256, 0, st>>>(p);
  else if (p.N <= 2048) w8_grad_rows_kernel<F16, GATED, ACT, 1><<<rows, 256, 0, st>>>(p);
  else if (p.N <= 8192) w8_grad_rows_kernel<F16, GATED, ACT, 2><<<rows, 512, 0, st>>>(p);
  else if (p.N <= 16384) w8_grad_rows_kernel<F16, GATED, ACT, 2><<<rows, 1024, 0, st>>>(p);
  else w8_grad_rows_kernel<F16, GATED, ACT, 4><<<rows, 1024, 0, st>>>(p);
  return hipGetLastError();
}

template <bool F16>
hipError_t launch_back(const W8Back& p, hipStream_t st) {
  const bool gated = p.G != nullptr;
  const int steps = int((gated ? 2 : 1) * p.Np / 64);
  hipError_t e = !gated             ? launch_rows<F16, false, kSilu>(p, st)
                 : p.act == kSilu ? launch_rows<F16, true, kSilu>(p, st)
                                  : launch_rows<F16, true, kGelu>(p, st);
  if (e != hipSuccess) return e;
  if (p.few) return launch_w8_back_few(p, st);
  const dim3 grid(unsigned(p.Np / 64), unsigned(p.K / 64), gated ? 2 : 1);
  w8_transpose_kernel<<<grid, 256, 0, st>>>(p);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int tiles_t = int((p.T + BN - 1) / BN), tiles_k = int((p.K + BM - 1) / BM);
  if (!p.cut.runs) {
    w8_back_gemm_kernel<F16, false>
        <<<unsigned(tiles_t * tiles_k), NT, 0, st>>>(p, steps, tiles_t, tiles_k);
    return hipGetLastError();
  }
  const int cut = tiles_t * tiles_k - p.cut.full;
  w8_back_gemm_kernel<F16, true>
      <<<unsigned(p.cut.full + cut * p.cut.runs), NT, 0, st>>>(p, steps, tiles_t, tiles_k);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  w8_back_gemm_sum_kernel<F16><<<dim3(unsigned(cut), 4, 8), 256, 0, st>>>(p, tiles_t, tiles_k);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_w8_back(const W8Back& p, hipStream_t st) {
  return p.f16 ? launch_back<true>(p, st) : launch_back<false>(p, st);
}

}  // namespace awq
