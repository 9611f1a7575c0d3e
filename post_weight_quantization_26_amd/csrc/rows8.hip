// Rows in 8 bits with one step each, the operands of the 8-bit products: a
// token's activations, or an output channel's weights times the scales s.
//
//   x' = fl32(x·s_k);  m = max(max |x'|, 2^-100);  step = fl32(m / 127)
//   code = rint(fl32(x'·fl32(127 / m)));  x^ = fl32(code·step)
//
// the arithmetic of an 8-bit checkpoint (act8.h) over a whole row: codes in
// -127..127, a row that holds a NaN or an infinity gets the step NaN.
#include "row_block.h"
#include "w8.h"

namespace awq {
namespace {

// Bound by HBM. A row stays in registers between its maximum and its codes, so
// X is read once; s comes from the caches.
template <int DT, int W, int V>
__global__ __launch_bounds__(kRowThreads<W>) void quantize_rows8_kernel(
    const void* __restrict__ X, const float* __restrict__ s, int64_t T, int K,
    int8_t* __restrict__ codes, float* __restrict__ steps) {
  __shared__ uint32_t red[16];
  const int64_t row = row_of<W>(blockIdx.x);
  if (row >= T) return;   // W = 1: no barrier follows; otherwise row < T
  const int t = row_thread<W>();
  float x[V][8];
#pragma unroll
  for (int c = 0; c < V; ++c) load_piece<DT, W>(X, row * K, K, c, t, x[c]);
  if (s) {
#pragma unroll
    for (int c = 0; c < V; ++c) {
      float f[8];
      load_piece<0, W>(s, 0, K, c, t, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[c][e] *= f[e];
    }
  }
  quantize_row<W, V>(x, row, K, t, red, codes, steps);
}

// x^ = code·step, 8 codes of a row a thread, 4 rows a workgroup apart loaded
// together. Bound by HBM.
template <int DT>
__global__ __launch_bounds__(256) void dequantize_rows8_kernel(const int8_t* __restrict__ codes,
                                                               const float* __restrict__ steps,
                                                               int64_t pieces, uint32_t per_row,
                                                               int K, void* __restrict__ X) {
  constexpr int U = 4;
  const int64_t p0 = int64_t(blockIdx.x) * (256 * U) + threadIdx.x;
  int64_t row[U];
  int col[U];
  float s[U];
  uint2 c[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t p = p0 + 256 * u;
    if (p >= pieces) break;
    row[u] = uint32_t(p) / per_row;      // pieces < 2^32
    col[u] = int(uint32_t(p) - uint32_t(row[u]) * per_row) * 8;
    s[u] = steps[row[u]];
    if (col[u] + 8 <= K) __builtin_memcpy(&c[u], codes + row[u] * K + col[u], 8);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (p0 + 256 * u >= pieces) break;
    const int64_t at = row[u] * K + col[u];
    if (col[u] + 8 <= K) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = float(int8_t(c[u].x >> (8 * e))) * s[u];
        v[4 + e] = float(int8_t(c[u].y >> (8 * e))) * s[u];
      }
      store_piece<DT, 1>(X, at, 8, 0, 0, v);
    } else {
      for (int e = 0; col[u] + e < K; ++e) store1<DT>(X, at + e, float(codes[at + e]) * s[u]);
    }
  }
}

template <int DT, int W, int V>
hipError_t launch_quantize(const QuantizeRows8& p, hipStream_t st) {
  quantize_rows8_kernel<DT, W, V><<<row_grid<W, V>(p.T), row_block<W, V>(p.K), 0, st>>>(
      p.X, p.s, p.T, int(p.K), p.codes, p.steps);
  return hipGetLastError();
}

// K up to 512·W·V. 16 columns a lane where a row fits 16 waves so: 28672 rows of 8192
// take 118 us, with 8 a lane 142, with 32 124.
template <int DT>
hipError_t launch_quantize_t(const QuantizeRows8& p, hipStream_t st) {
  if (p.K <= 512) return launch_quantize<DT, 1, 1>(p, st);
  if (p.K <= 1024) return launch_quantize<DT, 1, 2>(p, st);
  if (p.K <= 16384) return launch_quantize<DT, 16, 2>(p, st);
  if (p.K <= 32768) return launch_quantize<DT, 16, 4>(p, st);
  if (p.K <= 65536) return launch_quantize<DT, 16, 8>(p, st);
  return hipErrorInvalidValue;
}

template <int DT>
hipError_t launch_dequantize_t(const int8_t* codes, const float* steps, int64_t T, int64_t K,
                               void* X, hipStream_t st) {
  const int64_t per_row = (K + 7) / 8, pieces = T * per_row;
  if (pieces >= int64_t(1) << 32) return hipErrorInvalidValue;
  dequantize_rows8_kernel<DT><<<unsigned((pieces + 1023) / 1024), 256, 0, st>>>(
      codes, steps, pieces, uint32_t(per_row), int(K), X);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_rows8(const QuantizeRows8& p, int dtype, hipStream_t st) {
  if (dtype == 0) return launch_quantize_t<0>(p, st);
  if (dtype == 1) return launch_quantize_t<1>(p, st);
  return launch_quantize_t<2>(p, st);
}

hipError_t launch_dequantize_rows8(const int8_t* codes, const float* steps, int dtype, int64_t T,
                                   int64_t K, void* X, hipStream_t st) {
  if (dtype == 0) return launch_dequantize_t<0>(codes, steps, T, K, X, st);
  if (dtype == 1) return launch_dequantize_t<1>(codes, steps, T, K, X, st);
  return launch_dequantize_t<2>(codes, steps, T, K, X, st);
}

}  // namespace awq
