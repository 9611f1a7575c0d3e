// Gradient of the 8-bit products, fewer tokens: dx[t][k] = E_t·Σ_c A[t][c]·q[c][k]
// straight from the codes, with no transposed layer in memory.
//
// The contraction runs over the layer's rows, the matrix instruction wants 8
// consecutive of them per lane. A lane loads 8 bytes (channels k) of each of 8
// rows c; byte i of the 8 is then one operand of the block of channels
// kb + 8·(l % 16) + i, so 8 blocks of 16 channels come from 8 loads of whole
// 128-byte lines, 3 vector instructions per two codes (w8_back.h), and no
// exchange between lanes. Block i's row r is channel kb + 8r + i: a lane ends up
// with 8 consecutive channels of a token, one 16-byte store.
//
// A workgroup owns 128 channels and 16·TB tokens; its waves take parts of the
// contraction (nothing is shared until their sums meet in LDS, in order), and
// runs of it go to more workgroups, whose float32 sums a second launch adds. The
// next 32 rows are loaded ahead. Bound by HBM up to some 64 tokens (each 64 read
// the codes again, from the caches), then by loads and conversion.
#include "w8_back.h"

namespace awq {
namespace {

constexpr int kBackWaves = 4;

// Waves of a SIMD: 8·TB accumulators of 4 registers leave room for 4, 3 or 2. Left
// to itself the compiler took 364 registers at TB = 4 (300 tokens of 11008x4096:
// 72 us instead of 59).
constexpr int back_waves(int tb) { return tb == 4 ? 2 : tb == 2 ? 3 : 4; }

template <bool F16, int TB, bool RUNS>
__global__ __launch_bounds__(kBackWaves * 64)
__attribute__((amdgpu_waves_per_eu(back_waves(TB)))) void w8_back_few_kernel(const W8Back p, int tiles_t) {
  __shared__ floatx4 sums[2][8 * TB * 64];
  // (scalars: the matrix instructions ignore the execution mask)
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  // an XCD's channel tiles with all their token tiles one after the other
  const int xcd = blockIdx.x & 7, id = blockIdx.x >> 3;
  const int tk = id / tiles_t * 8 + xcd, tt = id % tiles_t;
  const int64_t kb = int64_t(tk) * 128;
  if (kb >= p.K) return;
  const int tb = int((p.T + 15) >> 4);
  const int per_layer = int(p.Np >> 5), blocks = p.G ? 2 * per_layer : per_layer;
  const int parts = kBackWaves * p.runs, part = int(blockIdx.y) * kBackWaves + wave;
  const int last = int(int64_t(blocks) * (part + 1) / parts);
  int at = int(int64_t(blocks) * part / parts);

  // the lane's operand of A: 16 bytes of block (at, token block); token blocks
  // past the last are the last one again, not stored
  const uint4* a[TB];
#pragma unroll
  for (int j = 0; j < TB; ++j) {
    const int b = tt * TB + j;
    a[j] = reinterpret_cast<const uint4*>(p.A) + int64_t(b < tb ? b : tb - 1) * 64 + lane;
  }
  struct Batch {
    uint2 q[8];
    uint4 a[TB];
  };
  auto load = [&](Batch& d, int block) {
    if (block >= last) return;
    const bool second = block >= per_layer;
    const int8_t* q = (second ? p.u.q : p.w.q) + kb + 8 * r;
    const int64_t row = int64_t(second ? block - per_layer : block) * 32 + 8 * g;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // rows past N meet zeros of A
      const int64_t n = row + j < p.N ? row + j : p.N - 1;
      d.q[j] = *reinterpret_cast<const uint2*>(q + n * p.K);
    }
#pragma unroll
    for (int j = 0; j < TB; ++j) d.a[j] = a[j][int64_t(block) * tb * 64];
  };
  floatx4 acc[8][TB] = {};
  auto use = [&](const Batch& d, int block) {
    if (block >= last) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        h[j] = i < 4 ? codes_to_f16(d.q[2 * j].x, d.q[2 * j + 1].x, byte_pair(i))
                     : codes_to_f16(d.q[2 * j].y, d.q[2 * j + 1].y, byte_pair(i - 4));
      const f16x8_t f = __builtin_bit_cast(f16x8_t, make_uint4(h[0], h[1], h[2], h[3]));
#pragma unroll
      for (int j = 0; j < TB; ++j)
        acc[i][j] = mfma_16x16x32(f, __builtin_bit_cast(f16x8_t, d.a[j]), acc[i][j]);
    }
  };
  Batch d0, d1;
  load(d0, at);
  for (; at < last; at += 2) {
    load(d1, at + 1);
    use(d0, at);
    load(d0, at + 2);
    use(d1, at + 1);
  }

  // ((0 + 2) + (1 + 3)): waves 2 and 3, then wave 1, hand theirs over
  auto hand = [&](floatx4* to) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < TB; ++j) to[(i * TB + j) * 64 + lane] = acc[i][j];
  };
  auto take = [&](const floatx4* from) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < TB; ++j) acc[i][j] += from[(i * TB + j) * 64 + lane];
  };
  if (wave >= 2) hand(sums[wave - 2]);
  __syncthreads();
  if (wave < 2) take(sums[wave]);
  __syncthreads();
  if (wave == 1) hand(sums[0]);
  __syncthreads();
  if (wave) return;
  take(sums[0]);
#pragma unroll
  for (int j = 0; j < TB; ++j) {
    const int64_t t = (int64_t(tt) * TB + j) * 16 + r;
    if (t >= p.T) continue;
    const float e = RUNS ? 1.f : p.E[t];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int64_t k = kb + 8 * (4 * g + v);
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = acc[i][j][v] * e;
      if constexpr (RUNS)
        store8<0>(p.partial, (int64_t(blockIdx.y) * p.T + t) * p.K + k, y);
      else
        store8<F16 ? 2 : 1>(p.dX, t * p.K + k, y);
    }
  }
}

// Adds the runs' sums in their order: 8 channels of a token a thread.
template <bool F16>
__global__ __launch_bounds__(256) void w8_back_sum_kernel(const W8Back p) {
  const int64_t i = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 8, n = p.T * p.K;
  if (i >= n) return;
  float s[8];
  load8<0>(p.partial, i, s);
  for (int r = 1; r < p.runs; ++r) {
    float v[8];
    load8<0>(p.partial, int64_t(r) * n + i, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] += v[e];
  }
  const float e = p.E[i / p.K];
#pragma unroll
  for (int k = 0; k < 8; ++k) s[k] *= e;
  store8<F16 ? 2 : 1>(p.dX, i, s);
}

template <bool F16, int TB>
hipError_t launch_few(const W8Back& p, hipStream_t st) {
  const int tiles_t = int((p.T + 16 * TB - 1) / (16 * TB));
  const int64_t tiles_k = p.K / 128;
  const dim3 grid(unsigned((tiles_k + 7) / 8 * 8 * tiles_t), unsigned(p.runs));
  if (p.runs == 1) {
    w8_back_few_kernel<F16, TB, false><<<grid, kBackWaves * 64, 0, st>>>(p, tiles_t);
    return hipGetLastError();
  }
  w8_back_few_kernel<F16, TB, true><<<grid, kBackWaves * 64, 0, st>>>(p, tiles_t);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  w8_back_sum_kernel<F16><<<unsigned((p.T * p.K / 8 + 255) / 256), 256, 0, st>>>(p);
  return hipGetLastError();
}

template <bool F16>
hipError_t launch_few_t(const W8Back& p, hipStream_t st) {
  if (p.tile_t == 16) return launch_few<F16, 1>(p, st);
  if (p.tile_t == 32) return launch_few<F16, 2>(p, st);
  return launch_few<F16, 4>(p, st);
}

}  // namespace

// p.A in operand order, Np a multiple of 32.
hipError_t launch_w8_back_few(const W8Back& p, hipStream_t st) {
  return p.f16 ? launch_few_t<true>(p, st) : launch_few_t<false>(p, st);
}

}  // namespace awq
