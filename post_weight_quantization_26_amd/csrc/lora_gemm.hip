// The wide half of the low-rank product, fused into the shared projection:
//
//   O[t][o] = Σ_c V[t][c]·Wd[o][c] + Σ_j q_t[j]·U_a[o][j],   a = ids[t],
//
// with Wd the packed layer rounded once to the 16-bit type (forward Ŵ [N, K],
// backward Ŵᵀ [K, N]), q_t = c_a·P[t] as two 16-bit halves (lora_down.hip) and
// U = B (forward) or Aᵀ (backward). The 256x256 main loop is the W4A16 GEMM's
// (gemm_core.h). The low-rank part is a few more MFMA steps on the same
// float32 accumulators: 2r / 32 steps per
// adapter in the tile against C / 32, so r = 16 over 4096 channels adds 1%
// of the work, and no float32 output ever goes to memory and back.
//
// It comes first, while the main loop's first copies are in flight, and the
// main loop adds to it.
//
// A tile's tokens may have any adapters. Where a wave's 128 rows have the same
// one (a prompt's), its U is loaded once for all of them. Otherwise, or where
// a q is scaled, each block of 16 rows takes every adapter it holds into fresh
// registers and keeps the rows that belong to it (a select, not a product
// with zero: an adapter's NaN stays with its own tokens).
#include "gemm_core.h"
#include "lora.h"
#include "lora_common.h"

namespace awq {
namespace {

__shared__ int sid[BM];
__shared__ float sE[BM];

// The low-rank part of one row block (rows row0 .. + 15) added to d.
template <bool F16>
__device__ __forceinline__ void expand_mixed(const LoraUp& u, const int* ids, const float* es,
                                             floatx4 (&d)[8], int64_t row0, int64_t col0,
                                             int64_t M, int64_t N) {
  typedef typename Operand<F16>::type V;
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const int nb8 = u.r / 8, steps = u.RW / 32;
  const int id = ids[lr];
  const int64_t row = row0 + lr;
  const uint16_t* qrow = u.Q + (row < M ? row : M - 1) * u.RW + 8 * lg;
  for (int a = next_adapter(id, -1, -1, u.L); a < u.L; a = next_adapter(id, -1, a, u.L)) {
    floatx4 t[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] = floatx4{0.f, 0.f, 0.f, 0.f};
    const uint16_t* ucol = u.U + int64_t(a) * N * u.r;
    int jb = lg % nb8;
    for (int s = 0; s < steps; ++s) {
      const V fq = __builtin_bit_cast(V, *reinterpret_cast<const uint4*>(qrow + 32 * s));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t col = col0 + 16 * j + lr;
        const V fu = __builtin_bit_cast(
            V, *reinterpret_cast<const uint4*>(ucol + (col < N ? col : N - 1) * u.r + 8 * jb));
        t[j] = mfma_16x16x32(fq, fu, t[j]);
      }
      jb = (jb + 4) % nb8;
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const bool mine = ids[4 * lg + v] == a;
      const float e = F16 ? es[4 * lg + v] : 1.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j][v] = mine ? __builtin_fmaf(e, t[j][v], d[j][v]) : d[j][v];
    }
  }
}

// The low-rank part of a wave's 128x128 outputs (rows row0 .., columns col0 ..
// of the problem). sid holds the tile's ids (-1: no adapter, or past the last
// token), sE the power of two that each token's q is scaled down by.
template <bool F16>
__device__ __forceinline__ void expand(const LoraUp& u, floatx4 (&acc)[8][8], int wm,
                                       int64_t row0, int64_t col0, int64_t M, int64_t N) {
  typedef typename Operand<F16>::type V;
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const int id0 = sid[wm * 128 + lane], id1 = sid[wm * 128 + 64 + lane];
  const int a = __builtin_amdgcn_readfirstlane(id0);
  bool same = __ballot(id0 == a && id1 == a) == ~0ull;
  if constexpr (F16)
    same = same &&
           __ballot(sE[wm * 128 + lane] == 1.f && sE[wm * 128 + 64 + lane] == 1.f) == ~0ull;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
  if (same) {
    if (a < 0) return;
    const int nb8 = u.r / 8, steps = u.RW / 32;
    const uint16_t* ucol = u.U + int64_t(a) * N * u.r;
    int jb = lg % nb8;                 // chunk 4·s + lg of [hi | lo], modulo r / 8
    for (int s = 0; s < steps; ++s) {
      V fu[8], fq[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t col = col0 + 16 * j + lr;
        fu[j] = __builtin_bit_cast(
            V, *reinterpret_cast<const uint4*>(ucol + (col < N ? col : N - 1) * u.r + 8 * jb));
      }
      jb = (jb + 4) % nb8;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t row = row0 + 16 * i + lr;
        fq[i] = __builtin_bit_cast(
            V, *reinterpret_cast<const uint4*>(u.Q + (row < M ? row : M - 1) * u.RW + 32 * s +
                                               8 * lg));
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = mfma_16x16x32(fq[i], fu[j], acc[i][j]);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    expand_mixed<F16>(u, &sid[wm * 128 + 16 * i], &sE[wm * 128 + 16 * i], acc[i], row0 + 16 * i,
                      col0, M, N);
}

// V [M, ldv] and Wd [N, ldw] with C columns each (a multiple of 64).
template <bool F16>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(1, 1)))
void lora_gemm_kernel(const uint16_t* __restrict__ X, int64_t ldv,
                      const uint16_t* __restrict__ Wd, int64_t ldw, int64_t M, int64_t N,
                      int64_t C, int tiles_m, int tiles_n, LoraUp u, uint16_t* __restrict__ O) {
  int tm, tn;
  if (!tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn)) return;
  const int64_t m0 = int64_t(tm) * BM, n0 = int64_t(tn) * BN;
  const int64_t rows_a = M - m0 < BM ? M - m0 : BM;
  const int64_t rows_b = N - n0 < BN ? N - n0 : BN;
  {
    const int64_t t = m0 + threadIdx.x;
    const int id = t < M ? u.ids[t] : -1;
    sid[threadIdx.x] = id >= 0 && id < u.L ? id : -1;
    if (F16) sE[threadIdx.x] = id >= 0 && id < u.L ? u.E[t] : 1.f;
  }
  GemmCtx64 c;
  gemm_setup64(c, X + m0 * ldv, rows_a, ldv, Wd + n0 * ldw, rows_b, ldw, C, false);
  __syncthreads();
  dma64<0>(c, 0);

  // lane l of block (i, j) holds column l % 16 and rows 4·(l/16) + v
  const int lane = threadIdx.x & 63;
  const int wm = c.wave >> 1, wn = c.wave & 1;
  const int64_t wrow = m0 + wm * 128, wcol = n0 + wn * 128;
  floatx4 acc[8][8];
  expand<F16>(u, acc, wm, wrow, wcol, M, N);
  // the accumulators are written by now; the first MFMA on them comes after
  // the main loop's barrier
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) asm volatile("" : "+a"(acc[i][j]));
  asm volatile("s_nop 15" ::: "memory");
  gemm_mainloop16<F16, true>(c, acc);

  const int64_t row0 = wrow + 4 * (lane >> 4);
  const int64_t col0 = wcol + (lane & 15);
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t col = col0 + j * 16;
      if (col >= N) continue;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int64_t row = row0 + i * 16 + v;
        if (row < M) O[row * N + col] = round16<F16>(acc[i][j][v]);
      }
    }
}

}  // namespace

// 512·ldv, 512·ldw < 2^31; 16-byte aligned rows; C a multiple of 64.
hipError_t launch_lora_gemm(const uint16_t* V, int64_t ldv, const uint16_t* Wd, int64_t ldw,
                            int64_t M, int64_t N, int64_t C, const LoraUp& u, int f16,
                            uint16_t* O, hipStream_t st) {
  if (C % 64 || ldv % 8 || ldw % 8 || u.r < 8 || u.r % 8) return hipErrorInvalidValue;
  const int tiles_m = int((M + BM - 1) / BM), tiles_n = int((N + BN - 1) / BN);
  const unsigned blocks = unsigned(gemm_blocks(tiles_m, tiles_n));
  if (f16)
    lora_gemm_kernel<true><<<blocks, NT, 0, st>>>(V, ldv, Wd, ldw, M, N, C, tiles_m, tiles_n, u,
                                                  O);
  else
    lora_gemm_kernel<false><<<blocks, NT, 0, st>>>(V, ldv, Wd, ldw, M, N, C, tiles_m, tiles_n, u,
                                                   O);
  return hipGetLastError();
}

}  // namespace awq
