// Arguments of the 8-bit layer's kernels (rows8.hip, norm.hip, w8_*.hip),
// shared with abi.cpp.
#pragma once

#include "device_common.h"

namespace awq {

// Rows of X [T, K] (times s [K], if given) to codes and steps.
struct QuantizeRows8 {
  const void* X;
  const float* s;
  int64_t T, K;
  int8_t* codes;
  float* steps;
};
hipError_t launch_quantize_rows8(const QuantizeRows8& p, int dtype, hipStream_t st);
hipError_t launch_dequantize_rows8(const int8_t* codes, const float* steps, int dtype, int64_t T,
                                   int64_t K, void* X, hipStream_t st);

// A norm of the rows of X [T, K].
struct Norm {
  const void* X;
  const void* gamma;   // [K], X's type or float32 (gamma32)
  const void* beta;    // like gamma, or NULL
  bool gamma32, rms;
  float eps;
  int64_t T, K;
  void* Y;             // [T, K], or NULL
  float* stats;        // [T, 2]: mean, 1 / deviation; or NULL
  int8_t* codes;       // [T, K] with steps [T], or NULL
  float* steps;
};
hipError_t launch_norm(const Norm& p, int dtype, hipStream_t st);

// Its gradient. partial: [2 (1 without dbeta), groups, Kp] float32 sums.
struct NormBack {
  const void* dY;
  const void* X;
  const float* stats;
  const void* gamma;
  bool gamma32, rms;
  int64_t T, K, Kp, groups;
  float* partial;
  void* dX;
  void* dgamma;        // gamma's type
  void* dbeta;         // or NULL
};
hipError_t launch_norm_back(const NormBack& p, int dtype, hipStream_t st);

// 256x256 tiles: those from `full` (a multiple of 256) on are cut into runs of the
// contraction, whose accumulators go to part [cut tiles, runs, 256·256]. runs 0:
// none is.
struct W8Cut {
  int full, runs;
  float* part;
};

// One 8-bit layer: codes [N, K], steps [N].
struct W8Layer {
  const int8_t* q;
  const float* steps;
};

// Y[t][n] = xs_t·w_n·Σ_k x[t][k]·q[n][k] + bias[n], or with a second layer u
// H[t][n] = act(G)·U. act: 0 silu, 1 gelu.
struct W8Product {
  const int8_t* x;
  const float* xs;
  W8Layer w, u;        // u.q NULL: a plain product
  const uint16_t* bias;
  int64_t T, N, K;
  int act;
  bool f16;
  uint16_t* Y;
  uint16_t* G;         // [T, N] products before the activation, or NULL
  uint16_t* U;
  // a few hundred tokens: rows of A (128 or 256) and tokens of a tile, runs of the
  // contraction, and for more than one run their sums [runs, layers, T, ldp]
  int tile_n, tile_t, runs;
  int64_t ldp;
  int* partial;
  W8Cut cut;           // many tokens
};
hipError_t launch_w8_few(const W8Product& p, hipStream_t st);
hipError_t launch_w8_mid(const W8Product& p, hipStream_t st);
hipError_t launch_w8_gemm(const W8Product& p, hipStream_t st);

// dX[t][k] = Σ_n (dY[t][n]·w_n)·q[n][k], or of a gated pair from dH, G and U.
struct W8Back {
  const uint16_t* dY;
  const uint16_t* G;   // NULL: a plain product
  const uint16_t* U;
  W8Layer w, u;
  int64_t T, N, K, Np; // Np: N rounded up to 64
  int act;
  bool f16;
  uint16_t* A;         // fp16 operand of [T, C], C = Np (twice that for a pair)
  float* E;            // [T] factor of a row of A
  uint16_t* B;         // many tokens: [K, C] codes as fp16
  uint16_t* dX;
  uint16_t* dG;        // a pair's
  uint16_t* dU;
  bool vec;            // the steps are 16-byte aligned
  bool few;            // no transposed layer: tokens of a tile, runs of the
  int tile_t, runs;    // contraction and, for more than one, their sums [runs, T, K]
  float* partial;
  W8Cut cut;           // many tokens
};
hipError_t launch_w8_back(const W8Back& p, hipStream_t st);

}  // namespace awq
