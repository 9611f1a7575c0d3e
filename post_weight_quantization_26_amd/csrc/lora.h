// Arguments of the low-rank adapter kernels (lora*.hip), shared with abi.cpp.
#pragma once

#include "device_common.h"

namespace awq {

constexpr int kLoraRankMax = 128;

// The packed 4-bit layer (quantize_pack's layout).
struct LoraLayer {
  const int32_t* qweight;
  const int32_t* qzeros;
  const uint16_t* scales;
  int64_t N, K;
  int group;
};

// The adapters and the tokens' ids.
struct LoraSet {
  const uint16_t* A;      // [L, r, K]
  const uint16_t* B;      // [L, N, r]
  const float* scaling;   // [L]
  const int32_t* ids;     // [T]
  int L, r;
};

// What follows the narrow product's partial sums: nothing (another launch adds
// them up), their sums, or these beside the dequantisation of w into Wd.
enum class LoraAfter { kNothing, kSums, kSumsAndLayer };
// The narrow product P[t][j] = Σ_c V[t][c]·M_a[j][c] (lora_down.hip).
struct LoraDown {
  LoraAfter after;
  LoraLayer w;
  uint16_t* Wd;           // [N, K]
  const uint16_t* V;      // [T, ldv]
  const uint16_t* M;      // [L, r, ldm]
  const float* scaling;
  const int32_t* ids;
  int64_t T, C, ldv, ldm; // C a multiple of 128
  int L, r, f16, S;       // S: runs of the contraction
  float* part;            // [S, T, r] their sums
  float* H;               // [T, r] or NULL; rows without an adapter get zeros
  const float* Hin;       // [T, r], with Ps
  float* Ps;              // P in the gradients' operand order, sorted by pos, or NULL
  float* Hs;              // Hin likewise
  const int32_t* pos;
  uint16_t* Q;            // [T, RW]: c·P as halves hi [r], lo [r], zeros up to RW, or NULL
  int RW;                 // 2r rounded up to 64
  float* E;               // [T] the power of two that Q is scaled down by
  int8_t* codes;          // [T, C] 8-bit checkpoint of V, or NULL
  float* steps;           // [T, C / 128]
};
hipError_t launch_lora_down(const LoraDown& p, hipStream_t st);

// The wide product's operands for a fused epilogue (lora_gemm.hip).
struct LoraUp {
  const uint16_t* Q;      // [T, RW]
  const float* E;         // [T]
  const int32_t* ids;     // [T]
  const uint16_t* U;      // [L, N, r]
  int L, r, RW;
};
// Tiles past the first `full` are cut into `runs` of the contraction (0 or 1:
// none is); part holds a 256x256 float32 tile for each of them.
struct LoraSplit {
  int full, runs;
  float* part;
};
hipError_t launch_lora_gemm(const uint16_t* V, int64_t ldv, const uint16_t* Wd, int64_t ldw,
                            int64_t M, int64_t N, int64_t C, const LoraUp& u,
                            const LoraSplit& sp, int f16, uint16_t* O, hipStream_t st);

// The float32 decode for N not a multiple of 16 (w4a16.hip).
hipError_t launch_w4a16_gemv(const uint16_t* X, int64_t T, int64_t N, int64_t K,
                             const int32_t* qweight, const int32_t* qzeros,
                             const uint16_t* scales, int group, int f16, int64_t kpw,
                             float* partial, hipStream_t st);

// Few tokens, forward (lora_few.hip).
struct LoraFew {
  const uint16_t* X;      // [T, K]
  int64_t T;
  LoraLayer w;
  LoraSet s;
  uint16_t* Y;            // [T, N]
  float* H;               // [T, r] or NULL
  float* partial;         // [S, T, N]
  float* hpart;           // [S2, T, r]
  int S, S2, kpw;         // runs of k of the two products; k rows per wave of the shared one
  int tiles, col_blocks;  // T > 16: token tiles and column blocks
  int gshift, gemv, f16;  // log2 of the group; T <= 16: the float32 decode
};
hipError_t launch_lora_few(const LoraFew& p, hipStream_t st);
// Its second launch alone.
hipError_t launch_lora_few_finish(const LoraFew& p, hipStream_t st);

// Few tokens, the shared product of the gradient (lora_few_back.hip).
struct LoraFewBack {
  const uint16_t* dY;     // [T, Np], zeros past N
  int64_t T, Np;
  LoraLayer w;
  float* partial;         // [S, T, K]
  int S, npw;             // runs of n; n per wave
  int tiles, col_blocks;
  int gshift, f16;
  LoraDown down;          // its sums are added up beside the product
};
hipError_t launch_lora_few_back(const LoraFewBack& p, hipStream_t st);

// A piece of one adapter's run of sorted tokens: positions pos .. pos + n - 1;
// slot of its partial sums, or -1 where it is the whole run.
struct LoraPiece {
  int a, pos, n, slot;
};
constexpr int kLoraMaxPiece = 2048;

// The gradient's preparation (lora_prep.hip).
struct LoraPrep {
  LoraLayer w;
  LoraSet s;
  int64_t T, Np;          // Np: N rounded up to 128
  int piece, f16;
  const uint16_t* dY;
  uint16_t* Wt;           // [K, Np], or NULL
  uint16_t* Bt;           // [L, r, Np]
  uint16_t* At;           // [L, K, r], or NULL
  uint16_t* dYp;          // [T, Np], or NULL where N = Np
  int* token;             // [Tp] token at each position
  int* pos;               // [T] position of each token with an adapter
  LoraPiece* pieces;      // adapters in order, one piece at least for each
  int* n_pieces;
  int* slots;             // [L] pieces of each adapter
  int* first_slot;        // [L]
  int* last_pos;          // [L]
};
struct LoraPrepGrid {
  uint32_t tb, ta, dq, pad;
  int waves;
};
hipError_t launch_lora_prep(const LoraPrep& p, hipStream_t st);

// The adapters' gradients (lora_grad.hip).
struct LoraGrad {
  const uint16_t* dY;     // [T, N]
  const void* X;          // [T, K] 16-bit, or int8 codes (then steps is set)
  const float* steps;     // [T, K / 128] or NULL
  const float* Gs;        // dY·B and H in operand order: [Tp / 32][16 ranks][lane][8]
  const float* Hs;
  const float* scaling;
  const int* token;
  const LoraPiece* pieces;
  const int* n_pieces;
  const int* slots;
  const int* first_slot;
  int64_t N, K;
  int L, r, f16;
  float* partial;         // [slots, (K + N)·r]
  uint16_t* dA;           // [L, r, K]
  uint16_t* dB;           // [L, N, r]
};
hipError_t launch_lora_grad(const LoraGrad& p, int pieces, bool sums, hipStream_t st);

// Activation checkpoints: codes [T, K] int8, steps [T, K / 128] float32.
hipError_t launch_act_pack8(const void* X, int dtype, int64_t T, int64_t K, int8_t* codes,
                            float* steps, hipStream_t st);
hipError_t launch_act_unpack8(const int8_t* codes, const float* steps, int dtype, int64_t T,
                              int64_t K, void* X, hipStream_t st);

}  // namespace awq
