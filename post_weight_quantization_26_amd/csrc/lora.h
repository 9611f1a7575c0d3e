// Arguments of the low-rank adapter kernels (lora.hip), shared with abi.cpp.
#pragma once

#include "device_common.h"

namespace awq {

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

struct LoraForward {
  const uint16_t* X;      // [T, K]
  int64_t T;
  LoraLayer w;
  LoraSet s;
  uint16_t* Y;            // [T, N]
  float* H;               // [T, r]
  int f16;
};

struct LoraBackward {
  const uint16_t* dY;     // [T, N]
  const void* X;          // [T, K] 16-bit, or int8 codes (then steps is set)
  const float* steps;     // [T, K / 128] or NULL
  const float* H;         // [T, r]
  int64_t T;
  LoraLayer w;
  LoraSet s;
  float* G;               // [T, r]
  uint16_t* dX;           // [T, K] or NULL
  uint16_t* dA;           // [L, r, K]
  uint16_t* dB;           // [L, N, r]
  int f16;
};

hipError_t launch_lora_forward(const LoraForward& p, hipStream_t st);
hipError_t launch_lora_backward(const LoraBackward& p, hipStream_t st);

// Activation checkpoints: codes [T, K] int8, steps [T, K / 128] float32.
hipError_t launch_act_pack8(const void* X, int dtype, int64_t T, int64_t K, int8_t* codes,
                            float* steps, hipStream_t st);
hipError_t launch_act_unpack8(const int8_t* codes, const float* steps, int dtype, int64_t T,
                              int64_t K, void* X, hipStream_t st);

}  // namespace awq
