// The sums of the narrow product (lora_down.hip, lora_few_back.hip).
#pragma once

#include "lora.h"
#include "lora_common.h"

namespace awq {
namespace {

// A wave per token (4 to a workgroup): the sum of its partial sums, in order, as H, in the
// gradients' operand order (with Hin in the same), and as the wide product's
// operand c_a·P in two 16-bit halves hi = rnd(v), lo = rnd(v - hi), which lose at most u² (bf16: 2^-16) of v. fp16 halves are
// scaled by a power of two where a row's largest value lies outside [2^-3,
// 2^14), so that neither half overflows and lo keeps 2^-22 of the largest.
template <bool F16>
__device__ __forceinline__ void lora_combine(const LoraDown& p, int64_t block) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  const int64_t t = block * 4 + wave;
  if (t >= p.T) return;
  const int a = p.ids[t];
  const bool has = a >= 0 && a < p.L;
  if (!has && !p.H) return;
  float v[2] = {0.f, 0.f}, h[2] = {0.f, 0.f};
  if (has)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int j = lane + 64 * k;
      if (j >= p.r) continue;
      const float* src = p.part + t * p.r + j;
#pragma unroll 4
      for (int s = 0; s < p.S; ++s) v[k] += src[int64_t(s) * p.T * p.r];
      if (p.Hin) h[k] = p.Hin[t * p.r + j];
    }
  if (p.H)
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (lane + 64 * k < p.r) p.H[t * p.r + lane + 64 * k] = v[k];
  if (!has) return;
  const float c = p.scaling[a];
  int e = 0;
  if constexpr (F16) {
    float m = fmaxf(fabsf(v[0]), fabsf(v[1]));
#pragma unroll
    for (int o = 32; o; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    const float cm = fabsf(c) * m;
    if (!(cm >= 0x1p-3f && cm < 0x1p14f)) e = exponent_of(cm);
  }
  const float down = exp2i(-e);
  uint16_t* q = p.Q + t * p.RW;
  const int pos = p.Ps ? p.pos[t] : 0;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int j = lane + 64 * k;
    if (j >= p.r) continue;
    if (p.Ps) {
      // [step of 32 positions][16 ranks][lane][8 positions] (lora_grad.hip)
      const int64_t at = ((int64_t(pos >> 5) * ((p.r + 15) / 16) + (j >> 4)) * 64 +
                          ((pos >> 3) & 3) * 16 + (j & 15)) * 8 + (pos & 7);
      p.Ps[at] = v[k];
      p.Hs[at] = h[k];
    }
    if (!p.Q) continue;
    const float s = c * v[k] * down;
    const uint16_t hi = round16<F16>(s);
    q[j] = hi;
    q[p.r + j] = round16<F16>(s - widen16<F16>(hi));
  }
  if (p.Q)
    for (int j = 2 * p.r + lane; j < p.RW; j += 64) q[j] = 0;
  if (lane == 0 && p.Q) p.E[t] = exp2i(e);
}

}  // namespace
}  // namespace awq
