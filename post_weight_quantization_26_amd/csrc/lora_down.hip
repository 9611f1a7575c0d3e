// The narrow half of the low-rank product,
//
//   P[t][j] = Σ_c V[t][c]·M_a[j][c],   a = ids[t], j < r <= 128,
//
// forward with V = X and M = A, backward with V = dY and M = Bᵀ (transposed
// by the preparation). One pass over V; M_a comes from L2.
//
// A workgroup takes 16·MT tokens; its 8 waves take the 128-wide blocks of the
// contraction in turn, so 16 tokens of 4096 channels are 32 blocks, 4 a wave,
// with every load of a block in flight at once. v_mfma_f32_16x16x32 operands
// come straight from memory: lane l holds 8 consecutive c of token l % 16 and
// of rank row l % 16. The waves meet in LDS in a fixed order.
//
// Tokens may have any adapters: the workgroup walks the distinct adapters of
// its tokens in rising order and each pass keeps the rows that belong to it
// (a long prompt has one; 16 decoding requests have up to 16, whose A_a are
// then all read, as they must be). An MFMA row depends on its own token only
// and rows of other adapters are dropped, not masked by zeros, so neither a
// token's nor an adapter's NaN reaches another.
//
// Output: P in float32 (H or, in sorted order and transposed, Gᵀ), and the
// operand of the wide half: c_a·P as two 16-bit halves hi = rnd(v), lo =
// rnd(v - hi), which lose at most u² (bf16: 2^-16) of v. fp16 halves are
// scaled by a power of two where a row's largest value lies outside [2^-3,
// 2^14), so that neither half overflows and lo keeps 2^-22 of the largest.
#include "act8.h"
#include "gemm_types.h"
#include "lora.h"
#include "lora_common.h"

namespace awq {
namespace {

constexpr int kDownWaves = 8;
constexpr int kDownThreads = 64 * kDownWaves;

// H as the gradients read it: transposed, in sorted order. 64 tokens a
// workgroup, a wave per token at a time.
__device__ __forceinline__ void transpose_h(const LoraDown& p, int64_t block) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int i = wave; i < 64; i += kDownWaves) {
    const int64_t t = block * 64 + i;
    if (t >= p.T) return;
    const int id = p.ids[t];
    if (id < 0 || id >= p.L) continue;
    const int pos = p.pos[t];
    float m = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int j = lane + 64 * h;
      if (j >= p.r) continue;
      const float v = p.Hin[t * p.r + j];
      p.Ht[int64_t(j) * p.ldp + pos] = v;
      m = fmaxf(m, fabsf(v));
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    if (lane == 0) p.h_max[pos] = m;
  }
}

// JB·16 >= min(r, 64): rank columns per pass (r above 64 takes two passes).
template <bool F16, int MT, int JB, bool PACK8>
__global__ __launch_bounds__(kDownThreads) void lora_down_kernel(LoraDown p) {
  typedef typename Operand<F16>::type V;
  constexpr int R = 16 * MT;
  __shared__ float red[kDownWaves][R][17];
  __shared__ float prod[R][kLoraRankMax + 1];
  __shared__ int sid[R];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int64_t t0 = int64_t(blockIdx.x) * R;
  if (t0 >= p.T) return transpose_h(p, int64_t(blockIdx.x) - (p.T + R - 1) / R);
  if (tid < R) sid[tid] = t0 + tid < p.T ? p.ids[t0 + tid] : -1;
  __syncthreads();
  const int my_id = lane < R ? sid[lane] : -1;

  // rows past the last token read the last one and are never stored
  const uint16_t* vrow[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int64_t t = t0 + 16 * m + lr;
    vrow[m] = p.V + (t < p.T ? t : p.T - 1) * p.ldv + 8 * lg;
  }
  const int nb = int(p.C / 128);
  bool pack = PACK8;
  int a = next_adapter(my_id, -1, -1, p.L);
  // tokens without an adapter: H is zero
  if (p.H)
    for (int e = tid; e < R * p.r; e += kDownThreads) {
      const int row = e / p.r;
      if (t0 + row < p.T && (sid[row] < 0 || sid[row] >= p.L))
        p.H[(t0 + row) * p.r + (e - row * p.r)] = 0.f;
    }
  while (a < p.L || pack) {
    const int am = a < p.L ? a : 0;   // no adapter at all: the pass only packs
    for (int j0 = 0; j0 < p.r; j0 += 16 * JB) {
      const uint16_t* mrow[JB];
#pragma unroll
      for (int q = 0; q < JB; ++q) {
        const int j = j0 + 16 * q + lr;
        mrow[q] = p.M + (int64_t(am) * p.r + (j < p.r ? j : p.r - 1)) * p.ldm + 8 * lg;
      }
      floatx4 acc[MT][JB];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int q = 0; q < JB; ++q) acc[m][q] = floatx4{0.f, 0.f, 0.f, 0.f};
      for (int b = wave; b < nb; b += kDownWaves) {
        uint4 x[MT][4], w[JB][4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
#pragma unroll
          for (int m = 0; m < MT; ++m)
            x[m][s] = *reinterpret_cast<const uint4*>(vrow[m] + int64_t(b) * 128 + 32 * s);
#pragma unroll
          for (int q = 0; q < JB; ++q)
            w[q][s] = *reinterpret_cast<const uint4*>(mrow[q] + int64_t(b) * 128 + 32 * s);
        }
        if constexpr (PACK8) {
          // the block's 128 channels of a token lie in the 4 lanes lr + 16·i
          if (pack && j0 == 0) {
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              float v[4][8];
              uint32_t mx = 0;
#pragma unroll
              for (int s = 0; s < 4; ++s) {
                const uint32_t ww[4] = {x[m][s].x, x[m][s].y, x[m][s].z, x[m][s].w};
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  v[s][e] = widen16<F16>(uint16_t(ww[e >> 1] >> (16 * (e & 1))));
                const uint32_t u = act8_abs_max(v[s]);
                mx = mx > u ? mx : u;
              }
#pragma unroll
              for (int o = 16; o <= 32; o *= 2) {
                const uint32_t u = __shfl_xor(mx, o);
                mx = mx > u ? mx : u;
              }
              const Act8Scale sc = act8_scale(mx);
              const int64_t t = t0 + 16 * m + lr;
              if (t < p.T) {
#pragma unroll
                for (int s = 0; s < 4; ++s)
                  *reinterpret_cast<uint2*>(p.codes + t * p.C + int64_t(b) * 128 + 32 * s +
                                            8 * lg) = act8_codes(v[s], sc);
                if (lg == 0) p.steps[t * nb + b] = sc.step;
              }
            }
          }
        }
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int q = 0; q < JB; ++q)
              acc[m][q] = mfma_16x16x32(__builtin_bit_cast(V, x[m][s]),
                                        __builtin_bit_cast(V, w[q][s]), acc[m][q]);
      }
      // lane l holds rows 4·(l / 16) + v and column l % 16 of every block
#pragma unroll
      for (int q = 0; q < JB; ++q) {
        if (j0 + 16 * q >= p.r) break;
        __syncthreads();
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int v = 0; v < 4; ++v) red[wave][16 * m + 4 * lg + v][lr] = acc[m][q][v];
        __syncthreads();
        for (int e = tid; e < R * 16; e += kDownThreads) {
          const int row = e >> 4, j = e & 15;
          float s = red[0][row][j];
#pragma unroll
          for (int w = 1; w < kDownWaves; ++w) s += red[w][row][j];
          if (j0 + 16 * q + j < p.r) prod[row][j0 + 16 * q + j] = s;
        }
      }
    }
    pack = false;
    __syncthreads();
    if (a < p.L) {
      const float c = p.scaling[a];
      for (int row = wave; row < R; row += kDownWaves) {
        const int64_t t = t0 + row;
        if (sid[row] != a) continue;   // (rows past T have the id -1)
        float v[2], m = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int j = lane + 64 * h;
          v[h] = j < p.r ? prod[row][j] : 0.f;
          m = fmaxf(m, fabsf(v[h]));
        }
#pragma unroll
        for (int o = 32; o; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
        const float cm = fabsf(c) * m;
        int e = 0;
        if (F16 && !(cm >= 0x1p-3f && cm < 0x1p14f)) e = exponent_of(cm);
        const float down = exp2i(-e);
        uint16_t* q = p.Q + t * p.RW;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int j = lane + 64 * h;
          if (j >= p.r) continue;
          if (p.H) p.H[t * p.r + j] = v[h];
          if (p.Pt) p.Pt[int64_t(j) * p.ldp + p.pos[t]] = v[h];
          const float s = c * v[h] * down;
          const uint16_t hi = round16<F16>(s);
          q[j] = hi;
          q[p.r + j] = round16<F16>(s - widen16<F16>(hi));
        }
        for (int j = 2 * p.r + lane; j < p.RW; j += 64) q[j] = 0;
        if (lane == 0) {
          p.E[t] = exp2i(e);
          if (p.row_max) p.row_max[p.pos[t]] = m;
        }
      }
    }
    a = a < p.L ? next_adapter(my_id, -1, a, p.L) : p.L;
    __syncthreads();
  }
}

template <bool F16, int MT, int JB>
hipError_t launch_jb(const LoraDown& p, hipStream_t st) {
  // the tokens' tiles, then H's
  const unsigned grid =
      unsigned((p.T + 16 * MT - 1) / (16 * MT) + (p.Hin ? (p.T + 63) / 64 : 0));
  if (p.codes) lora_down_kernel<F16, MT, JB, true><<<grid, kDownThreads, 0, st>>>(p);
  else lora_down_kernel<F16, MT, JB, false><<<grid, kDownThreads, 0, st>>>(p);
  return hipGetLastError();
}

template <bool F16, int MT>
hipError_t launch_mt(const LoraDown& p, hipStream_t st) {
  if (p.r <= 16) return launch_jb<F16, MT, 1>(p, st);
  if (p.r <= 32) return launch_jb<F16, MT, 2>(p, st);
  return launch_jb<F16, MT, 4>(p, st);
}

template <bool F16>
hipError_t launch_f(const LoraDown& p, hipStream_t st) {
  // Wider token tiles read each adapter's M from L2 less often; they are
  // taken once they still give a workgroup to every CU.
  if (p.T >= 16 * 4 * 256) return launch_mt<F16, 4>(p, st);
  if (p.T >= 16 * 2 * 256) return launch_mt<F16, 2>(p, st);
  return launch_mt<F16, 1>(p, st);
}

}  // namespace

hipError_t launch_lora_down(const LoraDown& p, hipStream_t st) {
  if (p.C % 128 || p.r < 8 || p.r > kLoraRankMax || p.r % 8) return hipErrorInvalidValue;
  return p.f16 ? launch_f<true>(p, st) : launch_f<false>(p, st);
}

}  // namespace awq
