// Gradients of the adapters,
//
//   dA_a[j][k] = c_a·Σ_t P[t][j]·X[t][k],   dB_a[n][j] = c_a·Σ_t dY[t][n]·H[t][j]
//
// over the tokens t of a, P = dY·B_a: products with a long contraction (tokens)
// and one narrow side (r). Both are Zᵀ·S with Z = X or dY, read once, and S
// the narrow side in the plan's sorted order. Bound by the reads of Z, with S,
// which every workgroup reads for its 128 columns, from L2: fp16, 2051 tokens of
// 4096x11008, rank 32: 21 us for 62 MB of Z; bf16, 8192 tokens of 11008x4096,
// rank 64, 8-bit X: 61 to 67 us for 213 MB. (S as halves from memory, and S loaded a
// step ahead, were no faster.)
//
// A workgroup takes 128 columns of Z, up to 64 ranks and one piece of a run;
// its 4 waves take every fourth step of 32 tokens. Z's rows, gathered through
// the plan, go to LDS by DMA a step ahead (a wave's own part: no barriers), 16
// lanes to a row's 256 bytes. A lane reads back 8 channels of 8 tokens; 32 byte
// permutes turn that 8x8 block into 8 MFMA operands of 8 tokens each, channel
// 8·(l % 16) + i for operand i. S lies in operand order ([step][16 ranks][lane]
// [8 tokens], lora_down.hip), so its loads are contiguous.
// S comes as float32 and is split in registers into two 16-bit halves, so
// that its rounding is u² (bf16 2^-16). fp16 halves are scaled by a power of two
// that takes the largest |S| of their rank so far to 2^14 (a value 2^-17 times
// as large still keeps 2^-22 of itself); where a step's is larger, the rank's
// sums are scaled down to match. Each rank has its own: a small one beside a
// large one, or beside one that is infinite, keeps its bits.
//
// An 8-bit checkpoint of X enters as its codes, exact in either 16-bit type, and
// its steps go into S: a strip of 128 channels has one step per token. The
// operands have the adapters' type: with fp16 ones under bf16 adapters g·step
// would leave their range where g itself does not.
//
// The waves add up in LDS in a fixed order. A run of one piece is finished
// here; pieces of a longer run leave float32 sums that lora_grad_sum_kernel adds
// in order. Runs never share a piece and padding repeats a run's last token
// with S = 0, so no adapter sees another's values.
#include "gemm_types.h"
#include "lora.h"
#include "lora_common.h"
#include "lora_stage.h"

namespace awq {
namespace {

constexpr int kGradWaves = 4;
constexpr int kGradStrip = 128;

typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

// Per wave: 32 tokens x 128 channels of Z.
typedef uint4 GradStage[kGradWaves][512];
static_assert(sizeof(GradStage) == 64 * kGradStrip * 4, "half of the waves' meeting place");

// Byte b of a word as a float32 number (a conversion with a byte select).
__device__ __forceinline__ float code_of(uint32_t w, int b) { return float(int8_t(w >> (8 * b))); }

template <bool F16, bool X8, int JB>
__device__ __forceinline__ void grad_piece(const LoraGrad& p, const LoraPiece& pc, bool is_a,
                                           int64_t strip, int j0, GradStage& z0, GradStage& z1,
                                           int* tokens) {
  constexpr int kCopies = X8 ? 4 : 8;          // 1 KiB each
  typedef typename Operand<F16>::type V;
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  const int64_t C = is_a ? p.K : p.N;
  const int jbs = (p.r + 15) / 16;
  const float* S = (is_a ? p.Gs : p.Hs) + int64_t(pc.pos / 32) * jbs * 512 + j0 / 16 * 512;
  const int64_t c0 = strip * kGradStrip;
  const int64_t KB = p.K / 128;

  // the piece's tokens, its padding included (positions are multiples of 32)
  const int padded = (pc.n + 31) / 32 * 32;
  for (int i = threadIdx.x; i < padded; i += 64 * kGradWaves) tokens[i] = p.token[pc.pos + i];
  __syncthreads();
  // Copy i brings rows 4i .. + 3 (8-bit: 8i .. + 7), 16 (8) lanes to a row; lanes
  // past the last column reread it.
  const char* Z = is_a ? static_cast<const char*>(p.X) : reinterpret_cast<const char*>(p.dY);
  constexpr int kRowLanes = X8 ? 8 : 16, kRows = 64 / kRowLanes, kBytes = X8 ? 1 : 2;
  const int64_t cb = (c0 + lane % kRowLanes * (16 / kBytes)) * kBytes;
  const int64_t colb = cb < C * kBytes ? cb : C * kBytes - 16;
  auto copy = [&](GradStage& st, int s) {
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      const int tok = tokens[s + kRows * i + lane / kRowLanes];
      __builtin_amdgcn_global_load_lds(
          (const __attribute__((address_space(1))) void*)(Z + int64_t(tok) * C * kBytes + colb),
          AWQ_LORA_LDS(st[wave] + 64 * i), 16, 0, 0);
    }
  };
  floatx4 acc[JB][8];
#pragma unroll
  for (int q = 0; q < JB; ++q)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[q][i] = floatx4{0.f, 0.f, 0.f, 0.f};
  // fp16: the exponent of the largest |S| so far of rank 16·q + lr
  int top[JB];
#pragma unroll
  for (int q = 0; q < JB; ++q) top[q] = kLeastExponent;

  auto use = [&](const GradStage& st, const float4 (&sv)[JB][2], const float (&step)[8], int s) {
    V sh[JB], sl[JB];
#pragma unroll
    for (int q = 0; q < JB; ++q) {
      const float4 a = sv[q][0], b = sv[q][1];
      float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if constexpr (X8) v[e] *= step[e];
        if (s + 8 * lg + e >= pc.n) v[e] = 0.f;
      }
      if constexpr (F16) {
        float m = fabsf(v[0]);
#pragma unroll
        for (int e = 1; e < 8; ++e) m = fmaxf(m, fabsf(v[e]));
        m = fmaxf(m, __shfl_xor(m, 16));
        m = fmaxf(m, __shfl_xor(m, 32));
        const int now = exponent_of(m);
        if (__ballot(now > top[q])) {
          const int to = now > top[q] ? now : top[q];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int down = __shfl(top[q] - to, 4 * lg + u);   // of the sums' rank
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[q][i][u] = __builtin_ldexpf(acc[q][i][u], down);
          }
          top[q] = to;
        }
        const float scale = exp2i(14 - top[q]);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= scale;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        hi[e] = pack2<F16>(v[2 * e], v[2 * e + 1]);
        lo[e] = pack2<F16>(v[2 * e] - widen16<F16>(uint16_t(hi[e])),
                          v[2 * e + 1] - widen16<F16>(uint16_t(hi[e] >> 16)));
      }
      sh[q] = __builtin_bit_cast(V, make_uint4(hi[0], hi[1], hi[2], hi[3]));
      sl[q] = __builtin_bit_cast(V, make_uint4(lo[0], lo[1], lo[2], lo[3]));
    }
    uint32_t z[8][X8 ? 2 : 4];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (X8) {
        const uint2 x =
            reinterpret_cast<const uint2*>(st[wave])[(8 * lg + e) * 16 + lr];
        z[e][0] = F16 ? x.x ^ 0x80808080u : x.x;
        z[e][1] = F16 ? x.y ^ 0x80808080u : x.y;
      } else {
        const uint4 x = st[wave][(8 * lg + e) * 16 + lr];
        z[e][0] = x.x;
        z[e][1] = x.y;
        z[e][2] = x.z;
        z[e][3] = x.w;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (X8 && !F16) {
          // the upper halves of two float32 codes
          w[e] = __builtin_amdgcn_perm(__float_as_uint(code_of(z[2 * e + 1][i >> 2], i & 3)),
                                       __float_as_uint(code_of(z[2 * e][i >> 2], i & 3)),
                                       0x07060302u);
        } else if constexpr (X8) {
          constexpr uint32_t kZero = 0x0C000C00u;
          const uint32_t b = i & 3;
          const uint32_t x = __builtin_amdgcn_perm(z[2 * e + 1][i >> 2], z[2 * e][i >> 2],
                                                   kZero | ((4u + b) << 16) | b);
          // fp16 1024 + (code + 128), less 1152: the code
          const f16x2_t v = __builtin_bit_cast(f16x2_t, x | 0x64006400u) -
                            f16x2_t{_Float16(1152.f), _Float16(1152.f)};
          w[e] = __builtin_bit_cast(uint32_t, v);
        } else {
          w[e] = __builtin_amdgcn_perm(z[2 * e + 1][i >> 1], z[2 * e][i >> 1],
                                       i & 1 ? 0x07060302u : 0x05040100u);
        }
      }
      const V zv = __builtin_bit_cast(V, make_uint4(w[0], w[1], w[2], w[3]));
#pragma unroll
      for (int q = 0; q < JB; ++q) {
        acc[q][i] = mfma_16x16x32(sh[q], zv, acc[q][i]);
        acc[q][i] = mfma_16x16x32(sl[q], zv, acc[q][i]);
      }
    }
  };
  // One step: S of this one, the copies of the next, a wait for all but the
  // copies, then the products. (Rank blocks past r read the last one again.)
  auto step = [&](const GradStage& st, GradStage& other, int s) {
    float4 sv[JB][2];
    float stp[8];
#pragma unroll
    for (int q = 0; q < JB; ++q) {
      const int jb = j0 / 16 + q < jbs ? q : jbs - 1 - j0 / 16;
      const float4* src =
          reinterpret_cast<const float4*>(S + (int64_t(s / 32) * jbs + jb) * 512) + 2 * lane;
      sv[q][0] = src[0];
      sv[q][1] = src[1];
    }
    if constexpr (X8)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        stp[e] = p.steps[int64_t(tokens[s + 8 * lg + e]) * KB + strip];
    wait_lds();
    fence();
    const int next = s + 32 * kGradWaves;
    if (next < pc.n) {
      copy(other, next);
      fence();
      wait_vmem<kCopies>();
    } else {
      wait_vmem<0>();
    }
    fence();
    use(st, sv, stp, s);
  };
  if (32 * wave < pc.n) {
    copy(z0, 32 * wave);
    for (int s = 32 * wave; s < pc.n; s += 64 * kGradWaves) {
      step(z0, z1, s);
      if (s + 32 * kGradWaves < pc.n) step(z1, z0, s + 32 * kGradWaves);
    }
  }
  __syncthreads();
  float(*const red[2])[kGradStrip] = {reinterpret_cast<float(*)[kGradStrip]>(&z0),
                                      reinterpret_cast<float(*)[kGradStrip]>(&z1)};
  // lane l holds channel 8·(l % 16) + i and ranks 16·q + 4·(l / 16) + v
  const float post = pc.n ? p.scaling[pc.a] : 0.f;   // no tokens: zeros
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    if (wave >> 1 == half) {
      float(*R)[kGradStrip] = red[wave & 1];
#pragma unroll
      for (int q = 0; q < JB; ++q)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          float* row = &R[16 * q + 4 * lg + v][8 * lr];
          const int up = F16 ? __shfl(top[q], 4 * lg + v) - 14 : 0;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float4 x = make_float4(acc[q][4 * h][v], acc[q][4 * h + 1][v], acc[q][4 * h + 2][v],
                                   acc[q][4 * h + 3][v]);
            if constexpr (F16)
              x = make_float4(__builtin_ldexpf(x.x, up), __builtin_ldexpf(x.y, up),
                              __builtin_ldexpf(x.z, up), __builtin_ldexpf(x.w, up));
            if (half) {
              const float4 y = *reinterpret_cast<const float4*>(row + 4 * h);
              x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
            }
            *reinterpret_cast<float4*>(row + 4 * h) = x;
          }
        }
    }
    __syncthreads();
  }
  // 8 consecutive values of the output's rows per thread: channels of dA
  // [r, K], ranks of dB [N, r]
  const int ranks = p.r - j0 < 16 * JB ? p.r - j0 : 16 * JB;
  const int items = ranks / 8 * kGradStrip;
  for (int e = threadIdx.x; e < items; e += 64 * kGradWaves) {
    int j, c;
    float v[8];
    if (is_a) {
      j = e / (kGradStrip / 8);
      c = e % (kGradStrip / 8) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = (red[0][j][c + i] + red[1][j][c + i]) * post;
    } else {
      c = e % kGradStrip;
      j = e / kGradStrip * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = (red[0][j + i][c] + red[1][j + i][c]) * post;
    }
    if (c0 + c >= C) continue;
    const int64_t at = is_a ? int64_t(j0 + j) * C + c0 + c : (c0 + c) * p.r + j0 + j;
    if (pc.slot < 0) {
      uint16_t* out = (is_a ? p.dA : p.dB) + int64_t(pc.a) * p.r * C + at;
      *reinterpret_cast<uint4*>(out) = make_uint4(pack2<F16>(v[0], v[1]), pack2<F16>(v[2], v[3]),
                                                  pack2<F16>(v[4], v[5]), pack2<F16>(v[6], v[7]));
    } else {
      float* out = p.partial + (int64_t(pc.slot) * (p.K + p.N) + (is_a ? 0 : p.K)) * p.r + at;
      *reinterpret_cast<float4*>(out) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(out + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
}

// Grid: strips of X then of dY; pieces; blocks of 16·JB ranks.
template <bool F16, bool X8, int JB>
__global__ __launch_bounds__(64 * kGradWaves, 2) void lora_grad_kernel(LoraGrad p) {
  // separate arrays, so that the compiler can tell the stage being read from
  // the one being filled
  __shared__ GradStage z0, z1;
  __shared__ int tokens[kLoraMaxPiece];
  if (int(blockIdx.y) >= *p.n_pieces) return;
  const LoraPiece pc = p.pieces[blockIdx.y];
  const int64_t sa = p.K / kGradStrip, strip = blockIdx.x;
  const int j0 = int(blockIdx.z) * 16 * JB;
  if (strip < sa) grad_piece<F16, X8, JB>(p, pc, true, strip, j0, z0, z1, tokens);
  else grad_piece<F16, false, JB>(p, pc, false, strip - sa, j0, z0, z1, tokens);
}

// The sum of a longer run's pieces, in order; 8 values per thread.
template <bool F16>
__global__ __launch_bounds__(256) void lora_grad_sum_kernel(LoraGrad p) {
  const int a = int(blockIdx.y), n = p.slots[a];
  if (n < 2) return;
  const int64_t ra = p.K * p.r, all = (p.K + p.N) * p.r;
  const int64_t i = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 8;
  if (i >= all) return;
  const float* src = p.partial + int64_t(p.first_slot[a]) * all + i;
  float v[8] = {};
  for (int q = 0; q < n; ++q) {
    const float4 x = *reinterpret_cast<const float4*>(src + q * all);
    const float4 y = *reinterpret_cast<const float4*>(src + q * all + 4);
    v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
    v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
  }
  uint16_t* out = i < ra ? p.dA + a * ra + i : p.dB + a * (all - ra) + (i - ra);
  *reinterpret_cast<uint4*>(out) = make_uint4(pack2<F16>(v[0], v[1]), pack2<F16>(v[2], v[3]),
                                              pack2<F16>(v[4], v[5]), pack2<F16>(v[6], v[7]));
}

template <bool F16, bool X8>
void launch_x8(const LoraGrad& p, int pieces, hipStream_t st) {
  const unsigned strips = unsigned(p.K / kGradStrip + (p.N + kGradStrip - 1) / kGradStrip);
  if (p.r <= 16)
    lora_grad_kernel<F16, X8, 1><<<dim3(strips, pieces, 1), 64 * kGradWaves, 0, st>>>(p);
  else if (p.r <= 32)
    lora_grad_kernel<F16, X8, 2><<<dim3(strips, pieces, 1), 64 * kGradWaves, 0, st>>>(p);
  else
    lora_grad_kernel<F16, X8, 4><<<dim3(strips, pieces, (p.r + 63) / 64), 64 * kGradWaves, 0,
                                   st>>>(p);
}

template <bool F16>
hipError_t launch_f(const LoraGrad& p, int pieces, bool sums, hipStream_t st) {
  if (p.steps) launch_x8<F16, true>(p, pieces, st);
  else launch_x8<F16, false>(p, pieces, st);
  if (sums) {
    const unsigned blocks = unsigned(((p.K + p.N) * p.r / 8 + 255) / 256);
    lora_grad_sum_kernel<F16><<<dim3(blocks, p.L), 256, 0, st>>>(p);
  }
  return hipGetLastError();
}

}  // namespace

// pieces: at least the plan's; sums: whether a run may have more than one.
hipError_t launch_lora_grad(const LoraGrad& p, int pieces, bool sums, hipStream_t st) {
  if (p.K % kGradStrip || p.N % 8 || p.r % 8 || pieces > 65535) return hipErrorInvalidValue;
  return p.f16 ? launch_f<true>(p, pieces, sums, st) : launch_f<false>(p, pieces, sums, st);
}

}  // namespace awq
