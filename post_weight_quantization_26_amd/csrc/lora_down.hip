// The narrow half of the low-rank product,
//
//   P[t][j] = Σ_c V[t][c]·M_a[j][c],   a = ids[t], j < r <= 128,
//
// forward with V = X and M = A, backward with V = dY and M = Bᵀ (transposed
// by the preparation), in two launches: float32 partial sums over runs of the
// contraction, then their sum and what the other kernels read of it.
//
// A workgroup takes 64 tokens and a run of 128-wide blocks; its 4 waves take
// 16 tokens each and share the tile of M, so V is read once and M once per 64
// tokens. Both go to LDS by DMA (lora_stage.h), the next block in flight while
// one is used. Bound by the reads of V; runs are chosen to keep every CU busy.
//
// Tokens may have any adapters: the workgroup walks the distinct adapters of
// its tokens, each a pass that keeps the rows belonging to it (the passes are
// dealt to up to 4 workgroups, so a tile where one prompt ends and the next
// begins takes no longer than another). An MFMA row depends on its own token
// only and rows of other adapters are dropped, not masked by zeros, so
// neither a token's nor an adapter's NaN reaches another.
#include "act8.h"
#include "lora.h"
#include "lora_common.h"
#include "lora_stage.h"

namespace awq {
namespace {

constexpr int kDownWaves = 4;
constexpr int kDownThreads = 64 * kDownWaves;

// Two stages; separate arrays, so that the compiler can tell the one being
// read from the one being filled.
template <int JB>
struct DownLds {
  uint4 x[kDownWaves][kTile16], m[JB][kTile16];
};

struct DownCtx {
  __amdgpu_buffer_rsrc_t rsV, rsM;
  uint32_t voff[4], moff;
  int mstep;     // bytes from one 16-row tile of M to the next
  int wave;
};

template <int JB>
__device__ __forceinline__ void down_copy(const DownCtx& c, DownLds<JB>& l, int k) {
#pragma unroll
  for (int i = 0; i < 4; ++i) tile_copy(c.rsV, c.voff[i], k, l.x[c.wave], i);
  // wave w copies rows 4w .. + 3 of each tile of M
#pragma unroll
  for (int q = 0; q < JB; ++q)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(c.rsM, AWQ_LORA_LDS(l.m[q] + c.wave * 64), 16, c.moff,
                                             q * c.mstep + 2 * k, 0, 0);
}

template <bool F16, int JB>
__device__ __forceinline__ void down_block(const DownLds<JB>& l, int wave, floatx4 (&acc)[JB]) {
  typedef typename Operand<F16>::type V;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const V x = __builtin_bit_cast(V, tile_read(l.x[wave], s));
#pragma unroll
    for (int q = 0; q < JB; ++q)
      acc[q] = mfma_16x16x32(x, __builtin_bit_cast(V, tile_read(l.m[q], s)), acc[q]);
  }
}

// The 8-bit checkpoint of the wave's 16 tokens x 128 channels at block b.
template <bool F16, int JB>
__device__ __forceinline__ void down_pack(const DownLds<JB>& l, const LoraDown& p, int wave,
                                          int64_t t0, int b) {
  const int lane = threadIdx.x & 63, c = lane & 15;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 4 * i + (lane >> 4);
    const int64_t t = t0 + row;
    const uint4 x = tile_chunk(l.x[wave], row, c);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = widen16<F16>(uint16_t(w[e >> 1] >> (16 * (e & 1))));
    const Act8 q = act8_block(v, [](uint32_t m) { return row16_max(m); });
    if (t < p.T) {
      *reinterpret_cast<uint2*>(p.codes + t * p.C + int64_t(b) * 128 + 8 * c) = q.codes;
      if (c == 0) p.steps[t * (p.C / 128) + b] = q.step;
    }
  }
}

// Grid: token tiles, runs, slots. JB·16 >= r.
template <bool F16, int JB, bool PACK8>
__global__ __launch_bounds__(kDownThreads) void lora_down_kernel(LoraDown p) {
  __shared__ DownLds<JB> st0, st1;
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  const int64_t t0 = int64_t(blockIdx.x) * 64, tw = t0 + 16 * wave;
  const int nb = int(p.C / 128), slots = int(gridDim.z), slot = int(blockIdx.z);
  const int b0 = int(int64_t(nb) * blockIdx.y / p.S), b1 = int(int64_t(nb) * (blockIdx.y + 1) / p.S);
  const int id = t0 + lane < p.T ? p.ids[t0 + lane] : -1;

  DownCtx c;
  const int64_t rows = p.T - t0 < 64 ? p.T - t0 : 64;
  c.rsV = rows_rsrc(p.V + t0 * p.ldv, rows, p.ldv);
  c.wave = wave;
#pragma unroll
  for (int i = 0; i < 4; ++i) c.voff[i] = tile_offset(16 * wave, i, p.ldv);
  c.moff = tile_offset(0, wave, p.ldm);
  c.mstep = int(16 * p.ldm * 2);

  uint64_t left = __ballot(id >= 0 && id < p.L);
  bool pack = PACK8 && slot == 0;
  int turn = 0;
  while (left || pack) {
    // no adapter at all: the pass only packs, over adapter 0
    int a = 0;
    uint64_t mine = 0;
    if (left) {
      a = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
      mine = __ballot(id == a);
      left &= ~mine;
      if (turn++ % slots != slot) continue;
    }
    c.rsM = rows_rsrc(p.M + int64_t(a) * p.r * p.ldm, p.r, p.ldm);
    floatx4 acc[JB];
#pragma unroll
    for (int q = 0; q < JB; ++q) acc[q] = floatx4{0.f, 0.f, 0.f, 0.f};
    auto use = [&](const DownLds<JB>& l, int b) {
      if constexpr (PACK8) {
        if (pack) down_pack<F16, JB>(l, p, wave, tw, b);
      }
      down_block<F16, JB>(l, wave, acc);
    };
    // one barrier per block: every wave's copies of the block have landed, and
    // every wave has read what the next copies overwrite
    auto ready = [&] {
      __builtin_amdgcn_s_waitcnt(0xF | (3 << 14) | (0x7 << 4));   // lgkmcnt(0)
      wait_vmem<0>();
      __builtin_amdgcn_s_barrier();
    };
    down_copy(c, st0, b0 * 128);
    for (int b = b0; b < b1; b += 2) {
      ready();
      if (b + 1 < b1) down_copy(c, st1, (b + 1) * 128);
      use(st0, b);
      if (b + 1 >= b1) break;
      ready();
      if (b + 2 < b1) down_copy(c, st0, (b + 2) * 128);
      use(st1, b + 1);
    }
    pack = false;
    // lane l holds rows 4·(l / 16) + v and ranks 16·q + l % 16
    const uint32_t own = uint32_t(mine >> (16 * wave)) & 0xFFFFu;
    float* out = p.part + (int64_t(blockIdx.y) * p.T + tw + 4 * lg) * p.r + lr;
#pragma unroll
    for (int q = 0; q < JB; ++q)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (((own >> (4 * lg + v)) & 1u) && 16 * q + lr < p.r)
          out[int64_t(v) * p.r + 16 * q] = acc[q][v];
    __syncthreads();   // the next pass's copies overwrite what slower waves read
  }
}

// A wave per token: the sum of its partial sums, in order, as H, in the
// gradients' operand order (with Hin in the same), and as the wide product's
// operand c_a·P in two 16-bit halves hi = rnd(v), lo = rnd(v - hi), which lose at most u² (bf16: 2^-16) of v. fp16 halves are
// scaled by a power of two where a row's largest value lies outside [2^-3,
// 2^14), so that neither half overflows and lo keeps 2^-22 of the largest.
template <bool F16>
__global__ __launch_bounds__(256) void lora_combine_kernel(LoraDown p) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  const int64_t t = int64_t(blockIdx.x) * 4 + wave;
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
  float m = fmaxf(fabsf(v[0]), fabsf(v[1])), mh = fmaxf(fabsf(h[0]), fabsf(h[1]));
#pragma unroll
  for (int o = 32; o; o >>= 1) {
    m = fmaxf(m, __shfl_xor(m, o));
    mh = fmaxf(mh, __shfl_xor(mh, o));
  }
  const float c = p.scaling[a], cm = fabsf(c) * m;
  int e = 0;
  if (F16 && !(cm >= 0x1p-3f && cm < 0x1p14f)) e = exponent_of(cm);
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
  if (lane == 0) {
    if (p.Q) p.E[t] = exp2i(e);
    if (p.Ps) {
      p.row_max[pos] = m;
      p.h_max[pos] = mh;
    }
  }
}

template <bool F16, int JB>
void launch_jb(const LoraDown& p, dim3 grid, hipStream_t st) {
  if (p.codes) lora_down_kernel<F16, JB, true><<<grid, kDownThreads, 0, st>>>(p);
  else lora_down_kernel<F16, JB, false><<<grid, kDownThreads, 0, st>>>(p);
}

template <bool F16>
hipError_t launch_f(const LoraDown& p, hipStream_t st) {
  const dim3 grid(unsigned((p.T + 63) / 64), unsigned(p.S), unsigned(p.L < 4 ? p.L : 4));
  if (p.r <= 16) launch_jb<F16, 1>(p, grid, st);
  else if (p.r <= 32) launch_jb<F16, 2>(p, grid, st);
  else if (p.r <= 64) launch_jb<F16, 4>(p, grid, st);
  else launch_jb<F16, 8>(p, grid, st);
  lora_combine_kernel<F16><<<unsigned((p.T + 3) / 4), 256, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace

// 128·ldv, 256·ldm < 2^31.
hipError_t launch_lora_down(const LoraDown& p, hipStream_t st) {
  if (p.C % 128 || p.r < 8 || p.r > kLoraRankMax || p.r % 8 || p.S < 1 || p.S > p.C / 128)
    return hipErrorInvalidValue;
  return p.f16 ? launch_f<true>(p, st) : launch_f<false>(p, st);
}

}  // namespace awq
