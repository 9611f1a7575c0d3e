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
// one is used. Bound by the reads of V; runs are chosen to keep every CU busy:
// bf16, 8192 tokens of 4096 channels, rank 16, with the checkpoint 23 us (102 MB,
// 4.4 TB/s); of 11008 channels, rank 64, 52 us (182 MB, 3.5 TB/s).
//
// Tokens may have any adapters: the workgroup walks the distinct adapters of
// its tokens, each a pass that keeps the rows belonging to it (the passes are
// dealt to up to 4 workgroups, so a tile where one prompt ends and the next
// begins takes no longer than another). An MFMA row depends on its own token
// only and rows of other adapters are dropped, not masked by zeros, so
// neither a token's nor an adapter's NaN reaches another.
#include "act8.h"
#include "lora.h"
#include "lora_combine.h"
#include "lora_common.h"
#include "lora_stage.h"
#include "w4a16_dequant.h"

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

template <bool F16>
__global__ __launch_bounds__(256) void lora_combine_kernel(LoraDown p) {
  lora_combine<F16>(p, blockIdx.x);
}
// The layer's dequantisation beside it: both come before the wide product and
// neither needs the other.
template <bool F16, bool WIDE>
__global__ __launch_bounds__(256, 8) void lora_combine_dequant_kernel(LoraDown p, LoraLayer w,
                                                                   uint16_t* __restrict__ Wd,
                                                                   int combines) {
  if (int(blockIdx.x) < combines) return lora_combine<F16>(p, blockIdx.x);
  const int64_t t = int64_t(int(blockIdx.x) - combines) * 256 + threadIdx.x;
  if constexpr (WIDE)
    dequant_words4<F16>(t, w.qweight, w.qzeros, w.scales, w.N, w.K, w.group, Wd);
  else dequant_words<F16>(t, w.qweight, w.qzeros, w.scales, w.N, w.K, w.group, Wd);
}

template <bool F16, int JB>
void launch_jb(const LoraDown& p, dim3 grid, hipStream_t st) {
  if (p.codes) lora_down_kernel<F16, JB, true><<<grid, kDownThreads, 0, st>>>(p);
  else lora_down_kernel<F16, JB, false><<<grid, kDownThreads, 0, st>>>(p);
}

template <bool F16>
void launch_sums(const LoraDown& p, hipStream_t st) {
  const unsigned combines = unsigned((p.T + 31) / 32 * 8);   // a multiple of the 8 XCDs
  if (p.after == LoraAfter::kSums) {
    lora_combine_kernel<F16><<<combines, 256, 0, st>>>(p);
  } else if (p.w.N % 32 == 0) {
    const unsigned grid = combines + unsigned((p.w.K / 8 * (p.w.N / 32) + 255) / 256);
    lora_combine_dequant_kernel<F16, true><<<grid, 256, 0, st>>>(p, p.w, p.Wd, int(combines));
  } else {
    const unsigned grid = combines + unsigned((p.w.K / 8 * (p.w.N / 8) + 255) / 256);
    lora_combine_dequant_kernel<F16, false><<<grid, 256, 0, st>>>(p, p.w, p.Wd, int(combines));
  }
}

template <bool F16>
hipError_t launch_f(const LoraDown& p, hipStream_t st) {
  const dim3 grid(unsigned((p.T + 63) / 64), unsigned(p.S), unsigned(p.L < 4 ? p.L : 4));
  if (p.r <= 16) launch_jb<F16, 1>(p, grid, st);
  else if (p.r <= 32) launch_jb<F16, 2>(p, grid, st);
  else if (p.r <= 64) launch_jb<F16, 4>(p, grid, st);
  else launch_jb<F16, 8>(p, grid, st);
  if (p.after != LoraAfter::kNothing) launch_sums<F16>(p, st);
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
