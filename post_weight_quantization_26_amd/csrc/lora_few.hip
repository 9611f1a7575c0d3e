// Low-rank adapters for few tokens (decoding requests, short prompts), in two
// launches:
//
//  1. the shared product as float32 partial sums over runs of k, and beside
//     it, in workgroups of their own, the narrow products A_a·x;
//  2. the sum of the partials, the wide product B_a·h of each token's adapter,
//     one rounding, and H if it is wanted.
//
// Both are bound by the bytes of the packed layer and of the adapters in use:
// nothing but partial sums goes to memory in between, and the adapters' reads
// overlap the layer's.
//
// The shared product, T <= 16: the matrix-core decode of w4a16.hip (exact Ŵ).
// Above: a wave takes 16·MT tokens x 128 outputs and a run of k. Lane l holds
// k rows 8·(l / 16) .. + 7 of word column l % 16, so nibble r of its 8 words
// is the MFMA operand of outputs 8·(l % 16) + r; the words become the rounded
// Ŵ in registers, as the dequantisation pass rounds it:
//   the codes of two k rows, put in the halves of a word by one byte permute,
//   turn into fp16 numbers B + q by one and-or (B = 1024 for the low nibble
//   of a byte, 64 for the high one);
//   fp16: (B + q) - (B + z) exactly, times scale, rounded once;
//   bf16: float32 fma((B + q), scale, -(B + z)·scale), which is (q - z)·scale
//   exactly, rounded once.
// Each word serves 16·MT tokens. X and the words come through LDS by copies of
// 16 bytes a lane, a stage or two ahead of their use.
//
// What bounds it is the issue of vector instructions, not the memory: nibble by
// nibble 4.5 of them make a pair of weights, one MFMA per 16 tokens uses four
// pairs, and a SIMD starts one of either every 4.7 cycles, however many waves
// it has (with every read of X and the words from one cached place the time is
// the same; without the MFMAs, or without the dequantisation, it is a quarter
// less). 28672x8192, bf16, no adapters: 64 tokens 52 us, 32 tokens 36 us, 17
// tokens 33 us; loads of single words to registers in place of the copies: 53
// and 41. Tried and slower: eight waves that share X (56), 128 tokens a wave
// (55 against 44 us for 200 tokens of 4096x11008).
#include <type_traits>

#include "lora.h"
#include "lora_few.h"
#include "w4a16_mgemv.h"

namespace awq {
namespace {

// ---------------------------------------------------------------------------
// launch 1: the narrow product
// ---------------------------------------------------------------------------

// Slots for the distinct adapters of a tile of 16 tokens.
__host__ __device__ inline int few_slots(const LoraFew& p) {
  const int rows = p.T < 16 ? int(p.T) : 16;
  return rows < p.s.L ? rows : p.s.L;
}
// Workgroup (tile of 16 tokens, slot, block of 16 ranks, run of k): the 16 x 16
// block of P of the tile's slot-th adapter for all rows that have it, as a
// float32 partial sum.
__device__ __forceinline__ void few_down_index(const LoraFew& p, int id, int& tile, int& slot,
                                               int& jb, int& ks) {
  const int jbs = (p.s.r + 15) / 16, slots = few_slots(p);
  ks = id % p.S2;
  id /= p.S2;
  jb = id % jbs;
  id /= jbs;
  slot = id % slots;
  tile = id / slots;
}

// A wave's stage: a 16-row tile of X and one of A (lora_stage.h).
struct FewStage {
  uint4 *x, *a;
};
typedef float FewRed[kFewWaves][16][17];     // the waves' meeting

template <bool F16>
__device__ __forceinline__ void few_down(const LoraFew& p, int id, FewStage s0, FewStage s1,
                                         FewRed& red) {
  typedef typename Operand<F16>::type V;
  int tile, slot, jb, ks;
  few_down_index(p, id, tile, slot, jb, ks);
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  const int64_t t0 = int64_t(tile) * 16, K = p.w.K;
  const int my = t0 + lr < p.T ? p.s.ids[t0 + lr] : -1;
  uint32_t left = uint32_t(__ballot(my >= 0 && my < p.s.L)) & 0xFFFFu, mine;
  int a;
  while (true) {
    if (!left) return;
    a = __builtin_amdgcn_readlane(my, __builtin_ctz(left));
    mine = uint32_t(__ballot(my == a)) & 0xFFFFu;
    if (slot-- == 0) break;
    left &= ~mine;
  }
  const int nb = int(K / 128), b0 = int(int64_t(nb) * ks / p.S2),
            b1 = int(int64_t(nb) * (ks + 1) / p.S2);
  const int64_t rows = p.T - t0 < 16 ? p.T - t0 : 16;
  const int ranks = p.s.r - 16 * jb < 16 ? p.s.r - 16 * jb : 16;
  const auto rsX = rows_rsrc(p.X + t0 * K, rows, K);
  const auto rsA = rows_rsrc(p.s.A + (int64_t(a) * p.s.r + 16 * jb) * K, ranks, K);
  uint32_t off[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) off[i] = tile_offset(0, i, K);
  auto copy = [&](const FewStage& st, int b) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      tile_copy(rsX, off[i], 128 * b, st.x, i);
      tile_copy(rsA, off[i], 128 * b, st.a, i);
    }
  };
  floatx4 acc = {0.f, 0.f, 0.f, 0.f};
  auto use = [&](const FewStage& st) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
      acc = mfma_16x16x32(__builtin_bit_cast(V, tile_read(st.x, s)),
                          __builtin_bit_cast(V, tile_read(st.a, s)), acc);
  };
  // a wave reads only what it copied itself: waits, no barriers
  for (int b = b0 + wave; b < b1; b += 2 * kFewWaves) {
    copy(s0, b);
    if (b + kFewWaves < b1) copy(s1, b + kFewWaves);
    wait_vmem<0>();
    fence();
    use(s0);
    if (b + kFewWaves < b1) use(s1);
    wait_lds();
    fence();
  }
  __syncthreads();
#pragma unroll
  for (int v = 0; v < 4; ++v) red[wave][4 * lg + v][lr] = acc[v];
  __syncthreads();
  const int i = threadIdx.x >> 4, jj = threadIdx.x & 15;
  if (((mine >> i) & 1u) && 16 * jb + jj < p.s.r)
    p.hpart[(int64_t(ks) * p.T + t0 + i) * p.s.r + 16 * jb + jj] =
        ((red[0][i][jj] + red[1][i][jj]) + red[2][i][jj]) + red[3][i][jj];
}

// ---------------------------------------------------------------------------
// launch 1: the shared product, T > 16
// ---------------------------------------------------------------------------

// Stages of 64 k rows. The packed words of a wave lie, for each block of 32 k
// rows, in the order of their use: word e of lane l (k row 8·(l / 16) + e, word
// column l % 16) at 64·e + l.
typedef uint4 FewQ[kFewWaves][2 * 128];

// The zero points and scales of the group that one (group size 32) or two (64,
// 128) blocks lie in.
struct FewGroup {
  uint32_t z;
  uint4 s;
};
// What its nibbles need of it: -(B + z)·scale (bf16), or B + z as a pair (fp16).
template <bool F16>
struct FewZeros {
  typename std::conditional<F16, f16x2_t, float>::type v[8];
};

// Codes R of words a and b in the halves of a word, as fp16 numbers B + q.
template <int R>
__device__ __forceinline__ f16x2_t few_code(uint32_t a, uint32_t b, const uint32_t (&base)[2]) {
  constexpr uint32_t kSel = 0x0C000C00u | uint32_t(4 + R / 2) << 16 | uint32_t(R / 2);
  constexpr uint32_t kMask = R & 1 ? 0x00F000F0u : 0x000F000Fu;
  return __builtin_bit_cast(f16x2_t, (__builtin_amdgcn_perm(b, a, kSel) & kMask) | base[R & 1]);
}
template <int R>
__device__ __forceinline__ _Float16 few_scale(const FewGroup& gr) {
  const uint32_t sw = R / 2 == 0 ? gr.s.x : R / 2 == 1 ? gr.s.y : R / 2 == 2 ? gr.s.z : gr.s.w;
  return __builtin_bit_cast(_Float16, uint16_t(sw >> (16 * (R & 1))));
}
template <bool F16, int R = 0>
__device__ __forceinline__ void few_zeros(FewZeros<F16>& n, const FewGroup& gr,
                                          const uint32_t (&base)[2]) {
  if constexpr (R < 8) {
    const f16x2_t z = few_code<R>(gr.z, gr.z, base);
    if constexpr (F16) n.v[R] = z;
    else n.v[R] = -(float(z[0]) * float(few_scale<R>(gr)));
    few_zeros<F16, R + 1>(n, gr, base);
  }
}
// The operands of a block: nibble R of the 8 words, pair E of k rows 2E, 2E + 1.
template <bool F16>
struct FewBlock {
  const uint32_t (&w)[8];
  const FewGroup& gr;
  const FewZeros<F16>& n;
  const uint32_t (&base)[2];
  __device__ static constexpr int word(int e) { return e; }
  template <int R, int E>
  __device__ __forceinline__ void pair(uint32_t& lo, uint32_t& hi) const {
    const f16x2_t q = few_code<R>(w[2 * E], w[2 * E + 1], base);
    const _Float16 s = few_scale<R>(gr);
    if constexpr (F16) {
      lo = __builtin_bit_cast(uint32_t, (q - n.v[R]) * f16x2_t{s, s});
    } else {
      lo = __builtin_bit_cast(uint32_t, __builtin_fmaf(float(q[0]), float(s), n.v[R]));
      hi = __builtin_bit_cast(uint32_t, __builtin_fmaf(float(q[1]), float(s), n.v[R]));
    }
  }
};

// WIDE: N a multiple of 32, rows of packed words 16-byte aligned.
template <bool F16, int MT, bool G32, bool WIDE>
__device__ __forceinline__ void few_product(const LoraFew& p, int id, int blocks, FewX<MT>& sx,
                                            FewQ& q0, FewQ& q1) {
  typedef typename Operand<F16>::type V;
  constexpr int R = 16 * MT;
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  const int64_t N = p.w.N, K = p.w.K, N8 = N / 8;
  // XCD i takes a contiguous run of (run of k, column block, token tile)
  // indices, token tiles fastest: the tiles that read the same packed words
  // and neighbouring column blocks, whose row segments share cache lines, meet
  // in one L2
  int tt, cb, s;
  {
    const int q = blocks / 8, rem = blocks % 8, xi = id % 8;
    int l = xi * q + (xi < rem ? xi : rem) + id / 8;
    tt = l % p.tiles;
    l /= p.tiles;
    cb = l % p.col_blocks;
    s = l / p.col_blocks;
  }
  const int64_t t0 = int64_t(tt) * R, n0 = int64_t(cb) * kFewCols;
  const int kw0 = (s * kFewWaves + wave) * p.kpw;
  const int kw1 = kw0 + p.kpw < int(K) ? kw0 + p.kpw : int(K);
  floatx4 acc[8][MT];
#pragma unroll
  for (int r = 0; r < 8; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[r][m] = floatx4{0.f, 0.f, 0.f, 0.f};
  if (kw0 < kw1) {
    const FewRows x = few_rows<MT>(p.X, t0, p.T, K);
    // (stages past the run read its last one)
    auto copy_x = [&](int kb) { few_copy_rows<MT>(x, sx[wave], kb < kw1 ? kb : kw1 - 64); };
    // The wave's rows of packed words (less than 2^31 bytes). WIDE: four words
    // a lane; words past the row are the next row's (or, past the last row,
    // zero), and never stored. Else one word a lane, column 0's past N.
    const int rowb = int(N8 * 4);
    const auto rsQ = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<int32_t*>(p.w.qweight) + int64_t(kw0) * N8, 0,
        int(uint32_t((kw1 - kw0) * N8 * 4)), 0x00020000);
    const int64_t col = n0 / 8 + lr < N8 ? n0 / 8 + lr : 0;
    const uint32_t qoff =
        WIDE ? uint32_t((int64_t(8 * (lane >> 2 & 3) + lg) * N8 + n0 / 8 + 4 * (lane & 3)) * 4)
             : uint32_t((int64_t(8 * lg) * N8 + col) * 4);
    auto copy_q = [&](FewQ& st, int kb) {
      const int k = kb < kw1 ? kb : kw1 - 64;
      const uint32_t at = uint32_t(k - kw0) * uint32_t(rowb);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if constexpr (WIDE) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rsQ, AWQ_LORA_LDS(st[wave] + 128 * h + 64 * i), 16, qoff,
                int(at + uint32_t((32 * h + 4 * i) * rowb)), 0, 0);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rsQ, AWQ_LORA_LDS(st[wave] + 128 * h + 16 * e), 4, qoff,
                int(at + uint32_t((32 * h + e) * rowb)), 0, 0);
        }
      }
    };
    const uint32_t zoff = uint32_t(col * 4), soff = uint32_t(col * 16);
    const auto rsZ = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<int32_t*>(p.w.qzeros), 0, int((K >> p.gshift) * N8 * 4), 0x00020000);
    const auto rsS = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint16_t*>(p.w.scales), 0, int((K >> p.gshift) * N * 2), 0x00020000);
    constexpr int kGroups = G32 ? 2 : 1;      // of a stage
    auto load_groups = [&](FewGroup(&gr)[kGroups], int kb) {
      const int k = kb < kw1 ? kb : kw1 - 64;
#pragma unroll
      for (int h = 0; h < kGroups; ++h) {
        const int g = (k + 32 * h) >> p.gshift;
        gr[h].z = __builtin_amdgcn_raw_buffer_load_b32(rsZ, zoff, g * rowb, 0);
        const auto v = __builtin_amdgcn_raw_buffer_load_b128(
            rsS, soff, int(uint32_t(g) * uint32_t(rowb) * 4u), 0);
        gr[h].s = make_uint4(v[0], v[1], v[2], v[3]);
      }
    };
    // fp16 1024 and 64, opaque so that they stay in registers (with the mask in
    // a scalar one, and-or is one instruction)
    uint32_t base[2] = {0x64006400u, 0x54005400u};
    asm volatile("" : "+v"(base[0]), "+v"(base[1]));
    FewGroup g0[kGroups], g1[kGroups];
    // A stage's X is copied a stage ahead, its words and groups two. A wave
    // reads only what it copied itself: waits, no barriers. The order of the
    // copies here is the loop's, so that its waits cover nothing else.
    copy_q(q0, kw0);
    fence();
    load_groups(g0, kw0);
    fence();
    copy_x(kw0);
    fence();
    copy_q(q1, kw0 + 64);
    fence();
    load_groups(g1, kw0 + 64);
    fence();
    constexpr int kBehind = (WIDE ? 4 : 16) + 2 * kGroups;   // what was asked for after a stage's X
    auto stage = [&](FewQ& st, FewGroup(&gr)[kGroups], int kb) {
      fence();
      wait_vmem<kBehind>();
      fence();
      V xv[2][MT];
      uint32_t w[2][8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          w[h][e] = reinterpret_cast<const uint32_t*>(st[wave])[512 * h + 64 * e + lane];
#pragma unroll
        for (int m = 0; m < MT; ++m)
          xv[h][m] = __builtin_bit_cast(V, sx[wave][x.at[h] + 128 * m]);
      }
      fence();
      wait_lds();      // read before they are copied over
      fence();
      copy_x(kb + 64);
      fence();
      copy_q(st, kb + 128);
      fence();
      FewZeros<F16> n;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (G32 || h == 0) few_zeros<F16>(n, gr[G32 ? h : 0], base);
        FewBlock<F16> b{w[h], gr[G32 ? h : 0], n, base};
        few_block<F16, MT>(b, xv[h], acc);
      }
      fence();
      load_groups(gr, kb + 128);
      fence();
    };
    // kpw and K are multiples of 128 (a way out between the two stages makes the
    // allocator spill the accumulators)
    for (int kb = kw0; kb < kw1; kb += 128) {
      stage(q0, g0, kb);
      stage(q1, g1, kb + 64);
    }
    wait_vmem<0>();
    // here, not behind the branch: there the compiler may copy accumulators first
    few_settle<MT>(acc);
  }
  // lane l holds outputs 8·(l % 16) + r, tokens 16·m + 4·(l / 16) + v
  float* const out = p.partial + (int64_t(s) * p.T + t0 + 4 * lg) * N + n0 + 8 * lr;
  const int64_t left = p.T - t0 - 4 * lg;
  const bool in = n0 + 8 * lr < N;
  auto store = [&](int u, int m, const floatx4 (&x)[2]) {
    if (!in) return;
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (16 * m + v < left)
        *reinterpret_cast<float2*>(out + (16 * m + v) * N + 2 * u) = make_float2(x[0][v], x[1][v]);
  };
  AWQ_FEW_MEET(acc, sx, wave, lane, MT, store)
}

// One stage of X and two of packed words in LDS, in arrays of their own so that
// the compiler can tell the one being read from those being filled; the narrow
// product's two stages lie over them.
template <bool F16, int MT, bool G32, bool WIDE>
__global__ __launch_bounds__(64 * kFewWaves, 2) void lora_few_kernel(LoraFew p, int downs) {
  __shared__ uint4 sx[kFewWaves * 2 * kTile16], q0[kFewWaves * kTile16], q1[kFewWaves * kTile16];
  static_assert(sizeof(FewX<MT>) <= sizeof(sx) && sizeof(FewQ) == sizeof(q0), "");
  const int id = int(blockIdx.x), wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  if (id < downs)
    few_down<F16>(p, id, {sx + 2 * wave * kTile16, sx + (2 * wave + 1) * kTile16},
                  {q0 + wave * kTile16, q1 + wave * kTile16}, reinterpret_cast<FewRed&>(sx));
  else
    few_product<F16, MT, G32, WIDE>(p, id - downs, int(gridDim.x) - downs,
                                    reinterpret_cast<FewX<MT>&>(sx),
                                    reinterpret_cast<FewQ&>(q0), reinterpret_cast<FewQ&>(q1));
}

// T <= 16, N a multiple of 16.
template <bool F16, int G, int TV>
__global__ __launch_bounds__(64 * kFewWaves, 2) void lora_decode_kernel(LoraFew p, int downs,
                                                                       int gx, int gy) {
  __shared__ union {
    uint4 down[kFewWaves][4][kTile16];
    FewRed red;
    MgRed mg[kMgWaves];
  } sm;
  const int id = int(blockIdx.x), wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  if (id < downs)
    few_down<F16>(p, id, {sm.down[wave][0], sm.down[wave][1]},
                  {sm.down[wave][2], sm.down[wave][3]}, sm.red);
  else
    mgemv_workgroup<F16, 4, G, TV>(p.X, p.T, p.w.N, p.w.K, p.w.qweight, p.w.qzeros, p.w.scales,
                                   p.kpw, p.partial, id - downs, gx, gy, sm.mg);
}

template <bool F16>
__global__ __launch_bounds__(64 * kFewWaves) void lora_few_down_kernel(LoraFew p) {
  __shared__ union {
    uint4 down[kFewWaves][4][kTile16];
    FewRed red;
  } sm;
  const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  few_down<F16>(p, int(blockIdx.x), {sm.down[wave][0], sm.down[wave][1]},
                {sm.down[wave][2], sm.down[wave][3]}, sm.red);
}

// ---------------------------------------------------------------------------
// launch 2
// ---------------------------------------------------------------------------

// Workgroup: 32 outputs x 16 tokens. NC·32 >= r. Its 4 waves share the work
// by reads, not by outputs: each takes every fourth run of partial sums and
// every fourth adapter among the rows, with all their loads in flight, and
// they add up in LDS in order. The rows' h (summed over the runs of k) become
// two 16-bit halves in LDS, as in lora_down.hip; an adapter takes one pass of
// MFMAs whose rows are kept where they belong to it.
// Bound by the reads of B, once per 16 tokens, and of the partial sums: 64 tokens
// with any of 48 adapters, rank 32, 28672 outputs (about 88 MB of B for the 62 MB
// that the 34 adapters in use hold, 15 MB of sums) 21 us; 200 tokens of 6
// adapters, rank 8, 4096 outputs (13 MB of sums) 9.8 us. Partial sums read in
// the MFMA's layout, a dword a lane: 27 and 13 us. B through LDS: 35 and 17.5.
constexpr int kFinishCols = 32;

template <bool F16, int NC>
__global__ __launch_bounds__(64 * kFewWaves) void lora_few_finish_kernel(LoraFew p) {
  typedef typename Operand<F16>::type V;
  constexpr int RP = 32 * NC, NB = NC == 4 ? 2 : 4;   // adapters in flight per wave
  __shared__ union {
    float h[16][RP + 1];
    float y[kFewWaves][16][kFinishCols + 1];
  } sm;
  __shared__ __align__(16) uint16_t q[2][16][RP + 8];
  __shared__ __align__(16) float part[kFewWaves][16][kFinishCols + 4];
  __shared__ float se[16];
  const int tid = threadIdx.x, lane = tid & 63, lr = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t t0 = int64_t(blockIdx.y) * 16, N = p.w.N, n0 = int64_t(blockIdx.x) * kFinishCols;
  const int r = p.s.r;
  const int my = t0 + lr < p.T ? p.s.ids[t0 + lr] : -1;
  const uint32_t valid = uint32_t(__ballot(my >= 0 && my < p.s.L)) & 0xFFFFu;
  int64_t col[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int64_t n = n0 + 16 * c + lr;
    col[c] = n < N ? n : N - 1;
  }

  // this wave's next adapters (every fourth distinct one) and their rows; mask
  // 0 when there are none left
  uint32_t left = valid;
  int turn = 0;
  auto next = [&](int& a, uint32_t& mask) {
    a = 0;
    mask = 0;
    while (left) {
      const int id = __builtin_amdgcn_readlane(my, __builtin_ctz(left));
      const uint32_t m = uint32_t(__ballot(my == id)) & 0xFFFFu;
      left &= ~m;
      if ((turn++ & (kFewWaves - 1)) == wave) {
        a = id;
        mask = m;
        return;
      }
    }
  };
  int a[NB];
  uint32_t mask[NB];
  uint4 u[NB][2][NC];
  auto load = [&] {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      next(a[b], mask[b]);
      if (!mask[b]) continue;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint16_t* row = p.s.B + (int64_t(a[b]) * N + col[c]) * r;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
          const int j = 32 * k + 8 * lg;
          u[b][c][k] = *reinterpret_cast<const uint4*>(row + (j < r ? j : r - 8));
        }
      }
    }
  };
  load();
  // h of the rows
  for (int e = tid; e < 16 * RP; e += 64 * kFewWaves) {
    const int i = e / RP, j = e % RP;
    const int64_t t = t0 + i;
    float h = 0.f;
    if (((valid >> i) & 1u) && j < r) {
      const float* src = p.hpart + t * r + j;
#pragma unroll 4
      for (int ks = 0; ks < p.S2; ++ks) h += src[int64_t(ks) * p.T * r];
    }
    sm.h[i][j] = h;
    if (p.H && blockIdx.x == 0 && t < p.T && j < r) p.H[t * r + j] = h;
  }
  // this wave's runs of the shared product: lane l takes 8 outputs of row l / 4
  // (rows past T read the last one, columns past N the first ones)
  {
    const int row = lane >> 2, c = (lane & 3) * 8;
    const int64_t t = t0 + row < p.T ? t0 + row : p.T - 1;
    const float* src = p.partial + t * N + (n0 + c < N ? n0 + c : 0);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), z = x;
#pragma unroll 4
    for (int s = wave; s < p.S; s += kFewWaves) {
      const float4 a0 = *reinterpret_cast<const float4*>(src + int64_t(s) * p.T * N);
      const float4 a1 = *reinterpret_cast<const float4*>(src + int64_t(s) * p.T * N + 4);
      x = make_float4(x.x + a0.x, x.y + a0.y, x.z + a0.z, x.w + a0.w);
      z = make_float4(z.x + a1.x, z.y + a1.y, z.z + a1.z, z.w + a1.w);
    }
    *reinterpret_cast<float4*>(&part[wave][row][c]) = x;
    *reinterpret_cast<float4*>(&part[wave][row][c + 4]) = z;
  }
  float y[2][4] = {};
  __syncthreads();
  for (int i = wave; i < 16; i += kFewWaves) {
    const int id = __builtin_amdgcn_readlane(my, i);
    const float c = (valid >> i) & 1u ? p.s.scaling[id] : 0.f;
    float m = 0.f;
    for (int j = lane; j < RP; j += 64) m = fmaxf(m, fabsf(sm.h[i][j]));
#pragma unroll
    for (int o = 32; o; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    const float cm = fabsf(c) * m;
    int e = 0;
    if (F16 && !(cm >= 0x1p-3f && cm < 0x1p14f)) e = exponent_of(cm);
    const float down = exp2i(-e);
    if (lane == 0) se[i] = exp2i(e);
    for (int j = lane; j < RP; j += 64) {
      const float s = c * sm.h[i][j] * down;
      const uint16_t hi = round16<F16>(s);
      q[0][i][j] = hi;
      q[1][i][j] = round16<F16>(s - widen16<F16>(hi));
    }
  }
  __syncthreads();
  V qh[NC], ql[NC];
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    qh[k] = __builtin_bit_cast(V, *reinterpret_cast<const uint4*>(&q[0][lr][32 * k + 8 * lg]));
    ql[k] = __builtin_bit_cast(V, *reinterpret_cast<const uint4*>(&q[1][lr][32 * k + 8 * lg]));
  }
  while (true) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if (!mask[b]) continue;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        floatx4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < NC; ++k) {
          d = mfma_16x16x32(qh[k], __builtin_bit_cast(V, u[b][c][k]), d);
          d = mfma_16x16x32(ql[k], __builtin_bit_cast(V, u[b][c][k]), d);
        }
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int i = 4 * lg + v;
          const float add = F16 ? se[i] * d[v] : d[v];
          y[c][v] = (mask[b] >> i) & 1u ? y[c][v] + add : y[c][v];
        }
      }
    }
    if (!left) break;
    load();
  }
  // (every wave has read sm.h: the barrier above)
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int v = 0; v < 4; ++v) sm.y[wave][4 * lg + v][16 * c + lr] = y[c][v];
  __syncthreads();
  for (int e = tid; e < 16 * kFinishCols; e += 64 * kFewWaves) {
    const int i = e / kFinishCols, c = e % kFinishCols;
    const float s = (((part[0][i][c] + part[1][i][c]) + part[2][i][c]) + part[3][i][c]) +
                    (((sm.y[0][i][c] + sm.y[1][i][c]) + sm.y[2][i][c]) + sm.y[3][i][c]);
    if (t0 + i < p.T && n0 + c < N) p.Y[(t0 + i) * N + n0 + c] = round16<F16>(s);
  }
}

template <bool F16, int MT>
void launch_few(const LoraFew& p, int downs, unsigned grid, hipStream_t st) {
  // copies of 16 bytes a lane where rows of words allow it, else of 4 bytes:
  // 91.1 against 94.6 us for a call of 64 tokens of 28672x8192, bf16, rank 32, 48
  // adapters, 67.0 against 69.6 with 32 tokens
  const bool wide = p.w.N % 32 == 0;
  if (p.w.group == 32) {
    if (wide) lora_few_kernel<F16, MT, true, true><<<grid, 256, 0, st>>>(p, downs);
    else lora_few_kernel<F16, MT, true, false><<<grid, 256, 0, st>>>(p, downs);
  } else {
    if (wide) lora_few_kernel<F16, MT, false, true><<<grid, 256, 0, st>>>(p, downs);
    else lora_few_kernel<F16, MT, false, false><<<grid, 256, 0, st>>>(p, downs);
  }
}

template <bool F16, int G>
void launch_decode(const LoraFew& p, int downs, int gx, int gy, hipStream_t st) {
  const unsigned grid = unsigned(downs + gx * gy);
  if (p.T == 1) lora_decode_kernel<F16, G, 1><<<grid, 256, 0, st>>>(p, downs, gx, gy);
  else if (p.T == 2) lora_decode_kernel<F16, G, 2><<<grid, 256, 0, st>>>(p, downs, gx, gy);
  else lora_decode_kernel<F16, G, 4><<<grid, 256, 0, st>>>(p, downs, gx, gy);
}

template <bool F16>
hipError_t launch_finish(const LoraFew& p, hipStream_t st) {
  const dim3 grid(unsigned((p.w.N + kFinishCols - 1) / kFinishCols), unsigned((p.T + 15) / 16));
  if (p.s.r <= 32) lora_few_finish_kernel<F16, 1><<<grid, 256, 0, st>>>(p);
  else if (p.s.r <= 64) lora_few_finish_kernel<F16, 2><<<grid, 256, 0, st>>>(p);
  else lora_few_finish_kernel<F16, 4><<<grid, 256, 0, st>>>(p);
  return hipGetLastError();
}

template <bool F16>
hipError_t launch_few(LoraFew p, hipStream_t st) {
  const int jbs = (p.s.r + 15) / 16;
  const int downs = int((p.T + 15) / 16) * few_slots(p) * jbs * p.S2;
  if (p.T <= 16 && p.gemv) {
    const hipError_t e =
        launch_w4a16_gemv(p.X, p.T, p.w.N, p.w.K, p.w.qweight, p.w.qzeros, p.w.scales,
                          p.w.group, F16, p.kpw, p.partial, st);
    if (e != hipSuccess) return e;
    lora_few_down_kernel<F16><<<unsigned(downs), 256, 0, st>>>(p);
  } else if (p.T <= 16) {
    const int gx = int((p.w.N + kMgCols * 8 - 1) / (kMgCols * 8));
    if (p.w.group == 32) launch_decode<F16, 32>(p, downs, gx, p.S, st);
    else if (p.w.group == 64) launch_decode<F16, 64>(p, downs, gx, p.S, st);
    else launch_decode<F16, 128>(p, downs, gx, p.S, st);
  } else {
    const unsigned grid = unsigned(downs + p.tiles * p.col_blocks * p.S);
    if (p.T <= 32) launch_few<F16, 2>(p, downs, grid, st);
    else launch_few<F16, 4>(p, downs, grid, st);
  }
  return launch_finish<F16>(p, st);
}

}  // namespace

hipError_t launch_lora_few(const LoraFew& p, hipStream_t st) {
  return p.f16 ? launch_few<true>(p, st) : launch_few<false>(p, st);
}

hipError_t launch_lora_few_finish(const LoraFew& p, hipStream_t st) {
  return p.f16 ? launch_finish<true>(p, st) : launch_finish<false>(p, st);
}

}  // namespace awq
