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
// Each word serves 16·MT tokens. The 4 waves' runs meet in LDS, in order.
#include "gemm_types.h"
#include "lora.h"
#include "lora_common.h"
#include "lora_stage.h"
#include "w4a16_mgemv.h"

namespace awq {
namespace {

constexpr int kFewWaves = 4;
constexpr int kFewCols = 128;     // outputs per workgroup (T > 16)

typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

// ---------------------------------------------------------------------------
// launch 1: the narrow product
// ---------------------------------------------------------------------------

// Workgroup (tile of 16 tokens, row, block of 16 ranks, run of k): if `row` is
// the first of the tile with its adapter, the adapter's 16 x 16 block of P for
// all rows of the tile that have it, as a float32 partial sum.
__device__ __forceinline__ void few_down_index(const LoraFew& p, int id, int& tile, int& row,
                                               int& jb, int& ks) {
  const int jbs = (p.s.r + 15) / 16, rows = p.T < 16 ? int(p.T) : 16;
  ks = id % p.S2;
  id /= p.S2;
  jb = id % jbs;
  id /= jbs;
  row = id % rows;
  tile = id / rows;
}

// Per wave and stage: a 16-row tile of X and one of A (lora_stage.h).
typedef uint4 FewStage[kFewWaves][2][kTile16];

template <bool F16>
__device__ __forceinline__ void few_down(const LoraFew& p, int id, FewStage& s0, FewStage& s1) {
  typedef typename Operand<F16>::type V;
  int tile, row, jb, ks;
  few_down_index(p, id, tile, row, jb, ks);
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  const int64_t t0 = int64_t(tile) * 16, K = p.w.K;
  const int my = t0 + lr < p.T ? p.s.ids[t0 + lr] : -1;
  const int a = __builtin_amdgcn_readlane(my, row);
  const uint32_t mine = uint32_t(__ballot(my == a)) & 0xFFFFu;
  if (a < 0 || a >= p.s.L || int(__builtin_ctz(mine)) != row) return;
  const int nb = int(K / 128), b0 = int(int64_t(nb) * ks / p.S2),
            b1 = int(int64_t(nb) * (ks + 1) / p.S2);
  const int64_t rows = p.T - t0 < 16 ? p.T - t0 : 16;
  const int ranks = p.s.r - 16 * jb < 16 ? p.s.r - 16 * jb : 16;
  const auto rsX = rows_rsrc(p.X + t0 * K, rows, K);
  const auto rsA = rows_rsrc(p.s.A + (int64_t(a) * p.s.r + 16 * jb) * K, ranks, K);
  uint32_t off[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) off[i] = tile_offset(0, i, K);
  auto copy = [&](FewStage& st, int b) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      tile_copy(rsX, off[i], 128 * b, st[wave][0], i);
      tile_copy(rsA, off[i], 128 * b, st[wave][1], i);
    }
  };
  floatx4 acc = {0.f, 0.f, 0.f, 0.f};
  auto use = [&](const FewStage& st) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
      acc = mfma_16x16x32(__builtin_bit_cast(V, tile_read(st[wave][0], s)),
                          __builtin_bit_cast(V, tile_read(st[wave][1], s)), acc);
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
  float(*red)[16][17] = reinterpret_cast<float(*)[16][17]>(&s0);
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

// A block of 32 k rows of the packed words; the zero points and scales of the
// group that one (group size 32) or two (64, 128) blocks lie in.
struct FewWords {
  uint32_t w[8];
};
struct FewGroup {
  uint32_t z;
  uint4 s;
};
constexpr int kFewSlots = 4;

// Per wave and stage: 16·MT tokens x 64 channels of X, rows of 8 chunks of 16
// bytes, chunk c of row i at c ^ (i / 2) % 8.
template <int MT>
using FewX = uint4[kFewWaves][16 * MT * 8];

// The MFMA operand of nibble R: its 8 codes, one per word, as rounded Ŵ.
template <bool F16, int R>
__device__ __forceinline__ uint4 few_operand(const uint32_t (&w)[8], uint32_t z,
                                             const uint32_t (&sw)[4],
                                             const uint32_t (&base)[2]) {
  constexpr uint32_t kSel = 0x0C000C00u | uint32_t(4 + R / 2) << 16 | uint32_t(R / 2);
  constexpr uint32_t kMask = R & 1 ? 0x00F000F0u : 0x000F000Fu;
  const uint32_t kBase = base[R & 1];
  const f16x2_t zb =
      __builtin_bit_cast(f16x2_t, (__builtin_amdgcn_perm(z, z, kSel) & kMask) | kBase);
  const _Float16 sc =
      __builtin_bit_cast(_Float16, uint16_t(sw[R / 2] >> (16 * (R & 1))));
  uint32_t out[4];
  if constexpr (F16) {
    const f16x2_t s2 = {sc, sc};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const f16x2_t q = __builtin_bit_cast(
          f16x2_t, (__builtin_amdgcn_perm(w[2 * e + 1], w[2 * e], kSel) & kMask) | kBase);
      const f16x2_t d = q - zb;
      out[e] = __builtin_bit_cast(uint32_t, d * s2);
    }
  } else {
    const float s = float(sc), nzs = -(float(zb[0]) * s);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const f16x2_t q = __builtin_bit_cast(
          f16x2_t, (__builtin_amdgcn_perm(w[2 * e + 1], w[2 * e], kSel) & kMask) | kBase);
      const float lo = __builtin_fmaf(float(q[0]), float(sc), nzs);
      const float hi = __builtin_fmaf(float(q[1]), float(sc), nzs);
      out[e] = pack2<false>(lo, hi);
    }
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// The accumulators stay in AGPRs through inline asm: 128 of them among the
// vector registers make the allocator spill at two waves per SIMD. The
// compiler puts no wait states around asm: s_nop 1 covers an operand that the
// instruction before wrote, and few_settle the reads at the end.
#define AWQ_FEW_MFMA(TYPE, V)                                                               \
  __device__ __forceinline__ void mfma_few(floatx4(&c)[2], const V(&a)[2], const V& b) {   \
    asm("s_nop 1\n\tv_mfma_f32_16x16x32_" TYPE " %0, %2, %4, %0\n\t"                       \
        "v_mfma_f32_16x16x32_" TYPE " %1, %3, %4, %1"                                       \
        : "+a"(c[0]), "+a"(c[1])                                                            \
        : "v"(a[0]), "v"(a[1]), "v"(b));                                                    \
  }                                                                                         \
  __device__ __forceinline__ void mfma_few(floatx4(&c)[4], const V(&a)[4], const V& b) {   \
    asm("s_nop 1\n\tv_mfma_f32_16x16x32_" TYPE " %0, %4, %8, %0\n\t"                       \
        "v_mfma_f32_16x16x32_" TYPE " %1, %5, %8, %1\n\t"                                   \
        "v_mfma_f32_16x16x32_" TYPE " %2, %6, %8, %2\n\t"                                   \
        "v_mfma_f32_16x16x32_" TYPE " %3, %7, %8, %3"                                       \
        : "+a"(c[0]), "+a"(c[1]), "+a"(c[2]), "+a"(c[3])                                    \
        : "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]), "v"(b));                              \
  }
AWQ_FEW_MFMA("bf16", bf16x8_t)
AWQ_FEW_MFMA("f16", f16x8_t)
#undef AWQ_FEW_MFMA
template <int MT>
__device__ __forceinline__ void few_settle(floatx4 (&acc)[8][MT]) {
  asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
#pragma unroll
  for (int r = 0; r < 8; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) asm volatile("" : "+a"(acc[r][m]));
}

template <bool F16, int MT>
__device__ __forceinline__ void few_block(const FewWords& sl, const FewGroup& gr,
                                          const FewX<MT>& x, uint32_t xat,
                                          const uint32_t (&base)[2], floatx4 (&acc)[8][MT]) {
  typedef typename Operand<F16>::type V;
  V xv[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
    xv[m] = __builtin_bit_cast(V, (&x[0][0])[xat + 128 * m]);
  const uint32_t sw[4] = {gr.s.x, gr.s.y, gr.s.z, gr.s.w};
#define AWQ_FEW_NIBBLE(R)                                                              \
  {                                                                                    \
    const V b = __builtin_bit_cast(V, few_operand<F16, R>(sl.w, gr.z, sw, base));      \
    mfma_few(acc[R], xv, b);                                                           \
  }
  AWQ_FEW_NIBBLE(0) AWQ_FEW_NIBBLE(1) AWQ_FEW_NIBBLE(2) AWQ_FEW_NIBBLE(3)
  AWQ_FEW_NIBBLE(4) AWQ_FEW_NIBBLE(5) AWQ_FEW_NIBBLE(6) AWQ_FEW_NIBBLE(7)
#undef AWQ_FEW_NIBBLE
}

// s0, s1: the wave's X stages and, at the end, the meeting of the waves.
template <bool F16, int MT, bool G32>
__device__ __forceinline__ void few_product(const LoraFew& p, int id, int blocks, FewX<MT>& s0,
                                            FewX<MT>& s1) {
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
  // Lanes past N read column 0 and are never stored; token rows past T read as
  // zero.
  const int64_t col = n0 / 8 + lr < N8 ? n0 / 8 + lr : 0;
  const uint32_t qoff = uint32_t((int64_t(8 * lg) * N8 + col) * 4);
  const uint32_t zoff = uint32_t(col * 4), soff = uint32_t(col * 16);
  const auto rsX = rows_rsrc(p.X + t0 * K, p.T - t0 < R ? p.T - t0 : R, K);
  uint32_t xoff[2];      // rows 8i + l / 8 of X: the swizzle repeats every 16 rows
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = 8 * i + (lane >> 3);
    xoff[i] = uint32_t((row * K + ((lane & 7) ^ (row >> 1)) * 8) * 2);
  }
  const int xstep = int(16 * K * 2);
  auto copy_x = [&](FewX<MT>& st, int k) {
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsX, AWQ_LORA_LDS(st[wave] + 64 * i), 16,
                                               xoff[i & 1], (i >> 1) * xstep + 2 * k, 0, 0);
  };
  // The wave's rows of packed words (at most a quarter of N·K / 2 <= 2^33
  // bytes), and the layer's zero points and scales, as buffer resources: one
  // lane offset each, everything else in scalar registers.
  const int kw = kw0 < kw1 ? kw0 : 0, rowb = int(N8 * 4);
  const auto rsQ = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<int32_t*>(p.w.qweight) + int64_t(kw) * N8, 0,
      int(uint32_t((kw1 - kw0 > 0 ? kw1 - kw0 : 0) * N8 * 4)), 0x00020000);
  const auto rsZ = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<int32_t*>(p.w.qzeros), 0, int((K >> p.gshift) * N8 * 4), 0x00020000);
  const auto rsS = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint16_t*>(p.w.scales), 0, int((K >> p.gshift) * N * 2), 0x00020000);
  // blocks past the wave's last one read it again (and are not used)
  auto load_words = [&](FewWords& sl, int kb) {
    const int k = kb < kw1 ? kb : kw1 - 32;
    const uint32_t at = uint32_t(k - kw0) * uint32_t(rowb);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      sl.w[e] = __builtin_amdgcn_raw_buffer_load_b32(rsQ, qoff, int(at + uint32_t(e * rowb)), 0);
  };
  auto load_group = [&](FewGroup& gr, int kb) {
    const int g = (kb < kw1 ? kb : kw1 - 32) >> p.gshift;
    gr.z = __builtin_amdgcn_raw_buffer_load_b32(rsZ, zoff, g * rowb, 0);
    const auto v = __builtin_amdgcn_raw_buffer_load_b128(
        rsS, soff, int(uint32_t(g) * uint32_t(rowb) * 4u), 0);
    gr.s = make_uint4(v[0], v[1], v[2], v[3]);
  };
  floatx4 acc[8][MT];
#pragma unroll
  for (int r = 0; r < 8; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[r][m] = floatx4{0.f, 0.f, 0.f, 0.f};
  if (kw0 < kw1) {
    // fp16 1024 and 64, opaque so that they stay in registers (with the mask in
    // a scalar one, and-or is one instruction)
    uint32_t base[2] = {0x64006400u, 0x54005400u};
    asm volatile("" : "+v"(base[0]), "+v"(base[1]));
    // where the lane's operand of 32-channel step h lies in a stage (as opaque:
    // two registers, not one for every stage and token block)
    uint32_t xat[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      xat[h] = uint32_t(wave * (R * 8) + lr * 8 + ((4 * h + lg) ^ (lr >> 1)));
    asm volatile("" : "+v"(xat[0]), "+v"(xat[1]));
    FewWords sl[kFewSlots];
    FewGroup gr[G32 ? 4 : 2];
    copy_x(s0, kw0);
    fence();
#pragma unroll
    for (int i = 0; i < kFewSlots; ++i) {
      load_words(sl[i], kw0 + 32 * i);
      if (G32 || i % 2) load_group(gr[G32 ? i : i / 2], kw0 + 32 * i);
    }
    // kpw and K are multiples of 128: two stages of X, four slots of words.
    // A stage's copies are followed by the loads of two slots and their groups
    // (the first stage's by twice that), which may be outstanding when it is
    // read. A wave reads only what it copied itself, so no barrier is needed.
    constexpr int kBehind = 16 + (G32 ? 4 : 2);
    for (int kb = kw0; kb < kw1; kb += 128) {
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        fence();
        wait_lds();
        wait_vmem<kBehind>();
        fence();
        if (st == 0) copy_x(s1, kb + 64);
        else copy_x(s0, kb + 128);
        fence();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int i = 2 * st + h, next = kb + 32 * (kFewSlots + i);
          few_block<F16, MT>(sl[i], gr[G32 ? i : st], st == 0 ? s0 : s1, xat[h], base, acc);
          __builtin_amdgcn_sched_barrier(0);
          load_words(sl[i], next);
          if (G32 || h) load_group(gr[G32 ? i : st], next);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
    wait_vmem<0>();
  }
  few_settle<MT>(acc);
  __syncthreads();
  float* const red[2] = {reinterpret_cast<float*>(&s0), reinterpret_cast<float*>(&s1)};
  // lane l holds outputs 8·(l % 16) + r, tokens 16·m + 4·(l / 16) + v
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    if (wave >> 1 == half) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          float* row = red[wave & 1] + (16 * m + 4 * lg + v) * kFewCols + 8 * lr;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float4 x = make_float4(acc[4 * h][m][v], acc[4 * h + 1][m][v], acc[4 * h + 2][m][v],
                                   acc[4 * h + 3][m][v]);
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
  for (int e = threadIdx.x; e < R * kFewCols / 4; e += 64 * kFewWaves) {
    const int i = e / (kFewCols / 4), c = e % (kFewCols / 4) * 4;
    if (t0 + i >= p.T || n0 + c >= N) continue;
    const float4 x = *reinterpret_cast<const float4*>(red[0] + i * kFewCols + c);
    const float4 y = *reinterpret_cast<const float4*>(red[1] + i * kFewCols + c);
    *reinterpret_cast<float4*>(p.partial + (int64_t(s) * p.T + t0 + i) * N + n0 + c) =
        make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
  }
}

template <bool F16, int MT, bool G32>
__global__ __launch_bounds__(64 * kFewWaves, 2) void lora_few_kernel(LoraFew p, int downs) {
  // two stages each; separate arrays, so that the compiler can tell the one
  // being read from the one being filled
  constexpr int kStage = sizeof(FewX<MT>) > sizeof(FewStage) ? sizeof(FewX<MT>) : sizeof(FewStage);
  __shared__ uint4 s0[kStage / 16], s1[kStage / 16];
  const int id = int(blockIdx.x);
  if (id < downs)
    few_down<F16>(p, id, reinterpret_cast<FewStage&>(s0), reinterpret_cast<FewStage&>(s1));
  else
    few_product<F16, MT, G32>(p, id - downs, int(gridDim.x) - downs,
                              reinterpret_cast<FewX<MT>&>(s0),
                              reinterpret_cast<FewX<MT>&>(s1));
}

// T <= 16, N a multiple of 16.
template <bool F16, int G, int TV>
__global__ __launch_bounds__(64 * kFewWaves, 2) void lora_decode_kernel(LoraFew p, int downs,
                                                                       int gx, int gy) {
  __shared__ union {
    FewStage down[2];
    MgRed mg[kMgWaves];
  } sm;
  const int id = int(blockIdx.x);
  if (id < downs) few_down<F16>(p, id, sm.down[0], sm.down[1]);
  else
    mgemv_workgroup<F16, 4, G, TV>(p.X, p.T, p.w.N, p.w.K, p.w.qweight, p.w.qzeros, p.w.scales,
                                   p.kpw, p.partial, id - downs, gx, gy, sm.mg);
}

template <bool F16>
__global__ __launch_bounds__(64 * kFewWaves) void lora_few_down_kernel(LoraFew p) {
  __shared__ FewStage s0, s1;
  few_down<F16>(p, int(blockIdx.x), s0, s1);
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
  // this wave's runs of the shared product (rows past T read the last one)
  float y[2][4] = {};
  {
    const float* src[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int64_t t = t0 + 4 * lg + v;
      src[v] = p.partial + (t < p.T ? t : p.T - 1) * N;
    }
#pragma unroll 4
    for (int s = wave; s < p.S; s += kFewWaves)
#pragma unroll
      for (int v = 0; v < 4; ++v)
#pragma unroll
        for (int c = 0; c < 2; ++c) y[c][v] += src[v][int64_t(s) * p.T * N + col[c]];
  }
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
    const float s = ((sm.y[0][i][c] + sm.y[1][i][c]) + sm.y[2][i][c]) + sm.y[3][i][c];
    if (t0 + i < p.T && n0 + c < N) p.Y[(t0 + i) * N + n0 + c] = round16<F16>(s);
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
hipError_t launch_few(LoraFew p, hipStream_t st) {
  const int jbs = (p.s.r + 15) / 16, rows = p.T < 16 ? int(p.T) : 16;
  const int downs = int((p.T + 15) / 16) * rows * jbs * p.S2;
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
    if (p.T <= 32) {
      if (p.w.group == 32) lora_few_kernel<F16, 2, true><<<grid, 256, 0, st>>>(p, downs);
      else lora_few_kernel<F16, 2, false><<<grid, 256, 0, st>>>(p, downs);
    } else {
      if (p.w.group == 32) lora_few_kernel<F16, 4, true><<<grid, 256, 0, st>>>(p, downs);
      else lora_few_kernel<F16, 4, false><<<grid, 256, 0, st>>>(p, downs);
    }
  }
  const dim3 grid(unsigned((p.w.N + kFinishCols - 1) / kFinishCols), unsigned((p.T + 15) / 16));
  if (p.s.r <= 32) lora_few_finish_kernel<F16, 1><<<grid, 256, 0, st>>>(p);
  else if (p.s.r <= 64) lora_few_finish_kernel<F16, 2><<<grid, 256, 0, st>>>(p);
  else lora_few_finish_kernel<F16, 4><<<grid, 256, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_lora_few(const LoraFew& p, hipStream_t st) {
  return p.f16 ? launch_few<true>(p, st) : launch_few<false>(p, st);
}

}  // namespace awq
