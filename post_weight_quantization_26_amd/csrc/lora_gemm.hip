// The wide half of the low-rank product, fused into the shared projection:
//
//   O[t][o] = Σ_c V[t][c]·Wd[o][c] + Σ_j q_t[j]·U_a[o][j],   a = ids[t],
//
// with Wd the packed layer rounded once to the 16-bit type (forward Ŵ [N, K],
// backward Ŵᵀ [K, N]), q_t = c_a·P[t] as two 16-bit halves (lora_down.hip) and
// U = B (forward) or Aᵀ (backward). The 256x256 main loop is the W4A16 GEMM's
// (gemm_core.h). The low-rank part is a few more MFMA steps on the same
// float32 accumulators: 2r / 32 steps per
// adapter in the tile against C / 32, so r = 16 over 4096 channels adds 1%
// of the work, and no float32 output ever goes to memory and back. They come
// first, through the main loop's own LDS ring, and the main loop adds to them.
//
// A tile's tokens may have any adapters. Each distinct one is an item of 64
// columns of q and U at a time: the copy that brings the tile's rows of q to
// LDS points the rows of other tokens past the buffer's end, where they read
// as zero, so the items of any mix are ordinary MFMA steps. A zero times an
// infinity would be NaN for somebody else's token, so the tile of U is looked
// over in LDS first: a value that is not finite becomes zero there and its
// column is marked for that adapter, whose own tokens get NaN at the store.
//
// One workgroup per CU and 256 CUs: tiles past a multiple of 256 would leave
// most CUs idle for a whole tile's time. Those last tiles are cut into runs of
// the contraction instead (LoraSplit), whose float32 accumulators go out in
// register order (1 KiB per store) and are added, in order, by a second kernel.
//
// Bound by the matrix cores: bf16, 8192 tokens of 4096x4096, rank 16, 212 us
// (1300 TFLOP/s; the W4A16 GEMM without adapters runs at 1285 to 1322), 4096
// tokens of 28672x8192, rank 16 and 5 adapters, 1430 to 1510 us (1280 to 1350).
// 1777 tokens of 11008x4096, rank 64: 153 us and 10 for the cut tiles' sums.
#include "gemm_core.h"
#include "lora.h"
#include "lora_common.h"

namespace awq {
namespace {

__shared__ __align__(16) int sid[BM];   // adapter of each row (-1: none, or past the end)
__shared__ int slist[BM];        // the first rows of the distinct adapters
__shared__ int sfirst[BM];       // first row with the same adapter
__shared__ uint32_t smark[BM][8];  // columns of U that are not finite, at that row
__shared__ __align__(16) float sE[BM];  // the power of two a row's q is scaled down by
__shared__ int scount[5];        // distinct adapters by wave; whether any column is marked

struct LowCtx {
  __amdgpu_buffer_rsrc_t rsQ;
  uint32_t qoff[2];    // copy j's lane offset in the tile's rows of q, for even and odd j
  uint32_t urow;       // the lane's row of U for copy 0
  int chunk[2];        // its 16-byte chunk, for even and odd j
  int id[8];           // the adapter of copy j's row
  int n, real, chunks;     // items: distinct adapters x 64-column chunks, made even
                       // by one whose rows of q are all zero
};

constexpr uint32_t kLowOob = 0x80000000u;

// Lists the tile's distinct adapters. All threads; rows' ids are in sid.
__device__ __forceinline__ int list_adapters() {
  const int i = threadIdx.x, lane = i & 63, wave = i >> 6;
  const int id = sid[i];
  int first = i;
  if (__syncthreads_and(id == sid[0])) {
    first = 0;
  } else {
    // from the last row down, so that the first match is the one that stays
#pragma unroll 8
    for (int k = BM / 4 - 1; k >= 0; --k) {
      const int4 x = reinterpret_cast<const int4*>(sid)[k];
      first = x.w == id ? 4 * k + 3 : first;
      first = x.z == id ? 4 * k + 2 : first;
      first = x.y == id ? 4 * k + 1 : first;
      first = x.x == id ? 4 * k : first;
    }
  }
  sfirst[i] = first;
  const uint64_t lead = __ballot(id >= 0 && first == i);
  if (lane == 0) scount[wave] = __popcll(lead);
  __syncthreads();
  int at = __popcll(lead & ((1ull << lane) - 1));
  for (int w = 0; w < wave; ++w) at += scount[w];
  if (id >= 0 && first == i) slist[at] = i;
  const int n = scount[0] + scount[1] + scount[2] + scount[3];
  __syncthreads();
  return n;
}

// Item q (an adapter's 64 columns) to stage S.
template <int S>
__device__ __forceinline__ void low_copy(const LowCtx& l, const LoraUp& u, int wave, int q,
                                         int64_t n0, int64_t N) {
  const bool pad = q >= l.real;
  const int a = __builtin_amdgcn_readfirstlane(sid[slist[pad ? 0 : q / l.chunks]]);
  const int kt = q % l.chunks, want = pad ? -2 : a;
  const int64_t rows = N - n0 < BN ? N - n0 : BN;
  const auto rsU = tile_rsrc(u.U + (int64_t(a) * N + n0) * u.r, rows, u.r);
  const int nb8 = u.r / 8;
  uint32_t uoff[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    uoff[h] = l.urow * u.r * 2 + uint32_t((8 * kt + l.chunk[h]) % nb8) * 16;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        l.rsQ, AWQ_LDS(stage64_a<S>() + (wave * 8 + j) * 64), 16,
        l.id[j] == want ? l.qoff[j & 1] + uint32_t(kt * 128) : kLowOob, j * 16 * u.RW, 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsU, AWQ_LDS(stage64_b<S>() + (wave * 8 + j) * 64),
                                             16, uoff[j & 1], j * 16 * u.r, 0, 0);
  }
}

// Zeroes and marks what is not finite in stage S's U.
template <bool F16, int S>
__device__ __forceinline__ void low_check(int first_row) {
  constexpr uint32_t kExp = F16 ? 0x7C007C00u : 0x7F807F80u;
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  u16x2 least = {0xFFFF, 0xFFFF};     // 0 in a half: an exponent of all ones
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint4 x = stage64_b<S>()[threadIdx.x + 256 * k];
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      least = __builtin_elementwise_min(least, __builtin_bit_cast(u16x2, ~w[e] & kExp));
  }
  if (least[0] != 0 && least[1] != 0) return;
  scount[4] = 1;
  for (int k = 0; k < 8; ++k) {
    const int at = threadIdx.x + 256 * k;
    uint32_t* w = reinterpret_cast<uint32_t*>(&stage64_b<S>()[at]);
    bool bad = false;
    for (int e = 0; e < 4; ++e) {
      uint32_t v = w[e];
      if ((~v & kExp & 0xFFFFu) == 0) v &= 0xFFFF0000u;
      if ((~v & kExp & 0xFFFF0000u) == 0) v &= 0xFFFFu;
      bad = bad || v != w[e];
      w[e] = v;
    }
    if (bad) atomicOr(&smark[first_row][(at >> 3) >> 5], 1u << ((at >> 3) & 31));
  }
}

// Item q from stage S, with the next item's copies, or the main loop's first,
// in flight (the last item is in stage 1).
template <bool F16, int S>
__device__ __forceinline__ void low_item(const GemmCtx64& c, const LowCtx& l, const LoraUp& u,
                                         int q, floatx4 (&acc)[8][8], int64_t n0, int64_t N) {
  typedef typename Operand<F16>::type V;
  __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
  __builtin_amdgcn_s_waitcnt(wait_vm(0));
  region_barrier();
  if (q + 1 < l.n) low_copy<S ^ 1>(l, u, c.wave, q + 1, n0, N);
  else if constexpr (S == 1) dma64<0>(c, 0);
  low_check<F16, S>(slist[q < l.real ? q / l.chunks : 0]);
  __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
  region_barrier();
  int rdA[2], rdB[2];
  frag_offsets16(c, rdA, rdB);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    V fa[8], fb[8];
#pragma unroll
    for (int r = 0; r < 16; ++r) frag16<S>(rdA[h], rdB[h], r, fa, fb);
    mfma_8x8(acc, fa, fb);
  }
}

// The low-rank part of the tile, and the main loop's first copies.
template <bool F16>
__device__ __forceinline__ void low_rank(const GemmCtx64& c, const LoraUp& u,
                                         floatx4 (&acc)[8][8], int64_t m0, int64_t rows_a,
                                         int64_t n0, int64_t N) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
      asm volatile("" : "+a"(acc[i][j]));   // in AGPRs from the start
    }
  LowCtx l;
  l.chunks = u.RW / 64;
  l.real = __builtin_amdgcn_readfirstlane(list_adapters()) * l.chunks;
  l.n = (l.real + 1) & ~1;
  const int lane = threadIdx.x & 63;
  l.rsQ = tile_rsrc(u.Q + m0 * u.RW, rows_a, u.RW);
  l.urow = uint32_t(c.wave * 64 + (lane >> 3));
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l.chunk[h] = (lane & 7) ^ (((lane >> 4) + 4 * h) & 7);
    l.qoff[h] = (l.urow * u.RW + l.chunk[h] * 8) * 2;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) l.id[j] = sid[l.urow + 8 * j];
  if (l.n == 0) dma64<0>(c, 0);
  else low_copy<0>(l, u, c.wave, 0, n0, N);
  // (one plain loop: with more control flow around the pinned accumulators
  // the allocator spills them)
  for (int q = 0; q < l.n; q += 2) {
    low_item<F16, 0>(c, l, u, q, acc, n0, N);
    low_item<F16, 1>(c, l, u, q + 1, acc, n0, N);
  }
  if constexpr (F16) {
    // (the last MFMAs have drained before their sums are read)
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) asm volatile("" : "+a"(acc[i][j]));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 e4 =
          *reinterpret_cast<const float4*>(&sE[(c.wave >> 1) * 128 + 16 * i + 4 * (lane >> 4)]);
      const float e[4] = {e4.x, e4.y, e4.z, e4.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[i][j][v] *= e[v];
        asm volatile("" : "+a"(acc[i][j]));
      }
    }
  }
}

// V [M, ldv] and Wd [N, ldw] with C columns each (a multiple of 64).
// SPLIT: workgroups below sp.full take whole tiles, the others run s of a tile.
template <bool F16, bool SPLIT>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(1, 1)))
void lora_gemm_kernel(const uint16_t* __restrict__ X, int64_t ldv,
                      const uint16_t* __restrict__ Wd, int64_t ldw, int64_t M, int64_t N,
                      int64_t C, int tiles_m, int tiles_n, LoraUp u, LoraSplit sp,
                      uint16_t* __restrict__ O) {
  int tm, tn, run = 0, slot = -1;
  int64_t k0 = 0, k1 = C;
  if constexpr (SPLIT) {
    // XCD i takes a contiguous run of tiles (token tiles fastest), and of the
    // (tile, run) units behind them
    int tile;
    const int id = int(blockIdx.x);
    if (id < sp.full) {
      tile = (id % 8) * (sp.full / 8) + id / 8;
    } else {
      const int v = id - sp.full, units = int(gridDim.x) - sp.full, q = units / 8,
                rem = units % 8, x = v % 8;
      slot = x * q + (x < rem ? x : rem) + v / 8;
      tile = sp.full + slot / sp.runs;
      run = slot % sp.runs;
      const int kt = int(C / BK64);
      k0 = int64_t(kt * run / sp.runs) * BK64;
      k1 = int64_t(kt * (run + 1) / sp.runs) * BK64;
    }
    tm = tile % tiles_m;
    tn = tile / tiles_m;
  } else {
    if (!tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn)) return;
  }
  const int64_t m0 = int64_t(tm) * BM, n0 = int64_t(tn) * BN;
  const int64_t rows_a = M - m0 < BM ? M - m0 : BM;
  const int64_t rows_b = N - n0 < BN ? N - n0 : BN;
  {
    // (only the first run of a cut tile takes the low-rank part)
    const int64_t t = m0 + threadIdx.x;
    const int id = t < M && run == 0 ? u.ids[t] : -1;
    sid[threadIdx.x] = id >= 0 && id < u.L ? id : -1;
    if (F16) sE[threadIdx.x] = id >= 0 && id < u.L ? u.E[t] : 1.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) smark[threadIdx.x][k] = 0;
    if (threadIdx.x == 0) scount[4] = 0;
  }
  GemmCtx64 c;
  gemm_setup64(c, X + m0 * ldv + k0, rows_a, ldv, Wd + n0 * ldw + k0, rows_b, ldw, k1 - k0, false);
  __syncthreads();

  // lane l of block (i, j) holds column l % 16 and rows 4·(l/16) + v
  const int lane = threadIdx.x & 63;
  const int wm = c.wave >> 1, wn = c.wave & 1;
  floatx4 acc[8][8];
  low_rank<F16>(c, u, acc, m0, rows_a, n0, N);
  // the accumulators are written by now; the first MFMA on them comes after
  // the main loop's barrier
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) asm volatile("" : "+a"(acc[i][j]));
  asm volatile("s_nop 15" ::: "memory");
  // (uniform, and said so again: past the code above the compiler held some
  // of these in vector registers and looped over each copy's lanes)
  c.stepA = __builtin_amdgcn_readfirstlane(c.stepA);
  c.stepB = __builtin_amdgcn_readfirstlane(c.stepB);
  c.KT = __builtin_amdgcn_readfirstlane(c.KT);
  gemm_mainloop16<F16, true>(c, acc);

  const int64_t wrow = m0 + wm * 128, wcol = n0 + wn * 128;
  if (SPLIT && slot >= 0) {
    floatx4* out = reinterpret_cast<floatx4*>(sp.part) + (int64_t(slot) * 4 + c.wave) * 4096 + lane;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) out[(i * 8 + j) * 64] = acc[i][j];
  } else {
    const int64_t row0 = wrow + 4 * (lane >> 4);
    const int64_t col0 = wcol + (lane & 15);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t col = col0 + j * 16;
        if (col >= N) continue;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int64_t row = row0 + i * 16 + v;
          if (row < M) O[row * N + col] = round16<F16>(acc[i][j][v]);
        }
      }
  }
  if (scount[4] == 0) return;
  // Rare: NaN over the outputs whose row's adapter has a column that is not
  // finite, a thread per row, after every thread's stores.
  __syncthreads();
  const int row = threadIdx.x;
  if (sid[row] < 0) return;
  for (int w = 0; w < 8; ++w)
    for (uint32_t m = smark[sfirst[row]][w]; m; m &= m - 1) {
      const int col = 32 * w + __builtin_ctz(m);
      if (SPLIT && slot >= 0) {
        const int64_t wave = (row >> 7) * 2 + (col >> 7);
        const int block = ((row & 127) >> 4) * 8 + ((col & 127) >> 4);
        sp.part[(((int64_t(slot) * 4 + wave) * 64 + block) * 64 + ((row & 15) >> 2) * 16 +
                 (col & 15)) * 4 + (row & 3)] = __uint_as_float(0x7FC00000u);
      } else if (n0 + col < N) {
        O[(m0 + row) * N + n0 + col] = F16 ? 0x7E00 : 0x7FC0;
      }
    }
}

// Workgroup (cut tile, wave, block row i): 16 rows x 128 columns, the runs'
// sums added in order, turned through LDS into 16-byte stores.
template <bool F16>
__global__ __launch_bounds__(256) void lora_gemm_sum_kernel(LoraSplit sp, int tiles_m, int64_t M,
                                                            int64_t N, uint16_t* __restrict__ O) {
  __shared__ __align__(16) uint16_t tile[16][136];
  const int cut = int(blockIdx.x), wave = int(blockIdx.y), i = int(blockIdx.z);
  const int lane = threadIdx.x & 63, q = threadIdx.x >> 6;
  const int t = sp.full + cut, tm = t % tiles_m, tn = t / tiles_m;
  const int64_t row0 = int64_t(tm) * BM + (wave >> 1) * 128 + 16 * i;
  const int64_t col0 = int64_t(tn) * BN + (wave & 1) * 128;
  if (row0 >= M || col0 >= N) return;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int j = q + 4 * h;
    const floatx4* src = reinterpret_cast<const floatx4*>(sp.part) +
                         (int64_t(cut) * sp.runs * 4 + wave) * 4096 + (i * 8 + j) * 64 + lane;
    floatx4 s = src[0];
#pragma unroll 4
    for (int r = 1; r < sp.runs; ++r) s += src[int64_t(r) * 4 * 4096];
#pragma unroll
    for (int v = 0; v < 4; ++v) tile[4 * (lane >> 4) + v][16 * j + (lane & 15)] = round16<F16>(s[v]);
  }
  __syncthreads();
  const int r = threadIdx.x >> 4, c = (threadIdx.x & 15) * 8;
  if (row0 + r < M && col0 + c < N)
    *reinterpret_cast<uint4*>(O + (row0 + r) * N + col0 + c) =
        *reinterpret_cast<const uint4*>(&tile[r][c]);
}

template <bool F16>
hipError_t launch_f(const uint16_t* V, int64_t ldv, const uint16_t* Wd, int64_t ldw, int64_t M,
                    int64_t N, int64_t C, const LoraUp& u, const LoraSplit& sp, uint16_t* O,
                    hipStream_t st) {
  const int tiles_m = int((M + BM - 1) / BM), tiles_n = int((N + BN - 1) / BN);
  if (sp.runs < 2) {
    lora_gemm_kernel<F16, false><<<unsigned(gemm_blocks(tiles_m, tiles_n)), NT, 0, st>>>(
        V, ldv, Wd, ldw, M, N, C, tiles_m, tiles_n, u, sp, O);
    return hipGetLastError();
  }
  const int cut = tiles_m * tiles_n - sp.full;
  lora_gemm_kernel<F16, true><<<unsigned(sp.full + cut * sp.runs), NT, 0, st>>>(
      V, ldv, Wd, ldw, M, N, C, tiles_m, tiles_n, u, sp, O);
  lora_gemm_sum_kernel<F16><<<dim3(unsigned(cut), 4, 8), 256, 0, st>>>(sp, tiles_m, M, N, O);
  return hipGetLastError();
}

}  // namespace

// 512·ldv, 512·ldw < 2^31; 16-byte aligned rows; C a multiple of 64, N of 8;
// sp from the host's rule for these sizes.
hipError_t launch_lora_gemm(const uint16_t* V, int64_t ldv, const uint16_t* Wd, int64_t ldw,
                            int64_t M, int64_t N, int64_t C, const LoraUp& u,
                            const LoraSplit& sp, int f16, uint16_t* O, hipStream_t st) {
  if (C % 64 || N % 8 || ldv % 8 || ldw % 8 || u.r < 8 || u.r % 8 || sp.runs > C / 64 ||
      sp.full % 256)
    return hipErrorInvalidValue;
  return f16 ? launch_f<true>(V, ldv, Wd, ldw, M, N, C, u, sp, O, st)
             : launch_f<false>(V, ldv, Wd, ldw, M, N, C, u, sp, O, st);
}

}  // namespace awq
