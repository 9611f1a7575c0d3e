// What the gradient of a low-rank call needs laid out first, in one launch
// (each part is independent of the others and takes its own workgroups):
//
//  * the plan: tokens sorted by adapter (a stable counting sort, so equal
//    calls give equal orders), each adapter's run starting at a multiple of
//    32 positions, and the runs cut into pieces of at most `piece` tokens;
//  * Ŵᵀ [K, Np]: the packed layer rounded once to the 16-bit type in the order
//    it is packed in (N padded with zeros to Np, a multiple of 128);
//  * Bᵀ [L, r, Np] and Aᵀ [L, K, r] of the adapters that have tokens, so that
//    every MFMA operand of the products over N and r is contiguous;
//  * dY padded to Np columns, where N is no multiple of 128.
//
// Bound by the layer's bytes (2.5 per weight): 4096x11008 23 us, 4.9 TB/s. With few
// tokens (no layer) by the latency of the plan and the transposes, 6.4 us.
#include "lora.h"
#include "lora_common.h"

namespace awq {
namespace {

constexpr int kPrepThreads = 1024;
constexpr int kPrepWaves = kPrepThreads / 64;

// The distinct ids (0 <= id < L) of a wave's 64 lanes, each with the mask of
// its lanes, in the order of their first lanes.
template <class F>
__device__ __forceinline__ void for_each_id(int id, int L, const F& f) {
  uint64_t left = __ballot(id >= 0 && id < L);
  while (left) {
    const int first = __builtin_ctzll(left);
    const int a = __builtin_amdgcn_readlane(id, first);
    const uint64_t mask = __ballot(id == a) & left;
    f(a, mask);
    left &= ~mask;
  }
}

// Exclusive sums over the workgroup's threads of three counts.
__device__ __forceinline__ void block_scan3(int (&v)[3], int* lds) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int x[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    x[i] = v[i];
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
      const int y = __shfl_up(x[i], o);
      if (lane >= o) x[i] += y;
    }
    if (lane == 63) lds[wave * 3 + i] = x[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    int base = 0;
    for (int w = 0; w < wave; ++w) base += lds[w * 3 + i];
    v[i] = base + x[i] - v[i];
  }
  __syncthreads();
}

// hist: [waves][L] counts, then running positions; scan: 3 ints per wave.
__device__ void plan(const LoraPrep& p, int waves, int* hist, int* scan) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int L = p.s.L;
  for (int i = tid; i < waves * L; i += kPrepThreads) hist[i] = 0;
  __syncthreads();
  const int64_t span = (p.T + int64_t(waves) * 64 - 1) / (int64_t(waves) * 64) * 64;
  const int64_t lo = int64_t(wave) * span;
  const int64_t hi = wave >= waves ? lo : lo + span < p.T ? lo + span : p.T;
  int* mine = hist + wave * L;
  for (int64_t t = lo; t < hi; t += 64)
    for_each_id(t + lane < hi ? p.s.ids[t + lane] : -1, L, [&](int a, uint64_t mask) {
      if (lane == 0) mine[a] += __popcll(mask);
    });
  __syncthreads();
  // adapters a0 .. a1 - 1 of this thread: padded positions, pieces, pieces
  // that share an adapter (those leave partial sums)
  const int per = (L + kPrepThreads - 1) / kPrepThreads;
  const int a0 = tid * per < L ? tid * per : L, a1 = a0 + per < L ? a0 + per : L;
  int v[3] = {0, 0, 0};
  for (int a = a0; a < a1; ++a) {
    int n = 0;
    for (int w = 0; w < waves; ++w) n += hist[w * L + a];
    const int np = n ? (n + p.piece - 1) / p.piece : 1;
    v[0] += (n + 31) / 32 * 32;
    v[1] += np;
    v[2] += np > 1 ? np : 0;
  }
  block_scan3(v, scan);
  for (int a = a0; a < a1; ++a) {
    int n = 0;
    for (int w = 0; w < waves; ++w) {
      const int h = hist[w * L + a];
      hist[w * L + a] = v[0] + n;
      n += h;
    }
    const int np = n ? (n + p.piece - 1) / p.piece : 1;
    p.first_slot[a] = np > 1 ? v[2] : -1;
    p.slots[a] = np;
    p.last_pos[a] = v[0] + n - 1;
    for (int q = 0; q < np; ++q)
      p.pieces[v[1] + q] = LoraPiece{a, v[0] + q * p.piece,
                                     n - q * p.piece < p.piece ? n - q * p.piece : p.piece,
                                     np > 1 ? v[2] + q : -1};
    v[0] += (n + 31) / 32 * 32;
    v[1] += np;
    v[2] += np > 1 ? np : 0;
    if (a == L - 1) *p.n_pieces = v[1];
  }
  __syncthreads();
  for (int64_t t = lo; t < hi; t += 64) {
    const int id = t + lane < hi ? p.s.ids[t + lane] : -1;
    for_each_id(id, L, [&](int a, uint64_t mask) {
      const int base = mine[a];
      __builtin_amdgcn_wave_barrier();
      if (id == a && t + lane < hi) {
        const int pos = base + __popcll(mask & ((1ull << lane) - 1));
        p.token[pos] = int(t + lane);
        p.pos[t + lane] = pos;
        // the run's padding repeats its last token
        if (pos == p.last_pos[a])
          for (int q = pos + 1; q % 32; ++q) p.token[q] = int(t + lane);
      }
      __builtin_amdgcn_wave_barrier();
      if (lane == 0) mine[a] = base + __popcll(mask);
      __builtin_amdgcn_wave_barrier();
    });
  }
}

// Thread (kb, j): k rows 8kb .. + 7 of word column j (one group: its scales and
// zero points are loaded once), one 16-byte store per row.
template <bool F16>
__device__ __forceinline__ void dequant_t(const LoraPrep& p, int64_t i) {
#pragma clang fp contract(off)
  const int64_t N8 = p.w.N / 8, P8 = p.Np / 8;
  if (i >= p.w.K / 8 * P8) return;
  const int64_t kb = i / P8, j = i - kb * P8, k0 = kb * 8;
  uint16_t* out = p.Wt + k0 * p.Np + 8 * j;
  if (j >= N8) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      *reinterpret_cast<uint4*>(out + e * p.Np) = make_uint4(0, 0, 0, 0);
    return;
  }
  uint32_t w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = uint32_t(p.w.qweight[(k0 + e) * N8 + j]);
  const int64_t g = k0 / p.w.group;
  const uint32_t zw = uint32_t(p.w.qzeros[g * N8 + j]);
  const uint4 s4 = *reinterpret_cast<const uint4*>(p.w.scales + g * p.w.N + 8 * j);
  const uint32_t sw[4] = {s4.x, s4.y, s4.z, s4.w};
  float sc[8], zf[8];
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    sc[r] = f16_to_f32(uint16_t(sw[r >> 1] >> (16 * (r & 1))));
    zf[r] = float((zw >> (4 * r)) & 15u);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    uint32_t h[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float a = (float((w[e] >> (8 * r)) & 15u) - zf[2 * r]) * sc[2 * r];
      const float b = (float((w[e] >> (8 * r + 4)) & 15u) - zf[2 * r + 1]) * sc[2 * r + 1];
      h[r] = pack2<F16>(a, b);
    }
    *reinterpret_cast<uint4*>(out + e * p.Np) = make_uint4(h[0], h[1], h[2], h[3]);
  }
}

// Whether any token has adapter a (all threads of the workgroup agree).
__device__ __forceinline__ bool used(const LoraPrep& p, int a) {
  int hit = 0;
  for (int64_t t = threadIdx.x; t < p.T && !hit; t += kPrepThreads) hit = p.s.ids[t] == a;
  return __syncthreads_or(hit) != 0;
}

// 64 columns c of one adapter: rows [r][C] of A to [C][r] of Aᵀ.
__device__ __forceinline__ void transpose_a(const LoraPrep& p, int64_t tile, uint16_t* lds) {
  const int64_t tiles = p.w.K / 64;
  const int a = int(tile / tiles), r = p.s.r;
  if (!used(p, a)) return;
  const int64_t k0 = (tile % tiles) * 64;
  for (int e = threadIdx.x; e < r * 8; e += kPrepThreads) {
    const int j = e >> 3, q = e & 7;
    const uint4 x = *reinterpret_cast<const uint4*>(p.s.A + (int64_t(a) * r + j) * p.w.K + k0 +
                                                    8 * q);
    const uint32_t ww[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int h = 0; h < 8; ++h) lds[(8 * q + h) * (r + 2) + j] = uint16_t(ww[h >> 1] >> (16 * (h & 1)));
  }
  __syncthreads();
  uint32_t* out = reinterpret_cast<uint32_t*>(p.At + (int64_t(a) * p.w.K + k0) * r);
  for (int e = threadIdx.x; e < 64 * r / 2; e += kPrepThreads) {
    const int k = e / (r / 2), j = 2 * (e - k * (r / 2));
    out[e] = uint32_t(lds[k * (r + 2) + j]) | uint32_t(lds[k * (r + 2) + j + 1]) << 16;
  }
}

// 64 rows n of one adapter: [N][r] of B to [r][Np] of Bᵀ (zeros past N).
__device__ __forceinline__ void transpose_b(const LoraPrep& p, int64_t tile, uint16_t* lds) {
  const int64_t tiles = p.Np / 64;
  const int a = int(tile / tiles), r = p.s.r;
  if (!used(p, a)) return;
  const int64_t n0 = (tile % tiles) * 64;
  for (int e = threadIdx.x; e < 64 * r / 8; e += kPrepThreads) {
    const int n = e / (r / 8), q = e - n * (r / 8);
    uint4 x = make_uint4(0, 0, 0, 0);
    if (n0 + n < p.w.N)
      x = *reinterpret_cast<const uint4*>(p.s.B + (int64_t(a) * p.w.N + n0 + n) * r + 8 * q);
    const uint32_t ww[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int h = 0; h < 8; ++h) lds[(8 * q + h) * 66 + n] = uint16_t(ww[h >> 1] >> (16 * (h & 1)));
  }
  __syncthreads();
  for (int e = threadIdx.x; e < r * 32; e += kPrepThreads) {
    const int j = e >> 5, n = 2 * (e & 31);
    *reinterpret_cast<uint32_t*>(p.Bt + (int64_t(a) * r + j) * p.Np + n0 + n) =
        uint32_t(lds[j * 66 + n]) | uint32_t(lds[j * 66 + n + 1]) << 16;
  }
}

__device__ __forceinline__ void pad_dy(const LoraPrep& p, int64_t i) {
  const int64_t P8 = p.Np / 8;
  if (i >= p.T * P8) return;
  const int64_t t = i / P8, j = i - t * P8;
  uint4 x = make_uint4(0, 0, 0, 0);
  if (8 * j < p.w.N) x = *reinterpret_cast<const uint4*>(p.dY + t * p.w.N + 8 * j);
  *reinterpret_cast<uint4*>(p.dYp + t * p.Np + 8 * j) = x;
}

template <bool F16>
__global__ __launch_bounds__(kPrepThreads) void lora_prep_kernel(LoraPrep p, LoraPrepGrid g) {
  extern __shared__ int lds[];
  __shared__ int scan[3 * kPrepWaves];
  uint32_t b = blockIdx.x;
  if (b < 1) return plan(p, g.waves, lds, scan);
  b -= 1;
  if (b < g.tb) return transpose_b(p, b, reinterpret_cast<uint16_t*>(lds));
  b -= g.tb;
  if (b < g.ta) return transpose_a(p, b, reinterpret_cast<uint16_t*>(lds));
  b -= g.ta;
  if (b < g.dq) return dequant_t<F16>(p, int64_t(b) * kPrepThreads + threadIdx.x);
  b -= g.dq;
  pad_dy(p, int64_t(b) * kPrepThreads + threadIdx.x);
}

}  // namespace

hipError_t launch_lora_prep(const LoraPrep& p, hipStream_t st) {
  LoraPrepGrid g{};
  const int L = p.s.L, r = p.s.r;
  g.waves = kPrepWaves;                 // [waves][L] counts within 60 KiB of LDS
  while (g.waves * L > 15 * 1024) g.waves /= 2;
  auto blocks = [](int64_t n) { return uint32_t((n + kPrepThreads - 1) / kPrepThreads); };
  g.tb = uint32_t(L * (p.Np / 64));
  if (p.At) g.ta = uint32_t(L * (p.w.K / 64));
  if (p.Wt) g.dq = blocks(p.w.K / 8 * (p.Np / 8));
  g.pad = p.dYp ? blocks(p.T * (p.Np / 8)) : 0;
  size_t lds = size_t(g.waves) * L * 4;
  const size_t tr = size_t(64) * (r + 2) * 2 > size_t(r) * 66 * 2 ? size_t(64) * (r + 2) * 2
                                                                  : size_t(r) * 66 * 2;
  if (tr > lds) lds = tr;
  const uint32_t grid = 1 + g.tb + g.ta + g.dq + g.pad;
  auto kernel = p.f16 ? lora_prep_kernel<true> : lora_prep_kernel<false>;
  kernel<<<grid, kPrepThreads, lds, st>>>(p, g);
  return hipGetLastError();
}

}  // namespace awq
