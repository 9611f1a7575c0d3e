// The gradient of the input for few tokens, without a dequantised layer:
//
//   dX[t][k] = Σ_n dY[t][n]·Ŵ[n][k] + Σ_j c_a·P[t][j]·A_a[j][k],
//
// the shared product here as float32 partial sums over runs of n, the rest by
// the forward call's second launch (lora_few.hip) with Aᵀ in B's place.
//
// As in the forward product a wave takes 16·MT tokens x 128 outputs, now
// channels k, and a run of n. A packed word holds 8 consecutive n of one k:
// that is one lane's operand, so word (k = 16·R + l % 16, n = 8·(l / 16) ..)
// makes operand R of a block of 32 n. One shift and four and-ors turn it into
// fp16 pairs of nibbles (i, i + 4), and the products with the group's scales
// into Ŵ as the dequantisation pass rounds it (lora_few.hip); scales and zero
// points vary along n and, by group, along k.
//   bf16: float32 fma((B + q), scale, -(B + z)·scale), two of them rounded to a
//   pair of consecutive n;
//   fp16: pairs (i, i + 4), and dY's chunks permuted to match.
// Words past N belong to other rows; their scales read as zero, and so does dY
// there.
//
// Bound by the issue of vector instructions, as the forward product. In place of
// a pass that writes Ŵᵀ and 256x256 tiles: the whole gradient of 64 tokens, bf16,
// rank 16, 91 instead of 265 us at 28672x8192, 38 instead of 55 at 4096x4096.
#include "lora.h"
#include "lora_combine.h"
#include "lora_few.h"

namespace awq {
namespace {

// A wave's stage of 64 n: the packed words of 128 k rows, 8 words each (word w
// of row k at w ^ 4·(k / 8 % 2), which keeps reads of 16 rows free of bank
// conflicts), and by group the scales (8 chunks of 8) and zero points (8 words).
struct BackSlot {
  uint4 w[128 * 2], s[64], z[16];
};

// Pair i of a word: nibbles i and i + 4 as fp16 numbers B + q (B = 1024 for
// even i, 64 for odd).
template <int I>
__device__ __forceinline__ f16x2_t back_code(uint32_t w, const uint32_t (&base)[2]) {
  const uint32_t x = I >= 2 ? w >> 8 : w;
  return __builtin_bit_cast(f16x2_t, (x & (I & 1 ? 0x00F000F0u : 0x000F000Fu)) | base[I & 1]);
}
// A group's scales and zero points for the lane's 8 n: -(B + z)·scale and the
// scales as they are (bf16), or both as pairs (i, i + 4) (fp16).
template <bool F16>
struct BackZeros {
  float z[8];
  uint32_t s[4];
};
template <>
struct BackZeros<true> {
  f16x2_t z[4], s[4];
};
__device__ __forceinline__ _Float16 half_of(uint32_t w, int hi) {
  return __builtin_bit_cast(_Float16, uint16_t(w >> (16 * hi)));
}
template <bool F16, int I = 0>
__device__ __forceinline__ void back_zeros(BackZeros<F16>& n, uint32_t z, const uint4& s,
                                           const uint32_t (&base)[2]) {
  if constexpr (I < 4) {
    const uint32_t sw[4] = {s.x, s.y, s.z, s.w};
    const f16x2_t c = back_code<I>(z, base);
    const uint32_t lo = sw[I / 2], hi = sw[2 + I / 2];
    if constexpr (F16) {
      n.z[I] = c;
      n.s[I] = __builtin_bit_cast(
          f16x2_t, __builtin_amdgcn_perm(hi, lo, I & 1 ? 0x07060302u : 0x05040100u));
    } else {
      n.s[I] = sw[I];
      n.z[I] = -(float(c[0]) * float(half_of(lo, I & 1)));
      n.z[I + 4] = -(float(c[1]) * float(half_of(hi, I & 1)));
    }
    back_zeros<F16, I + 1>(n, z, s, base);
  }
}

// The operands of a block of 32 n. NG: groups in 128 channels; operand R belongs
// to group R·NG / 8, whose scales are read from the stage a group ahead. Words in
// the order of their codes: bf16 takes the low halves of two pairs as word 0 (or
// 1), their high halves as word 2 (or 3).
template <bool F16, int NG>
struct BackBlock {
  const uint32_t (&w)[8];
  const BackSlot& st;
  int at;                 // the lane's 8 n in a group's row of the stage
  const uint32_t (&base)[2];
  uint32_t z;
  uint4 s;
  BackZeros<F16> n;
  f16x2_t c[2];
  __device__ __forceinline__ void read(int g) {
    z = reinterpret_cast<const uint32_t*>(st.z)[8 * g + at];
    s = st.s[8 * g + at];
  }
  __device__ static constexpr int word(int e) { return F16 || e == 0 || e == 3 ? e : 3 - e; }
  template <int R, int E>
  __device__ __forceinline__ void pair(uint32_t& lo, uint32_t& hi) {
    if constexpr (E == 0 && R % (8 / NG) == 0) {
      back_zeros<F16>(n, z, s, base);
      if constexpr (R + 8 / NG < 8) read(R * NG / 8 + 1);
    }
    if constexpr (F16) {
      lo = __builtin_bit_cast(uint32_t, (back_code<E>(w[R], base) - n.z[E]) * n.s[E]);
    } else {
      if constexpr (E % 2 == 0) {
        c[0] = back_code<E>(w[R], base);
        c[1] = back_code<E + 1>(w[R], base);
      }
      constexpr int kH = E & 1, kN = (E & 2) + 4 * kH;      // n = kN, kN + 1
      lo = __builtin_bit_cast(uint32_t, __builtin_fmaf(float(c[0][kH]),
                                                       float(half_of(n.s[kN / 2], 0)), n.z[kN]));
      hi = __builtin_bit_cast(uint32_t, __builtin_fmaf(float(c[1][kH]),
                                                       float(half_of(n.s[kN / 2], 1)),
                                                       n.z[kN + 1]));
    }
  }
};

// WIDE: N a multiple of 32, rows of packed words 16-byte aligned.
template <bool F16, int MT, int NG, bool WIDE>
__global__ __launch_bounds__(64 * kFewWaves, 2) void lora_few_back_kernel(LoraFewBack p) {
  // the narrow product's sums, by the workgroups behind (the last launch but
  // one has left their parts; a launch of its own took 4 us)
  const int blocks = p.tiles * p.col_blocks * p.S;
  if (int(blockIdx.x) >= blocks) return lora_combine<F16>(p.down, int(blockIdx.x) - blocks);
  typedef typename Operand<F16>::type V;
  constexpr uint32_t kOob = 0x80000000u;
  __shared__ uint4 xs[kFewWaves * 16 * MT * 8];
  __shared__ BackSlot q0[kFewWaves], q1[kFewWaves];
  FewX<MT>& sx = reinterpret_cast<FewX<MT>&>(xs);
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  const int64_t N = p.w.N, K = p.w.K, N8 = N / 8;
  // XCD i takes a contiguous run of (run of n, column block, token tile)
  // indices, token tiles fastest, as the forward product
  int tt, cb, s;
  {
    const int id = int(blockIdx.x);
    const int q = blocks / 8, rem = blocks % 8, xi = id % 8;
    int l = xi * q + (xi < rem ? xi : rem) + id / 8;
    tt = l % p.tiles;
    l /= p.tiles;
    cb = l % p.col_blocks;
    s = l / p.col_blocks;
  }
  const int64_t t0 = int64_t(tt) * 16 * MT, k0 = int64_t(cb) * kFewCols;
  const int n0 = (s * kFewWaves + wave) * p.npw;
  const int n1 = n0 + p.npw < int(p.Np) ? n0 + p.npw : int(p.Np);
  floatx4 acc[8][MT];
#pragma unroll
  for (int r = 0; r < 8; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[r][m] = floatx4{0.f, 0.f, 0.f, 0.f};
  if (n0 < n1) {
    const FewRows x = few_rows<MT>(p.dY, t0, p.T, p.Np);
    // (stages past the run read its last one)
    auto copy_x = [&](int nb) { few_copy_rows<MT>(x, sx[wave], nb < n1 ? nb : n1 - 64); };
    // 128 rows of at most N / 2 < 2^21 bytes
    const int rowb = int(N8 * 4);
    const auto rsQ = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<int32_t*>(p.w.qweight) + k0 * N8, 0, int(128 * N8 * 4), 0x00020000);
    uint32_t qoff[2];
    if constexpr (WIDE) {
      qoff[0] = uint32_t((lane >> 1) * rowb + (((lane & 1) ^ (lane >> 4 & 1)) * 16));
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        qoff[i] = uint32_t((lane >> 3) * rowb + ((lane & 7) ^ (4 * i)) * 4);
    }
    const int64_t g0 = k0 >> p.gshift;
    const auto rsS = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint16_t*>(p.w.scales) + g0 * N, 0, int(NG * N * 2), 0x00020000);
    const auto rsZ = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<int32_t*>(p.w.qzeros) + g0 * N8, 0, int(NG * N8 * 4), 0x00020000);
    const int lc = lane & 7, lgr = lane >> 3;
    const uint32_t soff = uint32_t((lgr * N + 8 * lc) * 2), zoff = uint32_t((lgr * N8 + lc) * 4);
    auto copy_q = [&](BackSlot& st, int nb) {
      const int n = nb < n1 ? nb : n1 - 64;
      if constexpr (WIDE) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          __builtin_amdgcn_raw_ptr_buffer_load_lds(rsQ, AWQ_LORA_LDS(st.w + 64 * i), 16, qoff[0],
                                                   32 * i * rowb + n / 2, 0, 0);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          __builtin_amdgcn_raw_ptr_buffer_load_lds(rsQ, AWQ_LORA_LDS(st.w + 16 * i), 4,
                                                   qoff[i & 1], 8 * i * rowb + n / 2, 0, 0);
      }
      const bool in = lgr < NG && n + 8 * lc < int(N);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsS, AWQ_LORA_LDS(st.s), 16, in ? soff : kOob,
                                               2 * n, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsZ, AWQ_LORA_LDS(st.z), 4, in ? zoff : kOob, n / 2,
                                               0, 0);
    };
    // fp16 1024 and 64, opaque so that they stay in registers
    uint32_t base[2] = {0x64006400u, 0x54005400u};
    asm volatile("" : "+v"(base[0]), "+v"(base[1]));
    uint32_t wat[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) wat[h] = uint32_t(lr * 8 + ((4 * h + lg) ^ (4 * (lr >> 3))));
    // A stage's activations are copied a stage ahead, its words two. A wave
    // reads only what it copied itself: waits, no barriers.
    copy_q(q0[wave], n0);
    fence();
    copy_x(n0);
    fence();
    copy_q(q1[wave], n0 + 64);
    fence();
    constexpr int kBehind = (WIDE ? 4 : 16) + 2;   // what was asked for after a stage's dY
    auto stage = [&](BackSlot& st, int nb) {
      fence();
      wait_vmem<kBehind>();
      fence();
      V xv[2][MT];
      uint32_t w[2][8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          uint4 d = sx[wave][x.at[h] + 128 * m];
          if constexpr (F16)
            d = make_uint4(__builtin_amdgcn_perm(d.z, d.x, 0x05040100u),
                           __builtin_amdgcn_perm(d.z, d.x, 0x07060302u),
                           __builtin_amdgcn_perm(d.w, d.y, 0x05040100u),
                           __builtin_amdgcn_perm(d.w, d.y, 0x07060302u));
          xv[h][m] = __builtin_bit_cast(V, d);
        }
#pragma unroll
        for (int r = 0; r < 8; ++r)
          w[h][r] = reinterpret_cast<const uint32_t*>(st.w)[wat[h] + 128 * r];
      }
      fence();
      wait_lds();      // read before they are copied over
      fence();
      copy_x(nb + 64);
      fence();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        BackBlock<F16, NG> b{w[h], st, 4 * h + lg, base};
        b.read(0);
        few_block<F16, MT>(b, xv[h], acc);
      }
      fence();
      wait_lds();
      fence();
      copy_q(st, nb + 128);
      fence();
    };
    // (npw and Np are multiples of 128)
    for (int nb = n0; nb < n1; nb += 128) {
      stage(q0[wave], nb);
      stage(q1[wave], nb + 64);
    }
    wait_vmem<0>();
    few_settle<MT>(acc);
  }
  // lane l holds channels 16·R + l % 16, tokens 16·m + 4·(l / 16) + v
  float* const out = p.partial + (int64_t(s) * p.T + t0 + 4 * lg) * K + k0 + lr;
  const int64_t left = p.T - t0 - 4 * lg;
  auto store = [&](int u, int m, const floatx4 (&y)[2]) {
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (16 * m + v < left) {
        out[(16 * m + v) * K + 32 * u] = y[0][v];
        out[(16 * m + v) * K + 32 * u + 16] = y[1][v];
      }
  };
  AWQ_FEW_MEET(acc, sx, wave, lane, MT, store)
}

template <bool F16, int MT, int NG>
void launch_ng(const LoraFewBack& p, hipStream_t st) {
  const unsigned grid = unsigned(p.tiles * p.col_blocks * p.S + (p.T + 3) / 4);
  if (p.w.N % 32 == 0) lora_few_back_kernel<F16, MT, NG, true><<<grid, 256, 0, st>>>(p);
  else lora_few_back_kernel<F16, MT, NG, false><<<grid, 256, 0, st>>>(p);
}
template <bool F16, int MT>
void launch_mt(const LoraFewBack& p, hipStream_t st) {
  if (p.w.group == 128) launch_ng<F16, MT, 1>(p, st);
  else if (p.w.group == 64) launch_ng<F16, MT, 2>(p, st);
  else launch_ng<F16, MT, 4>(p, st);
}
template <bool F16>
void launch_f(const LoraFewBack& p, hipStream_t st) {
  if (p.T <= 32) launch_mt<F16, 2>(p, st);
  else launch_mt<F16, 4>(p, st);
}

}  // namespace

hipError_t launch_lora_few_back(const LoraFewBack& p, hipStream_t st) {
  if (p.w.K % kFewCols || p.Np % 128 || p.npw % 128 || p.w.N % 8) return hipErrorInvalidValue;
  if (p.f16) launch_f<true>(p, st);
  else launch_f<false>(p, st);
  return hipGetLastError();
}

}  // namespace awq
