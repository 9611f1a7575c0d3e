// The main loop of the 256x256 tiles of the 8-bit products: 256 rows of A (output
// channels) x 256 rows of B (tokens), 128 bytes of the contraction a k-tile (128 codes
// or 64 16-bit numbers).
//
//  * Four waves in 2x2, one a SIMD, each 128x128 outputs as 8x8 blocks of 16x16 in
//    AGPRs; a k-tile is 128 matrix instructions a wave, 2048 cycles.
//  * A k-tile's rows of A or of B, 32 KiB, come by buffer_load ... lds into one of 5
//    units that fill the LDS: the next k-tile's B in a region's first half, the A of
//    the one after it in the second.
//    With two stages of both and every copy in the first half, where the address unit
//    was busy all the time, 2051 tokens of a pair 28672x8192 took 888 us instead of
//    840, the gradient of 4096 tokens of a pair 11008x4096 685 instead of 641. Units of
//    64 bytes of A and B, 4 ahead, took more (8192 tokens of 4096x11008: 313 instead of
//    261): half a line a request, so twice the requests to L2.
//  * The waves meet once a k-tile; the wait there leaves A's copies in flight.
//  * The card runs these loops at 1.9 of its 2.4 GHz; at that clock the matrix cores
//    are busy for 70 of 100 cycles.
#pragma once

#include "gemm_core.h"
#include "w8_ring_range.h"

namespace awq {
namespace {

// 16 codes an operand; the accumulator's registers hold 4 int32 sums (whose zero is
// the float's).
__device__ __forceinline__ void mfma16(floatx4& c, const i8x16_t& a, const i8x16_t& b) {
  asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}
__device__ __forceinline__ void mfma16_first(floatx4& c, const i8x16_t& a, const i8x16_t& b) {
  asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, 0" : "=a"(c) : "v"(a), "v"(b));
}

constexpr int kRing = 5;

// One array each: the compiler can tell the units being read from those being filled.
__shared__ uint4 ring0[STAGE64], ring1[STAGE64], ring2[STAGE64], ring3[STAGE64], ring4[STAGE64];
template <int U>
__device__ __forceinline__ uint4* ring_unit() {
  constexpr int u = U % kRing;
  return u == 0 ? ring0 : u == 1 ? ring1 : u == 2 ? ring2 : u == 3 ? ring3 : ring4;
}

template <class T>
__device__ __forceinline__ const T* uniform(const T* p) {
  const uint64_t u = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(u)),
                 hi = __builtin_amdgcn_readfirstlane(uint32_t(u >> 32));
  return reinterpret_cast<const T*>(uint64_t(hi) << 32 | lo);
}
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// One operand's next k-tile to copy: rows of `row` bytes, the next k-tile `next` bytes
// on. Rows past the last valid one, and k-tiles past the end, read as zero. All but v
// scalar, and said to be: else every copy is a loop over the lanes' resources (4096
// tokens of 4096x11008: 165 instead of 150 us).
struct RingSide {
  const char* at;
  int64_t next;
  RingRange range;
  int v[2], rows;       // the lane's offset in even and odd copies; bytes of 8 rows
  // wave_row: the first row that the wave copies, from `first`
  // (a panel's length alone does not tell: one token's panels are 128 bytes, too)
  __device__ __forceinline__ void set(RingKind kind, const void* first, int valid, int row,
                                      int wave_row, int64_t to_next, int tiles) {
    at = uniform(static_cast<const char*>(first));
    next = to_next;
    range = ring_range(kind, uniform(valid), row, uniform(tiles));
    rows = 8 * row;
#pragma unroll
    for (int j = 0; j < 2; ++j) v[j] = ring_offset(wave_row, threadIdx.x & 63, j, row);
  }
  // copy j of the wave's 8: 8 rows into unit U
  template <int U>
  __device__ __forceinline__ void copy(int wave, int j) const {
    const __amdgpu_buffer_rsrc_t rs =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(at), 0, range.bytes, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, AWQ_LDS(ring_unit<U>() + (wave * 8 + j) * 64), 16,
                                             v[j & 1], j * rows, 0, 0);
  }
  __device__ __forceinline__ void advance() {
    at += next;
    range.advance();
  }
};
struct RingCtx {
  RingSide a, b;
  int wave;
};

// Fragment r of a k-step: B's blocks first (the first row of blocks needs them all).
template <int UA, class V>
__device__ __forceinline__ void ring_frag(int rda, int rdb, int r, V (&fa)[8], V (&fb)[8]) {
  if (r < 8) fb[r] = __builtin_bit_cast(V, ring_unit<UA + 1>()[rdb + r * 128]);
  else fa[r - 8] = __builtin_bit_cast(V, ring_unit<UA>()[rda + (r - 8) * 128]);
}

// K-tile t with A in unit UA (2t) and B in UA + 1: the previous one's k-step 1 (f1)
// carries k-step 0's reads and the copies of the next B, k-step 0 (f0) carries k-step
// 1's reads and the copies of the A after next, into the previous k-tile's units.
template <int UA, bool PREV, class V>
__device__ __forceinline__ void ring_region(RingCtx& c, const int (&rda)[2], const int (&rdb)[2],
                                            floatx4 (&acc)[8][8], V (&f0a)[8], V (&f0b)[8],
                                            V (&f1a)[8], V (&f1b)[8]) {
#pragma unroll
  for (int m = 0; m < 64; ++m) {
    if (PREV) mfma16(acc[m >> 3][m & 7], f1a[m >> 3], f1b[m & 7]);
    if (m % 4 == 3) ring_frag<UA>(rda[0], rdb[0], m / 4, f0a, f0b);
    if (m % 8 == 4) c.b.template copy<UA + 3>(c.wave, m / 8);
  }
  c.b.advance();
#pragma unroll
  for (int m = 0; m < 64; ++m) {
    if (PREV) mfma16(acc[m >> 3][m & 7], f0a[m >> 3], f0b[m & 7]);
    else mfma16_first(acc[m >> 3][m & 7], f0a[m >> 3], f0b[m & 7]);
    if (m % 4 == 3) ring_frag<UA>(rda[1], rdb[1], m / 4, f1a, f1b);
    if (m % 8 == 4) c.a.template copy<UA + 4>(c.wave, m / 8);
  }
  c.a.advance();
  __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
  __builtin_amdgcn_s_waitcnt(wait_vm(8));
  region_barrier();
}

// Writes every accumulator and ends with them safe to read and the LDS free.
template <class V>
__device__ __forceinline__ void ring_mainloop(RingCtx& c, floatx4 (&acc)[8][8]) {
  // lane l reads row l % 16 of a block of 16, chunk l / 16 of a k-step's 4
  const int lane = threadIdx.x & 63;
  int rda[2], rdb[2];
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) {
    rda[ks] = swz64((c.wave >> 1) * 128 + (lane & 15), 4 * ks + (lane >> 4));
    rdb[ks] = swz64((c.wave & 1) * 128 + (lane & 15), 4 * ks + (lane >> 4));
  }
  int n = c.a.range.left;
#pragma unroll
  for (int j = 0; j < 8; ++j) c.a.template copy<0>(c.wave, j);
  c.a.advance();
#pragma unroll
  for (int j = 0; j < 8; ++j) c.b.template copy<1>(c.wave, j);
  c.b.advance();
#pragma unroll
  for (int j = 0; j < 8; ++j) c.a.template copy<2>(c.wave, j);
  c.a.advance();
  __builtin_amdgcn_s_waitcnt(wait_vm(8));
  region_barrier();
  V f0a[8], f0b[8], f1a[8], f1b[8];
  ring_region<0, false>(c, rda, rdb, acc, f0a, f0b, f1a, f1b);
  for (; __builtin_expect(n > 5, 1); n -= 5) {
    ring_region<2, true>(c, rda, rdb, acc, f0a, f0b, f1a, f1b);
    ring_region<4, true>(c, rda, rdb, acc, f0a, f0b, f1a, f1b);
    ring_region<1, true>(c, rda, rdb, acc, f0a, f0b, f1a, f1b);
    ring_region<3, true>(c, rda, rdb, acc, f0a, f0b, f1a, f1b);
    ring_region<0, true>(c, rda, rdb, acc, f0a, f0b, f1a, f1b);
  }
  if (__builtin_expect(n > 1, 1)) ring_region<2, true>(c, rda, rdb, acc, f0a, f0b, f1a, f1b);
  if (__builtin_expect(n > 2, 1)) ring_region<4, true>(c, rda, rdb, acc, f0a, f0b, f1a, f1b);
  if (__builtin_expect(n > 3, 1)) ring_region<1, true>(c, rda, rdb, acc, f0a, f0b, f1a, f1b);
  if (__builtin_expect(n > 4, 1)) ring_region<3, true>(c, rda, rdb, acc, f0a, f0b, f1a, f1b);
#pragma unroll
  for (int m = 0; m < 64; ++m) mfma16(acc[m >> 3][m & 7], f1a[m >> 3], f1b[m & 7]);
  // the compiler sees no MFMA in the asm, so it inserts no wait before the
  // accumulators are read; the empty statements tie every read to the nops
  asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) asm volatile("" : "+a"(acc[i][j]));
  __builtin_amdgcn_s_waitcnt(wait_vm(0));   // the copies (of zeros) past the end
  region_barrier();
}

}  // namespace
}  // namespace awq
