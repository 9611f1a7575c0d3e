// 16-row operand tiles of the low-rank kernels, staged through LDS.
//
// An MFMA operand read straight from memory touches 16 rows per 16 bytes of
// each, lane by lane: measured, a 64-lane load of that shape costs 64 cache
// accesses where a row-contiguous one costs 8 to 16. So tiles go to LDS with
// buffer_load_dwordx4 ... lds, whole 256-byte row segments at a time (128
// channels of a 16-bit type), and operands are read from there. The 16-byte
// chunk c of row i sits at chunk c ^ (i % 16), so the 16 lanes of an operand
// read (one chunk of 16 rows) hit all 64 banks.
#pragma once

#include "gemm_types.h"

namespace awq {
namespace {

#define AWQ_LORA_LDS(p) ((__attribute__((address_space(3))) void*)(p))

constexpr int kTileChunks = 16;              // 16-byte chunks per row (128 channels)
constexpr int kTile16 = 16 * kTileChunks;    // uint4 per 16-row tile

// s_waitcnt vmcnt(n) with the other counters left alone (gfx9 encoding).
template <int N>
__device__ __forceinline__ void wait_vmem() {
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

__device__ __forceinline__ void wait_lds() {   // lgkmcnt(0)
  __builtin_amdgcn_s_waitcnt(0xF | (3 << 14) | (0x7 << 4));
}

// Keeps memory operations and instructions on their side of it.
__device__ __forceinline__ void fence() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Rows of a matrix with `ld` elements per row, as a buffer resource: offsets
// past the last row read as zero. rows·ld·2 < 2^31.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const uint16_t* base, int64_t rows,
                                                            int64_t ld) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(base), 0, int(rows * ld * 2),
                                           0x00020000);
}

// Lane offset (bytes) of copy i (4 rows: 4i .. + 3) of a 16-row tile whose
// first row is row0.
__device__ __forceinline__ uint32_t tile_offset(int row0, int i, int64_t ld) {
  const int lane = threadIdx.x & 63;
  const int row = 4 * i + (lane >> 4);
  return uint32_t(((int64_t(row0) + row) * ld + ((lane & 15) ^ row) * 8) * 2);
}

// Copy i of a tile (1 KiB) at channel k of its rows.
__device__ __forceinline__ void tile_copy(__amdgpu_buffer_rsrc_t rs, uint32_t off, int k,
                                          uint4* tile, int i) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, AWQ_LORA_LDS(tile + i * 64), 16, off, 2 * k, 0,
                                           0);
}

// The operand of 32-channel step s: row l % 16, channels 32·s + 8·(l / 16) ..
__device__ __forceinline__ uint4 tile_read(const uint4* tile, int s) {
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  return tile[lr * kTileChunks + ((4 * s + lg) ^ lr)];
}

// Row i of a tile, chunk c.
__device__ __forceinline__ uint4 tile_chunk(const uint4* tile, int i, int c) {
  return tile[i * kTileChunks + (c ^ i)];
}

}  // namespace
}  // namespace awq
