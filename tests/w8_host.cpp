// The plans of the 8-bit products and the ranges of their 256x256 main loop, on the host:
// built together with validate.cpp by test_w8_host_cpu.py.
#include <algorithm>
#include <array>
#include <cstring>

#include "awq_internal.h"
#include "w8_phi.h"
#include "w8_ring_range.h"

using namespace awq;

// Replays every copy of one operand by one wave as ring_mainloop issues them, also those
// past the end. k-tile i begins next·i bytes after `first`, its row r's 128 bytes row·r
// further on; of the wave's 64 rows from wave_row those below `valid` exist, in an
// allocation of `size` bytes.
struct Replay {
  int64_t past = INT64_MIN;   // bytes that an admitted copy reaches past the allocation
  int64_t missed = 0;         // copies of existing rows that are refused
  int64_t stray = 0;          // copies of other rows, or past the last k-tile, that are not

  void operand(RingRange range, int64_t first, int64_t next, int row, int wave_row, int valid,
               int64_t size, int tiles) {
    for (int i = 0; i < tiles + 2; ++i, range.advance())
      for (int j = 0; j < 8; ++j)
        for (int lane = 0; lane < 64; ++lane) {
          // the hardware's check takes the bytes as unsigned
          const int64_t off = ring_offset(wave_row, lane, j & 1, row) + int64_t(j) * 8 * row;
          const bool admitted = off + 16 <= int64_t(uint32_t(range.bytes));
          const int r = wave_row + 8 * j + (lane >> 3);
          const bool there = i < tiles && r < valid;
          missed += there && !admitted;
          stray += admitted && !there;
          if (admitted) past = std::max(past, first + next * i + off + 16 - size);
          if (admitted && first + next * i + off < 0) ++stray;
        }
  }
};

// A first, a last but one and a last tile.
static std::array<int64_t, 3> edges(int64_t tiles) {
  return {0, std::max<int64_t>(0, tiles - 2), tiles - 1};
}

static void answer(const Replay& r, int64_t* out) {
  out[0] = r.past;
  out[1] = r.missed;
  out[2] = r.stray;
}

// form (0 few, 1 mid, 2 big), tile_n, tile_t, runs, cut.full, cut.runs, bytes
extern "C" void w8_host_plan(int64_t T, int64_t N, int64_t K, int32_t layers, int64_t* out) {
  const W8Plan l = w8_plan(T, N, K, layers);
  const int64_t v[] = {int64_t(l.form), l.tile_n, l.tile_t, l.runs, l.cut.full, l.cut.runs,
                       int64_t(l.bytes)};
  memcpy(out, v, sizeof v);
}

// few, tile_t, runs, cut.full, cut.runs, bytes
extern "C" void w8_host_back_plan(int64_t T, int64_t N, int64_t K, int32_t layers, int64_t* out) {
  const W8BackLayout l = w8_back_layout(T, N, K, layers);
  const int64_t v[] = {l.few, l.tile_t, l.runs, l.cut.full, l.cut.runs, int64_t(l.total)};
  memcpy(out, v, sizeof v);
}

// A product in the 256x256 form (w8_gemm.hip), its contraction in `runs` runs.
extern "C" void w8_host_replay(int64_t T, int64_t N, int64_t K, int32_t layers, int32_t runs,
                               int64_t* out) {
  const int64_t channels = layers == 2 ? 128 : 256;
  const int steps = int(K / 128);
  Replay rep;
  for (int run = 0; run < runs; ++run) {
    const int k0 = steps * run / runs, k1 = steps * (run + 1) / runs;
    for (int wave = 0; wave < 4; ++wave) {
      for (int64_t tt : edges(ceil_div(T, 256))) {
        const int64_t t0 = tt * 256;
        const int valid = int(std::min<int64_t>(T - t0, 256));
        rep.operand(ring_range(RingKind::kRows, valid, int(K), k1 - k0), t0 * K + k0 * 128, 128,
                    int(K), wave * 64, valid, T * K, k1 - k0);
      }
      for (int64_t tn : edges(ceil_div(N, channels))) {
        const int64_t n0 = tn * channels;
        if (layers == 2) {
          const PairRows rows = pair_rows(n0, wave, N);
          rep.operand(ring_range(RingKind::kRows, rows.valid, int(K), k1 - k0),
                      rows.first * K + k0 * 128, 128, int(K), 0, rows.valid, N * K, k1 - k0);
        } else {
          const int valid = int(std::min<int64_t>(N - n0, 256));
          rep.operand(ring_range(RingKind::kRows, valid, int(K), k1 - k0), n0 * K + k0 * 128, 128,
                      int(K), wave * 64, valid, N * K, k1 - k0);
        }
      }
    }
  }
  answer(rep, out);
}

// A gradient through the transposed layer (w8_back.hip): both operands in panels of 64 of
// the contraction, 128 bytes a row.
extern "C" void w8_host_back_replay(int64_t T, int64_t N, int64_t K, int32_t layers, int32_t runs,
                                    int64_t* out) {
  const int64_t C = layers * ceil_div(N, 64) * 64;
  const int steps = int(C / 64);
  Replay rep;
  for (int run = 0; run < runs; ++run) {
    const int k0 = steps * run / runs, k1 = steps * (run + 1) / runs;
    for (int wave = 0; wave < 4; ++wave)
      for (int64_t rows : {K, T})
        for (int64_t tile : edges(ceil_div(rows, 256))) {
          const int64_t o0 = tile * 256, panel = rows * 128;
          const int valid = int(std::min<int64_t>(rows - o0, 256));
          rep.operand(ring_range(RingKind::kPanels, valid, 128, k1 - k0), k0 * panel + o0 * 128,
                      panel, 128, wave * 64, valid, rows * C * 2, k1 - k0);
        }
  }
  answer(rep, out);
}

// The fit of erfcx(x / √2) / 2 with its own coefficients, exactly evaluated.
extern "C" void w8_host_phi(const double* x, int64_t n, double* y) {
  for (int64_t i = 0; i < n; ++i) {
    const double t = 1 / (1 + double(kPhiT) * x[i]);
    double q = 0;
    for (const float c : kPhi) q = q * t + double(c);
    y[i] = t * q;
  }
}

extern "C" int64_t w8_host_row_threads(int64_t K) { return row_threads(K); }
