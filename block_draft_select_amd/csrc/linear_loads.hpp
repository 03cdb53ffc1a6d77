// Where the 8-bit product's kernels read their operands: arrays of 8-bit rows
// as buffers, and each lane's place in them.  Constant expressions, so that a test
// on the host goes through every load.
//
// A load of a buffer is checked against its size: 16 bytes that begin at the size
// or behind it are not read.  Only the lane's own offset is sure to be part of
// that check (the scalar one is taken from the size before the comparison, which
// does not say what holds once it is the larger one), so row and piece of k all
// go there, and rows behind the last one, or pieces behind its end, need no clamp.
#pragma once

#include <cstdint>

#include "dflash.h"

namespace dfk {

constexpr int kTileCh = 256;       // channels of a tile
constexpr int kBufferRows = 256;   // that a block reaches over
constexpr int kLdsBytes = 163840;
static_assert((int64_t)kBufferRows * DFLASH_I8_STRIDE_MAX < INT32_MAX - 2 * DFLASH_H_MAX, "offsets in 32 bits");

// bytes of an array's rows from `row` on, of what a block reaches
constexpr int buffer_bytes(int64_t row, int64_t rows, int64_t stride, int H) {
  const int64_t behind = rows - 1 - row;
  return (int)((behind < kBufferRows - 1 ? behind : kBufferRows - 1) * stride) + (H + 15) / 16 * 16;
}

// place l % 8 of row l / 8 (in LDS) holds this piece of 128 bytes
constexpr int load_piece(int lane) { return ((lane & 7) ^ (lane >> 3)) * 16; }

// ---- tiles: a wave's loads of a stage, eight rows each

template <int TT>
struct TileLoads {
  static constexpr int BM = 32 * TT, SB = (kTileCh + BM) * 128, NB = kLdsBytes / SB;
  static constexpr int PER = (kTileCh + BM) / 64;  // loads a wave: four of channels, then tokens
  static_assert(NB >= 2, "a stage in use, one landing");
};

// the channel of a wave's i-th load (of the 64 that a pair of waves brings): rows 8 (j % 2) .. of tile j / 2, row
// i of tile c being channel 16 (i / 4) + 4 c + i % 4
constexpr int tile_channel(int wave, int lane, int i) {
  const int j = (wave & 1) * 4 + i;
  return 32 * (j & 1) + 4 * (j >> 1) + (lane >> 5) * 16 + (lane >> 3 & 3);
}

template <int TT>
constexpr int tile_token(int wave, int lane, int i) {
  return 8 * (wave * (TT / 2) + i - 4) + (lane >> 3);
}

// where the row's stage number s lies (behind the last one: behind the row, or in it again)
constexpr int tile_stage(int s, int rot, int n_st) { return s + rot < n_st || rot == 0 ? s + rot : s + rot - n_st; }

// ---- streamed weights: a wave's two loads of a step, eight rows each

constexpr int stream_channel(int lane, int i) { return 8 * i + (lane >> 3); }

}  // namespace dfk
