// attn_tiles.h -- what the attention kernels that hold 32 queries a wavefront and 64-key tiles in
// LDS share: the range of their probabilities, and where a tile's pieces sit.
#pragma once

#include "attn_device.h"

namespace nvq {

constexpr int kKeys = 64;  // of a tile
constexpr int kTileWaves = 4;  // wavefronts of a workgroup

// A score may pass the running maximum by 2^SLACK before everything is rescaled; probabilities are
// taken times 2^SHIFT.  In bfloat16 they are at most 1 with it: values reach to the top of float32, and
// times 2^SLACK they would pass it where the result does not.  In binary16 together 2^15, all that the type has room for: it keeps its 11
// bits of a probability down to 2^-25 of the largest (17 nats) and holds them down to 2^-36.  (With 2^8
// and 2^0, keys 16 nats below a heavy one whose values are 0 were off by 9 times the half unit.  The smaller slack
// costs nothing at scores of width 1 and 1.6 % at width 3: 8192 tokens 675 and 696 us.)
template <typename T>
struct Range {
  static constexpr float SLACK = 8.0f, SHIFT = -8.0f;
};
template <>
struct Range<_Float16> {
  static constexpr float SLACK = 4.0f, SHIFT = 11.0f;
};
// What is taken from a score (base 2) with the running maximum m
template <typename T>
__device__ __forceinline__ float score_base(float m) {
  return (m == -__builtin_inff() ? 0.0f : m) - Range<T>::SHIFT;
}

// A staged tile of 64 key (or value) rows: where its 16-byte pieces sit.  The rows follow one
// another; within a row the pieces are exchanged by row bits, so that the lanes of one LDS
// read, which take one piece of different rows (keys), or 32 bytes of each of four rows
// (values, transposed), fall on different banks (64 of 4 bytes).
template <int NB>
struct Stage {
  static constexpr int ROW = 64 * NB, PIECES = 4 * NB, BYTES = kKeys * ROW;
  static constexpr int LOADS = BYTES / 1024 / kTileWaves;  // 1 KB loads of a wavefront
  // (an exchange stays inside aligned groups of 16, 8 or 4 pieces, so it fits any row)
  static __device__ __forceinline__ int key_piece(int row, int i) {
    return PIECES % 16 == 0 ? i ^ (row & 15) : PIECES % 8 == 0 ? i ^ ((row >> 1) & 7) : i ^ ((row >> 2) & 3);
  }
  static __device__ __forceinline__ int value_piece(int row, int i) {
    return PIECES % 16 == 0 ? i ^ ((row & 3) << 2) : PIECES % 8 == 0 ? i ^ ((row & 2) << 1) : i;
  }
};

}  // namespace nvq
