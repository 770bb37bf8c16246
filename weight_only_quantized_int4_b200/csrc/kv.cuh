// Layout of the 4-bit key / value cache (include/qmm.h), shared by its kernels.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace qk {

constexpr int kKvTile = 16;   // tokens per tile, the unit the cache is made of

// A tile of 16 tokens of one head: key codes, value codes (16 rows of D / 2
// bytes each), key parameters, value parameters ([16][G], a scale or a
// (scale, zero) pair of fp16).
__host__ __device__ constexpr int kv_param_bytes(int mode) { return mode == kASYM ? 4 : 2; }
__host__ __device__ constexpr int kv_tile_bytes(int dim, int G, int mode) {
  return kKvTile * (dim + 2 * G * kv_param_bytes(mode));
}

// Place, in 32-bit words of a key row, of the row's natural word n (dims 8n ..
// 8n + 7) for a token at place `tok` of its tile.  n = 4w + t: lane t of a
// quad finds its words w = 0 .. 3 (dims 32w + 8t ..) in one 16-byte piece, so a
// group of 32 dims is one w of all four lanes.  256 dims: two pieces per lane,
// swapped for odd tokens so that two rows' reads hit different banks.
__host__ __device__ constexpr int kv_key_word(int dim, int n, int tok) {
  const int w = n >> 2, t = n & 3;
  if (dim == 64) return 2 * t + w;
  int piece = t + 4 * (w >> 2);
  if (dim == 256) piece ^= 4 * (tok & 1);
  return 4 * piece + (w & 3);
}
// The same for a value row: a lane group g reads D / 8 consecutive dims (a
// piece of D / 16 bytes); the pieces of different tokens are exchanged so that
// the four tokens a warp reads at once hit different banks.
__host__ __device__ constexpr int kv_val_piece(int dim, int piece, int tok) {
  if (dim == 128) return piece ^ (4 * ((tok >> 1) & 1));
  if (dim == 256) return piece ^ (2 * (tok & 3));
  return piece;
}
__host__ __device__ constexpr int kv_val_word(int dim, int n, int tok) {
  const int per = dim / 64;
  return kv_val_piece(dim, n / per, tok) * per + n % per;
}

}  // namespace qk
