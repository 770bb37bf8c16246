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

// Nibbles (0, 4), (1, 5), (2, 6), (3, 7) of w minus the integer behind the
// biases: bias = 1024 + z, bias16 = -(64 + z), both exact in fp16.
__device__ __forceinline__ void decode_nibbles(uint32_t w, uint32_t bias, uint32_t bias16, uint32_t (&a)[4]) {
  const uint32_t w8 = w >> 8;
  a[0] = hsub2_u(lop3_and_or(w, 0x000F000Fu, 0x64006400u), bias);
  a[1] = hfma2_u(lop3_and_or(w, 0x00F000F0u, 0x64006400u), 0x2C002C00u, bias16);
  a[2] = hsub2_u(lop3_and_or(w8, 0x000F000Fu, 0x64006400u), bias);
  a[3] = hfma2_u(lop3_and_or(w8, 0x00F000F0u, 0x64006400u), 0x2C002C00u, bias16);
}
// The biases of a pair of zero-points (fp16, integers 0 .. 15): 1024 + z and
// -64 - z by exact fp16 additions.
__device__ __forceinline__ void zero_biases(uint32_t z, uint32_t& bias, uint32_t& bias16) {
  bias = hfma2_u(z, 0x3C003C00u, 0x64006400u);
  bias16 = hfma2_u(z, 0xBC00BC00u, 0xD400D400u);
}

__device__ __forceinline__ uint32_t hmul2_u16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

}  // namespace qk
