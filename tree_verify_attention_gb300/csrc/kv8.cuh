// The 8-bit cache with a scale for each block of 64 positions and head:
// layout and limits shared by its writer, its reader and its attention.
//
// Block b of a head holds positions [64 b, 64 b + 64). A complete block is
// 64 * D signed codes for K, as many for V, and one f32 scale each; the value
// is code * scale. K codes lie as [D / 16][64][16] bytes (16 dims of one
// position innermost), V codes as [4][D][16] (16 positions of one dim
// innermost): a warp of the attention that owns 32 positions (K) or 32 dims
// (V) then reads its codes as consecutive 16-byte pieces, and two blocks in
// a row are the 128 keys of one tile. The open block, and the one before it,
// are kept as bf16 rows in tail slot (b & 1).
#pragma once

#include "common.cuh"

namespace dfv {

constexpr int kBlk = 64;   // positions per scale

// Magnitudes from 2^40 on (and infinities, NaN) are not stored: they enter
// as zeros and are reported. A block whose largest magnitude is below 2^-40
// is stored as zeros. Scales then lie in [2^-47, 2^33], which leaves the
// softmax's combined exponents far inside the f32 range.
constexpr uint32_t kBigBits = 0x5380u;    // bf16 2^40
constexpr uint32_t kSmallBits = 0x2B80u;  // bf16 2^-40

__host__ __device__ constexpr int kv8_blocks(int capacity) { return (capacity + kBlk - 1) / kBlk; }

// Bytes from a head's first K (V) code to the piece of (position t of block
// b, piece j of 16 dims), and of (group g of 16 positions, dim c).
__device__ __forceinline__ int64_t kv8_k_piece(int64_t b, int t, int j, int d) {
  return b * kBlk * d + (j * kBlk + t) * 16;
}
__device__ __forceinline__ int64_t kv8_v_piece(int64_t b, int g, int c, int d) {
  return b * kBlk * d + (static_cast<int64_t>(g) * d + c) * 16;
}

inline bool kv8_cache_ok(const dfv_kv8_cache* c) {
  return c && c->n_kv_heads >= 1 && c->n_kv_heads <= 65535 && c->capacity >= 1 &&
         c->capacity <= (1 << 30) && c->state && c->k_codes && c->v_codes && c->k_scale &&
         c->v_scale && c->k_tail && c->v_tail && aligned(c->state, 4) && aligned(c->k_codes, 128) &&
         aligned(c->v_codes, 128) && aligned(c->k_scale, 4) && aligned(c->v_scale, 4) &&
         aligned(c->k_tail, 32) && aligned(c->v_tail, 32);   // read 32 bytes at a time
}

inline bool kv8_dim_ok(int d) { return d == 64 || d == 128 || d == 256; }

}  // namespace dfv
