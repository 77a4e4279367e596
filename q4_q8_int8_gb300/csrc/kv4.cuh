// The 4-bit key/value cache's layout.
//
// A cache is [pages][kv_heads][page_size / 16] tiles of 18 D bytes, a tile
// being 16 tokens of one head:
//   8 D bytes  key codes      D bytes  key scales (float16)
//   8 D bytes  value codes    D bytes  value scales
// A value is (code - 8) * scale with one scale per 32 values of a token; the
// scale has at most 8 significant bits and is at most 8160, so that every
// value is a float16 (|code - 8| <= 8 adds three bits).
//
// The codes lie as the A operand of a 16 x 8 x 16 matrix product wants them:
// word [i / 4][lane][i % 4] holds lane's eight values of a 16 x 16 block, i the
// block of 16 dimensions.  With lane = 4 r + c, the block is tokens x
// dimensions for keys (r, r + 8 the tokens, 2 c, 2 c + 1 and those + 8 the
// dimensions) and dimensions x tokens for values.  A byte is dimensions x (low
// nibble) and x + 8 (high) of one token, so that a token can be written without
// reading its neighbours; masking a word with 0x000F000F or 0x00F000F0, and
// the same after a shift by 8, leaves the operand's four registers.
//   keys    token t, dimension 16 i + x (+ 8), x < 8:
//           lane 4 (t % 8) + x / 2, byte t / 8 + 2 (x % 2)
//   values  lane 4 x + (t % 8) / 2, byte t / 8 + 2 (t % 2)
// Scales follow the lanes: keys [t % 8][t / 8][block], values
// [(t % 8) / 2][block][t / 8][t % 2].
#pragma once
#include <stdint.h>

namespace mmq {
namespace kv4 {

constexpr int kTokens = 16;        // of a tile
constexpr float kTop = 8160.f;     // largest scale

__host__ __device__ constexpr int tile_bytes(int D) { return 18 * D; }
__host__ __device__ constexpr int key_scales(int D) { return 8 * D; }
__host__ __device__ constexpr int value_codes(int D) { return 9 * D; }
__host__ __device__ constexpr int value_scales(int D) { return 17 * D; }

// Byte offsets in a tile: token t < 16, block i of 16 dimensions, x < 8.
__host__ __device__ constexpr int key_byte(int t, int i, int x) {
    return (i / 4) * 512 + (t % 8) * 64 + (x / 2) * 16 + (i % 4) * 4 + 2 * (x % 2) + t / 8;
}
template <int D>
__host__ __device__ constexpr int value_byte(int t, int i, int x) {
    return value_codes(D) + (i / 4) * 512 + x * 64 + ((t % 8) / 2) * 16 + (i % 4) * 4 + 2 * (t % 2) + t / 8;
}
template <int D>
__host__ __device__ constexpr int key_scale(int t, int block) {
    return key_scales(D) + 2 * (((t % 8) * 2 + t / 8) * (D / 32) + block);
}
template <int D>
__host__ __device__ constexpr int value_scale(int t, int block) {
    return value_scales(D) + 2 * ((((t % 8) / 2) * (D / 32) + block) * 4 + (t / 8) * 2 + t % 2);
}

}  // namespace kv4
}  // namespace mmq
