// kv4.cuh -- the 4-bit form of cached keys and values, and where its bytes are.
//
// 32 neighbouring values of a head share one scale s = bf16(max|x| / 7); a value's code is
// x / s rounded to the nearest integer (ties to even) within -7 .. 7, held as the nibble
// code + 8.  4.5 bits a value.  The scale is rounded before the codes are taken, so code * s
// is the value that is read back, and bf16 keeps the scale's range that of the inputs.  A
// group that holds an infinity or a NaN gets a NaN scale: it reads back as NaN, never as
// plausible numbers.  (Integers rather than e2m1: same bits and error on normal data, and an
// integer nibble becomes a bf16 with one AND-OR, 0x4300 | u being 128 + u.)
//
// A page holds `page` tokens (a multiple of 16) of one K/V head.  The decode kernel multiplies
// 16 tokens at a time on m16n8k16 fragments (lane 4 g + t: row g, columns of t), and the bytes
// lie as its lanes load them:
//   K codes   token rows of d / 2 bytes: the 32-bit word t * (d / 32) + c holds the eight
//             values 32 c + 8 t + 0 .. 7, so that lane (g, t) reads its words of token g as one
//             16-byte load (d = 128).
//   V codes   tiles of 16 tokens (8 d bytes): token k's four values 32 c + 4 g + 0 .. 3 are the
//             16-bit word ((((k / 8) * 8 + g) * 4 + (k % 8) / 2) * 2 + k % 2) * (d / 32) + c
//             of the tile: lane (g, t) reads tokens 2t, 2t + 1 and then 2t + 8, 2t + 9 as one
//             load each, without bank conflicts (token rows conflict four ways).
//   K scales  [token][d / 32]
//   V scales  [token / 2][d / 32][token % 2]: a lane's two tokens' scales as one packed pair.
#pragma once

#include <cstdint>

namespace fa {

constexpr int kTileTokens = 16;
constexpr int kMaxTokens = 0x7fffff00;  // of a request: token numbers, and a tile's more, stay within int

// Byte offset of word (t, c) in a K token row.
__host__ __device__ constexpr int kv4_k_word(int d, int t, int c) { return 4 * (t * (d / 32) + c); }
// Byte offset of 16-bit word (g, c) of token `slot` in a page's V codes.
__host__ __device__ constexpr size_t kv4_v_half(int d, int slot, int g, int c) {
    const int k = slot % 16;
    return static_cast<size_t>(slot / 16) * 8 * d +
           2 * (((((k / 8) * 8 + g) * 4 + (k % 8) / 2) * 2 + k % 2) * (d / 32) + c);
}
// Index of token `slot`'s scale of group c in a page's V scales.
__host__ __device__ constexpr size_t kv4_v_scale(int d, int slot, int c) {
    return static_cast<size_t>(slot / 2) * 2 * (d / 32) + 2 * c + slot % 2;
}

}  // namespace fa
