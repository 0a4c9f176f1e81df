// The 4-bit cache of keys and values.
//
// For each token, kv head and group of G channels: codes c = 0..15 and two fp16 numbers
// s, m; the value is m + s * c.  With x the group's 16-bit values clamped to +-65504,
//   m = fp16(min x), s = fp16((max x - min x) / 15), c = clamp(rint((x - m) / s), 0, 15)
// (c = 0 where s = 0).
//
// A page holds `page` tokens of every kv head: [kv head][block of 32 tokens], each block
// contiguous, block_bytes(D, D / G) bytes: [K codes 16 D | V codes 16 D | K params | V params].
// Codes lie as the matrix instruction 16x16x32 takes them, so that a wave loads operands
// straight into registers:
//   K codes  32-bit words [tile 2][lane 64][D/32]: word j of lane l is token 16 tile + l%16,
//            channels 32 j + 8 (l/16) + e, e = 0..7 (rows of K: the product K q^T)
//   V codes  32-bit words [D/64][lane 64][4]: word w of lane l at h is channel
//            64 h + 16 w + l%16, tokens slot_token(l/16, e), e = 0..7 (rows of V^T)
//   in both, e sits at nibble nib_pos(e), as in the repacked weights
//   params   fp16 [D/G][s, m][32]; token t at token_slot(t)
// The order of the tokens in V's words is that in which K q^T leaves its two tiles in a
// lane's registers (4 (l/16) + i of tile 0, then of tile 1), so the probabilities go to the
// second product without moving between lanes; s and m of a lane's tokens are 16 bytes.
#pragma once
#include "internal.h"
#include "rows16.h"

namespace w4a16 {

__host__ __device__ constexpr int kv4_block_bytes(int D, int groups) {
  return 32 * D + 256 * groups;
}
__host__ __device__ constexpr int kv4_slot_token(int g, int e) {
  return e < 4 ? 4 * g + e : 16 + 4 * g + e - 4;
}
__host__ __device__ constexpr int kv4_token_slot(int t) {
  return 8 * ((t >> 2) & 3) + 4 * (t >> 4) + (t & 3);
}

// The new tokens of sequence b: rows first .. first + n - 1, the last at position len - 1.
// What the device arrays say is brought into range here, whatever they hold.
struct Kv4Seq {
  int first, n, len;
};
__device__ __forceinline__ Kv4Seq kv4_seq(const int* rows, const int* lens, int b, int tokens,
                                          int max_new) {
  Kv4Seq s;
  int lo = rows[b], hi = rows[b + 1];
  lo = lo < 0 ? 0 : lo > tokens ? tokens : lo;
  hi = hi < lo ? lo : hi > tokens ? tokens : hi;
  s.first = lo;
  s.n = hi - lo < max_new ? hi - lo : max_new;
  s.len = lens[b] < 0 ? 0 : lens[b];
  // tokens past max_new are left alone: the ones served are the first of the sequence
  s.len -= (hi - lo) - s.n;
  return s;
}
// Page of block `blk` (32 tokens) of sequence b, -1 if the table has none for it.
__device__ __forceinline__ int kv4_page(const int* table, int b, int blk, int page_blocks, int W,
                                        int pages) {
  const int at = blk / page_blocks;
  if (blk < 0 || at >= W) return -1;
  const int p = table[(size_t)b * W + at];
  return p >= 0 && p < pages ? p : -1;
}

}  // namespace w4a16
