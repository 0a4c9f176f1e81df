// What the attention kernels over the 4-bit cache share: operands made from codes, and which
// workgroup does which part (kv4_attention.hip, kv4_prefill.hip, kv4_tree_wide.hip).
#pragma once
#include "kv4.h"

namespace w4a16 {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kKv4Lazy = 7.f;       // how far a logit may exceed a column's reference
constexpr float kKv4Lift = 8.f;       // p is held times 2^8
// Reference of a column that has seen nothing, the lowest number: no finite logit is below it.
constexpr float kKv4None = -0x1.fffffep127f;

__device__ __forceinline__ half2v as_half2(uint32_t w) { return __builtin_bit_cast(half2v, w); }
__device__ __forceinline__ uint32_t as_word(half2v h) { return __builtin_bit_cast(uint32_t, h); }

// the eight codes of a word as fp16 subnormals, channels 2, 3, 6, 7 times 16
__device__ __forceinline__ half8v codes_subnormal(uint32_t w) {
  const uint32_t v = w >> 8;
  return __builtin_bit_cast(half8v, u32x4v{w & 0x000F000Fu, w & 0x00F000F0u, v & 0x000F000Fu,
                                           v & 0x00F000F0u});
}
// (w & mask) | bits in one instruction, which the compiler splits in two; its result goes to
// vector instructions only
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t bits) {
  uint32_t r;
  asm("v_and_or_b32 %0, %1, %2, %3" : "=v"(r) : "v"(w), "s"(mask), "v"(bits));
  return r;
}
// the eight values m + s c of a word; s and m of its tokens in the same order
__device__ __forceinline__ half8v values(uint32_t w, const u32x4v& s, const u32x4v& m) {
  const uint32_t v = w >> 8;
  const half2v one = {(_Float16)-1024.f, (_Float16)-1024.f};
  const half2v up = {(_Float16)0.0625f, (_Float16)0.0625f};
  const half2v off = {(_Float16)-64.f, (_Float16)-64.f};
  const uint32_t low = 0x000F000Fu, high = 0x00F000F0u, magic = 0x64006400u;
  const half2v c0 = as_half2(and_or(w, low, magic)) + one;
  const half2v c1 = __builtin_elementwise_fma(as_half2(and_or(w, high, magic)), up, off);
  const half2v c2 = as_half2(and_or(v, low, magic)) + one;
  const half2v c3 = __builtin_elementwise_fma(as_half2(and_or(v, high, magic)), up, off);
  // A group whose s was rounded up can pass 65504; NaN stays NaN.  (The saturating mode of
  // fp16 results would do the first for nothing, but in that mode the matrix instructions
  // turn a NaN sum into 0.)
  const half2v most = {(_Float16)65504.f, (_Float16)65504.f};
  auto value = [&](half2v c, uint32_t sw, uint32_t mw) {
    return as_word(__builtin_elementwise_minimum(
        __builtin_elementwise_fma(c, as_half2(sw), as_half2(mw)), most));
  };
  return __builtin_bit_cast(half8v, u32x4v{value(c0, s[0], m[0]), value(c1, s[1], m[1]),
                                           value(c2, s[2], m[2]), value(c3, s[3], m[3])});
}

// The exponent d by which a query row of largest magnitude `top` is scaled into fp16's top
// binade.
__device__ __forceinline__ int query_exponent(float top) {
  const int d = 15 - ((int)(__float_as_uint(top) >> 23) - 127);
  return top == 0.f ? 0 : d < -112 ? -112 : d > 100 ? 100 : d;
}

// A workgroup's part: one tile of a sequence's columns for one kv head, and blocks
// [blk0, blk1) of the cache.
struct Kv4Place {
  Kv4Seq s;
  int b, head, tile;
  int chunk, chunks;   // which of the tile's chunks, and how many there are
  int slot0;           // workspace slot of the tile's first chunk
  int span;            // blocks that a tile of the sequence can see
};

// TREE: the new tokens are the nodes of a tree.  Each sees the tokens held before the tree
// (those in the window of its position, which is as deep as it is) and the nodes that its bits
// name, so every tile of a sequence has the same blocks.
//
// Blocks that a tile of TC columns of the sequence can see, at least 1.
template <int TC, bool TREE>
__device__ __forceinline__ int kv4_span(const Kv4AttendArgs& p, const Kv4Seq& s, int ratio) {
  int span = (s.len >> 5) + ((s.len & 31) != 0);
  const int most = p.width * (p.page / 32);
  span = span < most ? span : most;
  if (p.window > 0) {
    const long long w = ((long long)p.window + (TREE ? s.n : TC / ratio + 1)) / 32 + 2;
    span = span < w ? span : (int)w;
  }
  return span < 1 ? 1 : span;
}

// A launch without chunks can have more workgroups than one dimension of a grid takes (2^32
// threads: 1024 sequences of 8 kv heads of which one brings 32768 tokens): rows of 2^20.
constexpr unsigned kKv4GridRow = 1u << 20;
inline dim3 kv4_grid(unsigned n) {
  return n <= kKv4GridRow ? dim3(n) : dim3(kKv4GridRow, (n + kKv4GridRow - 1) / kKv4GridRow);
}

// Where a launch without chunks starts: workgroups go round robin to the 8 XCDs, each with
// an L2 of its own, so that the tiles of one (sequence, kv head) take one residue of 8 and
// share the cached bytes.
__device__ __forceinline__ bool kv4_place_whole(const Kv4AttendArgs& p, Kv4Place& w) {
  const unsigned id = blockIdx.x + blockIdx.y * kKv4GridRow;
  const unsigned unit = id % 8 + 8 * (id / 8 / p.col_tiles);
  if (unit >= (unsigned)p.heads * p.batch) return false;
  // the last tiles see the most: they start first
  w.tile = p.col_tiles - 1 - (int)(id / 8 % p.col_tiles);
  w.head = unit % p.heads;
  w.b = unit / p.heads;
  w.s = kv4_seq(p.rows, p.lens, w.b, p.tokens, p.max_new);
  w.chunk = 0;
  w.chunks = 1;
  w.slot0 = 0;
  w.span = 1;
  return true;
}

// Sums of x over the lanes up to each one.
__device__ __forceinline__ uint32_t wave_sums(uint32_t x) {
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x111, 0xF, 0xF, false);  // row_shr 1
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x112, 0xF, 0xF, false);  // row_shr 2
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x114, 0xF, 0xF, false);  // row_shr 4
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x118, 0xF, 0xF, false);  // row_shr 8
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x142, 0xA, 0xF, false);  // row_bcast 15
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x143, 0xC, 0xF, false);  // row_bcast 31
  return x;
}

// The lengths are known on the device only, and sequences of one batch differ widely, so
// every workgroup works out the same division from them: the blocks of all tiles in a row,
// in the order (sequence, kv head, tile), cut into equal stripes, one per workgroup.  A
// stripe's first and last tile may be shared with its neighbours.
// To begin, join and hand over a tile costs a workgroup about 4 us, as much as 16 blocks (tiles of
// 128 columns: as 4), so a tile counts as `lead` blocks more than it has.  Where stripes of the least size
// p.chunk are enough for all, every tile is rounded up to whole stripes instead, and no
// workgroup has two.
template <int TC, bool TREE>
struct Kv4Stripes {
  static constexpr int kLead = TC >= 128 ? 4 : 16;
  uint32_t total, stripe;
  int lead;

  struct Lane {          // a lane's sequence of a group of 64
    Kv4Seq s;
    int span, tiles;
    uint32_t size, upto; // what its tiles count together, and those of the lanes up to it
  };
  __device__ __forceinline__ uint32_t tile_size(int span) const {
    return lead ? span + lead : (span + stripe - 1) / stripe * stripe;
  }
  __device__ __forceinline__ Lane fetch(const Kv4AttendArgs& p, int b0, int ratio) const {
    const int b = b0 + (threadIdx.x & 63);
    Lane x{{0, 0, 0}, 1, 0, 0u, 0u};
    if (b < p.batch) {
      x.s = kv4_seq(p.rows, p.lens, b, p.tokens, p.max_new);
      x.span = kv4_span<TC, TREE>(p, x.s, ratio);
      x.tiles = (int)(((long long)x.s.n * ratio + TC - 1) / TC);
      // past 2^29 blocks in all a sequence's tiles count as one block each: the last
      // stripe of a tile takes what is left of it
      if ((uint64_t)x.tiles * p.heads * x.span > (1u << 29) / (unsigned)p.batch) x.span = 1;
    }
    resize(p, x);
    return x;
  }
  __device__ __forceinline__ void resize(const Kv4AttendArgs& p, Lane& x) const {
    x.size = (uint32_t)x.tiles * p.heads * tile_size(x.span);
    x.upto = wave_sums(x.size);
  }
  // n: how many stripes.  Returns the lanes of the first 64 sequences.
  __device__ __forceinline__ Lane init(const Kv4AttendArgs& p, int ratio, uint32_t n) {
    lead = 0;
    stripe = p.chunk;
    total = 0;
    Lane x;
    for (int b0 = 0; b0 < p.batch; b0 += 64) {
      x = fetch(p, b0, ratio);
      total += __builtin_amdgcn_readlane(x.upto, 63);
    }
    if (total <= stripe * n) return x;
    lead = kLead;
    total = 0;
    for (int b0 = 0; b0 < p.batch; b0 += 64) {
      if (p.batch > 64) x = fetch(p, b0, ratio);
      else resize(p, x);
      total += __builtin_amdgcn_readlane(x.upto, 63);
    }
    stripe = (total + n - 1) / n;
    return x;
  }
  // The tile at place `at` (< total); u0: where it starts, x: lanes of the first 64 sequences
  __device__ __forceinline__ void find(const Kv4AttendArgs& p, uint32_t at, int ratio, Lane& x,
                                       Kv4Seq& seq, int& b, int& head, int& tile, int& tile_span,
                                       uint32_t& u0) const {
    uint32_t base = 0;
    int b0 = 0;
    uint64_t hit;
    for (;;) {
      if (p.batch > 64) x = fetch(p, b0, ratio);
      hit = __ballot(at - base < x.upto && at - base >= x.upto - x.size);
      if (hit) break;
      base += __builtin_amdgcn_readlane(x.upto, 63);
      b0 += 64;
    }
    const int l = __builtin_ctzll(hit);
    b = b0 + l;
    seq.first = __builtin_amdgcn_readlane(x.s.first, l);
    seq.n = __builtin_amdgcn_readlane(x.s.n, l);
    seq.len = __builtin_amdgcn_readlane(x.s.len, l);
    tile_span = __builtin_amdgcn_readlane(x.span, l);
    const int nt = __builtin_amdgcn_readlane(x.tiles, l);
    base += __builtin_amdgcn_readlane(x.upto - x.size, l);
    const uint32_t size = tile_size(tile_span), t = (at - base) / size;
    u0 = base + t * size;
    tile = t % nt;
    head = t / nt;
  }
};

// A launch with chunks: the lengths are known on the device only, and sequences of one batch
// differ widely, so every wave works out the same division from them: all tiles' blocks
// together, cut into about p.target equal chunks.  Slot numbers run over (sequence, kv head,
// tile, chunk).  `id` is a slot, or with BY_TILE the number of a tile (its chunk is then 0).
template <int TC, bool BY_TILE>
__device__ __forceinline__ bool kv4_place_chunk(const Kv4AttendArgs& p, int id, Kv4Place& w) {
  const int lane = threadIdx.x & 63, ratio = p.q_heads / p.heads;
  Kv4Seq s{};
  int span = 0, tiles = 0;
  auto fetch = [&](int b) {
    tiles = 0;
    span = 1;
    if (b < p.batch) {
      s = kv4_seq(p.rows, p.lens, b, p.tokens, p.max_new);
      span = kv4_span<TC, false>(p, s, ratio);
      tiles = (int)(((long long)s.n * ratio + TC - 1) / TC);
    }
  };
  float total = 0.f;
  for (int b0 = 0; b0 < p.batch; b0 += 64) {
    fetch(b0 + lane);
    total += (float)tiles * (float)span;
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) total += __shfl_xor(total, off);
  total *= (float)p.heads;
  const float even = __builtin_ceilf(total / (float)p.target);
  const int least = even > 1e9f ? 1000000000 : (int)even > p.chunk ? (int)even : p.chunk;
  int slot = 0, tile0 = 0;
  for (int b0 = 0; b0 < p.batch; b0 += 64) {
    if (p.batch > 64) fetch(b0 + lane);
    int size = (span + p.chunks - 1) / p.chunks;  // p.chunks: the most a tile may have
    size = size > least ? size : least;
    const int n = (span + size - 1) / size;
    long long want = (long long)p.heads * tiles * n;
    const int mine = want > (1 << 24) ? 1 << 24 : (int)want;
    want = (long long)p.heads * tiles;
    const int mine_t = want > (1 << 24) ? 1 << 24 : (int)want;
    int upto = mine, upto_t = mine_t;  // sums over the lanes up to this one
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int a = __shfl_up(upto, off), t = __shfl_up(upto_t, off);
      if (lane >= off) {
        upto += a;
        upto_t += t;
      }
    }
    const int from = BY_TILE ? tile0 + upto_t - mine_t : slot + upto - mine;
    const uint64_t hit = __ballot(id >= from && id < from + (BY_TILE ? mine_t : mine));
    if (hit) {
      const int l = __builtin_ctzll(hit);
      w.b = b0 + l;
      w.s.first = __builtin_amdgcn_readlane(s.first, l);
      w.s.n = __builtin_amdgcn_readlane(s.n, l);
      w.s.len = __builtin_amdgcn_readlane(s.len, l);
      w.span = __builtin_amdgcn_readlane(span, l);
      w.chunks = __builtin_amdgcn_readlane(n, l);
      const int nt = __builtin_amdgcn_readlane(tiles, l);
      const int s0 = slot + __builtin_amdgcn_readlane(upto - mine, l);
      const int t0 = tile0 + __builtin_amdgcn_readlane(upto_t - mine_t, l);
      const int t = BY_TILE ? id - t0 : (id - s0) / w.chunks;
      w.chunk = BY_TILE ? 0 : (id - s0) % w.chunks;
      w.tile = t % nt;
      w.head = t / nt;
      w.slot0 = s0 + t * w.chunks;
      // rows that overlap can ask for more than the launch has: such tiles are left out whole
      return w.slot0 + w.chunks <= p.slots && t0 + t < p.tiles;
    }
    slot += __builtin_amdgcn_readlane(upto, 63);
    tile0 += __builtin_amdgcn_readlane(upto_t, 63);
    if (slot > id && !BY_TILE) return false;
    if (tile0 > p.tiles || slot > p.slots) return false;
  }
  return false;
}

// Tokens that the columns of a tile can see, and the workgroup's blocks of them: blocks
// [from, to) counted from the tile's first, to < 0: all that are left.
struct Kv4Range {
  int i0, i1;          // first and last new token of the tile
  int from;            // position of the sequence's first new token
  int lo, hi;          // tokens that any column can see
  int blk0, blk1;
};
template <int TC, bool TREE>
__device__ __forceinline__ Kv4Range kv4_range(const Kv4AttendArgs& p, const Kv4Seq& s, int tile,
                                              int ratio, int from, int to) {
  Kv4Range r;
  r.i0 = tile * TC / ratio;
  const int end = (tile * TC + TC - 1) / ratio;
  r.i1 = end < s.n - 1 ? end : s.n - 1;
  r.from = s.len - s.n;
  r.hi = r.from + (TREE ? s.n : r.i1 + 1);
  const long long lo = p.window > 0 ? (long long)r.from + (TREE ? 0 : r.i0) - p.window + 1 : 0;
  r.lo = lo < 0 ? 0 : (int)lo;
  const int most = p.width * (p.page / 32);
  int stop = r.hi <= 0 ? 0 : (r.hi >> 5) + ((r.hi & 31) != 0);
  stop = stop < most ? stop : most;
  r.blk0 = r.lo / 32 + from;
  r.blk1 = to < 0 || r.lo / 32 + to > stop ? stop : r.lo / 32 + to;
  return r;
}

// TREE: the first token that node `row` of the sequence sees of those before the tree (their
// number is `from`; node r.from + j of the cache is node j).
__device__ __forceinline__ int kv4_tree_first(const Kv4AttendArgs& p, const Kv4Seq& s, int row) {
  if (p.window <= 0) return 0;
  int d = p.depth[row];
  d = d < 0 ? 0 : d > s.n - 1 ? s.n - 1 : d;
  const long long first = (long long)(s.len - s.n) + d - p.window + 1;
  return first < 0 ? 0 : (int)first;
}
// TREE: a token that some columns of a tile see and others do not may hold NaN (a rejected branch
// may not spoil the accepted one), and the matrix instruction makes 0 x NaN of it for the others.
// A NaN is in s or m, and makes a whole group of the token's channels NaN: so s and m are cleared
// and the columns that see the token get the group's NaN by themselves.
//
// Whether a word of two fp16 numbers may hold a NaN (infinities do no harm in being looked at).
__device__ __forceinline__ uint32_t maybe_nan(uint32_t w) {
  return ((w & 0x7C007C00u) + 0x04000400u) & 0x80008000u;
}
// The tokens, of the eight of lane group g, whose s or m is NaN, a bit each; their s and m become 0.
__device__ __forceinline__ uint32_t clear_nan_tokens(u32x4v& s, u32x4v& m, int g) {
  uint32_t bits = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int up = 16 * (e & 1);
    const uint32_t a = s[e >> 1] >> up & 0x7FFFu, b = m[e >> 1] >> up & 0x7FFFu;
    if (a > 0x7C00u || b > 0x7C00u) {
      bits |= 1u << e;
      s[e >> 1] &= ~(0xFFFFu << up);
      m[e >> 1] &= ~(0xFFFFu << up);
    }
  }
  // kv4_slot_token of each, with nothing that a compiler could keep for the next block
  return (bits & 0x0Fu) << (4 * g) | (bits & 0xF0u) << (12 + 4 * g);
}

// TREE: which of the 32 tokens from t0 on node `row` sees, a bit each.
__device__ __forceinline__ uint32_t kv4_tree_sees(const Kv4AttendArgs& p, const Kv4Seq& s, int row,
                                                  int first, int t0) {
  const int rel = t0 - (s.len - s.n);  // the node at t0
  uint32_t sees = 0;
  if (rel < 0) {
    sees = rel <= -32 ? 0xFFFFFFFFu : (1u << -rel) - 1u;
    if (first > t0) sees = first - t0 >= 32 ? 0u : sees & (0xFFFFFFFFu << (first - t0));
  }
  if (rel > -32) {
    const uint32_t* bits = p.mask + (size_t)row * p.words;
    uint32_t nodes;
    if (rel < 0) {
      nodes = bits[0] << -rel;
    } else {
      const int at = rel >> 5;
      const uint32_t a = at < p.words ? bits[at] : 0u;
      const uint32_t b = at + 1 < p.words ? bits[at + 1] : 0u;
      nodes = (uint32_t)(((uint64_t)b << 32 | a) >> (rel & 31));
    }
    const int left = s.n - rel;  // nodes from t0 on
    sees |= left >= 32 ? nodes : left <= 0 ? 0u : nodes & ((1u << left) - 1u);
  }
  return sees;
}

}  // namespace w4a16
