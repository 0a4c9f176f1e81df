// Attention of new tokens over the 4-bit cache (kv4.h has the format).
//
// The columns of a kv head's problem are (new token i, query head of the group): column
// i * ratio + h.  A tile of 16 columns is one operand of the matrix instruction and stays
// in registers; keys and values stream past it in blocks of 32 tokens, with the running
// maximum and sum of the softmax per column, so every cached byte is read once per tile.
//
//   K q^T   A = codes of K, B = q.  A code c masked out of its word is the fp16 subnormal
//           c * 2^-24 (16 c * 2^-24 for every second pair: those channels of q are divided
//           by 16), which the matrix instruction multiplies exactly: no conversion.  Per
//           group of channels, logit = s_t * (sum c q) + m_t * (sum q), in fp32.
//           q is first scaled per row by a power of two into fp16's top binade, exact for
//           every value within 2^-25 of the row's largest, so bf16 rows take the same path.
//   softmax in powers of two.  The reference of a column moves only when a logit exceeds it
//           by 7, then the sums so far are scaled; p = 2^(x - ref + 8) <= 2^15 is summed in fp32.
//           For the second product it is rounded to fp16 (2^-11: an eighth of bf16's own
//           step), and for fp16 rows split into hi + lo, 22 bits, so that V's rounding is the
//           only one beside that of the result: 1.65 to 1.33 times the error of rounding
//           alone, at no more (tiles of 8) or 8 more matrix instructions a block.
//   V^T p^T A = V = m_t + s_t c in fp16 (one rounding of the exact value, 2^-11), B = p, which
//           is where K q^T left it.  Values past 65504 (a group whose s was rounded up)
//           become 65504.
//
// A token is seen by a column if its position is at most the column's own, more than the
// column's less the window (window > 0), and its page is in the table.  Blocks that are
// not seen whole by every column take the masked path, which also clears s and m of
// the tokens that no column sees: what a page holds there may be anything.
// A column that sees nothing gives 0 and a log-sum of -infinity.
//
// TREE: the new tokens are the nodes of a drafted tree, and what a column sees of the last
// blocks is 32 bits that its node's mask gives for them; everything before the tree is as above.
// In those blocks a NaN stays with the columns that see its token (clear_nan_tokens).
//
// The blocks of all tiles are cut into equal stripes, one for each of the workgroups that
// the card holds at once; the sums of a tile that stripes share are joined in order.
//
// Bound: loads in flight for large caches, latency for small ones.  48 requests to 8192 tokens,
// 64 query heads on 8 of 128 channels, groups of 64: 234 MB in 59 us, 4.0 TB/s (a plain read:
// 6.3; 50 us with what the 256 MiB cache keeps of an earlier pass over the same bytes); contexts
// of 131072 and 16538 tokens, groups of 32: 189 MB in 66 us, 2.9 TB/s (51 us); 3999 tokens of 32
// heads: 17 MB in 13.1 us, of which 0.7 us find the part, 1.5 us load q, 2.4 us stream 2 blocks
// a wave, 1.8 us hand the sums over and 3 us join them.  512 stripes, two to a compute unit,
// which is what the registers allow: over the same bytes again 256 / 512 / 768 / 1024 take 59 /
// 50 / 60 / 57 us on the first and 58 / 51 / 76 / 87 on the second.  Equal stripes without the
// `lead` of a tile: 75 us on the first.  Tiles of 8 columns against 16 where both fit: 50
// against 57 us on the first.
// Registers: 193 to 227 with 128 channels, two waves to a SIMD.  With groups of 32 the two
// blocks and their s and m do not fit into 256: 17 are spilled in tiles of 8, 41 to 45 in tiles
// of 16.  TREE: 163 to 238, with groups of 32 29 to 48 spilled; 26 nodes and 2000 tokens of 32 heads
// (two tiles a head) 16.5 us.  56 to 84 scalar registers of the division into stripes lie in vector registers.
#include "kv4_attend.h"

namespace w4a16 {

namespace {

constexpr int AW = 4;              // waves of a workgroup, which share its blocks

// Columns of a sequence above which tiles have 128 (kv4_prefill.hip).  16 against 128, 64 query
// heads on 8, contexts of 8 x 8192 / 32 x 2048 / 1 x 32768 tokens, us:
//   32 columns 32 / 32 / 36 against 68 / 65 / 39;   96: 51 / 61 / 53 against 67 / 73 / 47
//   128: 63 / 71 / 61 against 71 / 73 / 50;         256: 112 / 107 / 104 against 105 / 97 / 76
constexpr int kPrefillColumns = 128;

// One block of 32 tokens of one kv head in a wave's registers.
// With tiles of 8 columns a lane needs K's s and m for 4 tokens only (those of tile r / 8).
template <int D, int NG, int TC>
struct Block {
  typedef uint32_t kparam __attribute__((ext_vector_type(TC / 4)));
  uint32_t k[2][D / 32];
  u32x4v v[D / 64];
  kparam ks[NG], km[NG];
  u32x4v vs[NG], vm[NG];

  __device__ __forceinline__ void load(const char* base, int lane) {
    const int g = lane >> 4;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if constexpr (D == 128) {
        const u32x4v x = *reinterpret_cast<const u32x4v*>(base + (t * 64 + lane) * 16);
#pragma unroll
        for (int j = 0; j < 4; ++j) k[t][j] = x[j];
      } else {
        const u32x2v x = *reinterpret_cast<const u32x2v*>(base + (t * 64 + lane) * 8);
        k[t][0] = x[0];
        k[t][1] = x[1];
      }
    }
#pragma unroll
    for (int h = 0; h < D / 64; ++h)
      v[h] = *reinterpret_cast<const u32x4v*>(base + 16 * D + (h * 64 + lane) * 16);
    const char* par = base + 32 * D + 16 * g;
    const char* kpar = par + (TC == 8 ? lane & 8 : 0);
#pragma unroll
    for (int q = 0; q < NG; ++q) {
      ks[q] = *reinterpret_cast<const kparam*>(kpar + 128 * q);
      km[q] = *reinterpret_cast<const kparam*>(kpar + 128 * q + 64);
      vs[q] = *reinterpret_cast<const u32x4v*>(par + 128 * (NG + q));
      vm[q] = *reinterpret_cast<const u32x4v*>(par + 128 * (NG + q) + 64);
    }
  }
};

template <class V>
__device__ __forceinline__ float half_at(const V& v, int e) {
  return e & 1 ? hi16<false>(v[e >> 1]) : lo16<false>(v[e >> 1]);
}
// the value of lane l ^ 8 (lanes of 16 turned by 8)
__device__ __forceinline__ uint32_t swap8(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x128, 0xF, 0xF, false);
}

// TC: columns of a tile, 16, or 8 where a sequence has no more than 8.  With 8, columns 8..15
// of the matrix instructions serve the same columns again: K q^T leaves tile 0's tokens in
// lanes r < 8 and tile 1's in the others, so each logit is worked on once, and V^T p^T
// takes p's upper part from lanes r < 8 and its lower part (fp16 rows) from the others.
template <int D, int NG, int TC, bool BF, bool TREE>
__global__ __launch_bounds__(64 * AW, 2) void kv4_attend_kernel(Kv4AttendArgs p) {
  constexpr int J = D / 32, JG = J / NG, NT = D / 16;
  constexpr int E = TC / 2;       // logits of a lane in a block
  __shared__ f32x4 red_o[AW][NT][64];
  __shared__ float red_ml[8][8][2];  // [wave][column], or [part][column] of the last join
  __shared__ int arrived;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int r = lane & 15, g = lane >> 4;
  const int ratio = p.q_heads / p.heads;
  Kv4Stripes<TC, TREE> stripes;
  typename Kv4Stripes<TC, TREE>::Lane lanes;
  uint32_t pos = 0, stop = 1;
  if (p.slots) {
    lanes = stripes.init(p, ratio, gridDim.x);
    pos = blockIdx.x * stripes.stripe;
    stop = pos + stripes.stripe < stripes.total ? pos + stripes.stripe : stripes.total;
  }
  for (bool again = false; pos < stop; again = true) {
  Kv4Seq seq;
  int b, head, tile, span = 1;
  uint32_t u0 = 0, r0 = 0, r1 = 1;  // this stripe's part of the tile: blocks [r0, r1)
  if (p.slots) {
    // fetched again (from cache) for a further tile rather than held in registers
    if (again && p.batch <= 64) lanes = stripes.fetch(p, 0, ratio);
    stripes.find(p, pos, ratio, lanes, seq, b, head, tile, span, u0);
    u0 += stripes.lead;
    r0 = pos > u0 ? pos - u0 : 0;
    pos = u0 - stripes.lead + stripes.tile_size(span);
    if (stop <= u0) break;  // it has the lead of a tile only
    r1 = stop - u0 < (uint32_t)span ? stop - u0 : (uint32_t)span;
    if (r0 >= r1) continue;  // what rounds a tile up to whole stripes
  } else {
    Kv4Place w;
    if (!kv4_place_whole(p, w)) return;
    seq = w.s;
    b = w.b;
    head = w.head;
    tile = w.tile;
    pos = 1;
  }
  const Kv4Range rg =
      kv4_range<TC, TREE>(p, seq, tile, ratio, r0, r1 == (uint32_t)span ? -1 : (int)r1);
  if (rg.i0 >= seq.n) return;  // a tile past the sequence's last, in a launch without stripes
  const int rc = TC == 8 ? r & 7 : r;
  const int col = tile * TC + rc, ci = col / ratio;
  const bool live = ci < seq.n;
  const int qh = head * ratio + col % ratio;
  const int row = seq.first + (live ? ci : 0);
  // tokens seen: column [first, last], any column [lo, hi), every column [all_lo, all_hi)
  const int lo = rg.lo, hi = rg.hi;
  // (TREE: those before the tree; its own blocks always take the masked path)
  const int last = live ? rg.from + ci : -1;
  const int first = TREE ? kv4_tree_first(p, seq, row) : p.window > 0 ? last - p.window + 1 : 0;
  const int all_hi = TREE ? rg.from : rg.from + rg.i0 + 1;
  const int all_lo = p.window > 0 ? rg.from + (TREE ? seq.n - 1 : rg.i1) - p.window + 1 : 0;

  const int page_blocks = p.page / 32;
  const size_t page_bytes = (size_t)p.heads * page_blocks * kv4_block_bytes(D, NG);
  const char* head_base = p.cache + (size_t)head * page_blocks * kv4_block_bytes(D, NG);
  const int* table = p.table + (size_t)b * p.width;

  // A wave's blocks blk0 + wave, + AW, ...: the next block's loads are in flight while one is
  // worked on, and its page number is fetched one block earlier still, before those loads,
  // so that no wait for it waits for them.  Blocks without a page are passed over; a load
  // past the last block reads some block of the table.
  const int b1 = rg.blk1;
  int blk = rg.blk0 + wave;
  int entry = blk / page_blocks, off = blk - entry * page_blocks;
  auto look_up = [&]() { return table[entry < p.width ? entry : p.width - 1]; };
  auto valid = [&](int pg) { return pg >= 0 && pg < p.pages; };
  auto advance = [&]() {
    blk += AW;
    off += AW;
    while (off >= page_blocks) {
      off -= page_blocks;
      ++entry;
    }
  };
  auto base_of = [&](int pg, int o_) {
    pg = __builtin_amdgcn_readfirstlane(pg);
    return head_base + (size_t)(valid(pg) ? pg : 0) * page_bytes +
           (size_t)o_ * kv4_block_bytes(D, NG);
  };
  Block<D, NG, TC> kv0, kv1;
  const bool any = blk < b1;
  int pg0 = 0, pg1 = 0, blk0 = blk, blk1 = 0, off1 = 0;
  if (any) {
    pg0 = look_up();
    const int off0 = off;
    advance();
    pg1 = look_up();
    blk1 = blk;
    off1 = off;
    kv0.load(base_of(pg0, off0), lane);
  }

  // q, scaled, and its sums per group of channels (times 2^-24, the codes' unit)
  half8v qf[TC == 8 ? 2 : 1][J];
  float qsum[NG], cf, more;
  {
    float f[J][8], top = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const u32x4v x = *reinterpret_cast<const u32x4v*>(p.q + (size_t)row * p.ldq +
                                                        (size_t)qh * D + 32 * j + 8 * g);
      unpack8<BF>(x, f[j]);
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(f[j][e]));
    }
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    const int d = query_exponent(top);
    const float up = __builtin_ldexpf(1.f, d);
#pragma unroll
    for (int q = 0; q < NG; ++q) qsum[q] = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float h[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = f[j][e] * up;
        qsum[j / JG] += x;
        h[e] = e & 2 ? x * 0.0625f : x;
      }
      const u32x4v x = pack8<false>(h);
      if constexpr (TC == 8) {
        const u32x4v zero = {0u, 0u, 0u, 0u};
        qf[0][j] = __builtin_bit_cast(half8v, r < 8 ? x : zero);
        qf[1][j] = __builtin_bit_cast(half8v, r < 8 ? zero : x);
      } else {
        qf[0][j] = __builtin_bit_cast(half8v, x);
      }
    }
#pragma unroll
    for (int q = 0; q < NG; ++q) {
      qsum[q] += __shfl_xor(qsum[q], 16);
      qsum[q] += __shfl_xor(qsum[q], 32);
      qsum[q] *= 0x1p-24f;
    }
    // bf16 queries past 2^91 need more than fp32 has in one factor
    const int over = BF && d < -76 ? -76 - d : 0;
    cf = __builtin_ldexpf(p.scale * 1.4426950408889634f, 24 - d - over);
    more = __builtin_ldexpf(1.f, over);
  }
  const bool big = BF && __ballot(more != 1.f) != 0;

  f32x4 o[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) o[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  float ref = kKv4None, sum = 0.f;

  auto process = [&](Block<D, NG, TC>& kv, int blk) {
    const int t0 = blk * 32;
    // logits of the lane's tokens: kv4_slot_token(g, e), or with TC == 8 the four of tile r / 8
    float x[E];
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = 0.f;
#pragma unroll
    for (int t = 0; t < E / 4; ++t)
#pragma unroll
      for (int q = 0; q < NG; ++q) {
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = q * JG; j < (q + 1) * JG; ++j) {
          acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes_subnormal(kv.k[t][j]), qf[0][j], acc,
                                                       0, 0, 0);
          if constexpr (TC == 8)
            acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes_subnormal(kv.k[1][j]), qf[1][j],
                                                         acc, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = 4 * t + i;
          x[e] = __builtin_fmaf(half_at(kv.ks[q], e), acc[i],
                                __builtin_fmaf(half_at(kv.km[q], e), qsum[q], x[e]));
        }
      }
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] *= cf;
    if (big) {
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] *= more;
    }
    if (t0 < all_lo || t0 + 32 > all_hi) {
      uint32_t sees = 0, any = 0;  // TREE: tokens that the column, that any column sees
      if constexpr (TREE) {
        sees = any = live ? kv4_tree_sees(p, seq, row, first, t0) : 0u;
#pragma unroll
        for (int off = 1; off < TC; off <<= 1) any |= (uint32_t)__shfl_xor((int)any, off);
      }
      // (TREE: bits of the lane's tokens, kv4_slot_token, at places that all lanes have alike)
      const uint32_t mine = sees >> (TC == 8 ? 4 * g + 2 * (r & 8) : 4 * g), some = any >> (4 * g);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int t = TC == 8 ? 4 * g + e + 2 * (r & 8) : kv4_slot_token(g, e);
        if (TREE ? (mine >> kv4_slot_token(0, e) & 1u) == 0 : t0 + t < first || t0 + t > last)
          x[e] = -INFINITY;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int t = kv4_slot_token(g, e);
        if (TREE ? (some >> kv4_slot_token(0, e) & 1u) == 0 : t0 + t < lo || t0 + t >= hi) {
#pragma unroll
          for (int q = 0; q < NG; ++q) {
            const uint32_t keep = e & 1 ? 0x0000FFFFu : 0xFFFF0000u;
            kv.vs[q][e >> 1] &= keep;
            kv.vm[q][e >> 1] &= keep;
          }
        }
      }
      if constexpr (TREE) {
#pragma unroll
        for (int q = 0; q < NG; ++q) {
          uint32_t odd = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) odd |= maybe_nan(kv.vs[q][i]) | maybe_nan(kv.vm[q][i]);
          if (__ballot(odd != 0) == 0) continue;
          uint32_t bits = clear_nan_tokens(kv.vs[q], kv.vm[q], g);
          bits |= (uint32_t)__shfl_xor((int)bits, 16);
          bits |= (uint32_t)__shfl_xor((int)bits, 32);
          const float add = (sees & bits) != 0 ? NAN : 0.f;
#pragma unroll
          for (int t = q * NT / NG; t < (q + 1) * NT / NG; ++t) o[t] += add;
        }
      }
    }
    float top = x[0];
#pragma unroll
    for (int e = 1; e < E; ++e) top = fmaxf(top, x[e]);
    if (__ballot(top > ref + kKv4Lazy) != 0) {
      if constexpr (TC == 8) top = fmaxf(top, __uint_as_float(swap8(__float_as_uint(top))));
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      const float next = fmaxf(ref, top);
      const float f = __builtin_amdgcn_exp2f(ref - next);
      ref = next;
      sum *= f;
#pragma unroll
      for (int t = 0; t < NT; ++t) o[t] *= f;
    }
    float pr[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
#pragma clang fp contract(off)  // ref is some x cf rounded: so has to be each that it is taken from
      pr[e] = __builtin_amdgcn_exp2f(x[e] - ref + kKv4Lift);
      sum += pr[e];
    }
    half8v ph, pl;
    uint32_t hw[E / 2], lw[E / 2];
#pragma unroll
    for (int e = 0; e < E; e += 2) hw[e / 2] = pack16<false>(pr[e], pr[e + 1]);
    if constexpr (!BF) {
#pragma unroll
      for (int e = 0; e < E; e += 2)
        lw[e / 2] = pack16<false>(pr[e] - lo16<false>(hw[e / 2]), pr[e + 1] - hi16<false>(hw[e / 2]));
    }
    if constexpr (TC == 8) {
      // lanes r < 8 get tile 1's upper parts, the others tile 0's lower parts
      uint32_t got[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) got[i] = swap8(BF ? hw[i] : r < 8 ? lw[i] : hw[i]);
      if constexpr (BF)
        ph = __builtin_bit_cast(half8v, u32x4v{hw[0], hw[1], got[0], got[1]});
      else
        ph = __builtin_bit_cast(half8v, u32x4v{r < 8 ? hw[0] : got[0], r < 8 ? hw[1] : got[1],
                                               r < 8 ? got[0] : lw[0], r < 8 ? got[1] : lw[1]});
    } else {
      ph = __builtin_bit_cast(half8v, u32x4v{hw[0], hw[1], hw[2], hw[3]});
      if constexpr (!BF) pl = __builtin_bit_cast(half8v, u32x4v{lw[0], lw[1], lw[2], lw[3]});
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int q = t * 16 / (D / NG);
      const half8v vf = values(kv.v[t >> 2][t & 3], kv.vs[q], kv.vm[q]);
      o[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, ph, o[t], 0, 0, 0);
      if constexpr (!BF && TC == 16)
        o[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, pl, o[t], 0, 0, 0);
    }
  };

  if (any) {
    for (;;) {
      advance();
      int pgn = look_up(), offn = off;
      kv1.load(base_of(pg1, off1), lane);
      if (valid(pg0)) process(kv0, blk0);
      if (blk1 >= b1) break;
      pg0 = pgn;
      blk0 = blk;
      advance();
      pgn = look_up();
      kv0.load(base_of(pg0, offn), lane);
      offn = off;
      if (valid(pg1)) process(kv1, blk1);
      if (blk0 >= b1) break;
      pg1 = pgn;
      blk1 = blk;
      off1 = offn;
    }
  }
  sum += __shfl_xor(sum, 16);
  sum += __shfl_xor(sum, 32);
  if constexpr (TC == 8) sum += __uint_as_float(swap8(__float_as_uint(sum)));

  // joins the waves: the tile's reference and sum, and rows 16 (wave + AW k) .. of its o
  float m, l;
  f32x4 v[NT / AW];
  auto join = [&]() {
#pragma unroll
    for (int t = 0; t < NT; ++t) red_o[wave][t][lane] = o[t];
    if (g == 0) {
      red_ml[wave][r & 7][r >> 3] = ref;
      red_ml[AW + wave][r & 7][r >> 3] = sum;
    }
    __syncthreads();
    m = kKv4None;
    l = 0.f;
    float f[AW];
#pragma unroll
    for (int i = 0; i < AW; ++i) m = fmaxf(m, red_ml[i][r & 7][r >> 3]);
#pragma unroll
    for (int i = 0; i < AW; ++i) {
      f[i] = __builtin_amdgcn_exp2f(red_ml[i][r & 7][r >> 3] - m);
      l += f[i] * red_ml[AW + i][r & 7][r >> 3];
    }
#pragma unroll
    for (int k = 0; k < NT / AW; ++k) {
      v[k] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < AW; ++i) {
        f32x4 x = red_o[i][wave + AW * k][lane];
        if constexpr (TC == 8 && !BF) x += red_o[i][wave + AW * k][lane ^ 8];
        v[k] += x * f[i];
      }
    }
  };
  join();
  const bool mine = live && r < TC;
  if (r0 == 0 && r1 == (uint32_t)span) {
    if (mine) {
      const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
      for (int k = 0; k < NT / AW; ++k) {
        v[k] *= inv;
        *reinterpret_cast<u32x2v*>(p.out + (size_t)row * p.ldo + (size_t)qh * D +
                                   16 * (wave + AW * k) + 4 * g) =
            u32x2v{pack16<BF>(v[k][0], v[k][1]), pack16<BF>(v[k][2], v[k][3])};
      }
      if (wave == 0 && g == 0 && p.lse != nullptr)
        p.lse[(size_t)row * p.q_heads + qh] = (m + log2f(l) - kKv4Lift) * 0.6931471805599453f;
    }
    __syncthreads();
    continue;
  }
  // A shared tile: the sums go to the workspace ([column][D], and m, l per column), slot
  // 2 w + 1 for the stripe w in which the tile starts, 2 w for the others.  The last
  // workgroup to arrive joins them, in the order of the stripes.
  const uint32_t w0 = u0 / stripes.stripe, w1 = (u0 + span - 1) / stripes.stripe;
  {
    const size_t slot = 2 * blockIdx.x + (blockIdx.x == w0);
    if (mine) {
#pragma unroll
      for (int k = 0; k < NT / AW; ++k) {
        float* at = p.part_o + (slot * TC + rc) * D + 16 * (wave + AW * k) + 4 * g;
        put8(at, v[k][0], v[k][1]);
        put8(at + 2, v[k][2], v[k][3]);
      }
      if (wave == 0 && g == 0) put8(p.part_ml + (slot * TC + rc) * 2, m, l);
    }
  }
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  if (threadIdx.x == 0)
    arrived = __hip_atomic_fetch_add(p.counters + w0, 1, __ATOMIC_RELAXED,
                                     __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  const bool last_one = arrived == (int)(w1 - w0);
  __syncthreads();
  if (!last_one) continue;
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  if (threadIdx.x == 0)
    __hip_atomic_store(p.counters + w0, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  // Eight columns at a time: a thread takes 4 channels of one of them from every `parts`-th
  // stripe, and the parts meet in LDS (fewer columns: more parts).
  constexpr int NL = D / 4;
  static_assert(8 * NL <= AW * NT * 64 && 8 * NL <= 64 * AW, "the parts fit");
  f32x4* sums = &red_o[0][0][0];         // [z][NL]
  const int z = threadIdx.x / NL, c4 = threadIdx.x % NL;
#pragma unroll 1
  for (int c8 = 0; c8 < TC; c8 += 8) {
    const int cols = (seq.n * ratio - tile * TC) - c8;  // live columns, of the eight and on
    if (cols <= 0) break;
    const int shift = cols > 4 ? 3 : cols > 2 ? 2 : cols > 1 ? 1 : 0, parts = 8 >> shift;
    const int i = z & ((1 << shift) - 1);
    f32x4 so = {0.f, 0.f, 0.f, 0.f};
    float sm = kKv4None, sl = 0.f;
    if (z < 8 && i < cols) {
      // eight stripes' loads in flight; past the last one its own again, with weight 0
      for (uint32_t k0 = w0 + (z >> shift); k0 <= w1; k0 += 8 * parts) {
        f32x4 x[8];
        float cm[8], cl[8], next = sm;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t k = k0 + j * parts <= w1 ? k0 + j * parts : w1;
          const size_t slot = (size_t)2 * k + (k == w0);
          get16(p.part_o + (slot * TC + c8 + i) * D + 4 * c4, x[j]);
          get8(p.part_ml + (slot * TC + c8 + i) * 2, cm[j], cl[j]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) next = fmaxf(next, cm[j]);
        const float fa = __builtin_amdgcn_exp2f(sm - next);
        sm = next;
        sl *= fa;
        so *= fa;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (k0 + j * parts > w1) break;
          const float fb = __builtin_amdgcn_exp2f(cm[j] - next);
          sl += cl[j] * fb;
          so += x[j] * fb;
        }
      }
      sums[z * NL + c4] = so;
      if (c4 == 0) {
        red_ml[z][0][0] = sm;
        red_ml[z][0][1] = sl;
      }
    }
    __syncthreads();
    if (z < (1 << shift) && i < cols) {
      float tm = kKv4None, tl = 0.f;
      f32x4 to = {0.f, 0.f, 0.f, 0.f};
      for (int k = z; k < 8; k += 1 << shift) tm = fmaxf(tm, red_ml[k][0][0]);
      for (int k = z; k < 8; k += 1 << shift) {
        const float f = __builtin_amdgcn_exp2f(red_ml[k][0][0] - tm);
        tl += f * red_ml[k][0][1];
        to += sums[k * NL + c4] * f;
      }
      to *= tl > 0.f || tl != tl ? 1.f / tl : 0.f;
      const int tc = tile * TC + c8 + i;
      const size_t trow = seq.first + tc / ratio;
      const int th = head * ratio + tc % ratio;
      *reinterpret_cast<u32x2v*>(p.out + trow * p.ldo + (size_t)th * D + 4 * c4) =
          u32x2v{pack16<BF>(to[0], to[1]), pack16<BF>(to[2], to[3])};
      if (c4 == 0 && p.lse != nullptr)
        p.lse[trow * p.q_heads + th] = (tm + log2f(tl) - kKv4Lift) * 0.6931471805599453f;
    }
    __syncthreads();
  }
  }
}

typedef void (*AttendFn)(Kv4AttendArgs);
template <int TC, bool BF, bool TREE>
AttendFn attend_kernel(int D, int groups) {
  if (D == 128)
    return groups == 1 ? kv4_attend_kernel<128, 1, TC, BF, TREE>
                       : groups == 2 ? kv4_attend_kernel<128, 2, TC, BF, TREE>
                                     : kv4_attend_kernel<128, 4, TC, BF, TREE>;
  return groups == 1 ? kv4_attend_kernel<64, 1, TC, BF, TREE>
                     : kv4_attend_kernel<64, 2, TC, BF, TREE>;
}
template <bool TREE>
AttendFn attend_kernel(int cols, bool bf, int D, int groups) {
  if (cols == 8)
    return bf ? attend_kernel<8, true, TREE>(D, groups) : attend_kernel<8, false, TREE>(D, groups);
  return bf ? attend_kernel<16, true, TREE>(D, groups) : attend_kernel<16, false, TREE>(D, groups);
}

// Tiles of 128 columns for trees, or of 16?  A block takes a workgroup 0.42 us in a tile of 16 and
// 2 us in one of 128, a tile costs 10 and 4 blocks more, and tiles of 128 take 11 us more to hand
// over and join; of several sequences the lengths are taken for half of what they may be.  16
// against 128, 64 query heads on 8, us: 128 columns, contexts to 8 x 8192 / 1 x 32768 / 32 x 2048 /
// 64 x 300 tokens 69 / 60 / 75 / 58 against 57 / 58 / 60 / 31; 96 columns, 8 x 8192 / 32 x 2048:
// 41 / 55 against 47 / 50; 104 columns, 2 x 131072: 250 against 163; 256 columns, 8 x 8192: 126
// against 96; 512 columns, 1 x 4000: 41 against 40; 64 columns, 4 x 131072: 248 against 287.
// The rule has one price for all types, heads and groups (fp16, 128 channels, groups of 64).  The
// others, 8 x 8192 tokens of 128 / 96 / 64 columns: bf16 51 / 46 / 51 against 44 / 48 / 54; groups of
// 128 64 / 54 / 40 against 54 / 53 / 48; groups of 32 91 / 67 / 57 against 60 / 53 / 60, bf16 77 /
// 72 / 61 against 50 / 55 / 56; 64 channels 45 / 31 / 25 against 40 / 38 / 32.  It is wrong by up to
// 1.3 for groups of 32 and 96 columns, and by 1.1 for 64 channels, 512 columns over 1 x 4000 (29
// against 31).  Nor does it count how long a tile is looked for among many sequences: 128 columns
// of 2048 x 300 tokens 1725 against 1099, of 8192 x 150 6133 against 8275.
bool wide_tree(int batch, long long columns, int max_new, int max_len, int heads, int window) {
  double span = (max_len + 31.0) / 32;
  if (batch > 1) span /= 2;
  const double near = ((double)window + max_new) / 32 + 2;
  if (window > 0 && span > near) span = near;
  const double units = (double)batch * heads;
  const double narrow = 0.42 * units * (double)((columns + 15) / 16) * (span + 10);
  const double wide = 2.0 * units * (double)((columns + 127) / 128) * (span + 4) + 11.0 * KV4_STRIPES;
  return wide < narrow;
}

}  // namespace

size_t kv4_attend_most_floats(int cols, int D) {
  // two slots a stripe of narrow tiles; fewer than target + target chunks of wide ones
  return (size_t)2 * KV4_STRIPES * cols * (D + 2) + (cols == 128 ? KV4_STRIPES * KV4_TREE_SHARED : 0);
}

Kv4AttendPlan kv4_attend_plan(int batch, int tokens, int max_new, int max_len, int q_heads,
                              int heads, int D, int window, bool tree) {
  Kv4AttendPlan p{};
  const int ratio = q_heads / heads;
  const long long columns = (long long)max_new * ratio;
  p.cols = columns <= 8 ? 8 : columns <= kPrefillColumns ? 16 : 128;
  if (tree && columns > 8) p.cols = wide_tree(batch, columns, max_new, max_len, heads, window) ? 128 : 16;
  p.col_tiles = (int)((columns + p.cols - 1) / p.cols);
  // tiles there can be: each sequence rounds up, and rows are not shared
  long long tiles = ((long long)tokens * ratio + p.cols - 1) / p.cols + batch;
  if (tiles > (long long)batch * p.col_tiles) tiles = (long long)batch * p.col_tiles;
  tiles *= heads;
  // blocks a tile can see: the window of its first token up to its last
  long long span = ((long long)max_len + 31) / 32;
  const long long near = ((long long)window + (tree ? max_new : p.cols / ratio + 1)) / 32 + 2;
  if (window > 0 && span > near) span = near;
  if (p.cols == 128 && !tree) {
    // Chunks of 8 / 16 / 32 blocks at least, us: 32 new tokens of 8 sequences on 2 kv heads, to
    // 16384: 55 / 47 / 56; 200 on 4, 2000: 33 / 35 / 49; 64 of 4 on 8, to 4096: 65 / 65 / 60;
    // 1024 on 1, 1024: 26 / 32 / 47; no difference above.  Chunks for 256 / 512 / 768 / 1024
    // workgroups: 512 on 8, 8192: 296 / 244 / 254 / 250; 512 of 2 on 1, 16384: 163 / 142 / 111 /
    // 129; 130 on 8, 131072: 1843 / 1432 / 1286 / 1207.
    p.target = KV4_STRIPES;
    p.chunk = 16;
    p.chunks = (int)((span + p.chunk - 1) / p.chunk);
    if (p.chunks <= 1 || tiles >= p.target || batch > 1024) {
      p.chunks = 1;
      return p;  // enough tiles by themselves
    }
    long long slots = p.target + tiles;
    if (slots > tiles * p.chunks) slots = tiles * p.chunks;
    p.slots = (int)slots;
    p.tiles = (int)tiles;
  } else {
    // Stripes of 4 / 8 / 16 / 32 blocks at least, single tokens, us: one sequence of 1000 tokens
    // on 8 kv heads 9.5 / 10.2 / 11.7 / 11.5, of 4000 13.8 / 11.6 / 11.8 / 14.8, of 16000 25.4 /
    // 25.9 / 16.5 / 16.6; six to 4000 15.9 / 15.2 / 12.5 / 15.3, to 16000 26 each; 24 to 1000
    // 16.1 / 16.1 / 16.0 / 12.5, to 16000 55 each.
    // Tiles of 128 columns (trees), 8 / 12 / 16 / 24: 128 columns over 1 x 32768 tokens 58 / 58 / 59 /
    // 63, 8 x 8192 57 / 57 / 58 / 62, 64 x 300 39 / 31 / 31 / 32; 512 over 1 x 4000 41 / 40 / 43 / 47.
    p.chunk = p.cols == 128 ? 12 : 8;
    long long stripes = tiles * ((span + p.chunk - 1) / p.chunk);
    // Trees only, and always stripes: two at least, since one tile of twelve blocks is never worth
    // 128 columns (wide_tree: 77 us of workgroups at most against 5640 at least).
    const bool wide = p.cols == 128;
    if (!wide && (batch > 1024 || stripes <= tiles)) return p;
    // Trees, tiles of 16 over short contexts: whole tiles where there are enough of them, since
    // to share one costs as much as 16 blocks.  In stripes against whole, us: 3 trees of 93 nodes
    // to 275 tokens, 64 query heads on 32, 37 / 29; 32 of 10 to 600, 64 on 8, 33 / 24; 64 of 4 to
    // 500 29 / 22; 64 of 8 to 1000 49 / 46; 32 of 8 to 2048 44 / 46.
    if (tree && !wide && tiles >= KV4_STRIPES && span <= 32) return p;
    // Trees, tiles of 16: 32 parts of a tile at most, which one workgroup joins.  16 / 32 / 48 / 64 /
    // no limit: 9 nodes over 36083 tokens, 8 heads on 1, 32 / 29 / 30 / 35 / 55; 16 over 100000
    // 59 / 44 / 54 / 54 / 55; 4 over 100000, 16 on 2, 59 / 43 / 41 / 41 / 74.
    if (tree && !wide && stripes > 32 * tiles) stripes = 32 * tiles;
    if (stripes > KV4_STRIPES) stripes = KV4_STRIPES;
    p.target = (int)stripes;
    p.tiles = tiles < (1 << 24) ? (int)tiles : 1 << 24;
    p.slots = 2 * (int)stripes;
    if (!wide) p.counters = (size_t)stripes;
  }
  p.floats = (size_t)p.slots * p.cols * (D + 2);
  if (tree && p.cols == 128) p.floats += (size_t)p.target * KV4_TREE_SHARED;
  return p;
}

hipError_t launch_kv4_attend(const Kv4AttendPlan& plan, const Kv4AttendArgs& args, int D, int groups,
                             bool bf, hipStream_t st) {
  Kv4AttendArgs a = args;
  a.col_tiles = plan.col_tiles;
  a.target = plan.target;
  a.chunk = plan.chunk;
  a.chunks = plan.chunks;
  a.slots = plan.slots;
  a.tiles = plan.tiles;
  if (plan.cols == 128)
    return a.mask ? launch_kv4_tree_wide(a, D, groups, bf, st)
                  : launch_kv4_prefill(a, D, groups, bf, st);
  const long long units = ((long long)a.heads * a.batch + 7) / 8 * 8;
  const unsigned grid = plan.slots ? plan.target : (unsigned)(units * plan.col_tiles);
  const AttendFn fn = a.mask ? attend_kernel<true>(plan.cols, bf, D, groups)
                             : attend_kernel<false>(plan.cols, bf, D, groups);
  hipLaunchKernelGGL(fn, kv4_grid(grid), dim3(64 * AW), 0, st, a);
  return hipGetLastError();
}

}  // namespace w4a16
