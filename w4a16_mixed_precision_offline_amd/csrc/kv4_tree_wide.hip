// Attention of large trees of drafted tokens over the 4-bit cache: tiles of 128 columns.
// kv4_prefill.hip has the mathematics and the operands' layout.
//
// All tiles of a sequence have the same blocks here, since every node sees what was held before
// the tree.  The blocks of all tiles are cut into equal stripes, one to a workgroup
// (Kv4Stripes); a stripe's part of a tile that others share goes to the workspace, and
// a second kernel joins a tile's parts in their order.
//
// What each of a block's tokens is to each column is worked out once, by the waves that unpack the
// block: 32 bits a column in LDS, where the block reaches into the tree or out of the window;
// there a NaN stays with the columns that see its token (clear_nan_tokens).
//
// Bound: matrix and vector instructions, of which the card overlaps two fifths at best (a probe
// of alternating phases, two waves to a SIMD: 644 ns where 432 and 360 are the parts).  Tiles
// all full and of equal length (16 sequences of 64 nodes and 8192 tokens, 64 query heads on 8 of
// 128 channels, groups of 64): 275 GFLOP in 483 us, 0.57 PFLOP/s (bf16 rows 401 us; groups of 128
// 464 us; a large fp16 product runs at 1.16).  Left out, of 513 us, the second part of p is worth
// 100 us, LDS reads 93, unpacking and its loads 85, exponentials and sums 38; one workgroup to a
// compute unit instead of two takes 707.  32 to 64 nodes and up to 8192 tokens: 100 GFLOP in 225
// us, of which 13 join 67 MB of parts; two trees of 13 nodes, contexts of 131072 and less, groups
// of 32: 161 us.
// Registers: 236 with groups of 64 (places in LDS and in the pages are worked out again for each
// stage: kept, they made 256 and spills).  4 are spilled with groups of 32.
// Measured, not kept: 8 waves of 32 columns over one stage (478 us where 513, but half-empty tiles
// of 256: 272 us where 250); K's operands read ahead of the block before, or of the unpacking, and
// no barriers for the scheduler (no difference within 3%).
#include "kv4_wide.h"

namespace w4a16 {

namespace {

constexpr int WS = 2;  // blocks of a stage

// What a stripe says of the tile that starts in it and goes on in others: `last` is the last of
// them, 0 if there is no such tile.
struct Shared {
  int first, n, head, tile;
  uint32_t last;
};
static_assert(sizeof(Shared) <= KV4_TREE_SHARED * sizeof(float), "it fits the workspace");

template <int D, int NG>
struct TreeStage {
  u32x4v k[WS][D / 16][64];
  u32x4v v[WS][2][D / 32][64];
  u32x4v m[WS][64];
  float s[WS][NG][32];
  uint32_t sees[WS][PTC];
  uint32_t nans[WS][NG];  // tokens whose V is NaN in a group, of a block of kind 2
  int kind[WS];  // 0: nobody looks at it, 1: all columns see all of it, 2: `sees` says what
};

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}

template <int D, int NG, bool BF>
__global__ __launch_bounds__(256, 2) void kv4_tree_wide_kernel(Kv4AttendArgs p) {
  constexpr int J = D / 16, JG = J / NG, CT = D / 32;
  __shared__ TreeStage<D, NG> lds[2];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int c = lane & 31, h = lane >> 5;
  const int half = wave & 1, mine = wave >> 1;  // what the wave unpacks of a stage
  const int ratio = p.q_heads / p.heads;
  const int page_blocks = p.page / 32;
  const size_t page_bytes = (size_t)p.heads * page_blocks * kv4_block_bytes(D, NG);

  // Of the two workgroups of a compute unit one goes first where both want the matrix or the vector
  // unit; alike, they want the same one at the same time (16 trees to 8192: 250 -> 233 us).
  if (blockIdx.x & 256) __builtin_amdgcn_s_setprio(2);
  // the channels of the m operand that stand for no group stay 0
  for (int i = threadIdx.x; i < 2 * WS * 64; i += 256)
    lds[i / (WS * 64)].m[i / 64 % WS][i % 64] = u32x4v{0u, 0u, 0u, 0u};

  Kv4Stripes<PTC, true> stripes;
  typename Kv4Stripes<PTC, true>::Lane lanes = stripes.init(p, ratio, gridDim.x);
  uint32_t place = blockIdx.x * stripes.stripe;
  const uint32_t stop =
      place + stripes.stripe < stripes.total ? place + stripes.stripe : stripes.total;
  Shared* shared = reinterpret_cast<Shared*>(p.part_shared) + blockIdx.x;
  const bool tells = threadIdx.x == 0;
  if (tells) shared->last = 0;
  for (bool again = false; place < stop; again = true) {
    Kv4Seq seq;
    int b, head, tile, span;
    uint32_t u0;
    if (again && p.batch <= 64) lanes = stripes.fetch(p, 0, ratio);
    stripes.find(p, place, ratio, lanes, seq, b, head, tile, span, u0);
    u0 += stripes.lead;
    const uint32_t r0 = place > u0 ? place - u0 : 0;
    place = u0 - stripes.lead + stripes.tile_size(span);
    if (stop <= u0) break;  // it has the lead of a tile only
    const uint32_t r1 = stop - u0 < (uint32_t)span ? stop - u0 : (uint32_t)span;
    if (r0 >= r1) continue;  // what rounds a tile up to whole stripes
    const bool last_part = r1 == (uint32_t)span;
    if (r0 == 0 && !last_part && tells)
      *shared = Shared{seq.first, seq.n, head, tile, (u0 + span - 1) / stripes.stripe};
    const Kv4Range rg = kv4_range<PTC, true>(p, seq, tile, ratio, r0, last_part ? -1 : (int)r1);
    const int b1 = rg.blk1;
    // every column sees the tokens [all_lo, rg.from)
    const int all_lo = p.window > 0 ? rg.from + seq.n - p.window : 0;
    const char* head_base = p.cache + (size_t)head * page_blocks * kv4_block_bytes(D, NG);
    const int* table = p.table + (size_t)b * p.width;

    const int col = tile * PTC + 32 * wave + c, ci = col / ratio;
    const bool live = ci < seq.n;
    const bool idle = (tile * PTC + 32 * wave) / ratio >= seq.n;  // the wave has no column
    const int qh = head * ratio + col % ratio;
    const int row = seq.first + (live ? ci : 0);
    half8v qf[J], qm;
    float cf;
    wide_queries<D, NG, BF>(p, row, qh, h, qf, qm, cf);

    f32x16 o[CT];
#pragma unroll
    for (int t = 0; t < CT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[t][i] = 0.f;
    float ref = kKv4None, sum = 0.f;
    uint32_t nan_groups = 0;  // groups of channels in which the column has seen a NaN
    bool far = false;  // of the whole wave: some column's reference is past kFar

    Piece<D, NG> piece;
    auto look_up = [&](int blk) {
      const int at = blk / page_blocks;
      return table[at < p.width ? at : p.width - 1];
    };
    auto valid = [&](int blk, int pg) { return blk < b1 && pg >= 0 && pg < p.pages; };
    auto fetch = [&](int blk, int pg) {
      int lane_ = lane;
      asm volatile("" : "+v"(lane_));
      piece.load(head_base + (size_t)(valid(blk, pg) ? pg : 0) * page_bytes +
                     (size_t)(blk % page_blocks) * kv4_block_bytes(D, NG),
                 half, lane_);
    };
    auto unpack = [&](TreeStage<D, NG>& st, int blk, int pg) {
      constexpr int W = D / 32;
      int lane_ = lane;
      asm volatile("" : "+v"(lane_));  // places are worked out again rather than kept
      const int t0 = blk * 32, g = lane_ >> 4, r = lane_ & 15;
      const bool look = valid(blk, pg), some = t0 < all_lo || t0 + 32 > rg.from;
      if (half == 0 && lane == 0) st.kind[mine] = look ? 1 + some : 0;
      if (!look) return;
      if (some) {
        uint32_t any = 0;
        for (int x = lane_; x < PTC; x += 64) {
          const int i = (tile * PTC + x) / ratio;
          uint32_t sees = 0;
          if (i < seq.n)
            sees = kv4_tree_sees(p, seq, seq.first + i, kv4_tree_first(p, seq, seq.first + i), t0);
          any |= sees;
          if (half == 0) st.sees[mine][x] = sees;
        }
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) any |= (uint32_t)__shfl_xor((int)any, off);
        // what no column sees may be anything: its s and m become 0
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if ((any >> kv4_slot_token(g, e) & 1u) == 0) {
            const uint32_t keep = e & 1 ? 0x0000FFFFu : 0xFFFF0000u;
#pragma unroll
            for (int i = 0; i < Piece<D, NG>::GH; ++i) {
              piece.vs[i][e >> 1] &= keep;
              piece.vm[i][e >> 1] &= keep;
            }
          }
        constexpr int GH = Piece<D, NG>::GH;
        uint32_t odd = 0;
#pragma unroll
        for (int i = 0; i < GH; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) odd |= maybe_nan(piece.vs[i][j]) | maybe_nan(piece.vm[i][j]);
        const bool look_close = __ballot(odd != 0) != 0;
#pragma unroll
        for (int i = 0; i < GH; ++i) {
          uint32_t bits = 0;
          if (look_close) {
            bits = clear_nan_tokens(piece.vs[i], piece.vm[i], g);
            bits |= (uint32_t)__shfl_xor((int)bits, 16);
            bits |= (uint32_t)__shfl_xor((int)bits, 32);
          }
          // (with one group both waves of a block have it, and say the same)
          if (lane == 0) st.nans[mine][(NG >= 2 ? half * GH : 0) + i] = bits;
        }
      }
      // K: token 16 half + r, channels 32 j + 8 g ..
#pragma unroll
      for (int j = 0; j < W; ++j)
        st.k[mine][2 * j + (g >> 1)][32 * (g & 1) + 16 * half + r] =
            __builtin_bit_cast(u32x4v, codes_subnormal(piece.k[j]));
      // V: channels 16 (W half + i) + r, tokens of word g
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const int c16 = W * half + i;
        const int q = NG >= 2 ? i * NG / (2 * W) : 0;
        st.v[mine][g >> 1][c16 >> 1][32 * (g & 1) + 16 * (i & 1) + r] =
            __builtin_bit_cast(u32x4v, values(piece.v[i], piece.vs[q], piece.vm[q]));
      }
      const int id = half * 64 + lane_;
      if (id < 32 * NG) {
        const int q = id / 32, t = id % 32;
        st.s[mine][q][t] = lo16<false>(piece.ks) * 0x1p16f;
        uint16_t* at = reinterpret_cast<uint16_t*>(&st.m[mine][32 * (q / 2) + t]) + 3 * (q & 1);
        at[0] = at[1] = at[2] = (uint16_t)piece.km;
      }
    };

    f32x16 zero;
#pragma unroll
    for (int i = 0; i < 16; ++i) zero[i] = 0.f;

    auto process = [&](const TreeStage<D, NG>& st, int i_blk, bool some) {
      half8v kf[J], vf[2][CT];
      const half8v mf = __builtin_bit_cast(half8v, st.m[i_blk][lane]);
#pragma unroll
      for (int j = 0; j < J; ++j)
        kf[j] = __builtin_bit_cast(half8v, st.k[i_blk][j / NG + j % NG * JG][lane]);
      __builtin_amdgcn_sched_barrier(0);
      f32x16 x = __builtin_amdgcn_mfma_f32_32x32x16_f16(mf, qm, zero, 0, 0, 0);
      f32x16 acc[NG];
#pragma unroll
      for (int j = 0; j < J; ++j)
        acc[j % NG] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
            kf[j], qf[j / NG + j % NG * JG], j < NG ? zero : acc[j % NG], 0, 0, 0);
#pragma unroll
      for (int q = 0; q < NG; ++q)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const f32x4 s = *reinterpret_cast<const f32x4*>(&st.s[i_blk][q][8 * k + 4 * h]);
#pragma unroll
          for (int i = 4 * k; i < 4 * k + 4; ++i)
            x[i] = __builtin_fmaf(s[i & 3], acc[q][i], x[i]);
        }
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int t = 0; t < CT; ++t)
          vf[s][t] = __builtin_bit_cast(half8v, st.v[i_blk][s][t][lane]);
      __builtin_amdgcn_sched_barrier(0);
      if (some) {
        const uint32_t sees = st.sees[i_blk][32 * wave + c] >> (4 * h);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if ((sees >> (8 * (i >> 2) + (i & 3)) & 1u) == 0) x[i] = -INFINITY;
#pragma unroll
        for (int q = 0; q < NG; ++q) {
          const uint32_t nans = __builtin_amdgcn_readfirstlane(st.nans[i_blk][q]);
          if (nans == 0) continue;
          if ((st.sees[i_blk][32 * wave + c] & nans) != 0) nan_groups |= 1u << q;
        }
      }
      float top = max3(x[0], x[1], x[2]);
#pragma unroll
      for (int i = 3; i < 15; i += 2) top = max3(top, x[i], x[i + 1]);
      top = max3(top, x[15], x[15]);
      top *= cf;
      float by = cf;
      if (__ballot(top > ref + kKv4Lazy) != 0 || far) {
#pragma clang fp contract(off)
        top = fmaxf(top, __shfl_xor(top, 32));
        const float next = fmaxf(ref, top);
        const float f = __builtin_amdgcn_exp2f(ref - next);
        ref = next;
        sum *= f;
#pragma unroll
        for (int t = 0; t < CT; ++t) o[t] *= f;
        far = __ballot(ref != kKv4None && fabsf(ref) > kFar) != 0;
        if (far) {
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = x[i] * cf - ref;
          by = 1.f;
        }
      }
      const float base = far ? kKv4Lift : kKv4Lift - ref;
      float pr[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        pr[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[i], by, base));
        sum += pr[i];
      }
      half8v pb[2], pl[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        u32x4v hi, lo;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = pr[4 * s + 8 * (i >> 1) + 2 * (i & 1)];
          const float b_ = pr[4 * s + 8 * (i >> 1) + 2 * (i & 1) + 1];
          hi[i] = pack16<false>(a, b_);
          if constexpr (!BF)
            lo[i] = pack16<false>(__builtin_fmaf(lo16<false>(hi[i]), -1.f, a),
                                  __builtin_fmaf(hi16<false>(hi[i]), -1.f, b_));
        }
        pb[s] = __builtin_bit_cast(half8v, hi);
        if constexpr (!BF) pl[s] = __builtin_bit_cast(half8v, lo);
      }
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int t = 0; t < CT; ++t)
          o[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf[s][t], pb[s], o[t], 0, 0, 0);
      if constexpr (!BF) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int t = 0; t < CT; ++t)
            o[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf[s][t], pl[s], o[t], 0, 0, 0);
      }
    };

    // The next stage's bytes are in flight while a stage is worked on; a page number is fetched
    // a stage earlier still.  With two stages in LDS one barrier is enough: whoever is past it
    // has worked on the stage before, which is the one written over next.
    int blk = rg.blk0;
    if (blk < b1) {
      int pg = look_up(blk + mine), next = look_up(blk + WS + mine);
      fetch(blk + mine, pg);
      __syncthreads();  // m is cleared, or the last tile's stages are no longer read
      for (int buf = 0;; buf ^= 1) {
        unpack(lds[buf], blk + mine, pg);
        __syncthreads();
        pg = next;
        if (blk + WS < b1) {
          next = look_up(blk + 2 * WS + mine);
          fetch(blk + WS + mine, pg);
        }
        if (!idle) {
#pragma unroll 1
          for (int i = 0; i < WS; ++i) {
            const int kind = __builtin_amdgcn_readfirstlane(lds[buf].kind[i]);
            if (kind != 0) process(lds[buf], i, kind == 2);
          }
        }
        blk += WS;
        if (blk >= b1) break;
      }
    }

    if (__ballot(nan_groups != 0) != 0) {
#pragma unroll
      for (int t = 0; t < CT; ++t) o[t] += nan_groups >> (t * NG / CT) & 1u ? NAN : 0.f;
    }
    sum += __shfl_xor(sum, 32);
    int col_ = tile * PTC + 32 * wave + c;
    asm volatile("" : "+v"(col_));  // worked out again rather than kept in registers
    const int ci_ = col_ / ratio, qh_ = head * ratio + col_ % ratio, row_ = seq.first + ci_;
    const bool live_ = ci_ < seq.n;
    if (r0 != 0 || !last_part) {
      // slot 2 w + 1 for the stripe w in which the tile's blocks start, 2 w for the others
      const size_t slot = 2 * blockIdx.x + (blockIdx.x == u0 / stripes.stripe);
      float* po = p.part_o + slot * PTC * D;
#pragma unroll
      for (int t = 0; t < CT; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<f32x4*>(po + (((wave * CT + t) * 4 + k) * 64 + lane) * 4) =
              f32x4{o[t][4 * k], o[t][4 * k + 1], o[t][4 * k + 2], o[t][4 * k + 3]};
      if (h == 0) {
        float* ml = p.part_ml + (slot * PTC + 32 * wave + c) * 2;
        ml[0] = ref;
        ml[1] = sum;
      }
    } else if (live_) {
      const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
      uint16_t* dst = p.out + (size_t)row_ * p.ldo + (size_t)qh_ * D + 4 * h;
#pragma unroll
      for (int t = 0; t < CT; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<u32x2v*>(dst + 32 * t + 8 * k) =
              u32x2v{pack16<BF>(o[t][4 * k] * inv, o[t][4 * k + 1] * inv),
                     pack16<BF>(o[t][4 * k + 2] * inv, o[t][4 * k + 3] * inv)};
      if (h == 0 && p.lse != nullptr)
        p.lse[(size_t)row_ * p.q_heads + qh_] = (ref + log2f(sum) - kKv4Lift) * 0.6931471805599453f;
    }
  }
}

// Joins the parts of the tile that starts in a stripe and goes on past it, if there is one.
// Grid: (D / (8 KN), stripes): a workgroup has 8 KN channels of the tile's 128 columns, a thread
// 4 KN of one.  The channels go first, since workgroups go round robin to the 8 XCDs: tiles of
// even lengths start in stripes that one XCD would have all of.
template <int D, bool BF, int KN>
__global__ __launch_bounds__(256) void kv4_tree_join_kernel(Kv4AttendArgs p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = lane & 31, h = lane >> 5, t = blockIdx.x * KN / 4, k0 = blockIdx.x * KN % 4;
  const uint32_t first = blockIdx.y;
  const int ratio = p.q_heads / p.heads;
  const Shared x = reinterpret_cast<const Shared*>(p.part_shared)[first];
  if (x.last == 0) return;
  const int col = x.tile * PTC + 32 * wave + c, ci = col / ratio;
  if (ci >= x.n) return;
  const int qh = x.head * ratio + col % ratio, row = x.first + ci;
  float m = kKv4None, l = 0.f;
  f32x4 o[KN];
#pragma unroll
  for (int k = 0; k < KN; ++k) o[k] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 16 / KN
  for (uint32_t i = first; i <= x.last; ++i) {
    const size_t slot = 2 * (size_t)i + (i == first);
    const float* ml = p.part_ml + (slot * PTC + 32 * wave + c) * 2;
    const f32x4* at = reinterpret_cast<const f32x4*>(p.part_o + slot * PTC * D) +
                      ((wave * (D / 32) + t) * 4 + k0) * 64 + lane;
    f32x4 v[KN];
#pragma unroll
    for (int k = 0; k < KN; ++k) v[k] = at[64 * k];
    const float cm = ml[0], cl = ml[1];
    const float next = fmaxf(m, cm);
    const float a = __builtin_amdgcn_exp2f(m - next), f = __builtin_amdgcn_exp2f(cm - next);
    m = next;
    l = l * a + cl * f;
#pragma unroll
    for (int k = 0; k < KN; ++k) o[k] = o[k] * a + v[k] * f;
  }
  const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
  uint16_t* dst = p.out + (size_t)row * p.ldo + (size_t)qh * D + 32 * t + 8 * k0 + 4 * h;
#pragma unroll
  for (int k = 0; k < KN; ++k) {
    o[k] *= inv;
    *reinterpret_cast<u32x2v*>(dst + 8 * k) =
        u32x2v{pack16<BF>(o[k][0], o[k][1]), pack16<BF>(o[k][2], o[k][3])};
  }
  if (blockIdx.x == 0 && h == 0 && p.lse != nullptr)
    p.lse[(size_t)row * p.q_heads + qh] = (m + log2f(l) - kKv4Lift) * 0.6931471805599453f;
}

typedef void (*TreeFn)(Kv4AttendArgs);
template <bool BF>
TreeFn tree_kernel(int D, int groups) {
  if (D == 128)
    return groups == 1   ? kv4_tree_wide_kernel<128, 1, BF>
           : groups == 2 ? kv4_tree_wide_kernel<128, 2, BF>
                         : kv4_tree_wide_kernel<128, 4, BF>;
  return groups == 1 ? kv4_tree_wide_kernel<64, 1, BF> : kv4_tree_wide_kernel<64, 2, BF>;
}
template <int KN>
TreeFn join_kernel(int D, bool bf) {
  if (D == 128) return bf ? kv4_tree_join_kernel<128, true, KN> : kv4_tree_join_kernel<128, false, KN>;
  return bf ? kv4_tree_join_kernel<64, true, KN> : kv4_tree_join_kernel<64, false, KN>;
}

}  // namespace

hipError_t launch_kv4_tree_wide(const Kv4AttendArgs& a, int D, int groups, bool bf,
                                hipStream_t st) {
  hipLaunchKernelGGL(bf ? tree_kernel<true>(D, groups) : tree_kernel<false>(D, groups),
                     dim3(a.target), dim3(256), 0, st, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // Many tiles of few parts: 32 channels a workgroup, few of many: 8.  8 against 32: 384 tiles of
  // 2 or 3 parts 17 against 13 us, 16 tiles of 32 parts 13 against 18.
  if (a.target >= 8 * a.tiles)
    hipLaunchKernelGGL(join_kernel<1>(D, bf), dim3(D / 8, a.target), dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL(join_kernel<4>(D, bf), dim3(D / 32, a.target), dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace w4a16
