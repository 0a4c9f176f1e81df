// Attention of many new tokens over the 4-bit cache: tiles of 128 columns (kv4_attention.hip
// has the mathematics, and tiles of 16).
//
// With 16 columns a wave unpacks a block of the cache for 16 matrix instructions.  Here a
// workgroup unpacks it once for 128 columns, into LDS, in the order in which the matrix
// instruction 32x32x16 takes its operands: every read is 16 bytes a lane, side by side.
//   K    codes as fp16 subnormals (exact), 32 tokens x 16 channels an operand
//   V^T  m + s c in fp16 (one rounding), 32 channels x 16 tokens an operand: K q^T leaves a
//        lane the tokens 4 h + 8 k + i of its column (h = lane / 32, k, i = 0..3), which are
//        the tokens of the cache's words 2 s + h, s = 0, 1, so p goes from one product to
//        the other inside the lane
//   m    logit = sum_g s_g (sum c q)_g + m_g (sum q)_g: the second part is a product as well,
//        of m with (sum q) split into three fp16 numbers (33 bits), one matrix instruction
//        a block; what is left per logit is one fma with s per group.
// A wave has 32 columns and streams stages of 64 tokens; the next stage's bytes are loaded
// into registers before a stage is worked on and unpacked into the other half of LDS after
// it, with one barrier a stage.
//
// For fp16 rows p is hi + lo, 22 bits, as with the smaller tiles, at 8 matrix instructions
// more on 17: with p rounded once the result's error is 1.65 times that of its own rounding,
// with lo 1.33 times, and 4 sequences of 512 new tokens take 611 us instead of 480.  bf16
// rows, whose own step is 2^-9, do without (424 us).
//
// Bound: matrix and vector instructions together.  4 sequences of 4109 to 8192 tokens, 512
// of them new, 64 query heads on 8 of 128 channels: 370 GFLOP in 611 us (601 to 634 from card
// to card), 0.61 PFLOP/s, half of the rate of a large fp16 product (1.2 PFLOP/s), 1060 us with
// tiles of 16.  Counters: the matrix unit busy 45% and the vector unit 51% of the time, LDS 27%;
// two waves of 208 to 240 registers fit a SIMD and take turns badly.  Measured, not kept: one
// block's product issued beside the exponentials of the block before it (with p hi + lo 640 us,
// registers spill), two sums per product instead of one dependent chain (637 us), longest
// sequences first (no difference).
#include "kv4_attend.h"

namespace w4a16 {

namespace {

constexpr int PTC = 128;  // columns of a workgroup
constexpr int PS = 2;     // blocks of a stage

// p's exponent is x cf - ref + 8 in one fma.  ref is some x cf rounded, so past 2^26 their
// difference alone can lift p out of fp16: past this reference x cf is rounded first.
constexpr float kFar = 0x1p20f;

template <int D, int NG>
struct Stage {
  u32x4v k[PS][D / 16][64];
  u32x4v v[PS][2][D / 32][64];
  u32x4v m[PS][64];
  float s[PS][NG][32];
};

// What a thread loads of a stage: wave w serves block w / 2, half w % 2.
template <int D, int NG>
struct Piece {
  static constexpr int W = D / 32;                 // words of a K or V item
  static constexpr int GH = NG >= 2 ? NG / 2 : 1;  // groups of half a row's channels
  uint32_t k[W], v[W];
  u32x4v vs[GH], vm[GH];
  uint32_t ks, km;

  __device__ __forceinline__ void load(const char* base, int half, int lane) {
    typedef uint32_t words __attribute__((ext_vector_type(W)));
    const words a = *reinterpret_cast<const words*>(base + (half * 64 + lane) * (4 * W));
    const words b = *reinterpret_cast<const words*>(
        base + 16 * D + (D == 128 ? (half * 64 + lane) * 16 : lane * 16 + 8 * half));
#pragma unroll
    for (int i = 0; i < W; ++i) {
      k[i] = a[i];
      v[i] = b[i];
    }
    const char* par = base + 32 * D;
#pragma unroll
    for (int i = 0; i < GH; ++i) {
      const int q = (NG >= 2 ? half * GH : 0) + i;
      const char* at = par + 128 * (NG + q) + 16 * (lane >> 4);
      vs[i] = *reinterpret_cast<const u32x4v*>(at);
      vm[i] = *reinterpret_cast<const u32x4v*>(at + 64);
    }
    const int id = half * 64 + lane;  // token id % 32, group id / 32
    if (id < 32 * NG) {
      const uint16_t* at =
          reinterpret_cast<const uint16_t*>(par + 128 * (id / 32)) + kv4_token_slot(id % 32);
      ks = at[0];
      km = at[32];
    }
  }
};

// Grid without chunks: 8 x tiles x (units / 8); with: one workgroup per chunk.
template <int D, int NG, bool BF>
__global__ __launch_bounds__(256, 2) void kv4_prefill_kernel(Kv4AttendArgs p) {
  constexpr int J = D / 16, JG = J / NG, CT = D / 32;
  __shared__ Stage<D, NG> lds[2];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int c = lane & 31, h = lane >> 5;
  const int ratio = p.q_heads / p.heads;
  Kv4Place w;
  if (!(p.slots ? kv4_place_chunk<PTC, false>(p, blockIdx.x, w) : kv4_place_whole(p, w))) return;
  const int size = (w.span + w.chunks - 1) / w.chunks;
  const Kv4Range rg = kv4_range<PTC>(p, w.s, w.tile, ratio, w.chunk * size,
                                     w.chunk == w.chunks - 1 ? -1 : (w.chunk + 1) * size);
  if (rg.i0 >= w.s.n) return;
  const int col = w.tile * PTC + 32 * wave + c, ci = col / ratio;
  const bool live = ci < w.s.n;
  const int qh = w.head * ratio + col % ratio;
  const int row = w.s.first + (live ? ci : 0);
  // tokens seen: column [first, last], any column [lo, hi) (of the wave: [wlo, whi)), every
  // column of the wave [all_lo, all_hi)
  const int last = live ? rg.from + ci : -1;
  const int first = p.window > 0 ? last - p.window + 1 : 0;
  const int w0 = (w.tile * PTC + 32 * wave) / ratio;
  const int wl = (w.tile * PTC + 32 * wave + 31) / ratio;
  const int w1 = wl < w.s.n - 1 ? wl : w.s.n - 1;
  const int whi = w0 < w.s.n ? rg.from + w1 + 1 : 0;
  const int wlo = p.window > 0 ? rg.from + w0 - p.window + 1 : 0;
  const int all_hi = wl < w.s.n ? rg.from + w0 + 1 : 0;
  const int all_lo = p.window > 0 ? rg.from + w1 - p.window + 1 : 0;

  half8v qf[J], qm;
  float cf;
  {
    float top = 0.f;
    u32x4v raw[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      raw[j] = *reinterpret_cast<const u32x4v*>(p.q + (size_t)row * p.ldq + (size_t)qh * D +
                                                16 * j + 8 * h);
      float f[8];
      unpack8<BF>(raw[j], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(f[e]));
    }
    top = fmaxf(top, __shfl_xor(top, 32));
    const int d = query_exponent(top);
    const float up = __builtin_ldexpf(1.f, d);
    float qsum[NG];
#pragma unroll
    for (int q = 0; q < NG; ++q) qsum[q] = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float f[8], x[8];
      unpack8<BF>(raw[j], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = f[e] * up;
        qsum[j / JG] += x[e];
        if (e & 2) x[e] *= 0.0625f;
      }
      qf[j] = __builtin_bit_cast(half8v, pack8<false>(x));
    }
    // (sum q) / 2^8 of a group as three fp16 numbers: groups 0, 1 at channels 0..5 of the
    // operand, groups 2, 3 at 8..13
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.f;
#pragma unroll
    for (int q = 0; q < NG; ++q) {
      float y = (qsum[q] + __shfl_xor(qsum[q], 32)) * 0x1p-8f;
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const float z = lo16<false>(to16<false>(y));
        y -= z;
        if (h == q / 2) x[3 * (q & 1) + k] = z;
      }
    }
    qm = __builtin_bit_cast(half8v, pack8<false>(x));
    // above 0, which would make NaN of a masked logit; what is less leaves nothing of the others
    cf = fmaxf(__builtin_ldexpf(p.scale * 1.4426950408889634f, 8 - d), 0x1p-126f);
  }

  f32x16 o[CT];
#pragma unroll
  for (int t = 0; t < CT; ++t)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[t][i] = 0.f;
  float ref = kKv4None, sum = 0.f;
  bool far = false;  // of the whole wave: some column's reference is past kFar

  const int page_blocks = p.page / 32;
  const size_t page_bytes = (size_t)p.heads * page_blocks * kv4_block_bytes(D, NG);
  const char* head_base = p.cache + (size_t)w.head * page_blocks * kv4_block_bytes(D, NG);
  const int* table = p.table + (size_t)w.b * p.width;
  const int b1 = rg.blk1;

  // A block's page as the table has it, which is loaded ahead of use; is it one to read?
  auto look_up = [&](int blk) {
    const int at = blk / page_blocks;
    return table[at < p.width ? at : p.width - 1];
  };
  auto valid = [&](int blk, int pg) { return blk < b1 && pg >= 0 && pg < p.pages; };
  Piece<D, NG> piece;
  const int half = wave & 1, mine = wave >> 1;
  auto fetch = [&](int blk, int pg) {
    piece.load(head_base + (size_t)(valid(blk, pg) ? pg : 0) * page_bytes +
                   (size_t)(blk % page_blocks) * kv4_block_bytes(D, NG),
               half, lane);
  };
  auto unpack = [&](Stage<D, NG>& st, int blk, int pg) {
    constexpr int W = D / 32;
    const int t0 = blk * 32, g = lane >> 4, r = lane & 15;
    if (!valid(blk, pg)) return;  // nobody looks at it
    // what no column sees may be anything: its s and m become 0
    if (t0 < rg.lo || t0 + 32 > rg.hi) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int pos = t0 + kv4_slot_token(g, e);
        if (pos < rg.lo || pos >= rg.hi) {
          const uint32_t keep = e & 1 ? 0x0000FFFFu : 0xFFFF0000u;
#pragma unroll
          for (int i = 0; i < Piece<D, NG>::GH; ++i) {
            piece.vs[i][e >> 1] &= keep;
            piece.vm[i][e >> 1] &= keep;
          }
        }
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
    const int id = half * 64 + lane;
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

  auto process = [&](const Stage<D, NG>& st, int i_blk, int t0) {
    // Both products' operands are read ahead of them, at once: read one by one beside the
    // matrix instructions they cost 10% more.
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
        for (int i = 4 * k; i < 4 * k + 4; ++i) x[i] = __builtin_fmaf(s[i & 3], acc[q][i], x[i]);
      }
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int t = 0; t < CT; ++t) vf[s][t] = __builtin_bit_cast(half8v, st.v[i_blk][s][t][lane]);
    __builtin_amdgcn_sched_barrier(0);
    if (t0 < all_lo || t0 + 32 > all_hi) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int pos = t0 + 4 * h + 8 * (i >> 2) + (i & 3);
        if (pos < first || pos > last) x[i] = -INFINITY;
      }
    }
    float top = x[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) top = fmaxf(top, x[i]);
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
        const float b = pr[4 * s + 8 * (i >> 1) + 2 * (i & 1) + 1];
        hi[i] = pack16<false>(a, b);
        if constexpr (!BF) lo[i] = pack16<false>(a - lo16<false>(hi[i]), b - hi16<false>(hi[i]));
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

  int blk = rg.blk0;
  if (blk < b1) {
    // the channels of the m operand that stand for no group
    for (int i = threadIdx.x; i < 2 * PS * 64; i += 256)
      lds[i / (PS * 64)].m[i / 64 % PS][i % 64] = u32x4v{0u, 0u, 0u, 0u};
    int pg[PS], nx[PS], more[PS];
#pragma unroll
    for (int i = 0; i < PS; ++i) {
      pg[i] = look_up(blk + i);
      nx[i] = look_up(blk + PS + i);
    }
    fetch(blk + mine, mine ? pg[1] : pg[0]);
    __syncthreads();
    unpack(lds[0], blk + mine, mine ? pg[1] : pg[0]);
    __syncthreads();
    int buf = 0;
    for (;;) {
      const int next = blk + PS;
      if (next < b1) {
#pragma unroll
        for (int i = 0; i < PS; ++i) more[i] = look_up(next + PS + i);
        fetch(next + mine, mine ? nx[1] : nx[0]);
      }
#pragma unroll
      for (int i = 0; i < PS; ++i) {
        const int t0 = 32 * (blk + i);
        if (valid(blk + i, pg[i]) && t0 < whi && t0 + 32 > wlo) process(lds[buf], i, t0);
      }
      if (next >= b1) break;
      unpack(lds[buf ^ 1], next + mine, mine ? nx[1] : nx[0]);
      __syncthreads();
      buf ^= 1;
      blk = next;
#pragma unroll
      for (int i = 0; i < PS; ++i) {
        pg[i] = nx[i];
        nx[i] = more[i];
      }
    }
  }

  sum += __shfl_xor(sum, 32);
  if (w.chunks > 1) {
    float* po = p.part_o + (size_t)(w.slot0 + w.chunk) * PTC * D;
#pragma unroll
    for (int t = 0; t < CT; ++t)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        *reinterpret_cast<f32x4*>(po + (((wave * CT + t) * 4 + k) * 64 + lane) * 4) =
            f32x4{o[t][4 * k], o[t][4 * k + 1], o[t][4 * k + 2], o[t][4 * k + 3]};
    if (h == 0) {
      float* ml = p.part_ml + ((size_t)(w.slot0 + w.chunk) * PTC + 32 * wave + c) * 2;
      ml[0] = ref;
      ml[1] = sum;
    }
    return;
  }
  if (!live) return;
  const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
  uint16_t* dst = p.out + (size_t)row * p.ldo + (size_t)qh * D + 4 * h;
#pragma unroll
  for (int t = 0; t < CT; ++t)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      *reinterpret_cast<u32x2v*>(dst + 32 * t + 8 * k) =
          u32x2v{pack16<BF>(o[t][4 * k] * inv, o[t][4 * k + 1] * inv),
                 pack16<BF>(o[t][4 * k + 2] * inv, o[t][4 * k + 3] * inv)};
  if (h == 0 && p.lse != nullptr)
    p.lse[(size_t)row * p.q_heads + qh] = (ref + log2f(sum) - kKv4Lift) * 0.6931471805599453f;
}

// Joins a tile's chunks, in their order.  Grid: (tiles, D / 8): a workgroup has 8 channels of
// the tile's 128 columns, a thread 4 of one.
template <int D, bool BF>
__global__ __launch_bounds__(256) void kv4_prefill_join_kernel(Kv4AttendArgs p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = lane & 31, h = lane >> 5, t = blockIdx.y >> 2, k = blockIdx.y & 3;
  const int ratio = p.q_heads / p.heads;
  Kv4Place w;
  if (!kv4_place_chunk<PTC, true>(p, blockIdx.x, w) || w.chunks == 1) return;
  const int col = w.tile * PTC + 32 * wave + c, ci = col / ratio;
  if (ci >= w.s.n) return;
  const int qh = w.head * ratio + col % ratio, row = w.s.first + ci;
  float m = kKv4None, l = 0.f;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int i = 0; i < w.chunks; ++i) {
    const size_t slot = w.slot0 + i;
    const float* ml = p.part_ml + (slot * PTC + 32 * wave + c) * 2;
    const f32x4 v = *reinterpret_cast<const f32x4*>(
        p.part_o + slot * PTC * D + (((wave * (D / 32) + t) * 4 + k) * 64 + lane) * 4);
    const float cm = ml[0], cl = ml[1];
    const float next = fmaxf(m, cm);
    const float a = __builtin_amdgcn_exp2f(m - next), f = __builtin_amdgcn_exp2f(cm - next);
    m = next;
    l = l * a + cl * f;
    o = o * a + v * f;
  }
  o *= l > 0.f || l != l ? 1.f / l : 0.f;
  *reinterpret_cast<u32x2v*>(p.out + (size_t)row * p.ldo + (size_t)qh * D + 32 * t + 8 * k + 4 * h) =
      u32x2v{pack16<BF>(o[0], o[1]), pack16<BF>(o[2], o[3])};
  if (blockIdx.y == 0 && h == 0 && p.lse != nullptr)
    p.lse[(size_t)row * p.q_heads + qh] = (m + log2f(l) - kKv4Lift) * 0.6931471805599453f;
}

typedef void (*PrefillFn)(Kv4AttendArgs);
template <bool BF>
PrefillFn prefill_kernel(int D, int groups) {
  if (D == 128)
    return groups == 1 ? kv4_prefill_kernel<128, 1, BF>
                       : groups == 2 ? kv4_prefill_kernel<128, 2, BF> : kv4_prefill_kernel<128, 4, BF>;
  return groups == 1 ? kv4_prefill_kernel<64, 1, BF> : kv4_prefill_kernel<64, 2, BF>;
}

}  // namespace

hipError_t launch_kv4_prefill(const Kv4AttendArgs& a, int D, int groups, bool bf, hipStream_t st) {
  const long long units = ((long long)a.heads * a.batch + 7) / 8 * 8;
  const unsigned grid = a.slots ? a.slots : (unsigned)(units * a.col_tiles);
  hipLaunchKernelGGL(bf ? prefill_kernel<true>(D, groups) : prefill_kernel<false>(D, groups),
                     kv4_grid(grid), dim3(256), 0, st, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.slots == 0) return e;
  auto join = D == 128 ? (bf ? kv4_prefill_join_kernel<128, true> : kv4_prefill_join_kernel<128, false>)
                       : (bf ? kv4_prefill_join_kernel<64, true> : kv4_prefill_join_kernel<64, false>);
  hipLaunchKernelGGL(join, dim3(a.tiles, D / 8), dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace w4a16
