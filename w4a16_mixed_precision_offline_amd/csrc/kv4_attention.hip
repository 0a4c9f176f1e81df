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
//           only one beside that of the result: 1.6 to 1.3 times the error of rounding
//           alone, at 16 more matrix instructions a block, which a stream from HBM hides.
//   V^T p^T A = V = m_t + s_t c in fp16 (one rounding of the exact value, 2^-11), B = p, which
//           is where K q^T left it.  Values past 65504 (a group whose s was rounded up)
//           saturate (MODE.FP16_OVFL).
//
// A token is seen by a column if its position is at most the column's own, more than the
// column's less the window (window > 0), and its page is in the table.  Blocks that are
// not seen whole by every column take the masked path, which also clears s and m of
// the tokens that no column sees: what a page holds there may be anything.
// A column that sees nothing gives 0 and a log-sum of -infinity.
//
// Few columns and long contexts: the token axis is cut into chunks, one workgroup each,
// whose sums a second kernel joins in order.
#include "kv4.h"

namespace w4a16 {

namespace {

constexpr int AW = 4;              // waves of a workgroup, which share its blocks
constexpr float kLazy = 7.f;       // how far a logit may exceed the reference
constexpr float kLift = 8.f;       // p is held times 2^8
constexpr float kNone = -1e30f;    // reference of a column that has seen nothing

// fp16 results past 65504 become 65504 instead of infinity, for the rest of the wave
__device__ __forceinline__ void saturate_fp16() {
  __builtin_amdgcn_s_setreg((0 << 11) | (23 << 6) | 1, 1);  // MODE, bit 23, one bit
}

__device__ __forceinline__ half2v as_half2(uint32_t w) { return __builtin_bit_cast(half2v, w); }
__device__ __forceinline__ uint32_t as_word(half2v h) { return __builtin_bit_cast(uint32_t, h); }

// the eight codes of a word as fp16 subnormals, channels 2, 3, 6, 7 times 16
__device__ __forceinline__ half8v codes_subnormal(uint32_t w) {
  const uint32_t v = w >> 8;
  return __builtin_bit_cast(half8v, u32x4v{w & 0x000F000Fu, w & 0x00F000F0u, v & 0x000F000Fu,
                                           v & 0x00F000F0u});
}
// the eight values m + s c of a word; s and m of its tokens in the same order
__device__ __forceinline__ half8v values(uint32_t w, const u32x4v& s, const u32x4v& m) {
  const uint32_t v = w >> 8;
  const half2v one = {(_Float16)-1024.f, (_Float16)-1024.f};
  const half2v up = {(_Float16)0.0625f, (_Float16)0.0625f};
  const half2v off = {(_Float16)-64.f, (_Float16)-64.f};
  const half2v c0 = as_half2((w & 0x000F000Fu) | 0x64006400u) + one;
  const half2v c1 = __builtin_elementwise_fma(as_half2((w & 0x00F000F0u) | 0x64006400u), up, off);
  const half2v c2 = as_half2((v & 0x000F000Fu) | 0x64006400u) + one;
  const half2v c3 = __builtin_elementwise_fma(as_half2((v & 0x00F000F0u) | 0x64006400u), up, off);
  return __builtin_bit_cast(
      half8v, u32x4v{as_word(__builtin_elementwise_fma(c0, as_half2(s[0]), as_half2(m[0]))),
                     as_word(__builtin_elementwise_fma(c1, as_half2(s[1]), as_half2(m[1]))),
                     as_word(__builtin_elementwise_fma(c2, as_half2(s[2]), as_half2(m[2]))),
                     as_word(__builtin_elementwise_fma(c3, as_half2(s[3]), as_half2(m[3])))});
}

// One block of 32 tokens of one kv head in a wave's registers.
template <int D, int NG>
struct Block {
  uint32_t k[2][D / 32];
  u32x4v v[D / 64];
  u32x4v ks[NG], km[NG], vs[NG], vm[NG];

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
#pragma unroll
    for (int q = 0; q < NG; ++q) {
      ks[q] = *reinterpret_cast<const u32x4v*>(par + 128 * q);
      km[q] = *reinterpret_cast<const u32x4v*>(par + 128 * q + 64);
      vs[q] = *reinterpret_cast<const u32x4v*>(par + 128 * (NG + q));
      vm[q] = *reinterpret_cast<const u32x4v*>(par + 128 * (NG + q) + 64);
    }
  }
};

__device__ __forceinline__ float half_at(const u32x4v& v, int e) {
  return e & 1 ? hi16<false>(v[e >> 1]) : lo16<false>(v[e >> 1]);
}

// Grid: chunks x column tiles x kv heads x sequences, chunks fastest.
template <int D, int NG, bool BF>
__global__ __launch_bounds__(64 * AW) void kv4_attend_kernel(Kv4AttendArgs p) {
  constexpr int J = D / 32, JG = J / NG, NT = D / 16;
  __shared__ f32x4 red_o[AW][NT][64];
  __shared__ float red_m[AW][16], red_l[AW][16];
  saturate_fp16();
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int r = lane & 15, g = lane >> 4;
  unsigned id = blockIdx.x;
  const int chunk = id % p.chunks;
  id /= p.chunks;
  const int tile = id % p.col_tiles;
  id /= p.col_tiles;
  const int head = id % p.heads, b = id / p.heads;
  const int ratio = p.q_heads / p.heads;
  const Kv4Seq s = kv4_seq(p.rows, p.lens, b, p.tokens, p.max_new);
  const int i0 = tile * 16 / ratio;               // first and last new token of the tile
  if (i0 >= s.n) return;
  const int i1 = (tile * 16 + 15) / ratio < s.n - 1 ? (tile * 16 + 15) / ratio : s.n - 1;
  const int from = s.len - s.n;
  const int col = tile * 16 + r, ci = col / ratio;
  const bool live = ci < s.n;
  const int qh = head * ratio + col % ratio;
  const int row = s.first + (live ? ci : 0);
  // tokens seen: column [first, last], any column [lo, hi), every column [all_lo, all_hi)
  const int last = live ? from + ci : -1;
  const int first = p.window > 0 ? last - p.window + 1 : 0;
  const int hi = from + i1 + 1;
  int lo = p.window > 0 ? from + i0 - p.window + 1 : 0;
  lo = lo < 0 ? 0 : lo;
  const int all_hi = from + i0 + 1;
  const int all_lo = p.window > 0 ? from + i1 - p.window + 1 : 0;

  // q, scaled, and its sums per group of channels (times 2^-24, the codes' unit)
  half8v qf[J];
  float qsum[NG], cf;
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
    int d = 15 - ((int)(__float_as_uint(top) >> 23) - 127);
    d = top == 0.f ? 0 : d < -112 ? -112 : d > 100 ? 100 : d;
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
      qf[j] = __builtin_bit_cast(half8v, pack8<false>(h));
    }
#pragma unroll
    for (int q = 0; q < NG; ++q) {
      qsum[q] += __shfl_xor(qsum[q], 16);
      qsum[q] += __shfl_xor(qsum[q], 32);
      qsum[q] *= 0x1p-24f;
    }
    cf = __builtin_ldexpf(p.scale * 1.4426950408889634f, 24 - d);
  }

  f32x4 o[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) o[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  float ref = kNone, sum = 0.f;

  // this workgroup's blocks: its chunk of [lo, hi), the last chunk taking what is left
  const int b0 = lo / 32 + chunk * (p.chunk / 32);
  const int end = (hi + 31) / 32;
  const int b1 = chunk == p.chunks - 1 || b0 + p.chunk / 32 > end ? end
                                                                           : b0 + p.chunk / 32;
  const int page_blocks = p.page / 32;
  const size_t page_bytes = (size_t)p.heads * page_blocks * kv4_block_bytes(D, NG);
  const char* head_base = p.cache + (size_t)head * page_blocks * kv4_block_bytes(D, NG);
  const int* table = p.table + (size_t)b * p.width;

  auto process = [&](Block<D, NG>& kv, int blk) {
    const int t0 = blk * 32;
    // logits of the lane's 8 tokens kv4_slot_token(g, e)
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.f;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int q = 0; q < NG; ++q) {
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < JG; ++j)
          acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes_subnormal(kv.k[t][q * JG + j]),
                                                       qf[q * JG + j], acc, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = 4 * t + i;
          x[e] = __builtin_fmaf(half_at(kv.ks[q], e), acc[i],
                                __builtin_fmaf(half_at(kv.km[q], e), qsum[q], x[e]));
        }
      }
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= cf;
    if (t0 < all_lo || t0 + 32 > all_hi) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int pos = t0 + kv4_slot_token(g, e);
        if (pos < first || pos > last) x[e] = -INFINITY;
        if (pos < lo || pos >= hi) {
#pragma unroll
          for (int q = 0; q < NG; ++q) {
            const uint32_t keep = e & 1 ? 0x0000FFFFu : 0xFFFF0000u;
            kv.vs[q][e >> 1] &= keep;
            kv.vm[q][e >> 1] &= keep;
          }
        }
      }
    }
    float top = x[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) top = fmaxf(top, x[e]);
    if (__ballot(top > ref + kLazy) != 0) {
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      const float next = fmaxf(ref, top);
      const float f = __builtin_amdgcn_exp2f(ref - next);
      ref = next;
      sum *= f;
#pragma unroll
      for (int t = 0; t < NT; ++t) o[t] *= f;
    }
    float pr[8], rest[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      pr[e] = __builtin_amdgcn_exp2f(x[e] - ref + kLift);
      sum += pr[e];
    }
    const u32x4v pw = pack8<false>(pr);
    const half8v ph = __builtin_bit_cast(half8v, pw);
    half8v pl;
    if constexpr (!BF) {
#pragma unroll
      for (int e = 0; e < 8; ++e) rest[e] = pr[e] - half_at(pw, e);
      pl = __builtin_bit_cast(half8v, pack8<false>(rest));
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int q = t * 16 / (D / NG);
      const half8v vf = values(kv.v[t >> 2][t & 3], kv.vs[q], kv.vm[q]);
      o[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, ph, o[t], 0, 0, 0);
      if constexpr (!BF) o[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, pl, o[t], 0, 0, 0);
    }
  };

  // A wave's blocks b0 + wave, + AW, ...: the next block's loads are in flight while one is
  // worked on, and its page number is fetched one block earlier still.  Blocks without a
  // page are passed over; a load past the last block reads the last one again.
  int blk = b0 + wave;
  int entry = blk / page_blocks, off = blk - entry * page_blocks;
  auto look_up = [&]() {
    const int pg = entry < p.width && blk < b1 ? table[entry] : -1;
    return pg >= 0 && pg < p.pages ? pg : -1;
  };
  auto advance = [&]() {
    blk += AW;
    off += AW;
    while (off >= page_blocks) {
      off -= page_blocks;
      ++entry;
    }
  };
  auto base_of = [&](int pg, int o_) {
    return head_base + (size_t)(pg < 0 ? 0 : pg) * page_bytes +
           (size_t)o_ * kv4_block_bytes(D, NG);
  };
  if (blk < b1) {
    Block<D, NG> kv0, kv1;
    int pg0 = look_up(), blk0 = blk;
    kv0.load(base_of(pg0, off), lane);
    advance();
    int pg1 = look_up(), blk1 = blk, off1 = off;
    for (;;) {
      kv1.load(base_of(pg1, off1), lane);
      advance();
      int pgn = look_up(), offn = off;
      if (pg0 >= 0) process(kv0, blk0);
      if (blk1 >= b1) break;
      pg0 = pgn;
      blk0 = blk;
      kv0.load(base_of(pg0, offn), lane);
      advance();
      pgn = look_up();
      offn = off;
      if (pg1 >= 0) process(kv1, blk1);
      if (blk0 >= b1) break;
      pg1 = pgn;
      blk1 = blk;
      off1 = offn;
    }
  }

  // join the waves
  sum += __shfl_xor(sum, 16);
  sum += __shfl_xor(sum, 32);
#pragma unroll
  for (int t = 0; t < NT; ++t) red_o[wave][t][lane] = o[t];
  if (g == 0) {
    red_m[wave][r] = ref;
    red_l[wave][r] = sum;
  }
  __syncthreads();
  float m = kNone, l = 0.f, f[AW];
#pragma unroll
  for (int w = 0; w < AW; ++w) m = fmaxf(m, red_m[w][r]);
#pragma unroll
  for (int w = 0; w < AW; ++w) {
    f[w] = __builtin_amdgcn_exp2f(red_m[w][r] - m);
    l += f[w] * red_l[w][r];
  }
  if (!live) return;
  const size_t at = (size_t)row * p.q_heads + qh;
  const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
  for (int k = 0; k < NT / AW; ++k) {
    const int t = wave + AW * k;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < AW; ++w) v += red_o[w][t][lane] * f[w];
    if (p.chunks > 1) {
      *reinterpret_cast<f32x4*>(
          p.part_o + ((size_t)chunk * p.tokens * p.q_heads + at) * D + 16 * t + 4 * g) = v;
    } else {
      v *= inv;
      *reinterpret_cast<u32x2v*>(p.out + (size_t)row * p.ldo + (size_t)qh * D + 16 * t + 4 * g) =
          u32x2v{pack16<BF>(v[0], v[1]), pack16<BF>(v[2], v[3])};
    }
  }
  if (wave == 0 && g == 0) {
    if (p.chunks > 1) {
      float* ml = p.part_ml + 2 * ((size_t)chunk * p.tokens * p.q_heads + at);
      ml[0] = m;
      ml[1] = l;
    } else if (p.lse != nullptr) {
      p.lse[at] = (m + log2f(l) - kLift) * 0.6931471805599453f;
    }
  }
}

// Joins the chunks of a (token, query head): one workgroup, D / 4 lanes to a chunk, so that
// a thread's loads do not wait for each other; the lanes' sums meet in LDS in order.
// Grid: (new tokens of a sequence, query heads, sequences).
template <int D, bool BF>
__global__ __launch_bounds__(256) void kv4_join_kernel(Kv4AttendArgs p) {
  constexpr int L = D / 4, NC = 256 / L;
  __shared__ f32x4 red_o[NC][L];
  __shared__ float red_m[NC], red_l[NC];
  saturate_fp16();
  const Kv4Seq s = kv4_seq(p.rows, p.lens, blockIdx.z, p.tokens, p.max_new);
  if ((int)blockIdx.x >= s.n) return;
  const int qh = blockIdx.y, z = threadIdx.x / L, c = threadIdx.x % L;
  const int row = s.first + blockIdx.x;
  const size_t at = (size_t)row * p.q_heads + qh, step = (size_t)p.tokens * p.q_heads;
  float m = kNone, l = 0.f;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  auto add = [&](float mk, float lk, const f32x4& v) {
    const float next = fmaxf(m, mk);
    const float a = __builtin_amdgcn_exp2f(m - next), f = __builtin_amdgcn_exp2f(mk - next);
    m = next;
    l = l * a + lk * f;
    o = o * a + v * f;
  };
#pragma unroll 4
  for (int k = z; k < p.chunks; k += NC) {
    const float* ml = p.part_ml + 2 * (k * step + at);
    add(ml[0], ml[1], *reinterpret_cast<const f32x4*>(p.part_o + (k * step + at) * D + 4 * c));
  }
  red_o[z][c] = o;
  if (c == 0) {
    red_m[z] = m;
    red_l[z] = l;
  }
  __syncthreads();
  if (z != 0) return;
#pragma unroll
  for (int k = 1; k < NC; ++k) add(red_m[k], red_l[k], red_o[k][c]);
  o *= l > 0.f || l != l ? 1.f / l : 0.f;
  *reinterpret_cast<u32x2v*>(p.out + (size_t)row * p.ldo + (size_t)qh * D + 4 * c) =
      u32x2v{pack16<BF>(o[0], o[1]), pack16<BF>(o[2], o[3])};
  if (c == 0 && p.lse != nullptr) p.lse[at] = (m + log2f(l) - kLift) * 0.6931471805599453f;
}

typedef void (*AttendFn)(Kv4AttendArgs);
template <bool BF>
AttendFn attend_kernel(int D, int groups) {
  if (D == 128)
    return groups == 1 ? kv4_attend_kernel<128, 1, BF>
                       : groups == 2 ? kv4_attend_kernel<128, 2, BF> : kv4_attend_kernel<128, 4, BF>;
  return groups == 1 ? kv4_attend_kernel<64, 1, BF> : kv4_attend_kernel<64, 2, BF>;
}

}  // namespace

Kv4AttendPlan kv4_attend_plan(int batch, int tokens, int max_new, int max_len, int q_heads,
                              int heads, int D, int window) {
  Kv4AttendPlan p;
  p.col_tiles = (int)(((long long)max_new * (q_heads / heads) + 15) / 16);
  // tokens any tile can see: the window of its first token up to its last
  long long span = max_len;
  if (window > 0 && span > (long long)window + 47) span = (long long)window + 47;
  const long long wgs = (long long)p.col_tiles * heads * batch;
  long long chunks = (1024 + wgs - 1) / wgs;
  long long chunk = (span + chunks - 1) / chunks;
  chunk = chunk < 256 ? 256 : (chunk + 31) / 32 * 32;
  p.chunk = (int)chunk;
  p.chunks = (int)((span + chunk - 1) / chunk);
  if (p.chunks < 1) p.chunks = 1;
  p.floats = p.chunks > 1 ? (size_t)p.chunks * tokens * q_heads * (D + 2) : 0;
  return p;
}

hipError_t launch_kv4_attend(const Kv4AttendPlan& plan, const Kv4AttendArgs& args, int D, int groups,
                             bool bf, hipStream_t st) {
  Kv4AttendArgs a = args;
  a.chunk = plan.chunk;
  a.chunks = plan.chunks;
  a.col_tiles = plan.col_tiles;
  const dim3 grid((unsigned)plan.chunks * plan.col_tiles * a.heads * a.batch);
  hipLaunchKernelGGL(bf ? attend_kernel<true>(D, groups) : attend_kernel<false>(D, groups), grid,
                     dim3(64 * AW), 0, st, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || plan.chunks == 1) return e;
  const dim3 jgrid(a.max_new, a.q_heads, a.batch);
  auto join = D == 128 ? (bf ? kv4_join_kernel<128, true> : kv4_join_kernel<128, false>)
                       : (bf ? kv4_join_kernel<64, true> : kv4_join_kernel<64, false>);
  hipLaunchKernelGGL(join, jgrid, dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace w4a16
