// Writing new tokens into the 4-bit cache, and reading tokens back from it (kv4.h has the
// format).
//
// One wave serves the tokens of one block of 32 of one kv head, keys or values: it owns
// every word it writes, so nothing needs an atomic and tokens that were in the block before
// keep their bits.  A lane loads 8 channels of a token at a time in the order of K's words
// (token l%16, channels 32 j + 8 (l/16)), so a group's minimum and maximum take two lane
// exchanges and K's words are stored as they stand.  V's words hold 8 tokens of a channel
// instead: the same words go through LDS and an 8 x 8 transposition of nibbles in registers.
//
// Bound: HBM and vector instructions.  Prompts of 9 requests (13807 tokens, 8 kv heads of 128
// bf16 channels): 25 us written (74 MB, 3.0 TB/s; a large copy: 4.9, a sum of two arrays: 5.9), 17 us read back (4.3
// TB/s); one token of each of 64 requests: 5.7 us and 3.6 us, chains of dependent loads.  The
// quotient by the divider for every code took 28 us and 8.4 us.
#include "kv4.h"

namespace w4a16 {

namespace {

// 8 x 8 nibbles: nibble j of word i becomes nibble i of word j.
__device__ __forceinline__ void transpose_nibbles(uint32_t* w) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = w[i], b = w[i + 4];
    w[i] = (a & 0xFFFFu) | (b << 16);
    w[i + 4] = (a >> 16) | (b & 0xFFFF0000u);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int i = (k & 1) + 4 * (k >> 1);
    const uint32_t a = w[i], b = w[i + 2];
    w[i] = (a & 0x00FF00FFu) | ((b & 0x00FF00FFu) << 8);
    w[i + 2] = ((a >> 8) & 0x00FF00FFu) | (b & 0xFF00FF00u);
  }
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const uint32_t a = w[i], b = w[i + 1];
    w[i] = (a & 0x0F0F0F0Fu) | ((b & 0x0F0F0F0Fu) << 4);
    w[i + 1] = ((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u);
  }
}

// index of channel c's word of V (tokens of lane group g) in the block's V words
__device__ __forceinline__ int v_word(int c, int g) {
  return ((c >> 6) * 64 + 16 * g + (c & 15)) * 4 + ((c >> 4) & 3);
}

// Grid: (blocks a sequence's new tokens can touch, kv heads x {K, V}, sequences).
template <int D, int NG, bool BF>
__global__ __launch_bounds__(64) void kv4_append_kernel(Kv4CacheArgs p) {
  constexpr int J = D / 32;
  constexpr int JG = J / NG;  // words of a token and lane in one group
  __shared__ uint32_t words[32][D / 8 + 1];
  const int lane = threadIdx.x;
  const int r = lane & 15, g = lane >> 4;
  const int head = blockIdx.y >> 1, is_v = blockIdx.y & 1, b = blockIdx.z;
  const Kv4Seq s = kv4_seq(p.rows, p.lens, b, p.tokens, p.max_new);
  const int from = s.len - s.n;  // position of the first new token
  const int start = from < 0 ? 0 : from;
  const int blk = start / 32 + blockIdx.x;
  if (blk * 32 >= s.len || s.n <= 0) return;
  const int page = kv4_page(p.table, b, blk, p.page / 32, p.width, p.pages);
  if (page < 0) return;
  char* block = p.cache + ((size_t)page * p.heads + head) * (size_t)(p.page / 32) *
                              kv4_block_bytes(D, NG) +
                (size_t)(blk % (p.page / 32)) * kv4_block_bytes(D, NG);
  const uint16_t* src = is_v ? p.v : p.k;
  const size_t ld = is_v ? p.ldv : p.ldk;
  uint16_t* params = reinterpret_cast<uint16_t*>(block + 32 * D + (is_v ? 128 * NG : 0));
  // V's words: 8 channels of a lane, the tokens of lane group tg; those that also hold other
  // tokens are fetched while the new ones are worked on
  const int oct = lane >> 2, tg = lane & 3;
  uint32_t* vdst = reinterpret_cast<uint32_t*>(block + 16 * D);
  uint32_t old[8], mask = 0;
  if (is_v && oct < D / 8) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int pos = blk * 32 + kv4_slot_token(tg, e);
      if (pos >= start && pos < s.len) mask |= 15u << (4 * nib_pos(e));
    }
    if (mask != 0 && mask != 0xFFFFFFFFu) {
#pragma unroll
      for (int e = 0; e < 8; ++e) old[e] = vdst[v_word(8 * oct + e, tg)];
    }
  }
  uint32_t word[2][J];
  bool fresh[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int pos = blk * 32 + 16 * t + r;
    fresh[t] = pos >= start && pos < s.len;
#pragma unroll
    for (int j = 0; j < J; ++j) word[t][j] = 0;
    if (__ballot(fresh[t]) == 0) continue;
    u32x4v x[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      x[j] = u32x4v{0u, 0u, 0u, 0u};
      if (fresh[t])
        x[j] = *reinterpret_cast<const u32x4v*>(src + (size_t)(s.first + pos - from) * ld +
                                                (size_t)head * D + 32 * j + 8 * g);
    }
#pragma unroll
    for (int q = 0; q < NG; ++q) {
      float f[JG][8];
      float lo = INFINITY, hi = -INFINITY, bad = 0.f;
#pragma unroll
      for (int j = 0; j < JG; ++j) {
        unpack8<BF>(x[q * JG + j], f[j]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (f[j][e] != f[j][e]) bad = NAN;
          f[j][e] = fminf(fmaxf(f[j][e], -65504.f), 65504.f);
          lo = fminf(lo, f[j][e]);
          hi = fmaxf(hi, f[j][e]);
        }
      }
#pragma unroll
      for (int off = 16; off <= 32; off <<= 1) {
        lo = fminf(lo, __shfl_xor(lo, off));
        hi = fmaxf(hi, __shfl_xor(hi, off));
        bad += __shfl_xor(bad, off);
      }
      // a NaN makes the whole group read as NaN
      const _Float16 mh = (_Float16)(lo + bad), sh = (_Float16)((hi - lo) / 15.f);
      const float m = (float)mh, sc = (float)sh;
      if (g == 0 && fresh[t]) {
        uint16_t* at = params + q * 64 + kv4_token_slot(16 * t + r);
        at[0] = __builtin_bit_cast(uint16_t, sh);
        at[32] = __builtin_bit_cast(uint16_t, mh);
      }
      // (x - m) / s rounded: a product with 1 / s is off by less than 3e-6 of a code, so only
      // where one lies closer to a half than that the quotient itself has to decide
      const float inv = sc > 0.f ? __builtin_amdgcn_rcpf(sc) : 0.f;
      bool close = false;
#pragma unroll
      for (int j = 0; j < JG; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float c = (f[j][e] - m) * inv, n = __builtin_rintf(c);
          close |= fabsf(c - n) > 0.49999f;
          word[t][q * JG + j] |= (uint32_t)(int)fminf(fmaxf(n, 0.f), 15.f) << (4 * nib_pos(e));
        }
      if (__ballot(close) != 0) {
#pragma unroll
        for (int j = 0; j < JG; ++j) {
          uint32_t w = 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float c = sc > 0.f ? __builtin_rintf((f[j][e] - m) / sc) : 0.f;
            w |= (uint32_t)(int)fminf(fmaxf(c, 0.f), 15.f) << (4 * nib_pos(e));
          }
          word[t][q * JG + j] = w;
        }
      }
    }
  }
  if (!is_v) {
    uint32_t* dst = reinterpret_cast<uint32_t*>(block);
#pragma unroll
    for (int t = 0; t < 2; ++t)
      if (fresh[t]) {
        uint32_t* at = dst + (t * 64 + lane) * J;
        if constexpr (J == 4)
          *reinterpret_cast<u32x4v*>(at) =
              u32x4v{word[t][0], word[t][1], word[t][2], word[t][3]};
        else
          *reinterpret_cast<u32x2v*>(at) = u32x2v{word[t][0], word[t][1]};
      }
    return;
  }
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int j = 0; j < J; ++j) words[16 * t + r][4 * j + g] = word[t][j];
  __syncthreads();
  if (mask == 0) return;  // also the lanes past D / 8
  uint32_t w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) w[nib_pos(e)] = words[kv4_slot_token(tg, e)][oct];
  transpose_nibbles(w);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t x = w[nib_pos(e)];
    vdst[v_word(8 * oct + e, tg)] = mask == 0xFFFFFFFFu ? x : (old[e] & ~mask) | (x & mask);
  }
}

// The values of the same tokens, read from the cache into rows of k and v (zeros where the
// table has no page).  Same grid.
template <int D, int NG, bool BF>
__global__ __launch_bounds__(64) void kv4_gather_kernel(Kv4GatherArgs p) {
  constexpr int J = D / 32;
  constexpr int G = D / NG;
  const int lane = threadIdx.x;
  const int head = blockIdx.y >> 1, is_v = blockIdx.y & 1, b = blockIdx.z;
  const Kv4Seq s = kv4_seq(p.rows, p.lens, b, p.tokens, p.max_new);
  const int from = s.len - s.n;
  const int start = from < 0 ? 0 : from;
  const int blk = start / 32 + blockIdx.x;
  if (blk * 32 >= s.len || s.n <= 0) return;
  const int page = kv4_page(p.table, b, blk, p.page / 32, p.width, p.pages);
  const char* block = p.cache + ((size_t)(page < 0 ? 0 : page) * p.heads + head) *
                                    (size_t)(p.page / 32) * kv4_block_bytes(D, NG) +
                      (size_t)(blk % (p.page / 32)) * kv4_block_bytes(D, NG);
  uint16_t* out = is_v ? p.v : p.k;
  const size_t ld = is_v ? p.ldv : p.ldk;
  const _Float16* params =
      reinterpret_cast<const _Float16*>(block + 32 * D + (is_v ? 128 * NG : 0));
  // eight channels 8 oct .. + 7 of token t of the block, in nibble order in w
  auto put = [&](int t, int oct, uint32_t w) {
    const int pos = blk * 32 + t;
    if (pos < start || pos >= s.len) return;
    float f[8];
    if (page < 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = 0.f;
    } else {
      const _Float16* at = params + (8 * oct / G) * 64 + kv4_token_slot(t);
      const float sc = (float)at[0], m = (float)at[32];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        f[e] = __builtin_fmaf(sc, (float)((w >> (4 * nib_pos(e))) & 15u), m);
    }
    *reinterpret_cast<u32x4v*>(out + (size_t)(s.first + pos - from) * ld + (size_t)head * D +
                               8 * oct) = pack8<BF>(f);
  };
  if (!is_v) {
    const uint32_t* src = reinterpret_cast<const uint32_t*>(block);
    const int r = lane & 15, g = lane >> 4;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int j = 0; j < J; ++j) put(16 * t + r, 4 * j + g, src[(t * 64 + lane) * J + j]);
    return;
  }
  const int oct = lane >> 2, tg = lane & 3;
  if (oct >= D / 8) return;
  const uint32_t* src = reinterpret_cast<const uint32_t*>(block + 16 * D);
  uint32_t w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) w[nib_pos(e)] = src[v_word(8 * oct + e, tg)];
  transpose_nibbles(w);
#pragma unroll
  for (int e = 0; e < 8; ++e) put(kv4_slot_token(tg, e), oct, w[nib_pos(e)]);
}

template <bool BF, template <int, int, bool> class F, class Args>
void by_layout(int D, int groups, dim3 grid, hipStream_t st, const Args& a) {
  if (D == 128) {
    if (groups == 1) F<128, 1, BF>::run(grid, st, a);
    else if (groups == 2) F<128, 2, BF>::run(grid, st, a);
    else F<128, 4, BF>::run(grid, st, a);
  } else {
    if (groups == 1) F<64, 1, BF>::run(grid, st, a);
    else F<64, 2, BF>::run(grid, st, a);
  }
}
template <int D, int NG, bool BF>
struct Append {
  static void run(dim3 grid, hipStream_t st, const Kv4CacheArgs& a) {
    hipLaunchKernelGGL((kv4_append_kernel<D, NG, BF>), grid, dim3(64), 0, st, a);
  }
};
template <int D, int NG, bool BF>
struct Gather {
  static void run(dim3 grid, hipStream_t st, const Kv4GatherArgs& a) {
    hipLaunchKernelGGL((kv4_gather_kernel<D, NG, BF>), grid, dim3(64), 0, st, a);
  }
};

// blocks of 32 that max_new tokens in a row can touch
unsigned touched(int max_new) { return (unsigned)(((long long)max_new + 62) / 32); }

}  // namespace

hipError_t launch_kv4_append(const Kv4CacheArgs& a, int D, int groups, bool bf, hipStream_t st) {
  const dim3 grid(touched(a.max_new), 2 * a.heads, a.batch);
  if (bf) by_layout<true, Append>(D, groups, grid, st, a);
  else by_layout<false, Append>(D, groups, grid, st, a);
  return hipGetLastError();
}

hipError_t launch_kv4_gather(const Kv4GatherArgs& a, int D, int groups, bool bf, hipStream_t st) {
  const dim3 grid(touched(a.max_new), 2 * a.heads, a.batch);
  if (bf) by_layout<true, Gather>(D, groups, grid, st, a);
  else by_layout<false, Gather>(D, groups, grid, st, a);
  return hipGetLastError();
}

}  // namespace w4a16
