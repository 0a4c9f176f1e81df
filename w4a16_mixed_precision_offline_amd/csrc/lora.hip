// Low-rank adapters of many requests beside one projection.
//
//   Y[m] = base[m] + scale[a] * (X[m] A[a]^T) B[a]^T,   a = ids[m]  (none: Y[m] = base[m])
//
// Two products: T = X A^T has r <= 128 columns and the whole of K to sum over, Y = T B^T has
// r to sum over and all of N to write.  So T's sum is split over K across workgroups (each
// slice writes its fp32 part, the second kernel adds the slices in order: the same bits
// every time, no atomics), and the second kernel is split over N.
//
// Rows are taken in tiles.  Of the rows of a tile that share an adapter the first is the
// leader: a leader's products run over the whole tile (a matrix instruction's 16 columns are
// there anyway) and only its own adapter's rows are kept.  One prompt per adapter gives
// one leader per tile; a decode batch of different adapters gives one per row, and each
// adapter is read once per tile, which is what bounds such a batch.
//
// T is held in fp32.  For the second product it goes to the matrix instruction as a sum of
// two 16-bit numbers, hi + lo: 22 bits in fp16 (after a power of two per row that puts its
// largest |T| in [1, 2), so that neither overflow nor underflow touches it), 16 bits in
// bf16, whose own step is 2^-9.
//
// Bound: HBM for many rows, latency for few.  4096 rows, 8192 x 8192, rank 64: 79 us a call for
// 201 MB of X, base and Y, 2.5 TB/s (a sum of two arrays: 5.9): X A^T 28 us (67 MB, its loads
// four steps at a time; 37 us one at a time), the split 5 us, T B^T 36 us (134 MB).  48 rows
// with 40 adapters of rank 16, 8192 x 10240: 6.2 and 8.0 us in the kernels, 15.2 a call; one row,
// 4096 x 4096: 3.3 and 3.9 us, 9.7 a call.  2048 rows of rank 128: 88 us (39, 9 and 35): X A^T
// with 128 KiB of LDS, one workgroup to a compute unit, T B^T with 20 to 23 registers spilled.
// Measured, not kept: the slices joined by the last workgroup to arrive (the kernels of 4096
// rows together 80 us instead of 69).
#include "internal.h"
#include "rows16.h"

namespace w4a16 {

namespace {

constexpr int LW = 4;  // waves of a workgroup

template <bool BF>
__device__ __forceinline__ f32x4 mfma16(const u32x4v& a, const u32x4v& b, const f32x4& c) {
  if constexpr (BF)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8v, a),
                                                   __builtin_bit_cast(bf16x8v, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8v, a),
                                                  __builtin_bit_cast(half8v, b), c, 0, 0, 0);
}

// Lane l's adapter: that of row m0 + l of a tile of 16 * TM rows (-1: none).
template <int TM>
__device__ __forceinline__ int tile_id(const int* ids, int m0, int M, int adapters) {
  const int lane = threadIdx.x & 63;
  const int id = lane < 16 * TM && m0 + lane < M ? ids[m0 + lane] : -1;
  return id >= 0 && id < adapters ? id : -1;
}
// The leaders a workgroup still has to serve, as a mask of the rows it may look at: all of
// the tile (TM > 1), or row z alone, if no earlier row has its adapter (TM == 1).
template <int TM>
__device__ __forceinline__ uint64_t tile_todo(int id, int z) {
  if constexpr (TM > 1) return __ballot(id >= 0);
  const int a = __builtin_amdgcn_readlane(id, z);
  const uint64_t same = __ballot(id == a && id >= 0);
  return same != 0 && __builtin_ctzll(same) == z ? same : 0;
}

// Sums one row's slices of T (columns 8 g .. of every 32) and splits the sum into operands
// hi and lo, 64 lanes apart for each 32 columns; returns the power of two that they were
// divided by.
template <int KR, bool BF>
__device__ __forceinline__ float split_row(const float* T, size_t step, int slices, size_t row,
                                           int rank, int g, bool live, u32x4v* hi, u32x4v* lo) {
  float v[KR][8];
  float top = 0.f;
#pragma unroll
  for (int q = 0; q < KR; ++q) {
    const int c = 32 * q + 8 * g;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[q][e] = 0.f;
    if (live && c < rank) {
      const float* p = T + row + c;
#pragma unroll 8
      for (int s = 0; s < slices; ++s) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(p + (size_t)s * step);
        const f32x4 y = *reinterpret_cast<const f32x4*>(p + (size_t)s * step + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[q][e] += x[e];
          v[q][4 + e] += y[e];
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[q][e]));
  }
  float down = 1.f, up = 1.f;
  if constexpr (!BF) {
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    // 2^-e and 2^e, both normal; an infinite or NaN row keeps its infinities and NaN
    int ex = (int)(__float_as_uint(top) >> 23) - 127;
    ex = ex < -100 ? -100 : ex > 100 ? 100 : ex;
    down = __uint_as_float((uint32_t)(127 - ex) << 23);
    up = __uint_as_float((uint32_t)(127 + ex) << 23);
  }
#pragma unroll
  for (int q = 0; q < KR; ++q) {
    float h[8], l[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = v[q][e] * down;
      h[e] = lo16<BF>(to16<BF>(x));
      l[e] = fabsf(h[e]) < INFINITY ? x - h[e] : 0.f;
    }
    hi[64 * q] = pack8<BF>(h);
    lo[64 * q] = pack8<BF>(l);
  }
  return up;
}

// T[slice][m][rp] (rp: the rank rounded up to 16) = X[m][its slice of K] A[a]^T.
// Grid: (slices of K, tiles of 16 TM rows, TM == 1 ? leaders : 1).
template <int TM, int RT, bool BF>
__global__ __launch_bounds__(64 * LW, RT * TM <= 16 ? 2 : 1) void lora_shrink_kernel(
    const uint16_t* __restrict__ X, const uint16_t* __restrict__ A, const int* __restrict__ ids,
    float* __restrict__ T, int M, int K, int rank, int adapters, int ldx, int kslice) {
  __shared__ f32x4 red[LW][RT * TM][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int r = lane & 15, g = lane >> 4;
  const int m0 = blockIdx.y * 16 * TM;
  const int id = tile_id<TM>(ids, m0, M, adapters);
  uint64_t todo = tile_todo<TM>(id, blockIdx.z);
  const int k0 = blockIdx.x * kslice;
  const int k1 = k0 + kslice < K ? k0 + kslice : K;
  const int rp = (rank + 15) & ~15;
  while (todo) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
    todo &= ~__ballot(id == a);
    const uint16_t* Aa = A + (size_t)a * rank * K;
    f32x4 acc[RT][TM];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int t = 0; t < TM; ++t) acc[i][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    // a wave's part of the slice lies together: 16 rows' 64-byte pieces of one load and the
    // next share cache lines
    const int kw = kslice / LW;
    const int ka = k0 + kw * wave, kb = ka + kw < k1 ? ka + kw : k1;
    // rows past A's or X's last repeat it: what comes of them is not stored
    const uint16_t *ap[RT], *xp[TM];
#pragma unroll
    for (int i = 0; i < RT; ++i)
      ap[i] = Aa + (size_t)(16 * i + r < rank ? 16 * i + r : rank - 1) * K + 8 * g;
#pragma unroll
    for (int t = 0; t < TM; ++t)
      xp[t] = X + (size_t)(m0 + 16 * t + r < M ? m0 + 16 * t + r : M - 1) * ldx + 8 * g;
    // the loads of U steps go out together
    constexpr int U = RT + TM <= 8 ? 4 : 2;
    int kk = ka;
    for (; kk + 32 * U <= kb; kk += 32 * U) {
      u32x4v af[U][RT], xf[U][TM];
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int t = 0; t < TM; ++t) xf[u][t] = *reinterpret_cast<const u32x4v*>(xp[t] + kk + 32 * u);
#pragma unroll
        for (int i = 0; i < RT; ++i) af[u][i] = *reinterpret_cast<const u32x4v*>(ap[i] + kk + 32 * u);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int t = 0; t < TM; ++t) acc[i][t] = mfma16<BF>(af[u][i], xf[u][t], acc[i][t]);
    }
    for (; kk + 32 <= kb; kk += 32) {
      u32x4v af[RT], xf[TM];
#pragma unroll
      for (int i = 0; i < RT; ++i) af[i] = *reinterpret_cast<const u32x4v*>(ap[i] + kk);
#pragma unroll
      for (int t = 0; t < TM; ++t) xf[t] = *reinterpret_cast<const u32x4v*>(xp[t] + kk);
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int t = 0; t < TM; ++t) acc[i][t] = mfma16<BF>(af[i], xf[t], acc[i][t]);
    }
    if (kk < kb) {  // K's last columns; their lanes past the end stay out of both operands
      u32x4v af[RT], xf[TM];
      const bool in = kk + 8 * g < kb;
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        af[i] = u32x4v{0u, 0u, 0u, 0u};
        if (in) af[i] = *reinterpret_cast<const u32x4v*>(ap[i] + kk);
      }
#pragma unroll
      for (int t = 0; t < TM; ++t) {
        xf[t] = u32x4v{0u, 0u, 0u, 0u};
        if (in) xf[t] = *reinterpret_cast<const u32x4v*>(xp[t] + kk);
      }
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int t = 0; t < TM; ++t) acc[i][t] = mfma16<BF>(af[i], xf[t], acc[i][t]);
    }
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int t = 0; t < TM; ++t) red[wave][i * TM + t][lane] = acc[i][t];
    __syncthreads();
    // lane: rows 16 i + 4 g .. + 3 of A, row m0 + 16 t + r of X
    for (int p = wave; p < RT * TM; p += LW) {
      f32x4 v = red[0][p][lane];
#pragma unroll
      for (int w = 1; w < LW; ++w) v += red[w][p][lane];
      const int i = p / TM, t = p - i * TM;
      const int mine = __shfl(id, 16 * t + r);
      const int m = m0 + 16 * t + r;
      if (mine == a && 16 * i < rp) {
        float* at = T + ((size_t)blockIdx.x * M + m) * rp + 16 * i + 4 * g;
        *reinterpret_cast<f32x4*>(at) = v;
      }
    }
    __syncthreads();
  }
}

// With tiles of many rows the sums are split once, S[tile][hi, lo][row tile][KR][64] and ups[m],
// for all workgroups that share a tile in the product with B (summed by each of them, 4096
// rows of rank 64 took 12 us more).  Grid: (row tiles of a tile, tiles), one wave each.
template <int TM, int KR, bool BF>
__global__ __launch_bounds__(64) void lora_split_kernel(
    const float* __restrict__ T, const int* __restrict__ ids, u32x4v* __restrict__ S,
    float* __restrict__ ups, int M, int rank, int adapters, int slices) {
  const int lane = threadIdx.x, r = lane & 15, g = lane >> 4, t = blockIdx.x;
  const int m = blockIdx.y * 16 * TM + 16 * t + r, rp = (rank + 15) & ~15;
  const int id = m < M ? ids[m] : -1;
  u32x4v* hi = S + ((size_t)blockIdx.y * 2 * TM + t) * KR * 64 + lane;
  const float up = split_row<KR, BF>(T, (size_t)M * rp, slices, (size_t)m * rp, rank, g,
                                     id >= 0 && id < adapters, hi, hi + (size_t)TM * KR * 64);
  if (g == 0) ups[m] = up;
}

// Y = base + scale (sum over slices of T) B^T.  A wave takes 64 columns at a time: row i of
// matrix tile t stands for column 16 (i / 4) + 4 t + i % 4, so that a lane ends with 16
// columns side by side.  Grid: (column pieces, tiles, TM == 1 ? leaders + 1 : 1); the last
// z of TM == 1 copies the rows without an adapter.
template <int TM, int KR, bool BF>
__global__ __launch_bounds__(64 * LW, 2) void lora_expand_kernel(
    const float* __restrict__ T, const u32x4v* __restrict__ S, const float* __restrict__ S_ups,
    const uint16_t* __restrict__ B, const int* __restrict__ ids, const float* __restrict__ scale, const uint16_t* base, uint16_t* Y, int M, int N, int rank,
    int adapters, int ldy, int slices, int ncols) {
  __shared__ u32x4v split[2][TM][KR][64];  // T's tile as hi and lo operands
  __shared__ float ups[16 * TM];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int r = lane & 15, g = lane >> 4;
  const int m0 = blockIdx.y * 16 * TM;
  const int id = tile_id<TM>(ids, m0, M, adapters);
  const int n0 = blockIdx.x * ncols + 64 * wave;
  const int n1 = (int)(blockIdx.x + 1) * ncols < N ? (int)(blockIdx.x + 1) * ncols : N;
  const bool copy = TM > 1 || blockIdx.z == 16;
  uint64_t todo = TM == 1 && copy ? 0 : tile_todo<TM>(id, blockIdx.z);
  if (copy && base != Y) {
#pragma unroll
    for (int t = 0; t < TM; ++t) {
      const int m = m0 + 16 * t + r;
      const int mine = __shfl(id, 16 * t + r);
      if (m < M && mine < 0)
        for (int nn = n0; nn < n1; nn += 64 * LW) {
          const int n = nn + 16 * g;
          const size_t at = (size_t)m * ldy + n;
          if (n < n1)
            *reinterpret_cast<u32x4v*>(Y + at) = *reinterpret_cast<const u32x4v*>(base + at);
          if (n + 8 < n1)
            *reinterpret_cast<u32x4v*>(Y + at + 8) =
                *reinterpret_cast<const u32x4v*>(base + at + 8);
        }
    }
  }
  const int rp = (rank + 15) & ~15;
  if constexpr (TM > 1) {
    u32x4v* all = &split[0][0][0][0];
#pragma unroll
    for (int i = threadIdx.x; i < 2 * TM * KR * 64; i += 64 * LW)
      all[i] = S[(size_t)blockIdx.y * (2 * TM * KR * 64) + i];
    if (threadIdx.x < 16 * TM) ups[threadIdx.x] = S_ups[m0 + threadIdx.x];
    __syncthreads();
  }
  while (todo) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
    todo &= ~__ballot(id == a);
    const uint16_t* Ba = B + (size_t)a * rank * N;
    const float sc = scale[a];
    // The operands of 64 columns.  Rows of B and of base past the last repeat it: what comes
    // of them is not stored.
    struct Columns {
      u32x4v bf[4][KR], b0[TM], b1[TM];
    };
    auto load = [&](Columns& c, int nn) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int n = nn + 16 * (r >> 2) + 4 * t + (r & 3);
        const uint16_t* row = Ba + (size_t)(n < N ? n : N - 1) * rank;
#pragma unroll
        for (int q = 0; q < KR; ++q) {
          const int k = 32 * q + 8 * g;
          c.bf[t][q] = u32x4v{0u, 0u, 0u, 0u};
          if (k < rank) c.bf[t][q] = *reinterpret_cast<const u32x4v*>(row + k);
        }
      }
      const int n = nn + 16 * g;
#pragma unroll
      for (int mt = 0; mt < TM; ++mt) {
        const int m = m0 + 16 * mt + r < M ? m0 + 16 * mt + r : M - 1;
        const uint16_t* row = base + (size_t)m * ldy;
        c.b0[mt] = c.b1[mt] = u32x4v{0u, 0u, 0u, 0u};
        if (TM > 1 || __shfl(id, r) == a) {  // the other leaders' rows are not for this one
          c.b0[mt] = *reinterpret_cast<const u32x4v*>(row + (n < N ? n : N - 8));
          c.b1[mt] = *reinterpret_cast<const u32x4v*>(row + (n + 8 < N ? n + 8 : N - 8));
        }
      }
    };
    if constexpr (TM == 1) {
      if (wave == 0) {
        const float up = sc * split_row<KR, BF>(
            T, (size_t)M * rp, slices, (size_t)(m0 + r) * rp, rank, g, __shfl(id, r) == a,
            &split[0][0][0][lane], &split[1][0][0][lane]);
        if (g == 0) ups[r] = up;
      }
      __syncthreads();
    }
    float up[TM];
    bool mine[TM];
#pragma unroll
    for (int t = 0; t < TM; ++t) {
      up[t] = TM == 1 ? ups[r] : sc * ups[16 * t + r];
      mine[t] = __shfl(id, 16 * t + r) == a;
    }
    for (int nn = n0; nn < n1; nn += 64 * LW) {
      Columns c;
      load(c, nn);
      const int n = nn + 16 * g;
#pragma unroll
      for (int mt = 0; mt < TM; ++mt) {
        const size_t at = (size_t)(m0 + 16 * mt + r) * ldy + n;
        f32x4 acc[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < KR; ++q) {
          const u32x4v hi = split[0][mt][q][lane], lo = split[1][mt][q][lane];
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            acc[t] = mfma16<BF>(c.bf[t][q], lo, acc[t]);
            acc[t] = mfma16<BF>(c.bf[t][q], hi, acc[t]);
          }
        }
        float y[8];
        unpack8<BF>(c.b0[mt], y);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = __builtin_fmaf(up[mt], acc[e >> 2][e & 3], y[e]);
        if (mine[mt] && n < n1) *reinterpret_cast<u32x4v*>(Y + at) = pack8<BF>(y);
        unpack8<BF>(c.b1[mt], y);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = __builtin_fmaf(up[mt], acc[2 + (e >> 2)][e & 3], y[e]);
        if (mine[mt] && n + 8 < n1) *reinterpret_cast<u32x4v*>(Y + at + 8) = pack8<BF>(y);
      }
    }
    __syncthreads();
  }
}

template <int TM, bool BF>
void shrink(dim3 grid, hipStream_t st, const uint16_t* X, const uint16_t* A, const int* ids,
            float* T, int M, int K, int rank, int adapters, int ldx, int kslice) {
  auto fn = rank <= 16 ? lora_shrink_kernel<TM, 1, BF>
                       : rank <= 32 ? lora_shrink_kernel<TM, 2, BF>
                                    : rank <= 64 ? lora_shrink_kernel<TM, 4, BF>
                                                 : lora_shrink_kernel<TM, 8, BF>;
  hipLaunchKernelGGL(fn, grid, dim3(64 * LW), 0, st, X, A, ids, T, M, K, rank, adapters, ldx,
                     kslice);
}
template <int TM, bool BF>
void expand(dim3 grid, hipStream_t st, const float* T, const u32x4v* S, const float* ups,
            const uint16_t* B, const int* ids,
            const float* scale, const uint16_t* base, uint16_t* Y, int M, int N, int rank,
            int adapters, int ldy, int slices, int ncols) {
  auto fn = rank <= 32 ? lora_expand_kernel<TM, 1, BF>
                       : rank <= 64 ? lora_expand_kernel<TM, 2, BF> : lora_expand_kernel<TM, 4, BF>;
  hipLaunchKernelGGL(fn, grid, dim3(64 * LW), 0, st, T, S, ups, B, ids, scale, base, Y, M, N, rank,
                     adapters, ldy, slices, ncols);
}

}  // namespace

namespace {
// workspace of the split sums and their powers of two (tiles of 64 rows)
size_t split_floats(int tiles, int tm, int rank) {
  const int kr = rank <= 32 ? 1 : rank <= 64 ? 2 : 4;
  return (size_t)tiles * (4 * 2 * tm * kr * 64 + 16 * tm);
}
}  // namespace

size_t lora_most_floats(int M, int rank) {
  // rows times slices: at most 256 or M in tiles of 16, 64 * 512 or M in tiles of 64
  const size_t rp = (rank + 15) / 16 * 16;
  if (M <= 512) return (M < 256 ? 256 : M) * rp;
  return (M < 32768 ? 32768 : M) * rp + split_floats((M + 63) / 64, 4, rank);
}

LoraPlan lora_make_plan(int M, int N, int K, int rank) {
  LoraPlan p;
  // Tiles of 64 rows share what they read of A and B, tiles of 16 work on an adapter that few of
  // their rows have with less waste.  8192 x 8192, rank 16, us, 16 against 64: 256 rows of 8
  // adapters in order 25 / 23, of 32 in any order 37 / 124; 512 rows 26 / 24 and 54 / 130;
  // 1024 rows 45 / 23 and 103 / 156.
  p.tm = M > 512 ? 4 : 1;
  p.tiles = (M + 16 * p.tm - 1) / (16 * p.tm);
  // workgroups: one per (leader, slice); M leaders are the most there can be of few rows
  const int leaders = p.tm == 1 ? M : p.tiles;
  p.kslice = 512;
  // fewer slices leave the second kernel less to add: 48 rows 14.4 us with 256, 15.6 with 512,
  // 17.2 with 128
  const int most = p.tm == 1 ? 256 : 512;
  while (p.kslice < K && ((long long)leaders * ((K + p.kslice - 1) / p.kslice) > most ||
                          (K + p.kslice - 1) / p.kslice > 16))
    p.kslice *= 2;
  p.slices = (K + p.kslice - 1) / p.kslice;
  // 4096 rows, the three kernels: 67 us with pieces of 512, 70 with 256 and with 1024
  p.ncols = 256;
  while (p.ncols < 512 && (long long)p.tiles * ((N + 2 * p.ncols - 1) / (2 * p.ncols)) >= 512)
    p.ncols *= 2;
  p.pieces = (N + p.ncols - 1) / p.ncols;
  p.floats = (size_t)p.slices * M * ((rank + 15) / 16 * 16);
  p.split = 0;
  if (p.tm > 1) {
    const int kr = rank <= 32 ? 1 : rank <= 64 ? 2 : 4;
    p.split = (size_t)p.tiles * 2 * p.tm * kr * 64;  // 16 bytes each
    p.floats += split_floats(p.tiles, p.tm, rank);
  }
  return p;
}

hipError_t lora_launch(const LoraPlan& p, const uint16_t* X, const uint16_t* A, const uint16_t* B,
                       const int* ids, const float* scale, const uint16_t* base, uint16_t* Y,
                       float* T, int M, int N, int K, int rank, int adapters, int ldx, int ldy,
                       bool bf, hipStream_t st) {
  const size_t rest = 4 * p.split + (size_t)p.tiles * 16 * p.tm;
  u32x4v* S = p.tm > 1 ? reinterpret_cast<u32x4v*>(T + (p.floats - rest)) : nullptr;
  float* ups = p.tm > 1 ? T + (p.floats - (size_t)p.tiles * 16 * p.tm) : nullptr;
  const dim3 g1(p.slices, p.tiles, p.tm == 1 ? 16 : 1);
  const dim3 g2(p.pieces, p.tiles, p.tm == 1 ? 17 : 1);
  if (p.tm == 1) {
    (bf ? shrink<1, true> : shrink<1, false>)(g1, st, X, A, ids, T, M, K, rank, adapters, ldx,
                                              p.kslice);
  } else {
    (bf ? shrink<4, true> : shrink<4, false>)(g1, st, X, A, ids, T, M, K, rank, adapters, ldx,
                                              p.kslice);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (p.tm > 1) {
    auto fn = rank <= 32 ? (bf ? lora_split_kernel<4, 1, true> : lora_split_kernel<4, 1, false>)
              : rank <= 64 ? (bf ? lora_split_kernel<4, 2, true> : lora_split_kernel<4, 2, false>)
                           : (bf ? lora_split_kernel<4, 4, true> : lora_split_kernel<4, 4, false>);
    hipLaunchKernelGGL(fn, dim3(4, p.tiles), dim3(64), 0, st, T, ids, S, ups, M, rank, adapters,
                       p.slices);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (p.tm == 1) {
    (bf ? expand<1, true> : expand<1, false>)(g2, st, T, S, ups, B, ids, scale, base, Y, M, N,
                                              rank, adapters, ldy, p.slices, p.ncols);
  } else {
    (bf ? expand<4, true> : expand<4, false>)(g2, st, T, S, ups, B, ids, scale, base, Y, M, N,
                                              rank, adapters, ldy, p.slices, p.ncols);
  }
  return hipGetLastError();
}

}  // namespace w4a16
