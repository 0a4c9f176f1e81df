// Residual addition, root-mean-square norm and the 8-bit rows of the W4A8 product.
//
//   h = rne16(x + r),  y = h * rsqrt(mean(h^2) + eps) * g,
//   s = max|y| / 448 (1 for a row of zeros),  y8 = e4m3(y / s)
//
// One workgroup holds one row in registers, so every input is read once.  Both things a row
// has to agree on, sum(h^2) and max|h g|, come from one pass and one exchange through LDS:
// y = inv * (h g) with inv > 0 common to the row, so max|y| = inv * max|h g| and
// y / s = (h g) * (448 / max|h g|), which needs no norm at all.  Sums are fp32.
//
// bf16 rows can leave the fp32 range, their squares above and below, their products with g
// too: such rows are worked out again in 64 bits, where nothing of theirs can, in twice the
// time.  True infinities and NaN end as the formula ends: a NaN makes the row's codes
// NaN, an infinity is a NaN among zeros, and s = 1 for both.
//
// Bound: HBM.  8192 x 8192 fp16: 470 MB in 81 us, 5.8 TB/s (a sum of two arrays: 5.9); 4096 x
// 65536 bf16: 373 us, 5.0 TB/s; one row of 4096: 2.6 us in the kernel, 5.6 us a call.
#include "internal.h"
#include "rows16.h"

namespace w4a16 {

namespace {

// Within these bounds fp32 loses nothing that counts: of a mean square above 2^-80, squares
// below 2^-126 are less than 2^-46; 448 / max|h g| is finite.  yscale is never below 2^-126,
// where fp32 begins to lose bits.
constexpr float kLeastMean = 0x1p-80f, kLeastTop = 0x1p-100f, kLeastScale = 0x1p-126f;

// A row that fp32 does not reach, from its beginning, in 64 bits.  It reads the row again
// (h, where it was written), two values at a time, so that it needs no more registers than
// the others.
template <int T, bool BF>
__device__ __forceinline__ void wide_row(const u32x4v* X, const u32x4v* R, const u32x4v* gamma,
                                         const u32x4v* H, u32x2v* Y8, float* yscale, u32x4v* Y,
                                         unsigned m, int K, float eps) {
  constexpr int NW = T / 64;
  __shared__ double red[NW][2];
  const int tid = threadIdx.x, pairs = K / 2;
  const size_t row = (size_t)m * pairs;
  const uint32_t* x = reinterpret_cast<const uint32_t*>(H != nullptr ? H : X) + row;
  const uint32_t* r = H != nullptr || R == nullptr ? nullptr
                                                   : reinterpret_cast<const uint32_t*>(R) + row;
  const uint32_t* g = reinterpret_cast<const uint32_t*>(gamma);
  auto h_pair = [&](int c) {
    const uint32_t a = x[c];
    if (r == nullptr) return a;
    return pack16<BF>(lo16<BF>(a) + lo16<BF>(r[c]), hi16<BF>(a) + hi16<BF>(r[c]));
  };
  double ss = 0., top = 0.;
#pragma unroll 1
  for (int c = tid; c < pairs; c += T) {
    const uint32_t h = h_pair(c);
    const double a = lo16<BF>(h), b = hi16<BF>(h);
    ss += a * a + b * b;
    top = fmax(top, fmax(fabs(a * lo16<BF>(g[c])), fabs(b * hi16<BF>(g[c]))));
  }
  for (int off = 32; off >= 1; off >>= 1) {
    ss += __shfl_xor(ss, off);
    top = fmax(top, __shfl_xor(top, off));
  }
  if ((tid & 63) == 0) {
    red[tid >> 6][0] = ss;
    red[tid >> 6][1] = top;
  }
  __syncthreads();
  ss = red[0][0];
  top = red[0][1];
#pragma unroll 1
  for (int w = 1; w < NW; ++w) {
    ss += red[w][0];
    top = fmax(top, red[w][1]);
  }
  const double mean = ss / K + eps;
  const double inv = mean == 0. ? 0. : 1. / sqrt(mean);  // a row of zeros stays zeros
  const double exact = inv * top / 448.;
  float s = 1.f;
  double up = inv;  // infinite and NaN rows, rows of zeros
  if (exact > 0. && exact < INFINITY) {
    s = fmaxf((float)exact, kLeastScale);
    up = inv / s;
  } else if (exact == INFINITY) {
    up = 0.;
  }
  if (tid == 0) yscale[m] = s;
#pragma unroll 1
  for (int c = tid; c < pairs; c += T) {
    const uint32_t h = h_pair(c);
    const double a = lo16<BF>(h), b = hi16<BF>(h), ga = lo16<BF>(g[c]), gb = hi16<BF>(g[c]);
    const int code =
        __builtin_amdgcn_cvt_pk_fp8_f32((float)(a * ga * up), (float)(b * gb * up), 0, false);
    reinterpret_cast<uint16_t*>(Y8)[row + c] = (uint16_t)code;
    if (Y != nullptr)
      reinterpret_cast<uint32_t*>(Y)[row + c] =
          pack16<BF>((float)(a * inv * ga), (float)(b * inv * gb));
  }
}

// Rows past the first 2^20 lie in further rows of the grid, whose dimensions take 2^32 threads.
constexpr unsigned kGridRow = 1u << 20;

// T threads, CH 16-byte chunks of a row in each.
template <int T, int CH, bool BF>
__global__ __launch_bounds__(T) void rmsnorm_kernel(const u32x4v* X, const u32x4v* R,
                                                    const u32x4v* __restrict__ gamma, u32x4v* H,
                                                    u32x2v* __restrict__ Y8,
                                                    float* __restrict__ yscale, u32x4v* Y, int M,
                                                    int K, float eps) {
  constexpr int NW = T / 64;
  __shared__ float red[NW][3];
  const int tid = threadIdx.x;
  const int chunks = K / 8;
  const unsigned m = blockIdx.x + blockIdx.y * kGridRow;
  if (m >= (unsigned)M) return;
  const size_t row = (size_t)m * chunks;
  u32x4v h[CH], gm[CH];
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    const int c = tid + j * T;
    h[j] = u32x4v{0u, 0u, 0u, 0u};
    gm[j] = h[j];
    if (c < chunks) {
      h[j] = X[row + c];
      gm[j] = gamma[c];
    }
  }
  if (R != nullptr) {
    u32x4v r[CH];
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = tid + j * T;
      r[j] = c < chunks ? R[row + c] : u32x4v{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      float a[8], b[8];
      unpack8<BF>(h[j], a);
      unpack8<BF>(r[j], b);
#pragma unroll
      for (int e = 0; e < 8; ++e) a[e] += b[e];
      h[j] = pack8<BF>(a);
    }
  }
  if (H != nullptr) {
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = tid + j * T;
      if (c < chunks) H[row + c] = h[j];
    }
  }
  // the row's sum of squares and largest |h g|
  auto reduce = [&](float& ss, float& top) {
    ss = 0.f;
    top = 0.f;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      float a[8], g[8];
      unpack8<BF>(h[j], a);
      unpack8<BF>(gm[j], g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ss = __builtin_fmaf(a[e], a[e], ss);
        top = fmaxf(top, fabsf(a[e] * g[e]));
      }
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
      ss += __shfl_xor(ss, off);
      top = fmaxf(top, __shfl_xor(top, off));
    }
    if constexpr (NW > 1) {
      if ((tid & 63) == 0) {
        red[tid >> 6][0] = ss;
        red[tid >> 6][1] = top;
      }
      __syncthreads();
      ss = red[0][0];
      top = red[0][1];
#pragma unroll
      for (int w = 1; w < NW; ++w) {
        ss += red[w][0];
        top = fmaxf(top, red[w][1]);
      }
    }
  };
  float ss, top;
  reduce(ss, top);
  const float mean = ss / (float)K + eps;
  float inv = rsqrtf(mean);
  float s = inv * top * (1.f / 448.f);
  float up = 448.f / top;
  // All of this is the same for the whole workgroup (the ballots show it to the compiler).
  // A sum of 0 is a row of zeros, as padding has them, or one too small for fp32.
  bool zeros = false;
  if (__ballot(ss == 0.f) != 0) {
    uint32_t bits = 0;
#pragma unroll
    for (int j = 0; j < CH; ++j) bits |= h[j][0] | h[j][1] | h[j][2] | h[j][3];
    const bool some = __ballot((bits & 0x7FFF7FFFu) != 0) != 0;
    if ((tid & 63) == 0) red[tid >> 6][2] = some ? 1.f : 0.f;
    __syncthreads();
    float any = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) any += red[w][2];
    zeros = __ballot(any == 0.f) != 0;
  }
  const bool narrow = ss < INFINITY && mean >= kLeastMean && top >= kLeastTop &&
                      s >= kLeastScale && s < INFINITY;
  if (zeros) {
    inv = 0.f;
    up = s = 1.f;
  } else if (__ballot(!narrow) != 0) {
    wide_row<T, BF>(X, R, gamma, H, Y8, yscale, Y, m, K, eps);
    return;
  }
  if (tid == 0) yscale[m] = s;
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    const int c = tid + j * T;
    if (c >= chunks) continue;
    // Unpacked again: the compiler would hold what it has unpacked since the sums.  Gamma too
    // only where registers would spill; with 256 threads, 8192 x 8192, 81.4 us instead of 80.6.
    asm("" : "+v"(h[j]));
    if constexpr (T == 1024) asm("" : "+v"(gm[j]));
    float a[8], g[8], y[8];
    unpack8<BF>(h[j], a);
    unpack8<BF>(gm[j], g);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = a[e] * g[e] * up;
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], lo, true);
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[4], y[5], 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[6], y[7], hi, true);
    Y8[row + c] = u32x2v{(uint32_t)lo, (uint32_t)hi};
    if (Y != nullptr) {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = a[e] * inv * g[e];
      Y[row + c] = pack8<BF>(y);
    }
  }
}

typedef void (*NormFn)(const u32x4v*, const u32x4v*, const u32x4v*, u32x4v*, u32x2v*, float*,
                       u32x4v*, int, int, float);
template <bool BF>
NormFn norm_kernel(int threads, int ch) {
  if (threads == 256)
    return ch <= 1 ? rmsnorm_kernel<256, 1, BF>
                   : ch <= 2 ? rmsnorm_kernel<256, 2, BF> : rmsnorm_kernel<256, 4, BF>;
  return ch <= 1 ? rmsnorm_kernel<1024, 1, BF>
                 : ch <= 2 ? rmsnorm_kernel<1024, 2, BF>
                           : ch <= 4 ? rmsnorm_kernel<1024, 4, BF> : rmsnorm_kernel<1024, 8, BF>;
}

}  // namespace

hipError_t launch_rmsnorm(const uint16_t* X, const uint16_t* R, const uint16_t* gamma, uint16_t* H,
                          uint8_t* Y8, float* yscale, uint16_t* Y, int M, int K, float eps, bool bf,
                          hipStream_t st) {
  if (M <= 0 || K <= 0 || K % 8 != 0 || K > NORM_MAX_K) return hipErrorInvalidValue;
  const int chunks = K / 8;
  // 4096 rows of 4096 / 8192 values: 18.7 / 34.8 us with 256 threads, 23.8 / 37.7 with 1024; 1024
  // rows of 8192: 11.2 / 12.7; 256 rows of 4096: 5.8 / 5.3; 1 to 64 rows: 5.7 / 5.7.  Past 8192
  // values 256 threads would need more than 4 chunks each
  const int threads = chunks <= 1024 ? 256 : 1024;
  const int ch = (chunks + threads - 1) / threads;
  NormFn fn = bf ? norm_kernel<true>(threads, ch) : norm_kernel<false>(threads, ch);
  const dim3 grid = (unsigned)M <= kGridRow ? dim3(M) : dim3(kGridRow, (M - 1) / kGridRow + 1);
  hipLaunchKernelGGL(fn, grid, dim3(threads), 0, st, reinterpret_cast<const u32x4v*>(X),
                     reinterpret_cast<const u32x4v*>(R), reinterpret_cast<const u32x4v*>(gamma),
                     reinterpret_cast<u32x4v*>(H), reinterpret_cast<u32x2v*>(Y8), yscale,
                     reinterpret_cast<u32x4v*>(Y), M, K, eps);
  return hipGetLastError();
}

}  // namespace w4a16
