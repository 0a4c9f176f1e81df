// What the kernels whose tiles have 128 columns share (kv4_prefill.hip, kv4_tree_wide.hip).
#pragma once
#include "kv4_attend.h"

namespace w4a16 {

constexpr int PTC = 128;  // columns of a workgroup

// p's exponent is x cf - ref + 8 in one fma.  ref is some x cf rounded, so past 2^26 their
// difference alone can lift p out of fp16: past this reference x cf is rounded first.
constexpr float kFar = 0x1p20f;

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

// The operands of a wave's columns (column lane % 32: row, query head qh; h = lane / 32): q
// scaled into fp16, its sums per group of channels, and the factor of the logits.
template <int D, int NG, bool BF>
__device__ __forceinline__ void wide_queries(const Kv4AttendArgs& p, int row, int qh, int h,
                                             half8v* qf, half8v& qm, float& cf) {
  constexpr int J = D / 16, JG = J / NG;
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

}  // namespace w4a16
