// 16-bit rows (fp16 or bf16) in the operators around the product: conversions to and from
// fp32, and sums handed from workgroup to workgroup, shared by rmsnorm.hip, lora.hip, kv4_cache.hip and
// kv4_attention.hip.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w4a16 {

typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef _Float16 half8v __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8v __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2v __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4v __attribute__((ext_vector_type(4)));

// BF: the 16 bits are bf16, else fp16
template <bool BF>
__device__ __forceinline__ float lo16(uint32_t w) {
  if constexpr (BF) return __uint_as_float(w << 16);
  return (float)__builtin_bit_cast(_Float16, (uint16_t)(w & 0xFFFFu));
}
template <bool BF>
__device__ __forceinline__ float hi16(uint32_t w) {
  if constexpr (BF) return __uint_as_float(w & 0xFFFF0000u);
  return (float)__builtin_bit_cast(_Float16, (uint16_t)(w >> 16));
}
// nearest-even, NaN stays NaN
template <bool BF>
__device__ __forceinline__ uint32_t to16(float f) {
  if constexpr (BF) return __builtin_bit_cast(uint16_t, (__bf16)f);
  return __builtin_bit_cast(uint16_t, (_Float16)f);
}
template <bool BF>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  if constexpr (BF) return to16<BF>(a) | (to16<BF>(b) << 16);
  typedef float pair __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(pair{a, b}, half2v));
}
// eight 16-bit values of a 16-byte chunk
template <bool BF>
__device__ __forceinline__ void unpack8(const u32x4v& v, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = lo16<BF>(v[i]);
    f[2 * i + 1] = hi16<BF>(v[i]);
  }
}
template <bool BF>
__device__ __forceinline__ u32x4v pack8(const float* f) {
  return u32x4v{pack16<BF>(f[0], f[1]), pack16<BF>(f[2], f[3]), pack16<BF>(f[4], f[5]),
                pack16<BF>(f[6], f[7])};
}

// Workgroups on different XCDs hand their sums over with relaxed agent-scope accesses, which
// are coherent across the L2s by themselves; what orders them is that all of a workgroup's
// stores have completed (s_waitcnt) before it counts itself in.
__device__ __forceinline__ void put8(float* p, float a, float b) {
  const uint64_t v = (uint64_t)__float_as_uint(b) << 32 | __float_as_uint(a);
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p), v, __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void get8(const float* p, float& a, float& b) {
  const uint64_t v = __hip_atomic_load(reinterpret_cast<uint64_t*>(const_cast<float*>(p)),
                                       __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  a = __uint_as_float((uint32_t)v);
  b = __uint_as_float((uint32_t)(v >> 32));
}
__device__ __forceinline__ void get16(const float* p, f32x4& x) {
  float a, b, c, d;
  get8(p, a, b);
  get8(p + 2, c, d);
  x = f32x4{a, b, c, d};
}

}  // namespace w4a16
