// Rotary positions: each pair (a, b) of a head's first `rot` channels is turned by the angle
// of its frequency and of its token's position on that frequency's axis:
//   w = pos[axis[i]][t] * freq[i];  (a, b) -> (a cos w - b sin w, b cos w + a sin w)
// Pair i is channels (i, i + rot/2) or (2 i, 2 i + 1).
//
// The angle is formed in 64 bits in turns, where its whole part can be dropped exactly; what is
// left has fp32's full precision at any position (in fp32 a position of 10^6 alone would be off
// by 0.03 radians).  A token's angles serve all its heads, so a workgroup makes them once, one
// thread an angle, and keeps cosines and sines in LDS.
//
// An item is 8 pairs of one head (two loads of 16 bytes), or 16 channels that are only copied.
// Bound: HBM for prompts, latency for single tokens.
#include "internal.h"
#include "rows16.h"

namespace w4a16 {

namespace {

constexpr int RT = 256;     // threads of a workgroup
constexpr int RU = 4;       // items of a thread with loads in flight

// Grid: (groups of TT tokens, pieces of a token's items).
template <int TT, bool BF, bool NEIGHBOURS>
__global__ __launch_bounds__(RT) void rotary_kernel(RotaryArgs p) {
  extern __shared__ float turned[];  // [TT][rot / 2] cosines, then sines
  const int half = p.rot / 2;
  float* cosines = turned;
  float* sines = turned + TT * half;
  const int t0 = blockIdx.x * TT;
  const int live = p.tokens - t0 < TT ? p.tokens - t0 : TT;
  const unsigned first = blockIdx.y * (unsigned)p.piece;
  const unsigned end = first + p.piece < (unsigned)p.items ? first + p.piece : (unsigned)p.items;
  const unsigned turns = p.rot / 16;  // a head's items that are turned

  struct Item {
    const uint16_t* src;
    uint16_t* dst;
    int second;   // channels from the first eight to the second, 0: there are none
    unsigned item;
  };
  auto place = [&](int t, unsigned u) {
    Item x;
    const unsigned h = p.items_head == 1 ? u : __umulhi(u, p.magic);
    x.item = u - h * p.items_head;
    int c;
    if (x.item < turns) {
      c = NEIGHBOURS ? 16 * x.item : 8 * x.item;
      x.second = NEIGHBOURS ? 8 : half;
    } else {
      c = 16 * x.item;  // = rot + 16 (item - rot / 16)
      x.second = c + 16 <= p.head ? 8 : 0;
    }
    const bool is_k = h >= (unsigned)p.q_heads;
    const size_t at = (size_t)(is_k ? h - p.q_heads : h) * p.head + c;
    x.src = (is_k ? p.k + (size_t)(t0 + t) * p.ldk : p.q + (size_t)(t0 + t) * p.ldq) + at;
    x.dst = (is_k ? p.ko + (size_t)(t0 + t) * p.ldko : p.qo + (size_t)(t0 + t) * p.ldqo) + at;
    return x;
  };
  Item it[RU];
  u32x4v a[RU], b[RU];
  auto load = [&](int t, unsigned u0) {
#pragma unroll
    for (int i = 0; i < RU; ++i) {
      const unsigned u = u0 + i * RT;
      if (u >= end) break;
      it[i] = place(t, u);
      a[i] = *reinterpret_cast<const u32x4v*>(it[i].src);
      if (it[i].second) b[i] = *reinterpret_cast<const u32x4v*>(it[i].src + it[i].second);
    }
  };
  const unsigned u0 = first + threadIdx.x;
  load(0, u0);  // in flight while the angles are worked out

  for (int x = threadIdx.x; x < live * half; x += RT) {
    const int t = x / half, i = x - t * half;
    int axis = p.axis ? p.axis[i] : 0;
    axis = axis < 0 ? 0 : axis >= p.axes ? p.axes - 1 : axis;
    const int pos = p.pos[(size_t)axis * p.ldpos + t0 + t];
    const double w = (double)pos * ((double)p.freq[i] * 0.15915494309189535);  // 1 / 2 pi
    float s, c;
    sincospif(2.f * (float)(w - __builtin_rint(w)), &s, &c);
    cosines[t * half + i] = c;
    sines[t * half + i] = s;
  }
  __syncthreads();

  auto store = [&](int t, unsigned u0) {
#pragma unroll
    for (int i = 0; i < RU; ++i) {
      if (u0 + i * RT >= end) break;
      if (it[i].item < turns) {
        const float* c = cosines + t * half + 8 * it[i].item;
        const float* s = sines + t * half + 8 * it[i].item;
        float x[8], y[8], cs[8], sn[8];
        unpack8<BF>(a[i], x);
        unpack8<BF>(b[i], y);
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          const f32x4 cc = *reinterpret_cast<const f32x4*>(c + e);
          const f32x4 ss = *reinterpret_cast<const f32x4*>(s + e);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            cs[e + j] = cc[j];
            sn[e + j] = ss[j];
          }
        }
        float v[8], w[8];
        if constexpr (NEIGHBOURS) {
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            v[e] = x[e] * cs[e / 2] - x[e + 1] * sn[e / 2];
            v[e + 1] = x[e + 1] * cs[e / 2] + x[e] * sn[e / 2];
            w[e] = y[e] * cs[4 + e / 2] - y[e + 1] * sn[4 + e / 2];
            w[e + 1] = y[e + 1] * cs[4 + e / 2] + y[e] * sn[4 + e / 2];
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            v[e] = x[e] * cs[e] - y[e] * sn[e];
            w[e] = y[e] * cs[e] + x[e] * sn[e];
          }
        }
        a[i] = pack8<BF>(v);
        b[i] = pack8<BF>(w);
      }
      *reinterpret_cast<u32x4v*>(it[i].dst) = a[i];
      if (it[i].second) *reinterpret_cast<u32x4v*>(it[i].dst + it[i].second) = b[i];
    }
  };
  for (int t = 0; t < live; ++t)
    for (unsigned u = u0; u < end; u += RU * RT) {
      if (t != 0 || u != u0) load(t, u);
      store(t, u);
    }
}

template <bool BF, bool NEIGHBOURS>
void run(int tt, dim3 grid, size_t lds, hipStream_t st, const RotaryArgs& a) {
  if (tt == 1)
    hipLaunchKernelGGL((rotary_kernel<1, BF, NEIGHBOURS>), grid, dim3(RT), lds, st, a);
  else
    hipLaunchKernelGGL((rotary_kernel<4, BF, NEIGHBOURS>), grid, dim3(RT), lds, st, a);
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs& args, bool neighbours, bool bf, hipStream_t st) {
  RotaryArgs a = args;
  // what is not turned stays where it is if q and k are turned in place
  const bool copy = a.qo != a.q || (a.kv_heads > 0 && a.ko != a.k);
  a.items_head = a.rot / 16 + (copy ? (a.head - a.rot + 15) / 16 : 0);
  a.magic = a.items_head == 1 ? 0 : (uint32_t)((((uint64_t)1 << 32) + a.items_head - 1) / a.items_head);
  a.items = (a.q_heads + a.kv_heads) * a.items_head;
  const int tt = a.tokens >= 2048 ? 4 : 1;
  a.piece = a.items;
  const dim3 grid((a.tokens + tt - 1) / tt, (a.items + a.piece - 1) / a.piece);
  const size_t lds = (size_t)tt * a.rot * sizeof(float);
  if (bf) neighbours ? run<true, true>(tt, grid, lds, st, a) : run<true, false>(tt, grid, lds, st, a);
  else neighbours ? run<false, true>(tt, grid, lds, st, a) : run<false, false>(tt, grid, lds, st, a);
  return hipGetLastError();
}

}  // namespace w4a16
