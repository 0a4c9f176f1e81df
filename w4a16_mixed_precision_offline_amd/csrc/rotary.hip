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
// An item is 8 pairs of one head, or 16 channels that are only copied: two runs of 8 channels, half
// of the turned (copied) channels apart, so that the lanes of a load or store lie side by side
// (neighbouring runs instead: 114 us where 110 below).
//
// Bound: HBM for prompts, latency for single tokens.  16384 tokens of 64 + 8 heads of 128
// channels, half of them turned, into other rows: 604 MB in 110 us, 5.5 TB/s (a large copy: 4.85);
// 5041 of 40 + 8, three axes: 124 MB in 21.5 us; one token 2.3 us.
#include "internal.h"
#include "rows16.h"

namespace w4a16 {

namespace {

constexpr int RT = 256;     // threads of a workgroup
constexpr int RU = 4;       // items of a thread with loads in flight

// Grid: (tokens, pieces of a token's items).  PAST: stores go past the caches.
template <bool BF, bool NEIGHBOURS, bool PAST>
__global__ __launch_bounds__(RT) void rotary_kernel(RotaryArgs p) {
  extern __shared__ float turned[];  // [rot / 2] cosines, then sines
  const int half = p.rot / 2;
  float* cosines = turned;
  float* sines = turned + half;
  const size_t t = blockIdx.x;
  const unsigned first = blockIdx.y * (unsigned)p.piece;
  const unsigned end = first + p.piece < (unsigned)p.items ? first + p.piece : (unsigned)p.items;
  const unsigned turns = p.rot / 16;  // a head's items that are turned

  struct Item {
    const uint16_t* src;
    uint16_t* dst;
    int second;   // channels from the first eight to the second, 0: there are none
    unsigned item;
  };
  auto place = [&](unsigned u) {
    Item x;
    const unsigned h = p.items_head == 1 ? u : __umulhi(u, p.magic);
    x.item = u - h * p.items_head;
    int c;
    if (x.item < turns) {
      c = 8 * x.item;
      x.second = half;
    } else {
      const int apart = 8 * (p.items_head - turns);
      c = p.rot + 8 * (x.item - turns);
      x.second = c + apart < p.head ? apart : 0;
    }
    const bool is_k = h >= (unsigned)p.q_heads;
    const size_t at = (size_t)(is_k ? h - p.q_heads : h) * p.head + c;
    x.src = (is_k ? p.k + t * p.ldk : p.q + t * p.ldq) + at;
    x.dst = (is_k ? p.ko + t * p.ldko : p.qo + t * p.ldqo) + at;
    return x;
  };
  Item it[RU];
  u32x4v a[RU], b[RU];
  auto load = [&](unsigned u0) {
#pragma unroll
    for (int i = 0; i < RU; ++i) {
      const unsigned u = u0 + i * RT;
      if (u >= end) break;
      it[i] = place(u);
      a[i] = *reinterpret_cast<const u32x4v*>(it[i].src);
      if (it[i].second) b[i] = *reinterpret_cast<const u32x4v*>(it[i].src + it[i].second);
    }
  };
  const unsigned u0 = first + threadIdx.x;
  load(u0);  // in flight while the angles are worked out

  for (int i = threadIdx.x; i < half; i += RT) {
    int axis = p.axis ? p.axis[i] : 0;
    axis = axis < 0 ? 0 : axis >= p.axes ? p.axes - 1 : axis;
    const int pos = p.pos[(size_t)axis * p.ldpos + t];
    const double w = (double)pos * ((double)p.freq[i] * 0.15915494309189535);  // 1 / 2 pi
    float s, c;
    sincospif(2.f * (float)(w - __builtin_rint(w)), &s, &c);
    cosines[i] = c;
    sines[i] = s;
  }
  __syncthreads();

  auto store = [&](unsigned u0) {
#pragma unroll
    for (int i = 0; i < RU; ++i) {
      if (u0 + i * RT >= end) break;
      if (it[i].item < turns) {
        // neighbours: pairs 4 item .. + 3 of the first run, and half a head's pairs on of the second
        const int at = NEIGHBOURS ? 4 * it[i].item : 8 * it[i].item, on = NEIGHBOURS ? half / 2 : 4;
        float x[8], y[8], cs[8], sn[8];
        unpack8<BF>(a[i], x);
        unpack8<BF>(b[i], y);
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          const f32x4 cc = *reinterpret_cast<const f32x4*>(cosines + at + (e ? on : 0));
          const f32x4 ss = *reinterpret_cast<const f32x4*>(sines + at + (e ? on : 0));
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
      u32x4v* first = reinterpret_cast<u32x4v*>(it[i].dst);
      u32x4v* second = reinterpret_cast<u32x4v*>(it[i].dst + it[i].second);
      if constexpr (PAST) {
        __builtin_nontemporal_store(a[i], first);
        if (it[i].second) __builtin_nontemporal_store(b[i], second);
      } else {
        *first = a[i];
        if (it[i].second) *second = b[i];
      }
    }
  };
  for (unsigned u = u0; u < end; u += RU * RT) {
    if (u != u0) load(u);
    store(u);
  }
}

typedef void (*RotaryFn)(RotaryArgs);
template <bool BF, bool PAST>
RotaryFn rotary_kernel_of(bool neighbours) {
  return neighbours ? rotary_kernel<BF, true, PAST> : rotary_kernel<BF, false, PAST>;
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs& args, bool neighbours, bool bf, hipStream_t st) {
  RotaryArgs a = args;
  // what is not turned stays where it is if q and k are turned in place
  const bool copy = a.qo != a.q || (a.kv_heads > 0 && a.ko != a.k);
  a.items_head = a.rot / 16 + (copy ? (a.head - a.rot + 15) / 16 : 0);
  a.magic = a.items_head == 1 ? 0 : (uint32_t)((((uint64_t)1 << 32) + a.items_head - 1) / a.items_head);
  a.items = (a.q_heads + a.kv_heads) * a.items_head;
  // A workgroup has a token; up to 512 tokens its items are shared by several, one item a thread:
  // 1 / 64 / 256 tokens of 64 + 8 heads 2.3 / 2.9 / 3.6 us instead of 2.9 / 3.8 / 4.1.  From 512 on
  // there is no difference, and each angle is made once.  Four tokens a workgroup instead of
  // one: no difference up to 16384.
  a.piece = a.tokens <= 512 ? RT : a.items;
  const dim3 grid(a.tokens, (a.items + a.piece - 1) / a.piece);
  const size_t lds = (size_t)a.rot * sizeof(float);
  // Stores past the caches where a run of lanes fills whole lines of 128 bytes: 5041 tokens of 40 + 8
  // heads of 128 channels 21.5 us instead of 27.5; with half of each head turned (runs of 64
  // bytes) 16384 tokens take 117 us that way and 110 the other.  What reads the rows next takes
  // as long either way.
  const bool lines = a.rot >= 128 && (a.items_head == a.rot / 16 || a.head - a.rot >= 128);
  const bool past = a.tokens > 512 && lines;
  const auto fn = bf ? (past ? rotary_kernel_of<true, true>(neighbours) : rotary_kernel_of<true, false>(neighbours))
                     : (past ? rotary_kernel_of<false, true>(neighbours) : rotary_kernel_of<false, false>(neighbours));
  hipLaunchKernelGGL(fn, grid, dim3(RT), lds, st, a);
  return hipGetLastError();
}

}  // namespace w4a16
