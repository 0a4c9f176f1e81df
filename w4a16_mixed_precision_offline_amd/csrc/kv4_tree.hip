// Trees of drafted tokens: what the other operators take, from the nodes' parents.
//
// A node's line is the node, its parent, its parent's parent and so on.  One thread walks the
// line of a node, over the sequence's parents in LDS; since a parent lies before its node (others
// are taken for none), every step goes down, the bits of a word come in one piece and the walk
// ends.  Bound: latency: 26 nodes 1.9 us, 64 trees of 125 to 250 nodes 3.7 us.  The walk is as long
// as the tree is deep: a chain of 64 / 256 / 1024 / 4096 nodes takes 7 / 26 / 117 / 1250 us, 4096
// nodes in two levels 260 us (a thread writes a row's 128 words).
#include "kv4.h"

namespace w4a16 {

namespace {

// Grid: sequences.
__global__ __launch_bounds__(1024) void kv4_tree_kernel(Kv4TreeArgs p) {
  extern __shared__ int16_t up[];  // parents of the sequence's nodes, -1: none
  const Kv4Seq s = kv4_seq(p.rows, p.lens, blockIdx.x, p.tokens, p.max_new);
  for (int i = threadIdx.x; i < s.n; i += blockDim.x) {
    const int j = p.parent[s.first + i];
    up[i] = (int16_t)(j >= 0 && j < i ? j : -1);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < s.n; i += blockDim.x) {
    const size_t row = s.first + i;
    uint32_t* out = p.mask + row * p.words;
    int w = p.words - 1, depth = 0;
    uint32_t bits = 0;
    for (int j = i;;) {
      for (; w > j >> 5; --w) {
        out[w] = bits;
        bits = 0;
      }
      if (depth < p.window) bits |= 1u << (j & 31);
      j = up[j];
      if (j < 0) break;
      ++depth;
    }
    for (; w >= 0; --w) {
      out[w] = bits;
      bits = 0;
    }
    if (p.depth) p.depth[row] = depth;
    if (p.pos) p.pos[row] = s.len - s.n + depth;
  }
}

}  // namespace

hipError_t launch_kv4_tree(const Kv4TreeArgs& a, hipStream_t st) {
  const int threads = a.max_new >= 1024 ? 1024 : (a.max_new + 63) / 64 * 64;
  hipLaunchKernelGGL(kv4_tree_kernel, dim3(a.batch), dim3(threads), a.max_new * sizeof(int16_t), st,
                     a);
  return hipGetLastError();
}

}  // namespace w4a16
