// Pages of the 4-bit cache: which sequence has which (fork), and tokens moved inside a
// sequence (compact).  Both serve all layers of a model in one call, `stride` bytes apart.
#include "kv4.h"

namespace w4a16 {

namespace {

// ---- fork ----------------------------------------------------------------------------------
// One workgroup decides about the pages (a bit for each in LDS); nothing depends on the order in
// which its threads come along: bits are set, and of several rows the lowest number is kept.
// A second kernel copies what has to be copied, and writes what is left of the table.
//
// Bound: a chain of dependent loads, then HBM.  64 rows of 8 searches, 56 of which copy half a page
// in 32 layers of 8 heads of 128 channels (64 MB read and written): 9.4 us decide and 15 copy,
// 4.2 TB/s in pieces of 4.6 and 9.2 KB.  256 rows of up to 8192 tokens, one page in 64: 13 and 4 us.
// With every row's entries one after another, pages' bytes one by one and rows read again instead
// of kept: 23 us.
constexpr int FT = 1024;  // its threads
static_assert(KV4_FORK_ROWS <= 2 * FT, "a thread has two rows");

// A row of the new table: the old row and what it keeps of it.
struct ForkRow {
  int old, keep, whole, part, entries;  // entries: of the new row that have a page
};
__device__ __forceinline__ ForkRow fork_row(const Kv4ForkArgs& p, int r) {
  ForkRow x;
  x.old = p.parent[r];
  const int most = p.width * p.page;
  x.keep = 0;
  if (x.old >= 0 && x.old < p.batch) {
    const int len = p.lens[x.old];
    x.keep = p.keep ? p.keep[r] : len;
    x.keep = x.keep < len ? x.keep : len;
    x.keep = x.keep < 0 ? 0 : x.keep < most ? x.keep : most;
  } else {
    x.old = 0;
  }
  int room = p.room ? p.room[r] : 0;
  room = room < x.keep ? x.keep : room < most ? room : most;
  x.whole = x.keep / p.page;
  x.part = x.keep % p.page != 0;
  x.entries = room / p.page + (room % p.page != 0);
  return x;
}
__device__ __forceinline__ int fork_entry(const Kv4ForkArgs& p, int row, int at) {
  const int page = p.table[(size_t)row * p.width + at];
  return page >= 0 && page < p.pages ? page : -1;
}

__device__ __forceinline__ uint32_t slot_of(int page, uint32_t slots) {
  return ((uint32_t)page * 2654435761u >> 12) & (slots - 1);
}

// Sums of x over the threads before each one, and over all.
__device__ __forceinline__ int sums_before(int x, int* part, int& all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int upto = x;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int y = __shfl_up(upto, off);
    if (lane >= off) upto += y;
  }
  if (lane == 63) part[wave] = upto;
  __syncthreads();
  int before = 0;
  all = 0;
  for (int i = 0; i < FT / 64; ++i) {
    if (i < wave) before += part[i];
    all += part[i];
  }
  __syncthreads();
  return before + upto - x;
}

__global__ __launch_bounds__(FT) void kv4_fork_kernel(Kv4ForkArgs p, int slots) {
  extern __shared__ int lds[];
  const int words = (p.pages + 31) / 32, per = (words + FT - 1) / FT;
  uint32_t* taken = reinterpret_cast<uint32_t*>(lds);  // [words]: a page is held or pinned
  int* key = lds + words;       // [slots]: a page that rows want to go on in
  int* low = key + slots;       // [slots]: the lowest of them
  int* old = low + slots;       // [rows]
  int* whole = old + p.rows;    // [rows]; then the first entry that gets a new page
  int* start = whole + p.rows;  // [rows]: pages given to the rows before
  int* free_upto = start + p.rows;  // [FT]: free pages in the words of the threads before
  __shared__ int part[FT / 64];
  const int tid = threadIdx.x;

  // rows tid and tid + FT, in registers: their loads are in flight beside those of `pinned`
  ForkRow row[2];
  int page[2];  // the last one of which a part is kept, -1: there is none
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (k * FT + tid < p.rows) row[k] = fork_row(p, k * FT + tid);
  // a wave makes two words of 64 pages' bytes, eight times in flight
  for (int w0 = 2 * (tid >> 6); w0 < words; w0 += 8 * 2 * (FT / 64)) {
    bool held[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = 32 * (w0 + j * 2 * (FT / 64)) + (tid & 63);
      held[j] = i >= p.pages || (p.pinned && p.pinned[i] != 0);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint64_t bits = __ballot(held[j]);
      const int w = w0 + j * 2 * (FT / 64) + (tid & 63);
      if ((tid & 63) < 2 && w < words) taken[w] = (uint32_t)(bits >> (32 * (tid & 63)));
    }
  }
  for (int i = tid; i < slots; i += FT) {
    key[i] = -1;
    low[i] = p.rows;
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int r = k * FT + tid;
    page[k] = -1;
    if (r >= p.rows) continue;
    p.lens_out[r] = row[k].keep;
    old[r] = row[k].old;
    whole[r] = row[k].whole;
    if (row[k].part) page[k] = fork_entry(p, row[k].old, row[k].whole);
  }
  __syncthreads();
  {
    // Pages held whole: 16 threads to a row, more where there are fewer than 64 rows, with 8
    // entries each in flight.
    int wide = FT;
    while (wide > 16 && wide * p.rows > FT) wide >>= 1;
    for (int r = tid / wide; r < p.rows; r += FT / wide) {
      const int n = whole[r], from = old[r];
      for (int i0 = tid % wide; i0 < n; i0 += 8 * wide) {
        int x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int i = i0 + j * wide;
          x[j] = p.table[(size_t)from * p.width + (i < n ? i : i0)];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (x[j] >= 0 && x[j] < p.pages) atomicOr(taken + (x[j] >> 5), 1u << (x[j] & 31));
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (page[k] < 0) continue;
    // twice as many slots as rows: there is always a free one
    for (uint32_t i = slot_of(page[k], slots);; i = (i + 1) & (slots - 1)) {
      const int was = atomicCAS(key + i, -1, page[k]);
      if (was == -1 || was == page[k]) {
        atomicMin(low + i, k * FT + tid);
        break;
      }
    }
  }
  __syncthreads();
  // who goes on in its last page, and how many pages each row is given
  int mine[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int r = k * FT + tid;
    if (r >= p.rows) continue;
    const ForkRow& x = row[k];
    mine[k] = x.entries - x.whole - x.part;
    int at = x.whole + x.part;
    if (x.part) {
      if (page[k] >= 0) {
        uint32_t i = slot_of(page[k], slots);
        while (key[i] != page[k]) i = (i + 1) & (slots - 1);
        // read before it is set for this row itself; the others of this page find `low` another
        if (low[i] != r || (taken[page[k] >> 5] >> (page[k] & 31) & 1u) != 0) {
          ++mine[k];
          at = x.whole;
        } else {
          atomicOr(taken + (page[k] >> 5), 1u << (page[k] & 31));
        }
      }
      if (at != x.whole) p.table_out[(size_t)r * p.width + x.whole] = page[k];
    }
    whole[r] = at;
  }
  __syncthreads();
  int need = 0;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (k * FT >= p.rows) break;
    int all;
    const int before = sums_before(mine[k], part, all);
    if (k * FT + tid < p.rows) start[k * FT + tid] = need + before;
    need += all;
  }
  int spare;
  {
    int n = 0;
    for (int w = tid * per; w < (tid + 1) * per && w < words; ++w) n += 32 - __popc(taken[w]);
    free_upto[tid] = sums_before(n, part, spare);
  }
  if (tid == 0 && p.missing) *p.missing = need > spare ? need - spare : 0;
  __syncthreads();
  for (int k = tid; k < need; k += FT) {
    int r = 0;  // the last row that starts at or before k
    for (int lo = 0, hi = p.rows; lo < hi;) {
      const int mid = (lo + hi) / 2;
      if (start[mid] <= k) {
        r = mid;
        lo = mid + 1;
      } else {
        hi = mid;
      }
    }
    int page = -1;
    if (k < spare) {
      int t = 0;
      for (int lo = 0, hi = FT; lo < hi;) {
        const int mid = (lo + hi) / 2;
        if (free_upto[mid] <= k) {
          t = mid;
          lo = mid + 1;
        } else {
          hi = mid;
        }
      }
      int left = k - free_upto[t], w = t * per;
      uint32_t bits = ~taken[w];
      while (left >= __popc(bits)) {
        left -= __popc(bits);
        bits = ~taken[++w];
      }
      for (; left > 0; --left) bits &= bits - 1;
      page = 32 * w + __builtin_ctz(bits);
    }
    p.table_out[(size_t)r * p.width + whole[r] + k - start[r]] = page;
  }
}

// What is left of the new table, and the copies of last pages: blocks that have something in
// them.  Grid: (waves / 4 that share the kv heads of all layers, groups of `group` <= 64 rows).
template <int D, int NG>
__global__ __launch_bounds__(256) void kv4_fork_copy_kernel(Kv4ForkArgs p, int group) {
  const int r0 = blockIdx.y * group;
  const int rows = p.rows - r0 < group ? p.rows - r0 : group;
  const unsigned all = (unsigned)rows * p.width;
  for (unsigned i = blockIdx.x * 256 + threadIdx.x; i < all; i += gridDim.x * 256) {
    const int r = r0 + (int)(i / p.width), at = i % p.width;
    const ForkRow x = fork_row(p, r);
    if (at < x.whole) p.table_out[(size_t)r * p.width + at] = fork_entry(p, x.old, at);
    else if (at >= x.entries) p.table_out[(size_t)r * p.width + at] = -1;
  }
  const int lane = threadIdx.x & 63;
  const int unit = __builtin_amdgcn_readfirstlane((int)(blockIdx.x * 4 + (threadIdx.x >> 6)));
  if (unit >= p.layers * p.heads) return;
  const size_t head_bytes = (size_t)(p.page / 32) * kv4_block_bytes(D, NG);
  int from = -1, to = -1, size = 0;
  if (lane < rows) {
    const ForkRow x = fork_row(p, r0 + lane);
    if (x.part) {
      from = fork_entry(p, x.old, x.whole);
      to = p.table_out[(size_t)(r0 + lane) * p.width + x.whole];
      size = (x.keep % p.page + 31) / 32 * kv4_block_bytes(D, NG);
    }
  }
  char* base = p.cache + (size_t)(unit / p.heads) * p.stride + (size_t)(unit % p.heads) * head_bytes;
  for (uint64_t go = __ballot(from >= 0 && to >= 0 && to != from); go; go &= go - 1) {
    const int l = __builtin_ctzll(go);
    const u32x4v* src = reinterpret_cast<const u32x4v*>(
        base + (size_t)__builtin_amdgcn_readlane(from, l) * p.heads * head_bytes);
    u32x4v* dst = reinterpret_cast<u32x4v*>(
        base + (size_t)__builtin_amdgcn_readlane(to, l) * p.heads * head_bytes);
    const int n = __builtin_amdgcn_readlane(size, l) / 16;
    // eight loads in flight; stores past the caches (15 us instead of 19 for the 64 rows above)
    for (int i0 = lane; i0 < n; i0 += 8 * 64) {
      u32x4v x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i0 + 64 * j < n) x[j] = src[i0 + 64 * j];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i0 + 64 * j < n) __builtin_nontemporal_store(x[j], dst + i0 + 64 * j);
    }
  }
}

// ---- compact -------------------------------------------------------------------------------
// A wave serves the accepted nodes of one sequence in one layer and kv head, eight at a time.
// Node path[j] goes to place j <= path[j], so what a later node brings has not been written
// over by an earlier one, and within eight all is read before any of it is written.  Of K a lane
// has one of a node's four runs of words; of V it has one or two channels, whose nibbles lie in
// words with other tokens': it reads the (at most three) words that eight places in a row lie
// in, and no other lane writes those.
//
// Bound: HBM, in pieces of 16 to 256 bytes.  149 moved tokens of 48 sequences in 64 layers of 8 heads
// of 128 channels: 22 MB of tokens, for which 76 MB go to and from memory, in 38 us; one sequence,
// 32 layers, 4.5 us.
template <int D, int NG>
__global__ __launch_bounds__(256) void kv4_compact_kernel(Kv4CompactArgs p, int waves) {
  constexpr int W = D / 32;  // words of a run of K
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(blockIdx.x * 4 + (threadIdx.x >> 6)));
  const int b = blockIdx.y;
  const Kv4Seq s = kv4_seq(p.rows, p.lens, b, p.tokens, p.max_new);
  int count = p.count[b];
  count = count < 0 ? 0 : count;
  count = count < p.max_path ? count : p.max_path;
  count = count < s.n ? count : s.n;
  const int from = s.len - s.n;
  if (wave == 0 && lane == 0) p.lens_out[b] = from + count > 0 ? from + count : 0;
  const int page_blocks = p.page / 32;
  const size_t head_bytes = (size_t)page_blocks * kv4_block_bytes(D, NG);
  for (int j0 = 0; j0 < count; j0 += 8) {
    // lane j < 8: where node path[j0 + j] lies and where it goes
    const int j = j0 + (lane & 7);
    int node = j;
    if (j < count) node = p.path[(size_t)b * p.max_path + j];
    bool go = j < count && node > j && node < s.n && from + j >= 0;
    int src_page = -1, dst_page = -1;
    const int src = from + node, dst = from + j;
    if (go) {
      src_page = kv4_page(p.table, b, src >> 5, page_blocks, p.width, p.pages);
      dst_page = kv4_page(p.table, b, dst >> 5, page_blocks, p.width, p.pages);
    }
    go = go && src_page >= 0 && dst_page >= 0;
    const uint32_t goes = (uint32_t)__ballot(go) & 0xFFu;
    if (goes == 0) continue;
    // bytes from a head's first page to the blocks, the same for every unit
    auto block_at = [&](int page, int pos) {
      return (size_t)(page < 0 ? 0 : page) * p.heads * head_bytes +
             (size_t)((pos >> 5) % page_blocks) * kv4_block_bytes(D, NG);
    };
    const size_t src_at = block_at(src_page, src), dst_at = block_at(dst_page, dst);
    auto of_lane = [](size_t x, int l) {
      return (size_t)(uint32_t)__builtin_amdgcn_readlane((int)x, l) |
             (size_t)(uint32_t)__builtin_amdgcn_readlane((int)(x >> 32), l) << 32;
    };
    auto of_each = [](size_t x, int l) {
      return (size_t)(uint32_t)__shfl((int)x, l) | (size_t)(uint32_t)__shfl((int)(x >> 32), l) << 32;
    };
    // K: lane 4 i + g < 32 has run g of node i; parameters: lanes 8 i .. 8 i + 7 have node i's
    typedef uint32_t run __attribute__((ext_vector_type(W)));
    const int ki = (lane >> 2) & 7, pi = lane >> 3;
    const bool kgo = lane < 32 && (goes >> ki & 1u) != 0, pgo = (goes >> pi & 1u) != 0;
    auto k_place = [&](int pos) {
      return (size_t)(((pos >> 4 & 1) * 64 + 16 * (lane & 3) + (pos & 15)) * W * 4);
    };
    constexpr int NP = 4 * NG;  // K's and V's s and m of each group
    auto p_place = [&](int pos) {
      return (size_t)(32 * D + 2 * ((lane & 7) * 32 + kv4_token_slot(pos & 31)));
    };
    const size_t k_src = of_each(src_at, ki) + k_place(__shfl(src, ki));
    const size_t k_dst = of_each(dst_at, ki) + k_place(__shfl(dst, ki));
    const size_t p_src = of_each(src_at, pi) + p_place(__shfl(src, pi));
    const size_t p_dst = of_each(dst_at, pi) + p_place(__shfl(dst, pi));
    // V: channels 64 h + lane; the words of a block of lane group tg
    const int v_lane = 16 * D + ((lane & 15) * 4 + (lane >> 4)) * 4;
    const int d0 = from + j0, skew = d0 & 3;
    // the places of nodes j0 .. j0 + 7 that lie in group y of four, which share a word
    auto group_of = [&](int y) { return goes & (uint32_t)((0xFULL << (4 * y)) >> skew); };
    for (int unit = wave; unit < p.layers * p.heads; unit += waves) {
      char* base = p.cache + (size_t)(unit / p.heads) * p.stride +
                   (size_t)(unit % p.heads) * head_bytes;
      run kw;
      if (kgo) kw = *reinterpret_cast<const run*>(base + k_src);
      uint16_t par[(NP + 7) / 8];
#pragma unroll
      for (int i = 0; i < (NP + 7) / 8; ++i)
        if (pgo && 8 * i + (lane & 7) < NP)
          par[i] = *reinterpret_cast<const uint16_t*>(base + p_src + 512 * i);
      uint32_t code[D / 64][8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (goes >> i & 1u) {
          const int tg = (__builtin_amdgcn_readlane(src, i) >> 2) & 3;
          const char* at = base + of_lane(src_at, i) + 256 * tg;
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            code[h][i] = *reinterpret_cast<const uint32_t*>(at + v_lane + 1024 * h);
        }
      uint32_t word[3][D / 64];
#pragma unroll
      for (int y = 0; y < 3; ++y)
        if (const uint32_t in = group_of(y)) {
          const int i = __builtin_ctz(in);
          const char* at = base + of_lane(dst_at, i) + 256 * (((d0 + i) >> 2) & 3);
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            word[y][h] = *reinterpret_cast<const uint32_t*>(at + v_lane + 1024 * h);
        }
      if (kgo) *reinterpret_cast<run*>(base + k_dst) = kw;
#pragma unroll
      for (int i = 0; i < (NP + 7) / 8; ++i)
        if (pgo && 8 * i + (lane & 7) < NP)
          *reinterpret_cast<uint16_t*>(base + p_dst + 512 * i) = par[i];
#pragma unroll
      for (int y = 0; y < 3; ++y)
        if (const uint32_t in = group_of(y)) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if ((in >> i & 1u) == 0) continue;
            const int ts = __builtin_amdgcn_readlane(src, i), td = d0 + i;
            const int ss = 4 * nib_pos(((ts >> 4) & 1) * 4 + (ts & 3));
            const int sd = 4 * nib_pos(((td >> 4) & 1) * 4 + (td & 3));
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              word[y][h] = (word[y][h] & ~(15u << sd)) | ((code[h][i] >> ss & 15u) << sd);
          }
          const int i = __builtin_ctz(in);
          char* at = base + of_lane(dst_at, i) + 256 * (((d0 + i) >> 2) & 3);
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            *reinterpret_cast<uint32_t*>(at + v_lane + 1024 * h) = word[y][h];
        }
    }
  }
}

}  // namespace

hipError_t launch_kv4_fork(const Kv4ForkArgs& a, int D, int groups, hipStream_t st) {
  int slots = 64;
  while (slots < 2 * a.rows) slots *= 2;
  const size_t lds = ((a.pages + 31) / 32 + 2 * slots + 3 * a.rows + FT) * sizeof(int);
  constexpr int most = (KV4_FORK_PAGES / 32 + 4 * KV4_FORK_ROWS + 3 * KV4_FORK_ROWS + FT) * sizeof(int);
  hipError_t e = hipSuccess;
  // the same for every call, since another thread's smaller one may come between this and the launch
  if (lds > 65536)
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(kv4_fork_kernel),
                            hipFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kv4_fork_kernel, dim3(1), dim3(FT), lds, st, a, slots);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  // A wave has one layer's kv head, and one row up to 16384 waves (two for every one that the
  // card holds at a time), more rows past that.  Four heads a wave instead, which look up once
  // what there is to do: 24 us where one takes 20 (64 rows of which 56 copy, 32 layers of 8 heads).
  const int units = a.layers * a.heads;
  long long group = (long long)units * a.rows / 16384;
  group = group < 1 ? 1 : group > 64 ? 64 : group;
  const dim3 grid((units + 3) / 4, (unsigned)((a.rows + group - 1) / group));
  auto fn = D == 128 ? (groups == 1   ? kv4_fork_copy_kernel<128, 1>
                        : groups == 2 ? kv4_fork_copy_kernel<128, 2>
                                      : kv4_fork_copy_kernel<128, 4>)
                     : (groups == 1 ? kv4_fork_copy_kernel<64, 1> : kv4_fork_copy_kernel<64, 2>);
  hipLaunchKernelGGL(fn, grid, dim3(256), 0, st, a, (int)group);
  return hipGetLastError();
}

hipError_t launch_kv4_compact(const Kv4CompactArgs& a, int D, int groups, hipStream_t st) {
  // Units of a wave: two where that leaves 8192 waves.  1 / 2 / 4 / 8 / 16 units a wave: 40 / 38 / 40 /
  // 49 / 70 us for 48 sequences, 64 layers of 8 heads.
  const int units = a.layers * a.heads;
  long long each = (long long)units * a.batch / 8192;
  each = each < 1 ? 1 : each > 2 ? 2 : each;
  const int groups4 = (int)((units + 4 * each - 1) / (4 * each));
  auto fn = D == 128 ? (groups == 1   ? kv4_compact_kernel<128, 1>
                        : groups == 2 ? kv4_compact_kernel<128, 2>
                                      : kv4_compact_kernel<128, 4>)
                     : (groups == 1 ? kv4_compact_kernel<64, 1> : kv4_compact_kernel<64, 2>);
  hipLaunchKernelGGL(fn, dim3(groups4, a.batch), dim3(256), 0, st, a, 4 * groups4);
  return hipGetLastError();
}

}  // namespace w4a16
