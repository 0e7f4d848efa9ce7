// Embedding lookup and its gradient.
//
//   forward   out[i] = scale * table[id_i]           (id_i < 0: zeros)
//   backward  dtable[v] = scale * sum_{i: id_i = v} dout[i]   [+ dtable[v]]
//
// Both move bytes and compute next to nothing.  The gradient adds the rows of
// equal ids in an order that their positions fix, in fp32, and rounds once, so that
// it is the same for every run: the (id, position) pairs are sorted stably, the
// sorted list is cut into runs, one block sums each run,
// and ids that cross a cut are joined from the runs' partial sums in a fixed order.
// Work is even over blocks however often an id comes.  Blocks of the same
// launch write the zeros of the rows that no id names.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "internal.h"
#include "ptx.cuh"
#include "vocab.h"

namespace dmuon {
namespace {

// ---------------------------------------------------------- rows of 8 values
template <bool BF16>
__device__ __forceinline__ void load8(const void* p, float (&v)[8]) {
  if (BF16) {
    const uint4 q = *static_cast<const uint4*>(p);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    const float4 a = static_cast<const float4*>(p)[0], b = static_cast<const float4*>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}

template <bool BF16>
__device__ __forceinline__ void store8(void* p, const float (&v)[8]) {
  if (BF16) {
    *static_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                         pack_bf16x2(v[6], v[7]));
  } else {
    static_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    static_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

template <bool BF16>
__device__ __forceinline__ float load1(const void* p) {
  return BF16 ? bf16_bits_to_f32(*static_cast<const uint16_t*>(p)) : *static_cast<const float*>(p);
}
template <bool BF16>
__device__ __forceinline__ void store1(void* p, float v) {
  if (BF16)
    *static_cast<uint16_t*>(p) = to_bf16_bits(v);
  else
    *static_cast<float*>(p) = v;
}
template <bool BF16>
__device__ __forceinline__ const void* at(const void* p, int64_t i) {
  return static_cast<const char*>(p) + i * (BF16 ? 2 : 4);
}
template <bool BF16>
__device__ __forceinline__ void* at(void* p, int64_t i) {
  return static_cast<char*>(p) + i * (BF16 ? 2 : 4);
}

// -------------------------------------------------------------------- forward
// One warp takes 1024 columns of one token: four 16-byte (bf16) loads a lane
// in flight.  VEC: rows start on 16 bytes and dim % 8 == 0.
constexpr int kFwdCols = 1024;

template <bool TB, bool OB, bool VEC>
__global__ void __launch_bounds__(256) embed_forward_kernel(const EmbedForward E) {
  pdl_launch();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int segs = (E.dim + kFwdCols - 1) / kFwdCols;
  const int64_t tasks = E.n * segs, warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); t < tasks; t += warps) {
    const int64_t i = t / segs;
    const int c0 = static_cast<int>(t - i * segs) * kFwdCols;
    bool bad = false;
    const int id = load_id(E.ids, i, &bad);
    if (bad && lane == 0) atomicCAS(E.err, 0, kErrBadIndex);
    const void* src = at<TB>(E.table, static_cast<int64_t>(id < 0 ? 0 : id) * E.ld_table);
    void* dst = at<OB>(E.out, i * E.ld_out);
    if (VEC) {
      float v[4][8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = c0 + 256 * k + 8 * lane;
        if (id >= 0 && c < E.dim) load8<TB>(at<TB>(src, c), v[k]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = c0 + 256 * k + 8 * lane;
        if (c >= E.dim) break;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[k][j] = id >= 0 ? v[k][j] * E.scale : 0.f;
        store8<OB>(at<OB>(dst, c), v[k]);
      }
    } else {
      const int end = min(E.dim, c0 + kFwdCols);
      for (int c = c0 + lane; c < end; c += 32) store1<OB>(at<OB>(dst, c), id >= 0 ? load1<TB>(at<TB>(src, c)) * E.scale : 0.f);
    }
  }
}

// ----------------------------------------------------------------------- sort
// Stable radix sort of (id, position), least significant digit first, at most
// 9 bits a pass.  A block takes kSortThreads * ITEMS pairs; warp w holds
// 32 * ITEMS consecutive ones (ITEMS rounds of one per lane).  Entries that
// are not counted get the key `vocab`, which sorts last.
constexpr int kSortThreads = 1024;
constexpr int kSortTile = 4096;  // pairs of a block in the sort over several launches
constexpr int kDigitBits = 9, kBins = 1 << kDigitBits;
constexpr int kClusterMost = 8, kClusterItems = 8;
constexpr int kOneLaunch = kSortThreads * kClusterMost * kClusterItems;

__device__ __forceinline__ uint32_t first_key(const EmbedBackward& E, int64_t i) {
  bool bad = false;
  const int id = load_id(E.ids, i, &bad);
  if (bad) atomicCAS(E.err, 0, kErrBadIndex);
  return id < 0 ? static_cast<uint32_t>(E.ids.vocab) : static_cast<uint32_t>(id);
}

// Ranks of this block's pairs among its pairs of the same digit: rank[k] within the
// warp, and cnt[w][d] the number in the warps before w.  Called by all threads;
// returns (thread d) the block's number of digit d.
template <int ITEMS>
__device__ __forceinline__ uint32_t block_ranks(const uint32_t (&digit)[ITEMS], const bool (&has)[ITEMS],
                                                uint16_t (*cnt)[kBins], uint32_t (&rank)[ITEMS]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t* mine = reinterpret_cast<uint32_t*>(cnt[warp]);
#pragma unroll
  for (int d = 0; d < kBins / 64; ++d) mine[d * 32 + lane] = 0;
  __syncwarp();
  // Lanes of the same digit, by a ballot per bit: 20.5 us for 32768 entries where
  // __match_any_sync took 23.
  uint32_t same[ITEMS];
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    const uint32_t m = __ballot_sync(0xffffffffu, has[k]);
    same[k] = has[k] ? m : ~m;
#pragma unroll
    for (int b = 0; b < kDigitBits; ++b) {
      const bool one = (digit[k] >> b) & 1u;
      const uint32_t v = __ballot_sync(0xffffffffu, one);
      same[k] &= one ? v : ~v;
    }
  }
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    const uint32_t before = has[k] ? cnt[warp][digit[k]] : 0u;
    rank[k] = before + __popc(same[k] & ((1u << lane) - 1u));
    __syncwarp();
    if (has[k] && lane == __ffs(same[k]) - 1) cnt[warp][digit[k]] = static_cast<uint16_t>(before + __popc(same[k]));
    __syncwarp();
  }
  __syncthreads();
  uint32_t total = 0;
  if (threadIdx.x < kBins) {
    uint32_t c[kSortThreads / 32];
#pragma unroll
    for (int w = 0; w < kSortThreads / 32; ++w) c[w] = cnt[w][threadIdx.x];
#pragma unroll
    for (int w = 0; w < kSortThreads / 32; ++w) {
      cnt[w][threadIdx.x] = static_cast<uint16_t>(total);
      total += c[w];
    }
  }
  __syncthreads();
  return total;
}

// Exclusive scan over the block's threads.
__device__ __forceinline__ uint32_t scan_threads(uint32_t v, uint32_t* tmp) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  if (lane == 31) tmp[warp] = s;
  __syncthreads();
  if (warp == 0) {
    uint32_t t = tmp[lane], x = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += u;
    }
    tmp[lane] = x - t;
  }
  __syncthreads();
  const uint32_t out = s - v + tmp[warp];
  __syncthreads();
  return out;
}

// Bit v of the map: some entry names row v.  Set where a key differs from the
// one before it in the sorted list, so once for each row.
__device__ __forceinline__ void mark_row(const EmbedBackward& E, uint32_t key, uint32_t before, bool first) {
  if (key < static_cast<uint32_t>(E.ids.vocab) && (first || before != key))
    atomicOr(E.present + (key >> 5), 1u << (key & 31));
}

__device__ __forceinline__ uint32_t ld_shared_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// Up to kCounted entries: every entry's place is counted, as the number of pairs
// before its own.  n^2 comparisons over all SMs are one step where the passes of a
// radix sort are a chain of them: 3.2 us with 1000 entries of 32000 rows, where the
// cluster below takes 8.9, and 6.1 for 10.5 with 4096 of 50257.  A block reads the
// whole list; two warps place four entries, each lane counting over a 64th of the
// list.  Equal keys before the entry's own quad (four entries) count, those in it
// up to the entry, those after it do not.  With `present` the blocks also share out
// the map's words, each looking through the list for its own, so that nothing has to
// be cleared before; that takes half of the time, and half of the entries is the
// limit (3000 of 128256: 7.4 us for 11.4 alone, but 58 for 55 in a call).
constexpr int kCounted = 4096, kCountThreads = 512, kCountEntries = 32, kMapWords = 1024;

__global__ void __launch_bounds__(kCountThreads) embed_count_kernel(const EmbedBackward E) {
  __shared__ __align__(16) uint32_t keys[kCounted];
  __shared__ uint32_t map[kMapWords];
  __shared__ uint32_t upper[kCountEntries];  // places counted by the second half of the warps
  const int n = static_cast<int>(E.n), padded = (n + 3) & ~3, t = threadIdx.x, lane = t & 31, warp = t >> 5;
  pdl_wait();
  pdl_launch();
  constexpr int kLoads = kCounted / kCountThreads;
  int id[kLoads];
  bool bad = false;
#pragma unroll
  for (int k = 0; k < kLoads; ++k) {
    const int i = t + k * kCountThreads;
    id[k] = i < n ? load_id(E.ids, i, &bad) : -1;
  }
  if (bad && blockIdx.x == 0) atomicCAS(E.err, 0, kErrBadIndex);
#pragma unroll
  for (int k = 0; k < kLoads; ++k) {
    const int i = t + k * kCountThreads;
    if (i < padded) keys[i] = i >= n ? 0xffffffffu : id[k] < 0 ? static_cast<uint32_t>(E.ids.vocab) : static_cast<uint32_t>(id[k]);
  }
  __syncthreads();
  constexpr int kHalf = kCountEntries / 4;  // warps that take four entries each; the others take the list's odd quads
  const int group = warp % kHalf, half = warp / kHalf;
  const int first = static_cast<int>(blockIdx.x) * kCountEntries + group * 4, own = first >> 2;
  uint32_t places[4] = {0, 0, 0, 0}, k[4] = {0, 0, 0, 0};
  if (first < n) {
    const uint4* quads = reinterpret_cast<const uint4*>(keys);
    const uint4 mine = quads[own];
    k[0] = mine.x; k[1] = mine.y; k[2] = mine.z; k[3] = mine.w;
#pragma unroll 2
    for (int q = 32 * half + lane; q < padded >> 2; q += 64) {
      const uint4 v = quads[q];
      const uint32_t equal = q < own ? 1u : 0u;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t below = k[e] + equal;  // keys are at most 2^24; the padding's places are not used
        places[e] += (v.x < below ? 1u : 0u) + (v.y < below ? 1u : 0u) + (v.z < below ? 1u : 0u) + (v.w < below ? 1u : 0u);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      places[e] = __reduce_add_sync(0xffffffffu, places[e]);
      if (half == 1 && lane == 0) upper[group * 4 + e] = places[e];
    }
  }
  __syncthreads();
  if (half == 0 && lane == 0) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (first + e >= n) continue;
      uint32_t to = places[e] + upper[group * 4 + e];
#pragma unroll
      for (int c = 0; c < e; ++c) to += k[c] == k[e] ? 1u : 0u;
      __stcg(E.key[0] + to, k[e]);
      __stcg(E.pos[0] + to, static_cast<uint32_t>(first + e));
    }
  }
  if (!E.present) return;
  const int words = (E.ids.vocab + 31) / 32, span = (words + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
  const int end = min(words, (static_cast<int>(blockIdx.x) + 1) * span);
  for (int w0 = static_cast<int>(blockIdx.x) * span; w0 < end; w0 += kMapWords) {
    const int here = min(kMapWords, end - w0);
    __syncthreads();  // the words before these are out
    for (int i = t; i < here; i += kCountThreads) map[i] = 0u;
    __syncthreads();
    for (int i = t; i < n; i += kCountThreads) {
      const int w = static_cast<int>(keys[i] >> 5) - w0;
      if (w >= 0 && w < here) atomicOr(map + w, 1u << (keys[i] & 31));
    }
    __syncthreads();
    for (int i = t; i < here; i += kCountThreads) E.present[w0 + i] = map[i];
  }
}

// Up to kOneLaunch entries: the whole sort in one launch of one cluster.  The
// CTAs read one another's digit counts through distributed shared memory, and
// the cluster barriers order the pairs that move through global memory.  With
// 8192 ids of a 128256-row table that is 8 us, where a histogram, a scan and a
// scatter for each pass took 28.
struct ClusterSort {
  uint16_t cnt[kSortThreads / 32][kBins];
  uint32_t hist[2][kBins];
  uint32_t base[kBins];
  uint32_t tmp[32];
};

template <int ITEMS>
__global__ void __launch_bounds__(kSortThreads) embed_sort_cluster_kernel(const EmbedBackward E, int passes, int bits) {
  __shared__ ClusterSort S;
  const int n = static_cast<int>(E.n);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank_in_cluster = static_cast<int>(cluster_ctarank()), ctas = static_cast<int>(gridDim.x);
  const int first = (rank_in_cluster * kSortThreads + warp * 32) * ITEMS + lane;
  uint32_t key[ITEMS], pos[ITEMS], digit[ITEMS], rank[ITEMS];
  bool has[ITEMS];
  pdl_launch();
  pdl_wait();
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    const int i = first + 32 * k;
    has[k] = i < n;
    pos[k] = static_cast<uint32_t>(i);
    key[k] = has[k] ? first_key(E, i) : 0u;
  }
  if (E.present) {
    const int words = (E.ids.vocab + 31) / 32;
    for (int i = rank_in_cluster * kSortThreads + static_cast<int>(threadIdx.x); i < words; i += ctas * kSortThreads) E.present[i] = 0u;
  }
  for (int p = 0; p < passes; ++p) {
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) digit[k] = (key[k] >> (p * bits)) & ((1u << bits) - 1u);
    const uint32_t mine = block_ranks<ITEMS>(digit, has, S.cnt, rank);
    uint32_t* hist = S.hist[p & 1];
    if (threadIdx.x < kBins) hist[threadIdx.x] = mine;
    cluster_sync_all();
    uint32_t before = 0, total = 0;
    if (threadIdx.x < kBins) {
      const uint32_t at = smem_u32(hist + threadIdx.x);
      for (int r = 0; r < ctas; ++r) {
        const uint32_t c = ld_shared_cluster_u32(mapa_shared(at, static_cast<uint32_t>(r)));
        before += r < rank_in_cluster ? c : 0u;
        total += c;
      }
    }
    const uint32_t b = scan_threads(total, S.tmp);
    if (threadIdx.x < kBins) S.base[threadIdx.x] = b + before;
    __syncthreads();
    const int to_buf = p & 1;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k)
      if (has[k]) {
        const uint32_t to = S.base[digit[k]] + S.cnt[warp][digit[k]] + rank[k];
        __stcg(E.key[to_buf] + to, key[k]);
        __stcg(E.pos[to_buf] + to, pos[k]);
      }
    __syncwarp();
    cluster_sync_all();  // every CTA's pairs are in place; every read of hist[p & 1] is done
    if (p + 1 < passes) {
#pragma unroll
      for (int k = 0; k < ITEMS; ++k)
        if (has[k]) {
          key[k] = load_l2(E.key[to_buf] + first + 32 * k);
          pos[k] = load_l2(E.pos[to_buf] + first + 32 * k);
        }
    }
  }
  if (E.present) {
    const uint32_t* sorted = E.key[(passes - 1) & 1];
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      const int i = first + 32 * k;
      if (i < n) mark_row(E, load_l2(sorted + i), i > 0 ? load_l2(sorted + i - 1) : 0u, i == 0);
    }
  }
}

constexpr int kSortItems = kSortTile / kSortThreads;

// Longer lists: per pass a histogram of each block, a scan over the blocks of
// each digit, and the scatter.  hist[digit][block]; hist[kBins * blocks + digit]: totals.
__global__ void __launch_bounds__(kSortThreads) embed_hist_kernel(const EmbedBackward E, int pass, int bits, int from) {
  __shared__ uint32_t h[kBins];
  for (int d = threadIdx.x; d < kBins; d += kSortThreads) h[d] = 0;
  __syncthreads();
  pdl_launch();
  pdl_wait();
  if (pass == 0 && E.present) {
    const int64_t words = (E.ids.vocab + 31) / 32;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kSortThreads + threadIdx.x; i < words; i += static_cast<int64_t>(gridDim.x) * kSortThreads)
      E.present[i] = 0u;
  }
  for (int k = 0; k < kSortItems; ++k) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kSortTile + k * kSortThreads + threadIdx.x;
    if (i < E.n) {
      const uint32_t key = pass == 0 ? first_key(E, i) : E.key[from][i];
      atomicAdd(&h[(key >> (pass * bits)) & ((1u << bits) - 1u)], 1u);  // integers: any order gives the same
    }
  }
  __syncthreads();
  for (int d = threadIdx.x; d < kBins; d += kSortThreads) E.hist[static_cast<int64_t>(d) * gridDim.x + blockIdx.x] = h[d];
}

__global__ void __launch_bounds__(kSortThreads) embed_scan_kernel(uint32_t* hist, int blocks) {
  __shared__ uint32_t tmp[32];
  __shared__ uint32_t chunk;
  pdl_launch();
  pdl_wait();
  uint32_t* h = hist + static_cast<int64_t>(blockIdx.x) * blocks;
  uint32_t base = 0;
  for (int b0 = 0; b0 < blocks; b0 += kSortThreads) {
    const int b = b0 + threadIdx.x;
    const uint32_t v = b < blocks ? h[b] : 0u;
    const uint32_t s = scan_threads(v, tmp);
    if (b < blocks) h[b] = base + s;
    if (threadIdx.x == kSortThreads - 1) chunk = s + v;
    __syncthreads();
    base += chunk;
    __syncthreads();
  }
  if (threadIdx.x == 0) hist[static_cast<int64_t>(kBins) * blocks + blockIdx.x] = base;
}

struct Scatter {
  uint16_t cnt[kSortThreads / 32][kBins];
  uint32_t base[kBins];
  uint32_t tmp[32];
};

__global__ void __launch_bounds__(kSortThreads) embed_scatter_kernel(const EmbedBackward E, int pass, int bits, int from) {
  __shared__ Scatter S;
  pdl_launch();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kSortTile + warp * 32 * kSortItems + lane;
  uint32_t key[kSortItems], pos[kSortItems], digit[kSortItems], rank[kSortItems];
  bool has[kSortItems];
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) {
    const int64_t i = i0 + 32 * k;
    has[k] = i < E.n;
    key[k] = pos[k] = 0;
    if (has[k]) {
      key[k] = pass == 0 ? first_key(E, i) : E.key[from][i];
      pos[k] = pass == 0 ? static_cast<uint32_t>(i) : E.pos[from][i];
    }
    digit[k] = (key[k] >> (pass * bits)) & ((1u << bits) - 1u);
  }
  const uint32_t total = threadIdx.x < kBins ? E.hist[static_cast<int64_t>(kBins) * gridDim.x + threadIdx.x] : 0u;
  const uint32_t b = scan_threads(total, S.tmp);
  if (threadIdx.x < kBins) S.base[threadIdx.x] = b + E.hist[static_cast<int64_t>(threadIdx.x) * gridDim.x + blockIdx.x];
  block_ranks<kSortItems>(digit, has, S.cnt, rank);
#pragma unroll
  for (int k = 0; k < kSortItems; ++k)
    if (has[k]) {
      const uint32_t to = S.base[digit[k]] + S.cnt[warp][digit[k]] + rank[k];
      E.key[from ^ 1][to] = key[k];
      E.pos[from ^ 1][to] = pos[k];
    }
}

__global__ void __launch_bounds__(kSortThreads) embed_mark_kernel(const EmbedBackward E, int from) {
  pdl_launch();
  pdl_wait();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kSortThreads + threadIdx.x;
  if (i < E.n) mark_row(E, E.key[from][i], i > 0 ? E.key[from][i - 1] : 0u, i == 0);
}

// ----------------------------------------------------------------------- sums
struct Runs {
  const uint32_t* key;
  const uint32_t* pos;
  int32_t run;        // sorted positions of a run, a multiple of 4
  int64_t n_runs;
  int32_t col_blocks;
  int32_t join_lanes, join_blocks;  // threads side by side in the join, and its column blocks
  int32_t zero_rows;                // rows of a warp that writes zeros
  int64_t ld_part;
};

// Adds to, or writes, VEC columns of a row.
template <bool GB, int VEC>
__device__ __forceinline__ void put_row(const EmbedBackward& E, uint32_t id, int c, const float (&acc)[VEC]) {
  void* dst = at<GB>(E.dtable, static_cast<int64_t>(id) * E.ld_dtable + c);
  if (VEC == 8) {
    float v[8];
    if (E.accumulate) {
      load8<GB>(dst, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = fmaf(E.scale, acc[j % VEC], v[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = E.scale * acc[j % VEC];
    }
    store8<GB>(dst, v);
  } else {
    store1<GB>(dst, E.accumulate ? fmaf(E.scale, acc[0], load1<GB>(dst)) : E.scale * acc[0]);
  }
}

// Zeros into rows that no entry names, by a warp each: four rows beside the sums (5001
// entries of 1031 x 1000 in fp32: 20.4 us a call, 22 with eight), eight where every
// block sorts the list first (100 entries of 50257 x 768: 19 us, 26 with four), 32 of
// at most kZeroShort bytes (5000 entries of 128256 x 256 in bf16: 27.6 us for 32;
// with rows of 2 KB they are too few warps, 22 us for 14 at 100 entries of 32000).
constexpr int kZeroShort = 512;
int zero_rows_of(int64_t row_bytes, int usual) { return row_bytes <= kZeroShort ? 32 : usual; }

// Row r0 + k for each bit k of `left`.
template <bool GB, bool VEC>
__device__ __forceinline__ void zero_marked(const EmbedBackward& E, int64_t r0, uint32_t left, int lane) {
  while (left) {
    const int k = __ffs(left) - 1;
    left &= left - 1;
    void* dst = at<GB>(E.dtable, (r0 + k) * E.ld_dtable);
    if (VEC) {
      const int n16 = E.dim / (GB ? 8 : 4);
#pragma unroll 4
      for (int c = lane; c < n16; c += 32) static_cast<uint4*>(dst)[c] = make_uint4(0, 0, 0, 0);
    } else {
      for (int c = lane; c < E.dim; c += 32) store1<GB>(at<GB>(dst, c), 0.f);
    }
  }
}

template <bool GB, bool VEC>
__device__ __forceinline__ void zero_rows(const EmbedBackward& E, int64_t r0, int most, int lane) {
  if (r0 >= E.ids.vocab) return;
  const int rows = static_cast<int>(min(static_cast<int64_t>(most), E.ids.vocab - r0));
  zero_marked<GB, VEC>(E, r0, (~load_l2(E.present + (r0 >> 5)) >> (r0 & 31)) & (0xffffffffu >> (32 - rows)), lane);
}

// VEC columns a thread.  n_runs * col_blocks blocks take a run and a column
// block each, four rows in flight; the others, spread evenly among them so
// that reads and writes share the memory all along, write zeros.  Four blocks an
// SM (64 registers a thread): 32768 entries added at 128256 x 4096 in bf16 take 128 us
// where three blocks take 137, and with five (and spills) 154.
template <bool DB, bool GB, int VEC>
__global__ void __launch_bounds__(256, 4) embed_sum_kernel(const EmbedBackward E, const Runs R) {
  __shared__ uint32_t keys[kEmbedRun + 2], pos[kEmbedRun];
  pdl_launch();
  pdl_wait();
  const uint64_t sums = static_cast<uint64_t>(R.n_runs) * R.col_blocks, all = gridDim.x;
  const uint64_t task = blockIdx.x * sums / all;  // sums in the blocks before this one
  if ((blockIdx.x + 1) * sums / all == task) {
    const int64_t zero = static_cast<int64_t>(blockIdx.x - task);
    zero_rows<GB, VEC == 8>(E, (zero * (blockDim.x >> 5) + (threadIdx.x >> 5)) * R.zero_rows, R.zero_rows, threadIdx.x & 31);
    return;
  }
  const int64_t run = static_cast<int64_t>(task) / R.col_blocks;
  const int col_block = static_cast<int>(static_cast<int64_t>(task) - run * R.col_blocks);
  const int64_t p0 = run * R.run;
  const uint32_t none = 0xffffffffu, dropped = static_cast<uint32_t>(E.ids.vocab);
  for (int k = threadIdx.x; k < R.run + 2; k += blockDim.x) {
    const int64_t p = p0 + k - 1;
    keys[k] = p >= 0 && p < E.n ? load_l2(R.key + p) : none;
    if (k >= 1 && k <= R.run && p < E.n) pos[k - 1] = load_l2(R.pos + p);
  }
  __syncthreads();
  const int c = (col_block * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x)) * VEC;
  if (c >= E.dim) return;
  float acc[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) acc[j] = 0.f;
  for (int k0 = 0; k0 < R.run; k0 += 4) {
    float v[4][VEC];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t id = keys[k0 + u + 1];
      if (id >= dropped) continue;  // padding, or past the list
      const void* src = at<DB>(E.dout, static_cast<int64_t>(pos[k0 + u]) * E.ld_dout + c);
      if (VEC == 8)
        load8<DB>(src, reinterpret_cast<float(&)[8]>(v[u]));
      else
        v[u][0] = load1<DB>(src);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = k0 + u;
      const uint32_t id = keys[k + 1];
      if (id >= dropped) return;
#pragma unroll
      for (int j = 0; j < VEC; ++j) acc[j] += v[u][j];
      const bool ends = keys[k + 2] != id;
      if (!ends && k + 1 < R.run) continue;
      const bool from_before = keys[0] == id;  // the list is sorted
      if (ends && !from_before) {
        put_row<GB, VEC>(E, id, c, acc);
      } else {
        float* part = E.partial + (2 * run + (from_before ? 0 : 1)) * R.ld_part + c;
#pragma unroll
        for (int j = 0; j < VEC; ++j) part[j] = acc[j];
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) acc[j] = 0.f;
    }
  }
}

// Joins an id that crosses cuts: run's tail, then the heads of the runs after it.
// An id that came often has dozens of heads, and a thread that added them alone was
// a chain of latencies: up to kJoinLanes threads take the columns and the block's
// others a share of the heads each (every S-th), joined in the shares' order.  5001
// entries on eight ids of width 1000 take 6.0 us instead of 8.1; 32768 Zipf ids of
// width 4096 12.9 instead of 15.4, and 24 with 64 lanes.
constexpr int kJoinThreads = 512, kJoinLanes = 128;

template <bool GB, int VEC>
__global__ void __launch_bounds__(kJoinThreads) embed_join_kernel(const EmbedBackward E, const Runs R) {
  __shared__ float sums[kJoinThreads * VEC];
  pdl_wait();
  pdl_launch();  // not before: blocks that wait here would hold the room of the next call's sort (21 us a call for 26 there)
  const int64_t run = blockIdx.x / R.join_blocks;
  const int64_t p0 = run * R.run, next = p0 + R.run;
  if (next >= E.n) return;
  const uint32_t none = 0xffffffffu;
  auto key_of_run = [&](int64_t k) { return next + k * R.run < E.n ? R.key[next + k * R.run] : none; };
  const uint32_t mine = key_of_run(threadIdx.x);
  const uint32_t id = R.key[next], last = R.key[next - 1], head_key = R.key[p0], before = p0 > 0 ? R.key[p0 - 1] : none;
  if (id >= static_cast<uint32_t>(E.ids.vocab) || last != id) return;
  if (head_key == id && before == id) return;  // began in an earlier run
  const int threads = static_cast<int>(blockDim.x);
  int more = __syncthreads_count(mine == id);
  int64_t heads = more;
  while (more == threads) {
    more = __syncthreads_count(key_of_run(heads + threadIdx.x) == id);
    heads += more;
  }
  const int lane = static_cast<int>(threadIdx.x) % R.join_lanes, share = static_cast<int>(threadIdx.x) / R.join_lanes;
  const int shares = threads / R.join_lanes;
  const int c = (static_cast<int>(blockIdx.x - run * R.join_blocks) * R.join_lanes + lane) * VEC;
  const bool live = c < E.dim;
  float acc[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) acc[j] = 0.f;
  if (live) {
    if (share == 0) {
      const float* tail = E.partial + (2 * run + 1) * R.ld_part + c;
#pragma unroll
      for (int j = 0; j < VEC; ++j) acc[j] = tail[j];
    }
    const float* head = E.partial + 2 * (run + 1) * R.ld_part + c;
#pragma unroll 8
    for (int64_t h = share; h < heads; h += shares) {
      if (VEC == 8) {
        const float4 a = *reinterpret_cast<const float4*>(head + 2 * h * R.ld_part);
        const float4 b = *reinterpret_cast<const float4*>(head + 2 * h * R.ld_part + 4);
        acc[0] += a.x; acc[1 % VEC] += a.y; acc[2 % VEC] += a.z; acc[3 % VEC] += a.w;
        acc[4 % VEC] += b.x; acc[5 % VEC] += b.y; acc[6 % VEC] += b.z; acc[7 % VEC] += b.w;
      } else {
        acc[0] += head[2 * h * R.ld_part];
      }
    }
  }
#pragma unroll
  for (int j = 0; j < VEC; ++j) sums[j * kJoinThreads + threadIdx.x] = acc[j];
  __syncthreads();
  if (share > 0 || !live) return;
  for (int k = 1; k < shares; ++k) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) acc[j] += sums[j * kJoinThreads + k * R.join_lanes + lane];
  }
  put_row<GB, VEC>(E, id, c, acc);
}

// ----------------------------------------------------------------- few entries
// Up to kFew entries, all in one launch: every block sorts the list by itself
// (each thread counts the pairs before its own), block i then sums the i-th
// distinct id, and the blocks after those write zeros.  17 entries added at
// width 4096 take 7 us of host and device each, where three launches took 13.
constexpr int kFew = 128;

template <bool DB, bool GB, int VEC>
__global__ void __launch_bounds__(256) embed_few_kernel(const EmbedBackward E, int col_blocks, int zero_rows) {
  __shared__ uint32_t raw[kFew], keys[kFew + 1], pos[kFew];
  __shared__ uint32_t starts[kFew / 32];
  const int n = static_cast<int>(E.n), t = threadIdx.x, lane = t & 31;
  const uint32_t dropped = static_cast<uint32_t>(E.ids.vocab);
  pdl_launch();
  pdl_wait();
  for (int i = t; i < n; i += blockDim.x) {
    bool bad = false;
    const int id = load_id(E.ids, i, &bad);
    if (bad && blockIdx.x == 0) atomicCAS(E.err, 0, kErrBadIndex);
    raw[i] = id < 0 ? dropped : static_cast<uint32_t>(id);
  }
  if (t == 0) keys[n] = dropped;
  __syncthreads();
  for (int i = t; i < n; i += blockDim.x) {
    const uint32_t key = raw[i];
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) rank += raw[j] < key || (raw[j] == key && j < i) ? 1 : 0;
    keys[rank] = key;
    pos[rank] = static_cast<uint32_t>(i);
  }
  __syncthreads();
  const int sums = n * col_blocks;
  if (static_cast<int>(blockIdx.x) >= sums) {
    // Zeros: a warp takes its rows and looks them up.
    const int64_t r0 = (static_cast<int64_t>(blockIdx.x - sums) * (blockDim.x >> 5) + (t >> 5)) * zero_rows;
    if (r0 >= E.ids.vocab) return;
    const int rows = static_cast<int>(min(static_cast<int64_t>(zero_rows), E.ids.vocab - r0));
    bool named = false;
    for (int j = lane; j < n; j += 32) named = named || (keys[j] >= r0 && keys[j] < r0 + rows);
    uint32_t left = 0xffffffffu >> (32 - rows);
    if (__any_sync(0xffffffffu, named)) {
      for (int j = 0; j < n; ++j)
        if (keys[j] >= r0 && keys[j] < r0 + rows) left &= ~(1u << (keys[j] - r0));
    }
    zero_marked<GB, VEC == 8>(E, r0, left, lane);
    return;
  }
  // The distinct ids' first places, found a warp (32 places) at a time.
  for (int i0 = t - lane; i0 < kFew; i0 += blockDim.x) {
    const int i = i0 + lane;
    const bool start = i < n && keys[i] < dropped && (i == 0 || keys[i - 1] != keys[i]);
    const uint32_t m = __ballot_sync(0xffffffffu, start);
    if (lane == 0) starts[i0 >> 5] = m;
  }
  __syncthreads();
  const int want = static_cast<int>(blockIdx.x) / col_blocks;
  int seen = 0, from = -1;
#pragma unroll
  for (int w = 0; w < kFew / 32; ++w) {
    const int here = __popc(starts[w]);
    if (from < 0 && want < seen + here) from = 32 * w + static_cast<int>(__fns(starts[w], 0, want - seen + 1));
    seen += here;
  }
  if (from < 0) return;
  const int c = ((static_cast<int>(blockIdx.x) - want * col_blocks) * static_cast<int>(blockDim.x) + t) * VEC;
  if (c >= E.dim) return;
  const uint32_t id = keys[from];
  int to = from + 1;
  while (keys[to] == id) ++to;
  float acc[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) acc[j] = 0.f;
  for (int k0 = from; k0 < to; k0 += 8) {
    float v[8][VEC];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (k0 + u >= to) continue;
      const void* src = at<DB>(E.dout, static_cast<int64_t>(pos[k0 + u]) * E.ld_dout + c);
      if (VEC == 8)
        load8<DB>(src, reinterpret_cast<float(&)[8]>(v[u]));
      else
        v[u][0] = load1<DB>(src);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (k0 + u >= to) continue;
#pragma unroll
      for (int j = 0; j < VEC; ++j) acc[j] += v[u][j];
    }
  }
  put_row<GB, VEC>(E, id, c, acc);
}

inline bool aligned16_rows(const void* p, int64_t ld, int bf16, int dim) {
  return dim % 8 == 0 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld * (bf16 ? 2 : 4) % 16 == 0;
}

// Positions of a run: short lists in short runs, so that about two blocks per SM
// share the memory latency; 64 at most, which bounds the partials at a 32nd of
// the rows read.
int run_length(int64_t n, int col_blocks) {
  int run = 4;
  while (run < kEmbedRun && n * col_blocks > static_cast<int64_t>(304) * 2 * run) run *= 2;
  return run;
}

int sum_threads(int64_t width) { return static_cast<int>(width >= 256 ? 256 : (width + 31) / 32 * 32); }

template <bool DB, bool GB>
cudaError_t launch_sums(const EmbedBackward& E, Runs R, int* launches, cudaStream_t st) {
  const bool vec = aligned16_rows(E.dout, E.ld_dout, DB, E.dim) && aligned16_rows(E.dtable, E.ld_dtable, GB, E.dim);
  const int width = vec ? E.dim / 8 : E.dim;
  const int threads = sum_threads(width);
  R.col_blocks = (width + threads - 1) / threads;
  R.run = run_length(E.n, R.col_blocks);
  R.n_runs = (E.n + R.run - 1) / R.run;
  const int64_t sums = R.n_runs * R.col_blocks;
  R.join_lanes = std::min(kJoinLanes, (width + 31) / 32 * 32);
  R.join_blocks = (width + R.join_lanes - 1) / R.join_lanes;
  R.zero_rows = zero_rows_of(static_cast<int64_t>(E.dim) * (GB ? 2 : 4), 4);
  const int64_t rows_per_block = threads / 32 * R.zero_rows;
  const int64_t zeros = E.present ? (E.ids.vocab + rows_per_block - 1) / rows_per_block : 0;
  cudaError_t e = launch_after(vec ? embed_sum_kernel<DB, GB, 8> : embed_sum_kernel<DB, GB, 1>,
                               dim3(static_cast<unsigned>(sums + zeros)), dim3(threads), 0, st, E, R);
  ++*launches;
  if (e == cudaSuccess && R.n_runs > 1) {
    e = launch_after(vec ? embed_join_kernel<GB, 8> : embed_join_kernel<GB, 1>, dim3(static_cast<unsigned>(R.n_runs * R.join_blocks)),
                     dim3(static_cast<unsigned>(kJoinThreads / R.join_lanes * R.join_lanes)), 0, st, E, R);
    ++*launches;
  }
  return e;
}

template <bool DB, bool GB>
cudaError_t launch_few(const EmbedBackward& E, int* launches, cudaStream_t st) {
  const bool vec = aligned16_rows(E.dout, E.ld_dout, DB, E.dim) && aligned16_rows(E.dtable, E.ld_dtable, GB, E.dim);
  const int width = vec ? E.dim / 8 : E.dim;
  const int threads = sum_threads(width), col_blocks = (width + threads - 1) / threads;
  const int zero_rows = zero_rows_of(static_cast<int64_t>(E.dim) * (GB ? 2 : 4), 8);
  const int64_t rows_per_block = threads / 32 * zero_rows;
  const int64_t zeros = E.accumulate ? 0 : (E.ids.vocab + rows_per_block - 1) / rows_per_block;
  ++*launches;
  return launch_after(vec ? embed_few_kernel<DB, GB, 8> : embed_few_kernel<DB, GB, 1>,
                      dim3(static_cast<unsigned>(E.n * col_blocks + zeros)), dim3(threads), 0, st, E, col_blocks, zero_rows);
}

// One launch of a cluster of `ctas` blocks.
cudaError_t launch_cluster_sort(void (*kernel)(EmbedBackward, int, int), int ctas, cudaStream_t st, const EmbedBackward& E,
                                int passes, int bits) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kSortThreads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, E, passes, bits);
}

template <bool TB, bool OB>
cudaError_t launch_forward(const EmbedForward& E, cudaStream_t st) {
  const bool vec = aligned16_rows(E.table, E.ld_table, TB, E.dim) && aligned16_rows(E.out, E.ld_out, OB, E.dim);
  const int64_t tasks = E.n * ((E.dim + kFwdCols - 1) / kFwdCols);
  const int64_t blocks = (tasks + 7) / 8;
  const unsigned grid = static_cast<unsigned>(blocks < 152 * 64 ? blocks : 152 * 64);
  return launch_after(vec ? embed_forward_kernel<TB, OB, true> : embed_forward_kernel<TB, OB, false>, dim3(grid), dim3(256), 0,
                      st, E);
}

}  // namespace

cudaError_t launch_embed_forward(const EmbedForward& E, cudaStream_t st) {
  if (E.table_bf16) return E.out_bf16 ? launch_forward<true, true>(E, st) : launch_forward<true, false>(E, st);
  return E.out_bf16 ? launch_forward<false, true>(E, st) : launch_forward<false, false>(E, st);
}

EmbedWs embed_backward_ws(int64_t n, int64_t vocab, int32_t dim) {
  EmbedWs W{};
  if (n <= kFew) return W;  // none
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) / 256 * 256;
    return at;
  };
  const int64_t blocks = n <= kOneLaunch ? 0 : (n + kSortTile - 1) / kSortTile;
  // Runs as launch_sums cuts them, for whichever vector width it takes.
  int64_t runs = 0;
  for (const int64_t width : {static_cast<int64_t>(dim), static_cast<int64_t>(dim) / 8}) {
    if (width < 1) continue;
    const int threads = sum_threads(width);
    const int run = run_length(n, static_cast<int>((width + threads - 1) / threads));
    if ((n + run - 1) / run > runs) runs = (n + run - 1) / run;
  }
  for (int k = 0; k < 2; ++k) {
    W.key[k] = take(static_cast<size_t>(n) * 4);
    W.pos[k] = take(static_cast<size_t>(n) * 4);
  }
  W.hist = take(static_cast<size_t>(kBins) * static_cast<size_t>(blocks + 1) * 4);
  W.present = take(static_cast<size_t>((vocab + 31) / 32) * 4);
  W.partial = take(static_cast<size_t>(runs) * 2 * static_cast<size_t>((dim + 7) / 8 * 8) * 4);
  W.bytes = off;
  return W;
}

cudaError_t launch_embed_backward(const EmbedBackward& E, int* launches, cudaStream_t st) {
  *launches = 0;
  if (E.n <= kFew) {
    if (E.dout_bf16) return E.dtable_bf16 ? launch_few<true, true>(E, launches, st) : launch_few<true, false>(E, launches, st);
    return E.dtable_bf16 ? launch_few<false, true>(E, launches, st) : launch_few<false, false>(E, launches, st);
  }
  int key_bits = 1;
  while ((int64_t(1) << key_bits) <= E.ids.vocab) ++key_bits;  // keys 0 .. vocab
  const int passes = (key_bits + kDigitBits - 1) / kDigitBits, bits = (key_bits + passes - 1) / passes;
  int sorted = (passes - 1) & 1;
  cudaError_t e = cudaSuccess;
  if (E.n <= (E.present ? kCounted / 2 : kCounted)) {
    e = launch_after(embed_count_kernel, dim3(static_cast<unsigned>((E.n + kCountEntries - 1) / kCountEntries)), dim3(kCountThreads), 0, st, E);
    sorted = 0;
    ++*launches;
  } else if (E.n <= kOneLaunch) {
    // One entry a thread while the cluster has room for more blocks.
    int ctas = 1, items = 1;
    while (ctas < kClusterMost && ctas * kSortThreads < E.n) ctas *= 2;
    while (ctas * kSortThreads * items < E.n) items *= 2;
    e = launch_cluster_sort(items == 1   ? embed_sort_cluster_kernel<1>
                            : items == 2 ? embed_sort_cluster_kernel<2>
                            : items == 4 ? embed_sort_cluster_kernel<4>
                                         : embed_sort_cluster_kernel<8>,
                            ctas, st, E, passes, bits);
    ++*launches;
  } else {
    const dim3 blocks(static_cast<unsigned>((E.n + kSortTile - 1) / kSortTile)), threads(kSortThreads);
    int from = 1;
    for (int p = 0; p < passes && e == cudaSuccess; ++p) {
      e = launch_after(embed_hist_kernel, blocks, threads, 0, st, E, p, bits, from);
      if (e == cudaSuccess) e = launch_after(embed_scan_kernel, dim3(kBins), threads, 0, st, E.hist, static_cast<int>(blocks.x));
      if (e == cudaSuccess) e = launch_after(embed_scatter_kernel, blocks, threads, 0, st, E, p, bits, from);
      from ^= 1;
      *launches += 3;
    }
    sorted = from;
    if (E.present && e == cudaSuccess) {
      e = launch_after(embed_mark_kernel, dim3(static_cast<unsigned>((E.n + kSortThreads - 1) / kSortThreads)), threads, 0, st, E, from);
      ++*launches;
    }
  }
  if (e != cudaSuccess) return e;
  Runs R = {};
  R.key = E.key[sorted];
  R.pos = E.pos[sorted];
  R.ld_part = (E.dim + 7) / 8 * 8;
  if (E.dout_bf16)
    return E.dtable_bf16 ? launch_sums<true, true>(E, R, launches, st) : launch_sums<true, false>(E, R, launches, st);
  return E.dtable_bf16 ? launch_sums<false, true>(E, R, launches, st) : launch_sums<false, false>(E, R, launches, st);
}

}  // namespace dmuon
