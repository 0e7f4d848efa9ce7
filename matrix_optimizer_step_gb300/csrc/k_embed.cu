// Embedding lookup and its gradient.
//
//   forward   out[i] = scale * table[id_i]           (id_i < 0: zeros)
//   backward  dtable[v] = scale * sum_{i: id_i = v} dout[i]   [+ dtable[v]]
//
// Both move bytes and compute next to nothing.  The gradient adds the rows of
// equal ids in the order of their positions, in fp32, and rounds once, so that
// it is the same for every run: the (id, position) pairs are sorted with a
// stable radix sort, the sorted list is cut into runs of kEmbedRun positions,
// one block sums each run, and ids that cross a cut are joined from the runs'
// partial sums in order.  Work is even over blocks however often an id comes.
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "ptx.cuh"
#include "vocab.h"

namespace dmuon {
namespace {

// ---------------------------------------------------------- rows of 8 values
template <bool BF16>
__device__ __forceinline__ void load8(const void* p, float (&v)[8]) {
  if (BF16) {
    const uint4 q = __ldg(static_cast<const uint4*>(p));
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    const float4 a = __ldg(static_cast<const float4*>(p)), b = __ldg(static_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}

// The same for memory that the kernel also writes.
template <bool BF16>
__device__ __forceinline__ void load8_rw(const void* p, float (&v)[8]) {
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
// 9 bits a pass.  A block takes 4096 pairs; warp w holds 128 consecutive ones
// (four rounds of one per lane).  Entries that are not counted get the key
// `vocab`, which sorts last.
constexpr int kSortThreads = 1024, kSortItems = 4, kSortTile = kSortThreads * kSortItems;
constexpr int kBins = 512;

__device__ __forceinline__ uint32_t first_key(const EmbedBackward& E, int64_t i) {
  bool bad = false;
  const int id = load_id(E.ids, i, &bad);
  if (bad) atomicCAS(E.err, 0, kErrBadIndex);
  return id < 0 ? static_cast<uint32_t>(E.ids.vocab) : static_cast<uint32_t>(id);
}

// Ranks of this block's pairs among its pairs of the same digit: rank[k] within the
// warp, and cnt[w][d] the number in the warps before w.  Called by all threads;
// total (thread d): the block's number of digit d.
__device__ __forceinline__ uint32_t block_ranks(const uint32_t (&digit)[kSortItems], const bool (&has)[kSortItems],
                                                uint16_t (*cnt)[kBins], uint32_t (&rank)[kSortItems]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int d = lane; d < kBins; d += 32) cnt[warp][d] = 0;
  __syncwarp();
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) {
    const uint32_t key = has[k] ? digit[k] : kBins + 1;
    const uint32_t mask = __match_any_sync(0xffffffffu, key);
    const uint32_t before = has[k] ? cnt[warp][digit[k]] : 0u;
    rank[k] = before + __popc(mask & ((1u << lane) - 1u));
    __syncwarp();
    if (has[k] && lane == __ffs(mask) - 1) cnt[warp][digit[k]] = static_cast<uint16_t>(before + __popc(mask));
    __syncwarp();
  }
  __syncthreads();
  uint32_t total = 0;
  if (threadIdx.x < kBins)
    for (int w = 0; w < kSortThreads / 32; ++w) {
      const uint32_t c = cnt[w][threadIdx.x];
      cnt[w][threadIdx.x] = static_cast<uint16_t>(total);
      total += c;
    }
  __syncthreads();
  return total;
}

// Exclusive scan of the first kBins threads' values (others pass 0).
__device__ __forceinline__ uint32_t scan_bins(uint32_t v, uint32_t* tmp) {
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

struct SmallSort {
  uint16_t cnt[kSortThreads / 32][kBins];
  uint32_t key[kSortTile], pos[kSortTile];
  uint32_t base[kBins];
  uint32_t tmp[32];
};

// Up to kSortTile entries: the whole sort in one block.
__global__ void __launch_bounds__(kSortThreads) embed_sort_small_kernel(const EmbedBackward E, int passes, int bits) {
  extern __shared__ uint8_t smem_raw[];
  SmallSort& S = *reinterpret_cast<SmallSort*>(smem_raw);
  const int n = static_cast<int>(E.n);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t key[kSortItems], pos[kSortItems], digit[kSortItems], rank[kSortItems];
  bool has[kSortItems];
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) {
    const int i = warp * 32 * kSortItems + 32 * k + lane;
    has[k] = i < n;
    pos[k] = static_cast<uint32_t>(i);
    key[k] = has[k] ? first_key(E, i) : 0u;
  }
  for (int p = 0; p < passes; ++p) {
#pragma unroll
    for (int k = 0; k < kSortItems; ++k) digit[k] = (key[k] >> (p * bits)) & ((1u << bits) - 1u);
    const uint32_t total = block_ranks(digit, has, S.cnt, rank);
    const uint32_t b = scan_bins(threadIdx.x < kBins ? total : 0u, S.tmp);
    if (threadIdx.x < kBins) S.base[threadIdx.x] = b;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kSortItems; ++k)
      if (has[k]) {
        const uint32_t to = S.base[digit[k]] + S.cnt[warp][digit[k]] + rank[k];
        S.key[to] = key[k];
        S.pos[to] = pos[k];
      }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kSortItems; ++k) {
      const int i = warp * 32 * kSortItems + 32 * k + lane;
      if (has[k]) {
        key[k] = S.key[i];
        pos[k] = S.pos[i];
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) {
    const int i = warp * 32 * kSortItems + 32 * k + lane;
    if (has[k]) {
      E.key[0][i] = key[k];
      E.pos[0][i] = pos[k];
    }
  }
}

// Longer lists: per pass a histogram of each block, a scan over the blocks of
// each digit, and the scatter.  hist[digit][block]; hist[kBins * blocks + digit]: totals.
__global__ void __launch_bounds__(kSortThreads) embed_hist_kernel(const EmbedBackward E, int pass, int bits, int from) {
  __shared__ uint32_t h[kBins];
  for (int d = threadIdx.x; d < kBins; d += kSortThreads) h[d] = 0;
  __syncthreads();
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
  uint32_t* h = hist + static_cast<int64_t>(blockIdx.x) * blocks;
  uint32_t base = 0;
  for (int b0 = 0; b0 < blocks; b0 += kSortThreads) {
    const int b = b0 + threadIdx.x;
    const uint32_t v = b < blocks ? h[b] : 0u;
    const uint32_t s = scan_bins(v, tmp);
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
  const uint32_t b = scan_bins(total, S.tmp);
  if (threadIdx.x < kBins) S.base[threadIdx.x] = b + E.hist[static_cast<int64_t>(threadIdx.x) * gridDim.x + blockIdx.x];
  block_ranks(digit, has, S.cnt, rank);
#pragma unroll
  for (int k = 0; k < kSortItems; ++k)
    if (has[k]) {
      const uint32_t to = S.base[digit[k]] + S.cnt[warp][digit[k]] + rank[k];
      E.key[from ^ 1][to] = key[k];
      E.pos[from ^ 1][to] = pos[k];
    }
}

// ----------------------------------------------------------------------- sums
struct Runs {
  const uint32_t* key;
  const uint32_t* pos;
  int64_t n_runs;
  int64_t ld_part;
};

// VEC columns a thread; blockIdx.x is the run, blockIdx.y the column block.
template <bool DB, bool GB, int VEC>
__device__ __forceinline__ void put_row(const EmbedBackward& E, uint32_t id, int c, const float (&acc)[VEC]) {
  void* dst = at<GB>(E.dtable, static_cast<int64_t>(id) * E.ld_dtable + c);
  if (VEC == 8) {
    float v[8];
    if (E.accumulate) {
      load8_rw<GB>(dst, v);
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

template <bool DB, bool GB, int VEC>
__global__ void __launch_bounds__(256) embed_sum_kernel(const EmbedBackward E, const Runs R) {
  __shared__ uint32_t keys[kEmbedRun + 2], pos[kEmbedRun];
  const int64_t run = blockIdx.x;
  const int64_t p0 = run * kEmbedRun;
  const uint32_t none = 0xffffffffu, dropped = static_cast<uint32_t>(E.ids.vocab);
  for (int k = threadIdx.x; k < kEmbedRun + 2; k += blockDim.x) {
    const int64_t p = p0 + k - 1;
    keys[k] = p >= 0 && p < E.n ? R.key[p] : none;
    if (k >= 1 && k <= kEmbedRun && p < E.n) pos[k - 1] = R.pos[p];
  }
  __syncthreads();
  const int c = (blockIdx.y * blockDim.x + threadIdx.x) * VEC;
  if (c >= E.dim) return;
  float acc[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) acc[j] = 0.f;
  int seg0 = 0;
  for (int k0 = 0; k0 < kEmbedRun; k0 += 4) {
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
      if (!ends && k + 1 < kEmbedRun) continue;
      const bool from_before = seg0 == 0 && keys[0] == id;
      if (ends && !from_before) {
        put_row<DB, GB, VEC>(E, id, c, acc);
      } else {
        float* part = E.partial + (2 * run + (from_before ? 0 : 1)) * R.ld_part + c;
#pragma unroll
        for (int j = 0; j < VEC; ++j) part[j] = acc[j];
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) acc[j] = 0.f;
      seg0 = k + 1;
    }
  }
}

// Joins an id that crosses cuts: run's tail, then the heads of the runs after it.
template <bool DB, bool GB, int VEC>
__global__ void __launch_bounds__(256) embed_join_kernel(const EmbedBackward E, const Runs R) {
  const int64_t run = blockIdx.x;
  const int64_t next = (run + 1) * kEmbedRun;
  if (next >= E.n) return;
  const uint32_t id = R.key[next];
  if (id >= static_cast<uint32_t>(E.ids.vocab) || R.key[next - 1] != id) return;
  const int64_t p0 = run * kEmbedRun;
  if (R.key[p0] == id && p0 > 0 && R.key[p0 - 1] == id) return;  // began in an earlier run
  int64_t heads = 0;
  for (;;) {
    const int64_t p = next + (heads + threadIdx.x) * kEmbedRun;
    const int more = __syncthreads_count(p < E.n && R.key[p] == id);
    heads += more;
    if (more < static_cast<int>(blockDim.x)) break;
  }
  const int c = (blockIdx.y * blockDim.x + threadIdx.x) * VEC;
  if (c >= E.dim) return;
  float acc[VEC];
  const float* tail = E.partial + (2 * run + 1) * R.ld_part + c;
#pragma unroll
  for (int j = 0; j < VEC; ++j) acc[j] = tail[j];
  const float* head = E.partial + 2 * (run + 1) * R.ld_part + c;
#pragma unroll 4
  for (int64_t h = 0; h < heads; ++h)
#pragma unroll
    for (int j = 0; j < VEC; ++j) acc[j] += head[2 * h * R.ld_part + j];
  put_row<DB, GB, VEC>(E, id, c, acc);
}

// Rows that no entry names become zeros.  A warp takes 32 rows: each lane looks
// its row up in the sorted list, then the warp writes the absent ones.
template <bool GB, bool VEC>
__global__ void __launch_bounds__(256) embed_zero_kernel(const EmbedBackward E, const Runs R) {
  const int lane = threadIdx.x & 31;
  const int64_t r0 = (static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5)) * 32;
  if (r0 >= E.ids.vocab) return;
  const int64_t row = r0 + lane;
  int64_t lo = 0, hi = E.n;
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (static_cast<int64_t>(R.key[mid]) < row)
      lo = mid + 1;
    else
      hi = mid;
  }
  const bool absent = row < E.ids.vocab && !(lo < E.n && static_cast<int64_t>(R.key[lo]) == row);
  uint32_t left = __ballot_sync(0xffffffffu, absent);
  while (left) {
    const int k = __ffs(left) - 1;
    left &= left - 1;
    void* dst = at<GB>(E.dtable, (r0 + k) * E.ld_dtable);
    if (VEC) {
      const int n16 = E.dim / (GB ? 8 : 4);
      for (int c = lane; c < n16; c += 32) static_cast<uint4*>(dst)[c] = make_uint4(0, 0, 0, 0);
    } else {
      for (int c = lane; c < E.dim; c += 32) store1<GB>(at<GB>(dst, c), 0.f);
    }
  }
}

inline bool aligned16_rows(const void* p, int64_t ld, int bf16, int dim) {
  return dim % 8 == 0 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld * (bf16 ? 2 : 4) % 16 == 0;
}

template <bool DB, bool GB>
cudaError_t launch_sums(const EmbedBackward& E, const Runs& R, int* launches, cudaStream_t st) {
  const bool vec = aligned16_rows(E.dout, E.ld_dout, DB, E.dim) && aligned16_rows(E.dtable, E.ld_dtable, GB, E.dim);
  const int width = (E.dim + (vec ? 7 : 0)) / (vec ? 8 : 1);
  const int threads = width >= 256 ? 256 : (width + 31) / 32 * 32;
  const dim3 grid(static_cast<unsigned>(R.n_runs), static_cast<unsigned>((width + threads - 1) / threads));
  if (!E.accumulate) {
    const unsigned blocks = static_cast<unsigned>((E.ids.vocab + 255) / 256);
    if (vec)
      embed_zero_kernel<GB, true><<<blocks, 256, 0, st>>>(E, R);
    else
      embed_zero_kernel<GB, false><<<blocks, 256, 0, st>>>(E, R);
    ++*launches;
  }
  if (vec)
    embed_sum_kernel<DB, GB, 8><<<grid, threads, 0, st>>>(E, R);
  else
    embed_sum_kernel<DB, GB, 1><<<grid, threads, 0, st>>>(E, R);
  ++*launches;
  if (R.n_runs > 1) {
    if (vec)
      embed_join_kernel<DB, GB, 8><<<grid, threads, 0, st>>>(E, R);
    else
      embed_join_kernel<DB, GB, 1><<<grid, threads, 0, st>>>(E, R);
    ++*launches;
  }
  return cudaGetLastError();
}

template <bool TB, bool OB>
cudaError_t launch_forward(const EmbedForward& E, cudaStream_t st) {
  const bool vec = aligned16_rows(E.table, E.ld_table, TB, E.dim) && aligned16_rows(E.out, E.ld_out, OB, E.dim);
  const int64_t tasks = E.n * ((E.dim + kFwdCols - 1) / kFwdCols);
  const int64_t blocks = (tasks + 7) / 8;
  const unsigned grid = static_cast<unsigned>(blocks < 152 * 64 ? blocks : 152 * 64);
  if (vec)
    embed_forward_kernel<TB, OB, true><<<grid, 256, 0, st>>>(E);
  else
    embed_forward_kernel<TB, OB, false><<<grid, 256, 0, st>>>(E);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_embed_forward(const EmbedForward& E, cudaStream_t st) {
  if (E.table_bf16) return E.out_bf16 ? launch_forward<true, true>(E, st) : launch_forward<true, false>(E, st);
  return E.out_bf16 ? launch_forward<false, true>(E, st) : launch_forward<false, false>(E, st);
}

EmbedWs embed_backward_ws(int64_t n, int32_t dim) {
  EmbedWs W{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) / 256 * 256;
    return at;
  };
  const int64_t blocks = (n + kSortTile - 1) / kSortTile, runs = (n + kEmbedRun - 1) / kEmbedRun;
  for (int k = 0; k < 2; ++k) {
    W.key[k] = take(static_cast<size_t>(n) * 4);
    W.pos[k] = take(static_cast<size_t>(n) * 4);
  }
  W.hist = take(static_cast<size_t>(kBins) * static_cast<size_t>(blocks + 1) * 4);
  W.partial = take(static_cast<size_t>(runs) * 2 * static_cast<size_t>((dim + 7) / 8 * 8) * 4);
  W.bytes = off;
  return W;
}

cudaError_t launch_embed_backward(const EmbedBackward& E, int* launches, cudaStream_t st) {
  *launches = 0;
  int key_bits = 1;
  while ((int64_t(1) << key_bits) <= E.ids.vocab) ++key_bits;  // keys 0 .. vocab
  const int passes = (key_bits + 8) / 9, bits = (key_bits + passes - 1) / passes;
  int from = 0;
  if (E.n <= kSortTile) {
    static unsigned long long attr_mask = 0;
    if (attr_needed_on_current_device(&attr_mask)) {
      cudaError_t e = cudaFuncSetAttribute(embed_sort_small_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           static_cast<int>(sizeof(SmallSort)));
      if (e != cudaSuccess) return e;
      attr_note_current_device(&attr_mask);
    }
    embed_sort_small_kernel<<<1, kSortThreads, sizeof(SmallSort), st>>>(E, passes, bits);
    ++*launches;
  } else {
    const int blocks = static_cast<int>((E.n + kSortTile - 1) / kSortTile);
    for (int p = 0; p < passes; ++p) {
      embed_hist_kernel<<<blocks, kSortThreads, 0, st>>>(E, p, bits, from);
      embed_scan_kernel<<<kBins, kSortThreads, 0, st>>>(E.hist, blocks);
      embed_scatter_kernel<<<blocks, kSortThreads, 0, st>>>(E, p, bits, from);
      from ^= 1;
      *launches += 3;
    }
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  Runs R;
  R.key = E.key[from];
  R.pos = E.pos[from];
  R.n_runs = (E.n + kEmbedRun - 1) / kEmbedRun;
  R.ld_part = (E.dim + 7) / 8 * 8;
  if (E.dout_bf16)
    return E.dtable_bf16 ? launch_sums<true, true>(E, R, launches, st) : launch_sums<true, false>(E, R, launches, st);
  return E.dtable_bf16 ? launch_sums<false, true>(E, R, launches, st) : launch_sums<false, false>(E, R, launches, st);
}

}  // namespace dmuon
