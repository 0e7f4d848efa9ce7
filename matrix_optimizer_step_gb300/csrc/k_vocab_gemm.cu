// The three products of the cross entropy over a head matrix, on CTA pairs
// (tcgen05, cta_group::2):
//   logits   Z  = X W^T     (tokens x vocabulary, K = width)
//   dX       dX = dZ W      (tokens x width,      K = vocabulary)
//   dW       dW = dZ^T X    (vocabulary x width,  K = tokens)
// bf16 operands, fp32 accumulation in TMEM.  Each output tile is 256 x 256
// and belongs to a cluster of two CTAs: CTA r loads rows [128r, 128r + 128)
// of the tile's A operand and of its B operand into a 5-stage ring, one
// thread of CTA 0 issues M = 256, N = 256, K = 16 MMAs that read both CTAs'
// shared memory, and each CTA's TMEM receives 128 rows of the accumulator.
// The accumulator is double-buffered (2 x 256 of the 512 TMEM columns), so
// the epilogue of a tile runs under the main loop of the next.
//
// The logits' epilogue never stores a logit.  Each thread owns one row and
// 128 columns: it takes their maximum m and the sum of 2^(z - m) over all but
// the target, with z = logit * log2(e), and writes that pair.  For the gradient it also leaves
// round((m - z) * 1024) as 16 bits: the exponential's argument in fixed point
// is within 2^-11 octaves, i.e. a relative error of at most 3.4e-4 in the
// probability, a quarter of the rounding to bf16 that d logits get anyway,
// where the logit itself rounded to 16 bits would be off by its size times
// 2^-9.  The logs turn into d logits once the row's sum is known
// (k_vocab_ce.cu), so the gradient needs no second logits product.
//
// Long tiles are handed out by a counter in global memory: the SMs do not run
// at one pace (with equal shares the first pair was done 5 % before the last),
// and the two gradient products' tiles differ in length.  One thread of CTA 0
// draws a number and puts it into a two-deep mailbox of both CTAs, and draws
// the next but one once every role of both has read it.  Which pair computes
// a tile does not change its result.  At 8192 x 128256 x 4096 that takes a
// gradient call from 17.1 to 16.6 ms.  A drawn number costs half a
// microsecond, so short tiles (vocab.cu says which) have fixed shares: drawn,
// 24 x 128256 x 4096 took 671 us for 620.
//
// Where a row's largest logits are wanted, four more warps of each CTA read its half of W's rows in shared memory beside
// the MMA, a row a lane, in the tiles of the first 256 tokens, and leave the largest norm of each 32: what
// bounds the rounding of a logit (k_logprobs.cu).  The producer of W waits for them in those tiles.  A call with
// alternatives takes 630 us for 616 without the norms at 1000 x 128256 x 4096, and 750 with a kernel of its own that reads W
// beside the product (795 behind it); with 64 tokens 232 for 223.
//
// Every wait is bounded; after a timeout the CTA records the error, stops
// issuing, and both CTAs meet at the final cluster barrier before the pair
// frees its TMEM.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "internal.h"
#include "ptx.cuh"
#include "vocab.h"
#include "vocab_rows.cuh"

namespace dmuon {
namespace {

constexpr int TILE = 256;
constexpr int BK = 64;
constexpr int STAGES = 5;  // with 4: 16.4 ms for 15.6 at 8192 x 128256 x 4096, 762 us for 719 at 4096 x 50257 x 768
constexpr int EPI = 8;  // epilogue warps: two per TMEM lane quarter, 128 columns each
constexpr int kSchedWarp = 3 + EPI;
constexpr int kThreads = (4 + EPI) * 32;
constexpr int kNormWarp = 4 + EPI, kNormWarps = 4;  // the first of the warps that take norms
constexpr uint32_t HALF_BYTES = 128 * BK * 2;
constexpr uint32_t STAGE_BYTES = 2 * HALF_BYTES;
constexpr uint32_t MN_BOX_BYTES = 64 * 64 * 2;
constexpr uint32_t kStaging = 2 * 4096;  // two boxes of 32 rows x 128 bytes per epilogue warp
constexpr int kMail = 2;  // tile numbers on their way to the roles
constexpr int kNumBars = 2 * STAGES + 2 + 2 + 1 + 2 * kMail + 2 * STAGES;
// Threads that read a tile number: both producers and the epilogue warps of two CTAs, and the MMA issuer.
constexpr uint32_t kReaders = 2 * (2 + EPI) + 1;
template <class Args>
constexpr bool kCanNorm = std::is_base_of<VocabLogProbs, Args>::value;
template <class Args>
__host__ __device__ inline float* norms_of(const Args& G) {
  if constexpr (kCanNorm<Args>)
    return G.norms;
  else
    return nullptr;
}
constexpr size_t kSmem = 1024 + STAGES * STAGE_BYTES + EPI * kStaging + kNumBars * 8 + 8 + 4 * kMail;
constexpr uint32_t kTmemCols = 512;
static_assert(kSmem <= 227 * 1024, "shared memory budget");
// Every CTA takes all of its SM's TMEM, so no second one may share the SM.
static_assert(kSmem > 114 * 1024, "one CTA per SM");

__device__ __forceinline__ uint64_t desc_k(uint32_t base, int kk) {
  return smem_desc_sw128(base + 32u * kk, 16u, 1024u);
}
__device__ __forceinline__ uint64_t desc_mn(uint32_t base, int kk) {
  return smem_desc_sw128(base + 2048u * kk, MN_BOX_BYTES, 1024u);
}

struct Tile {
  int product;           // index into VocabGrad::p; -1: no more
  int m0, n0, kb0, kb1, split;
};

// Tile number t >= 0 of a product.
__device__ __forceinline__ Tile place(const TileGrid& R, int t) {
  Tile T;
  T.product = 0;
  T.split = R.per_split.div(t);
  t -= T.split * static_cast<int>(R.per_split.d);
  const int g = R.per_group.div(t);
  t -= g * static_cast<int>(R.per_group.d);
  const bool full = (g + 1) * R.group_m <= R.tiles_m;
  const int n = full ? R.group.div(t) : R.last.div(t);
  T.m0 = (g * R.group_m + t - n * (full ? R.group_m : R.last_m)) * TILE;
  T.n0 = n * TILE;
  T.kb0 = T.split * R.kb_step;
  T.kb1 = min(R.kb_total, T.kb0 + R.kb_step);
  return T;
}

// Tile number t of the launch (-1: no more).
__device__ __forceinline__ Tile tile_at(const VocabLogits& G, int t) {
  Tile T;
  T.product = -1;
  return t < 0 ? T : place(G.grid, t);
}
__device__ __forceinline__ Tile tile_at(const VocabGrad& G, int t) {
  Tile T;
  T.product = -1;
  if (t < 0) return T;
  const int p = t >= G.n_units[0] ? 1 : 0;
  T = place(G.p[p].grid, p ? t - G.n_units[0] : t);
  T.product = p;
  return T;
}

__device__ __forceinline__ int tiles_in(const VocabLogits& G) { return G.grid.count(); }
__device__ __forceinline__ int tiles_in(const VocabGrad& G) { return G.n_units[0] + G.n_units[1]; }

// Shares fixed in advance: the numbers of one pair's tiles.  The first
// product's tiles go to the pairs in turn, then the second's; pairs with one
// of the first's fewer take `extra` of the second's before the others begin
// on those.
struct FixedShares {
  int pair, pairs, n0, n1, own0, mine, light, heavy, extras;
  __device__ __forceinline__ FixedShares(int n0_, int n1_, int extra) : n0(n0_), n1(n1_) {
    pair = blockIdx.x >> 1;
    pairs = gridDim.x >> 1;
    heavy = n0 % pairs;
    light = pairs - heavy;
    own0 = n0 / pairs + (pair < heavy ? 1 : 0);
    extras = min(light * extra, n1);
    mine = pair >= heavy && pair - heavy < extras ? (extras - (pair - heavy) + light - 1) / light : 0;
  }
  __device__ __forceinline__ int at(int i) const {
    if (i < own0) return pair + i * pairs;
    i -= own0;
    const int t = i < mine ? pair - heavy + i * light : extras + pair + (i - mine) * pairs;
    return t < n1 ? n0 + t : -1;
  }
};
__device__ __forceinline__ FixedShares fixed_shares(const VocabLogits& G) { return FixedShares(tiles_in(G), 0, 0); }
__device__ __forceinline__ FixedShares fixed_shares(const VocabGrad& G) {
  return FixedShares(G.n_units[0], G.n_units[1], G.extra);
}

__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Arrival on the other CTA's barrier that hands on no ordinary memory: the
// tensor-core fence before it orders the TMEM reads.  (With release semantics
// the arrival waits for all of the thread's earlier stores.)
__device__ __forceinline__ void arrive_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

__device__ __forceinline__ void st_shared_16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ void tma_add_3d(const CUtensorMap* map, uint32_t src, int c0, int c1, int c2) {
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// This thread's 128 accumulator columns.
__device__ __forceinline__ void load_columns(uint32_t t_lane, uint32_t (&r)[4][32]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) tmem_ld_32x32b_x32(t_lane + 32u * i, r[i]);
#pragma unroll
  for (int i = 0; i < 4; ++i) tmem_ld_wait_regs(r[i]);
}

// Box `buf` of the warp's staging (32 rows of 128 bytes, 128-byte swizzle):
// 16-byte piece j of row `lane`.
__device__ __forceinline__ uint32_t piece(uint32_t buf, int lane, int j) {
  return buf + static_cast<uint32_t>(lane) * 128u + (static_cast<uint32_t>(j ^ (lane & 7)) << 4);
}

// A whole 32-byte sector by one thread (aligned).
__device__ __forceinline__ void st_global_32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Columns past the vocabulary in a 32-column chunk starting at `col` do not count.
__device__ __forceinline__ void mask_columns(uint32_t (&r)[32], int col, int n) {
  if (col + 32 <= n) return;
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if (col + j >= n) r[j] = 0xff800000u;  // -inf
}

__device__ __forceinline__ float max_of(const uint32_t (&r)[32]) {
  float m[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    m[k] = __uint_as_float(r[k]);
#pragma unroll
    for (int j = k + 4; j < 32; j += 4) m[k] = fmaxf(m[k], __uint_as_float(r[j]));
  }
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// The accumulator is read twice, 32 columns at a time: once for the maximum
// and once for the sums and logs.  Holding all 128 columns in registers
// spills (168 registers a thread with 12 warps) and measured 2.1 times the
// time of the whole product at 4096 x 50257 x 768.
// `target`: of this thread's row, -1 for none.  Calls `release` once the last
// column has left the TMEM.
// ENT: also the sum of 2^(z - m) (z - m), of which the entropy is made; a z of -inf has no part in it.
// COARSE: VocabLogTop's logs.
template <bool ENT, bool COARSE, class Args, class Release>
__device__ __forceinline__ void logits_epilogue(const Args& G, uint32_t t_lane, int row, int target, int col0,
                                                Release release) {
  const float c = G.logit_scale_log2;
  const float minus_inf = __int_as_float(0xff800000);
  const int n = G.N;
  uint32_t ra[32], rb[32];
  float m = minus_inf;
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    tmem_ld_32x32b_x32(t_lane + 32u * i, ra);
    tmem_ld_32x32b_x32(t_lane + 32u * (i + 1), rb);
    tmem_ld_wait_regs(ra);
    tmem_ld_wait_regs(rb);
    mask_columns(ra, col0 + 32 * i, n);
    mask_columns(rb, col0 + 32 * (i + 1), n);
    m = fmaxf(m, fmaxf(max_of(ra), max_of(rb)));
  }
  m *= c;  // c > 0
  // Above every z by more than the rounding of the products below, so that no
  // distance comes out negative.
  // Only -inf and NaN: the pair is -inf and a sum of 0 or NaN, and takes no part in the row's maximum.
  if (m != minus_inf) m += fabsf(m) * 2.4e-7f;
  const float ref = m == minus_inf ? 0.f : m;
  const bool row_ok = row < G.M;
  const int at = target >= 0 ? target - col0 : -1;
  constexpr int kLogBytes = COARSE ? 1 : 2;
  char* logs = G.logs && row_ok ? reinterpret_cast<char*>(G.logs) + (static_cast<int64_t>(row) * G.ld_logs + col0) * kLogBytes : nullptr;
  const int stored = static_cast<int>(min(static_cast<int64_t>(kCeBlock), G.ld_logs - col0));  // a multiple of 64
  // A distance is rounded to the nearest unit by adding 2^23, whose low
  // mantissa bits then are the integer; past 64 octaves it stays at the largest.
  const float magic = 8388608.f, most = magic + 65535.f;
  float s[4] = {0.f, 0.f, 0.f, 0.f}, t[4] = {0.f, 0.f, 0.f, 0.f};
  auto chunk = [&](uint32_t (&q)[32], int i) {
    // The target's share of the sum is added by the row pass.
    if (__any_sync(0xffffffffu, (at >> 5) == i)) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (at == 32 * i + j) q[j] = 0xff800000u;  // -inf
    }
    mask_columns(q, col0 + 32 * i, n);
    uint32_t coarse[8];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      uint32_t w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float lo = fmaf(__uint_as_float(q[16 * p + 2 * k]), c, -ref);
        const float hi = fmaf(__uint_as_float(q[16 * p + 2 * k + 1]), c, -ref);
        const float e_lo = ex2(lo), e_hi = ex2(hi);
        s[k & 3] += e_lo;
        s[k & 3] += e_hi;
        if constexpr (ENT) {
          t[k & 3] = fmaf(e_lo, fmaxf(lo, kNoLogit), t[k & 3]);
          t[k & 3] = fmaf(e_hi, fmaxf(hi, kNoLogit), t[k & 3]);
        }
        if constexpr (COARSE) {
          const uint32_t two = pack_e4m3x2(-lo, -hi);
          coarse[4 * p + (k >> 1)] = k & 1 ? __byte_perm(coarse[4 * p + (k >> 1)], two, 0x5410) : two;
        } else {
          w[k] = __byte_perm(__float_as_uint(fminf(fmaf(lo, -kCeLogUnits, magic), most)),
                             __float_as_uint(fminf(fmaf(hi, -kCeLogUnits, magic), most)), 0x5410);
        }
      }
      if constexpr (!COARSE) {
        if (logs && 32 * i < stored) st_global_32(logs + 64 * i + 32 * p, w);
      }
    }
    if constexpr (COARSE) {
      if (logs && 32 * i < stored) st_global_32(logs + 32 * i, coarse);
    }
  };
  // The next chunk's load is in flight while one is worked on.
  tmem_ld_32x32b_x32(t_lane, ra);
  tmem_ld_wait_regs(ra);
  tmem_ld_32x32b_x32(t_lane + 32u, rb);
  chunk(ra, 0);
  tmem_ld_wait_regs(rb);
  tmem_ld_32x32b_x32(t_lane + 64u, ra);
  chunk(rb, 1);
  tmem_ld_wait_regs(ra);
  tmem_ld_32x32b_x32(t_lane + 96u, rb);
  chunk(ra, 2);
  tmem_ld_wait_regs(rb);
  release();
  chunk(rb, 3);
  if (row_ok)
    G.stats[static_cast<int64_t>(col0 / kCeBlock) * G.stats_ld + row] = make_float2(m, (s[0] + s[1]) + (s[2] + s[3]));
  if constexpr (ENT) {
    if (row_ok) G.weighted[static_cast<int64_t>(col0 / kCeBlock) * G.stats_ld + row] = (t[0] + t[1]) + (t[2] + t[3]);
  }
}

__device__ __forceinline__ void bf16_epilogue(const VgProduct& P, uint32_t (&r)[4][32], float alpha, int col0,
                                              int warp_row0, uint32_t staging, int lane) {
  if (lane == 0) bulk_wait_group_read<0>();
  __syncwarp();
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const uint32_t buf = staging + 4096u * b;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int j = 64 * b + 8 * p + 2 * k;
        w[k] = pack_bf16x2(alpha * __uint_as_float(r[j >> 5][j & 31]), alpha * __uint_as_float(r[(j + 1) >> 5][(j + 1) & 31]));
      }
      st_shared_16(piece(buf, lane, p), w[0], w[1], w[2], w[3]);
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_3d(&P.map_out, staging, col0, warp_row0, 0);
    if (col0 + 64 < P.N) tma_store_3d(&P.map_out, staging + 4096u, col0 + 64, warp_row0, 0);
    bulk_commit_group();
  }
}

__device__ __forceinline__ void f32_epilogue(const VgProduct& P, uint32_t (&r)[4][32], float alpha, int col0,
                                             int warp_row0, int split, uint32_t staging, int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (col0 + 32 * i >= P.N) break;
    const uint32_t buf = staging + 4096u * (i & 1);
    if (lane == 0) {
      if (i == 0)
        bulk_wait_group_read<0>();
      else
        bulk_wait_group_read<1>();
    }
    __syncwarp();
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = __float_as_uint(alpha * __uint_as_float(r[i][4 * p + k]));
      st_shared_16(piece(buf, lane, p), w[0], w[1], w[2], w[3]);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      if (P.add)
        tma_add_3d(&P.map_out, buf, col0 + 32 * i, warp_row0, split);
      else
        tma_store_3d(&P.map_out, buf, col0 + 32 * i, warp_row0, split);
      bulk_commit_group();
    }
  }
}

// bf16 rows that start anywhere: the warp packs its 32 x 128 block in shared
// memory and writes each row in whole 16-byte pieces with single values at
// the two ends.  (Two-byte stores of 32 columns at a time leave most 32-byte
// sectors written in two parts, which took twice the time.)
__device__ __forceinline__ void unaligned_bf16_epilogue(const VgProduct& P, uint32_t (&r)[4][32], float alpha, int col0,
                                                        int warp_row0, uint32_t staging, int lane) {
  if (lane == 0) bulk_wait_group_read<0>();  // stores of the other product
  __syncwarp();
#pragma unroll
  for (int p = 0; p < 16; ++p) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int j = 8 * p + 2 * k;
      w[k] = pack_bf16x2(alpha * __uint_as_float(r[j >> 5][j & 31]), alpha * __uint_as_float(r[(j + 1) >> 5][(j + 1) & 31]));
    }
    st_shared_16(piece(staging + 4096u * (p >> 3), lane, p & 7), w[0], w[1], w[2], w[3]);
  }
  __syncwarp();
  const int rows = min(32, P.M - warp_row0), cols = min(128, P.N - col0);
  const int part = lane & 15;
#pragma unroll 4
  for (int it = 0; it < 16; ++it) {
    const int row = 2 * it + (lane >> 4);
    if (row >= rows) continue;
    uint16_t* out = static_cast<uint16_t*>(P.out) + static_cast<int64_t>(warp_row0 + row) * P.ld_out + col0;
    // Columns 2 i and 2 i + 1 of the row.
    auto word = [&](int i) {
      uint32_t v;
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(piece(staging + 4096u * (i >> 5), row, (i >> 2) & 7) + 4u * (i & 3)));
      return v;
    };
    auto value = [&](int c) { return static_cast<uint16_t>(word(c >> 1) >> (16 * (c & 1))); };
    const int head = min(cols, static_cast<int>((8u - ((reinterpret_cast<uintptr_t>(out) >> 1) & 7u)) & 7u));
    const int pieces = (cols - head) >> 3, tail = head + 8 * pieces;
    if (part < pieces) {
      // Eight columns from head + 8 part on: four words, or five where that is odd.
      const int i = (head + 8 * part) >> 1;
      const uint32_t odd = head & 1, shift = 16 * odd;
      const uint32_t w0 = word(i), w1 = word(i + 1), w2 = word(i + 2), w3 = word(i + 3), w4 = odd ? word(i + 4) : 0u;
      *reinterpret_cast<uint4*>(out + head + 8 * part) =
          make_uint4(__funnelshift_r(w0, w1, shift), __funnelshift_r(w1, w2, shift), __funnelshift_r(w2, w3, shift),
                     __funnelshift_r(w3, w4, shift));
    }
    if (part < head) out[part] = value(part);
    if (tail + part < cols) out[tail + part] = value(tail + part);
  }
  __syncwarp();
}

// Without TMA: the warp turns each 32 x 32 block around in shared memory, so
// that a store instruction writes 32 neighbouring columns of one row.
__device__ __forceinline__ void direct_epilogue(const VgProduct& P, uint32_t (&r)[4][32], float alpha, int col0, int warp_row0,
                                                uint32_t staging, int lane) {
  if (lane == 0) bulk_wait_group_read<0>();  // stores of the other product
  const int rows = min(32, P.M - warp_row0);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (col0 + 32 * i >= P.N) break;
    const uint32_t buf = staging + 4096u * (i & 1);
    __syncwarp();
#pragma unroll
    for (int p = 0; p < 8; ++p) st_shared_16(piece(buf, lane, p), r[i][4 * p], r[i][4 * p + 1], r[i][4 * p + 2], r[i][4 * p + 3]);
    __syncwarp();
    const int col = col0 + 32 * i + lane;
    const int64_t at = static_cast<int64_t>(warp_row0) * P.ld_out + col;
    uint16_t* h = static_cast<uint16_t*>(P.out) + at;
    float* f = static_cast<float*>(P.out) + at;
    if (col < P.N) {
      for (int r0 = 0; r0 < rows; r0 += 8) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          uint32_t w;
          asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(piece(buf, r0 + k, lane >> 2) + 4u * (lane & 3)));
          v[k] = alpha * __uint_as_float(w);
        }
        if (P.add) {
          float old[8];
#pragma unroll
          for (int k = 0; k < 8; ++k)
            old[k] = r0 + k >= rows ? 0.f : P.out_bf16 ? bf16_bits_to_f32(h[(r0 + k) * P.ld_out]) : f[(r0 + k) * P.ld_out];
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] += old[k];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (r0 + k >= rows) break;
          if (P.out_bf16)
            h[(r0 + k) * P.ld_out] = to_bf16_bits(v[k]);
          else
            f[(r0 + k) * P.ld_out] = v[k];
        }
      }
    }
  }
  __syncwarp();
}

// The parts of a tile's product that differ between the two kernels.
__device__ __forceinline__ const CUtensorMap* operand_map(const VocabLogits& G, int, bool b) { return b ? &G.map_b : &G.map_a; }
__device__ __forceinline__ const CUtensorMap* operand_map(const VocabGrad& G, int p, bool b) {
  return b ? &G.p[p].map_b : &G.p[p].map_a;
}
__device__ __forceinline__ bool a_is_mn(const VocabLogits&, int) { return false; }
__device__ __forceinline__ bool a_is_mn(const VocabGrad& G, int p) { return G.p[p].a_mn != 0; }

// Args: VocabLogits, VocabLogProbs or VocabLogTop (B is vocabulary x width,
// K-contiguous), or VocabGrad (B is N-contiguous).
template <class Args, bool B_MN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads + (kCanNorm<Args> ? 32 * kNormWarps : 0), 1)
    vocab_gemm_kernel(const __grid_constant__ Args G) {
  constexpr bool LOGITS = !B_MN;
  constexpr int kProducerBWarp = 2 + EPI;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t ring = smem_u32(smem);
  const uint32_t staging = ring + STAGES * STAGE_BYTES;
  uint64_t* bar_mem = reinterpret_cast<uint64_t*>(smem + STAGES * STAGE_BYTES + EPI * kStaging);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_mem + kNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* mailbox = reinterpret_cast<volatile int*>(tmem_slot + 2);  // kMail tile numbers
  const uint32_t bar0 = smem_u32(bar_mem);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (STAGES + s); };
  auto tfull = [&](int a) { return bar0 + 8u * (2 * STAGES + a); };
  auto tempty = [&](int a) { return bar0 + 8u * (2 * STAGES + 2 + a); };
  const uint32_t drain = bar0 + 8u * (2 * STAGES + 4);
  auto mail_full = [&](int i) { return bar0 + 8u * (2 * STAGES + 5 + i); };
  auto mail_empty = [&](int i) { return bar0 + 8u * (2 * STAGES + 5 + kMail + i); };  // the leader's is used
  // A stage whose rows of W the norms' warps may read, and have read: in the tiles that they take norms in.
  auto readable = [&](int s) { return bar0 + 8u * (2 * STAGES + 5 + 2 * kMail + s); };
  auto read = [&](int s) { return bar0 + 8u * (3 * STAGES + 5 + 2 * kMail + s); };
  const bool norms = norms_of(G) != nullptr;

  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full(s), 2);  // one arrival per operand producer of the leader
      mbar_init(empty(s), 1);
      mbar_init(readable(s), 1);
      mbar_init(read(s), kNormWarps);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull(a), 1);
      mbar_init(tempty(a), 2 * EPI);
    }
    mbar_init(drain, 1);
    for (int i = 0; i < kMail; ++i) {
      mbar_init(mail_full(i), 1);
      mbar_init(mail_empty(i), kReaders + (norms ? 2 * kNormWarps : 0));
    }
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();  // both CTAs' barriers exist before any cross-CTA signal
  tc_fence_after();
  pdl_launch();
  pdl_wait();
  const uint32_t tmem_base = *tmem_slot;

  const bool drawn = G.drawn != 0;
  const FixedShares shares = fixed_shares(G);
  // The i-th tile of this pair, as every role reads it.
  auto next_tile = [&](int i, bool whole_warp) {
    if (!drawn) return tile_at(G, shares.at(i));
    const int at = i % kMail;
    int t = -1;
    if (mbar_wait_bounded_cluster(mail_full(at), static_cast<uint32_t>(i / kMail) & 1u, abort_flag, G.err, kErrTimeoutMailbox))
      t = mailbox[at];
    if (whole_warp) __syncwarp();
    if (!whole_warp || lane == 0) {
      if (leader)
        mbar_arrive(mail_empty(at));
      else
        mbar_arrive_cluster(mapa_shared(mail_empty(at), 0));
    }
    return tile_at(G, t);
  };

  if ((warp == 0 || warp == kProducerBWarp) && elect_one()) {
    // ------------------------------------ producers (A: warp 0, B: the last)
    const bool is_b = warp != 0;
    const uint32_t dst_off = is_b ? HALF_BYTES : 0u;
    const uint32_t leader_full0 = mapa_shared(full(0), 0);
    int stage = 0, filled = 0;
    uint32_t phase = 0;
    uint32_t to_read = 0, read_phase = 0;  // by stages
    bool ok = true;
    for (int i = 0; ok; ++i) {
      const Tile T = next_tile(i, false);
      if (T.product < 0) break;
      const bool has_norms = norms && is_b && T.m0 == 0;
      const CUtensorMap* map = operand_map(G, T.product, is_b);
      const bool mn = is_b ? B_MN : a_is_mn(G, T.product);
      const int row0 = (is_b ? T.n0 : T.m0) + 128 * static_cast<int>(rank);
      for (int kb = T.kb0; kb < T.kb1; ++kb) {
        if (!mbar_wait_bounded_cluster(empty(stage), phase ^ 1u, abort_flag, G.err, kErrTimeoutProducer)) {
          ok = false;
          break;
        }
        if constexpr (kCanNorm<Args>) {
          const uint32_t bit = 1u << stage;
          if (to_read & bit) {
            if (!mbar_wait_bounded(read(stage), read_phase & bit ? 1u : 0u, abort_flag, G.err, kErrTimeoutProducer)) {
              ok = false;
              break;
            }
            read_phase ^= bit;
          }
          to_read = has_norms ? to_read | bit : to_read & ~bit;
        }
        const uint32_t leader_full = leader_full0 + 8u * stage;
        if (leader) mbar_expect_tx(full(stage), 2 * HALF_BYTES);
        ++filled;
        const uint32_t dst = ring + stage * STAGE_BYTES + dst_off;
        if (!mn) {
          tma_load_3d_pair(dst, map, leader_full, kb * BK, row0, 0);
        } else {
          tma_load_3d_pair(dst, map, leader_full, row0, kb * BK, 0);
          tma_load_3d_pair(dst + MN_BOX_BYTES, map, leader_full, row0 + 64, kb * BK, 0);
        }
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok && leader) {
      // The leader's barriers count both CTAs' bytes: let every armed phase land
      // before the pair tears down.  Stage s was armed ceil((filled - s) / STAGES) times.
      for (int s = 0; s < STAGES && s < filled; ++s) {
        volatile int no_abort = 0;
        const int uses = (filled - s + STAGES - 1) / STAGES;
        mbar_wait_bounded_cluster(full(s), static_cast<uint32_t>(uses - 1) & 1u, &no_abort, nullptr, 0, 100000000ull);
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------- MMA issuer (leader only)
    if (leader && elect_one()) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      int use = 0;
      for (; ok; ++use) {
        const Tile T = next_tile(use, false);
        if (T.product < 0) break;
        const bool a_mn = a_is_mn(G, T.product);
        const uint32_t idesc = idesc_bf16_f32(TILE, TILE, a_mn, B_MN);
        // Descriptors of stage 0; a stage or a 16-deep step on is an addition to
        // the address field (units of 16 bytes).
        const uint64_t a0 = a_mn ? desc_mn(ring, 0) : desc_k(ring, 0);
        const uint64_t b0 = B_MN ? desc_mn(ring + HALF_BYTES, 0) : desc_k(ring + HALF_BYTES, 0);
        const uint32_t a_step = a_mn ? 2048u >> 4 : 32u >> 4;
        constexpr uint32_t b_step = B_MN ? 2048u >> 4 : 32u >> 4;
        if (!mbar_wait_bounded_cluster(tempty(use & 1), (static_cast<uint32_t>(use >> 1) & 1u) ^ 1u, abort_flag, G.err,
                                       kErrTimeoutMma))
          break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>((use & 1) * TILE);
        for (int kb = T.kb0; kb < T.kb1; ++kb) {
          if (!mbar_wait_bounded_cluster(full(stage), phase, abort_flag, G.err, kErrTimeoutMma)) {
            ok = false;
            break;
          }
          tc_fence_after();
          // Both CTAs' copies have landed: tells the norms' warps so, once the MMAs of the stage before are done.
          if (kCanNorm<Args> && norms && T.m0 == 0) umma_commit_pair_multicast(readable(stage), 0x3);
          const uint64_t ad = a0 + static_cast<uint32_t>(stage) * (STAGE_BYTES >> 4);
          const uint64_t bd = b0 + static_cast<uint32_t>(stage) * (STAGE_BYTES >> 4);
          umma_bf16_pair(d_tmem, ad, bd, idesc, kb != T.kb0 ? 1u : 0u);
#pragma unroll
          for (int kk = 1; kk < BK / 16; ++kk) umma_bf16_pair(d_tmem, ad + kk * a_step, bd + kk * b_step, idesc, 1u);
          umma_commit_pair_multicast(empty(stage), 0x3);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok) umma_commit_pair_multicast(tfull(use & 1), 0x3);
      }
      umma_commit_pair_multicast(drain, 0x1);
      volatile int no_abort = 0;
      mbar_wait_bounded_cluster(drain, 0, &no_abort, G.err, kErrTimeoutDrain);
    }
  } else if (warp >= 2 && warp < 2 + EPI) {
    // ------------------------------------------------------------ epilogue
    // A warp reaches the TMEM lanes of its warp index mod 4; the two warps of
    // a lane quarter take 128 columns each.
    const int quarter = warp & 3;
    const int half = (warp - 2) >> 2;
    const uint32_t my_staging = staging + static_cast<uint32_t>(warp - 2) * kStaging;
    int use = 0;
    float alpha = 1.f;
    if constexpr (!LOGITS) alpha = G.alpha ? *G.alpha : 1.f;
    for (;; ++use) {
      const Tile T = next_tile(use, true);
      if (T.product < 0) break;
      const int acc = use & 1;
      const int warp_row0 = T.m0 + 128 * static_cast<int>(rank) + 32 * quarter;
      const int col0 = T.n0 + 128 * half;
      int target = -1, rows, cols;
      if constexpr (LOGITS) {
        rows = G.M;
        cols = G.N;
        bool bad = false;
        if (G.targets.p && warp_row0 + lane < rows) target = load_id(G.targets, warp_row0 + lane, &bad);
      } else {
        rows = G.p[T.product].M;
        cols = G.p[T.product].N;
      }
      if (!mbar_wait_bounded_cluster(tfull(acc), static_cast<uint32_t>(use >> 1) & 1u, abort_flag, G.err,
                                     kErrTimeoutEpilogue))
        break;
      tc_fence_after();
      const uint32_t t_lane =
          tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(acc * TILE + 128 * half);
      // Hands the accumulator back: its columns have been read.
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (leader)
            mbar_arrive(tempty(acc));
          else
            arrive_relaxed(mapa_shared(tempty(acc), 0));
        }
      };
      if (warp_row0 >= rows || col0 >= cols) {  // warp-uniform
        release();
        continue;
      }
      if constexpr (LOGITS) {
        constexpr bool kCoarse = std::is_same<Args, VocabLogTop>::value;
        logits_epilogue<kCoarse || std::is_same<Args, VocabLogProbs>::value, kCoarse>(G, t_lane, warp_row0 + lane, target, col0, release);
      } else {
        const VgProduct& P = G.p[T.product];
        uint32_t r[4][32];
        load_columns(t_lane, r);
        release();
        if (P.direct && P.out_bf16 && !P.add)
          unaligned_bf16_epilogue(P, r, alpha, col0, warp_row0, my_staging, lane);
        else if (P.direct)
          direct_epilogue(P, r, alpha, col0, warp_row0, my_staging, lane);
        else if (P.out_bf16)
          bf16_epilogue(P, r, alpha, col0, warp_row0, my_staging, lane);
        else
          f32_epilogue(P, r, alpha, col0, warp_row0, T.split, my_staging, lane);
      }
    }
    if (lane == 0) bulk_wait_group<0>();
    __syncwarp();
  } else if (kCanNorm<Args> && warp >= kNormWarp) {
    // --------------------------------------------------------------- norms
    const int row = 32 * (warp - kNormWarp) + lane;  // of this CTA's half of the tile's rows of W
    int stage = 0;
    uint32_t phases = 0;  // by stages
    bool ok = norms;
    for (int i = 0; ok; ++i) {
      const Tile T = next_tile(i, true);
      if (T.product < 0) break;
      if (T.m0 != 0) {
        stage = (stage + T.kb1 - T.kb0) % STAGES;
        continue;
      }
      float s[4] = {0.f, 0.f, 0.f, 0.f};
      for (int kb = T.kb0; kb < T.kb1; ++kb) {
        const uint32_t bit = 1u << stage;
        ok = __all_sync(0xffffffffu, mbar_wait_bounded_cluster(readable(stage), phases & bit ? 1u : 0u, abort_flag, G.err, kErrTimeoutEpilogue));
        if (!ok) break;
        phases ^= bit;
        add_row_squares(smem + stage * STAGE_BYTES + HALF_BYTES, row, s);
        __syncwarp();
        if (lane == 0) mbar_arrive(read(stage));
        stage = stage + 1 == STAGES ? 0 : stage + 1;
      }
      const float most = warp_max((s[0] + s[1]) + (s[2] + s[3]));  // rows past the vocabulary are zeros
      const int v0 = T.n0 + 128 * static_cast<int>(rank) + row - lane;
      if constexpr (kCanNorm<Args>) {
        // Whole blocks of statistics, the last one's rows past the vocabulary too.
        if (ok && lane == 0 && v0 < (G.N + kCeBlock - 1) / kCeBlock * kCeBlock) G.norms[v0 / kNormRows] = largest_norm(most);
      }
    }
  }

  if (warp == kSchedWarp && !leader && blockIdx.x == 1) {
    // The other CTA's scheduling warp is free for the sums on the side.
    if constexpr (LOGITS) {
      if (G.norm.alpha) write_alpha(G.norm, lane);
    } else {
      if (G.total.total) write_total(G.total, lane);
    }
    __syncwarp();
  }
  if (drawn && warp == kSchedWarp && leader && lane == 0) {
    // ------------------------------------------------------ tile numbers
    const int total = tiles_in(G);
    for (int i = 0;; ++i) {
      const int at = i % kMail;
      if (!mbar_wait_bounded_cluster(mail_empty(at), (static_cast<uint32_t>(i / kMail) & 1u) ^ 1u, abort_flag, G.err,
                                     kErrTimeoutMailbox))
        break;
      int t = static_cast<int>(atomicAdd(G.counter, 1u));
      if (t >= total) t = -1;
      mailbox[at] = t;
      st_cluster_u32(mapa_shared(smem_u32(const_cast<int*>(mailbox)) + 4u * at, 1), static_cast<uint32_t>(t));
      mbar_arrive(mail_full(at));
      mbar_arrive_cluster(mapa_shared(mail_full(at), 1));
      if (t < 0) break;
    }
  }

  tc_fence_before();
  cluster_sync_all();  // all MMAs drained, no more cross-CTA traffic
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

template <class Args, bool B_MN>
cudaError_t launch(const Args& G, int64_t tiles, int n_pairs, cudaStream_t st) {
  static unsigned long long attr_mask = 0;
  if (attr_needed_on_current_device(&attr_mask)) {
    cudaError_t e = cudaFuncSetAttribute(vocab_gemm_kernel<Args, B_MN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(kSmem));
    if (e != cudaSuccess) return e;
    attr_note_current_device(&attr_mask);
  }
  if (tiles <= 0 || n_pairs <= 0) return cudaErrorInvalidValue;
  const int pairs = static_cast<int>(tiles < n_pairs ? tiles : n_pairs);
  const int threads = kThreads + (norms_of(G) ? 32 * kNormWarps : 0);
  return launch_after(vocab_gemm_kernel<Args, B_MN>, dim3(2 * pairs), dim3(threads), kSmem, st, G);
}

}  // namespace

cudaError_t launch_vocab_logits(const VocabLogits& G, int n_pairs, cudaStream_t st) {
  return launch<VocabLogits, false>(G, G.grid.count(), n_pairs, st);
}

cudaError_t launch_vocab_logits(const VocabLogProbs& G, int n_pairs, cudaStream_t st) {
  return launch<VocabLogProbs, false>(G, G.grid.count(), n_pairs, st);
}

cudaError_t launch_vocab_logits(const VocabLogTop& G, int n_pairs, cudaStream_t st) {
  return launch<VocabLogTop, false>(G, G.grid.count(), n_pairs, st);
}

cudaError_t launch_vocab_grad(const VocabGrad& G, int n_pairs, cudaStream_t st) {
  return launch<VocabGrad, true>(G, static_cast<int64_t>(G.n_units[0]) + G.n_units[1], n_pairs, st);
}

// CTA pairs that can be resident at once.
int vocab_gemm_max_pairs() {
  auto kernel = vocab_gemm_kernel<VocabLogits, false>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem)) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  cudaLaunchConfig_t cfg = {};  // the cluster shape comes from __cluster_dims__
  cfg.gridDim = dim3(2, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  return n;
}

}  // namespace dmuon
