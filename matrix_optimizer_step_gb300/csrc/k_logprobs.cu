// Row-wise kernels of the token log probabilities (the products are in
// k_vocab_gemm.cu and k_vocab_thin.cu): the rows' sums, their most likely
// entries, and the turn from fixed-point logs into d logits.
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "ptx.cuh"
#include "vocab.h"
#include "vocab_rows.cuh"

namespace dmuon {
namespace {

__device__ __forceinline__ float minus_inf() { return __int_as_float(0xff800000); }

// What the product's rounding may do to a logit, in octaves.  A step of the matrix instruction adds 16 products to the running
// sum: it lines the 17 up to the largest, keeps what reaches 2^-25 of that, and cuts the result off to 24 bits (measured
// with a term of 2^p and small ones beside it, before it or behind it: a small one of 1 counts whole to p = 25 and not at
// all from 26 on, and a sum past 2^23 loses its halves towards zero).  No product and no running sum is larger than |x| |w|
// (Cauchy and Schwarz), so a step is off by at most (17 2^-25 + 2^-23) |x| |w|, 10.5 roundoffs of it, whatever the signs of its
// terms; 13 are taken, which covers the rounding of the norms.  Where the width is cut into sums of their own, each is off by as many of
// its parts' norms, whose products add up to |x| |w| at most: `steps` are those of one.  Joined sums, the scale and the fixed-point
// logs: 32 more and 2^-9 octaves.
__device__ __forceinline__ float slack_unit(float x_squares, double logit_scale_log2, int steps) {
  const float norm = sqrtf(fmaxf(x_squares, 1e-30f));
  return norm * static_cast<float>(logit_scale_log2) * (static_cast<float>(13 * steps + 32) * 0x1p-24f);
}
// Largest norm of the rows of w of statistics block b.
__device__ __forceinline__ float block_norm(const float* norms, int stats_shift, int b) {
  if (stats_shift == kCeThinShift) return norms[b];
  const float4 q = reinterpret_cast<const float4*>(norms)[b];
  return fmaxf(fmaxf(q.x, q.y), fmaxf(q.z, q.w));
}
// Of a logit with a row of w of that norm.
__device__ __forceinline__ float logit_slack(float unit, float norm) {
  const float s = fmaf(unit, norm, 0x1p-9f);
  return s < __int_as_float(0x7f800000) ? s : __int_as_float(0x7f800000);  // 0 times infinity
}

// A value that at least k of the warp's values reach (PER of them a lane) and, unless
// values crowd there, not many more; -inf where k of them are not above it.
template <int PER>
__device__ __forceinline__ float reached_by(const float (&v)[PER], int k) {
  float top = v[0];
#pragma unroll
  for (int i = 1; i < PER; ++i) top = fmaxf(top, v[i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  auto reach = [&](float at) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) n += v[i] >= at ? 1 : 0;
    return __reduce_add_sync(0xffffffffu, n);
  };
  float step = 2.f, above = top, at = top - step;
  int n = reach(at);
  while (n < k) {
    if (step > 1e6f) return minus_inf();
    above = at;
    step *= 2.f;
    at = top - step;
    n = reach(at);
  }
  for (int i = 0; i < 10 && n > k + 2; ++i) {
    const float mid = 0.5f * (at + above);
    const int m = reach(mid);
    if (m >= k) {
      at = mid;
      n = m;
    } else {
      above = mid;
    }
  }
  return at;
}

// ---------------------------------------------------------- most likely entries
// The k largest logits of a row, equal ones by their numbers, in the order that
// sums of 64 bits give.  The row pass has bounded them from below and listed the
// blocks that may hold one.  The logs (16- or 8-bit distances to the blocks' maxima)
// bound each logit from both sides, to half a step and the product's rounding, and
// only entries that may be among the k are multiplied out again:
//   1. of the listed blocks' entries those whose upper bound reaches the row's, and of
//      these the ones that reach the k-th largest lower bound: k and a few more;
//   2. their logits as sums of fp32, with a bound of their error; those that lie
//      closer to another than both errors again, exact to about 48 bits.
// A block takes a row.  Below 512 rows, where its latency counts, it has the row pass's
// 16 warps and no launch of its own (4 warps in one: 207 us for 184 with 1 row at 128256 x 4096, 50 for 43
// with 128 at 50257 x 768); from there on 4.  Calls with 20 alternatives: 600 x 128256 x 1024 148 us (2 warps:
// 159, 8: 145, 16: 152), 4096 x 50257 x 768 256 (2: 252, 8: 271, 16: 311), 8192 x 32000 x 2048 765 (2: 773,
// 8: 827, 16: 872), all before the norms of w's rows were taken.  At 4096 x 50257 x 768 the pass itself takes 60 us from cold caches,
// with half of the issue slots and a sixth of the memory's rate in use.
//
// More candidates than there is room for (equal or nearly equal logits) are taken
// kWindow entries at a time; a row of zeros, all of whose logits are equal, is known without.
constexpr int kWindow = 128;     // candidate entries

// a + p without loss: the sum in a, what it rounds away in `lost` (Knuth's two-sum).
__device__ __forceinline__ void add_exactly(float& a, float& lost, float p) {
  const float s = a + p, back = s - a;
  lost += (a - (s - back)) + (p - back);
  a = s;
}

// Dot product of two bf16 rows on 16-byte boundaries to about 48 bits, the same in every lane.
__device__ __noinline__ double warp_dot_exact(const uint16_t* a, const uint16_t* b, int n, int lane) {
  float sum[4] = {0.f, 0.f, 0.f, 0.f}, lost[4] = {0.f, 0.f, 0.f, 0.f};
  for (int c = lane; c < n >> 3; c += 32) {
    const uint4 p = reinterpret_cast<const uint4*>(a)[c], q = reinterpret_cast<const uint4*>(b)[c];
    const uint32_t u[4] = {p.x, p.y, p.z, p.w}, v[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      add_exactly(sum[i], lost[i], __fmul_rn(__uint_as_float(u[i] << 16), __uint_as_float(v[i] << 16)));
      add_exactly(sum[i], lost[i], __fmul_rn(__uint_as_float(u[i] & 0xFFFF0000u), __uint_as_float(v[i] & 0xFFFF0000u)));
    }
  }
  for (int c = (n & ~7) + lane; c < n; c += 32) add_exactly(sum[0], lost[0], __fmul_rn(bf16_bits_to_f32(a[c]), bf16_bits_to_f32(b[c])));
  double d = 0.0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    d += static_cast<double>(sum[i]);
    if (isfinite(sum[i])) d += static_cast<double>(lost[i]);  // of an infinite sum nothing else is known
  }
  return warp_sum(d);
}

// Sum of each of N values over the warp's lanes; lane l has that of value l % N.
template <int N>
__device__ __forceinline__ float sum_values(float (&v)[N], int lane) {
#pragma unroll
  for (int d = N / 2; d > 0; d >>= 1) {
    const bool up = (lane & d) != 0;
#pragma unroll
    for (int j = 0; j < d; ++j) {
      const float keep = up ? v[j + d] : v[j], send = up ? v[j] : v[j + d];
      v[j] = keep + __shfl_xor_sync(0xffffffffu, send, d);
    }
  }
#pragma unroll
  for (int d = N; d < 32; d <<= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], d);
  return v[0];
}

// Two fp32 side by side, and two multiply-adds in one instruction.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ uint64_t pair_of_bf16(uint32_t w) { return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }
__device__ __forceinline__ void fma_pair(uint64_t& c, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c) : "l"(a), "l"(b));
}
__device__ __forceinline__ float sum_of_pair(uint64_t v) {
  float a, b;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
  return a + b;
}

// Dot products of x with N rows of w (all on 16-byte boundaries) in fp32, four chains a lane (64-bit sums of all
// candidates took a quarter of this kernel's time: an SM adds two a cycle).  No dot product is off by more than a roundoff of
// sum |x_k w_k| <= |x| |w| for each step of its longest chain; the norms cost less than that sum.
// Lane l returns what concerns row l % N.
struct DotBound {
  float z, error;
};
template <int N>
__device__ __forceinline__ DotBound warp_dots(const uint16_t* x, const uint16_t* const (&w)[N], int n, int lane) {
  uint64_t sum[N][2], ww[N], xx = 0;  // all bits zero: 0.f twice
#pragma unroll
  for (int r = 0; r < N; ++r) sum[r][0] = sum[r][1] = ww[r] = 0;
  constexpr int kAhead = N > 1 ? 2 : 8;
#pragma unroll kAhead
  for (int c = lane; c < n >> 3; c += 32) {
    uint4 q[N];
    const uint4 p = reinterpret_cast<const uint4*>(x)[c];
#pragma unroll
    for (int r = 0; r < N; ++r) q[r] = reinterpret_cast<const uint4*>(w[r])[c];
    const uint64_t u[4] = {pair_of_bf16(p.x), pair_of_bf16(p.y), pair_of_bf16(p.z), pair_of_bf16(p.w)};
#pragma unroll
    for (int i = 0; i < 4; ++i) fma_pair(xx, u[i], u[i]);
#pragma unroll
    for (int r = 0; r < N; ++r) {
      const uint64_t v[4] = {pair_of_bf16(q[r].x), pair_of_bf16(q[r].y), pair_of_bf16(q[r].z), pair_of_bf16(q[r].w)};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        fma_pair(sum[r][i & 1], u[i], v[i]);
        fma_pair(ww[r], v[i], v[i]);
      }
    }
  }
  for (int c = (n & ~7) + lane; c < n; c += 32) {
    const uint64_t u = pair(bf16_bits_to_f32(x[c]), 0.f);
    fma_pair(xx, u, u);
#pragma unroll
    for (int r = 0; r < N; ++r) {
      const uint64_t v = pair(bf16_bits_to_f32(w[r][c]), 0.f);
      fma_pair(sum[r][0], u, v);
      fma_pair(ww[r], v, v);
    }
  }
  float z[N], norm[N];
#pragma unroll
  for (int r = 0; r < N; ++r) {
    z[r] = sum_of_pair(sum[r][0]) + sum_of_pair(sum[r][1]);
    norm[r] = sum_of_pair(ww[r]);
  }
  float x2 = sum_of_pair(xx);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x2 += __shfl_xor_sync(0xffffffffu, x2, o);
  DotBound d;
  d.z = sum_values(z, lane);
  const float w2 = sum_values(norm, lane);
  // Two steps for each vector of a lane, one for its last element, seven between chains and lanes.  A part in 2^8 more than covers
  // what the norms' own sums round away.  Squares that leave the range of fp32 bound nothing.
  const int steps = 2 * ((n >> 3) / 32 + 1) + 8;
  const bool known = x2 > 1e-30f && w2 > 1e-30f;
  d.error = known ? sqrtf(x2) * sqrtf(w2) * (static_cast<float>(steps) * (0x1p-24f + 0x1p-32f)) : __int_as_float(0x7f800000);
  return d;
}

struct TopShared {
  float group[512];                 // a thread's largest lower bound
  double z[kWindow + kTopMost];     // where some were close: all of them, those exact
  float near[kWindow + kTopMost], error[kWindow + kTopMost];
  int32_t id[kWindow + kTopMost];
  uint8_t again[kWindow + kTopMost], rank[kWindow + kTopMost];
  float upper[kWindow], lower[kWindow];
  int32_t entry[kWindow];
  double best_z[kTopMost];
  int32_t best_id[kTopMost];
  int32_t n_entries, n_ids, close;
};

// By all WARPS of the block; `list`: the row's listed blocks, in either memory.
template <int WARPS>
__device__ __forceinline__ void top_of_row(const LpTop& T, int64_t row, const LpRow& R, const TopBlock* list, TopShared& S) {
  constexpr int kThreads = 32 * WARPS;
  constexpr int kDots = WARPS >= 16 ? 1 : 2;  // candidates that a warp takes at a time
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, thread = threadIdx.x;
  const int k = T.k;
  auto put = [&](int rank, int32_t id, float logprob) {
    if (T.ids64)
      static_cast<long long*>(T.ids)[row * k + rank] = id;
    else
      static_cast<int*>(T.ids)[row * k + rank] = id;
    if (T.logprobs) T.logprobs[row * k + rank] = logprob;
  };
  // A row that is not scored, or has no distribution (NaN, or infinite logits).
  if (!R.scored || !isfinite(R.top) || !isfinite(R.log_sum)) {
    if (thread < k) put(thread, -1, R.scored ? __int_as_float(0x7fc00000) : 0.f);
    return;
  }
  const uint8_t* logs = static_cast<const uint8_t*>(T.block) + row * T.ld_block * (T.coarse ? 1 : 2);
  const uint16_t* x = T.x + row * T.ld_x;
  // An entry that holds more than half is the row's maximum: its share of the sum, which is 1, is taken out and the rest set
  // against its own logit, so that what the product's sum rounded away of it takes no probability above 1.  Not below a half
  // then: the value falls with the logit from one formula to the other.  Beside the given token's logprob, whose
  // logit is summed apart, the others keep their places.  z_t: its z here, -inf where it is not among them.
  auto logprob = [&](double z, int32_t id, double z_t) {
    if (id == R.target) return R.logprob;
    const float d = static_cast<float>(z * T.logit_scale_log2 - R.top);
    float v = kLn2 * (d - R.log_sum);
    if (d > R.log_sum - 1.f) {
      const float share = T.stats_shift == kCeThinShift ? exp2f(-fabsf(R.top) * kThinAbove) : 1.f;
      v = fmaxf(-log1pf(fmaxf(exp2f(R.log_sum) - share, 0.f) / exp2f(d)), -kLn2);
    }
    if (R.target < 0) return v;
    return z > z_t || (z == z_t && id < R.target) ? fmaxf(v, R.logprob) : fminf(v, R.logprob);
  };
  if (thread == 0) S.n_entries = S.n_ids = S.close = 0;
  __syncthreads();

  // This lane's logs of a block, all ones (further off than logs go, or none) past the vocabulary.
  const int per_lane = (1 << T.stats_shift) / 32;
  auto load_entries = [&](int b) {
    const int c0 = (b << T.stats_shift) + lane * per_lane;
    uint2 w = make_uint2(0xffffffffu, 0xffffffffu);
    if (c0 < T.vocab) {
      if (T.coarse)
        w.x = *reinterpret_cast<const uint32_t*>(logs + c0);
      else if (per_lane == 4)
        w = *reinterpret_cast<const uint2*>(logs + 2 * c0);
      else
        w.x = *reinterpret_cast<const uint16_t*>(logs + 2 * c0);
    }
    return w;
  };
  // take(entry, upper and lower bound) for this lane's entries of a block with maximum m whose upper bound reaches `from`.
  // Few do, so their logs are compared as they are with what the bound leaves room for, a little more than it.  An infinite slack
  // (rows of w with infinities) leaves no bound, and none is below `from`.
  auto for_entries = [&](int b, float m, float slack, uint2 w, float from, auto&& take) {
    const int c0 = (b << T.stats_shift) + lane * per_lane;
    const float room = m + slack - from;
    uint32_t some = 0;  // bit j: entry j
    if (T.coarse) {
      // d (1 - 1/16) - 2^-10 <= room; codes without their sign are in the order of what they stand for, and NaN's is the last.
      const uint32_t most = pack_e4m3x2(fmaf(room, 1.25f, 0x1p-6f), 0.f) & 0x7fu;
#pragma unroll
      for (int j = 0; j < 4; ++j) some |= ((w.x >> (8 * j)) & 0x7fu) <= most ? 1u << j : 0u;
    } else {
      const float most = fmaf(room, kCeLogUnits, 2.f);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < per_lane) some |= static_cast<float>(((j & 2) ? w.y : w.x) >> (16 * (j & 1)) & 0xffffu) > most ? 0u : 1u << j;  // NaN: all
    }
    while (some) {
      const int j = __ffs(some) - 1;
      some &= some - 1;
      const int c = c0 + j;
      float z, wide;
      bool far;
      if (T.coarse) {
        // Sign, four bits of exponent (bias 7), three of mantissa: as an fp32's, times 2^120; what is below the first exponent stays exact.
        const uint32_t q = w.x >> (8 * j) & 0x7fu;
        const float d = __uint_as_float(q << 20) * 0x1p120f;
        z = m - d;
        wide = slack + fmaf(d, 0x1p-4f, 0x1p-10f);
        far = q >= 0x7eu;
      } else {
        const uint32_t q = ((j & 2) ? w.y : w.x) >> (16 * (j & 1)) & 0xffffu;
        z = m - static_cast<float>(q) * (1.f / kCeLogUnits);
        wide = slack + 0.5f / kCeLogUnits;
        far = q == 65535u;
      }
      if (!(z + wide < from) && c < T.vocab && c != R.target) take(c, z + wide, far ? minus_inf() : z - wide);
    }
  };
  // Logits of n candidates, then the first k of them in order: take(rank, z, id).
  auto in_order = [&](int n, auto&& take) {
    for (int i = warp * kDots; i < n; i += WARPS * kDots) {
      const uint16_t* w[kDots];
#pragma unroll
      for (int u = 0; u < kDots; ++u) w[u] = T.w + S.id[min(i + u, n - 1)] * T.ld_w;
      const DotBound d = warp_dots(x, w, T.dim, lane);
      if (lane < kDots && i + lane < n) {
        S.near[i + lane] = d.z;
        S.error[i + lane] = d.error;
      }
    }
    __syncthreads();
    for (int i = thread; i < n; i += kThreads) {
      const float z = S.near[i], e = S.error[i];
      bool close = !isfinite(z);
      int rank = 0;
      for (int j = 0; j < n; ++j) {
        const float other = S.near[j];
        rank += other > z;
        close = close || (j != i && fabsf(z - other) <= e + S.error[j]);
      }
      S.again[i] = close;
      S.rank[i] = rank;
      if (close) S.close = 1;
    }
    __syncthreads();
    if (!S.close) {
      for (int i = thread; i < n; i += kThreads)
        if (S.rank[i] < k) take(S.rank[i], static_cast<double>(S.near[i]), S.id[i]);
      return;
    }
    // Closer to another than both errors: once more, exact.
    for (int i = warp; i < n; i += WARPS) {
      const double z = S.again[i] ? warp_dot_exact(x, T.w + S.id[i] * T.ld_w, T.dim, lane) : static_cast<double>(S.near[i]);
      if (lane == 0) S.z[i] = z;
    }
    __syncthreads();
    for (int i = thread; i < n; i += kThreads) {
      const double z = S.z[i];
      const int32_t id = S.id[i];
      int rank = 0;
      for (int j = 0; j < n; ++j) rank += S.z[j] > z || (S.z[j] == z && S.id[j] < id);
      if (rank < k) take(rank, z, id);
    }
  };

  // This lane's entries of the listed blocks that reach `from`.
  auto for_list = [&](float from, auto&& take) {
    constexpr int kLoads = WARPS >= 16 ? 2 : 8;
    for (int i = warp; i < R.blocks; i += kLoads * WARPS) {
      TopBlock b[kLoads];
      uint2 w[kLoads];
#pragma unroll
      for (int u = 0; u < kLoads; ++u) b[u] = list[min(i + u * WARPS, R.blocks - 1)];
#pragma unroll
      for (int u = 0; u < kLoads; ++u) w[u] = load_entries(b[u].block);
#pragma unroll
      for (int u = 0; u < kLoads; ++u)
        if (i + u * WARPS < R.blocks) for_entries(b[u].block, b[u].max, b[u].slack, w[u], from, take);
    }
  };
  if (R.blocks <= kTopBlocks) {
    // Where fewer than k blocks or many close logits leave the row's bound low: a better one from the
    // largest lower bounds of each thread's entries (2162 x 1292 x 3264 with 20 alternatives 118 us, 3.2 ms without).
    float from = R.reached;
    for (int attempt = from == minus_inf() ? 1 : 0; attempt < 2; ++attempt) {
      if (attempt > 0) {
        float own = minus_inf();
        for_list(minus_inf(), [&](int, float, float lower) { own = fmaxf(own, lower); });
        S.group[thread] = own;
        __syncthreads();
        float g[WARPS];
#pragma unroll
        for (int i = 0; i < WARPS; ++i) g[i] = S.group[lane + 32 * i];
        from = fmaxf(from, reached_by<WARPS>(g, k));
        if (thread == 0) S.n_entries = 0;
        __syncthreads();
      }
      for_list(from, [&](int c, float upper, float lower) {
        const int at = atomicAdd(&S.n_entries, 1);
        if (at < kWindow) {
          S.entry[at] = c;
          S.upper[at] = upper;
          S.lower[at] = lower;
        }
      });
      __syncthreads();
      const int n = S.n_entries;
      if (n > kWindow) continue;
      if (warp == 0) {
        float v[kWindow / 32];
#pragma unroll
        for (int i = 0; i < kWindow / 32; ++i) v[i] = lane + 32 * i < n ? S.lower[lane + 32 * i] : minus_inf();
        const float reach = reached_by<kWindow / 32>(v, k);
        int count = R.target >= 0 ? 1 : 0;  // its log is not kept
        if (R.target >= 0 && lane == 0) S.id[0] = R.target;
#pragma unroll
        for (int i = 0; i < kWindow / 32; ++i) {
          const bool in = lane + 32 * i < n && !(S.upper[lane + 32 * i] < reach);
          const unsigned who = __ballot_sync(0xffffffffu, in);
          if (in) S.id[count + __popc(who & ((1u << lane) - 1u))] = S.entry[lane + 32 * i];
          count += __popc(who);
        }
        if (lane == 0) S.n_ids = count;
      }
      __syncthreads();
      in_order(S.n_ids, [&](int rank, double z, int32_t id) {
        // Not at the start: over 100 to 511 rows of 50257 x 768, 32000 x 2048 and 128256 x 1024 with 1 and 20
        // alternatives that is 3.4 % faster to 3.4 % slower, without a rule in the sizes, and on average slower
        // (1 row of 128256 x 4096 184.2 us for 183.3; 300 of 50257 x 768 with one 47.6 for 52.9).
        pdl_launch();
        put(rank, id, logprob(z, id, S.close ? S.z[0] : static_cast<double>(S.near[0])));  // the given token comes first
      });
      return;
    }
  }
  bool any = false;
  for (int c = lane; c < T.dim; c += 32) any = any || (x[c] & 0x7fffu) != 0;
  if (!__any_sync(0xffffffffu, any)) {
    if (thread < k) put(thread, thread, logprob(0.0, thread, 0.0));
    return;
  }
  // A few blocks at a time, each joined with the best before it.
  const int step = kWindow >> T.stats_shift;
  int best = 0;
  for (int b0 = 0; b0 < T.n_blocks; b0 += step) {
    __syncthreads();
    if (thread == 0) S.n_ids = S.close = 0;
    __syncthreads();
    for (int b = b0 + warp; b < min(b0 + step, T.n_blocks); b += WARPS) {
      const float m = T.stats[static_cast<int64_t>(b) * T.stats_ld + row].x, slack = logit_slack(R.unit, block_norm(T.norms, T.stats_shift, b));
      if (m + slack < R.reached) continue;
      for_entries(b, m, slack, load_entries(b), R.reached, [&](int c, float, float) { S.id[atomicAdd(&S.n_ids, 1)] = c; });
    }
    if (thread == 0 && R.target >= 0 && R.target >> T.stats_shift >= b0 && R.target >> T.stats_shift < b0 + step)
      S.id[atomicAdd(&S.n_ids, 1)] = R.target;
    __syncthreads();
    const int n = S.n_ids;
    if (n == 0) continue;
    if (thread < best) S.id[n + thread] = S.best_id[thread];
    __syncthreads();
    in_order(n + best, [&](int rank, double z, int32_t id) {
      S.best_z[rank] = z;
      S.best_id[rank] = id;
    });
    best = min(k, n + best);
  }
  __syncthreads();
  double z_t = static_cast<double>(minus_inf());
  for (int i = 0; i < best; ++i)
    if (S.best_id[i] == R.target) z_t = S.best_z[i];
  if (thread < best) put(thread, S.best_id[thread], logprob(S.best_z[thread], S.best_id[thread], z_t));
}

// Eight blocks an SM (72 registers, seven blocks: 8192 x 32000 x 2048 779 us for 750).
template <int WARPS>
__global__ void __launch_bounds__(32 * WARPS, 8) lp_top_kernel(const LpTop T) {
  __shared__ TopShared S;
  pdl_wait();
  const int64_t row = blockIdx.x;
  const LpRow R = T.rows_in[row];
  top_of_row<WARPS>(T, row, R, T.top_blocks + row * kTopBlocks, S);
}

// ------------------------------------------------------------------- row sums
// Joins a row's blocks, each with its maximum m_b, its sum s_b of 2^(z - m_b)
// and its sum t_b of 2^(z - m_b) (z - m_b), octaves, without the given token's:
//   M = max m_b,  S = sum_b s_b 2^(m_b - M),  T = sum_b 2^(m_b - M) (t_b + s_b (m_b - M)).
// With the given token's logit z_t, summed here in 64 bits as in the cross
// entropy, and o = 2^(z_t - M):
//   ln p_t  = ln(o / (S + o)),
//   entropy = ln 2 (log2(S + o) - (T + o (z_t - M)) / (S + o)),
// where every term of the second is positive but for the rounding of M, so that
// nothing cancels.  A token that holds more than half is the reference itself:
//   ln p_t = -log1p(S / o),  entropy = log1p(S / o) - ln 2 (T - S (z_t - M)) / (S + o),
// and both keep their digits however certain it is.  Blocks, widths and the
// copy of dW's operand are as in ce_rows_kernel.
//
// Where a row's k largest logits are wanted, the same pass bounds them: a value T that
// k of 256 groups of blocks reach with their maxima, found by bisection.  k entries
// lie there or above, so only blocks that reach T (k and a few more, listed
// for lp_top_kernel) hold one.  The maxima carry the product's rounding (slack_unit): a
// group counts with what its maximum is at least, a block reaches T with what its own is at most.  A thread takes the largest norm
// of its blocks for all of them.
struct Sums {
  float m, s, t;
};
__device__ __forceinline__ Sums join(const Sums& a, const Sums& b) {
  Sums r;
  r.m = fmaxf(a.m, b.m);
  if (r.m == minus_inf()) {  // nothing yet, or NaN
    r.s = a.s + b.s;
    r.t = a.t + b.t;
    return r;
  }
  const float da = fmaxf(a.m - r.m, kNoLogit), db = fmaxf(b.m - r.m, kNoLogit);
  const float fa = exp2f(da), fb = exp2f(db);
  r.s = a.s * fa + b.s * fb;
  r.t = fa * fmaf(a.s, da, a.t) + fb * fmaf(b.s, db, b.t);
  return r;
}

// Joined over lanes `step`, 2 step, ... 16 apart; both lanes of a pair join in the same order.
__device__ __forceinline__ Sums join_lanes(Sums sum, int step, int lane) {
  for (int o = step; o < 32; o <<= 1) {
    Sums other;
    other.m = __shfl_xor_sync(0xffffffffu, sum.m, o);
    other.s = __shfl_xor_sync(0xffffffffu, sum.s, o);
    other.t = __shfl_xor_sync(0xffffffffu, sum.t, o);
    sum = lane & o ? join(other, sum) : join(sum, other);
  }
  return sum;
}

// Few rows: 16 warps a row (WARPS), and where alternatives are wanted (TOP) the block goes on
// to them, without a launch and a way through memory.  1024 threads an SM: with the 79 registers that it would take, 4096 x 50257 x 768
// runs 270 us for 266 and 8192 x 32000 x 2048 754 for 745, but 600 x 128256 x 1024 163 for 167.
template <bool VEC, int WARPS, bool TOP>
__global__ void __launch_bounds__(WARPS * 32, WARPS > kRowWarps ? 2 : 4) lp_rows_kernel(const LpRows R, const LpTop T, int row_blocks) {
  constexpr int kGroups = 32 * WARPS, kWidth = WARPS > kRowWarps ? 1 : 8;  // groups of a row, and rows at most
  __shared__ Sums part[WARPS][kWidth];
  __shared__ double dots[WARPS];
  __shared__ float squares[WARPS];
  __shared__ float groups[kWidth][kGroups + 1], reached[kWidth];
  __shared__ int found[kWidth];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, width = kWidth == 1 ? 1 : R.width;
  if (!TOP) pdl_launch();  // else with the last of it
  pdl_wait();
  if (static_cast<int>(blockIdx.x) >= row_blocks) {
    const int64_t warps = static_cast<int64_t>(gridDim.x - row_blocks) * WARPS;
    for (int64_t r = static_cast<int64_t>(blockIdx.x - row_blocks) * WARPS + warp; r < R.rows; r += warps) {
      bool bad = false;
      const bool keep = !R.tokens.p || load_id(R.tokens, R.row0 + r, &bad) >= 0;
      for (int k = 0; k < R.copies; ++k)
        copy_row<VEC>(R.x + r * R.ld_x, R.x_copy + (r + k * R.rows) * R.ld_copy, R.dim, static_cast<int>(R.ld_copy), keep, lane);
    }
    return;
  }
  // The candidate blocks go to memory, or with TOP stay here.
  __shared__ TopBlock here[TOP ? kTopBlocks : 1];
  TopBlock* const list = TOP ? here : R.top_blocks;
  const int64_t list_rows = TOP ? 0 : kTopBlocks;
  if (blockIdx.x == 0 && threadIdx.x < 2) R.counters[threadIdx.x] = 0u;
  const int64_t base = static_cast<int64_t>(blockIdx.x) * width;
  const int shares = WARPS / width;
  const int64_t dot_row = base + warp / shares;
  bool bad = false;
  const int dot_target = R.tokens.p && dot_row < R.rows ? load_id(R.tokens, R.row0 + dot_row, &bad) : -1;
  Sums sum = {minus_inf(), 0.f, 0.f};
  const int64_t own_row = base + (lane & (width - 1));
  const int per_warp = 32 / width, stride = WARPS * per_warp;
  const int first_block = warp * per_warp + lane / width;
  float group[8];  // maxima of the blocks that are first, second, ... of eight
#pragma unroll
  for (int k = 0; k < 8; ++k) group[k] = minus_inf();
  Sums q[8];
  auto load = [&](int b) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int64_t at = static_cast<int64_t>(b + k * stride) * R.stats_ld + own_row;
      const bool in = own_row < R.rows && b + k * stride < R.n_blocks;
      const float2 ms = in ? R.stats[at] : make_float2(minus_inf(), 0.f);
      q[k] = Sums{ms.x, ms.y, in ? R.weighted[at] : 0.f};
    }
  };
  load(first_block);  // under way while the given token's logit is summed
  float norm = 0.f;  // largest of this thread's blocks
  if (R.k > 0) {
    // Shared among the lanes that have the same blocks, of other rows.
#pragma unroll 8
    for (int b = first_block + (lane & (width - 1)) * stride; b < R.n_blocks; b += width * stride)
      norm = fmaxf(norm, block_norm(R.norms, R.stats_shift, b));
    for (int o = 1; o < width; o <<= 1) norm = fmaxf(norm, __shfl_xor_sync(0xffffffffu, norm, o));
  }
  if (dot_row < R.rows && (dot_target >= 0 || R.k > 0)) {
    const uint16_t* x = R.x + dot_row * R.ld_x;
    float sq;
    const double d = warp_dot(x, dot_target >= 0 ? R.w + dot_target * R.ld_w : x, R.dim, warp % shares, shares, lane, &sq);
    if (lane == 0) {
      dots[warp] = d;
      squares[warp] = sq;
    }
  }
  if (own_row < R.rows) {
    for (int b = first_block; b < R.n_blocks; b += 8 * stride) {
      if (b != first_block) load(b);
#pragma unroll
      for (int k = 0; k < 8; ++k) group[k] = fmaxf(group[k], q[k].m);
      // The eight against their common maximum.
      Sums eight = {q[0].m, 0.f, 0.f};
#pragma unroll
      for (int k = 1; k < 8; ++k) eight.m = fmaxf(eight.m, q[k].m);
      const float ref = eight.m == minus_inf() ? 0.f : eight.m;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float d = fmaxf(q[k].m - ref, kNoLogit), f = exp2f(d);
        eight.s += f * q[k].s;
        eight.t += f * fmaf(q[k].s, d, q[k].t);
      }
      sum = join(sum, eight);
    }
  }
  sum = join_lanes(sum, width, lane);
  if (lane < width) part[warp][lane] = sum;
  float unit = 0.f, slack = 0.f;
  if (R.k > 0) {
    __syncthreads();  // squares
    for (int i = 0; i < shares; ++i) unit += squares[(lane & (width - 1)) * shares + i];
    unit = slack_unit(unit, R.logit_scale_log2, R.steps);
    slack = logit_slack(unit, norm);
    // Eight, four or one group of this thread: as many of a row as the block has threads.
#pragma unroll
    for (int o = 4; o > 0; o >>= 1)
      if (o >= width)
#pragma unroll
        for (int k = 0; k < o; ++k) group[k] = fmaxf(group[k], group[k + o]);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < kWidth && k < width) groups[lane & (width - 1)][(first_block * width + k)] = group[k] - slack;
    if (threadIdx.x < kWidth) found[threadIdx.x] = 0;
  }
  __syncthreads();
  if (R.k > 0) {
    if (warp < width) {
      float g[kGroups / 32];
#pragma unroll
      for (int i = 0; i < kGroups / 32; ++i) g[i] = groups[warp][lane + 32 * i];
      const float at = reached_by<kGroups / 32>(g, R.k);
      if (lane == 0) reached[warp] = at;
    }
    __syncthreads();
    if (own_row < R.rows) {
      const float from = reached[lane & (width - 1)];
      for (int b = first_block; b < R.n_blocks; b += 8 * stride) {
        float m[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          m[k] = b + k * stride < R.n_blocks ? R.stats[static_cast<int64_t>(b + k * stride) * R.stats_ld + own_row].x : minus_inf();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (b + k * stride >= R.n_blocks || m[k] + slack < from) continue;
          const int at = atomicAdd(&found[lane & (width - 1)], 1);
          if (at < kTopBlocks) list[own_row * list_rows + at] = TopBlock{b + k * stride, m[k], slack};
        }
      }
    }
    __syncthreads();
  }
  const int64_t r = base + lane;
  __shared__ LpRow info;
  auto finish = [&](const Sums& all) {
    const int64_t i = R.row0 + r;
    const int t = R.tokens.p ? load_id(R.tokens, i, &bad) : -1;
    if (bad) atomicCAS(R.err, 0, kErrBadIndex);
    LpRow o = {};
    if (R.k > 0) {
      o.reached = reached[lane];
      o.unit = unit;  // warp 0's lanes below `width` have their own rows
      o.blocks = found[lane];
    }
    o.target = t;
    o.scored = !R.tokens.p || t >= 0;
    float lse = 0.f, entropy = 0.f;
    if (o.scored) {
      float own = 0.f, dz = kNoLogit;
      if (t >= 0) {
        double z = 0.0;
        for (int k = 0; k < shares; ++k) z += dots[lane * shares + k];
        dz = static_cast<float>(z * R.logit_scale_log2 - all.m);
        own = exp2f(dz);
      }
      const float whole = all.s + own;
      o.top = all.m;
      o.log_sum = log2f(whole);
      lse = kLn2 * (all.m + o.log_sum);
      if (own > all.s) {
        o.logprob = -log1pf(all.s / own);
        entropy = -o.logprob - kLn2 * fmaf(-all.s, dz, all.t) / whole;
      } else {
        o.logprob = t >= 0 ? kLn2 * (dz - o.log_sum) : 0.f;
        entropy = kLn2 * (o.log_sum - fmaf(own, fmaxf(dz, kNoLogit), all.t) / whole);
      }
      // The rounding of M may leave the entropy of a nearly certain row that much below 0.  NaN stays.
      if (entropy < 0.f) entropy = 0.f;
      const float g = R.dlogprobs ? R.dlogprobs[i] : 0.f, h = R.dentropy ? R.dentropy[i] : 0.f;
      o.a = fmaf(h, entropy, g);
      o.b = kLn2 * h;
      const float p = own / whole;
      o.target_dz = g * (all.s / whole);
      // Of a token with no probability p ln p is 0.
      if (h != 0.f) o.target_dz -= p > 0.f ? h * p * (o.logprob + entropy) : 0.f;
      if (g == 0.f && h == 0.f) o.a = o.b = o.target_dz = 0.f;
    }
    if (R.logprobs) R.logprobs[i] = o.logprob;
    if (R.lse) R.lse[i] = lse;
    if (R.entropy) R.entropy[i] = entropy;
    if (TOP) info = o;
    R.out[r] = o;
  };
  if (warp == 0) {
    Sums all = {minus_inf(), 0.f, 0.f};
    for (int w = lane / width; w < WARPS; w += 32 / width) all = join(all, part[w][lane & (width - 1)]);
    all = join_lanes(all, width, lane);
    if (lane < width && r < R.rows) finish(all);
  }
  if constexpr (TOP) {
    __shared__ TopShared S;
    __syncthreads();
    const LpRow o = info;
    top_of_row<WARPS>(T, base, o, here, S);
  }
}

// ------------------------------------------------------------------- d logits
//   dz_v = g ([v = t] - p_v) - h p_v (ln p_v + H) = g [v = t] - p_v (a + b log2 p_v)
// with a = g + h H and b = h ln 2; the given token's comes from the row pass.
// As ce_dlogits_kernel, a read and a write of two bytes an entry.
template <bool LO>
__global__ void __launch_bounds__(kDlThreads) lp_dlogits_kernel(uint16_t* block, int64_t ld, int vocab, int stats_shift,
                                                                const float2* stats, int64_t stats_ld,
                                                                const LpRow* row_info, int64_t lo_rows) {
  pdl_launch();
  pdl_wait();
  const int64_t row = blockIdx.y;
  uint16_t* p = block + row * ld;
  const LpRow R = row_info[row];
  const int chunk = blockIdx.x, c0 = chunk * kDlCols + threadIdx.x * 8;
  const Logs L = load_logs(p, vocab, stats_shift, stats + row, stats_ld, chunk);
  const bool live = R.a != 0.f || R.b != 0.f || R.target_dz != 0.f;  // else zeros, whatever the row's logits are
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int c = c0 + k * kDlThreads * 8;
    if (c >= vocab) continue;
    const float top = (L.m[k] - R.top) - R.log_sum;
    const uint32_t w[4] = {L.q[k].x, L.q[k].y, L.q[k].z, L.q[k].w};
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = static_cast<float>(w[j] & 0xffffu);
      v[2 * j + 1] = static_cast<float>(w[j] >> 16);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float log_p = fmaf(v[j], -1.f / kCeLogUnits, top);
      v[j] = -ex2_approx(log_p) * fmaf(R.b, fmaxf(log_p, kNoLogit), R.a);
      if (c + j == R.target) v[j] = R.target_dz;
      if (!live) v[j] = 0.f;
    }
    *reinterpret_cast<uint4*>(p + c) =
        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    if (LO)
      *reinterpret_cast<uint4*>(p + lo_rows * ld + c) =
          make_uint4(pack_bf16x2_remainder(v[0], v[1]), pack_bf16x2_remainder(v[2], v[3]),
                     pack_bf16x2_remainder(v[4], v[5]), pack_bf16x2_remainder(v[6], v[7]));
  }
}

}  // namespace

cudaError_t launch_lp_rows(const LpRows& R, const LpTop& T, bool* top_done, cudaStream_t st) {
  const bool few = R.width == 1, top = few && T.k > 0;
  *top_done = top;
  if (T.k < 0 || T.k > kTopMost || T.k > T.vocab) return cudaErrorInvalidValue;
  const int warps = few ? 16 : kRowWarps;
  const int64_t row_blocks = (R.rows + R.width - 1) / R.width;
  const int64_t copy_blocks = R.x_copy ? (R.rows + warps - 1) / warps : 0;
  const bool vec = R.dim % 8 == 0 && R.ld_x % 8 == 0 && (reinterpret_cast<uintptr_t>(R.x) & 15u) == 0;
  auto kernel = top   ? (vec ? lp_rows_kernel<true, 16, true> : lp_rows_kernel<false, 16, true>)
                : few ? (vec ? lp_rows_kernel<true, 16, false> : lp_rows_kernel<false, 16, false>)
                      : (vec ? lp_rows_kernel<true, kRowWarps, false> : lp_rows_kernel<false, kRowWarps, false>);
  // Not before the product has ended: blocks that wait beside it cost it more than
  // the launch that they save (64 x 128256 x 4096 scores 177 us for 171, 600 x 128256 x 1024 126 for 114).
  return launch_ordered(false, kernel, dim3(static_cast<unsigned>(row_blocks + copy_blocks)), dim3(32 * warps), 0, st, R, T,
                        static_cast<int>(row_blocks));
}

cudaError_t launch_lp_top(const LpTop& T, cudaStream_t st) {
  if (T.k < 1 || T.k > kTopMost || T.k > T.vocab) return cudaErrorInvalidValue;
  return launch_after(lp_top_kernel<4>, dim3(static_cast<unsigned>(T.rows)), dim3(128), 0, st, T);
}

cudaError_t launch_lp_dlogits(uint16_t* block, int64_t ld, int64_t rows, int32_t vocab, int32_t stats_shift,
                              const float2* stats, int64_t stats_ld, const LpRow* row_info, int64_t lo_rows,
                              cudaStream_t st) {
  const int64_t per_launch = 65535;  // the grid's second dimension
  for (int64_t r = 0; r < rows; r += per_launch) {
    const int64_t n = rows - r < per_launch ? rows - r : per_launch;
    const dim3 grid(static_cast<unsigned>((vocab + kDlCols - 1) / kDlCols), static_cast<unsigned>(n));
    const cudaError_t e =
        launch_after(lo_rows > 0 ? lp_dlogits_kernel<true> : lp_dlogits_kernel<false>, grid, dim3(kDlThreads), 0, st,
                     block + r * ld, ld, static_cast<int>(vocab), static_cast<int>(stats_shift), stats + r, stats_ld, row_info + r, lo_rows);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace dmuon
