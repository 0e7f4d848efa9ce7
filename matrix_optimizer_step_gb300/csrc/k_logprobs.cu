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

template <bool VEC>
__global__ void __launch_bounds__(kRowWarps * 32) lp_rows_kernel(const LpRows R, int row_blocks) {
  __shared__ Sums part[kRowWarps][8];
  __shared__ double dots[kRowWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, width = R.width;
  pdl_launch();
  pdl_wait();
  if (static_cast<int>(blockIdx.x) >= row_blocks) {
    const int64_t warps = static_cast<int64_t>(gridDim.x - row_blocks) * kRowWarps;
    for (int64_t r = static_cast<int64_t>(blockIdx.x - row_blocks) * kRowWarps + warp; r < R.rows; r += warps) {
      bool bad = false;
      const bool keep = !R.tokens.p || load_id(R.tokens, R.row0 + r, &bad) >= 0;
      for (int k = 0; k < R.copies; ++k)
        copy_row<VEC>(R.x + r * R.ld_x, R.x_copy + (r + k * R.rows) * R.ld_copy, R.dim, static_cast<int>(R.ld_copy), keep, lane);
    }
    return;
  }
  if (blockIdx.x == 0 && threadIdx.x < 2) R.counters[threadIdx.x] = 0u;
  const int64_t base = static_cast<int64_t>(blockIdx.x) * width;
  const int shares = kRowWarps / width;
  const int64_t dot_row = base + warp / shares;
  bool bad = false;
  const int dot_target = R.tokens.p && dot_row < R.rows ? load_id(R.tokens, R.row0 + dot_row, &bad) : -1;
  Sums sum = {minus_inf(), 0.f, 0.f};
  const int64_t own_row = base + (lane & (width - 1));
  const int per_warp = 32 / width, stride = kRowWarps * per_warp;
  if (own_row < R.rows) {
    for (int b = warp * per_warp + lane / width; b < R.n_blocks; b += 8 * stride) {
      Sums q[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int64_t at = static_cast<int64_t>(b + k * stride) * R.stats_ld + own_row;
        const bool in = b + k * stride < R.n_blocks;
        const float2 ms = in ? R.stats[at] : make_float2(minus_inf(), 0.f);
        q[k] = Sums{ms.x, ms.y, in ? R.weighted[at] : 0.f};
      }
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
  for (int o = width; o < 32; o <<= 1) {
    Sums other;
    other.m = __shfl_xor_sync(0xffffffffu, sum.m, o);
    other.s = __shfl_xor_sync(0xffffffffu, sum.s, o);
    other.t = __shfl_xor_sync(0xffffffffu, sum.t, o);
    // Both lanes join in the same order.
    sum = lane & o ? join(other, sum) : join(sum, other);
  }
  if (lane < width) part[warp][lane] = sum;
  if (dot_target >= 0) {
    const double d = warp_dot(R.x + dot_row * R.ld_x, R.w + dot_target * R.ld_w, R.dim, warp % shares, shares, lane);
    if (lane == 0) dots[warp] = d;
  }
  __syncthreads();
  const int64_t r = base + lane;
  if (warp != 0 || lane >= width || r >= R.rows) return;
  Sums all = part[0][lane];
#pragma unroll
  for (int w = 1; w < kRowWarps; ++w) all = join(all, part[w][lane]);
  const int64_t i = R.row0 + r;
  const int t = R.tokens.p ? load_id(R.tokens, i, &bad) : -1;
  if (bad) atomicCAS(R.err, 0, kErrBadIndex);
  LpRow o = {};
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
  R.out[r] = o;
}

// ---------------------------------------------------------- most likely entries
// The k largest logits of a row, equal ones by their numbers, in the order that
// sums of 64 bits give.  A block takes a row; the logs (16-bit distances to the
// blocks' maxima) bound each logit from both sides, and only entries that may be
// among the k are multiplied out again:
//   1. the k-th largest of the blocks' maxima: k entries lie there or above, so
//      blocks further below hold none;
//   2. of the others' entries the k-th largest lower bound;
//   3. entries whose upper bound reaches it, k and one or two more: their logits
//      as sums of exact products, in two floats each, put in order.
// What a bound allows for besides the log's own half step is the product's
// rounding, taken as 2^-9 octaves and 2^-14 of the row's maximum.
// More candidates than there is room for (equal or nearly equal logits) are taken a few
// blocks at a time; a row of zeros, all of whose logits are equal, is known without.
constexpr int kCandidates = 256;

// Lane i holds the i-th largest value so far; `least` is the k-th.
struct WarpTop {
  float q, least;
  __device__ __forceinline__ WarpTop() : q(minus_inf()), least(minus_inf()) {}
  // Takes each lane's value.
  __device__ __forceinline__ void add(float v, int k, int lane) {
    unsigned more = __ballot_sync(0xffffffffu, v > least);
    while (more) {
      const float c = __shfl_sync(0xffffffffu, v, __ffs(more) - 1);
      more &= more - 1;
      if (c <= least) continue;
      const int at = __popc(__ballot_sync(0xffffffffu, q >= c));
      const float above = __shfl_up_sync(0xffffffffu, q, 1);
      q = lane < at ? q : lane == at ? c : above;
      least = __shfl_sync(0xffffffffu, q, k - 1);
    }
  }
};

// The k-th largest of all warps' values.
template <int WARPS>
__device__ __forceinline__ float block_least(const WarpTop& mine, int k, float (&lists)[WARPS][kTopMost], float* result) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  lists[warp][lane] = mine.q;
  __syncthreads();
  if (warp == 0) {
    WarpTop all;
    for (int w = 0; w < WARPS; ++w) all.add(lane < k ? lists[w][lane] : minus_inf(), k, lane);
    if (lane == 0) *result = all.least;
  }
  __syncthreads();
  return *result;
}

// a + p without loss: the sum in a, what it rounds away in `lost` (Knuth's two-sum).
__device__ __forceinline__ void add_exactly(float& a, float& lost, float p) {
  const float s = a + p, back = s - a;
  lost += (a - (s - back)) + (p - back);
  a = s;
}

// Dot product of two bf16 rows to about 48 bits, the same in every lane.
__device__ __forceinline__ double warp_dot_exact(const uint16_t* a, const uint16_t* b, int n, int lane) {
  float sum[4] = {0.f, 0.f, 0.f, 0.f}, lost[4] = {0.f, 0.f, 0.f, 0.f};
  int done = 0;
  if (((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b)) & 15u) == 0) {
    done = n & ~7;
#pragma unroll 4
    for (int c = lane; c < n >> 3; c += 32) {
      const uint4 p = reinterpret_cast<const uint4*>(a)[c], q = reinterpret_cast<const uint4*>(b)[c];
      const uint32_t u[4] = {p.x, p.y, p.z, p.w}, v[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        add_exactly(sum[i], lost[i], __fmul_rn(__uint_as_float(u[i] << 16), __uint_as_float(v[i] << 16)));
        add_exactly(sum[i], lost[i], __fmul_rn(__uint_as_float(u[i] & 0xFFFF0000u), __uint_as_float(v[i] & 0xFFFF0000u)));
      }
    }
  }
  for (int c = done + lane; c < n; c += 32) add_exactly(sum[0], lost[0], __fmul_rn(bf16_bits_to_f32(a[c]), bf16_bits_to_f32(b[c])));
  double d = 0.0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    d += static_cast<double>(sum[i]);
    if (isfinite(sum[i])) d += static_cast<double>(lost[i]);  // of an infinite sum nothing else is known
  }
  return warp_sum(d);
}

template <int WARPS>
struct TopShared {
  float lists[WARPS][kTopMost];
  double z[kTopMost + kCandidates];
  int32_t id[kTopMost + kCandidates];
  double best_z[kTopMost];
  int32_t best_id[kTopMost];
  float least;
  int32_t count;
  int32_t nonzero;
};

template <int WARPS>
__global__ void __launch_bounds__(WARPS * 32) lp_top_kernel(const LpTop T) {
  __shared__ TopShared<WARPS> S;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch();
  pdl_wait();
  const int64_t row = blockIdx.x;
  const LpRow R = T.rows_in[row];
  const int k = T.k;
  auto put = [&](int rank, int32_t id, float logprob) {
    if (T.ids64)
      static_cast<long long*>(T.ids)[row * k + rank] = id;
    else
      static_cast<int*>(T.ids)[row * k + rank] = id;
    if (T.logprobs) T.logprobs[row * k + rank] = logprob;
  };
  // A row that is not scored, or has no distribution (NaN, or infinite logits).
  const bool ok = isfinite(R.top) && isfinite(R.log_sum);
  if (!R.scored || !ok) {
    if (threadIdx.x < k) put(threadIdx.x, -1, R.scored ? __int_as_float(0x7fc00000) : 0.f);
    return;
  }
  const float2* stats = T.stats + row;
  const uint16_t* logs = T.block + row * T.ld_block;
  const uint16_t* x = T.x + row * T.ld_x;
  const float slack = 0x1p-9f + fabsf(R.top) * 0x1p-14f;
  const int per_lane = (1 << T.stats_shift) / 32;
  auto logprob = [&](double z, int32_t id) {
    return id == R.target ? R.logprob : kLn2 * (static_cast<float>(z * T.logit_scale_log2 - R.top) - R.log_sum);
  };

  // Maxima of the blocks [b0, b1), those at or above `from`, each with a whole warp.
  auto for_blocks = [&](int b0, int b1, float from, auto&& take) {
    for (int b = b0 + warp * 32; b < b1; b += WARPS * 32) {
      const float m = b + lane < b1 ? stats[static_cast<int64_t>(b + lane) * T.stats_ld].x : minus_inf();
      unsigned more = __ballot_sync(0xffffffffu, b + lane < b1 && m >= from);
      while (more) {
        const int at = __ffs(more) - 1;
        more &= more - 1;
        take(b + at, __shfl_sync(0xffffffffu, m, at));
      }
    }
  };
  // Entries of block b, one a lane at a time: number and log; 65535: further off than logs go, or no logit.
  auto for_entries = [&](int b, auto&& take) {
    const int c0 = (b << T.stats_shift) + lane * per_lane;
    uint16_t q[4] = {65535, 65535, 65535, 65535};
    if (c0 < T.vocab) {
      if (per_lane == 4) {
        const uint2 w = *reinterpret_cast<const uint2*>(logs + c0);
        q[0] = static_cast<uint16_t>(w.x);
        q[1] = static_cast<uint16_t>(w.x >> 16);
        q[2] = static_cast<uint16_t>(w.y);
        q[3] = static_cast<uint16_t>(w.y >> 16);
      } else {
        q[0] = logs[c0];
      }
    }
    for (int j = 0; j < per_lane; ++j) take(c0 + j, q[j]);
  };

  WarpTop maxima;
  for (int b = warp * 32; b < T.n_blocks; b += WARPS * 32)
    maxima.add(b + lane < T.n_blocks ? stats[static_cast<int64_t>(b + lane) * T.stats_ld].x : minus_inf(), k, lane);
  const float from = block_least<WARPS>(maxima, k, S.lists, &S.least) - 2.f * slack;

  WarpTop lower;
  for_blocks(0, T.n_blocks, from, [&](int b, float m) {
    for_entries(b, [&](int c, uint16_t q) {
      const bool in = c < T.vocab && c != R.target && q != 65535;
      lower.add(in ? m - (static_cast<float>(q) + 0.5f) * (1.f / kCeLogUnits) - slack : minus_inf(), k, lane);
    });
  });
  __syncthreads();  // S.least has been read
  const float reach = block_least<WARPS>(lower, k, S.lists, &S.least);

  // Candidates of the blocks [b0, b1) into S.id; their number.
  auto collect = [&](int b0, int b1) {
    __syncthreads();
    if (threadIdx.x == 0) S.count = 0;
    __syncthreads();
    for_blocks(b0, b1, from, [&](int b, float m) {
      for_entries(b, [&](int c, uint16_t q) {
        const float upper = m - (static_cast<float>(q) - 0.5f) * (1.f / kCeLogUnits) + slack;
        if (c < T.vocab && c != R.target && upper >= reach) {
          const int at = atomicAdd(&S.count, 1);
          if (at < kCandidates) S.id[at] = c;
        }
      });
    });
    // The given token's log is not kept.
    if (threadIdx.x == 0 && R.target >= 0 && R.target >> T.stats_shift >= b0 && R.target >> T.stats_shift < b1) {
      const int at = atomicAdd(&S.count, 1);
      if (at < kCandidates) S.id[at] = R.target;
    }
    __syncthreads();
    return S.count;
  };
  auto multiply = [&](int n) {
    for (int i = warp; i < n; i += WARPS) {
      const double z = warp_dot_exact(x, T.w + S.id[i] * T.ld_w, T.dim, lane);
      if (lane == 0) S.z[i] = z;
    }
    __syncthreads();
  };
  // The first k of n in order: take(rank, z, id).
  auto in_order = [&](int n, auto&& take) {
    for (int i = threadIdx.x; i < n; i += WARPS * 32) {
      const double z = S.z[i];
      const int32_t id = S.id[i];
      int rank = 0;
      for (int j = 0; j < n; ++j) rank += S.z[j] > z || (S.z[j] == z && S.id[j] < id);
      if (rank < k) take(rank, z, id);
    }
  };

  const int found = collect(0, T.n_blocks);
  if (found <= kCandidates) {
    multiply(found);
    in_order(found, [&](int rank, double z, int32_t id) { put(rank, id, logprob(z, id)); });
    return;
  }
  if (threadIdx.x == 0) S.nonzero = 0;
  __syncthreads();
  bool any = false;
  for (int c = threadIdx.x; c < T.dim; c += WARPS * 32) any = any || (x[c] & 0x7fffu) != 0;
  if (any) S.nonzero = 1;
  __syncthreads();
  if (!S.nonzero) {
    if (threadIdx.x < k) put(threadIdx.x, threadIdx.x, logprob(0.0, threadIdx.x));
    return;
  }
  // A few blocks at a time, each joined with the best before it.
  const int step = kCandidates >> T.stats_shift;
  int best = 0;
  for (int b0 = 0; b0 < T.n_blocks; b0 += step) {
    const int n = collect(b0, min(b0 + step, T.n_blocks));
    if (n == 0) continue;
    multiply(n);
    if (threadIdx.x < best) {
      S.z[n + threadIdx.x] = S.best_z[threadIdx.x];
      S.id[n + threadIdx.x] = S.best_id[threadIdx.x];
    }
    __syncthreads();
    in_order(n + best, [&](int rank, double z, int32_t id) {
      S.best_z[rank] = z;
      S.best_id[rank] = id;
    });
    best = min(k, n + best);
  }
  __syncthreads();
  if (threadIdx.x < best) put(threadIdx.x, S.best_id[threadIdx.x], logprob(S.best_z[threadIdx.x], S.best_id[threadIdx.x]));
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

cudaError_t launch_lp_rows(const LpRows& R, cudaStream_t st) {
  const int64_t row_blocks = (R.rows + R.width - 1) / R.width;
  const int64_t copy_blocks = R.x_copy ? (R.rows + kRowWarps - 1) / kRowWarps : 0;
  const bool vec = R.dim % 8 == 0 && R.ld_x % 8 == 0 && (reinterpret_cast<uintptr_t>(R.x) & 15u) == 0;
  return launch_after(vec ? lp_rows_kernel<true> : lp_rows_kernel<false>, dim3(static_cast<unsigned>(row_blocks + copy_blocks)),
                      dim3(kRowWarps * 32), 0, st, R, static_cast<int>(row_blocks));
}

cudaError_t launch_lp_top(const LpTop& T, cudaStream_t st) {
  if (T.k < 1 || T.k > kTopMost || T.k > T.vocab) return cudaErrorInvalidValue;
  // Few rows: more warps for each, since only their latency counts.
  if (T.rows <= 304) return launch_after(lp_top_kernel<32>, dim3(static_cast<unsigned>(T.rows)), dim3(1024), 0, st, T);
  return launch_after(lp_top_kernel<8>, dim3(static_cast<unsigned>(T.rows)), dim3(256), 0, st, T);
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
