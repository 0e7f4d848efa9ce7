// Row-wise kernels of the cross entropy (the products are in
// k_vocab_gemm.cu): the operand copy, the per-row sums, the turn from
// fixed-point logs into d logits, and the join of partial products.  All are
// bound by HBM or by latency; none takes a noticeable share of a training
// call next to its three products.
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "ptx.cuh"
#include "vocab.h"

namespace dmuon {
namespace {

constexpr float kLn2 = 0.69314718055994531f;

// Sum over the block's threads in a fixed order; the result is in thread 0.
__device__ __forceinline__ double block_sum(double v, double* smem) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
  if (threadIdx.x == 0)
    for (unsigned w = 0; w < blockDim.x / 32; ++w) s += smem[w];
  return s;
}

__global__ void __launch_bounds__(1024) ce_norm_kernel(const CeNorm N) {
  __shared__ double red[32];
  pdl_launch();
  pdl_wait();
  const double sum = block_sum(norm_share(N, threadIdx.x, blockDim.x), red);
  if (threadIdx.x == 0) put_alpha(N, sum);
}

// --------------------------------------------------------------- operand copy
// One warp per row; VEC: source rows start on 16 bytes and cols % 8 == 0.
template <bool VEC>
__device__ __forceinline__ void copy_row(const uint16_t* s, uint16_t* d, int cols, int ld_dst, bool keep, int lane) {
  if (VEC) {
    for (int c0 = lane * 8; c0 < cols; c0 += 1024) {
      uint4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        v[k] = keep && c0 + 256 * k < cols ? *reinterpret_cast<const uint4*>(s + c0 + 256 * k) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (c0 + 256 * k < cols) *reinterpret_cast<uint4*>(d + c0 + 256 * k) = v[k];
    }
  } else {
    for (int c0 = lane; c0 < ld_dst; c0 += 256) {
      uint16_t v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = keep && c0 + 32 * k < cols ? s[c0 + 32 * k] : uint16_t(0);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (c0 + 32 * k < ld_dst) d[c0 + 32 * k] = v[k];
    }
  }
}

template <bool VEC>
__global__ void __launch_bounds__(256) ce_copy_kernel(const uint16_t* src, int64_t ld_src, uint16_t* dst, int64_t ld_dst,
                                                      int64_t rows, int cols, IdList targets) {
  pdl_launch();
  pdl_wait();
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); row < rows; row += warps) {
    bool bad = false;
    const bool keep = !targets.p || load_id(targets, row, &bad) >= 0;
    copy_row<VEC>(src + row * ld_src, dst + row * ld_dst, cols, static_cast<int>(ld_dst), keep, threadIdx.x & 31);
  }
}

// ------------------------------------------------------------------- d logits
//   dz = weight (2^(m_b - lse - q / 1024) - [v = target])
// with the weight folded into the exponent; the factor common to all rows stays
// out, so that without weights a target's dz is rounded next to 1, not next to
// 1 / (number of tokens).  Eight entries (16 bytes) a thread, four at a time:
// 7.0 TB/s read and written at 4096 x 50257.
// LO: also the rest of the rounding, for the rows below.
constexpr int kDlThreads = 256;
constexpr int kDlCols = kDlThreads * 8 * 4;

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A thread's part of the entries [chunk * kDlCols, + kDlCols) of one row: the
// logs (from p) and their blocks' maxima (from the row's pairs) ...
struct Logs {
  uint4 q[4];
  float m[4];
};
__device__ __forceinline__ Logs load_logs(const uint16_t* p, int vocab, int stats_shift, const float2* stats, int64_t stats_ld,
                                          int chunk) {
  Logs L;
  const int c0 = chunk * kDlCols + threadIdx.x * 8;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int c = c0 + k * kDlThreads * 8;
    if (c < vocab) {
      L.q[k] = *reinterpret_cast<const uint4*>(p + c);
      L.m[k] = stats[static_cast<int64_t>(c >> stats_shift) * stats_ld].x;
    }
  }
  return L;
}
// ... and their d logits, in place.
template <bool LO>
__device__ __forceinline__ void put_dlogits(const Logs& L, uint16_t* p, int64_t lo_offset, int vocab, const CeRow& R, int chunk) {
  const int c0 = chunk * kDlCols + threadIdx.x * 8;
  const bool counted = R.weight != 0.f;  // else zeros, whatever the row's logits are
  const float lift = log2f(fabsf(R.weight)) - R.lse2;
  const uint32_t sign = __float_as_uint(R.weight) & 0x80000000u;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int c = c0 + k * kDlThreads * 8;
    if (c >= vocab) continue;
    const float top = L.m[k] + lift;
    const uint32_t w[4] = {L.q[k].x, L.q[k].y, L.q[k].z, L.q[k].w};
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = static_cast<float>(w[j] & 0xffffu);
      v[2 * j + 1] = static_cast<float>(w[j] >> 16);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = __uint_as_float(__float_as_uint(ex2_approx(fmaf(v[j], -1.f / kCeLogUnits, top))) ^ sign);
      if (c + j == R.target) v[j] = R.target_dz;
      if (!counted) v[j] = 0.f;
    }
    *reinterpret_cast<uint4*>(p + c) =
        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    if (LO)
      *reinterpret_cast<uint4*>(p + lo_offset + c) =
          make_uint4(pack_bf16x2_remainder(v[0], v[1]), pack_bf16x2_remainder(v[2], v[3]),
                     pack_bf16x2_remainder(v[4], v[5]), pack_bf16x2_remainder(v[6], v[7]));
  }
}

template <bool LO>
__global__ void __launch_bounds__(kDlThreads) ce_dlogits_kernel(uint16_t* block, int64_t ld, int vocab, int stats_shift,
                                                                const float2* stats, int64_t stats_ld,
                                                                const CeRow* row_info, int64_t lo_rows) {
  pdl_launch();
  pdl_wait();
  const int64_t row = blockIdx.y;
  uint16_t* p = block + row * ld;
  const CeRow R = row_info[row];
  const Logs L = load_logs(p, vocab, stats_shift, stats + row, stats_ld, blockIdx.x);
  put_dlogits<LO>(L, p, lo_rows * ld, vocab, R, blockIdx.x);
}

// ------------------------------------------------------------------- row sums
// Joins a row's (maximum, sum) pairs of all vocabulary blocks:
//   M = max m_b,  S = sum_b s_b 2^(m_b - M),
// and from them the row's loss.  S leaves the target out: its logit is summed
// here (one dot product a row; the product's fp32 sums truncate, which shows
// where one logit is large), and with o = 2^(z_t - M)
//   loss = ln((S + o) / o),
// as log1p(S / o) where the target holds more than half of the sum, so that
// the loss of a token that is all but certain keeps its digits: nothing is
// subtracted from a sum, and z_t - M is taken in 64 bits, an octave count's
// rounding to 32 being up to 2e-6 of the loss.
//
// A block takes `width` rows (1; from 512 on 4, so that a warp reads whole
// 32-byte sectors of pairs; from 2048 on 8, so that the blocks stay one wave:
// 4096 x 50257 in 14 us, 21 with 4) and its 8 warps share their vocabulary blocks and their dot
// products; what is left is a chain of memory latencies, so each is taken by
// as many threads as there are.  All joins run in a fixed order.  The blocks
// after those copy dW's operand.
//
// DL, for few rows: `chunks` blocks take a row each, all of them find its sum
// (a few KB from L2 again) and turn their part of its logs into d logits; the
// first also does the rest.  That saves a launch and its latency.
constexpr int kRowWarps = 8;

__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
  const float top = fmaxf(m, m2);
  if (top == __int_as_float(0xff800000)) {  // nothing yet
    s += s2;
    return;
  }
  s = s * exp2f(m - top) + s2 * exp2f(m2 - top);
  m = top;
}

// Joined over lanes `step`, 2 step, ... 16 apart.
__device__ __forceinline__ void join_lanes(float& m, float& s, int step) {
  for (int o = step; o < 32; o <<= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
    join(m, s, m2, s2);
  }
}

// This warp's share (of `shares`) of the dot product of two bf16 rows: a lane's
// part in fp32, their sum in 64 bits, the same in every lane.
__device__ __forceinline__ double warp_dot(const uint16_t* a, const uint16_t* b, int n, int share, int shares, int lane) {
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  const int start = share * 32 + lane, step = shares * 32;
  int done = 0;
  if (((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b)) & 15u) == 0) {
    done = n & ~7;
#pragma unroll 4
    for (int c = start; c < n >> 3; c += step) {
      const uint4 p = reinterpret_cast<const uint4*>(a)[c], q = reinterpret_cast<const uint4*>(b)[c];
      const uint32_t u[4] = {p.x, p.y, p.z, p.w}, v[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[i] = fmaf(__uint_as_float(u[i] << 16), __uint_as_float(v[i] << 16), acc[i]);
        acc[i] = fmaf(__uint_as_float(u[i] & 0xFFFF0000u), __uint_as_float(v[i] & 0xFFFF0000u), acc[i]);
      }
    }
  }
  for (int c = done + start; c < n; c += step) acc[0] = fmaf(bf16_bits_to_f32(a[c]), bf16_bits_to_f32(b[c]), acc[0]);
  return warp_sum(static_cast<double>((acc[0] + acc[1]) + (acc[2] + acc[3])));
}

template <bool VEC, bool DL>
__global__ void __launch_bounds__(kRowWarps * 32) ce_rows_kernel(const CeRows R, int row_blocks, int chunks) {
  __shared__ float sm[kRowWarps][8], ss[kRowWarps][8];
  __shared__ double dots[kRowWarps];
  __shared__ double red[32];
  __shared__ uint32_t last;
  __shared__ CeRow info;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, width = R.width;
  pdl_launch();
  pdl_wait();
  const int copy0 = DL ? row_blocks * chunks : row_blocks;
  if (static_cast<int>(blockIdx.x) >= copy0) {
    const int64_t warps = static_cast<int64_t>(gridDim.x - copy0) * kRowWarps;
    for (int64_t r = static_cast<int64_t>(blockIdx.x - copy0) * kRowWarps + warp; r < R.rows; r += warps) {
      bool bad = false;
      const bool keep = load_id(R.targets, R.row0 + r, &bad) >= 0;
      for (int k = 0; k < R.copies; ++k)
        copy_row<VEC>(R.x + r * R.ld_x, R.x_copy + (r + k * R.rows) * R.ld_copy, R.dim, static_cast<int>(R.ld_copy), keep, lane);
    }
    return;
  }
  if (blockIdx.x == 0 && threadIdx.x < 2) R.counters[threadIdx.x] = 0u;
  const int row_block = DL ? static_cast<int>(blockIdx.x) / chunks : static_cast<int>(blockIdx.x);
  const int chunk = DL ? static_cast<int>(blockIdx.x) - row_block * chunks : 0;
  const int64_t base = static_cast<int64_t>(row_block) * width;
  const int shares = kRowWarps / width;
  const int64_t dot_row = base + warp / shares;
  bool bad = false;
  const int dot_target = dot_row < R.rows ? load_id(R.targets, R.row0 + dot_row, &bad) : -1;
  Logs logs;  // on their way while the row's sum is found
  if (DL) logs = load_logs(R.block + base * R.ld_block, R.vocab, R.stats_shift, R.stats + base, R.stats_ld, chunk);
  {
    const int64_t r = base + (lane & (width - 1));
    const int per_warp = 32 / width, stride = kRowWarps * per_warp;
    float m = __int_as_float(0xff800000), s = 0.f;
    if (r < R.rows) {
      const float2* p = R.stats + r;
      int b = warp * per_warp + lane / width;
      for (; b < R.n_blocks; b += 8 * stride) {
        float2 q[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          q[k] = b + k * stride < R.n_blocks ? p[static_cast<int64_t>(b + k * stride) * R.stats_ld]
                                             : make_float2(__int_as_float(0xff800000), 0.f);
        float top = m;
#pragma unroll
        for (int k = 0; k < 8; ++k) top = fmaxf(top, q[k].x);
        const float ref = top == __int_as_float(0xff800000) ? 0.f : top;  // nothing but -inf yet: all sums are 0 or NaN
        s *= exp2f(m - ref);
#pragma unroll
        for (int k = 0; k < 8; ++k) s += q[k].y * exp2f(q[k].x - ref);
        m = top;
      }
    }
    join_lanes(m, s, width);
    if (lane < width) {
      sm[warp][lane] = m;
      ss[warp][lane] = s;
    }
  }
  if (dot_target >= 0) {
    const double d = warp_dot(R.x + dot_row * R.ld_x, R.w + dot_target * R.ld_w, R.dim, warp % shares, shares, lane);
    if (lane == 0) dots[warp] = d;
  }
  __syncthreads();
  if (warp == 0) {
    const int64_t r = base + lane;
    double weighted = 0.0, weight_sum = 0.0;
    if (lane < width && r < R.rows) {
      float m = sm[0][lane], s = ss[0][lane];
#pragma unroll
      for (int w = 1; w < kRowWarps; ++w) join(m, s, sm[w][lane], ss[w][lane]);
      const int64_t i = R.row0 + r;
      const int t = load_id(R.targets, i, &bad);
      if (bad && chunk == 0) atomicCAS(R.err, 0, kErrBadIndex);
      const float weight = t < 0 ? 0.f : R.weights ? R.weights[i] : 1.f;
      float loss = 0.f, lse2 = m + log2f(s), share = 0.f;  // share: 1 - p_target
      if (t >= 0) {
        double z = 0.0;
        for (int k = 0; k < shares; ++k) z += dots[lane * shares + k];
        const float dz = static_cast<float>(z * R.logit_scale_log2 - m);
        const float own = exp2f(dz), sum = s + own, l2 = log2f(sum);
        loss = own > s ? log1pf(s / own) : kLn2 * (l2 - dz);
        lse2 = m + l2;
        share = s / sum;
      }
      if (R.loss && chunk == 0) R.loss[i] = loss;
      if (R.lse && chunk == 0) R.lse[i] = t >= 0 ? kLn2 * lse2 : 0.f;
      CeRow o;
      o.lse2 = lse2;
      o.weight = weight;
      o.target_dz = -weight * share;
      o.target = t;
      if (DL)
        info = o;
      else if (R.out)
        R.out[r] = o;
      if (weight != 0.f) weighted = static_cast<double>(weight) * loss;
      weight_sum = weight;
    }
    if (R.partial && chunk == 0) {
      for (int o = 1; o < width; o <<= 1) {
        weighted += __shfl_xor_sync(0xffffffffu, weighted, o);
        weight_sum += __shfl_xor_sync(0xffffffffu, weight_sum, o);
      }
      if (lane == 0) R.partial[R.row0 / width + row_block] = make_double2(weighted, weight_sum);
    }
  }
  if (DL) {
    __syncthreads();
    const CeRow o = info;
    put_dlogits<true>(logs, R.block + base * R.ld_block, R.lo_rows * R.ld_block, R.vocab, o, chunk);
  }
  if (!R.total.total || chunk != 0) return;
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(R.ticket, 1u) == static_cast<uint32_t>(row_blocks) - 1u;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  double2 sums = total_share(R.total, threadIdx.x, blockDim.x);
  sums.x = block_sum(sums.x, red);
  sums.y = block_sum(sums.y, red);
  if (threadIdx.x == 0) {
    put_total(R.total, sums);
    *R.ticket = 0u;
  }
}

// ------------------------------------------------------------- partial sums
// VEC columns a thread.  LANES threads share an output's partials (thread i takes
// every LANES-th) and add theirs in a fixed order: a few tokens' gradient is a
// few thousand outputs of dozens of partials each, and the time is latency
// (one token of width 2080: 11 us with one thread each, 4 with eight).
template <int VEC, int LANES>
__global__ void __launch_bounds__(256) ce_finish_kernel(const float* part, int64_t ld_part, int64_t part_stride, int parts,
                                                        int64_t fold, void* out, int64_t ld_out, int out_bf16,
                                                        int accumulate, const float* alpha, int64_t rows, int cols) {
  pdl_launch();
  pdl_wait();
  constexpr int kOutputs = 32 / LANES;  // of a warp, neighbours in neighbouring lanes
  const int lane = threadIdx.x & 31, sub = lane / kOutputs;
  const int64_t per_row = cols / VEC, total = rows * per_row;
  const float f = alpha ? *alpha : 1.f;
  const int n = fold > 0 ? 2 * parts : parts;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  for (int64_t i0 = (static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5)) * kOutputs; i0 < total;
       i0 += warps * kOutputs) {
    const int64_t i = i0 + lane % kOutputs;
    const bool live = i < total;
    const int64_t r = live ? i / per_row : 0, c = live ? (i - r * per_row) * VEC : 0;
    float s[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) s[j] = 0.f;
    const float* p = part + r * ld_part + c;
    for (int k0 = sub; k0 < n; k0 += 4 * LANES) {
      float4 q[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int k = k0 + u * LANES;
        q[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k >= n || !live) continue;
        const float* at = p + (fold > 0 ? (k >> 1) * part_stride + (k & 1) * fold * ld_part : k * part_stride);
        if (VEC == 4)
          q[u] = *reinterpret_cast<const float4*>(at);
        else
          q[u].x = *at;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        s[0] += q[u].x;
        if (VEC == 4) {
          s[1 % VEC] += q[u].y;
          s[2 % VEC] += q[u].z;
          s[3 % VEC] += q[u].w;
        }
      }
    }
#pragma unroll
    for (int o = kOutputs; o < 32; o <<= 1)
#pragma unroll
      for (int j = 0; j < VEC; ++j) s[j] += __shfl_xor_sync(0xffffffffu, s[j], o);
    if (sub != 0 || !live) continue;
#pragma unroll
    for (int j = 0; j < VEC; ++j) s[j] *= f;
    if (out_bf16) {
      uint16_t* o = static_cast<uint16_t*>(out) + r * ld_out + c;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        if (accumulate) s[j] += bf16_bits_to_f32(o[j]);
        if (VEC == 1) o[j] = to_bf16_bits(s[j]);
      }
      if (VEC == 4) *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(s[0], s[1 % VEC]), pack_bf16x2(s[2 % VEC], s[3 % VEC]));
    } else {
      float* o = static_cast<float*>(out) + r * ld_out + c;
#pragma unroll
      for (int j = 0; j < VEC; ++j) o[j] = accumulate ? o[j] + s[j] : s[j];
    }
  }
}

}  // namespace

cudaError_t launch_ce_copy(const uint16_t* src, int64_t ld_src, uint16_t* dst, int64_t ld_dst, int64_t rows,
                           int32_t cols, const IdList& targets, cudaStream_t st) {
  const bool vec = cols % 8 == 0 && ld_src % 8 == 0 && (reinterpret_cast<uintptr_t>(src) & 15u) == 0;
  const int64_t blocks = (rows + 7) / 8;
  const int grid = static_cast<int>(blocks < 152 * 16 ? blocks : 152 * 16);
  return launch_after(vec ? ce_copy_kernel<true> : ce_copy_kernel<false>, dim3(grid), dim3(256), 0, st, src, ld_src, dst,
                      ld_dst, rows, static_cast<int>(cols), targets);
}

int ce_rows_width(int64_t n) { return n >= 2048 ? 8 : n >= 512 ? 4 : 1; }
// Up to 128 rows it is even or saves a microsecond; at 214 x 60556 it cost seven.
bool ce_rows_make_dlogits(int64_t n) { return n <= 128; }

cudaError_t launch_ce_norm(const CeNorm& N, cudaStream_t st) {
  return launch_after(ce_norm_kernel, dim3(1), dim3(1024), 0, st, N);
}

cudaError_t launch_ce_rows(const CeRows& R, cudaStream_t st) {
  const int64_t row_blocks = (R.rows + R.width - 1) / R.width;
  const int64_t copy_blocks = R.x_copy ? (R.rows + kRowWarps - 1) / kRowWarps : 0;
  const bool vec = R.dim % 8 == 0 && R.ld_x % 8 == 0 && (reinterpret_cast<uintptr_t>(R.x) & 15u) == 0;
  const int chunks = R.block ? (R.vocab + kDlCols - 1) / kDlCols : 1;
  static_assert(kDlThreads == kRowWarps * 32, "one block size");
  auto kernel = R.block ? (vec ? ce_rows_kernel<true, true> : ce_rows_kernel<false, true>)
                        : (vec ? ce_rows_kernel<true, false> : ce_rows_kernel<false, false>);
  return launch_after(kernel, dim3(static_cast<unsigned>(row_blocks * chunks + copy_blocks)), dim3(kRowWarps * 32), 0, st, R,
                      static_cast<int>(row_blocks), chunks);
}

cudaError_t launch_ce_dlogits(uint16_t* block, int64_t ld, int64_t rows, int32_t vocab, int32_t stats_shift,
                              const float2* stats, int64_t stats_ld, const CeRow* row_info, int64_t lo_rows,
                              cudaStream_t st) {
  const int64_t per_launch = 65535;  // the grid's second dimension
  for (int64_t r = 0; r < rows; r += per_launch) {
    const int64_t n = rows - r < per_launch ? rows - r : per_launch;
    const dim3 grid(static_cast<unsigned>((vocab + kDlCols - 1) / kDlCols), static_cast<unsigned>(n));
    const cudaError_t e =
        launch_after(lo_rows > 0 ? ce_dlogits_kernel<true> : ce_dlogits_kernel<false>, grid, dim3(kDlThreads), 0, st,
                     block + r * ld, ld, static_cast<int>(vocab), static_cast<int>(stats_shift), stats + r, stats_ld, row_info + r, lo_rows);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_ce_finish(const float* part, int64_t ld_part, int64_t part_stride, int parts, int64_t fold,
                             void* out, int64_t ld_out, int out_bf16, int accumulate, const float* alpha,
                             int64_t rows, int32_t cols, cudaStream_t st) {
  // Partials have pitches of four; the output's rows must start on four bf16.
  const bool vec = cols % 4 == 0 && ld_out % 4 == 0 && (reinterpret_cast<uintptr_t>(out) & 7u) == 0;
  const bool shared = (fold > 0 ? 2 * parts : parts) >= 8;
  const int64_t blocks = (rows * (vec ? cols / 4 : cols) * (shared ? 8 : 1) + 255) / 256;
  const int grid = static_cast<int>(blocks < 152 * 32 ? blocks : 152 * 32);
  auto kernel = vec ? (shared ? ce_finish_kernel<4, 8> : ce_finish_kernel<4, 1>)
                    : (shared ? ce_finish_kernel<1, 8> : ce_finish_kernel<1, 1>);
  return launch_after(kernel, dim3(grid), dim3(256), 0, st, part, ld_part, part_stride, parts, fold, out, ld_out, out_bf16,
                      accumulate, alpha, rows, static_cast<int>(cols));
}

}  // namespace dmuon
