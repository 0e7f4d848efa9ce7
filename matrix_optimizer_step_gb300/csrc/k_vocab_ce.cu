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

__device__ __forceinline__ float weight_of(const IdList& T, const float* weights, int64_t i, bool* bad) {
  return load_id(T, i, bad) < 0 ? 0.f : weights ? __ldg(weights + i) : 1.f;
}

// Sum over the block's threads in a fixed order; the result is in thread 0.
__device__ __forceinline__ double block_sum(double v, double* smem) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_down_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
  if (threadIdx.x == 0)
    for (unsigned w = 0; w < blockDim.x / 32; ++w) s += smem[w];
  return s;
}

// --------------------------------------------------------------- operand copy
// One warp per row; VEC: rows start on 16 bytes in both arrays and cols % 8 == 0.
template <bool VEC>
__global__ void ce_copy_kernel(const uint16_t* src, int64_t ld_src, uint16_t* dst, int64_t ld_dst, int64_t rows,
                               int cols, IdList targets, int has_targets, const float* weights, float* inv_norm) {
  if (inv_norm && blockIdx.x == 0) {
    __shared__ double smem[32];
    double s = 0.0;
    bool bad = false;
    for (int64_t i = threadIdx.x; i < rows; i += blockDim.x) s += weight_of(targets, weights, i, &bad);
    s = block_sum(s, smem);
    if (threadIdx.x == 0) *inv_norm = s != 0.0 ? static_cast<float>(1.0 / s) : 0.f;
  }
  if (!dst) return;  // only the norm is wanted
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); row < rows; row += warps) {
    bool bad = false;
    const bool keep = !has_targets || load_id(targets, row, &bad) >= 0;
    const uint16_t* s = src + row * ld_src;
    uint16_t* d = dst + row * ld_dst;
    if (VEC) {
      for (int c = lane * 8; c < cols; c += 256)
        *reinterpret_cast<uint4*>(d + c) = keep ? __ldg(reinterpret_cast<const uint4*>(s + c)) : make_uint4(0, 0, 0, 0);
    } else {
      for (int c = lane; c < ld_dst; c += 32) d[c] = keep && c < cols ? s[c] : uint16_t(0);
    }
  }
}

// ------------------------------------------------------------------- row sums
// Joins a row's (maximum, sum) pairs of all column blocks:
//   M = max m_b,  S = sum_b s_b 2^(m_b - M),  log2 sum = M + log2 S,
//   loss = ln2 ((M - z_t) + log2 S).
// A block takes 32 rows (one per lane, so a warp reads 32 neighbouring pairs)
// and its 32 warps take every 32nd column block; the warps' pairs are joined
// in a fixed order.  The last block of the last pass sums the losses.
constexpr int kRowWarps = 32;

__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
  const float top = fmaxf(m, m2);
  if (top == __int_as_float(0xff800000)) {  // nothing yet
    s += s2;
    return;
  }
  s = s * exp2f(m - top) + s2 * exp2f(m2 - top);
  m = top;
}

__global__ void __launch_bounds__(kRowWarps * 32) ce_rows_kernel(const CeRows R) {
  __shared__ float sm[kRowWarps][33], ss[kRowWarps][33];
  __shared__ double red[32];
  __shared__ uint32_t last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float m = __int_as_float(0xff800000), s = 0.f;
  if (r < R.rows) {
    const float2* p = R.stats + r;
    int b = warp;
    for (; b + 3 * kRowWarps < R.n_blocks; b += 4 * kRowWarps) {
      float2 q[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) q[k] = __ldg(p + static_cast<int64_t>(b + k * kRowWarps) * R.stats_ld);
#pragma unroll
      for (int k = 0; k < 4; ++k) join(m, s, q[k].x, q[k].y);
    }
    for (; b < R.n_blocks; b += kRowWarps) {
      const float2 q = __ldg(p + static_cast<int64_t>(b) * R.stats_ld);
      join(m, s, q.x, q.y);
    }
  }
  sm[warp][lane] = m;
  ss[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && r < R.rows) {
    const int warps = min(kRowWarps, R.n_blocks);
    for (int w = 1; w < warps; ++w) join(m, s, sm[w][lane], ss[w][lane]);
    const int64_t i = R.row0 + r;
    bool bad = false;
    const int t = load_id(R.targets, i, &bad);
    if (bad) atomicCAS(R.err, 0, kErrBadIndex);
    const float l2 = log2f(s), lse2 = m + l2;
    const float gap = t >= 0 ? (m - R.target_z[r]) + l2 : 0.f;  // log2(1 / p_target), octaves
    R.loss[i] = t >= 0 ? kLn2 * gap : 0.f;
    if (R.lse) R.lse[i] = t >= 0 ? kLn2 * lse2 : 0.f;
    if (R.out) {
      CeRow o;
      o.lse2 = lse2;
      o.coef = t < 0 ? 0.f : R.grad_scale * (R.weights ? R.weights[i] : 1.f) * (R.inv_norm ? *R.inv_norm : 1.f);
      o.target_dz = o.coef * expm1f(-kLn2 * gap);
      o.target = t;
      R.out[r] = o;
    }
  }
  if (!R.total) return;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(R.ticket, 1u) == gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  double sum = 0.0, norm = 0.0;
  bool bad = false;
  for (int64_t i = threadIdx.x; i < R.n; i += blockDim.x) {
    const float w = weight_of(R.targets, R.weights, i, &bad);
    if (w != 0.f) sum += static_cast<double>(w) * __ldcg(R.loss + i);
    norm += w;
  }
  sum = block_sum(sum, red);
  norm = block_sum(norm, red);
  if (threadIdx.x == 0) {
    *R.total = static_cast<float>(!R.mean ? sum : norm != 0.0 ? sum / norm : 0.0);
    *R.ticket = 0u;
  }
}

// ------------------------------------------------------------------- d logits
//   dz = coef (2^(m_b - lse - q / 1024) - [v = target])
// with the factor folded into the exponent.  Eight columns (16 bytes) a thread.
constexpr int kDlThreads = 256;
constexpr int kDlCols = kDlThreads * 8 * 4;

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__global__ void __launch_bounds__(kDlThreads) ce_dlogits_kernel(uint16_t* block, int64_t ld, int vocab,
                                                                const float2* stats, int64_t stats_ld,
                                                                const CeRow* row_info) {
  const int64_t row = blockIdx.y;
  const CeRow R = row_info[row];
  uint16_t* p = block + row * ld;
  const int c0 = blockIdx.x * kDlCols + threadIdx.x * 8;
  const bool counted = R.coef != 0.f;  // else zeros, whatever the row's logits are
  const float lift = log2f(fabsf(R.coef)) - R.lse2;
  const uint32_t sign = __float_as_uint(R.coef) & 0x80000000u;
  uint4 q[4];
  float m[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int c = c0 + k * kDlThreads * 8;
    if (c < vocab) {
      q[k] = *reinterpret_cast<const uint4*>(p + c);
      m[k] = __ldg(&stats[static_cast<int64_t>(c / kCeBlock) * stats_ld + row].x);
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int c = c0 + k * kDlThreads * 8;
    if (c >= vocab) continue;
    const float top = m[k] + lift;
    const uint32_t w[4] = {q[k].x, q[k].y, q[k].z, q[k].w};
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
    uint4 o;
    o.x = pack_bf16x2(v[0], v[1]);
    o.y = pack_bf16x2(v[2], v[3]);
    o.z = pack_bf16x2(v[4], v[5]);
    o.w = pack_bf16x2(v[6], v[7]);
    *reinterpret_cast<uint4*>(p + c) = o;
  }
}

// ------------------------------------------------------------- partial sums
__global__ void ce_finish_kernel(const float* part, int64_t ld_part, int64_t part_stride, int parts, void* out,
                                 int64_t ld_out, int out_bf16, int accumulate, int64_t rows, int cols) {
  const int64_t n = rows * cols;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t r = i / cols, c = i - r * cols;
    const float* p = part + r * ld_part + c;
    float s = p[0];
    for (int k = 1; k < parts; ++k) s += p[k * part_stride];
    if (out_bf16) {
      uint16_t* o = static_cast<uint16_t*>(out) + r * ld_out + c;
      if (accumulate) s += bf16_bits_to_f32(*o);
      *o = to_bf16_bits(s);
    } else {
      float* o = static_cast<float*>(out) + r * ld_out + c;
      *o = accumulate ? *o + s : s;
    }
  }
}

}  // namespace

cudaError_t launch_ce_copy(const uint16_t* src, int64_t ld_src, uint16_t* dst, int64_t ld_dst, int64_t rows,
                           int32_t cols, const IdList* targets, const float* weights, float* inv_norm,
                           cudaStream_t st) {
  const bool vec = cols % 8 == 0 && ld_src % 8 == 0 && ld_dst % 8 == 0 && cols == ld_dst &&
                   (reinterpret_cast<uintptr_t>(src) & 15u) == 0;
  const int64_t blocks = (rows + 7) / 8;
  const int grid = !dst ? 1 : static_cast<int>(blocks < 152 * 16 ? blocks : 152 * 16);
  const IdList ids = targets ? *targets : IdList{nullptr, 0, 0};
  if (vec)
    ce_copy_kernel<true><<<grid, 256, 0, st>>>(src, ld_src, dst, ld_dst, rows, cols, ids, targets != nullptr, weights, inv_norm);
  else
    ce_copy_kernel<false><<<grid, 256, 0, st>>>(src, ld_src, dst, ld_dst, rows, cols, ids, targets != nullptr, weights, inv_norm);
  return cudaGetLastError();
}

cudaError_t launch_ce_rows(const CeRows& R, cudaStream_t st) {
  ce_rows_kernel<<<static_cast<unsigned>((R.rows + 31) / 32), kRowWarps * 32, 0, st>>>(R);
  return cudaGetLastError();
}

cudaError_t launch_ce_dlogits(uint16_t* block, int64_t ld, int64_t rows, int32_t vocab, const float2* stats,
                              int64_t stats_ld, const CeRow* row_info, cudaStream_t st) {
  const int64_t per_launch = 65535;  // the grid's second dimension
  for (int64_t r = 0; r < rows; r += per_launch) {
    const int64_t n = rows - r < per_launch ? rows - r : per_launch;
    const dim3 grid(static_cast<unsigned>((vocab + kDlCols - 1) / kDlCols), static_cast<unsigned>(n));
    ce_dlogits_kernel<<<grid, kDlThreads, 0, st>>>(block + r * ld, ld, vocab, stats + r, stats_ld, row_info + r);
  }
  return cudaGetLastError();
}

cudaError_t launch_ce_finish(const float* part, int64_t ld_part, int64_t part_stride, int parts, void* out,
                             int64_t ld_out, int out_bf16, int accumulate, int64_t rows, int32_t cols,
                             cudaStream_t st) {
  const int64_t blocks = (rows * cols + 255) / 256;
  const int grid = static_cast<int>(blocks < 152 * 32 ? blocks : 152 * 32);
  ce_finish_kernel<<<grid, 256, 0, st>>>(part, ld_part, part_stride, parts, out, ld_out, out_bf16, accumulate, rows, cols);
  return cudaGetLastError();
}

}  // namespace dmuon
