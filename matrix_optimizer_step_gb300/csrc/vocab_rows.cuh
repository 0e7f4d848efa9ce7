// Pieces of the row-wise kernels of the vocabulary operators (k_vocab_ce.cu,
// k_logprobs.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "ptx.cuh"
#include "vocab.h"

namespace dmuon {
namespace {

constexpr float kLn2 = 0.69314718055994531f;
constexpr int kRowWarps = 8;  // of the kernels that find the rows' sums

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

// This warp's share (of `shares`) of the dot product of two bf16 rows: a lane's
// part in fp32, their sum in 64 bits, the same in every lane.  `squares`, if wanted: the sum of
// the squares of a's share.
__device__ __forceinline__ double warp_dot(const uint16_t* a, const uint16_t* b, int n, int share, int shares, int lane,
                                           float* squares = nullptr) {
  float acc[4] = {0.f, 0.f, 0.f, 0.f}, sq = 0.f;
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
        if (squares) {
          sq = fmaf(__uint_as_float(u[i] << 16), __uint_as_float(u[i] << 16), sq);
          sq = fmaf(__uint_as_float(u[i] & 0xFFFF0000u), __uint_as_float(u[i] & 0xFFFF0000u), sq);
        }
      }
    }
  }
  for (int c = done + start; c < n; c += step) {
    acc[0] = fmaf(bf16_bits_to_f32(a[c]), bf16_bits_to_f32(b[c]), acc[0]);
    if (squares) sq = fmaf(bf16_bits_to_f32(a[c]), bf16_bits_to_f32(a[c]), sq);
  }
  if (squares) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
    *squares = sq;
  }
  return warp_sum(static_cast<double>((acc[0] + acc[1]) + (acc[2] + acc[3])));
}

// Adds the squares of this lane's row of a stage of W in shared memory (64 columns, 128-byte swizzle): its eight
// 16-byte pieces in an order in which eight lanes read all banks.
__device__ __forceinline__ void add_row_squares(const uint8_t* stage, int row, float (&s)[4]) {
  const uint4* p = reinterpret_cast<const uint4*>(stage + row * 128);
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const uint4 q = p[c ^ (row & 7)];
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float lo = __uint_as_float(u[i] << 16), hi = __uint_as_float(u[i] & 0xFFFF0000u);
      s[i] = fmaf(hi, hi, fmaf(lo, lo, s[i]));
    }
  }
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Norm of the row of w with the largest sum of squares.  Squares below fp32's range count for nothing, so none is taken below 1e-15.
__device__ __forceinline__ float largest_norm(float squares) { return sqrtf(fmaxf(squares, 1e-30f)); }

constexpr int kDlThreads = 256;
constexpr int kDlCols = kDlThreads * 8 * 4;

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A thread's part of the entries [chunk * kDlCols, + kDlCols) of one row: the
// logs (from p) and their blocks' maxima (from the row's pairs).
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

}  // namespace
}  // namespace dmuon
