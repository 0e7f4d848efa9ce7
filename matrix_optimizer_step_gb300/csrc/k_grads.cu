// Norms of many gradients and their scaling.  Both are bound by HBM: a block
// takes a chunk of one tensor, and the tensors' pointers come as kernel
// arguments.
#include <cuda_runtime.h>
#include <stdint.h>

#include "grads.h"
#include "internal.h"
#include "ptx.cuh"
#include "vocab.h"

namespace dmuon {
namespace {

constexpr int kThreads = 256;

// Tensor of a chunk: the last whose first chunk is not behind it (tensors without
// elements have none and are skipped).
template <int CAP>
__device__ __forceinline__ int tensor_of(const GradBatch<CAP>& B, int chunk) {
  int lo = 0, hi = B.n;  // first[lo] <= chunk < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (B.first[mid] <= chunk)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Sum over the block in a fixed order, in every thread.
__device__ __forceinline__ double block_sum(double v, double* red) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
  for (int w = 0; w < kThreads / 32; ++w) s += red[w];
  return s;
}

// Whether this is the last of n blocks to get here; what the others wrote before is then visible.
__device__ __forceinline__ bool last_block(uint32_t* ticket, uint32_t n) {
  __shared__ bool last;
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(ticket, 1u) == n - 1u;
  }
  __syncthreads();
  if (last) __threadfence();
  return last;
}

// What concerns all tensors, from the sum of all squares; the ticket is handed back.
__device__ __forceinline__ void put_norm(const GradNorm& G, double squares) {
  const double norm = sqrt(squares), c = static_cast<double>(G.max_norm) / (norm + 1e-6);
  if (G.norm) *G.norm = static_cast<float>(norm);
  if (G.coef) *G.coef = c > 1.0 || isinf(G.max_norm) ? 1.f : static_cast<float>(c);  // NaN stays
  *G.ticket = 0u;
}

__device__ __forceinline__ void square(uint32_t pair, float scale, float& a, float& b) {
  const float lo = __uint_as_float(pair << 16) * scale, hi = __uint_as_float(pair & 0xFFFF0000u) * scale;
  a = fmaf(lo, lo, a);
  b = fmaf(hi, hi, b);
}

// This thread's share of the sum of (scale x)^2 over n elements; `bits` gathers all
// bits that are set.  The elements before the first 16-byte boundary and behind the
// last one go one by one.
template <bool BF16>
__device__ __forceinline__ float squares(const void* p, int n, float scale, uint32_t& bits) {
  constexpr int kSize = BF16 ? 2 : 4, kVec = 16 / kSize;
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  const int head = min(n, static_cast<int>(((16u - (at & 15u)) & 15u) / kSize));
  const int vectors = (n - head) / kVec, tail = head + vectors * kVec;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  auto one = [&](int i) {
    float v;
    if (BF16)
      v = bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
    else
      v = static_cast<const float*>(p)[i];
    bits |= __float_as_uint(v);
    v *= scale;
    s[0] = fmaf(v, v, s[0]);
  };
  if (static_cast<int>(threadIdx.x) < head) one(threadIdx.x);
  if (tail + static_cast<int>(threadIdx.x) < n) one(tail + threadIdx.x);
  const uint4* v = reinterpret_cast<const uint4*>(at + static_cast<uintptr_t>(head) * kSize);
  for (int i = threadIdx.x; i < vectors; i += 4 * kThreads) {
    uint4 q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) q[k] = i + k * kThreads < vectors ? v[i + k * kThreads] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t w[4] = {q[k].x, q[k].y, q[k].z, q[k].w};
      bits |= (w[0] | w[1]) | (w[2] | w[3]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (BF16) {
          square(w[j], scale, s[j], s[j ^ 1]);
        } else {
          const float x = __uint_as_float(w[j]) * scale;
          s[j] = fmaf(x, x, s[j]);
        }
      }
    }
  }
  return (s[0] + s[1]) + (s[2] + s[3]);
}

// Sum over the block of one fp32 value a thread, in a fixed order, in every thread.  (In 64 bits, of which an
// SM adds two a cycle, the blocks of a small call spent more time here than on their data.)
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  static_assert(kThreads == 256, "eight warps");
  return ((red[0] + red[1]) + (red[2] + red[3])) + ((red[4] + red[5]) + (red[6] + red[7]));
}

// A chunk's sum in fp32.  Where it leaves the range in which squares keep their
// digits (infinite, or below 2^-80 without all elements being zeros) the chunk is
// read again with a power of two that brings it back; the result is in 64 bits, so the call's
// sum neither overflows nor loses small tensors.
//
// WHOLE: few chunks, whose sums the last block joins, which saves a launch.
template <int CAP, bool WHOLE>
__global__ void __launch_bounds__(kThreads) grad_squares_kernel(const __grid_constant__ GradBatch<CAP> B, const GradNorm G, double* partial) {
  __shared__ float red[kThreads / 32];
  pdl_launch();
  pdl_wait();
  const int t = tensor_of(B, blockIdx.x);
  const bool bf16 = B.in_bf16[t] != 0;
  const int length = B.chunk >> (bf16 ? 1 : 2);
  const int64_t start = static_cast<int64_t>(blockIdx.x - B.first[t]) * length;
  const int n = static_cast<int>(min(static_cast<int64_t>(length), B.numel[t] - start));
  const void* p = static_cast<const char*>(B.in[t]) + start * (bf16 ? 2 : 4);
  uint32_t bits = 0;
  auto sum = [&](float scale) { return block_sum(bf16 ? squares<true>(p, n, scale, bits) : squares<false>(p, n, scale, bits), red); };
  const float plain = sum(1.f);
  double s = plain;
  const bool large = isinf(plain), small = plain < 0x1p-80f;
  if (large || (small && __syncthreads_or((bits & (bf16 ? 0x7fff7fffu : 0x7fffffffu)) != 0u)))
    s = large ? sum(0x1p-80f) * 0x1p160 : sum(0x1p100f) * 0x1p-200;
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
  if constexpr (WHOLE) {
    __shared__ double all[kGradWhole], of_tensor[kGradWholeTensors];
    __shared__ int first[kGradWholeTensors + 1];
    if (!last_block(G.ticket, gridDim.x)) return;
    for (int c = threadIdx.x; c < static_cast<int>(gridDim.x); c += kThreads) all[c] = __ldcg(partial + c);
    for (int i = threadIdx.x; i <= B.n; i += kThreads) first[i] = B.first[i];
    __syncthreads();
    // A thread a tensor of few chunks, a warp one of many.
    constexpr int kFew = 8;
    for (int i = threadIdx.x; i < B.n; i += kThreads) {
      const int c0 = first[i], c1 = first[i + 1];
      double q = 0.0;
      if (c1 - c0 <= kFew)
        for (int c = c0; c < c1; ++c) q += all[c];
      of_tensor[i] = q;
    }
    __syncthreads();
    for (int i = threadIdx.x >> 5; i < B.n; i += kThreads / 32) {
      const int c0 = first[i], c1 = first[i + 1];
      if (c1 - c0 <= kFew) continue;
      double q = 0.0;
      for (int c = c0 + (threadIdx.x & 31); c < c1; c += 32) q += all[c];
      q = warp_sum(q);
      if ((threadIdx.x & 31) == 0) of_tensor[i] = q;
    }
    __syncthreads();
    if (G.norms)
      for (int i = threadIdx.x; i < B.n; i += kThreads) G.norms[i] = static_cast<float>(sqrt(of_tensor[i]));
    if (threadIdx.x < 32) {
      double total = 0.0;
      for (int i = threadIdx.x; i < B.n; i += 32) total += of_tensor[i];
      total = warp_sum(total);
      if (threadIdx.x == 0) put_norm(G, total);
    }
  }
}

// A block a tensor; the last block of the call joins the tensors.
template <int CAP>
__global__ void __launch_bounds__(kThreads) grad_join_kernel(const __grid_constant__ GradBatch<CAP> B, const GradNorm G,
                                                             int64_t chunk0, int tensor0) {
  __shared__ double red[kThreads / 32];
  pdl_launch();
  pdl_wait();
  const int t = blockIdx.x;
  if (t < B.n) {
    double s = 0.0;
#pragma unroll 4
    for (int c = B.first[t] + threadIdx.x; c < B.first[t + 1]; c += kThreads) s += G.partial[chunk0 + c];
    s = block_sum(s, red);
    if (threadIdx.x == 0) {
      G.squares[tensor0 + t] = s;
      if (G.norms) G.norms[tensor0 + t] = static_cast<float>(sqrt(s));
    }
  }
  if (!last_block(G.ticket, static_cast<uint32_t>(max(G.n_total, 1)))) return;
  double s = 0.0;
  for (int i = threadIdx.x; i < G.n_total; i += kThreads) s += __ldcg(G.squares + i);
  s = block_sum(s, red);
  if (threadIdx.x == 0) put_norm(G, s);
}

template <bool IN_BF16, bool OUT_BF16>
__device__ __forceinline__ void scale_chunk(const void* in, void* out, int n, float f) {
  int done = 0;
  if (((reinterpret_cast<uintptr_t>(in) | reinterpret_cast<uintptr_t>(out)) & 15u) == 0) {
    done = n & ~7;
    for (int i = threadIdx.x; i < n >> 3; i += 2 * kThreads) {
      uint4 q[2][2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int at = i + k * kThreads;
        if (at >= n >> 3) continue;
        const uint4* p = static_cast<const uint4*>(in) + (IN_BF16 ? at : 2 * at);
        q[k][0] = p[0];
        if (!IN_BF16) q[k][1] = p[1];
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int at = i + k * kThreads;
        if (at >= n >> 3) continue;
        float v[8];
        if (IN_BF16) {
          const uint32_t w[4] = {q[k][0].x, q[k][0].y, q[k][0].z, q[k][0].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(w[j] << 16);
            v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
          }
        } else {
          const uint32_t w[8] = {q[k][0].x, q[k][0].y, q[k][0].z, q[k][0].w, q[k][1].x, q[k][1].y, q[k][1].z, q[k][1].w};
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= f;
        uint4* o = static_cast<uint4*>(out) + (OUT_BF16 ? at : 2 * at);
        if (OUT_BF16) {
          o[0] = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
        } else {
          o[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
          o[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
        }
      }
    }
  }
  for (int i = done + threadIdx.x; i < n; i += kThreads) {
    const float v = f * (IN_BF16 ? bf16_bits_to_f32(static_cast<const uint16_t*>(in)[i]) : static_cast<const float*>(in)[i]);
    if (OUT_BF16)
      static_cast<uint16_t*>(out)[i] = to_bf16_bits(v);
    else
      static_cast<float*>(out)[i] = v;
  }
}

// Chunks in falling order: after a norm the last ones read are still in L2.  A
// factor of 1 leaves what is scaled in place as it is.
template <int CAP>
__global__ void __launch_bounds__(kThreads) grad_scale_kernel(const __grid_constant__ GradBatch<CAP> B, const float* coef) {
  pdl_launch();
  pdl_wait();
  const float f = *coef;
  const int c = static_cast<int>(gridDim.x - 1u - blockIdx.x);
  const int t = tensor_of(B, c);
  if (f == 1.f && B.in[t] == B.out[t]) return;
  const bool in16 = B.in_bf16[t] != 0, out16 = B.out_bf16[t] != 0;
  const int length = B.chunk >> (in16 ? 1 : 2);
  const int64_t start = static_cast<int64_t>(c - B.first[t]) * length;
  const int n = static_cast<int>(min(static_cast<int64_t>(length), B.numel[t] - start));
  const void* in = static_cast<const char*>(B.in[t]) + start * (in16 ? 2 : 4);
  void* out = static_cast<char*>(B.out[t]) + start * (out16 ? 2 : 4);
  if (in16)
    out16 ? scale_chunk<true, true>(in, out, n, f) : scale_chunk<true, false>(in, out, n, f);
  else
    out16 ? scale_chunk<false, true>(in, out, n, f) : scale_chunk<false, false>(in, out, n, f);
}

}  // namespace

template <int CAP>
cudaError_t launch_grad_squares(const GradBatch<CAP>& B, const GradNorm& G, int64_t chunk0, bool whole, cudaStream_t st) {
  if (whole && B.first[B.n] > kGradWhole) return cudaErrorInvalidValue;
  return launch_after(whole ? grad_squares_kernel<CAP, true> : grad_squares_kernel<CAP, false>, dim3(static_cast<unsigned>(B.first[B.n])),
                      dim3(kThreads), 0, st, B, G, G.partial + chunk0);
}

template <int CAP>
cudaError_t launch_grad_join(const GradBatch<CAP>& B, const GradNorm& G, int64_t chunk0, int tensor0, cudaStream_t st) {
  return launch_after(grad_join_kernel<CAP>, dim3(static_cast<unsigned>(B.n > 0 ? B.n : 1)), dim3(kThreads), 0, st, B, G, chunk0, tensor0);
}

template <int CAP>
cudaError_t launch_grad_scale(const GradBatch<CAP>& B, const float* coef, cudaStream_t st) {
  return launch_after(grad_scale_kernel<CAP>, dim3(static_cast<unsigned>(B.first[B.n])), dim3(kThreads), 0, st, B, coef);
}

template cudaError_t launch_grad_squares(const GradBatch<kGradFew>&, const GradNorm&, int64_t, bool, cudaStream_t);
template cudaError_t launch_grad_squares(const GradBatch<kGradBatch>&, const GradNorm&, int64_t, bool, cudaStream_t);
template cudaError_t launch_grad_join(const GradBatch<kGradFew>&, const GradNorm&, int64_t, int, cudaStream_t);
template cudaError_t launch_grad_join(const GradBatch<kGradBatch>&, const GradNorm&, int64_t, int, cudaStream_t);
template cudaError_t launch_grad_scale(const GradBatch<kGradFew>&, const float*, cudaStream_t);
template cudaError_t launch_grad_scale(const GradBatch<kGradBatch>&, const float*, cudaStream_t);

}  // namespace dmuon
