// Private types of the gradient operators (grads.cu, k_grads.cu): norms of many
// tensors and clipping.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace dmuon {

// Tensors of one launch, handed over as kernel arguments: no table in device memory
// that calls on different streams or captured graphs would share.
template <int CAP>
struct GradBatch {
  const void* in[CAP];
  void* out[CAP];           // scaling only
  int64_t numel[CAP];
  int32_t first[CAP + 1];   // first chunk of each tensor, from the batch's first on
  uint8_t in_bf16[CAP], out_bf16[CAP];
  int32_t n;
  int32_t chunk;            // bytes of a chunk of `in`, a multiple of 32
};
constexpr int kGradBatch = 512, kGradFew = 32;  // two sizes of argument lists

// What a norm call leaves, all device memory; null: not wanted.
struct GradNorm {
  double* partial;      // sum of squares of each chunk of the call
  double* squares;      // and of each tensor
  int32_t n_total;      // tensors of the call
  float* norms;         // each tensor's
  float* norm;          // of all
  float* coef;          // min(1, max_norm / (norm + 1e-6))
  float max_norm;
  uint32_t* ticket;     // zero before and after
};

// Sums of squares of a batch's chunks into G.partial + chunk0; with `whole` (one batch,
// kGradWhole chunks and kGradWholeTensors tensors at most) the last block joins them too.
constexpr int kGradWhole = 2048, kGradWholeTensors = kGradBatch;
template <int CAP>
cudaError_t launch_grad_squares(const GradBatch<CAP>& B, const GradNorm& G, int64_t chunk0, bool whole, cudaStream_t st);
// Joins them: tensors [tensor0, tensor0 + B.n) of the call; the last block of the call's
// last batch writes what concerns all.
template <int CAP>
cudaError_t launch_grad_join(const GradBatch<CAP>& B, const GradNorm& G, int64_t chunk0, int tensor0, cudaStream_t st);
// out = *coef * in.
template <int CAP>
cudaError_t launch_grad_scale(const GradBatch<CAP>& B, const float* coef, cudaStream_t st);

}  // namespace dmuon
