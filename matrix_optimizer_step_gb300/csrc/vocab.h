// Private types of the vocabulary operators (vocab.cu, k_vocab_gemm.cu,
// k_vocab_ce.cu, k_embed.cu): softmax cross entropy over a head matrix and
// embedding lookup, each with its gradient.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace dmuon {

// Token ids and targets: 32- or 64-bit, as the caller has them.
struct IdList {
  const void* p;
  int32_t is64;
  int32_t vocab;
};

// Columns that one epilogue warp reduces: the softmax statistics of a row
// come as one (maximum, sum) pair for each block of this many columns.
constexpr int kCeBlock = 128;

// Fixed-point logs: a logit of the block is kept as the 16-bit distance to
// the block's maximum in units of 2^-10 octaves, cut off at 64 octaves.
constexpr float kCeLogUnits = 1024.f;

// One product D (M x N) = A (M x K) B (K x N) of the cross entropy, on CTA
// pairs with 256 x 256 tiles.
enum VocabGemmMode : int {
  kVgLogits = 0,  // softmax statistics of each row, optionally the logits' fixed-point logs
  kVgBf16 = 1,    // D as bf16
  kVgF32 = 2,     // D as fp32, stored or added; with splits > 1 one partial D for each split
};

struct VocabGemm {
  CUtensorMap map_a, map_b, map_out;
  int32_t M, N, K;
  int32_t tiles_m, tiles_n, splits;
  int32_t kb_total;      // 64-deep k-blocks of K
  int32_t group_m;       // row tiles that are walked together (operand reuse in L2)
  int32_t add;           // kVgF32: add to what `out` holds
  int* err;
  // kVgLogits
  float logit_scale_log2;  // logit scale times log2(e)
  int32_t store_logs;
  float2* stats;           // [column block][row]: maximum and sum of 2^(z - maximum), z in octaves
  int64_t stats_ld;
  float* target_z;         // [row]: the target's z
  IdList targets;          // of row 0 of this product
};

cudaError_t launch_vocab_gemm(int mode, bool a_mn, bool b_mn, const VocabGemm& G, int n_pairs, cudaStream_t st);
int vocab_gemm_max_pairs();

// ---- k_vocab_ce.cu
// Copy of `rows` x `cols` bf16 values into rows of pitch ld_dst (the columns
// up to ld_dst are zeros).  With targets, rows whose target is not counted
// become zeros; with norm, block 0 also writes 1 / (sum of the counted weights).
cudaError_t launch_ce_copy(const uint16_t* src, int64_t ld_src, uint16_t* dst, int64_t ld_dst, int64_t rows,
                           int32_t cols, const IdList* targets, const float* weights, float* inv_norm,
                           cudaStream_t st);

// Per-row outcome of the statistics, as the gradient pass reads it.
struct CeRow {
  float lse2;       // log2 of the softmax's sum, in octaves
  float coef;       // factor of (p - onehot) in d logits, 0 for a row that is not counted
  float target_dz;  // coef * (p_target - 1)
  int32_t target;   // -1: none
};

struct CeRows {
  const float2* stats;
  int64_t stats_ld;
  int32_t n_blocks;        // column blocks
  int64_t row0, rows;      // rows of this pass, as part of n
  int64_t n;
  const float* target_z;   // of row row0
  IdList targets;          // of row 0
  const float* weights;    // of row 0, or null
  const float* inv_norm;   // or null: 1
  float grad_scale;        // upstream factor times logit scale
  CeRow* out;              // of row row0, or null
  float* loss;             // of row 0, never null
  float* lse;              // of row 0, or null
  // The last pass sums the losses: total = sum(weight * loss) [/ sum(weight)].
  float* total;            // null: not in this pass
  int32_t mean;
  uint32_t* ticket;        // zero before and after
  int* err;
};
cudaError_t launch_ce_rows(const CeRows& R, cudaStream_t st);

// Fixed-point logs -> bf16 d logits, in place.
cudaError_t launch_ce_dlogits(uint16_t* block, int64_t ld, int64_t rows, int32_t vocab, const float2* stats,
                              int64_t stats_ld, const CeRow* row_info, cudaStream_t st);

// out (rows x cols, pitch ld_out) = sum over `parts` partials (pitch ld_part,
// part_stride elements apart) [+ out].
cudaError_t launch_ce_finish(const float* part, int64_t ld_part, int64_t part_stride, int parts, void* out,
                             int64_t ld_out, int out_bf16, int accumulate, int64_t rows, int32_t cols,
                             cudaStream_t st);

// ---- k_embed.cu
struct EmbedForward {
  IdList ids;
  int64_t n;
  const void* table;
  int64_t ld_table;
  int32_t table_bf16;
  void* out;
  int64_t ld_out;
  int32_t out_bf16;
  int32_t dim;
  float scale;
  int* err;
};
cudaError_t launch_embed_forward(const EmbedForward& E, cudaStream_t st);

struct EmbedBackward {
  IdList ids;
  int64_t n;
  const void* dout;
  int64_t ld_dout;
  int32_t dout_bf16;
  void* dtable;
  int64_t ld_dtable;
  int32_t dtable_bf16;
  int32_t accumulate;
  int32_t dim;
  float scale;
  int* err;
  // workspace (embed_backward_ws)
  uint32_t* key[2];
  uint32_t* pos[2];
  uint32_t* hist;
  float* partial;
};
// Sorted positions that one block of the summing kernel takes.
constexpr int kEmbedRun = 64;
struct EmbedWs {
  size_t key[2], pos[2], hist, partial, bytes;
};
EmbedWs embed_backward_ws(int64_t n, int32_t dim);
// Enqueues the launches; *launches counts them.
cudaError_t launch_embed_backward(const EmbedBackward& E, int* launches, cudaStream_t st);

// id of entry i, or -1 where there is none (negative: not counted; past the
// vocabulary: *bad is set).
__device__ __forceinline__ int32_t load_id(const IdList& L, int64_t i, bool* bad) {
  const int64_t v = L.is64 ? __ldg(static_cast<const long long*>(L.p) + i)
                           : static_cast<int64_t>(__ldg(static_cast<const int*>(L.p) + i));
  if (v < 0) return -1;
  if (v >= L.vocab) {
    *bad = true;
    return -1;
  }
  return static_cast<int32_t>(v);
}

}  // namespace dmuon
