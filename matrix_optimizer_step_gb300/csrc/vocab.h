// Private types of the vocabulary operators (vocab.cu, k_vocab_gemm.cu,
// k_vocab_ce.cu, k_embed.cu): softmax cross entropy over a head matrix and
// embedding lookup, each with its gradient.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace dmuon {

// Launch that may begin while the kernel before it on the stream ends: every
// kernel of the vocabulary operators calls pdl_wait before it touches memory,
// so only its set-up (barriers, TMEM, launch latency) runs early.
template <class... P, class... A>
inline cudaError_t launch_after(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// One lane of a warp whose lanes are all here, the same one every time.  The
// roles that one thread plays begin with it rather than with `lane == 0`: the
// compiler then knows that a single lane goes on and hands descriptors, tensor
// maps and barriers to the asynchronous instructions as they are.  Behind
// `lane == 0` the MMA issuer fell behind whenever an epilogue warp computed on
// its scheduler: the logits of 4096 x 50257 x 512 took 142 us instead of 113,
// of 8192 x 128256 x 4096 4.9 ms instead of 4.7; the thin product of one row and
// 128256 x 4096 weights 162 us instead of 155.
__device__ __forceinline__ bool elect_one() {
  uint32_t elected;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(elected));
  return elected != 0;
}

// All earlier work on the stream is done and visible.  What is read after it may
// have been written while this block was already resident (by the kernel before,
// ours or the caller's), so the kernels read with ordinary loads, which are
// ordered after the wait: the read-only path (ld.global.nc, __ldg) is for memory
// that nothing writes during a kernel's life, and its lines may be old ones.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// From L2, and not before the barrier or fence that it follows: what other blocks wrote.
__device__ __forceinline__ uint32_t load_l2(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.global.cg.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ double2 load_l2(const double2* p) {
  double2 v;
  asm volatile("ld.global.cg.v2.f64 {%0, %1}, [%2];" : "=d"(v.x), "=d"(v.y) : "l"(p) : "memory");
  return v;
}
// The next kernel's blocks may take free room from here on.
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Token ids and targets: 32- or 64-bit, as the caller has them.
struct IdList {
  const void* p;
  int32_t is64;
  int32_t vocab;
};

// id of entry i, or -1 where there is none (negative: not counted; past the
// vocabulary: *bad is set).
__device__ __forceinline__ int32_t load_id(const IdList& L, int64_t i, bool* bad) {
  const int64_t v = L.is64 ? static_cast<const long long*>(L.p)[i] : static_cast<int64_t>(static_cast<const int*>(L.p)[i]);
  if (v < 0) return -1;
  if (v >= L.vocab) {
    *bad = true;
    return -1;
  }
  return static_cast<int32_t>(v);
}

// Softmax statistics of a row come as one (maximum, sum) pair for each block
// of this many vocabulary entries: what one epilogue warp reduces.
constexpr int kCeBlock = 128;     // 256 x 256 tiles (k_vocab_gemm.cu)
constexpr int kCeThinBlock = 32;  // few tokens (k_vocab_thin.cu)
constexpr int kCeShift = 7, kCeThinShift = 5;
static_assert(kCeBlock == 1 << kCeShift && kCeThinBlock == 1 << kCeThinShift, "block shifts");

// Fixed-point logs: a logit is kept as the 16-bit distance to its block's
// maximum in units of 2^-10 octaves, cut off at 64 octaves.
constexpr float kCeLogUnits = 1024.f;

// Division by a constant of the launch: n / d for 0 <= n < 2^31, by the rounded-up
// reciprocal 2^32 + mul and a shift (Granlund and Montgomery, "Division by invariant
// integers using multiplication", 1994).
struct FastDiv {
  uint32_t mul, shift, d;
  __host__ void set(int32_t divisor) {
    d = static_cast<uint32_t>(divisor);
    shift = 0;
    while ((1ull << shift) < d) ++shift;
    mul = static_cast<uint32_t>(((1ull << 32) * ((1ull << shift) - d)) / d + 1);
  }
  __device__ __forceinline__ int div(int n) const {
    return static_cast<int>((__umulhi(static_cast<uint32_t>(n), mul) + static_cast<uint32_t>(n)) >> shift);
  }
};

// The tiles of one product on 256 x 256 tiles of CTA pairs, in the order of
// their numbers: by parts of K; within a part by groups of group_m row tiles;
// within a group column by column, the row tile fastest.  Tiles that run at
// the same time then share the group's A rows and a few B blocks in L2.
struct TileGrid {
  int32_t tiles_m, tiles_n, splits;
  int32_t kb_total, kb_step;  // 64-deep k-blocks, and those of one part
  int32_t group_m, last_m;    // row tiles of a group, and of the last one
  FastDiv per_split, per_group, group, last;
  // m x n x k, K in `parts` or fewer non-empty parts.
  __host__ void set(int64_t m, int64_t n, int64_t k, int parts, int group_rows) {
    tiles_m = static_cast<int32_t>((m + 255) / 256);
    tiles_n = static_cast<int32_t>((n + 255) / 256);
    kb_total = static_cast<int32_t>((k + 63) / 64);
    kb_step = (kb_total + parts - 1) / parts;
    splits = (kb_total + kb_step - 1) / kb_step;
    group_m = group_rows < tiles_m ? group_rows : tiles_m;
    last_m = tiles_m % group_m ? tiles_m % group_m : group_m;
    per_split.set(tiles_m * tiles_n);
    per_group.set(group_m * tiles_n);
    group.set(group_m);
    last.set(last_m);
  }
  __host__ __device__ int32_t count() const { return tiles_m * tiles_n * splits; }
};

// Factor of both gradients, scale [/ sum of the counted weights], which depends
// on no logit: a warp that the logits' kernel has to spare writes it.
struct CeNorm {
  float* alpha;                       // null: not wanted
  IdList targets;
  const float* weights;
  int64_t n;
  int32_t mean;
  float scale;
};

// L = sum(weight * loss) [/ sum(weight)] from the row blocks' sums: a warp that
// the gradients' kernel has to spare writes it.
struct CeTotal {
  float* total;                       // null: not wanted
  const double2* partial;
  int64_t parts;
  int32_t mean;
};

// Longer lists are summed by a whole block: one warp would outlast the product.
constexpr int64_t kSideSums = 16384;

// This thread's share of the sums, every `step`-th entry from `first` on, and
// what is written from the whole.
__device__ __forceinline__ double norm_share(const CeNorm& N, int first, int step) {
  double sum = 0.0;
  if (!N.mean) return sum;
#pragma unroll 8
  for (int64_t i = first; i < N.n; i += step) {
    bool bad = false;
    const int t = load_id(N.targets, i, &bad);
    sum += t < 0 ? 0.f : N.weights ? N.weights[i] : 1.f;
  }
  return sum;
}
__device__ __forceinline__ void put_alpha(const CeNorm& N, double sum) {
  *N.alpha = !N.mean ? N.scale : sum != 0.0 ? static_cast<float>(N.scale / sum) : 0.f;
}
__device__ __forceinline__ double2 total_share(const CeTotal& T, int first, int step) {
  double2 s = make_double2(0.0, 0.0);
#pragma unroll 8
  for (int64_t i = first; i < T.parts; i += step) {
    const double2 q = load_l2(T.partial + i);
    s.x += q.x;
    s.y += q.y;
  }
  return s;
}
__device__ __forceinline__ void put_total(const CeTotal& T, double2 s) {
  *T.total = static_cast<float>(!T.mean ? s.x : s.y != 0.0 ? s.x / s.y : 0.0);
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ void write_alpha(const CeNorm& N, int lane) {
  const double sum = warp_sum(norm_share(N, lane, 32));
  if (lane == 0) put_alpha(N, sum);
}
__device__ __forceinline__ void write_total(const CeTotal& T, int lane) {
  double2 s = total_share(T, lane, 32);
  s.x = warp_sum(s.x);
  s.y = warp_sum(s.y);
  if (lane == 0) put_total(T, s);
}

// Z = X W^T: statistics, optionally logs.
struct VocabLogits {
  CUtensorMap map_a, map_b;           // X, W
  int32_t M, N;                       // tokens, vocabulary
  TileGrid grid;
  int* err;
  float logit_scale_log2;             // logit scale times log2(e)
  uint16_t* logs;                     // [row][ld_logs], ld_logs a multiple of 64; or null
  int64_t ld_logs;
  float2* stats;                      // [block][row]: maximum, and sum of 2^(z - maximum) without the target's; z in octaves
  int64_t stats_ld;
  IdList targets;                     // of row 0 of this product
  uint32_t* counter;                  // zero before
  int32_t drawn;                      // tiles drawn from the counter, else fixed shares
  CeNorm norm;
};
cudaError_t launch_vocab_logits(const VocabLogits& G, int n_pairs, cudaStream_t st);

// One gradient product D (M x N) = alpha A B: B is k x n with contiguous
// columns, A is m x k, or k x m with a_mn.
struct VgProduct {
  CUtensorMap map_a, map_b, map_out;
  int32_t M, N;
  TileGrid grid;                      // grid.splits > 1: fp32 partials, one per part of K
  int32_t a_mn;
  int32_t out_bf16;                   // else fp32
  int32_t add;                        // add to what the output holds (bf16: `direct` only)
  // Rows that TMA cannot write, or a bf16 sum: stored from registers instead of through map_out.
  int32_t direct;
  void* out;
  int64_t ld_out;
};

// One launch for up to two products, the first's tiles first.
struct VocabGrad {
  VgProduct p[2];
  int32_t n_units[2];                 // tiles times parts
  uint32_t* counter;                  // zero before
  int32_t drawn;                      // tiles drawn from the counter, else fixed shares
  int32_t extra;                      // fixed shares: see fixed_tile
  const float* alpha;
  CeTotal total;
  int* err;
};
cudaError_t launch_vocab_grad(const VocabGrad& G, int n_pairs, cudaStream_t st);
int vocab_gemm_max_pairs();

// The products that read W, for few tokens (k_vocab_thin.cu).
constexpr int kThinRows = 256;        // token rows at most
struct VocabThin {
  CUtensorMap map_a, map_b;           // W; X or dZ
  int32_t M;                          // vocabulary (logits) or width (dX)
  int32_t tokens, np;                 // token rows, and those rounded up to 16
  int32_t tiles_m, splits, kb_total, kb_step;
  int32_t groups;                     // accumulators that K is cut into
  int* err;
  // logits
  float logit_scale_log2;
  uint16_t* logs;                     // [token][ld_logs], or null
  int64_t ld_logs;
  float2* stats;
  int64_t stats_ld;
  IdList targets;
  CeNorm norm;
  // dX: fp32 partials [split][token][ld_part]
  float* part;
  int64_t ld_part;
};
cudaError_t launch_vocab_thin(bool logits, const VocabThin& G, int n_ctas, cudaStream_t st);

// ---- k_vocab_ce.cu
// Copy of rows x cols bf16 values into rows of pitch ld_dst (a multiple of 8).
// With targets, rows that are not counted become zeros.
cudaError_t launch_ce_copy(const uint16_t* src, int64_t ld_src, uint16_t* dst, int64_t ld_dst, int64_t rows,
                           int32_t cols, const IdList& targets, cudaStream_t st);

// The factor alone, for long lists.
cudaError_t launch_ce_norm(const CeNorm& N, cudaStream_t st);

// Per-row outcome of the statistics, as the gradient pass reads it.
struct CeRow {
  float lse2;       // log2 of the softmax's sum, in octaves
  float weight;     // 0 for a row that is not counted
  float target_dz;  // weight * (p_target - 1)
  int32_t target;   // -1: none
};

struct CeRows {
  const float2* stats;
  int64_t stats_ld;
  int32_t n_blocks;        // vocabulary blocks
  int64_t row0, rows;      // rows of this pass
  IdList targets;          // of row 0
  const float* weights;    // of row 0, or null
  const uint16_t* x;       // of row row0
  const uint16_t* w;
  int64_t ld_x, ld_w;
  int32_t dim;
  double logit_scale_log2;
  CeRow* out;              // of row row0, or null
  // Few rows: the same launch turns the logs into d logits in two halves (launch_ce_dlogits says how). Null: not wanted.
  uint16_t* block;
  int64_t ld_block, lo_rows;
  int32_t vocab, stats_shift;
  float* loss;             // of row 0, or null
  float* lse;              // of row 0, or null
  // dW's operand: this pass's rows of x, zeros where the row is not counted; twice
  // (copies rows apart) for a gradient in two halves.  Null: not wanted.
  uint16_t* x_copy;
  int64_t ld_copy;
  int32_t copies;
  int32_t width;           // rows of a block: ce_rows_width(n)
  double2* partial;        // [row / width]: sums of weight * loss and weight; null without total
  CeTotal total;           // written by the last block
  uint32_t* ticket;        // zero before and after
  uint32_t* counters;      // the products' two tile counters, set to zero
  int* err;
};
int ce_rows_width(int64_t n);
// Whether launch_ce_rows makes the d logits too.
bool ce_rows_make_dlogits(int64_t n);
cudaError_t launch_ce_rows(const CeRows& R, cudaStream_t st);

// Fixed-point logs -> bf16 d logits (before the factor alpha), in place.  With
// lo_rows > 0 the rounding's rest goes, as bf16, to the row lo_rows below.
cudaError_t launch_ce_dlogits(uint16_t* block, int64_t ld, int64_t rows, int32_t vocab, int32_t stats_shift,
                              const float2* stats, int64_t stats_ld, const CeRow* row_info, int64_t lo_rows,
                              cudaStream_t st);

// out (rows x cols, pitch ld_out) = sum over `parts` partials (pitch ld_part,
// part_stride elements apart), with fold > 0 of their rows r and r + fold [+ out].
cudaError_t launch_ce_finish(const float* part, int64_t ld_part, int64_t part_stride, int parts, int64_t fold,
                             void* out, int64_t ld_out, int out_bf16, int accumulate, const float* alpha,
                             int64_t rows, int32_t cols, cudaStream_t st);

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
  uint32_t* present;  // one bit per table row: named by an entry; null when adding
  float* partial;
};
// Sorted positions that one block of the summing kernel takes at most.
constexpr int kEmbedRun = 64;
struct EmbedWs {
  size_t key[2], pos[2], hist, present, partial, bytes;
};
EmbedWs embed_backward_ws(int64_t n, int64_t vocab, int32_t dim);
// Enqueues the launches; *launches counts them.
cudaError_t launch_embed_backward(const EmbedBackward& E, int* launches, cudaStream_t st);

}  // namespace dmuon
