// Entry points of the vocabulary operators: argument checks, workspace layout
// and launch order of the cross entropy and of the embedding lookup (kernels:
// k_vocab_gemm.cu, k_vocab_ce.cu, k_embed.cu).
#include "vocab.h"

#include "runtime.h"

namespace dmuon {

// Encodes a tensor map of `count` slices of rows x inner elements (plan.cu).
int make_map_typed(EncodeTiledFn enc, CUtensorMap* out, CUtensorMapDataType type, int elem_bytes, const void* base,
                   int64_t inner, int64_t rows, int64_t count, int64_t ld, int64_t slice_stride, uint32_t box_inner,
                   uint32_t box_rows) {
  cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)rows, (cuuint64_t)count};
  cuuint64_t strides[2] = {(cuuint64_t)(ld * elem_bytes), (cuuint64_t)(slice_stride * elem_bytes)};
  cuuint32_t box[3] = {box_inner, box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = enc(out, type, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    char buf[200];
    snprintf(buf, sizeof buf, "cuTensorMapEncodeTiled failed (%d) for a %lld x %lld x %lld map", (int)r,
             (long long)inner, (long long)rows, (long long)count);
    return set_error(DMUON_ERR_CUDA, buf);
  }
  return DMUON_OK;
}

namespace {

// ------------------------------------------------------------ argument checks
struct Range {
  const void* p;
  int64_t bytes;
  bool written;
  const char* what;
};

// Bytes from the first to the last element of rows x cols at pitch ld.
int64_t span_bytes(int64_t rows, int64_t cols, int64_t ld, int64_t elem) {
  return rows <= 0 ? 0 : ((rows - 1) * ld + cols) * elem;
}

int check_ranges(const dmuon_context* ctx, const char* op, const Range* r, int n) {
  char buf[200];
  for (int i = 0; i < n; ++i)
    for (int j = i + 1; j < n; ++j) {
      if (!r[i].p || !r[j].p || (!r[i].written && !r[j].written)) continue;
      const uintptr_t a = reinterpret_cast<uintptr_t>(r[i].p), b = reinterpret_cast<uintptr_t>(r[j].p);
      if (r[i].bytes > 0 && r[j].bytes > 0 && a < b + r[j].bytes && b < a + r[i].bytes) {
        snprintf(buf, sizeof buf, "%s: %s overlaps %s (memory the call writes must not be shared)", op, r[i].what,
                 r[j].what);
        return set_error(DMUON_ERR_INVALID_ARG, buf);
      }
    }
  return DMUON_OK;
}

int check_pointers(const dmuon_context* ctx, const Range* r, int n) {
  for (int i = 0; i < n; ++i) {
    if (!r[i].p || r[i].bytes <= 0) continue;
    const int st = check_reachable(ctx, r[i].p, r[i].what, 0);
    if (st != DMUON_OK) return st;
  }
  return DMUON_OK;
}

int check_sizes(const char* op, int64_t n, int64_t vocab, int64_t dim) {
  char buf[160];
  if (n < 0 || n > INT32_MAX || vocab < 1 || vocab > (int64_t(1) << 24) || dim < 1 || dim > (int64_t(1) << 20)) {
    snprintf(buf, sizeof buf, "%s: %lld tokens, vocabulary %lld, width %lld (limits: 2^31 - 1, 2^24, 2^20)", op,
             (long long)n, (long long)vocab, (long long)dim);
    return set_error(DMUON_ERR_SHAPE, buf);
  }
  return DMUON_OK;
}

int check_ld(const char* op, const char* what, int64_t ld, int64_t dim) {
  char buf[160];
  if (ld < dim || ld > (int64_t(1) << 32)) {
    snprintf(buf, sizeof buf, "%s: row pitch %lld of %s (the width is %lld)", op, (long long)ld, what, (long long)dim);
    return set_error(DMUON_ERR_SHAPE, buf);
  }
  return DMUON_OK;
}

int check_type(const char* op, const char* what, int32_t t, bool f32_allowed) {
  if (t == DMUON_DTYPE_BF16 || (f32_allowed && t == DMUON_DTYPE_F32)) return DMUON_OK;
  char buf[160];
  snprintf(buf, sizeof buf, "%s: dtype %d of %s", op, t, what);
  return set_error(DMUON_ERR_DTYPE, buf);
}

int check_index(const char* op, int32_t t) {
  if (t == DMUON_INDEX_I32 || t == DMUON_INDEX_I64) return DMUON_OK;
  char buf[160];
  snprintf(buf, sizeof buf, "%s: index dtype %d", op, t);
  return set_error(DMUON_ERR_DTYPE, buf);
}

#define DM_TRY(call)                    \
  do {                                  \
    const int st_ = (call);             \
    if (st_ != DMUON_OK) return st_;    \
  } while (0)

// ------------------------------------------------------------------ workspace
// The vocabulary operators' own scratch: grown on demand, shared by all calls
// on the context.  A call on another stream than the last one waits for it.
int vocab_workspace(dmuon_context* ctx, size_t bytes, cudaStream_t s) {
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  DM_CUDA(cudaStreamIsCapturing(s, &cap));
  if (cap == cudaStreamCaptureStatusNone && ctx->vocab_used && ctx->vocab_stream != s)
    DM_CUDA(cudaStreamWaitEvent(s, ctx->vocab_done, 0));
  if (bytes > ctx->vocab_ws.bytes) {
    ctx->vocab_ws.release();
    const int st = dev_alloc(ctx->vocab_ws, bytes);
    if (st != DMUON_OK) return st;
  }
  if (!ctx->vocab_ticket.p) {
    const int st = dev_alloc(ctx->vocab_ticket, 256);
    if (st != DMUON_OK) return st;
    DM_CUDA(cudaMemset(ctx->vocab_ticket.p, 0, 256));
  }
  return DMUON_OK;
}

// After the last launch that uses the workspace.
int vocab_used(dmuon_context* ctx, cudaStream_t s) {
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  DM_CUDA(cudaStreamIsCapturing(s, &cap));
  if (cap != cudaStreamCaptureStatusNone) return DMUON_OK;
  if (!ctx->vocab_done) DM_CUDA(cudaEventCreateWithFlags(&ctx->vocab_done, cudaEventDisableTiming));
  DM_CUDA(cudaEventRecord(ctx->vocab_done, s));
  ctx->vocab_stream = s;
  ctx->vocab_used = true;
  return DMUON_OK;
}

struct Layout {
  size_t bytes = 0;
  size_t take(size_t n) {
    const size_t at = bytes;
    bytes += (n + 1023) / 1024 * 1024;
    return at;
  }
};

// ---------------------------------------------------------------- the products
// Whether TMA can address rows of this pitch.
bool tma_rows(const void* p, int64_t ld, int elem) { return aligned16(p) && ld * elem % 16 == 0; }

constexpr int kVgTile = 256;

// Parts that the K axis of an M x N product is cut into: few output tiles leave
// pairs idle, and every part costs a pass of its fp32 partial through memory.
// Unit: one k-block of one tile (256 x 256 x 64, about 0.27 us on a pair);
// 12 units is what a tile's pipeline fill and epilogue measured, and 24 KB
// of partial traffic take a unit at the copy rate.
int choose_splits(int64_t m, int64_t n, int64_t k, int pairs, bool need_partial) {
  const int64_t tiles = ((m + kVgTile - 1) / kVgTile) * ((n + kVgTile - 1) / kVgTile);
  const int64_t kb = (k + 63) / 64;
  if (tiles >= 4 * pairs) return 1;
  double best = 0.0;
  int parts = 1;
  for (int s = 1; s <= 64 && s <= kb; ++s) {
    const int64_t waves = (tiles * s + pairs - 1) / pairs;
    double cost = static_cast<double>(waves) * (static_cast<double>((kb + s - 1) / s) + 12.0);
    if (s > 1 || need_partial) cost += 10.0 + static_cast<double>(m) * static_cast<double>(n) * 4.0 * (2.0 * s + 1.0) / 1.8e6;
    if (s == 1 || cost < best * 0.95) {
      best = cost;
      parts = s;
    }
  }
  return parts;
}

struct Product {
  int64_t m, n, k;
  bool a_mn;
  const void* a;
  int64_t ld_a;  // rows x inner: m x k (or k x m when a_mn)
  const void* b;
  int64_t ld_b;  // k x n
  void* out;
  int64_t ld_out;
  bool out_bf16;
  bool keep;     // add to what `out` holds
  // fp32 partials, or null where the product writes `out` itself
  float* part;
  int64_t ld_part;
  int splits;
  bool first, last;  // first and last pass over the rows (dW)
};

int encode_2d(EncodeTiledFn enc, CUtensorMap* map, const void* p, int64_t inner, int64_t rows, int64_t ld, uint32_t box_inner,
              uint32_t box_rows) {
  return make_map_typed(enc, map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p, inner, rows, 1, ld, rows * ld, box_inner, box_rows);
}

void set_tiles(VocabGemm& G, int64_t m, int64_t n, int64_t k, int splits) {
  G.M = static_cast<int32_t>(m);
  G.N = static_cast<int32_t>(n);
  G.K = static_cast<int32_t>(k);
  G.tiles_m = static_cast<int32_t>((m + kVgTile - 1) / kVgTile);
  G.tiles_n = static_cast<int32_t>((n + kVgTile - 1) / kVgTile);
  G.kb_total = static_cast<int32_t>((k + 63) / 64);
  G.splits = splits;
  G.group_m = 8;
}

int run_product(dmuon_context* ctx, EncodeTiledFn enc, const Product& P, cudaStream_t s) {
  VocabGemm G = {};
  set_tiles(G, P.m, P.n, P.k, P.splits);
  G.err = static_cast<int*>(ctx->err.p);
  if (P.a_mn)
    DM_TRY(encode_2d(enc, &G.map_a, P.a, P.m, P.k, P.ld_a, 64, 64));
  else
    DM_TRY(encode_2d(enc, &G.map_a, P.a, P.k, P.m, P.ld_a, 64, 128));
  DM_TRY(encode_2d(enc, &G.map_b, P.b, P.n, P.k, P.ld_b, 64, 64));
  int mode = kVgF32;
  if (P.part) {
    DM_TRY(make_map_typed(enc, &G.map_out, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, P.part, P.n, P.m, P.splits, P.ld_part,
                          P.m * P.ld_part, 32, 32));
    G.add = P.first ? 0 : 1;
  } else if (P.out_bf16) {
    mode = kVgBf16;
    DM_TRY(encode_2d(enc, &G.map_out, P.out, P.n, P.m, P.ld_out, 64, 32));
  } else {
    DM_TRY(make_map_typed(enc, &G.map_out, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, P.out, P.n, P.m, 1, P.ld_out,
                          P.m * P.ld_out, 32, 32));
    G.add = P.keep || !P.first ? 1 : 0;
  }
  DM_TRY(timed_launch(ctx, -1, s, [&] { return launch_vocab_gemm(mode, P.a_mn, true, G, ctx->vocab_pairs, s); }));
  if (P.part && P.last)
    DM_TRY(timed_launch(ctx, -1, s, [&] {
      return launch_ce_finish(P.part, P.ld_part, P.m * P.ld_part, P.splits, P.out, P.ld_out, P.out_bf16, P.keep, P.m,
                              static_cast<int32_t>(P.n), s);
    }));
  return DMUON_OK;
}

// Whether a product of these properties may write its output itself.
bool writes_out(const void* out, int64_t ld, bool bf16, bool keep, bool one_pass, int splits) {
  if (splits > 1 || !tma_rows(out, ld, bf16 ? 2 : 4)) return false;
  return bf16 ? one_pass && !keep : true;
}

int cross_entropy_impl(dmuon_context* ctx, const dmuon_ce& C, cudaStream_t s) {
  const int64_t n = C.n_tokens, v = C.vocab, d = C.dim;
  const bool grads = C.dx || C.dw;
  const bool mean = (C.flags & DMUON_CE_MEAN) != 0, add_dw = (C.flags & DMUON_CE_ADD_DW) != 0;
  const bool dx_bf16 = C.dx_dtype == DMUON_DTYPE_BF16, dw_bf16 = C.dw_dtype == DMUON_DTYPE_BF16;
  if (n == 0) {
    if (C.total) DM_CUDA(cudaMemsetAsync(C.total, 0, sizeof(float), s));
    if (C.dw && !add_dw)
      DM_CUDA(cudaMemset2DAsync(C.dw, static_cast<size_t>(C.ld_dw * (dw_bf16 ? 2 : 4)), 0,
                                static_cast<size_t>(d * (dw_bf16 ? 2 : 4)), static_cast<size_t>(v), s));
    return DMUON_OK;
  }
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return set_error(DMUON_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  if (ctx->vocab_pairs == 0) ctx->vocab_pairs = vocab_gemm_max_pairs();
  const int pairs = ctx->vocab_pairs;
  if (pairs < 1) return set_error(DMUON_ERR_UNSUPPORTED, "cross_entropy: no CTA pair of the product kernel fits the device");

  // Rows of one pass: the block of fixed-point logs stays within its limit.
  // Without gradients there is no block and one pass takes all rows.
  const int64_t ld_block = round_up(v, 64);
  int64_t rows = n;
  if (grads) {
    const int64_t most = std::max<int64_t>(kVgTile, ctx->tune.ce_block_bytes / (2 * ld_block) / kVgTile * kVgTile);
    const int64_t passes = (n + most - 1) / most;
    rows = passes == 1 ? n : round_up((n + passes - 1) / passes, kVgTile);
  }
  const bool one_pass = rows >= n;
  const int n_blocks = static_cast<int>((v + kCeBlock - 1) / kCeBlock);
  const int64_t stats_ld = round_up(rows, 32);

  // Operand copies: rows that are not counted must read as zeros in dW's
  // product whatever they hold, and TMA needs rows on 16 bytes.
  const bool copy_x = C.dw != nullptr || !tma_rows(C.x, C.ld_x, 2);
  const bool copy_w = !tma_rows(C.w, C.ld_w, 2);
  const int64_t ld8 = round_up(d, 8), ld4 = round_up(d, 4);
  Layout L;
  const size_t off_x = copy_x ? L.take(static_cast<size_t>(n * ld8) * 2) : 0;
  const size_t off_w = copy_w ? L.take(static_cast<size_t>(v * ld8) * 2) : 0;
  const size_t off_stats = L.take(static_cast<size_t>(n_blocks * stats_ld) * sizeof(float2));
  const size_t off_z = L.take(static_cast<size_t>(rows) * 4);
  const size_t off_loss = C.loss ? 0 : L.take(static_cast<size_t>(n) * 4);
  const size_t off_norm = L.take(4);
  size_t off_block = 0, off_rows = 0, off_dx = 0, off_dw = 0;
  int dx_splits = 1, dw_splits = 1;
  bool dx_part = false, dw_part = false;
  if (grads) {
    off_block = L.take(static_cast<size_t>(rows * ld_block) * 2);
    off_rows = L.take(static_cast<size_t>(rows) * sizeof(CeRow));
    if (C.dx) {
      dx_splits = choose_splits(rows, d, v, pairs, !writes_out(C.dx, C.ld_dx, dx_bf16, false, true, 1));
      dx_part = !writes_out(C.dx, C.ld_dx, dx_bf16, false, true, dx_splits);
      if (dx_part) off_dx = L.take(static_cast<size_t>(dx_splits * rows * ld4) * 4);
    }
    if (C.dw) {
      dw_splits = choose_splits(v, d, rows, pairs, !writes_out(C.dw, C.ld_dw, dw_bf16, add_dw, one_pass, 1));
      dw_part = !writes_out(C.dw, C.ld_dw, dw_bf16, add_dw, one_pass, dw_splits);
      if (dw_part) off_dw = L.take(static_cast<size_t>(dw_splits * v * ld4) * 4);
    }
  }
  DM_TRY(vocab_workspace(ctx, L.bytes, s));
  char* ws = static_cast<char*>(ctx->vocab_ws.p);
  const IdList ids{C.targets, C.target_dtype == DMUON_INDEX_I64, static_cast<int32_t>(v)};
  auto ids_from = [&](int64_t row) {
    IdList q = ids;
    q.p = static_cast<const char*>(ids.p) + row * (ids.is64 ? 8 : 4);
    return q;
  };
  const uint16_t* x = C.x;
  const uint16_t* w = C.w;
  int64_t ld_x = C.ld_x, ld_w = C.ld_w;
  float* inv_norm = grads && mean ? reinterpret_cast<float*>(ws + off_norm) : nullptr;
  if (copy_x) {
    uint16_t* to = reinterpret_cast<uint16_t*>(ws + off_x);
    DM_TRY(timed_launch(ctx, -1, s, [&] {
      return launch_ce_copy(C.x, C.ld_x, to, ld8, n, static_cast<int32_t>(d), &ids, C.weights, inv_norm, s);
    }));
    x = to;
    ld_x = ld8;
  } else if (inv_norm) {
    DM_TRY(timed_launch(ctx, -1, s, [&] {
      return launch_ce_copy(nullptr, 0, nullptr, 0, n, static_cast<int32_t>(d), &ids, C.weights, inv_norm, s);
    }));
  }
  if (copy_w) {
    uint16_t* to = reinterpret_cast<uint16_t*>(ws + off_w);
    DM_TRY(timed_launch(ctx, -1, s, [&] {
      return launch_ce_copy(C.w, C.ld_w, to, ld8, v, static_cast<int32_t>(d), nullptr, nullptr, nullptr, s);
    }));
    w = to;
    ld_w = ld8;
  }
  float2* stats = reinterpret_cast<float2*>(ws + off_stats);
  float* target_z = reinterpret_cast<float*>(ws + off_z);
  float* loss = C.loss ? C.loss : reinterpret_cast<float*>(ws + off_loss);
  uint16_t* block = reinterpret_cast<uint16_t*>(ws + off_block);
  CeRow* row_info = reinterpret_cast<CeRow*>(ws + off_rows);

  for (int64_t r0 = 0; r0 < n; r0 += rows) {
    const int64_t nr = std::min(rows, n - r0);
    const bool first = r0 == 0, last = r0 + rows >= n;
    VocabGemm G = {};
    set_tiles(G, nr, v, d, 1);
    G.err = static_cast<int*>(ctx->err.p);
    DM_TRY(encode_2d(enc, &G.map_a, x + r0 * ld_x, d, nr, ld_x, 64, 128));
    DM_TRY(encode_2d(enc, &G.map_b, w, d, v, ld_w, 64, 128));
    if (grads) DM_TRY(encode_2d(enc, &G.map_out, block, v, nr, ld_block, 64, 32));
    G.logit_scale_log2 = C.logit_scale * 1.4426950408889634f;
    G.store_logs = grads;
    G.stats = stats;
    G.stats_ld = stats_ld;
    G.target_z = target_z;
    G.targets = ids_from(r0);
    DM_TRY(timed_launch(ctx, -1, s, [&] { return launch_vocab_gemm(kVgLogits, false, false, G, pairs, s); }));

    CeRows R = {};
    R.stats = stats;
    R.stats_ld = stats_ld;
    R.n_blocks = n_blocks;
    R.row0 = r0;
    R.rows = nr;
    R.n = n;
    R.target_z = target_z;
    R.targets = ids;
    R.weights = C.weights;
    R.inv_norm = inv_norm;
    R.grad_scale = C.grad_scale * C.logit_scale;
    R.out = grads ? row_info : nullptr;
    R.loss = loss;
    R.lse = C.lse;
    R.total = last ? C.total : nullptr;
    R.mean = mean;
    R.ticket = static_cast<uint32_t*>(ctx->vocab_ticket.p);
    R.err = static_cast<int*>(ctx->err.p);
    DM_TRY(timed_launch(ctx, -1, s, [&] { return launch_ce_rows(R, s); }));
    if (!grads) continue;

    DM_TRY(timed_launch(ctx, -1, s, [&] {
      return launch_ce_dlogits(block, ld_block, nr, static_cast<int32_t>(v), stats, stats_ld, row_info, s);
    }));
    if (C.dx) {
      Product P = {};
      P.m = nr; P.n = d; P.k = v;
      P.a = block; P.ld_a = ld_block;
      P.b = w; P.ld_b = ld_w;
      P.out = static_cast<char*>(C.dx) + r0 * C.ld_dx * (dx_bf16 ? 2 : 4);
      P.ld_out = C.ld_dx;
      P.out_bf16 = dx_bf16;
      P.part = dx_part ? reinterpret_cast<float*>(ws + off_dx) : nullptr;
      P.ld_part = ld4;
      P.splits = dx_splits;
      P.first = P.last = true;
      DM_TRY(run_product(ctx, enc, P, s));
    }
    if (C.dw) {
      Product P = {};
      P.m = v; P.n = d; P.k = nr;
      P.a_mn = true;
      P.a = block; P.ld_a = ld_block;
      P.b = x + r0 * ld_x; P.ld_b = ld_x;
      P.out = C.dw;
      P.ld_out = C.ld_dw;
      P.out_bf16 = dw_bf16;
      P.keep = add_dw;
      P.part = dw_part ? reinterpret_cast<float*>(ws + off_dw) : nullptr;
      P.ld_part = ld4;
      // The last pass may be shorter: every part needs a k-block of its own,
      // and its other parts already hold the earlier passes' sums.
      P.splits = static_cast<int>(std::min<int64_t>(dw_splits, (nr + 63) / 64));
      P.first = first;
      P.last = false;
      DM_TRY(run_product(ctx, enc, P, s));
      if (dw_part && last)
        DM_TRY(timed_launch(ctx, -1, s, [&] {
          return launch_ce_finish(P.part, ld4, v * ld4, dw_splits, C.dw, C.ld_dw, dw_bf16, add_dw, v,
                                  static_cast<int32_t>(d), s);
        }));
    }
  }
  return vocab_used(ctx, s);
}

}  // namespace
}  // namespace dmuon

using namespace dmuon;

extern "C" {

int dmuon_cross_entropy(dmuon_context* ctx, const dmuon_ce* args, void* stream) {
  clear_error();
  if (!ctx || !args) return set_error(DMUON_ERR_INVALID_ARG, "cross_entropy: null context or arguments");
  const dmuon_ce& C = *args;
  const char* op = "cross_entropy";
  DM_TRY(check_sizes(op, C.n_tokens, C.vocab, C.dim));
  // An empty list may come without memory.
  if (!C.w || (C.n_tokens > 0 && (!C.x || !C.targets)))
    return set_error(DMUON_ERR_INVALID_ARG, "cross_entropy: null x, w or targets");
  if (C.n_tokens > 0 && !C.loss && !C.lse && !C.total && !C.dx && !C.dw)
    return set_error(DMUON_ERR_INVALID_ARG, "cross_entropy: no output asked for");
  if (!finite(C.logit_scale) || C.logit_scale <= 0.f || !finite(C.grad_scale))
    return set_error(DMUON_ERR_INVALID_ARG, "cross_entropy: logit_scale must be positive, grad_scale finite");
  if (C.flags & ~uint32_t(DMUON_CE_MEAN | DMUON_CE_ADD_DW))
    return set_error(DMUON_ERR_INVALID_ARG, "cross_entropy: unknown flag bits");
  DM_TRY(check_type(op, "x", C.x_dtype, false));
  DM_TRY(check_type(op, "w", C.w_dtype, false));
  DM_TRY(check_index(op, C.target_dtype));
  DM_TRY(check_ld(op, "x", C.ld_x, C.dim));
  DM_TRY(check_ld(op, "w", C.ld_w, C.dim));
  if (C.dx) {
    DM_TRY(check_type(op, "dx", C.dx_dtype, true));
    DM_TRY(check_ld(op, "dx", C.ld_dx, C.dim));
  }
  if (C.dw) {
    DM_TRY(check_type(op, "dw", C.dw_dtype, true));
    DM_TRY(check_ld(op, "dw", C.ld_dw, C.dim));
  }
  const Range r[] = {
      {C.x, span_bytes(C.n_tokens, C.dim, C.ld_x, 2), false, "x"},
      {C.w, span_bytes(C.vocab, C.dim, C.ld_w, 2), false, "w"},
      {C.targets, C.n_tokens * (C.target_dtype == DMUON_INDEX_I64 ? 8 : 4), false, "targets"},
      {C.weights, C.n_tokens * 4, false, "weights"},
      {C.loss, C.n_tokens * 4, true, "loss"},
      {C.lse, C.n_tokens * 4, true, "lse"},
      {C.total, 4, true, "total"},
      {C.dx, span_bytes(C.n_tokens, C.dim, C.ld_dx, C.dx_dtype == DMUON_DTYPE_BF16 ? 2 : 4), true, "dx"},
      {C.dw, span_bytes(C.vocab, C.dim, C.ld_dw, C.dw_dtype == DMUON_DTYPE_BF16 ? 2 : 4), true, "dw"},
  };
  const int nr = static_cast<int>(sizeof r / sizeof r[0]);
  DM_TRY(check_ranges(ctx, op, r, nr));
  DeviceGuard guard(ctx->device);
  DM_TRY(ensure_device(ctx));
  DM_TRY(check_pointers(ctx, r, nr));
  return cross_entropy_impl(ctx, C, static_cast<cudaStream_t>(stream));
}

int dmuon_embed_forward(dmuon_context* ctx, const dmuon_embed* args, void* stream) {
  clear_error();
  if (!ctx || !args) return set_error(DMUON_ERR_INVALID_ARG, "embed_forward: null context or arguments");
  const dmuon_embed& A = *args;
  const char* op = "embed_forward";
  DM_TRY(check_sizes(op, A.n_tokens, A.vocab, A.dim));
  if (!A.table || (A.n_tokens > 0 && (!A.ids || !A.rows)))
    return set_error(DMUON_ERR_INVALID_ARG, "embed_forward: null ids, table or rows");
  if (!finite(A.scale)) return set_error(DMUON_ERR_INVALID_ARG, "embed_forward: non-finite scale");
  if (A.flags) return set_error(DMUON_ERR_INVALID_ARG, "embed_forward: unknown flag bits");
  DM_TRY(check_index(op, A.id_dtype));
  DM_TRY(check_type(op, "table", A.table_dtype, true));
  DM_TRY(check_type(op, "rows", A.row_dtype, true));
  DM_TRY(check_ld(op, "table", A.ld_table, A.dim));
  DM_TRY(check_ld(op, "rows", A.ld_rows, A.dim));
  const Range r[] = {
      {A.ids, A.n_tokens * (A.id_dtype == DMUON_INDEX_I64 ? 8 : 4), false, "ids"},
      {A.table, span_bytes(A.vocab, A.dim, A.ld_table, A.table_dtype == DMUON_DTYPE_BF16 ? 2 : 4), false, "table"},
      {A.rows, span_bytes(A.n_tokens, A.dim, A.ld_rows, A.row_dtype == DMUON_DTYPE_BF16 ? 2 : 4), true, "rows"},
  };
  DM_TRY(check_ranges(ctx, op, r, 3));
  DeviceGuard guard(ctx->device);
  DM_TRY(ensure_device(ctx));
  DM_TRY(check_pointers(ctx, r, 3));
  if (A.n_tokens == 0) return DMUON_OK;
  EmbedForward E = {};
  E.ids = IdList{A.ids, A.id_dtype == DMUON_INDEX_I64, static_cast<int32_t>(A.vocab)};
  E.n = A.n_tokens;
  E.table = A.table;
  E.ld_table = A.ld_table;
  E.table_bf16 = A.table_dtype == DMUON_DTYPE_BF16;
  E.out = A.rows;
  E.ld_out = A.ld_rows;
  E.out_bf16 = A.row_dtype == DMUON_DTYPE_BF16;
  E.dim = static_cast<int32_t>(A.dim);
  E.scale = A.scale;
  E.err = static_cast<int*>(ctx->err.p);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return timed_launch(ctx, -1, s, [&] { return launch_embed_forward(E, s); });
}

int dmuon_embed_backward(dmuon_context* ctx, const dmuon_embed* args, void* stream) {
  clear_error();
  if (!ctx || !args) return set_error(DMUON_ERR_INVALID_ARG, "embed_backward: null context or arguments");
  const dmuon_embed& A = *args;
  const char* op = "embed_backward";
  DM_TRY(check_sizes(op, A.n_tokens, A.vocab, A.dim));
  if (!A.table || (A.n_tokens > 0 && (!A.ids || !A.rows)))
    return set_error(DMUON_ERR_INVALID_ARG, "embed_backward: null ids, table or rows");
  if (!finite(A.scale)) return set_error(DMUON_ERR_INVALID_ARG, "embed_backward: non-finite scale");
  if (A.flags & ~uint32_t(DMUON_EMBED_ADD)) return set_error(DMUON_ERR_INVALID_ARG, "embed_backward: unknown flag bits");
  DM_TRY(check_index(op, A.id_dtype));
  DM_TRY(check_type(op, "table", A.table_dtype, true));
  DM_TRY(check_type(op, "rows", A.row_dtype, true));
  DM_TRY(check_ld(op, "table", A.ld_table, A.dim));
  DM_TRY(check_ld(op, "rows", A.ld_rows, A.dim));
  const int table_elem = A.table_dtype == DMUON_DTYPE_BF16 ? 2 : 4;
  const Range r[] = {
      {A.ids, A.n_tokens * (A.id_dtype == DMUON_INDEX_I64 ? 8 : 4), false, "ids"},
      {A.table, span_bytes(A.vocab, A.dim, A.ld_table, table_elem), true, "table"},
      {A.rows, span_bytes(A.n_tokens, A.dim, A.ld_rows, A.row_dtype == DMUON_DTYPE_BF16 ? 2 : 4), false, "rows"},
  };
  DM_TRY(check_ranges(ctx, op, r, 3));
  DeviceGuard guard(ctx->device);
  DM_TRY(ensure_device(ctx));
  DM_TRY(check_pointers(ctx, r, 3));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool add = (A.flags & DMUON_EMBED_ADD) != 0;
  if (A.n_tokens == 0) {
    if (!add)
      DM_CUDA(cudaMemset2DAsync(A.table, static_cast<size_t>(A.ld_table * table_elem), 0,
                                static_cast<size_t>(A.dim * table_elem), static_cast<size_t>(A.vocab), s));
    return DMUON_OK;
  }
  const EmbedWs W = embed_backward_ws(A.n_tokens, static_cast<int32_t>(A.dim));
  DM_TRY(vocab_workspace(ctx, W.bytes, s));
  char* ws = static_cast<char*>(ctx->vocab_ws.p);
  EmbedBackward E = {};
  E.ids = IdList{A.ids, A.id_dtype == DMUON_INDEX_I64, static_cast<int32_t>(A.vocab)};
  E.n = A.n_tokens;
  E.dout = A.rows;
  E.ld_dout = A.ld_rows;
  E.dout_bf16 = A.row_dtype == DMUON_DTYPE_BF16;
  E.dtable = A.table;
  E.ld_dtable = A.ld_table;
  E.dtable_bf16 = A.table_dtype == DMUON_DTYPE_BF16;
  E.accumulate = add;
  E.dim = static_cast<int32_t>(A.dim);
  E.scale = A.scale;
  E.err = static_cast<int*>(ctx->err.p);
  for (int k = 0; k < 2; ++k) {
    E.key[k] = reinterpret_cast<uint32_t*>(ws + W.key[k]);
    E.pos[k] = reinterpret_cast<uint32_t*>(ws + W.pos[k]);
  }
  E.hist = reinterpret_cast<uint32_t*>(ws + W.hist);
  E.partial = reinterpret_cast<float*>(ws + W.partial);
  int launches = 0;
  DM_TRY(timed_launch(ctx, -1, s, [&] { return launch_embed_backward(E, &launches, s); }));
  ctx->launches += launches - 1;  // timed_launch counted one
  return vocab_used(ctx, s);
}

}  // extern "C"
