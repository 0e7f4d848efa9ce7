// Entry points of the vocabulary operators: argument checks, workspace layout
// and launch order of the cross entropy, the log probabilities and the embedding
// lookup (kernels: k_vocab_gemm.cu, k_vocab_thin.cu, k_vocab_ce.cu, k_logprobs.cu, k_embed.cu).
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
  int64_t rows, row_bytes, pitch;  // in bytes; a list is one row
  int elem;  // element size, and the alignment that kernels rely on
  bool written;
  const char* what;
  // Bytes from the first to the last element.
  int64_t bytes() const { return rows <= 0 || row_bytes <= 0 ? 0 : (rows - 1) * pitch + row_bytes; }
};

Range matrix(const void* p, int64_t rows, int64_t cols, int64_t ld, int elem, bool written, const char* what) {
  return Range{p, rows, cols * elem, ld * elem, elem, written, what};
}
Range list(const void* p, int64_t n, int elem, bool written, const char* what) {
  return Range{p, 1, n * elem, n * elem, elem, written, what};
}

// Whether two ranges share a byte.  Matrices of one pitch may be column ranges of
// one buffer, whose rows lie between one another; of two pitches the spans are compared.
bool share_bytes(const Range& a, const Range& b) {
  if (!a.p || !b.p || a.bytes() <= 0 || b.bytes() <= 0) return false;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  if (pa >= pb + static_cast<uintptr_t>(b.bytes()) || pb >= pa + static_cast<uintptr_t>(a.bytes())) return false;
  if (a.rows == 1 || b.rows == 1) {
    // One row against many of `pitch`: it may lie in a gap.
    const Range& one = a.rows == 1 ? a : b;
    const Range& many = a.rows == 1 ? b : a;
    if (many.rows == 1 || one.p < many.p) return true;
    const int64_t at = static_cast<int64_t>(reinterpret_cast<uintptr_t>(one.p) - reinterpret_cast<uintptr_t>(many.p)) % many.pitch;
    return at < many.row_bytes || at + one.row_bytes > many.pitch;
  }
  if (a.pitch != b.pitch) return true;
  const Range& lo = pa <= pb ? a : b;
  const Range& hi = pa <= pb ? b : a;
  // Row starts of `hi` lie `at` bytes past row starts of `lo`, or past where they would be.
  const int64_t at = static_cast<int64_t>(pa <= pb ? pb - pa : pa - pb) % a.pitch;
  return at < lo.row_bytes || at + hi.row_bytes > a.pitch;
}

// Alignment of each, and no written range shared with another.
int check_ranges(const char* op, const Range* r, int n) {
  char buf[200];
  for (int i = 0; i < n; ++i)
    if (reinterpret_cast<uintptr_t>(r[i].p) % static_cast<uintptr_t>(r[i].elem) != 0) {
      snprintf(buf, sizeof buf, "%s: %s is not aligned to its %d-byte elements", op, r[i].what, r[i].elem);
      return set_error(DMUON_ERR_INVALID_ARG, buf);
    }
  for (int i = 0; i < n; ++i)
    for (int j = i + 1; j < n; ++j) {
      if ((r[i].written || r[j].written) && share_bytes(r[i], r[j])) {
        snprintf(buf, sizeof buf, "%s: %s overlaps %s (memory the call writes must not be shared)", op, r[i].what,
                 r[j].what);
        return set_error(DMUON_ERR_INVALID_ARG, buf);
      }
    }
  return DMUON_OK;
}

int check_pointers(const dmuon_context* ctx, const Range* r, int n) {
  for (int i = 0; i < n; ++i) {
    if (!r[i].p || r[i].bytes() <= 0) continue;
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
// The scratch of the vocabulary and the gradient operators: grown on demand, shared by all
// their calls on the context.  A call on another stream than the last one waits for it;
// streams are told apart by their ids, since a handle may stand for another stream
// than before (cudaStreamPerThread in each thread; a handle freed and given out again).
}  // namespace

int vocab_workspace(dmuon_context* ctx, size_t bytes, cudaStream_t s) {
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  DM_CUDA(cudaStreamIsCapturing(s, &cap));
  if (cap == cudaStreamCaptureStatusNone && ctx->vocab_used) {
    unsigned long long id = 0;
    DM_CUDA(cudaStreamGetId(s, &id));
    if (id != ctx->vocab_stream) DM_CUDA(cudaStreamWaitEvent(s, ctx->vocab_done, 0));
  }
  if (bytes > ctx->vocab_ws.bytes) {
    if (ctx->vocab_captured || cap != cudaStreamCaptureStatusNone) {
      // Captured graphs point into the old scratch, and a capture refuses to free memory:
      // it lives as long as the context, and stays in use if there is no other to be had.
      DevBuf next;
      const int st = dev_alloc(next, bytes);
      if (st != DMUON_OK) return st;
      try {
        ctx->vocab_retired.push_back(ctx->vocab_ws);
      } catch (...) {
        next.release();
        return set_error(DMUON_ERR_NOMEM, "host allocation failed");
      }
      ctx->vocab_ws = next;
      ctx->vocab_captured = false;
    } else {
      const int st = dev_alloc(ctx->vocab_ws, bytes);  // frees the old first
      if (st != DMUON_OK) return st;
    }
  }
  if (!ctx->vocab_ticket.p) {
    const int st = dev_alloc_zeroed(ctx->vocab_ticket, 256);
    if (st != DMUON_OK) return st;
  }
  if (cap != cudaStreamCaptureStatusNone) ctx->vocab_captured = true;
  return DMUON_OK;
}

// After the last launch that uses the workspace, also of a call that broke off
// with `st`; returns the call's status.
int end_use(dmuon_context* ctx, cudaStream_t s, int st) {
  const auto note = [&] {
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    cudaError_t e = cudaStreamIsCapturing(s, &cap);
    if (e != cudaSuccess || cap != cudaStreamCaptureStatusNone) return e;
    if (!ctx->vocab_done) e = cudaEventCreateWithFlags(&ctx->vocab_done, cudaEventDisableTiming);
    if (e == cudaSuccess) e = cudaEventRecord(ctx->vocab_done, s);
    if (e == cudaSuccess) e = cudaStreamGetId(s, &ctx->vocab_stream);
    ctx->vocab_used = ctx->vocab_used || e == cudaSuccess;
    return e;
  };
  const cudaError_t e = note();
  return st != DMUON_OK || e == cudaSuccess ? st : cuda_fail(e, "end of a call that uses the shared scratch");
}

namespace {

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

// Tokens up to which d logits always come in two halves.
constexpr int kHalvesTokens = 128;

// The products that read W run on k_vocab_thin.cu where that is faster.
//  Logits, microseconds of a call there / on 256 x 256 tiles, W from HBM.  Scores: 162 / 248
//  with 1 token and 169 / 185 with 64 at 128256 x 4096, 39 / 65 and 51 / 55 at 128256 x 768,
//  8.2 / 11 with 1 and 12 / 11 with 64 at 8000 x 256, 41 / 49 with 48 and 46 / 42 with 64 at
//  128256 x 512: to 64 tokens, narrow heads to 48.  With logs to write, two bytes at a time
//  there (gradient calls): 160 / 186 with 1 and 165 / 171 with 32 at 32000 x 4096, 302 / 304
//  with 24 and 314 / 306 with 32 at 128256 x 2048, 548 / 546 with 32 at 128256 x 4096; of
//  narrow heads 71 / 78 with 32 at 50257 x 768, 111 / 115 with 8, 116 / 115 with 16 and
//  135 / 122 with 32 at 128256 x 512, 236 / 245 with 8 and 270 / 251 with 16 at 250000 x 768:
//  to 32 tokens, and where the main loop is too short to hide the stores to 2.2 million logs.
bool thin_logits_pay(int64_t tokens, int64_t vocab, int64_t dim, bool logs) {
  if (!logs) return tokens <= (dim < 768 ? 48 : 64);
  return tokens <= 32 && (dim >= 2048 || tokens * vocab <= 2200000);
}
//  dX (with dW and the sum of the partials), by rows of d logits (two a token up to
//  128 tokens): 37 / 37 with 16 rows at 50257 x 768 but 4 us more before it, 53 / 58
//  with 16 and 62 / 64 with 128 at 32000 x 2048, 62 / 63 with 128 at 60000 x 1024,
//  330 / 427 with 48 at 128256 x 4096.  With 200 rows 78 / 73 at 32000 x 2048,
//  128 / 127 at 32000 x 4096, 191 / 210 at 100000 x 2048; with 250 rows 134 / 124 at
//  30000 x 4096, 231 / 237 at 60000 x 4096, 452 / 490 at 128256 x 4096.
bool thin_dx(int64_t rows, int64_t vocab, int64_t dim) {
  const int64_t entries = vocab * dim;
  return rows <= kThinRows / 2 ? entries > 55000000 : rows <= kThinRows && entries > 180000000;
}

// Row tiles that go through the columns together, so that L2 keeps them while the
// other operand passes once for all.  Logits: 184 us with 16 at 4096 x 50257 x 768,
// 190 with 8; 32 take 67 MB of X at 8192 x 128256 x 4096 and 5.07 ms for 4.82.  dX:
// 16 and 32 are 1 and 4 % slower than 8 at 8192 x 32000 x 2048.  dW (rows are the
// vocabulary): 4 are 0.8 % faster than 8 there, 16 1 % slower.
constexpr int kLogitsGroup = 16, kDxGroup = 8, kDwGroup = 4;

// Tiles of at least this many k-blocks are drawn (k_vocab_gemm.cu): half a
// microsecond a tile against 9 us and more of work.
constexpr int kDrawnBlocks = 32;

int64_t tiles_of(int64_t n) { return (n + kVgTile - 1) / kVgTile; }

// Costs in k-blocks of one 256 x 256 tile (about 0.27 us on a pair): what a
// tile adds to its main loop, a further launch, and the way of a partial's
// bytes through memory (written, read).
constexpr double kTileCost = 6.0, kLaunchCost = 12.0, kPartialBytesPerUnit = 1.8e6;

// Parts of equal length (the last may be shorter) that K is cut into when about `parts` are wanted: none is empty.
int whole_parts(int64_t k, int64_t parts) {
  const int64_t kb = (k + 63) / 64, step = (kb + parts - 1) / parts;
  return static_cast<int>((kb + step - 1) / step);
}

// Parts that the K axis of an M x N product is cut into.  Few output tiles
// leave pairs idle, and `other` k-blocks of further tiles share the launch;
// every part costs a pass of its fp32 partial through memory.
int choose_splits(int64_t m, int64_t n, int64_t k, double other, int pairs, bool need_partial) {
  const int64_t tiles = tiles_of(m) * tiles_of(n);
  const int64_t kb = (k + 63) / 64;
  double best = 0.0;
  int parts = 1;
  for (int s = 1; s <= 64 && s <= kb; ++s) {
    const double unit = static_cast<double>((kb + s - 1) / s) + kTileCost;
    const double units = static_cast<double>(tiles * s);
    // The pairs finish together, but not before the longest column of whole units.
    const double waves = std::ceil(units / pairs);
    double cost = other > 0 ? std::max((units * unit + other) / pairs, std::max(1.0, std::floor(units / pairs)) * unit) : waves * unit;
    if (s > 1 || need_partial) cost += kLaunchCost + static_cast<double>(m) * static_cast<double>(n) * 4.0 * (2.0 * s + 1.0) / kPartialBytesPerUnit;
    if (s == 1 || cost < best * 0.97) {
      best = cost;
      parts = s;
    }
  }
  return whole_parts(k, parts);
}

int encode_2d(EncodeTiledFn enc, CUtensorMap* map, const void* p, int64_t inner, int64_t rows, int64_t ld, uint32_t box_inner,
              uint32_t box_rows) {
  return make_map_typed(enc, map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p, inner, rows, 1, ld, rows * ld, box_inner, box_rows);
}

// A gradient's way out: written by its product, or as fp32 partials that a
// further kernel joins (several parts of K, two halves to fold, or a bf16 sum
// over passes).
struct Target {
  void* out = nullptr;
  int64_t ld = 0;
  bool bf16 = false, keep = false;
  int splits = 1;
  float* part = nullptr;
  int64_t ld_part = 0;
};

// Product D (m x n) = A B into T; `first`: first pass over the rows.
int encode_product(EncodeTiledFn enc, VgProduct* P, int64_t m, int64_t n, int64_t k, bool a_mn, const void* a, int64_t ld_a,
                   const void* b, int64_t ld_b, const Target& T, int splits, int group_m, bool first) {
  P->M = static_cast<int32_t>(m);
  P->N = static_cast<int32_t>(n);
  P->grid.set(m, n, k, splits, group_m);
  P->a_mn = a_mn;
  if (a_mn)
    DM_TRY(encode_2d(enc, &P->map_a, a, m, k, ld_a, 64, 64));
  else
    DM_TRY(encode_2d(enc, &P->map_a, a, k, m, ld_a, 64, 128));
  DM_TRY(encode_2d(enc, &P->map_b, b, n, k, ld_b, 64, 64));
  if (T.part) {
    P->add = !first;
    return make_map_typed(enc, &P->map_out, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, T.part, n, m, P->grid.splits, T.ld_part, m * T.ld_part, 32, 32);
  }
  P->out_bf16 = T.bf16;
  P->add = T.keep || !first;
  P->direct = !tma_rows(T.out, T.ld, T.bf16 ? 2 : 4) || (T.bf16 && P->add);
  P->out = T.out;
  P->ld_out = T.ld;
  if (P->direct) return DMUON_OK;
  if (T.bf16) return encode_2d(enc, &P->map_out, T.out, n, m, T.ld, 64, 32);
  return make_map_typed(enc, &P->map_out, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, T.out, n, m, 1, T.ld, m * T.ld, 32, 32);
}

// Cross entropy, or with P the log probabilities of the given tokens (C holds the
// arguments that both have).
int head_impl(dmuon_context* ctx, const dmuon_ce& C, const dmuon_logprobs* P, cudaStream_t s) {
  const int64_t n = C.n_tokens, v = C.vocab, d = C.dim;
  const bool grads = C.dx || C.dw;
  const int n_top = P && P->top_ids ? P->n_top : 0;
  const bool keep_logs = grads || n_top > 0;
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

  // Few tokens: a 256-row tile has room for d logits in two bf16 halves (value
  // and the rounding's rest), so they come at no cost, and with as few terms in
  // the gradients' sums one rounding would not average out.  More tokens take
  // them where the caller asks for it: both gradient products are then twice as
  // long, and what is left of a d logit's error is that of its 16-bit log.
  const bool halves = grads && (n <= kHalvesTokens || (C.flags & DMUON_CE_FINE_GRADS) != 0);

  // Rows of one pass: what is held for each (its logs, or without gradients and alternatives its
  // statistics) stays within the limit, and tiles are numbered in 32 bits.
  const int64_t ld_block = round_up(v, 64);
  const bool thin_logits = thin_logits_pay(n, v, d, keep_logs), coarse = n_top > 0 && !grads && !thin_logits;
  const int64_t row_bytes = (keep_logs ? (halves ? 4 : coarse ? 1 : 2) * ld_block : (P ? 12 : 8) * ((v + kCeBlock - 1) / kCeBlock)) +
                            (n_top > 0 ? static_cast<int64_t>(kTopBlocks * sizeof(TopBlock)) : 0);
  const int64_t most = std::max<int64_t>(kVgTile, std::min(ctx->tune.ce_block_bytes / row_bytes,
                                                           (int64_t(1) << 30) / tiles_of(v) * kVgTile) / kVgTile * kVgTile);
  int64_t rows = n;
  if (n > most) {
    const int64_t passes = (n + most - 1) / most;
    rows = round_up((n + passes - 1) / passes, kVgTile);
  }
  const bool one_pass = rows >= n;
  const int64_t token_rows = halves ? 2 * rows : rows;
  const bool thin_x = C.dx && thin_dx(token_rows, v, d);
  const int stats_shift = thin_logits ? kCeThinShift : kCeShift, stats_block = 1 << stats_shift;
  const bool rows_make_dlogits = !P && halves && ce_rows_make_dlogits(n);
  const int n_blocks = static_cast<int>((v + stats_block - 1) / stats_block);
  const int64_t stats_ld = rows >= 4 ? round_up(rows, 4) : rows;

  // Operand copies: TMA needs rows on 16 bytes, and rows that are not counted
  // must read as zeros in dW's product whatever they hold (the row pass makes
  // that copy where none is needed before it).  Rows off 128 bytes cost the
  // products on 256 x 256 tiles twice the L2 lines: with x at a pitch of 1000
  // elements the logits of 4000 x 32003 took 237 us, at 1024 they take 186.
  // x is small next to what it is multiplied by; a copy of w would cost as
  // much as it gains (20 of 186 us there).
  const bool off_lines = n >= 256 && d >= 128 && ((reinterpret_cast<uintptr_t>(C.x) | static_cast<uintptr_t>(C.ld_x * 2)) & 127u) != 0;
  const bool copy_x = off_lines || !tma_rows(C.x, C.ld_x, 2), copy_w = !tma_rows(C.w, C.ld_w, 2);
  const bool masked_first = copy_x && C.dw && !halves;  // that copy serves dW's product too
  const int64_t ld8 = round_up(d, n >= 256 ? 64 : 8), ld4 = round_up(d, 4);
  Layout L;
  const size_t off_x = copy_x ? L.take(static_cast<size_t>(n * ld8) * 2) : 0;
  const size_t off_w = copy_w ? L.take(static_cast<size_t>(v * ld8) * 2) : 0;
  const size_t off_stats = L.take(static_cast<size_t>(n_blocks * stats_ld) * sizeof(float2));
  const size_t off_weighted = P ? L.take(static_cast<size_t>(n_blocks * stats_ld) * sizeof(float)) : 0;
  const int width = ce_rows_width(n);
  const size_t off_partial = C.total ? L.take(static_cast<size_t>((n + width - 1) / width) * sizeof(double2)) : 0;
  size_t off_block = 0, off_rows = 0, off_alpha = 0, off_masked = 0, off_dx = 0, off_dw = 0;
  Target dx, dw;
  if (keep_logs) off_block = L.take(static_cast<size_t>(token_rows * ld_block) * (coarse ? 1 : 2));
  if (grads || P) off_rows = L.take(static_cast<size_t>(rows) * (P ? sizeof(LpRow) : sizeof(CeRow)));
  const size_t off_top = n_top > 0 ? L.take(static_cast<size_t>(rows) * kTopBlocks * sizeof(TopBlock)) : 0;
  const int32_t norm_groups = static_cast<int32_t>(round_up((v + kNormRows - 1) / kNormRows, 4));
  const size_t off_norms = n_top > 0 ? L.take(static_cast<size_t>(norm_groups) * sizeof(float)) : 0;
  if (grads) {
    off_alpha = L.take(4);
    bool dx_part = false, dw_part = false;
    if (C.dw) {
      if (!masked_first) off_masked = L.take(static_cast<size_t>(token_rows * ld8) * 2);
      dw.out = C.dw;
      dw.ld = C.ld_dw;
      dw.bf16 = dw_bf16;
      dw.keep = add_dw;
      dw_part = dw_bf16 && !one_pass;
      dw.splits = choose_splits(v, d, token_rows, 0.0, pairs, dw_part);
      dw_part = dw_part || dw.splits > 1;
      dw.ld_part = ld4;
      if (dw_part) off_dw = L.take(static_cast<size_t>(dw.splits * v * ld4) * 4);
    }
    if (C.dx) {
      dx.bf16 = dx_bf16;
      dx.ld = C.ld_dx;
      dx_part = halves || thin_x;
      if (thin_x) {
        // Tiles of 128 columns; parts of the vocabulary for a few tiles per SM.
        const int64_t tiles = (d + 127) / 128, kb = (v + 63) / 64;
        int64_t parts = (2 * ctx->num_sms + tiles - 1) / tiles;
        // Whole waves of CTAs, but at least 8 k-blocks in a part.
        if (parts * tiles > ctx->num_sms) parts = std::max<int64_t>(1, (2 * ctx->num_sms) / tiles);
        dx.splits = whole_parts(v, std::max<int64_t>(1, std::min<int64_t>(parts, kb / 8)));
      } else {
        const double other = C.dw ? static_cast<double>(tiles_of(v) * tiles_of(d) * dw.splits) *
                                        (static_cast<double>((token_rows + 63) / 64) / dw.splits + kTileCost)
                                  : 0.0;
        dx.splits = choose_splits(token_rows, d, v, other, pairs, dx_part);
      }
      dx_part = dx_part || dx.splits > 1;
      dx.ld_part = ld4;
      if (dx_part) off_dx = L.take(static_cast<size_t>(dx.splits * token_rows * ld4) * 4);
    }
    DM_TRY(vocab_workspace(ctx, L.bytes, s));
    char* ws = static_cast<char*>(ctx->vocab_ws.p);
    if (dx_part) dx.part = reinterpret_cast<float*>(ws + off_dx);
    if (dw_part) dw.part = reinterpret_cast<float*>(ws + off_dw);
  } else {
    DM_TRY(vocab_workspace(ctx, L.bytes, s));
  }
  char* ws = static_cast<char*>(ctx->vocab_ws.p);
  int* err = static_cast<int*>(ctx->err.p);
  const IdList ids{C.targets, C.target_dtype == DMUON_INDEX_I64, static_cast<int32_t>(v)};
  const uint16_t* x = C.x;
  const uint16_t* w = C.w;
  int64_t ld_x = C.ld_x, ld_w = C.ld_w;
  if (copy_x) {
    uint16_t* to = reinterpret_cast<uint16_t*>(ws + off_x);
    DM_TRY(timed_launch(ctx, -1, s, [&] { return launch_ce_copy(C.x, C.ld_x, to, ld8, n, static_cast<int32_t>(d), masked_first ? ids : IdList{}, s); }));
    x = to;
    ld_x = ld8;
  }
  if (copy_w) {
    uint16_t* to = reinterpret_cast<uint16_t*>(ws + off_w);
    DM_TRY(timed_launch(ctx, -1, s, [&] { return launch_ce_copy(C.w, C.ld_w, to, ld8, v, static_cast<int32_t>(d), IdList{}, s); }));
    w = to;
    ld_w = ld8;
  }
  float2* stats = reinterpret_cast<float2*>(ws + off_stats);
  uint16_t* block = reinterpret_cast<uint16_t*>(ws + off_block);
  float* weighted = reinterpret_cast<float*>(ws + off_weighted);
  CeRow* row_info = reinterpret_cast<CeRow*>(ws + off_rows);
  LpRow* lp_info = reinterpret_cast<LpRow*>(ws + off_rows);
  float* norms = n_top > 0 ? reinterpret_cast<float*>(ws + off_norms) : nullptr;
  float* alpha = reinterpret_cast<float*>(ws + off_alpha);
  uint16_t* masked = reinterpret_cast<uint16_t*>(ws + off_masked);
  uint32_t* counters = static_cast<uint32_t*>(ctx->vocab_ticket.p);  // two tile counters, one ticket
  const double scale_log2 = C.logit_scale * 1.4426950408889634;
  CeNorm norm = {};
  norm.alpha = grads ? alpha : nullptr;
  norm.targets = ids;
  norm.weights = C.weights;
  norm.n = n;
  norm.mean = mean;
  norm.scale = C.grad_scale * C.logit_scale;
  double2* partial = C.total ? reinterpret_cast<double2*>(ws + off_partial) : nullptr;
  const CeTotal total = {C.total, partial, (n + width - 1) / width, mean};
  const bool side_sums = n <= kSideSums;
  if (grads && !side_sums) {
    DM_TRY(timed_launch(ctx, -1, s, [&] { return launch_ce_norm(norm, s); }));
    norm.alpha = nullptr;
  }
  const bool total_later = side_sums && (C.dw || (C.dx && !thin_x));  // the gradients' kernel writes it

  for (int64_t r0 = 0; r0 < n; r0 += rows) {
    const int64_t nr = std::min(rows, n - r0);
    const bool first = r0 == 0, last = r0 + rows >= n;
    const int64_t k_rows = halves ? 2 * nr : nr;  // rows of d logits
    IdList here = ids;
    int32_t steps = static_cast<int32_t>((d + 15) / 16);
    if (ids.p) here.p = static_cast<const char*>(ids.p) + r0 * (ids.is64 ? 8 : 4);
    if (thin_logits) {
      VocabThin G = {};
      G.M = static_cast<int32_t>(v);
      G.tokens = static_cast<int32_t>(nr);
      G.np = static_cast<int32_t>(round_up(nr, 16));
      G.tiles_m = static_cast<int32_t>((v + 127) / 128);
      G.splits = 1;
      G.kb_total = G.kb_step = static_cast<int32_t>((d + 63) / 64);
      G.groups = std::max(1, std::min({4, G.kb_total / 16, 256 / G.np}));
      steps = 4 * ((G.kb_total + G.groups - 1) / G.groups);
      G.err = err;
      DM_TRY(encode_2d(enc, &G.map_a, w, d, v, ld_w, 64, 128));
      DM_TRY(encode_2d(enc, &G.map_b, x, d, nr, ld_x, 64, static_cast<uint32_t>(G.np)));
      G.logit_scale_log2 = static_cast<float>(scale_log2);
      G.logs = keep_logs ? block : nullptr;
      G.ld_logs = ld_block;
      G.stats = stats;
      G.stats_ld = stats_ld;
      G.targets = here;
      if (P) G.weighted = weighted;
      G.norms = norms;
      if (first) G.norm = norm;
      DM_TRY(timed_launch(ctx, -1, s, [&] { return launch_vocab_thin(true, G, ctx->num_sms, s); }));
    } else {
      VocabLogTop G = {};
      G.M = static_cast<int32_t>(nr);
      G.N = static_cast<int32_t>(v);
      G.grid.set(nr, v, d, 1, kLogitsGroup);
      G.err = err;
      DM_TRY(encode_2d(enc, &G.map_a, x + r0 * ld_x, d, nr, ld_x, 64, 128));
      DM_TRY(encode_2d(enc, &G.map_b, w, d, v, ld_w, 64, 128));
      G.logit_scale_log2 = static_cast<float>(scale_log2);
      G.logs = keep_logs ? block : nullptr;
      G.ld_logs = ld_block;
      G.stats = stats;
      G.stats_ld = stats_ld;
      G.targets = here;
      G.counter = counters;
      if (first) G.norm = norm;
      G.weighted = weighted;
      G.norms = first ? norms : nullptr;
      G.drawn = G.grid.kb_total >= kDrawnBlocks;
      DM_TRY(timed_launch(ctx, -1, s, [&] {
        return coarse ? launch_vocab_logits(G, pairs, s)
               : P    ? launch_vocab_logits(static_cast<const VocabLogProbs&>(G), pairs, s)
                      : launch_vocab_logits(static_cast<const VocabLogits&>(G), pairs, s);
      }));
    }

    if (P) {
      LpRows R = {};
      R.stats = stats;
      R.weighted = weighted;
      R.stats_ld = stats_ld;
      R.n_blocks = n_blocks;
      R.row0 = r0;
      R.rows = nr;
      R.tokens = ids;
      R.dlogprobs = grads ? P->dlogprobs : nullptr;
      R.dentropy = grads ? P->dentropy : nullptr;
      R.x = x + r0 * ld_x;
      R.w = w;
      R.ld_x = ld_x;
      R.ld_w = ld_w;
      R.dim = static_cast<int32_t>(d);
      R.vocab = static_cast<int32_t>(v);
      R.logit_scale_log2 = scale_log2;
      R.logprobs = P->logprobs;
      R.lse = P->lse;
      R.entropy = P->entropy;
      R.out = lp_info;
      R.x_copy = C.dw && !masked_first ? masked : nullptr;
      R.ld_copy = ld8;
      R.copies = halves ? 2 : 1;
      R.width = width;
      R.counters = counters;
      R.err = err;
      R.k = n_top;
      R.top_blocks = reinterpret_cast<TopBlock*>(ws + off_top);
      R.norms = norms;
      R.stats_shift = stats_shift;
      R.steps = steps;
      LpTop T = {};
      T.block = block;
      T.coarse = coarse;
      T.ld_block = ld_block;
      T.stats = stats;
      T.stats_ld = stats_ld;
      T.n_blocks = n_blocks;
      T.stats_shift = stats_shift;
      T.vocab = static_cast<int32_t>(v);
      T.rows_in = lp_info;
      T.top_blocks = R.top_blocks;
      T.norms = norms;
      T.rows = nr;
      T.x = R.x;
      T.w = w;
      T.ld_x = ld_x;
      T.ld_w = ld_w;
      T.dim = R.dim;
      T.logit_scale_log2 = scale_log2;
      T.k = n_top;
      T.ids64 = P->top_dtype == DMUON_INDEX_I64;
      if (n_top > 0) T.ids = static_cast<char*>(P->top_ids) + r0 * n_top * (T.ids64 ? 8 : 4);
      T.logprobs = P->top_logprobs ? P->top_logprobs + r0 * n_top : nullptr;
      bool top_done = false;
      DM_TRY(timed_launch(ctx, -1, s, [&] { return launch_lp_rows(R, T, &top_done, s); }));
      if (n_top > 0 && !top_done) DM_TRY(timed_launch(ctx, -1, s, [&] { return launch_lp_top(T, s); }));
      if (!grads) continue;
      DM_TRY(timed_launch(ctx, -1, s, [&] {
        return launch_lp_dlogits(block, ld_block, nr, static_cast<int32_t>(v), stats_shift, stats, stats_ld, lp_info,
                                 halves ? nr : 0, s);
      }));
    } else {
      CeRows R = {};
      R.stats = stats;
      R.stats_ld = stats_ld;
      R.n_blocks = n_blocks;
      R.row0 = r0;
      R.rows = nr;
      R.targets = ids;
      R.weights = C.weights;
      R.x = x + r0 * ld_x;
      R.w = w;
      R.ld_x = ld_x;
      R.ld_w = ld_w;
      R.dim = static_cast<int32_t>(d);
      R.logit_scale_log2 = scale_log2;
      R.out = grads ? row_info : nullptr;
      if (rows_make_dlogits) {
        R.block = block;
        R.ld_block = ld_block;
        R.lo_rows = nr;
        R.vocab = static_cast<int32_t>(v);
        R.stats_shift = stats_shift;
      }
      R.loss = C.loss;
      R.lse = C.lse;
      R.x_copy = C.dw && !masked_first ? masked : nullptr;
      R.ld_copy = ld8;
      R.copies = halves ? 2 : 1;
      R.width = width;
      R.partial = partial;
      if (last && !total_later) R.total = total;
      R.ticket = counters + 2;
      R.counters = counters;
      R.err = err;
      DM_TRY(timed_launch(ctx, -1, s, [&] { return launch_ce_rows(R, s); }));
      if (!grads) continue;

      if (!rows_make_dlogits)
        DM_TRY(timed_launch(ctx, -1, s, [&] {
          return launch_ce_dlogits(block, ld_block, nr, static_cast<int32_t>(v), stats_shift, stats, stats_ld, row_info,
                                   halves ? nr : 0, s);
        }));
    }
    if (C.dx) dx.out = static_cast<char*>(C.dx) + r0 * C.ld_dx * (dx_bf16 ? 2 : 4);
    VocabGrad G = {};
    G.counter = counters + 1;
    G.alpha = alpha;
    if (last && total_later) G.total = total;
    G.err = err;
    if (thin_x) {
      VocabThin T = {};
      T.M = static_cast<int32_t>(d);
      T.tokens = static_cast<int32_t>(k_rows);
      T.np = static_cast<int32_t>(round_up(k_rows, 16));
      T.tiles_m = static_cast<int32_t>((d + 127) / 128);
      T.kb_total = static_cast<int32_t>((v + 63) / 64);
      T.kb_step = (T.kb_total + dx.splits - 1) / dx.splits;
      T.splits = dx.splits;
      T.groups = 1;
      T.err = err;
      DM_TRY(encode_2d(enc, &T.map_a, w, d, v, ld_w, 64, 64));
      DM_TRY(encode_2d(enc, &T.map_b, block, v, k_rows, ld_block, 64, static_cast<uint32_t>(T.np)));
      T.part = dx.part;
      T.ld_part = dx.ld_part;
      DM_TRY(timed_launch(ctx, -1, s, [&] { return launch_vocab_thin(false, T, ctx->num_sms, s); }));
    } else if (C.dx) {
      DM_TRY(encode_product(enc, &G.p[0], k_rows, d, v, false, block, ld_block, w, ld_w, dx, dx.splits, kDxGroup, true));
      G.n_units[0] = G.p[0].grid.count();
    }
    if (C.dw) {
      // The last pass may be shorter: every part needs a k-block of its own,
      // and the parts it leaves out hold the earlier passes' sums.
      const int splits = static_cast<int>(std::min<int64_t>(dw.splits, (k_rows + 63) / 64));
      DM_TRY(encode_product(enc, &G.p[1], v, d, k_rows, true, block, ld_block, masked_first ? x + r0 * ld_x : masked, ld8, dw, splits, kDwGroup, first));
      G.n_units[1] = G.p[1].grid.count();
    }
    if (G.n_units[1] > 0) {
      const int u1 = G.p[1].grid.kb_step;
      G.drawn = u1 >= kDrawnBlocks;
      if (G.n_units[0] % pairs != 0)
        G.extra = static_cast<int32_t>((G.p[0].grid.kb_step + kTileCost) / (u1 + kTileCost) + 0.5);
    } else {
      G.drawn = 1;
    }
    if (G.n_units[0] + G.n_units[1] > 0)
      DM_TRY(timed_launch(ctx, -1, s, [&] { return launch_vocab_grad(G, pairs, s); }));
    if (dx.part)
      DM_TRY(timed_launch(ctx, -1, s, [&] {
        // The tile kernel has applied alpha already.
        return launch_ce_finish(dx.part, dx.ld_part, k_rows * dx.ld_part, dx.splits, halves ? nr : 0, dx.out, dx.ld, dx.bf16, 0,
                                thin_x ? alpha : nullptr, nr, static_cast<int32_t>(d), s);
      }));
    if (dw.part && last)
      DM_TRY(timed_launch(ctx, -1, s, [&] {
        return launch_ce_finish(dw.part, dw.ld_part, v * dw.ld_part, dw.splits, 0, C.dw, C.ld_dw, dw_bf16, add_dw, nullptr, v,
                                static_cast<int32_t>(d), s);
      }));
  }
  return DMUON_OK;
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
  if (C.flags & ~uint32_t(DMUON_CE_MEAN | DMUON_CE_ADD_DW | DMUON_CE_FINE_GRADS))
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
  const int id_size = C.target_dtype == DMUON_INDEX_I64 ? 8 : 4;
  const int dx_size = C.dx_dtype == DMUON_DTYPE_BF16 ? 2 : 4, dw_size = C.dw_dtype == DMUON_DTYPE_BF16 ? 2 : 4;
  const Range r[] = {
      matrix(C.x, C.n_tokens, C.dim, C.ld_x, 2, false, "x"),
      matrix(C.w, C.vocab, C.dim, C.ld_w, 2, false, "w"),
      list(C.targets, C.n_tokens, id_size, false, "targets"),
      list(C.weights, C.n_tokens, 4, false, "weights"),
      list(C.loss, C.n_tokens, 4, true, "loss"),
      list(C.lse, C.n_tokens, 4, true, "lse"),
      list(C.total, 1, 4, true, "total"),
      matrix(C.dx, C.n_tokens, C.dim, C.ld_dx, dx_size, true, "dx"),
      matrix(C.dw, C.vocab, C.dim, C.ld_dw, dw_size, true, "dw"),
  };
  const int nr = static_cast<int>(sizeof r / sizeof r[0]);
  DM_TRY(check_ranges(op, r, nr));
  DeviceGuard guard(ctx->device);
  DM_TRY(ensure_device(ctx));
  DM_TRY(check_pointers(ctx, r, nr));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int st = head_impl(ctx, C, nullptr, s);
  if (C.n_tokens == 0) return st;  // no scratch
  // A sequence that broke off may have left its counters up.
  if (st != DMUON_OK && ctx->vocab_ticket.p) cudaMemsetAsync(ctx->vocab_ticket.p, 0, 256, s);
  return end_use(ctx, s, st);
}

int dmuon_token_logprobs(dmuon_context* ctx, const dmuon_logprobs* args, void* stream) {
  clear_error();
  if (!ctx || !args) return set_error(DMUON_ERR_INVALID_ARG, "token_logprobs: null context or arguments");
  const dmuon_logprobs& P = *args;
  const char* op = "token_logprobs";
  DM_TRY(check_sizes(op, P.n_tokens, P.vocab, P.dim));
  const bool grads = P.dx || P.dw;
  // An empty list may come without memory.
  const bool some = P.n_tokens > 0;
  if (!P.w || (some && !P.x)) return set_error(DMUON_ERR_INVALID_ARG, "token_logprobs: null x or w");
  if (some && !P.logprobs && !P.lse && !P.entropy && !P.top_ids && !grads)
    return set_error(DMUON_ERR_INVALID_ARG, "token_logprobs: no output asked for");
  if (some && !P.tokens && (P.logprobs || P.dlogprobs))
    return set_error(DMUON_ERR_INVALID_ARG, "token_logprobs: log probabilities and their gradients need tokens");
  if (some && grads && !P.dlogprobs && !P.dentropy)
    return set_error(DMUON_ERR_INVALID_ARG, "token_logprobs: dx and dw need dlogprobs or dentropy");
  if (some && !grads && (P.dlogprobs || P.dentropy))
    return set_error(DMUON_ERR_INVALID_ARG, "token_logprobs: dlogprobs and dentropy without dx or dw");
  if (some && !P.top_ids && (P.n_top != 0 || P.top_logprobs))
    return set_error(DMUON_ERR_INVALID_ARG, "token_logprobs: alternatives asked for without top_ids");
  if (P.top_ids && (P.n_top < 1 || P.n_top > kTopMost || P.n_top > P.vocab))
    return set_error(DMUON_ERR_INVALID_ARG, "token_logprobs: n_top outside [1, min(32, vocab)]");
  if (!finite(P.logit_scale) || P.logit_scale <= 0.f || !finite(P.grad_scale))
    return set_error(DMUON_ERR_INVALID_ARG, "token_logprobs: logit_scale must be positive, grad_scale finite");
  if (P.flags & ~uint32_t(DMUON_CE_ADD_DW | DMUON_CE_FINE_GRADS))
    return set_error(DMUON_ERR_INVALID_ARG, "token_logprobs: unknown flag bits");
  DM_TRY(check_type(op, "x", P.x_dtype, false));
  DM_TRY(check_type(op, "w", P.w_dtype, false));
  if (P.tokens) DM_TRY(check_index(op, P.token_dtype));
  if (P.top_ids) DM_TRY(check_index(op, P.top_dtype));
  DM_TRY(check_ld(op, "x", P.ld_x, P.dim));
  DM_TRY(check_ld(op, "w", P.ld_w, P.dim));
  if (P.dx) {
    DM_TRY(check_type(op, "dx", P.dx_dtype, true));
    DM_TRY(check_ld(op, "dx", P.ld_dx, P.dim));
  }
  if (P.dw) {
    DM_TRY(check_type(op, "dw", P.dw_dtype, true));
    DM_TRY(check_ld(op, "dw", P.ld_dw, P.dim));
  }
  const int64_t n = P.n_tokens, n_top = P.top_ids ? P.n_top : 0;
  const int dx_size = P.dx_dtype == DMUON_DTYPE_BF16 ? 2 : 4, dw_size = P.dw_dtype == DMUON_DTYPE_BF16 ? 2 : 4;
  const Range r[] = {
      matrix(P.x, n, P.dim, P.ld_x, 2, false, "x"),
      matrix(P.w, P.vocab, P.dim, P.ld_w, 2, false, "w"),
      list(P.tokens, n, P.token_dtype == DMUON_INDEX_I64 ? 8 : 4, false, "tokens"),
      list(P.dlogprobs, n, 4, false, "dlogprobs"),
      list(P.dentropy, n, 4, false, "dentropy"),
      list(P.logprobs, n, 4, true, "logprobs"),
      list(P.lse, n, 4, true, "lse"),
      list(P.entropy, n, 4, true, "entropy"),
      list(P.top_ids, n * n_top, P.top_dtype == DMUON_INDEX_I64 ? 8 : 4, true, "top_ids"),
      list(P.top_logprobs, n * n_top, 4, true, "top_logprobs"),
      matrix(P.dx, n, P.dim, P.ld_dx, dx_size, true, "dx"),
      matrix(P.dw, P.vocab, P.dim, P.ld_dw, dw_size, true, "dw"),
  };
  const int nr = static_cast<int>(sizeof r / sizeof r[0]);
  DM_TRY(check_ranges(op, r, nr));
  dmuon_ce C = {};
  C.n_tokens = n;
  C.vocab = P.vocab;
  C.dim = P.dim;
  C.x = P.x;
  C.w = P.w;
  C.ld_x = P.ld_x;
  C.ld_w = P.ld_w;
  C.targets = P.tokens;
  C.dx = P.dx;
  C.dw = P.dw;
  C.ld_dx = P.ld_dx;
  C.ld_dw = P.ld_dw;
  C.target_dtype = P.token_dtype;
  C.dx_dtype = P.dx_dtype;
  C.dw_dtype = P.dw_dtype;
  C.logit_scale = P.logit_scale;
  C.grad_scale = P.grad_scale;
  C.flags = P.flags;
  DeviceGuard guard(ctx->device);
  DM_TRY(ensure_device(ctx));
  DM_TRY(check_pointers(ctx, r, nr));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int st = head_impl(ctx, C, &P, s);
  if (n == 0) return st;  // no scratch
  // A sequence that broke off may have left its counters up.
  if (st != DMUON_OK && ctx->vocab_ticket.p) cudaMemsetAsync(ctx->vocab_ticket.p, 0, 256, s);
  return end_use(ctx, s, st);
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
  const int id_size = A.id_dtype == DMUON_INDEX_I64 ? 8 : 4;
  const int table_elem = A.table_dtype == DMUON_DTYPE_BF16 ? 2 : 4, row_elem = A.row_dtype == DMUON_DTYPE_BF16 ? 2 : 4;
  const Range r[] = {
      list(A.ids, A.n_tokens, id_size, false, "ids"),
      matrix(A.table, A.vocab, A.dim, A.ld_table, table_elem, false, "table"),
      matrix(A.rows, A.n_tokens, A.dim, A.ld_rows, row_elem, true, "rows"),
  };
  DM_TRY(check_ranges(op, r, 3));
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
  const int id_size = A.id_dtype == DMUON_INDEX_I64 ? 8 : 4;
  const int table_elem = A.table_dtype == DMUON_DTYPE_BF16 ? 2 : 4, row_elem = A.row_dtype == DMUON_DTYPE_BF16 ? 2 : 4;
  const Range r[] = {
      list(A.ids, A.n_tokens, id_size, false, "ids"),
      matrix(A.table, A.vocab, A.dim, A.ld_table, table_elem, true, "table"),
      matrix(A.rows, A.n_tokens, A.dim, A.ld_rows, row_elem, false, "rows"),
  };
  DM_TRY(check_ranges(op, r, 3));
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
  const EmbedWs W = embed_backward_ws(A.n_tokens, A.vocab, static_cast<int32_t>(A.dim));
  if (W.bytes > 0) DM_TRY(vocab_workspace(ctx, W.bytes, s));
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
  E.present = add ? nullptr : reinterpret_cast<uint32_t*>(ws + W.present);
  E.partial = reinterpret_cast<float*>(ws + W.partial);
  int launches = 0;
  const int st = timed_launch(ctx, -1, s, [&] { return launch_embed_backward(E, &launches, s); });
  if (st == DMUON_OK) ctx->launches += launches - 1;  // timed_launch counted one
  return W.bytes > 0 ? end_use(ctx, s, st) : st;
}

}  // extern "C"
