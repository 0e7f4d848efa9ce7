// Entry points of the gradient operators: norms of many tensors and clipping
// (kernels: k_grads.cu).
#include "grads.h"

#include "runtime.h"

#include <new>

namespace dmuon {
namespace {

#define DM_TRY(call)                    \
  do {                                  \
    const int st_ = (call);             \
    if (st_ != DMUON_OK) return st_;    \
  } while (0)

constexpr int64_t kLongChunk = 131072;  // bytes of a chunk of a large call

int64_t elem_size(int32_t dtype) { return dtype == DMUON_DTYPE_BF16 ? 2 : 4; }

int validate_grads(const char* op, const dmuon_grad* gs, int32_t n, bool outs) {
  char buf[200];
  if (n < 0 || (n > 0 && !gs)) {
    snprintf(buf, sizeof buf, "%s: bad tensor list", op);
    return set_error(DMUON_ERR_INVALID_ARG, buf);
  }
  if (n > (1 << 24)) {
    snprintf(buf, sizeof buf, "%s: more than 2^24 tensors", op);
    return set_error(DMUON_ERR_SHAPE, buf);
  }
  for (int i = 0; i < n; ++i) {
    const dmuon_grad& g = gs[i];
    if (g.numel < 0 || g.numel > (int64_t(1) << 40)) {
      snprintf(buf, sizeof buf, "%s: tensor %d: numel %lld", op, i, (long long)g.numel);
      return set_error(DMUON_ERR_SHAPE, buf);
    }
    if ((g.grad_dtype != DMUON_DTYPE_F32 && g.grad_dtype != DMUON_DTYPE_BF16) ||
        (outs && g.out_dtype != DMUON_DTYPE_F32 && g.out_dtype != DMUON_DTYPE_BF16)) {
      snprintf(buf, sizeof buf, "%s: tensor %d: dtype", op, i);
      return set_error(DMUON_ERR_DTYPE, buf);
    }
    if (g.numel > 0 && (!g.grad || (outs && !g.out))) {
      snprintf(buf, sizeof buf, "%s: tensor %d: null grad%s", op, i, outs ? " or out" : "");
      return set_error(DMUON_ERR_INVALID_ARG, buf);
    }
    if (reinterpret_cast<uintptr_t>(g.grad) % elem_size(g.grad_dtype) != 0 ||
        (outs && reinterpret_cast<uintptr_t>(g.out) % elem_size(g.out_dtype) != 0)) {
      snprintf(buf, sizeof buf, "%s: tensor %d is not aligned to its elements", op, i);
      return set_error(DMUON_ERR_INVALID_ARG, buf);
    }
  }
  return DMUON_OK;
}

struct Span {
  uintptr_t lo, hi;
  int idx;  // -1: one of the call's results
  bool written;
};

// Memory that the call writes is shared with nothing else, but a tensor's out may be its grad.
int check_spans(const char* op, const dmuon_grad* gs, int n, bool outs, const float* norm, const float* norms, const float* coef,
                bool coef_written) {
  std::vector<Span> v;
  v.reserve(2 * static_cast<size_t>(n) + 3);
  const auto add = [&](const void* p, int64_t bytes, int idx, bool written) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    if (p && bytes > 0) v.push_back(Span{lo, lo + static_cast<uintptr_t>(bytes), idx, written});
  };
  for (int i = 0; i < n; ++i) {
    const bool in_place = outs && gs[i].out == gs[i].grad && gs[i].out_dtype == gs[i].grad_dtype;
    if (!in_place) add(gs[i].grad, gs[i].numel * elem_size(gs[i].grad_dtype), i, false);
    if (outs) add(gs[i].out, gs[i].numel * elem_size(gs[i].out_dtype), i, true);
  }
  add(norm, 4, -1, true);
  add(norms, 4 * static_cast<int64_t>(n), -1, true);
  add(coef, 4, -1, coef_written);
  std::sort(v.begin(), v.end(), [](const Span& a, const Span& b) { return a.lo < b.lo; });
  // Ends of what begins before: of what is written, and of anything.
  uintptr_t end_written = 0, end_any = 0;
  int who_written = 0, who_any = 0;
  for (const Span& s : v) {
    if (s.lo < (s.written ? end_any : end_written)) {
      const auto name = [](int i) { return i < 0 ? std::string("a result of the call") : "tensor " + std::to_string(i); };
      const std::string m = std::string(op) + ": " + name(s.written ? who_any : who_written) + " overlaps " + name(s.idx) +
                            " (memory the call writes must not be shared)";
      return set_error(DMUON_ERR_INVALID_ARG, m.c_str());
    }
    if (s.hi > end_any) {
      end_any = s.hi;
      who_any = s.idx;
    }
    if (s.written && s.hi > end_written) {
      end_written = s.hi;
      who_written = s.idx;
    }
  }
  return DMUON_OK;
}

// The checks that look at the whole list (before the device is touched) and that ask
// the driver, skipped for the descriptor arrays and results that passed them last;
// then the device is the context's.
int check_list(dmuon_context* ctx, const char* op, const dmuon_grad* gs, int n, bool outs, const float* norm, const float* norms,
               const float* coef, bool coef_written) {
  struct Rest {
    const void* p[3];
    int64_t flags;
  } rest = {{norm, norms, coef}, (outs ? 1 : 0) | (coef_written ? 2 : 0)};
  std::vector<uint8_t> key;
  keep_bytes(key, gs, n);
  key.insert(key.end(), reinterpret_cast<const uint8_t*>(&rest), reinterpret_cast<const uint8_t*>(&rest) + sizeof rest);
  for (const auto& k : ctx->checked_grads)
    if (k == key) return DMUON_OK;
  for (const float* p : {norm, norms, coef})
    if (reinterpret_cast<uintptr_t>(p) % sizeof(float) != 0) {
      const std::string m = std::string(op) + ": a result is not aligned to its elements";
      return set_error(DMUON_ERR_INVALID_ARG, m.c_str());
    }
  DM_TRY(check_spans(op, gs, n, outs, norm, norms, coef, coef_written));
  DM_TRY(ensure_device(ctx));
  for (int i = 0; i < n; ++i) {
    if (gs[i].numel == 0) continue;
    DM_TRY(check_reachable(ctx, gs[i].grad, "grad", i));
    if (outs) DM_TRY(check_reachable(ctx, gs[i].out, "out", i));
  }
  DM_TRY(check_reachable(ctx, norm, "norm", 0));
  if (n > 0) DM_TRY(check_reachable(ctx, norms, "norms", 0));
  DM_TRY(check_reachable(ctx, coef, "coef", 0));
  ctx->checked_grads[ctx->checked_next] = std::move(key);
  ctx->checked_next = (ctx->checked_next + 1) % dmuon_context::kCheckedGrads;
  return DMUON_OK;
}

// Bytes of a chunk (a multiple of `least`), by the number of chunks wanted.
int32_t chunk_bytes(const dmuon_grad* gs, int n, int64_t wanted, int64_t least) {
  int64_t total = 0;
  for (int i = 0; i < n; ++i) total += gs[i].numel * elem_size(gs[i].grad_dtype);
  int64_t chunk = std::min<int64_t>(round_up(total / wanted + 1, least), kLongChunk);
  // Chunks are numbered in 31 bits.
  while (total / chunk + n >= (int64_t(1) << 30)) chunk *= 2;
  return static_cast<int32_t>(chunk);
}

// An SM holds eight blocks.  Sums: one round of blocks as long as chunks of 128 KB do (their ends are what a
// small call waits for: three tensors of a small model 8.2 us in chunks of 4 KB, 7.1 of 16), then eight.  Scaling: at least four
// rounds, so that its last one is a small part (clipping 1e8 bf16 elements 109 us with two, 107.4 with four, 3e7 of fp32 into bf16 56.3
// and 55.3; 120 small tensors, 1.9e7 elements, 33.0 and 34.0).
int64_t round_of(const dmuon_context* ctx) { return int64_t(ctx->num_sms) * 8; }
int32_t norm_chunk(const dmuon_context* ctx, const dmuon_grad* gs, int n) {
  const int64_t round = round_of(ctx);
  const int32_t one = chunk_bytes(gs, n, std::max<int64_t>(round - n, round / 8), 16384);
  return one < kLongChunk ? one : chunk_bytes(gs, n, round * 8, 16384);
}
int32_t scale_chunk(const dmuon_context* ctx, const dmuon_grad* gs, int n) { return chunk_bytes(gs, n, round_of(ctx) * 4, 4096); }

int64_t chunks_of(const dmuon_grad& g, int32_t chunk) {
  const int64_t length = chunk / elem_size(g.grad_dtype);
  return (g.numel + length - 1) / length;
}

template <int CAP>
void fill_batch(GradBatch<CAP>& B, const dmuon_grad* gs, int n, int32_t chunk) {
  B.n = n;
  B.chunk = chunk;
  B.first[0] = 0;
  for (int i = 0; i < n; ++i) {
    B.in[i] = gs[i].grad;
    B.out[i] = gs[i].out;
    B.numel[i] = gs[i].numel;
    B.in_bf16[i] = gs[i].grad_dtype == DMUON_DTYPE_BF16;
    B.out_bf16[i] = gs[i].out_dtype == DMUON_DTYPE_BF16;
    B.first[i + 1] = B.first[i] + static_cast<int32_t>(chunks_of(gs[i], chunk));
  }
}

template <int CAP>
int norm_launches(dmuon_context* ctx, const dmuon_grad* gs, int n, int32_t chunk, const GradNorm& G, cudaStream_t s) {
  int64_t chunk0 = 0;
  for (int i = 0; i < std::max(n, 1); i += CAP) {
    GradBatch<CAP> B;
    fill_batch(B, gs + i, std::min(CAP, n - i), chunk);
    const int32_t chunks = B.first[B.n];
    const bool whole = n <= CAP && chunks > 0 && chunks <= kGradWhole && n <= kGradWholeTensors;
    if (chunks > 0) DM_TRY(timed_launch(ctx, -1, s, [&] { return launch_grad_squares(B, G, chunk0, whole, s); }));
    if (!whole) DM_TRY(timed_launch(ctx, -1, s, [&] { return launch_grad_join(B, G, chunk0, i, s); }));
    chunk0 += B.first[B.n];
  }
  return DMUON_OK;
}

template <int CAP>
int scale_launches(dmuon_context* ctx, const dmuon_grad* gs, int n, int32_t chunk, const float* coef, cudaStream_t s) {
  // The last tensors, which a norm has read last, first.
  for (int i = (n - 1) / CAP * CAP; i >= 0 && n > 0; i -= CAP) {
    GradBatch<CAP> B;
    fill_batch(B, gs + i, std::min(CAP, n - i), chunk);
    if (B.first[B.n] > 0) DM_TRY(timed_launch(ctx, -1, s, [&] { return launch_grad_scale(B, coef, s); }));
  }
  return DMUON_OK;
}

int scale_impl(dmuon_context* ctx, const dmuon_grad* gs, int n, const float* coef, cudaStream_t s) {
  const int32_t chunk = scale_chunk(ctx, gs, n);
  return n <= kGradFew ? scale_launches<kGradFew>(ctx, gs, n, chunk, coef, s) : scale_launches<kGradBatch>(ctx, gs, n, chunk, coef, s);
}

// Norms into the given results; with `scale` the outs too.
int norm_impl(dmuon_context* ctx, const dmuon_grad* gs, int n, float max_norm, float* norm, float* norms, float* coef, bool scale,
              cudaStream_t s) {
  const int32_t chunk = norm_chunk(ctx, gs, n);
  int64_t chunks = 0;
  for (int i = 0; i < n; ++i) chunks += chunks_of(gs[i], chunk);
  const size_t at_squares = static_cast<size_t>(chunks) * sizeof(double), at_coef = at_squares + static_cast<size_t>(n) * sizeof(double);
  DM_TRY(vocab_workspace(ctx, at_coef + 16, s));
  char* ws = static_cast<char*>(ctx->vocab_ws.p);
  if (scale && !coef) coef = reinterpret_cast<float*>(ws + at_coef);
  GradNorm G = {};
  G.partial = reinterpret_cast<double*>(ws);
  G.squares = reinterpret_cast<double*>(ws + at_squares);
  G.n_total = n;
  G.norms = norms;
  G.norm = norm;
  G.coef = coef;
  G.max_norm = max_norm;
  G.ticket = static_cast<uint32_t*>(ctx->vocab_ticket.p) + 4;
  const auto launches = [&]() -> int {
    DM_TRY(n <= kGradFew ? norm_launches<kGradFew>(ctx, gs, n, chunk, G, s) : norm_launches<kGradBatch>(ctx, gs, n, chunk, G, s));
    return scale ? scale_impl(ctx, gs, n, coef, s) : static_cast<int>(DMUON_OK);
  };
  const int st = launches();
  // A sequence that broke off may have left its ticket up.
  if (st != DMUON_OK) cudaMemsetAsync(ctx->vocab_ticket.p, 0, 256, s);
  return end_use(ctx, s, st);
}

// What the host's memory refuses does not leave a C entry as an exception.
template <class F>
int guarded(F&& call) {
  try {
    return call();
  } catch (const std::exception&) {
    return set_error(DMUON_ERR_NOMEM, "host allocation failed");
  }
}

int check_max_norm(const char* op, float max_norm) {
  if (max_norm > 0.f) return DMUON_OK;  // infinity: a factor of 1, whatever the norm
  char buf[120];
  snprintf(buf, sizeof buf, "%s: max_norm must be positive", op);
  return set_error(DMUON_ERR_INVALID_ARG, buf);
}

}  // namespace
}  // namespace dmuon

using namespace dmuon;

extern "C" {

int dmuon_grad_norm(dmuon_context* ctx, const dmuon_grad* gs, int32_t n, float max_norm, float* norm, float* norms, float* coef,
                    void* stream) {
  clear_error();
  return guarded([&]() -> int {
    const char* op = "grad_norm";
    if (!ctx) return set_error(DMUON_ERR_INVALID_ARG, "grad_norm: null context");
    DM_TRY(validate_grads(op, gs, n, false));
    if (!norm && !norms && !coef) return set_error(DMUON_ERR_INVALID_ARG, "grad_norm: no output asked for");
    if (coef) DM_TRY(check_max_norm(op, max_norm));
    DeviceGuard guard(ctx->device);
    DM_TRY(check_list(ctx, op, gs, n, false, norm, norms, coef, true));
    return norm_impl(ctx, gs, n, max_norm, norm, norms, coef, false, static_cast<cudaStream_t>(stream));
  });
}

int dmuon_clip_grads(dmuon_context* ctx, const dmuon_grad* gs, int32_t n, float max_norm, float* norm, float* norms, float* coef,
                     void* stream) {
  clear_error();
  return guarded([&]() -> int {
    const char* op = "clip_grads";
    if (!ctx) return set_error(DMUON_ERR_INVALID_ARG, "clip_grads: null context");
    DM_TRY(validate_grads(op, gs, n, true));
    DM_TRY(check_max_norm(op, max_norm));
    DeviceGuard guard(ctx->device);
    DM_TRY(check_list(ctx, op, gs, n, true, norm, norms, coef, true));
    return norm_impl(ctx, gs, n, max_norm, norm, norms, coef, true, static_cast<cudaStream_t>(stream));
  });
}

int dmuon_scale_grads(dmuon_context* ctx, const dmuon_grad* gs, int32_t n, const float* coef, void* stream) {
  clear_error();
  return guarded([&]() -> int {
    const char* op = "scale_grads";
    if (!ctx) return set_error(DMUON_ERR_INVALID_ARG, "scale_grads: null context");
    DM_TRY(validate_grads(op, gs, n, true));
    if (!coef) return set_error(DMUON_ERR_INVALID_ARG, "scale_grads: null factor");
    DeviceGuard guard(ctx->device);
    DM_TRY(check_list(ctx, op, gs, n, true, nullptr, nullptr, coef, false));
    return scale_impl(ctx, gs, n, coef, static_cast<cudaStream_t>(stream));
  });
}

}  // extern "C"
