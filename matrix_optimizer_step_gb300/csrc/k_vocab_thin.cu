// The cross entropy's two products that read the head matrix, for few tokens:
//   logits   Z^T  = W X^T       (vocabulary x tokens, K = width)
//   dX       dX^T = W^T dZ^T    (width x tokens,      K = vocabulary)
// With few token rows the time is W's way through memory, so W is the MMA's
// 128-row operand and the tokens are its short N side (16 to 256): the ring's 200 KB
// are 11 stages of W in flight per SM with 16 rows, 6 with 128 and 4 with 256, where
// the 256 x 256 tiles of k_vocab_gemm.cu would fill half of theirs with rows past
// the last token.  vocab.cu has the rules of size.  One CTA per tile (tcgen05, cta_group::1),
// persistent; warp 0 loads, warp 1 issues the MMAs, warps 2 to 5 drain, warp 6
// sums the gradients' common factor on the side.
// Memory sets the pace, not the SMs' shares: cutting the last round of tiles
// evenly over the SMs, or halving the ring, changes nothing.
//
// A drained column is a token and a lane a row of W, so a token's statistics
// go across lanes: 16 columns at a time are reduced together, each exchange
// halving the columns a lane still works on (16 shuffles for 16 maxima).
// A long K is cut into up to four accumulators that the epilogue adds: the
// MMA's running sum truncates, and with one token nothing averages that out
// (the loss at width 4096 came out 4e-6 off, relatively, from one accumulator).
// Every wait is bounded, as in k_vocab_gemm.cu.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "ptx.cuh"
#include "vocab.h"

namespace dmuon {
namespace {

constexpr int BM = 128, BK = 64;
constexpr int kThreads = 7 * 32;
constexpr uint32_t A_BYTES = BM * BK * 2;
constexpr uint32_t MN_BOX_BYTES = 64 * 64 * 2;
constexpr int kMaxStages = 12;
constexpr uint32_t kRingBytes = 200 * 1024;
constexpr int kNumBars = 2 * kMaxStages + 2 + 2 + 1;
constexpr size_t kSmem = 1024 + kRingBytes + kNumBars * 8 + 16;
static_assert(kSmem <= 227 * 1024, "shared memory budget");
static_assert(kSmem > 114 * 1024, "one CTA per SM");

__device__ __forceinline__ uint64_t desc_k(uint32_t base, int kk) {
  return smem_desc_sw128(base + 32u * kk, 16u, 1024u);
}
__device__ __forceinline__ uint64_t desc_mn(uint32_t base, int kk) {
  return smem_desc_sw128(base + 2048u * kk, MN_BOX_BYTES, 1024u);
}

__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// The wait, with the load's registers as operands: nothing that reads them moves before it.
__device__ __forceinline__ void tmem_wait_x16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
  tma_load_3d(dst, map, bar, c0, c1, 0);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Reduction of 16 columns over the warp's 32 lanes; lane l returns column l % 16.
template <class Op>
__device__ __forceinline__ float reduce16(float (&v)[16], int lane, Op op) {
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) {
    const bool up = (lane & d) != 0;
#pragma unroll
    for (int j = 0; j < d; ++j) {
      const float keep = up ? v[j + d] : v[j], send = up ? v[j] : v[j + d];
      v[j] = op(keep, __shfl_xor_sync(0xffffffffu, send, d));
    }
  }
  return op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 16));
}

// One warp's 32 vocabulary rows (v0 + lane) of 16 tokens from `token0` on.
__device__ __forceinline__ void thin_logits(const VocabThin& G, uint32_t (&r)[16], int v0, int token0, int lane) {
  const float c = G.logit_scale_log2;
  const float minus_inf = __int_as_float(0xff800000);
  const int v = v0 + lane;
  float t[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) t[j] = v < G.M ? __uint_as_float(r[j]) : minus_inf;
  const float top = reduce16(t, lane, [](float a, float b) { return fmaxf(a, b); });
  // Above every z by more than the rounding of the products below.
  float m = top * c;  // c > 0
  if (m != minus_inf) m += fabsf(m) * 2.4e-7f;
  const float ref = m == minus_inf ? 0.f : m;  // only -inf and NaN: as in k_vocab_gemm.cu
  const int token = token0 + (lane & 15);
  int target = -1;
  if (token < G.tokens) {
    bool bad = false;
    target = load_id(G.targets, token, &bad);
  }
  const float magic = 8388608.f, most = magic + 65535.f;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float mj = __shfl_sync(0xffffffffu, ref, j);
    const int tj = __shfl_sync(0xffffffffu, target, j);
    const float z = __uint_as_float(r[j]);
    // The target's share of the sum is added by the row pass.
    const float d = v < G.M && v != tj ? fmaf(z, c, -mj) : minus_inf;
    t[j] = ex2(d);
    if (G.logs && token0 + j < G.tokens && v < G.M)
      G.logs[static_cast<int64_t>(token0 + j) * G.ld_logs + v] =
          static_cast<uint16_t>(__float_as_uint(fminf(fmaf(d, -kCeLogUnits, magic), most)));
  }
  const float s = reduce16(t, lane, [](float a, float b) { return a + b; });
  if (lane < 16 && token < G.tokens) G.stats[static_cast<int64_t>(v0 / kCeThinBlock) * G.stats_ld + token] = make_float2(m, s);
}

template <bool LOGITS>
__global__ void __launch_bounds__(kThreads, 1) vocab_thin_kernel(const __grid_constant__ VocabThin G) {
  constexpr bool A_MN = !LOGITS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t ring = smem_u32(smem);
  uint64_t* bar_mem = reinterpret_cast<uint64_t*>(smem + kRingBytes);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_mem + kNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const uint32_t bar0 = smem_u32(bar_mem);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
  auto tfull = [&](int a) { return bar0 + 8u * (2 * kMaxStages + a); };
  auto tempty = [&](int a) { return bar0 + 8u * (2 * kMaxStages + 2 + a); };
  const uint32_t drain = bar0 + 8u * (2 * kMaxStages + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t stage_bytes = A_BYTES + static_cast<uint32_t>(G.np) * (BK * 2);
  const int stages = min(kMaxStages, static_cast<int>(kRingBytes / stage_bytes));
  uint32_t tmem_cols = 32;
  const uint32_t acc_cols = static_cast<uint32_t>(G.np * G.groups);
  while (tmem_cols < 2u * acc_cols) tmem_cols <<= 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull(a), 1);
      mbar_init(tempty(a), 4);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch();
  pdl_wait();
  const uint32_t tmem_base = *tmem_slot;
  // Tile t of this CTA: rows [m0, m0 + 128) of D^T, k-blocks [kb0, kb1).
  struct Tile {
    int m0, split, kb0, kb1;
  };
  const int ctas = static_cast<int>(gridDim.x), cta = static_cast<int>(blockIdx.x);
  const int n_tiles = (G.tiles_m * G.splits - cta + ctas - 1) / ctas;
  auto tile_at = [&](int t) {
    const int u = cta + t * ctas;
    Tile T;
    T.split = LOGITS ? 0 : u / G.tiles_m;
    T.m0 = (u - T.split * G.tiles_m) * BM;
    T.kb0 = T.split * G.kb_step;
    T.kb1 = min(G.kb_total, T.kb0 + G.kb_step);
    return T;
  };

  if (warp == 0) {
    if (elect_one()) {
      // ------------------------------------------------------------ producer
      tma_prefetch_map(&G.map_a);
      tma_prefetch_map(&G.map_b);
      int stage = 0, filled = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = 0; t < n_tiles && ok; ++t) {
        const Tile T = tile_at(t);
        for (int kb = T.kb0; kb < T.kb1; ++kb) {
          if (!mbar_wait_bounded(empty(stage), phase ^ 1u, abort_flag, G.err, kErrTimeoutProducer)) {
            ok = false;
            break;
          }
          const uint32_t dst = ring + stage * stage_bytes;
          mbar_expect_tx(full(stage), stage_bytes);
          ++filled;
          if (A_MN) {
            tma_load(dst, &G.map_a, full(stage), T.m0, kb * BK);
            tma_load(dst + MN_BOX_BYTES, &G.map_a, full(stage), T.m0 + 64, kb * BK);
          } else {
            tma_load(dst, &G.map_a, full(stage), kb * BK, T.m0);
          }
          tma_load(dst + A_BYTES, &G.map_b, full(stage), kb * BK, 0);
          if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        // Copies in flight land before the block leaves: stage s was filled
        // ceil((filled - s) / stages) times.
        for (int s = 0; s < stages && s < filled; ++s) {
          volatile int no_abort = 0;
          const int uses = (filled - s + stages - 1) / stages;
          mbar_wait_bounded(full(s), static_cast<uint32_t>(uses - 1) & 1u, &no_abort, nullptr, 0, 100000000ull);
        }
      }
    }
  } else if (warp == 6) {
    if (LOGITS && blockIdx.x == 0 && G.norm.alpha) write_alpha(G.norm, lane);
  } else if (warp == 1) {
    if (elect_one()) {
      // ---------------------------------------------------------- MMA issuer
      const uint32_t idesc = idesc_bf16_f32(BM, G.np, A_MN, false);
      int stage = 0, use = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (; use < n_tiles && ok; ++use) {
        const Tile T = tile_at(use);
        const int kb0 = T.kb0, kb1 = T.kb1;
        if (!mbar_wait_bounded(tempty(use & 1), (static_cast<uint32_t>(use >> 1) & 1u) ^ 1u, abort_flag, G.err, kErrTimeoutMma))
          break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(use & 1) * acc_cols;
        const int per_group = (kb1 - kb0 + G.groups - 1) / G.groups;
        int group = 0, left = per_group;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait_bounded(full(stage), phase, abort_flag, G.err, kErrTimeoutMma)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = ring + stage * stage_bytes, sb = sa + A_BYTES;
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk)
            umma_bf16(d_tmem + static_cast<uint32_t>(group * G.np), A_MN ? desc_mn(sa, kk) : desc_k(sa, kk), desc_k(sb, kk),
                      idesc, (left != per_group || kk != 0) ? 1u : 0u);
          if (--left == 0) {
            ++group;
            left = per_group;
          }
          umma_commit(empty(stage));
          if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok) umma_commit(tfull(use & 1));
      }
      umma_commit(drain);
      volatile int no_abort = 0;
      mbar_wait_bounded(drain, 0, &no_abort, G.err, kErrTimeoutDrain);
    }
  } else {
    // -------------------------------------------------------------- epilogue
    const int quarter = warp & 3;
    int use = 0;
    for (; use < n_tiles; ++use) {
      const Tile T = tile_at(use);
      const int split = T.split, row0 = T.m0 + 32 * quarter;
      const int acc = use & 1;
      if (!mbar_wait_bounded(tfull(acc), static_cast<uint32_t>(use >> 1) & 1u, abort_flag, G.err, kErrTimeoutEpilogue)) break;
      tc_fence_after();
      const uint32_t t_lane = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(acc) * acc_cols;
      if (row0 < G.M) {  // warp-uniform
        for (int c0 = 0; c0 < G.tokens; c0 += 16) {
          uint32_t r[16];
          tmem_ld_32x32b_x16(t_lane + static_cast<uint32_t>(c0), r);
          tmem_wait_x16(r);
          for (int g = 1; g < G.groups; ++g) {
            uint32_t more[16];
            tmem_ld_32x32b_x16(t_lane + static_cast<uint32_t>(g * G.np + c0), more);
            tmem_wait_x16(more);
#pragma unroll
            for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) + __uint_as_float(more[j]));
          }
          if (LOGITS) {
            thin_logits(G, r, row0, c0, lane);
          } else if (row0 + lane < G.M) {
            float* p = G.part + (static_cast<int64_t>(split) * G.tokens + c0) * G.ld_part + row0 + lane;
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (c0 + j < G.tokens) p[j * G.ld_part] = __uint_as_float(r[j]);
          }
          __syncwarp();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty(acc));
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, tmem_cols);
}

template <bool LOGITS>
cudaError_t launch_variant(const VocabThin& G, int n_ctas, cudaStream_t st) {
  static unsigned long long attr_mask = 0;
  if (attr_needed_on_current_device(&attr_mask)) {
    cudaError_t e = cudaFuncSetAttribute(vocab_thin_kernel<LOGITS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(kSmem));
    if (e != cudaSuccess) return e;
    attr_note_current_device(&attr_mask);
  }
  const int64_t tiles = static_cast<int64_t>(G.tiles_m) * G.splits;
  return launch_after(vocab_thin_kernel<LOGITS>, dim3(static_cast<unsigned>(tiles < n_ctas ? tiles : n_ctas)), dim3(kThreads),
                      kSmem, st, G);
}

}  // namespace

cudaError_t launch_vocab_thin(bool logits, const VocabThin& G, int n_ctas, cudaStream_t st) {
  if (G.M <= 0 || G.tokens <= 0 || G.np < G.tokens || G.np > kThinRows || G.np % 16 != 0 || G.groups < 1 ||
      2 * G.np * G.groups > 512 || n_ctas <= 0)
    return cudaErrorInvalidValue;
  return logits ? launch_variant<true>(G, n_ctas, st) : launch_variant<false>(G, n_ctas, st);
}

}  // namespace dmuon
