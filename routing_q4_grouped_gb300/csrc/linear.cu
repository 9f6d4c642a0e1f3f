// linear.cu — dense projection with its epilogue (moe_linear):
//
//   y[t][n] = act( sx[t] sw[n] sum_k x[t][k] w[n][k] + bias[n] ) + add[t][n]
//
// 16-bit or e4m3 operands, fp32 accumulation on the tensor cores. The weights are the
// MMA's A operand (128 output features, one per tensor-memory lane) and the tokens its B
// operand (up to 256 columns), so one token costs 16 columns and not 128 rows, and a
// feature's bias and scale are one register of its lane.
//
// A block keeps a ring of K-chunks (128 bytes of K of both operands, 128-byte swizzle)
// that one thread fills by TMA and one warp feeds to the tensor cores; two accumulators in
// tensor memory let 16 warps finish a tile while the next one is multiplied. Three modes:
//   kSingle  a block per tile, each block several tiles
//   kSplit   too few tiles for the multiprocessors: a cluster of 2, 4 or 8 blocks splits K;
//            each sends its partial sums to the block that finishes their tokens through
//            distributed shared memory, where they are added in the order of the blocks
//   kPair    many tiles: two blocks on neighbouring multiprocessors multiply one tile of 256
//            features (cta_group::2); each holds its 128 features and half of the tokens, so
//            a chunk of 256 x 256 costs each of them 32 KB of copies instead of 48
#include <algorithm>
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/moeq4_debug.h"
#include "internal.h"
#include "ptx.cuh"

namespace moeq4 {
namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;
constexpr int kEpiWarps = 16;              // four per tensor-memory lane quarter: an epilogue is
                                           // latency (8 warps: 4096 x 2048 -> 8192 with gelu
                                           // 106 us, with a residual 100; 16: 92 and 86)
constexpr int kParts = kEpiWarps / 4;      // warps that share a tile's tokens
constexpr int kThreads = 64 + 32 * kEpiWarps;   // warp 0: producer, warp 1: MMA issuer
constexpr int kRows = 128;                 // features per tile (MMA M)
constexpr int kChunk = 128;                // bytes of K per stage and row
constexpr int kMaxCols = 256;              // tokens per tile at most (MMA N)
constexpr int kMaxStages = 12;
constexpr int kMaxSplit = 8;
constexpr int kMaxSplitCols = 128;         // tokens per tile at most where K is split
constexpr int kBatch = 16;                 // tokens that an epilogue warp finishes at once
constexpr size_t kSmemMax = 227 * 1024;

enum Mode { kSingle, kSplit, kPair };

struct LinearArgs {
  int T, N;
  int nch;                   // K-chunks
  int cols;                  // tokens per tile, a multiple of 16
  int tiles_n, tiles_t;
  int band;                  // feature tiles that are gone through together for every token tile
  int stages;
  int acc, tcols;            // tensor-memory columns per accumulator, and of all (powers of two)
  uint32_t idesc;
  const float *x_scale, *w_scale, *bias;
  const void* add;
  void* out;
  int64_t add_row, out_row;
  int act;
  int32_t* err;
  uint64_t timeout_ns;
};

struct Ctl {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drained;
  uint32_t tmem;
  int abort, zero;
  uint32_t peer_ok[kMaxSplit][kEpiWarps];    // [block][warp]: its partial sums were sent
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t peer_addr(uint32_t saddr, uint32_t rank) {
  uint32_t d;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(saddr), "r"(rank));
  return d;
}
__device__ __forceinline__ void st_peer(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Arrives on barrier `bar` of block 0 of the cluster.
__device__ __forceinline__ void arrive_leader(uint64_t* bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                   peer_addr(smem_u32(bar), 0))
               : "memory");
}

// One K-chunk's copies: `bytes` expected on `bar`, features from row `fn` and tokens from row
// `ft` at element c0 of K, issued by one elected lane of a converged warp from one asm block
// (warp-uniform operands stay in uniform registers; behind a test of the lane each copy took
// about 250 cycles to issue). PAIR: both blocks' copies complete on block 0's barrier, at
// cluster address `bar`, and block 0 alone expects them (`expect`).
template <bool PAIR>
__device__ __forceinline__ void load_chunk(uint32_t dst_w, uint32_t dst_x, const CUtensorMap* tm_w,
                                           const CUtensorMap* tm_x, uint32_t bar, uint32_t own_bar,
                                           uint32_t bytes, bool expect, int32_t c0, int32_t fn,
                                           int32_t ft, uint64_t pol_w, uint64_t pol_x) {
#define MOEQ4_LOAD(GROUP)                                                                        \
  asm volatile(                                                                                  \
      "{\n\t.reg .pred e, p;\n\tsetp.ne.b32 p, %7, 0;\n\t"                                       \
      "elect.sync _|e, 0xffffffff;\n\tand.pred p, p, e;\n\t"                                     \
      "@p mbarrier.arrive.expect_tx.shared::cta.b64 _, [%5], %6;\n\t"                            \
      "@e cp.async.bulk.tensor.2d" GROUP ".shared::cluster.global.tile.mbarrier::complete_tx::"  \
      "bytes.L2::cache_hint [%0], [%2, {%8, %9}], [%4], %11;\n\t"                                \
      "@e cp.async.bulk.tensor.2d" GROUP ".shared::cluster.global.tile.mbarrier::complete_tx::"  \
      "bytes.L2::cache_hint [%1], [%3, {%8, %10}], [%4], %12;\n\t}" ::"r"(dst_w),                \
      "r"(dst_x), "l"(reinterpret_cast<uint64_t>(tm_w)), "l"(reinterpret_cast<uint64_t>(tm_x)),  \
      "r"(bar), "r"(own_bar), "r"(bytes), "r"(static_cast<uint32_t>(expect)), "r"(c0), "r"(fn),  \
      "r"(ft), "l"(pol_w), "l"(pol_x)                                                            \
      : "memory")
  if constexpr (PAIR) MOEQ4_LOAD(".cta_group::2");
  else MOEQ4_LOAD("");
#undef MOEQ4_LOAD
}

// One K-chunk (4 steps of 32 bytes of K) of D[features, tokens] += W X^T, issued by one
// elected lane of a converged warp. The first step accumulates only if `accumulate`.
#define MOEQ4_MMA_CHUNK(GROUP, KIND)                                                    \
  asm volatile(                                                                         \
      "{\n\t.reg .pred e, p;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"                  \
      "setp.ne.b32 p, %4, 0;\n\t"                                                       \
      "add.u64 a1, %1, 2;\n\tadd.u64 a2, %1, 4;\n\tadd.u64 a3, %1, 6;\n\t"             \
      "add.u64 b1, %2, 2;\n\tadd.u64 b2, %2, 4;\n\tadd.u64 b3, %2, 6;\n\t"             \
      "elect.sync _|e, 0xffffffff;\n\t"                                                 \
      "@e tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], %1, %2, %3, p;\n\t"      \
      "@e tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], a1, b1, %3, 1;\n\t"      \
      "@e tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], a2, b2, %3, 1;\n\t"      \
      "@e tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], a3, b3, %3, 1;\n\t}" ::  \
          "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)                           \
      : "memory")
template <bool E4M3, bool PAIR>
__device__ __forceinline__ void mma_chunk(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
  if constexpr (E4M3 && PAIR) MOEQ4_MMA_CHUNK("2", "f8f6f4");
  else if constexpr (E4M3) MOEQ4_MMA_CHUNK("1", "f8f6f4");
  else if constexpr (PAIR) MOEQ4_MMA_CHUNK("2", "f16");
  else MOEQ4_MMA_CHUNK("1", "f16");
}
#undef MOEQ4_MMA_CHUNK

// Arrives on `bar` (PAIR: of both blocks) when every product issued so far is complete.
template <bool PAIR>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if constexpr (PAIR) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
        ".multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
  } else {
    mma_commit_elect(bar);
  }
}

template <bool PAIR>
__device__ __forceinline__ void alloc_columns(uint32_t* dst, uint32_t n) {
  if constexpr (PAIR) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(dst)),
                 "r"(n)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    tmem_alloc(dst, n);
    tmem_relinquish();
  }
}
template <bool PAIR>
__device__ __forceinline__ void free_columns(uint32_t base, uint32_t n) {
  if constexpr (PAIR)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(n)
                 : "memory");
  else
    tmem_dealloc(base, n);
}

template <typename O>
__device__ __forceinline__ float to_f(O v);
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f(float v) { return v; }
template <typename O>
__device__ __forceinline__ O to_out(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 to_out(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half to_out(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float to_out(float v) { return v; }

// erf(x) to 1.5e-7 (M. Abramowitz and I. A. Stegun, "Handbook of Mathematical Functions",
// 1964, 7.1.26): a third of erff's instructions, next to results of 16 bits.
__device__ __forceinline__ float erf_near(float x) {
  const float z = fabsf(x), t = __fdividef(1.f, fmaf(0.3275911f, z, 1.f));
  float p = fmaf(1.061405429f, t, -1.453152027f);
  p = fmaf(p, t, 1.421413741f);
  p = fmaf(p, t, -0.284496736f);
  p = fmaf(p, t, 0.254829592f);
  return copysignf(fmaf(-p * t, __expf(-z * z), 1.f), x);
}

template <int M>
__device__ __forceinline__ void activate(float (&v)[M], int act) {
  switch (act) {
    case MOE_ACT_RELU:
#pragma unroll
      for (int j = 0; j < M; ++j) v[j] = v[j] < 0.f ? 0.f : v[j];   // (NaN stays)
      break;
    case MOE_ACT_SILU:
      // (a denominator above 2^126 gives 0, which the quotient has rounded to long before)
#pragma unroll
      for (int j = 0; j < M; ++j) v[j] = __fdividef(v[j], 1.f + __expf(-v[j]));
      break;
    case MOE_ACT_GELU:
#pragma unroll
      for (int j = 0; j < M; ++j)
        v[j] = 0.5f * v[j] * (1.f + erf_near(v[j] * 0.70710678118654752f));
      break;
    case MOE_ACT_GELU_TANH:
      // (1 + tanh u) / 2 = 1 / (1 + exp(-2u))
#pragma unroll
      for (int j = 0; j < M; ++j) {
        const float u = 0.79788456080286536f * fmaf(0.044715f * v[j] * v[j], v[j], v[j]);
        v[j] = __fdividef(v[j], 1.f + __expf(-2.f * u));
      }
      break;
    default: break;
  }
}

// M tokens t, t + step, ... of one feature n, of which the first `live` exist: what the
// epilogue reads of them (all loads before any store), and the results from their sums.
// Called by whole warps: a token's scale is held by one lane.
template <bool E4M3, typename O, int M>
struct Tokens {
  O add[M];
  float scale;               // of token t + lane * step

  __device__ __forceinline__ void load(const LinearArgs& a, int64_t t, int step, int live, int n,
                                       bool in) {
    if (E4M3) {
      const int lane = static_cast<int>(threadIdx.x & 31);
      scale = lane < min(live, M) ? a.x_scale[t + lane * step] : 0.f;
    }
    if (a.add && in) {
      const int64_t row = step * a.add_row;
      const O* p = static_cast<const O*>(a.add) + t * a.add_row + n;
      if (live >= M) {
#pragma unroll
        for (int j = 0; j < M; ++j, p += row) add[j] = *p;
      } else {
#pragma unroll
        for (int j = 0; j < M; ++j, p += row)
          if (j < live) add[j] = *p;
      }
    }
  }
  __device__ __forceinline__ void finish(const LinearArgs& a, float (&v)[M], int64_t t, int step,
                                         int live, int n, bool in, float ws, float bias) {
#pragma unroll
    for (int j = 0; j < M; ++j) {
      if (E4M3) v[j] = v[j] * __shfl_sync(kFull, scale, j) * ws;
      v[j] += bias;
    }
    activate(v, a.act);
    if (!in) return;
    if (a.add) {
#pragma unroll
      for (int j = 0; j < M; ++j) v[j] += to_f(add[j]);     // (not stored where j >= live)
    }
    const int64_t row = step * a.out_row;
    O* o = static_cast<O*>(a.out) + t * a.out_row + n;
    if (live >= M) {
#pragma unroll
      for (int j = 0; j < M; ++j, o += row) *o = to_out<O>(v[j]);
    } else {
#pragma unroll
      for (int j = 0; j < M; ++j, o += row)
        if (j < live) *o = to_out<O>(v[j]);
    }
  }
};

// Bytes of a ring stage: 128 features, and the tokens of a tile (kPair: half of them).
__host__ __device__ inline int stage_bytes(int cols, int mode) {
  return (kRows + (mode == kPair ? cols / 2 : cols)) * kChunk;
}

// Feature and token tile of a tile number: bands of `band` feature tiles, the features of a
// band going fastest, so that the tiles under way at one time share rows of both operands.
__device__ __forceinline__ void tile_at(const LinearArgs& a, int tile, int& fn, int& ft) {
  const int per = a.band * a.tiles_t, g = tile / per, r = tile - g * per;
  const int here = min(a.band, a.tiles_n - g * a.band);
  ft = r / here;
  fn = g * a.band + r - ft * here;
}

template <bool E4M3, typename O, int MODE>
__global__ void __launch_bounds__(kThreads)
    linear_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                  const LinearArgs a) {
  constexpr bool kIsPair = MODE == kPair, kIsSplit = MODE == kSplit;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int sb = stage_bytes(a.cols, MODE), ns = a.stages;
  // behind the ring: partial sums [source block][token][feature] (kSplit), then control
  float* parts = reinterpret_cast<float*>(smem + static_cast<size_t>(ns) * sb);
  Ctl& ctl = *reinterpret_cast<Ctl*>(reinterpret_cast<uint8_t*>(parts) +
                                     (kIsSplit ? static_cast<size_t>(a.cols) * kRows * 4 : 0));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t group = 1, rank = 0;              // blocks that share a tile
  if constexpr (MODE != kSingle) {
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(group));
    rank = cluster_rank();
  }
  if (tid == 0) {
    for (int s = 0; s < ns; ++s) {
      mbar_init(&ctl.full[s], 1);
      mbar_init(&ctl.empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctl.acc_full[s], 1);
      mbar_init(&ctl.acc_empty[s], kEpiWarps * (kIsPair ? 2 : 1));
    }
    mbar_init(&ctl.drained, 1);
    ctl.abort = 0;
    ctl.zero = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_x);
    tma_prefetch_desc(&tm_w);
  }
  if (warp == 1) alloc_columns<kIsPair>(&ctl.tmem, a.tcols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if constexpr (MODE != kSingle) cluster_arrive();   // (this block's barriers and memory may be used)
  if constexpr (kIsPair) cluster_wait();
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t tmem = ctl.tmem;
  const volatile int* abortp = &ctl.abort;
  const uint64_t lim = a.timeout_ns;
  const int tiles = a.tiles_n * a.tiles_t;
  const int first = static_cast<int>(blockIdx.x / group), step = static_cast<int>(gridDim.x / group);
  // this block's chunks of every tile
  const int c_lo = kIsSplit ? static_cast<int>(static_cast<int64_t>(a.nch) * rank / group) : 0;
  const int c_hi = kIsSplit ? static_cast<int>(static_cast<int64_t>(a.nch) * (rank + 1) / group) : a.nch;
  const int fw = kRows * (kIsPair ? 2 : 1);  // features of a tile
  const int f0 = kIsPair ? static_cast<int>(rank) * kRows : 0;   // this block's first one in it
  bool ok = true;
  int n0 = 0, t0 = 0;                        // of the tile that the epilogue holds at the end

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    const uint64_t pol = policy_evict_last();
    int st = 0, issued = 0;                  // stage, chunks requested
    uint32_t ph = 1;                         // parity of the phase before the stage's next use
    for (int tile = first; tile < tiles && ok; tile += step) {
      int fn, ft;
      tile_at(a, tile, fn, ft);
      const int tn = fn * fw + f0;
      const int tt = ft * a.cols + (kIsPair ? static_cast<int>(rank) * (a.cols / 2) : 0);
      for (int c = c_lo; c < c_hi; ++c, ++issued) {
        ok = __all_sync(kFull, mbar_wait(&ctl.empty[st], ph, abortp, lim));
        if (!ok) break;
        const uint32_t dst = smem_u32(smem) + st * sb, bar = smem_u32(&ctl.full[st]);
        constexpr int kElems = E4M3 ? kChunk : kChunk / 2;
        load_chunk<kIsPair>(dst, dst + kRows * kChunk, &tm_w, &tm_x,
                            kIsPair ? peer_addr(bar, 0) : bar, bar, kIsPair ? 2 * sb : sb,
                            !kIsPair || rank == 0, c * kElems, tn, tt, pol, pol);
        if (++st == ns) {
          st = 0;
          ph ^= 1;
        }
      }
    }
    if (!ok && lane == 0 && atomicExch(&ctl.abort, 1) == 0)
      atomicOr(a.err, MOE_DEVERR_PIPE_TIMEOUT);
    // Every copy has landed, and been multiplied, before the block's shared memory goes away:
    // the last use of each stage, oldest first.
    for (int i = min(issued, ns); i > 0; --i) {
      const int c = issued - i;
      mbar_wait(&ctl.empty[c % ns], (c / ns) & 1, &ctl.zero, 20000000ull);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------- MMA issuer
    if (rank == 0 || kIsSplit) {
      int st = 0, i = 0;                     // stage, tiles multiplied
      uint32_t ph = 0;
      for (int tile = first; tile < tiles && ok; tile += step, ++i) {
        const int b = i & 1;
        ok = __all_sync(kFull, mbar_wait(&ctl.acc_empty[b], ((i >> 1) & 1) ^ 1, abortp, lim));
        tc_fence_after();
        for (int c = c_lo; c < c_hi && ok; ++c) {
          ok = __all_sync(kFull, mbar_wait(&ctl.full[st], ph, abortp, lim));
          if (!ok) break;
          tc_fence_after();
          const uint32_t sa = smem_u32(smem) + st * sb;
          mma_chunk<E4M3, kIsPair>(tmem + b * a.acc, sdesc_k_sw128(sa),
                                   sdesc_k_sw128(sa + kRows * kChunk), a.idesc, c != c_lo);
          commit<kIsPair>(&ctl.empty[st]);
          if (++st == ns) {
            st = 0;
            ph ^= 1;
          }
        }
        if (ok) commit<kIsPair>(&ctl.acc_full[b]);
      }
      if (!ok && lane == 0 && atomicExch(&ctl.abort, 1) == 0)
        atomicOr(a.err, MOE_DEVERR_PIPE_TIMEOUT);
      // no product is under way when tensor memory is given back
      commit<kIsPair>(&ctl.drained);
      mbar_wait(&ctl.drained, 0, &ctl.zero, 20000000ull);
      __syncwarp();
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    // warp w reads tensor-memory lanes 32 (w % 4) .. (features n, one per lane) and every
    // kParts-th batch of tokens
    const int q = warp & 3, part = (warp - 2) >> 2;
    int i = 0;
    for (int tile = first; tile < tiles && ok; tile += step, ++i) {
      const int b = i & 1;
      int fn, ft;
      tile_at(a, tile, fn, ft);
      n0 = fn * fw + f0;
      t0 = ft * a.cols;
      const int n = n0 + q * 32 + lane, live = min(a.cols, a.T - t0);
      const bool in = n < a.N;
      Tokens<E4M3, O, kBatch> next;
      float bias = 0.f, ws = 1.f;
      if constexpr (!kIsSplit) {
        bias = in && a.bias ? a.bias[n] : 0.f;
        ws = in && E4M3 ? a.w_scale[n] : 1.f;
        next.load(a, t0 + part * kBatch, 1, live - part * kBatch, n, in);
      }
      ok = __all_sync(kFull, mbar_wait(&ctl.acc_full[b], (i >> 1) & 1, abortp, lim));
      if (!ok) break;
      tc_fence_after();
      const uint32_t taddr = tmem + b * a.acc + (static_cast<uint32_t>(q * 32) << 16);
      if constexpr (kIsSplit) cluster_wait();   // every block of the cluster has started
      const int per = a.cols / static_cast<int>(group);
      const int inv = (65536 + per - 1) / per;  // x / per = x inv >> 16 for x < 128
      for (int c = part * kBatch; c < live; c += kParts * kBatch) {
        uint32_t v[kBatch];
        tmem_ld_32x32b_x16(taddr + c, v);
        if constexpr (kIsSplit) {
          tmem_ld_wait();
          tmem_regs_ready(v);
          // tokens [r per, r per + per) are finished by block r
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            if (c + j >= live) break;
            const int owner = (c + j) * inv >> 16, at = c + j - owner * per;
            st_peer(peer_addr(smem_u32(parts + (rank * per + at) * kRows + q * 32 + lane), owner),
                    v[j]);
          }
        } else {
          Tokens<E4M3, O, kBatch> now = next;
          next.load(a, t0 + c + kParts * kBatch, 1, live - c - kParts * kBatch, n, in);
          tmem_ld_wait();
          tmem_regs_ready(v);
          float y[kBatch];
#pragma unroll
          for (int j = 0; j < kBatch; ++j) y[j] = __uint_as_float(v[j]);
          now.finish(a, y, t0 + c, 1, live - c, n, in, ws, bias);
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (kIsPair) arrive_leader(&ctl.acc_empty[b]);
        else mbar_arrive(&ctl.acc_empty[b]);
      }
    }
    if (!ok && lane == 0 && atomicExch(&ctl.abort, 1) == 0)
      atomicOr(a.err, MOE_DEVERR_PIPE_TIMEOUT);
  }
  if constexpr (kIsSplit) {
    // one tile per cluster. Each barrier is reached by every thread, whatever happened before
    // it; the epilogue's warps passed the first one above unless they gave up.
    if (warp < 2 || !ok) cluster_wait();
    if (warp >= 2 && lane < group)
      st_peer(peer_addr(smem_u32(&ctl.peer_ok[rank][warp - 2]), lane), ok ? 1u : 0u);
    __syncwarp();
    cluster_arrive();
    constexpr int kM = 8;                    // tokens at once, every kParts-th of the block's
    const int per = a.cols / static_cast<int>(group);
    const int part = (warp - 2) >> 2, f = (warp & 3) * 32 + lane, n = n0 + f;
    const int tb = t0 + static_cast<int>(rank) * per;      // this block's first token
    const int live = min(per, a.T - tb);
    const bool in = n < a.N;
    const auto left = [&](int at) { return live > at ? (live - at + kParts - 1) / kParts : 0; };
    Tokens<E4M3, O, kM> now;
    float bias = 0.f, ws = 1.f;
    if (warp >= 2) {
      bias = in && a.bias ? a.bias[n] : 0.f;
      ws = in && E4M3 ? a.w_scale[n] : 1.f;
      now.load(a, tb + part, kParts, left(part), n, in);
    }
    cluster_wait();
    if (warp >= 2) {
      bool all = true;                       // partial sums of these features
      for (uint32_t r = 0; r < group; ++r)
        for (int p = 0; p < kParts; ++p) all = all && ctl.peer_ok[r][((warp - 2) & 3) + 4 * p] != 0;
      for (int at = part; at < live && all; at += kParts * kM) {
        if (at != part) now.load(a, tb + at, kParts, left(at), n, in);
        float y[kM];
#pragma unroll
        for (int j = 0; j < kM; ++j) {
          y[j] = 0.f;
          if (at + kParts * j < live)
            for (uint32_t r = 0; r < group; ++r) y[j] += parts[(r * per + at + kParts * j) * kRows + f];
        }
        now.finish(a, y, tb + at, kParts, left(at), n, in, ws, bias);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (kIsPair) {
    // neither block leaves while the other's products or arrivals may still reach it
    cluster_arrive();
    cluster_wait();
  }
  if (warp == 1) {
    tc_fence_after();
    free_columns<kIsPair>(tmem, a.tcols);
  }
}

// Sizes of one call.
struct Plan {
  int mode, cols, splits, stages, acc, tcols;
  size_t smem;
};

int next_pow2(int v) {
  int p = 16;
  while (p < v) p *= 2;
  return p;
}

// Shared memory is asked for in proportion to tensor memory (228 KB and 512 columns per
// multiprocessor), so that whatever runs side by side never waits for columns: a block of a
// cluster that did would wait for blocks that may wait for it.
size_t smem_for(int tcols, size_t need) {
  const size_t least = static_cast<size_t>(tcols) * 228 * 1024 / 512 - 1024;
  return std::max(need, least);
}

// Cycles of a call by mode and tokens per tile; the least is taken. A chunk costs its products
// (2 cycles a column) or the copies that feed them.
Plan make_plan(int T, int N, int nch, int sms) {
  const int rows_n = (N + kRows - 1) / kRows;
  const int most = std::min(kMaxCols, (T + 15) / 16 * 16);
  double best = 1e300;
  Plan p{};
  const auto offer = [&](int mode, int cols, int splits, double cost) {
    if (cost >= best) return;
    best = cost;
    p.mode = mode;
    p.cols = cols;
    p.splits = splits;
  };
  for (int cols = 16; cols <= most; cols += 16) {
    const int64_t tiles_t = (T + cols - 1) / cols;
    const double chunk = std::max(2.0 * cols, stage_bytes(cols, kSingle) / 64.0);
    for (int splits = 1; splits <= kMaxSplit && splits <= nch; splits *= 2) {
      if (splits > 1 && cols > kMaxSplitCols) break;
      const double turns = static_cast<double>((rows_n * tiles_t * splits + sms - 1) / sms);
      offer(splits > 1 ? kSplit : kSingle, cols, splits,
            turns * ((nch + splits - 1) / splits * chunk + 100.0) + 8.0 * cols +
                (splits > 1 ? 1500.0 + 10.0 * cols : 0.0));
    }
    if (cols % 32 == 0 && sms >= 2) {
      const double pair = std::max(2.0 * cols, stage_bytes(cols, kPair) / 64.0);
      const double turns = static_cast<double>(((rows_n + 1) / 2 * tiles_t + sms / 2 - 1) / (sms / 2));
      offer(kPair, cols, 1, turns * (nch * pair + 100.0) + 8.0 * cols + 500.0);
    }
  }
  p.acc = next_pow2(p.cols);
  p.tcols = std::max(32, p.mode == kSplit ? p.acc : 2 * p.acc);
  const size_t fixed = 1024 + sizeof(Ctl) +
                       (p.mode == kSplit ? static_cast<size_t>(p.cols) * kRows * sizeof(float) : 0);
  const int sb = stage_bytes(p.cols, p.mode);
  const int room = static_cast<int>((kSmemMax - fixed) / sb);
  p.stages = std::min({room, kMaxStages, std::max(2, (nch + p.splits - 1) / p.splits)});
  p.smem = smem_for(p.tcols, fixed + static_cast<size_t>(p.stages) * sb);
  return p;
}

template <bool E4M3, typename O, int MODE>
cudaError_t launch(const CUtensorMap& tx, const CUtensorMap& tw, const LinearArgs& a, const Plan& p,
                   int sms, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(linear_kernel<E4M3, O, MODE>, kSmemMax, done);
  if (e != cudaSuccess) return e;
  const int64_t tiles = static_cast<int64_t>(a.tiles_n) * a.tiles_t;
  const int64_t blocks = MODE == kSplit  ? tiles * p.splits
                         : MODE == kPair ? 2 * std::min<int64_t>(tiles, sms / 2)
                                         : std::min<int64_t>(tiles, sms);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = p.smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = MODE == kPair ? 2 : p.splits;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = MODE == kSingle ? 1 : 2;
  return cudaLaunchKernelEx(&cfg, linear_kernel<E4M3, O, MODE>, tx, tw, a);
}

template <bool E4M3, typename O>
cudaError_t launch_out(const CUtensorMap& tx, const CUtensorMap& tw, const LinearArgs& a,
                       const Plan& p, int sms, cudaStream_t s) {
  return p.mode == kPair    ? launch<E4M3, O, kPair>(tx, tw, a, p, sms, s)
         : p.mode == kSplit ? launch<E4M3, O, kSplit>(tx, tw, a, p, sms, s)
                            : launch<E4M3, O, kSingle>(tx, tw, a, p, sms, s);
}

bool bad_align(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

}  // namespace
}  // namespace moeq4

extern "C" moe_status moe_linear(const moe_linear_args* l, void* stream) {
  using namespace moeq4;
  if (!l || l->T < 0 || l->N < 1 || l->K < 1) return MOE_ERR_ARG;
  const bool e4m3 = l->dtype == MOE_E4M3;
  if (!e4m3 && l->dtype != MOE_BF16 && l->dtype != MOE_F16) return MOE_ERR_ARG;
  // results: the operands' type or fp32; bf16, fp16 or fp32 from e4m3
  if (l->out_dtype < MOE_BF16 || l->out_dtype > MOE_F32 ||
      (!e4m3 && l->out_dtype != MOE_F32 && l->out_dtype != l->dtype) ||
      l->act < MOE_ACT_NONE || l->act > MOE_ACT_GELU_TANH)
    return MOE_ERR_ARG;
  const int es = e4m3 ? 1 : 2, os = l->out_dtype == MOE_F32 ? 4 : 2;
  if (l->K % (16 / es) || l->K > (1 << 20)) return MOE_ERR_SHAPE;
  if (!l->err || !l->w || (e4m3 && !l->w_scale) || (!e4m3 && (l->x_scale || l->w_scale)))
    return MOE_ERR_ARG;
  if (l->N > 1 && (l->w_row < l->K || l->w_row >= (1ll << 39) / es)) return MOE_ERR_SHAPE;
  if (l->T == 0) return MOE_OK;
  if (!l->x || !l->out || (e4m3 && !l->x_scale)) return MOE_ERR_ARG;
  if (l->T > 1 && (l->x_row < l->K || l->x_row >= (1ll << 39) / es || l->out_row < l->N ||
                   (l->add && l->add_row < 0)))
    return MOE_ERR_SHAPE;
  if (l->add == l->out && l->T > 1 && l->add_row != l->out_row) return MOE_ERR_ARG;
  if (l->out == l->x || l->out == l->w) return MOE_ERR_ARG;
  if (bad_align(l->x, 16) || bad_align(l->w, 16) || bad_align(l->out, os) ||
      bad_align(l->add, os) || bad_align(l->x_scale, 4) || bad_align(l->w_scale, 4) ||
      bad_align(l->bias, 4) || bad_align(l->err, 4) || (l->T > 1 && l->x_row * es % 16) ||
      (l->N > 1 && l->w_row * es % 16))
    return MOE_ERR_ALIGN;
  int sms = 0;
  const moe_status st = check_device(&sms);
  if (st != MOE_OK) return st;
  LinearArgs a{};
  a.T = l->T;
  a.N = l->N;
  const int elems = kChunk / es;
  a.nch = (l->K + elems - 1) / elems;
  const Plan p = make_plan(l->T, l->N, a.nch, sms);
  a.cols = p.cols;
  const int fw = p.mode == kPair ? 2 * kRows : kRows;
  a.tiles_n = (l->N - 1) / fw + 1;
  a.tiles_t = (l->T - 1) / p.cols + 1;
  if (static_cast<int64_t>(a.tiles_n) * a.tiles_t * p.splits > 0x7FFFFFFF - 1024) return MOE_ERR_SHAPE;
  a.stages = p.stages;
  a.acc = p.acc;
  a.tcols = p.tcols;
  a.band = p.mode == kPair ? 8 : 12;         // about the square root of the tiles under way
  // instruction descriptor: fp32 D, both operands K-major, M = features, N = cols; operand types
  // fp16 (0) or bf16 (1), or e4m3 (0)
  const uint32_t type = l->dtype == MOE_BF16 ? 1u : 0u;
  a.idesc = (1u << 4) | (type << 7) | (type << 10) | (static_cast<uint32_t>(p.cols >> 3) << 17) |
            (static_cast<uint32_t>(fw >> 4) << 24);
  a.x_scale = l->x_scale;
  a.w_scale = l->w_scale;
  a.bias = l->bias;
  a.add = l->add;
  a.out = l->out;
  a.add_row = l->add_row;
  a.out_row = l->out_row;
  a.act = l->act;
  a.err = l->err;
  a.timeout_ns = wait_timeout_ns();
  // a single row has no stride: any multiple of 16 bytes will do
  const uint64_t one = (static_cast<uint64_t>(l->K) * es + 15) / 16 * 16;
  CUtensorMap tx, tw;
  if (!map_rows(&tx, l->dtype, l->x, l->K, l->T, l->T > 1 ? l->x_row * es : one, elems,
                p.mode == kPair ? p.cols / 2 : p.cols) ||
      !map_rows(&tw, l->dtype, l->w, l->K, l->N, l->N > 1 ? l->w_row * es : one, elems, kRows))
    return MOE_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (e4m3)
    e = l->out_dtype == MOE_F32   ? launch_out<true, float>(tx, tw, a, p, sms, s)
        : l->out_dtype == MOE_F16 ? launch_out<true, __half>(tx, tw, a, p, sms, s)
                                  : launch_out<true, __nv_bfloat16>(tx, tw, a, p, sms, s);
  else
    e = l->out_dtype == MOE_F32   ? launch_out<false, float>(tx, tw, a, p, sms, s)
        : l->out_dtype == MOE_F16 ? launch_out<false, __half>(tx, tw, a, p, sms, s)
                                  : launch_out<false, __nv_bfloat16>(tx, tw, a, p, sms, s);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" moe_status moe_debug_linear_plan(int32_t T, int32_t N, int32_t K, int32_t dtype,
                                            int32_t sms, int32_t* plan) {
  using namespace moeq4;
  if (T < 1 || N < 1 || K < 1 || sms < 1 || !plan) return MOE_ERR_ARG;
  const int elems = dtype == MOE_E4M3 ? kChunk : kChunk / 2, nch = (K + elems - 1) / elems;
  const Plan p = make_plan(T, N, nch, sms);
  const int32_t v[7] = {p.cols, p.splits, p.stages, p.acc, p.tcols, static_cast<int32_t>(p.smem),
                        p.mode};
  for (int i = 0; i < 7; ++i) plan[i] = v[i];
  return MOE_OK;
}
