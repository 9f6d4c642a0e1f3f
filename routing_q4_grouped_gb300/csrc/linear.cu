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
// that one warp fills by TMA and another feeds to the tensor cores; two accumulators in
// tensor memory let 16 warps finish a tile while the next one is multiplied. The tensor
// cores' fp32 sums are cut off, not rounded: a sum loses about 2^-26 of itself at each step of
// 32 bytes of K, always towards zero. Next to results of 16 bits that is little (2^-14 at the
// longest K); for fp32 results the sum is taken in pieces of 32 steps, which the finishing warps
// add up in registers (2047 tokens, 2048 -> 256: 8.9 us instead of 8.3). Three modes, and a
// kernel of its own for few tokens (below):
//   kSingle  a block per tile, each block several tiles
//   kSplit   too few tiles for the multiprocessors: a cluster of 2, 4 or 8 blocks splits K;
//            each finishes a share of the tokens, reading the others' partial sums from their
//            shared memory, in the order of the blocks
//   kPair    many tiles: two blocks on neighbouring multiprocessors multiply one tile of 256
//            features (cta_group::2); each holds its 128 features and half of the tokens, so
//            a chunk of 256 x 256 costs each of them 32 KB of copies instead of 48
// Measured in bursts of 12 calls in a graph, and in a long row of calls, whose power lowers the
// clock: 8192^3 in bf16 541 to 557 and 625 us (2.0 and 1.76 PFLOP/s), in e4m3 with a residual 301
// to 321 and 354 us (3.5 and 3.1); 4096 tokens 2048 -> 8192 73 us (1.88) and 92, with bias and gelu
// 78 and 92; bound by the products, the first copies and the last tile's epilogue. 64 tokens
// 2048 -> 2048 7.5 us: by the plan's model 1.4 for the chunks (0.13 to 0.17 us each to issue and
// wait for, whatever their bytes), 2 for the start and 3.9 for the exchange of partial sums.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

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
constexpr int kPiece = 8;                  // K-chunks of a piece of an fp32 result's sum
constexpr int kMaxK = 65536;
constexpr int kMaxRows = 1 << 30;          // tokens, features
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
  int sub;                   // K-chunks per stage
  int cube;                  // one copy of each operand per stage: K is whole chunks
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
__device__ __forceinline__ uint32_t ld_peer(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
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

// A K-chunk's copies, or (CUBE) those of a whole stage's chunks: features from row `fn` and tokens
// from row `ft` at element c0 of K (CUBE: at chunk c0), completing on `bar`, on which `bytes` are
// expected first (0: they have been), issued by one elected lane of a converged warp from one asm
// block (warp-uniform operands stay in uniform registers; behind a test of the lane a chunk took
// 261 ns to issue, so 127). PAIR: both blocks' copies complete on block 0's barrier, at cluster
// address `bar`, and block 0 expects them all.
template <bool PAIR, bool CUBE>
__device__ __forceinline__ void load_chunk(uint32_t dst_w, uint32_t dst_x, const CUtensorMap* tm_w,
                                           const CUtensorMap* tm_x, uint32_t bar, uint32_t own_bar,
                                           uint32_t bytes, int32_t c0, int32_t fn, int32_t ft,
                                           uint64_t pol) {
#define MOEQ4_LOAD(GROUP, DIM, AT_W, AT_X)                                                       \
  asm volatile(                                                                                  \
      "{\n\t.reg .pred e, p;\n\tsetp.ne.b32 p, %6, 0;\n\t"                                       \
      "elect.sync _|e, 0xffffffff;\n\tand.pred p, p, e;\n\t"                                     \
      "@p mbarrier.arrive.expect_tx.shared::cta.b64 _, [%5], %6;\n\t"                            \
      "@e cp.async.bulk.tensor." DIM GROUP ".shared::cluster.global.tile.mbarrier::complete_tx::" \
      "bytes.L2::cache_hint [%0], [%2, " AT_W "], [%4], %10;\n\t"                                \
      "@e cp.async.bulk.tensor." DIM GROUP ".shared::cluster.global.tile.mbarrier::complete_tx::" \
      "bytes.L2::cache_hint [%1], [%3, " AT_X "], [%4], %10;\n\t}" ::"r"(dst_w),                 \
      "r"(dst_x), "l"(reinterpret_cast<uint64_t>(tm_w)), "l"(reinterpret_cast<uint64_t>(tm_x)),  \
      "r"(bar), "r"(own_bar), "r"(bytes), "r"(c0), "r"(fn), "r"(ft), "l"(pol), "r"(0)            \
      : "memory")
  if constexpr (PAIR && CUBE) MOEQ4_LOAD(".cta_group::2", "3d", "{%11, %8, %7}", "{%11, %9, %7}");
  else if constexpr (PAIR) MOEQ4_LOAD(".cta_group::2", "2d", "{%7, %8}", "{%7, %9}");
  else if constexpr (CUBE) MOEQ4_LOAD("", "3d", "{%11, %8, %7}", "{%11, %9, %7}");
  else MOEQ4_LOAD("", "2d", "{%7, %8}", "{%7, %9}");
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

// erfc(|y| / sqrt 2) / 2, by which a gelu multiplies a negative y (and one minus which, a positive
// one). Taken as exp(-y^2 / 2) times a polynomial in t = 1 / (1 + c |y|), it keeps its bits where
// 1 + erf would cancel. The polynomial is fitted to exp(y^2 / 2) erfc(|y| / sqrt 2) / 2 for |y| up
// to 15 (beyond, the exponential is 0) by least squares, weighted until the largest errors are
// level. Seven terms next to results of 16 bits: off by 5.6e-6 of the value at most, and by 1.2e-7
// of y. Ten next to fp32 results (WIDE): off by 1e-8, with their arithmetic by 4e-7.
template <bool WIDE>
__device__ __forceinline__ float gelu_tail(float y) {
  const float z = fabsf(y);
  if constexpr (WIDE) {
    const float t = __frcp_rn(fmaf(0.25f, z, 1.f));
    float p = fmaf(0.017177129f, t, -0.066118889f);
    p = fmaf(p, t, 0.059692319f);
    p = fmaf(p, t, 0.017385859f);
    p = fmaf(p, t, 0.022212096f);
    p = fmaf(p, t, 0.081368029f);
    p = fmaf(p, t, 0.073902480f);
    p = fmaf(p, t, 0.095089644f);
    p = fmaf(p, t, 0.099546343f);
    p = fmaf(p, t, 0.099744990f);
    return p * t * expf(-0.5f * z * z);
  } else {
    const float t = __fdividef(1.f, fmaf(0.34375f, z, 1.f));
    float p = fmaf(0.042991161f, t, -0.18733738f);
    p = fmaf(p, t, 0.23206683f);
    p = fmaf(p, t, -0.0053868666f);
    p = fmaf(p, t, 0.14686827f);
    p = fmaf(p, t, 0.13345376f);
    p = fmaf(p, t, 0.13734417f);
    return p * t * __expf(-0.5f * z * z);
  }
}

// y / (1 + exp(-w)) for a w of y's sign. The exponential is that of -|w|, so the denominator stays
// between 1 and 2 and a negative tail keeps its value until fp32 ends.
template <bool WIDE>
__device__ __forceinline__ float times_sigmoid(float y, float w) {
  const float e = WIDE ? expf(-fabsf(w)) : __expf(-fabsf(w));
  const float n = w < 0.f ? y * e : y;
  return WIDE ? __fdiv_rn(n, 1.f + e) : __fdividef(n, 1.f + e);
}

// WIDE: fp32 results, which take expf and rounded quotients.
template <bool WIDE, int M>
__device__ __forceinline__ void activate(float (&v)[M], int act) {
  switch (act) {
    case MOE_ACT_RELU:
#pragma unroll
      for (int j = 0; j < M; ++j) v[j] = v[j] < 0.f ? 0.f : v[j];   // (NaN stays)
      break;
    case MOE_ACT_SILU:
#pragma unroll
      for (int j = 0; j < M; ++j) v[j] = times_sigmoid<WIDE>(v[j], v[j]);
      break;
    case MOE_ACT_GELU:
#pragma unroll
      for (int j = 0; j < M; ++j) {
        const float p = gelu_tail<WIDE>(v[j]);
        v[j] *= v[j] < 0.f ? p : 1.f - p;
      }
      break;
    case MOE_ACT_GELU_TANH:
      // (1 + tanh u) / 2 = 1 / (1 + exp(-2u))
#pragma unroll
      for (int j = 0; j < M; ++j)
        v[j] = times_sigmoid<WIDE>(
            v[j], 1.5957691216057307f * fmaf(0.044715f * v[j] * v[j], v[j], v[j]));
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
    activate<sizeof(O) == 4>(v, a.act);
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

// Bytes of a K-chunk: 128 features, and the tokens of a tile (kPair: half of them).
__host__ __device__ inline int chunk_bytes(int cols, int mode) {
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
  constexpr bool kPieces = sizeof(O) == 4;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int cb = chunk_bytes(a.cols, MODE), xb = cb - kRows * kChunk;   // of a chunk, its tokens
  const int sb = a.sub * cb, ns = a.stages;
  Ctl& ctl = *reinterpret_cast<Ctl*>(smem + static_cast<size_t>(ns) * sb);
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
  if constexpr (kIsPair) {                   // the other block's barriers are set up
    cluster_arrive();
    cluster_wait();
  }
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
  constexpr int kElems = E4M3 ? kChunk : kChunk / 2;
  griddep_wait();
  griddep_launch_dependents();
  bool ok = true;
  int n0 = 0, t0 = 0;                        // of the tile that the epilogue holds at the end

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    const uint64_t pol = policy_evict_last();
    int issued = 0;                          // stages filled
    // (SUB chunks a stage, known to the compiler: counted at run time, 4096 tokens 2048 -> 2560
    // took 33.8 us instead of 28.3)
    const auto produce = [&](auto chunks) {
      constexpr int SUB = decltype(chunks)::value;
      int st = 0;                            // stage
      uint32_t ph = 1;                       // parity of the phase before the stage's next use
      for (int tile = first; tile < tiles && ok; tile += step) {
        int fn, ft;
        tile_at(a, tile, fn, ft);
        const int tn = fn * fw + f0;
        const int tt = ft * a.cols + (kIsPair ? static_cast<int>(rank) * (a.cols / 2) : 0);
        for (int c = c_lo; c < c_hi; c += SUB, ++issued) {
          ok = __all_sync(kFull, mbar_wait(&ctl.empty[st], ph, abortp, lim));
          if (!ok) break;
          const uint32_t own_bar = smem_u32(&ctl.full[st]);
          const uint32_t bar = kIsPair ? peer_addr(own_bar, 0) : own_bar;
          // a stage: the weights of its chunks, then the tokens of its chunks
          const uint32_t dst = smem_u32(smem) + st * sb, dst_x = dst + SUB * kRows * kChunk;
          if (SUB > 1 && a.cube) {           // (chunks behind the last: zeros)
            load_chunk<kIsPair, true>(dst, dst_x, &tm_w, &tm_x, bar, own_bar,
                                      kIsPair && rank != 0 ? 0 : SUB * cb * (kIsPair ? 2 : 1), c,
                                      tn, tt, pol);
          } else {
            const uint32_t all = (SUB == 1 ? cb : min(SUB, c_hi - c) * cb) * (kIsPair ? 2 : 1);
            const uint32_t bytes = kIsPair && rank != 0 ? 0 : all;
#pragma unroll
            for (int u = 0; u < SUB; ++u)
              if (u == 0 || c + u < c_hi)
                load_chunk<kIsPair, false>(dst + u * kRows * kChunk, dst_x + u * xb, &tm_w, &tm_x,
                                           bar, own_bar, u == 0 ? bytes : 0, (c + u) * kElems, tn,
                                           tt, pol);
          }
          if (++st == ns) {
            st = 0;
            ph ^= 1;
          }
        }
      }
    };
    if (a.sub == 1) produce(std::integral_constant<int, 1>{});
    else if (a.sub == 2) produce(std::integral_constant<int, 2>{});
    else produce(std::integral_constant<int, 4>{});
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
      const auto multiply = [&](auto chunks) {
        constexpr int SUB = decltype(chunks)::value;
        int st = 0, i = 0;                   // stage, sums completed
        uint32_t ph = 0;
        for (int tile = first; tile < tiles && ok; tile += step) {
          for (int lo = c_lo; lo < c_hi && ok; ++i) {
            const int hi = kPieces ? min(c_hi, lo + kPiece) : c_hi;
            const int b = i & 1;
            ok = __all_sync(kFull, mbar_wait(&ctl.acc_empty[b], ((i >> 1) & 1) ^ 1, abortp, lim));
            tc_fence_after();
            for (int c = lo; c < hi && ok; c += SUB) {
              ok = __all_sync(kFull, mbar_wait(&ctl.full[st], ph, abortp, lim));
              if (!ok) break;
              tc_fence_after();
              const uint32_t sa = smem_u32(smem) + st * sb;
#pragma unroll
              for (int u = 0; u < SUB; ++u)
                if (u == 0 || c + u < hi)
                  mma_chunk<E4M3, kIsPair>(
                      tmem + b * a.acc, sdesc_k_sw128(sa + u * kRows * kChunk),
                      sdesc_k_sw128(sa + SUB * kRows * kChunk + u * xb), a.idesc,
                      u != 0 || c != lo);
              commit<kIsPair>(&ctl.empty[st]);
              if (++st == ns) {
                st = 0;
                ph ^= 1;
              }
            }
            if (ok) commit<kIsPair>(&ctl.acc_full[b]);
            lo = hi;
          }
        }
      };
      if (a.sub == 1) multiply(std::integral_constant<int, 1>{});
      else if (a.sub == 2) multiply(std::integral_constant<int, 2>{});
      else multiply(std::integral_constant<int, 4>{});
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
    int i = 0;                               // sums read
    const auto give_back = [&](int b) {      // of an accumulator
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (kIsPair) arrive_leader(&ctl.acc_empty[b]);
        else mbar_arrive(&ctl.acc_empty[b]);
      }
    };
    for (int tile = first; tile < tiles && ok; tile += step) {
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
        if constexpr (!kPieces) next.load(a, t0 + part * kBatch, 1, live - part * kBatch, n, in);
      }
      // 16 tokens' sums: results (kSplit: partial sums [token][feature] over the ring, which
      // nothing uses any more)
      const auto put = [&](float (&y)[kBatch], int c, Tokens<E4M3, O, kBatch>& of) {
        if constexpr (kIsSplit) {
          float* part_sums = reinterpret_cast<float*>(smem) + c * kRows + q * 32 + lane;
#pragma unroll
          for (int j = 0; j < kBatch; ++j) part_sums[j * kRows] = y[j];
        } else {
          of.finish(a, y, t0 + c, 1, live - c, n, in, ws, bias);
        }
        __syncwarp();
      };
      if constexpr (kPieces) {
        constexpr int kMine = kMaxCols / (kParts * kBatch);   // batches of a warp at most
        float sum[kMine][kBatch];
#pragma unroll
        for (int m = 0; m < kMine; ++m)
#pragma unroll
          for (int j = 0; j < kBatch; ++j) sum[m][j] = 0.f;
        for (int lo = c_lo; lo < c_hi; lo += kPiece, ++i) {
          const int b = i & 1;
          ok = __all_sync(kFull, mbar_wait(&ctl.acc_full[b], (i >> 1) & 1, abortp, lim));
          if (!ok) break;
          tc_fence_after();
          const uint32_t taddr = tmem + b * a.acc + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll
          for (int m = 0; m < kMine; ++m) {
            const int c = (part + m * kParts) * kBatch;
            if (c < live) {
              uint32_t v[kBatch];
              tmem_ld_32x32b_x16(taddr + c, v);
              tmem_ld_wait();
              tmem_regs_ready(v);
#pragma unroll
              for (int j = 0; j < kBatch; ++j) sum[m][j] += __uint_as_float(v[j]);
            }
          }
          give_back(b);
        }
        if (!ok) break;
#pragma unroll
        for (int m = 0; m < kMine; ++m) {
          const int c = (part + m * kParts) * kBatch;
          if (c < live) {
            if constexpr (!kIsSplit) next.load(a, t0 + c, 1, live - c, n, in);
            put(sum[m], c, next);
          }
        }
      } else {
        const int b = i++ & 1;
        ok = __all_sync(kFull, mbar_wait(&ctl.acc_full[b], ((i - 1) >> 1) & 1, abortp, lim));
        if (!ok) break;
        tc_fence_after();
        const uint32_t taddr = tmem + b * a.acc + (static_cast<uint32_t>(q * 32) << 16);
        for (int c = part * kBatch; c < live; c += kParts * kBatch) {
          uint32_t v[kBatch];
          tmem_ld_32x32b_x16(taddr + c, v);
          Tokens<E4M3, O, kBatch> now = next;
          if constexpr (!kIsSplit)
            next.load(a, t0 + c + kParts * kBatch, 1, live - c - kParts * kBatch, n, in);
          tmem_ld_wait();
          tmem_regs_ready(v);
          float y[kBatch];
#pragma unroll
          for (int j = 0; j < kBatch; ++j) y[j] = __uint_as_float(v[j]);
          put(y, c, now);
        }
        give_back(b);
      }
    }
    if (!ok && lane == 0 && atomicExch(&ctl.abort, 1) == 0)
      atomicOr(a.err, MOE_DEVERR_PIPE_TIMEOUT);
  }
  if constexpr (kIsSplit) {
    // One tile per cluster. Every thread reaches the barriers, whatever happened before them.
    const int per = a.cols / static_cast<int>(group);
    const int part = (warp - 2) >> 2, f = (warp & 3) * 32 + lane, n = n0 + f;
    const int at0 = static_cast<int>(rank) * per;          // this block's first token of the tile
    const int live = min(per, a.T - t0 - at0);
    const bool in = n < a.N;
    constexpr int kM = 2;                    // tokens at once (little code: it runs once or twice)
    const auto left = [&](int at) { return live > at ? (live - at + kParts - 1) / kParts : 0; };
    Tokens<E4M3, O, kM> now;
    float bias = 0.f, ws = 1.f;
    if (warp >= 2) {
      bias = in && a.bias ? a.bias[n] : 0.f;
      ws = in && E4M3 ? a.w_scale[n] : 1.f;
      now.load(a, t0 + at0 + part, kParts, left(part), n, in);
    }
    __syncwarp();
    cluster_arrive();                        // the partial sums are written
    cluster_wait();
    if (warp >= 2) {
      // a block that gave up has no sums
      bool all = true;
      if (lane < group) all = ld_peer(peer_addr(smem_u32(&ctl.abort), lane)) == 0;
      all = __all_sync(kFull, all);
      for (int at = part; at < live && all; at += kParts * kM) {
        if (at != part) now.load(a, t0 + at0 + at, kParts, left(at), n, in);
        float y[kM];
#pragma unroll
        for (int j = 0; j < kM; ++j) {
          // (past the block's tokens: sums of another block's, or of no token, not written)
          const uint32_t place =
              smem_u32(smem) + (min(at0 + at + kParts * j, a.cols - 1) * kRows + f) * 4;
          uint32_t p[kMaxSplit];
#pragma unroll
          for (int r = 0; r < kMaxSplit; ++r)
            if (r < static_cast<int>(group)) p[r] = ld_peer(peer_addr(place, r));
          y[j] = 0.f;
#pragma unroll
          for (int r = 0; r < kMaxSplit; ++r)
            if (r < static_cast<int>(group)) y[j] += __uint_as_float(p[r]);
        }
        now.finish(a, y, t0 + at0 + at, kParts, left(at), n, in, ws, bias);
      }
    }
    __syncwarp();
    cluster_arrive();                        // nothing of the others' memory is read any more
    cluster_wait();
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

// -------------------------------------------------------------- few tokens
//
// Up to 16 tokens the weights' bytes are the work. A block takes 16 features, and its warps
// share out K: each multiplies 128 bytes of K of the 16 rows at a time by mma.sync, with the
// tokens as the 8-wide operand. A sum over K may be taken in any order, so a lane loads 16
// consecutive bytes of a row and uses them as the k-slots of two products; the tokens' lanes
// load the same places of x. No shared memory, barrier or copy engine stands between the loads
// and the products; the warps' sums meet in shared memory once, in the order of the warps.
// Plain loads: x, or fresh weights, may come from the kernel that still ended when this one
// started, and a load for data that no one writes (ld.global.nc) has no place there. They are
// also faster: one token, 8192 -> 2048 in bf16 7.9 us instead of 10.1, 8192 -> 8192 23.7, 27.0.

constexpr int kFewWarps = 16;              // at most
constexpr int kFewRows = 16;

template <bool E4M3, bool HALF>
__device__ __forceinline__ void mma_16x8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
#define MOEQ4_MMA_SYNC(OP)                                                                      \
  asm(OP " {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"                     \
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])                                          \
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1))
  if constexpr (E4M3) MOEQ4_MMA_SYNC("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32");
  else if constexpr (HALF) MOEQ4_MMA_SYNC("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32");
  else MOEQ4_MMA_SYNC("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32");
#undef MOEQ4_MMA_SYNC
}

struct FewArgs {
  const uint8_t *x, *w;
  int64_t x_row, w_row;      // bytes
  int k_bytes;               // of a row, a multiple of 16
  int early;                 // blocks that prefetch: one per multiprocessor
  LinearArgs l;
};

// NT groups of 8 tokens.
template <bool E4M3, bool HALF, typename O, int NT>
__global__ void __launch_bounds__(kFewWarps * 32, 2) linear_few_kernel(const FewArgs a) {
  __shared__ float part[kFewWarps][NT * 8][kFewRows + 1];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  const int n0 = blockIdx.x * kFewRows, warps = blockDim.x >> 5;
  // The first blocks ask for the start of their weights while the previous kernel ends: reads of
  // them wait for it, a prefetch into L2 does not (what that kernel writes reaches L2 all the
  // same). One token, 8192 -> 8192 in e4m3: 15.4 -> 15.0 us; whole rows, or all blocks: slower.
  if (blockIdx.x < a.early && tid < kFewRows && n0 + tid < a.l.N)
    bulk_prefetch_l2(a.w + static_cast<int64_t>(n0 + tid) * a.w_row, min(a.k_bytes, 4096));
  griddep_wait();
  griddep_launch_dependents();
  // rows past N repeat the last one, tokens past T the last token: nothing of them is written
  const uint8_t* wa = a.w + static_cast<int64_t>(min(n0 + g, a.l.N - 1)) * a.w_row + c * 16;
  const uint8_t* wb = a.w + static_cast<int64_t>(min(n0 + g + 8, a.l.N - 1)) * a.w_row + c * 16;
  const uint8_t* xp[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
    xp[i] = a.x + static_cast<int64_t>(min(i * 8 + g, a.l.T - 1)) * a.x_row + c * 16;
  float sum[NT][4];          // of pieces of 2 kU steps: the products' own sums are cut off
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) sum[i][j] = 0.f;
  constexpr int kU = NT == 1 ? 4 : 2;        // steps of 64 bytes whose loads go together
  const int last = a.k_bytes - c * 16;       // bytes of K from this lane's first place on
  for (int k0 = warp * 128; k0 < a.k_bytes; k0 += warps * 128 * (kU / 2)) {
    uint4 p[kU], q[kU], x[kU][NT];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int k = k0 + (u >> 1) * (warps * 128) + (u & 1) * 64;
      const bool in = k < last;
      const uint4 zero = make_uint4(0, 0, 0, 0);
      p[u] = in ? *reinterpret_cast<const uint4*>(wa + k) : zero;
      q[u] = in ? *reinterpret_cast<const uint4*>(wb + k) : zero;
#pragma unroll
      for (int i = 0; i < NT; ++i)
        x[u][i] = in ? *reinterpret_cast<const uint4*>(xp[i] + k) : zero;
    }
    float d[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) d[i][j] = 0.f;
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        mma_16x8<E4M3, HALF>(d[i], p[u].x, q[u].x, p[u].y, q[u].y, x[u][i].x, x[u][i].y);
        mma_16x8<E4M3, HALF>(d[i], p[u].z, q[u].z, p[u].w, q[u].w, x[u][i].z, x[u][i].w);
      }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[i][j] += d[i][j];
  }
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) part[warp][i * 8 + 2 * c + (j & 1)][g + (j >> 1) * 8] = sum[i][j];
  __syncthreads();
  for (int v = tid; v < NT * 8 * kFewRows; v += warps * 32) {
    const int t = v / kFewRows, r = v % kFewRows, n = n0 + r;
    if (t >= a.l.T || n >= a.l.N) continue;
    float y[1] = {0.f};
    for (int w = 0; w < warps; ++w) y[0] += part[w][t][r];
    if (E4M3) y[0] = y[0] * a.l.x_scale[t] * a.l.w_scale[n];
    if (a.l.bias) y[0] += a.l.bias[n];
    activate<sizeof(O) == 4>(y, a.l.act);
    if (a.l.add) y[0] += to_f(static_cast<const O*>(a.l.add)[t * a.l.add_row + n]);
    static_cast<O*>(a.l.out)[t * a.l.out_row + n] = to_out<O>(y[0]);
  }
}

template <bool E4M3, bool HALF, typename O>
cudaError_t launch_few(const FewArgs& a, cudaStream_t s) {
  // A warp for 256 elements of K, up to 16, or up to 8 where every multiprocessor has two blocks
  // anyway. Measured for one token, 16 and 8 warps: 2048 -> 2560 in bf16 3.4 and 3.3 us, 8192 ->
  // 2048 7.9 and 12.9, 2048 -> 8192 7.1 and 6.3; 8192 -> 8192 in e4m3 15.0 and 13.6. 2048 -> 2560
  // in e4m3 with 8 and 4 warps 2.8 and 3.4.
  const int blocks = (a.l.N - 1) / kFewRows + 1;
  const int most = blocks >= 2 * a.early ? kFewWarps / 2 : kFewWarps;
  const int per = E4M3 ? 256 : 512;          // bytes
  const dim3 grid(blocks), block(32 * std::min(most, (a.k_bytes + per - 1) / per));
  const auto kernel = a.l.T <= 8 ? linear_few_kernel<E4M3, HALF, O, 1>
                                 : linear_few_kernel<E4M3, HALF, O, 2>;
  return launch_pdl(kernel, grid, block, 0, s, a);
}

// Sizes of one call.
struct Plan {
  int mode, cols, splits, sub, stages, acc, tcols;
  bool pieces;
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

// Chunks per stage: a wait and a commit for several where their products are short. One token
// tile of 16 columns, 8192 -> 2048: 1, 2 and 4 chunks a stage 13.8, 12.1 and 11.5 us.
int chunks_per_stage(int cols, int chunks) {
  const int most = cols <= 16 ? 4 : cols <= 128 ? 2 : 1;
  return chunks >= most ? most : chunks >= 2 ? 2 : 1;
}

// Ring stages, tensor-memory columns and shared memory of a mode, tokens per tile and split.
void lay_out(Plan& p, int nch) {
  const int chunks = (nch + p.splits - 1) / p.splits, cb = chunk_bytes(p.cols, p.mode);
  p.acc = next_pow2(p.cols);
  p.tcols = std::max(32, p.mode == kSplit && !p.pieces ? p.acc : 2 * p.acc);
  const size_t fixed = 1024 + sizeof(Ctl);
  p.sub = chunks_per_stage(p.cols, chunks);
  const int sb = p.sub * cb;
  const int room = static_cast<int>((kSmemMax - fixed) / sb);
  p.stages = std::min({room, kMaxStages, std::max(2, (chunks + p.sub - 1) / p.sub)});
  p.smem = smem_for(p.tcols, fixed + static_cast<size_t>(p.stages) * sb);
}

// The mode, tokens per tile and split of the least time in a model of it (us), fitted to
// measurements: a K-chunk's time by columns, times the tiles that a multiprocessor takes in
// turn, but no less than the weights' bytes take, and a start and an end; those of a cluster
// grow with its size and their number. Model and measured, 2048 -> 2048: 64 tokens split by 4
// at 32 columns 7.5 and 7.2, by 8 9.9 and 9.0, not split 9.1 and 8.9; 2048 -> 8192: 4096 tokens
// in pairs 78 and 72, without 94 and 86; 8192 -> 8192: 16 tokens split by 2 25.6 and 24.1, not
// split 27.9 and 27.8.
Plan make_plan(int T, int N, int nch, bool pieces, int sms) {
  const int rows_n = (N + kRows - 1) / kRows;
  const int most = std::min(kMaxCols, (T + 15) / 16 * 16);
  const double bytes = static_cast<double>(N) * nch * kChunk;
  double best = 1e300;
  Plan p{};
  p.pieces = pieces;
  const auto offer = [&](int mode, int cols, int splits, double cost) {
    if (cost >= best) return;
    best = cost;
    p.mode = mode;
    p.cols = cols;
    p.splits = splits;
  };
  // 0.085 TB/s for each block, 6.8 for all
  const auto fetch = [&](double blocks) { return bytes / std::min(6.8e6, 0.085e6 * blocks); };
  for (int cols = 16; cols <= most; cols += 16) {
    const int64_t tiles_t = (T + cols - 1) / cols, tiles = rows_n * tiles_t;
    const double chunk = cols <= 16 ? 0.13 : std::max(0.175, 0.07 + 0.00125 * cols);
    offer(kSingle, cols, 1,
          std::max(static_cast<double>((tiles + sms - 1) / sms) * nch * chunk,
                   fetch(static_cast<double>(tiles))) + 3.2 + 0.011 * cols);
    if (cols % 32 == 0 && sms >= 2) {
      const int64_t pairs = (rows_n + 1) / 2 * tiles_t;
      offer(kPair, cols, 1,
            std::max(static_cast<double>((pairs + sms / 2 - 1) / (sms / 2)) * nch *
                         (0.165 + 0.0006 * cols),
                     fetch(2.0 * pairs)) + 4.2 + 0.011 * cols);
    }
    if (cols > kMaxSplitCols || tiles >= sms) continue;
    for (int splits = 2; splits <= kMaxSplit && splits <= nch; splits *= 2) {
      // Clusters side by side: all blocks of one find room within a group of multiprocessors
      // (8 of 19 on this device: 76, 36 and 15 clusters of 2, 4 and 8 blocks that have a
      // multiprocessor each, and a little more than twice that at half its shared memory).
      Plan q{};
      q.mode = kSplit;
      q.cols = cols;
      q.splits = splits;
      q.pieces = pieces;
      lay_out(q, nch);
      const int per_sm = static_cast<int>(kSmemMax + 1024) / static_cast<int>(q.smem + 1024);
      const int64_t room = std::max(1, sms / 8 * per_sm / splits * 8 - (per_sm == 1 ? 1 : 0));
      const double turns = static_cast<double>((tiles + room - 1) / room);
      const double blocks = static_cast<double>(std::min(tiles, room)) * splits;
      const double end = 1.9 + 0.13 * splits + 0.013 * blocks + 0.00015 * cols * cols;
      offer(kSplit, cols, splits,
            std::max(turns * ((nch + splits - 1) / splits) * chunk, fetch(blocks)) + turns * end + 2.0);
    }
  }
  lay_out(p, nch);
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

// Measured, few-token kernel and the better of the others, us: 1 token 2048 -> 2560 3.3 and 5.9,
// 8192 -> 8192 23.2 and 24.0, 2048 -> 16384 15.8 and 13.6; 16 tokens 2048 -> 4096 4.7 and 6.7,
// 2048 -> 8192 9.9 and 8.6, 8192 -> 2048 10.9 and 10.0, 8192 -> 8192 28.4 and 24.7.
bool take_few(int T, int N) { return (T <= 8 && N <= 8192) || (T <= 16 && N <= 4096); }

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
  if (l->K % (16 / es) || l->K > kMaxK || l->T > kMaxRows || l->N > kMaxRows) return MOE_ERR_SHAPE;
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
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (take_few(l->T, l->N)) {
    FewArgs f{};
    f.x = static_cast<const uint8_t*>(l->x);
    f.w = static_cast<const uint8_t*>(l->w);
    f.x_row = l->T > 1 ? l->x_row * es : 0;
    f.w_row = l->N > 1 ? l->w_row * es : 0;
    f.k_bytes = l->K * es;
    f.early = sms;
    f.l = a;
    cudaError_t e;
    if (e4m3)
      e = l->out_dtype == MOE_F32   ? launch_few<true, false, float>(f, s)
          : l->out_dtype == MOE_F16 ? launch_few<true, false, __half>(f, s)
                                    : launch_few<true, false, __nv_bfloat16>(f, s);
    else if (l->dtype == MOE_F16)
      e = l->out_dtype == MOE_F32 ? launch_few<false, true, float>(f, s)
                                  : launch_few<false, true, __half>(f, s);
    else
      e = l->out_dtype == MOE_F32 ? launch_few<false, false, float>(f, s)
                                  : launch_few<false, false, __nv_bfloat16>(f, s);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  }
  const Plan p = make_plan(l->T, l->N, a.nch, l->out_dtype == MOE_F32, sms);
  a.cols = p.cols;
  const int fw = p.mode == kPair ? 2 * kRows : kRows;
  a.tiles_n = (l->N - 1) / fw + 1;
  a.tiles_t = (l->T - 1) / p.cols + 1;
  if (static_cast<int64_t>(a.tiles_n) * a.tiles_t * p.splits > 0x7FFFFFFF - 1024) return MOE_ERR_SHAPE;
  a.stages = p.stages;
  a.sub = p.sub;
  a.acc = p.acc;
  a.tcols = p.tcols;
  a.band = p.mode == kPair ? 8 : 12;         // about the square root of the tiles under way
  // instruction descriptor: fp32 D, both operands K-major, M = features, N = cols; operand types
  // fp16 (0) or bf16 (1), or e4m3 (0)
  const uint32_t type = l->dtype == MOE_BF16 ? 1u : 0u;
  a.idesc = (1u << 4) | (type << 7) | (type << 10) | (static_cast<uint32_t>(p.cols >> 3) << 17) |
            (static_cast<uint32_t>(fw >> 4) << 24);
  // a single row has no stride: any multiple of 16 bytes will do
  const uint64_t one = (static_cast<uint64_t>(l->K) * es + 15) / 16 * 16;
  a.cube = l->K % elems == 0 && p.sub > 1;
  const int depth = a.cube ? p.sub : 1;
  CUtensorMap tx, tw;
  if (!map_rows(&tx, l->dtype, l->x, l->K, l->T, l->T > 1 ? l->x_row * es : one, elems,
                p.mode == kPair ? p.cols / 2 : p.cols, depth) ||
      !map_rows(&tw, l->dtype, l->w, l->K, l->N, l->N > 1 ? l->w_row * es : one, elems, kRows,
                depth))
    return MOE_ERR_CUDA;
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
                                            int32_t out_dtype, int32_t sms, int32_t* plan) {
  using namespace moeq4;
  if (T < 1 || N < 1 || K < 1 || sms < 1 || !plan) return MOE_ERR_ARG;
  const int elems = dtype == MOE_E4M3 ? kChunk : kChunk / 2, nch = (K + elems - 1) / elems;
  const Plan p = make_plan(T, N, nch, out_dtype == MOE_F32, sms);
  const int32_t v[8] = {p.cols, p.splits, p.stages, p.acc, p.tcols, static_cast<int32_t>(p.smem),
                        p.mode, p.sub};
  for (int i = 0; i < 8; ++i) plan[i] = v[i];
  return MOE_OK;
}
