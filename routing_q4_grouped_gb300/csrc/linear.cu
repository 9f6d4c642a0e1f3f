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
// tensor memory let four warps finish a tile while the next one is multiplied. Where the
// tiles are too few for the multiprocessors, a cluster of 2, 4 or 8 blocks splits K: each
// sends its partial sums to the block that finishes their tokens through distributed
// shared memory, where they are added in the order of the blocks.
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
constexpr int kThreads = 192;              // producer, MMA issuer, 4 epilogue warps
constexpr int kRows = 128;                 // features per tile (MMA M)
constexpr int kChunk = 128;                // bytes of K per stage and row
constexpr int kMaxCols = 256;              // tokens per tile at most (MMA N)
constexpr int kMaxStages = 12;
constexpr int kMaxSplit = 8;
constexpr int kMaxSplitCols = 128;         // tokens per tile at most where K is split
constexpr size_t kSmemMax = 227 * 1024;

struct LinearArgs {
  int T, N;
  int nch;                   // K-chunks
  int cols;                  // tokens per tile, a multiple of 16
  int tiles_n, tiles_t;
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
  uint32_t peer_ok[kMaxSplit][4];            // [block][warp]: its partial sums were sent
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

// One K-chunk (4 steps of 32 bytes of K) of D[features, tokens] += W X^T, issued by one
// elected lane of a converged warp. The first step accumulates only if `accumulate`.
template <bool E4M3>
__device__ __forceinline__ void mma_chunk(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
  if constexpr (E4M3) {
    asm volatile(
        "{\n\t.reg .pred e, p;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "add.u64 a1, %1, 2;\n\tadd.u64 a2, %1, 4;\n\tadd.u64 a3, %1, 6;\n\t"
        "add.u64 b1, %2, 2;\n\tadd.u64 b2, %2, 4;\n\tadd.u64 b3, %2, 6;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, b2, %3, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, b3, %3, 1;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred e, p;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "add.u64 a1, %1, 2;\n\tadd.u64 a2, %1, 4;\n\tadd.u64 a3, %1, 6;\n\t"
        "add.u64 b1, %2, 2;\n\tadd.u64 b2, %2, 4;\n\tadd.u64 b3, %2, 6;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, 1;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  }
}

template <typename O>
__device__ __forceinline__ float load_f(const O* p);
template <>
__device__ __forceinline__ float load_f(const __nv_bfloat16* p) { return __bfloat162float(*p); }
template <>
__device__ __forceinline__ float load_f(const __half* p) { return __half2float(*p); }
template <>
__device__ __forceinline__ float load_f(const float* p) { return *p; }
template <typename O>
__device__ __forceinline__ O to_out(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 to_out(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half to_out(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float to_out(float v) { return v; }

__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case MOE_ACT_RELU: return v < 0.f ? 0.f : v;               // (NaN stays)
    case MOE_ACT_SILU: return v / (1.f + expf(-v));
    case MOE_ACT_GELU: return 0.5f * v * (1.f + erff(v * 0.70710678118654752f));
    case MOE_ACT_GELU_TANH:
      return 0.5f * v * (1.f + tanhf(0.79788456080286536f * fmaf(0.044715f * v * v, v, v)));
    default: return v;
  }
}

// One element from its sum: scales, bias, activation, residual, one rounding.
template <bool E4M3, typename O>
__device__ __forceinline__ void finish(const LinearArgs& a, float v, int64_t t, int n, float ws,
                                       float bias) {
  if (E4M3) v = v * a.x_scale[t] * ws;
  v = activate(v + bias, a.act);
  if (a.add) v += load_f(static_cast<const O*>(a.add) + t * a.add_row + n);
  static_cast<O*>(a.out)[t * a.out_row + n] = to_out<O>(v);
}

__host__ __device__ inline int stage_bytes(int cols) { return (kRows + cols) * kChunk; }

template <bool E4M3, typename O, bool SPLIT>
__global__ void __launch_bounds__(kThreads)
    linear_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                  const LinearArgs a) {
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int sb = stage_bytes(a.cols), ns = a.stages;
  // behind the ring: partial sums [source block][token][feature] (split K), then control
  float* parts = reinterpret_cast<float*>(smem + static_cast<size_t>(ns) * sb);
  Ctl& ctl = *reinterpret_cast<Ctl*>(reinterpret_cast<uint8_t*>(parts) +
                                     (SPLIT ? static_cast<size_t>(a.cols) * kRows * 4 : 0));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t splits = 1, rank = 0;
  if constexpr (SPLIT) {
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(splits));
    rank = cluster_rank();
  }
  if (tid == 0) {
    for (int s = 0; s < ns; ++s) {
      mbar_init(&ctl.full[s], 1);
      mbar_init(&ctl.empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctl.acc_full[s], 1);
      mbar_init(&ctl.acc_empty[s], 4);
    }
    mbar_init(&ctl.drained, 1);
    ctl.abort = 0;
    ctl.zero = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_x);
    tma_prefetch_desc(&tm_w);
  }
  if (warp == 1) {
    tmem_alloc(&ctl.tmem, a.tcols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if constexpr (SPLIT) cluster_arrive();     // (this block's shared memory may be written to)
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t tmem = ctl.tmem;
  const volatile int* abortp = &ctl.abort;
  const uint64_t lim = a.timeout_ns;
  const int tiles = a.tiles_n * a.tiles_t;
  const int first = static_cast<int>(blockIdx.x / splits), step = static_cast<int>(gridDim.x / splits);
  // this block's chunks of every tile
  const int c_lo = static_cast<int>(static_cast<int64_t>(a.nch) * rank / splits);
  const int c_hi = static_cast<int>(static_cast<int64_t>(a.nch) * (rank + 1) / splits);
  bool ok = true;
  int n0 = 0, t0 = 0;                        // of the tile that the epilogue holds at the end

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      const uint64_t pol = policy_evict_last();
      int it = 0;                            // chunks requested
      for (int tile = first; tile < tiles && ok; tile += step) {
        const int tn = tile / a.tiles_t * kRows, tt = tile % a.tiles_t * a.cols;
        for (int c = c_lo; c < c_hi; ++c, ++it) {
          const int s = it % ns;
          if (!mbar_wait(&ctl.empty[s], ((it / ns) & 1) ^ 1, abortp, lim)) {
            ok = false;
            break;
          }
          uint8_t* st = smem + static_cast<size_t>(s) * sb;
          mbar_arrive_expect_tx(&ctl.full[s], sb);
          constexpr int kElems = E4M3 ? kChunk : kChunk / 2;
          tma_load_2d(st, &tm_w, &ctl.full[s], c * kElems, tn, pol);
          tma_load_2d(st + kRows * kChunk, &tm_x, &ctl.full[s], c * kElems, tt, pol);
        }
      }
      if (!ok) {
        if (atomicExch(&ctl.abort, 1) == 0) atomicOr(a.err, MOE_DEVERR_PIPE_TIMEOUT);
      }
      // every copy has landed before the block's shared memory goes away (at the end of a
      // whole run they have, and the waits return at once)
      for (int i = 1; i <= min(it, ns); ++i) {
        const int c = it - i;
        mbar_wait(&ctl.full[c % ns], (c / ns) & 1, &ctl.zero, 20000000ull);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------- MMA issuer
    int it = 0, i = 0;                       // chunks and tiles multiplied
    for (int tile = first; tile < tiles && ok; tile += step, ++i) {
      const int b = i & 1;
      ok = __all_sync(kFull, mbar_wait(&ctl.acc_empty[b], ((i >> 1) & 1) ^ 1, abortp, lim));
      tc_fence_after();
      for (int c = c_lo; c < c_hi && ok; ++c, ++it) {
        const int s = it % ns;
        ok = __all_sync(kFull, mbar_wait(&ctl.full[s], (it / ns) & 1, abortp, lim));
        if (!ok) break;
        tc_fence_after();
        const uint32_t sa = smem_u32(smem + static_cast<size_t>(s) * sb);
        mma_chunk<E4M3>(tmem + b * a.acc, sdesc_k_sw128(sa), sdesc_k_sw128(sa + kRows * kChunk),
                        a.idesc, c != c_lo);
        mma_commit_elect(&ctl.empty[s]);
      }
      if (ok) mma_commit_elect(&ctl.acc_full[b]);
    }
    if (!ok && lane == 0 && atomicExch(&ctl.abort, 1) == 0)
      atomicOr(a.err, MOE_DEVERR_PIPE_TIMEOUT);
    // no product is under way when tensor memory is given back
    mma_commit_elect(&ctl.drained);
    mbar_wait(&ctl.drained, 0, &ctl.zero, 20000000ull);
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- epilogue
    // warp w reads tensor-memory lanes 32 (w % 4) ..: features n, one per lane
    const int q = warp & 3;
    int i = 0;
    for (int tile = first; tile < tiles && ok; tile += step, ++i) {
      const int b = i & 1;
      n0 = tile / a.tiles_t * kRows;
      t0 = tile % a.tiles_t * a.cols;
      const int n = n0 + q * 32 + lane;
      const bool in = n < a.N;
      const float bias = in && a.bias ? a.bias[n] : 0.f;
      const float ws = in && E4M3 ? a.w_scale[n] : 1.f;
      ok = __all_sync(kFull, mbar_wait(&ctl.acc_full[b], (i >> 1) & 1, abortp, lim));
      if (!ok) break;
      tc_fence_after();
      const uint32_t taddr = tmem + b * a.acc + (static_cast<uint32_t>(q * 32) << 16);
      if constexpr (SPLIT) cluster_wait();   // every block of the cluster has started
      const int per = a.cols / static_cast<int>(splits);
      for (int c = 0; c < a.cols; c += 16) {
        uint32_t v[16];
        tmem_ld_32x32b_x16(taddr + c, v);
        tmem_ld_wait();
        tmem_regs_ready(v);
        if constexpr (SPLIT) {
          // tokens [r per, r per + per) are finished by block r
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            if (t0 + c + j >= a.T) break;
            const int owner = (c + j) / per, at = (c + j) % per;
            st_peer(peer_addr(smem_u32(parts + (rank * per + at) * kRows + q * 32 + lane), owner),
                    v[j]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int t = t0 + c + j;
            if (t >= a.T) break;
            if (in) finish<E4M3, O>(a, __uint_as_float(v[j]), t, n, ws, bias);
          }
          __syncwarp();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.acc_empty[b]);
    }
    if (!ok && lane == 0 && atomicExch(&ctl.abort, 1) == 0)
      atomicOr(a.err, MOE_DEVERR_PIPE_TIMEOUT);
  }
  if constexpr (SPLIT) {
    // one tile per cluster. Each barrier is reached by every thread, whatever happened before
    // it; the epilogue's warps passed the first one above unless they gave up.
    if (warp < 2 || !ok) cluster_wait();
    if (warp >= 2 && lane < splits)
      st_peer(peer_addr(smem_u32(&ctl.peer_ok[rank][warp & 3]), lane), ok ? 1u : 0u);
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    bool all = true;
    for (uint32_t r = 0; r < splits; ++r) all = all && ctl.peer_ok[r][warp & 3] != 0;
    if (warp >= 2 && all) {
      const int per = a.cols / static_cast<int>(splits);
      const int f = (warp & 3) * 32 + lane, n = n0 + f;
      if (n < a.N) {
        const float bias = a.bias ? a.bias[n] : 0.f, ws = E4M3 ? a.w_scale[n] : 1.f;
        for (int at = 0; at < per; ++at) {
          const int t = t0 + static_cast<int>(rank) * per + at;
          if (t >= a.T) break;
          float v = 0.f;
          for (uint32_t r = 0; r < splits; ++r) v += parts[(r * per + at) * kRows + f];
          finish<E4M3, O>(a, v, t, n, ws, bias);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, a.tcols);
  }
}

// Sizes of one call: tokens per tile, blocks that share a tile's K, ring stages.
struct Plan {
  int cols, splits, stages, acc, tcols;
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

Plan make_plan(int T, int N, int nch, int sms) {
  const int tiles_n = (N + kRows - 1) / kRows;
  const int most = std::min(kMaxCols, (T + 15) / 16 * 16);
  double best = 1e300;
  Plan p{};
  for (int splits = 1; splits <= kMaxSplit && splits <= nch; splits *= 2) {
    for (int cols = 16; cols <= most; cols += 16) {
      if (splits > 1 && cols > kMaxSplitCols) break;
      const int64_t tiles = static_cast<int64_t>(tiles_n) * ((T + cols - 1) / cols);
      // cycles: products, or the copies that feed them, and a start and an end per call
      const double chunk = std::max(2.0 * cols, stage_bytes(cols) / 64.0);
      const double turns = static_cast<double>((tiles * splits + sms - 1) / sms);
      const double cost = turns * ((nch + splits - 1) / splits * chunk + 100.0) + 8.0 * cols +
                          (splits > 1 ? 1500.0 + 10.0 * cols : 0.0);
      if (cost < best) {
        best = cost;
        p.cols = cols;
        p.splits = splits;
      }
    }
  }
  p.acc = next_pow2(p.cols);
  p.tcols = std::max(32, p.splits > 1 ? p.acc : 2 * p.acc);
  const size_t fixed = 1024 + sizeof(Ctl) +
                       (p.splits > 1 ? static_cast<size_t>(p.cols) * kRows * sizeof(float) : 0);
  const int room = static_cast<int>((kSmemMax - fixed) / stage_bytes(p.cols));
  p.stages = std::min({room, kMaxStages, std::max(2, (nch + p.splits - 1) / p.splits)});
  p.smem = smem_for(p.tcols, fixed + static_cast<size_t>(p.stages) * stage_bytes(p.cols));
  return p;
}

template <bool E4M3, typename O, bool SPLIT>
cudaError_t launch(const CUtensorMap& tx, const CUtensorMap& tw, const LinearArgs& a, const Plan& p,
                   int sms, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(linear_kernel<E4M3, O, SPLIT>, kSmemMax, done);
  if (e != cudaSuccess) return e;
  const int64_t tiles = static_cast<int64_t>(a.tiles_n) * a.tiles_t;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(SPLIT ? tiles * p.splits : std::min<int64_t>(tiles, sms)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = p.smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.splits;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = SPLIT ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, linear_kernel<E4M3, O, SPLIT>, tx, tw, a);
}

template <bool E4M3, typename O>
cudaError_t launch_out(const CUtensorMap& tx, const CUtensorMap& tw, const LinearArgs& a,
                       const Plan& p, int sms, cudaStream_t s) {
  return p.splits > 1 ? launch<E4M3, O, true>(tx, tw, a, p, sms, s)
                      : launch<E4M3, O, false>(tx, tw, a, p, sms, s);
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
  a.tiles_n = (l->N - 1) / kRows + 1;
  a.tiles_t = (l->T - 1) / p.cols + 1;
  if (static_cast<int64_t>(a.tiles_n) * a.tiles_t * p.splits > 0x7FFFFFFF - 1024) return MOE_ERR_SHAPE;
  a.stages = p.stages;
  a.acc = p.acc;
  a.tcols = p.tcols;
  // instruction descriptor: fp32 D, both operands K-major, M = 128, N = cols; operand types
  // fp16 (0) or bf16 (1), or e4m3 (0)
  const uint32_t type = l->dtype == MOE_BF16 ? 1u : 0u;
  a.idesc = (1u << 4) | (type << 7) | (type << 10) | (static_cast<uint32_t>(p.cols >> 3) << 17) |
            (static_cast<uint32_t>(kRows >> 4) << 24);
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
  if (!map_rows(&tx, l->dtype, l->x, l->K, l->T, l->T > 1 ? l->x_row * es : one, elems, p.cols) ||
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
  const int32_t v[6] = {p.cols, p.splits, p.stages, p.acc, p.tcols, static_cast<int32_t>(p.smem)};
  for (int i = 0; i < 6; ++i) plan[i] = v[i];
  return MOE_OK;
}
