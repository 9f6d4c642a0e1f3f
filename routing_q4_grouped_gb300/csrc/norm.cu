// norm.cu — residual addition and root-mean-square norm (moe_rms_norm), with the
// result in the input's type, in 8 bits with one scale per row, or both.
//
//   h = x + add,  r = 1 / sqrt(mean(h^2) + eps),  y = h r (weight + offset)
//   scale = max(max|y| / 448, 2^-126),  code = e4m3(y / scale)
//
// Each byte moves once and each element takes a few instructions, so many rows are
// bound by memory bandwidth and few rows by launch latency. A row is held in registers
// between its reductions (nothing is read twice): by 8, 16 or 32 lanes where it has up
// to 64 vectors of 16 bytes, by a block of up to 512 threads where it has more. Two
// vectors a thread: measured for 4096 rows of 2048 bf16 elements with a residual (67 MB)
// 11.9 us, one vector 13.2, four 12.6. 40 registers for 1536 threads on a
// multiprocessor: 8191 rows of 5120 into codes 50.4 us, with 64 registers 56.4.
// Measured bandwidth, of a copy's 6.7 TB/s: 6.7 for 4096 fp32 rows of 4096, 6.8 for
// 8191 bf16 rows of 5120, 5.8 into codes (33 instructions an element, issue slots 73 %
// used). 4096 rows that vectors of 16 bytes do not fit: of 2050 elements, two a load,
// 4.0; of 2047, one a load, 2.9.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "../../include/moeq4.h"
#include "internal.h"
#include "ptx.cuh"

namespace moeq4 {
namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;
constexpr int kMaxD = 16384;
constexpr float kCodeMax = 448.f;                    // largest e4m3 value
constexpr float kScaleMin = 1.17549435e-38f;         // 2^-126: its reciprocal is finite

struct NormArgs {
  const void *x, *add, *weight;
  void *sum, *out;
  uint8_t* codes;
  float* scales;
  int64_t x_row, x_head, add_row, add_head, sum_row, sum_head, out_row, out_head, c_row, c_head;
  int rows, H, D;            // rows = T * H
  int n;                     // vectors per row, D / V
  float eps, offset, inv_d;
};

template <typename E, int V>
struct alignas(V * sizeof(E)) Vec {
  E e[V];
};
template <int V>
struct alignas(V) Bytes {
  uint8_t e[V];
};
// Two e4m3 codes, the first in the low byte.
__device__ __forceinline__ uint32_t two_codes(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f(float v) { return v; }
template <typename E>
__device__ __forceinline__ E from_f(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float from_f(float v) { return v; }

// The elements of a vector as floats, and back, two at a time where they have 16 bits.
template <int V>
__device__ __forceinline__ void unpack(const Vec<__nv_bfloat16, V>& p, float (&f)[V]) {
  if constexpr (V % 2 == 0) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&p);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    f[0] = to_f(p.e[0]);
  }
}
template <int V>
__device__ __forceinline__ void unpack(const Vec<__half, V>& p, float (&f)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = to_f(p.e[i]);
}
template <int V>
__device__ __forceinline__ void unpack(const Vec<float, V>& p, float (&f)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = p.e[i];
}
template <typename E, int V>
__device__ __forceinline__ Vec<E, V> pack(const float (&f)[V]) {
  Vec<E, V> w;
  if constexpr (V % 2 == 0 && sizeof(E) == 2) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      if constexpr (std::is_same_v<E, __nv_bfloat16>)
        *reinterpret_cast<__nv_bfloat162*>(&w.e[i]) = __floats2bfloat162_rn(f[i], f[i + 1]);
      else
        *reinterpret_cast<__half2*>(&w.e[i]) = __floats2half2_rn(f[i], f[i + 1]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) w.e[i] = from_f<E>(f[i]);
  }
  return w;
}

// Sum and unsigned maximum over the lanes of a row: LANES neighbouring lanes of a warp
// (LANES <= 32), or the whole block (LANES = 0; `sh` holds two words per warp and is used by one
// call only; the order of the additions is fixed).
template <int LANES, bool MAX>
__device__ __forceinline__ void row_reduce(float& sum, uint32_t& most, float* sh) {
  constexpr int kFirst = (LANES == 0 ? 32 : LANES) / 2;
#pragma unroll
  for (int off = kFirst; off > 0; off >>= 1) {
    sum += __shfl_xor_sync(kFull, sum, off);
    if (MAX) most = max(most, __shfl_xor_sync(kFull, most, off));
  }
  if constexpr (LANES == 0) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) {
      sh[warp] = sum;
      if (MAX) sh[16 + warp] = __uint_as_float(most);
    }
    __syncthreads();
    sum = lane < warps ? sh[lane] : 0.f;             // (at most 16 warps)
    if (MAX) most = lane < warps ? __float_as_uint(sh[16 + lane]) : 0u;
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) {
      sum += __shfl_xor_sync(kFull, sum, off);
      if (MAX) most = max(most, __shfl_xor_sync(kFull, most, off));
    }
    sum = __shfl_sync(kFull, sum, 0);                // (lanes 16.. added up zeros)
    if (MAX) most = __shfl_sync(kFull, most, 0);
  }
}

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// What follows the loads: the sum's store, reductions, results. v holds h of row `row` (token t,
// head `head`): vector u of the row in thread tid = u % lanes. CODES: with the 8-bit result, whose
// largest magnitude is reduced together with the sum of squares, as that of h (weight + offset).
template <typename E, int V, int NV, int LANES, bool CODES>
__device__ __forceinline__ void finish_row(const NormArgs& a, float (&v)[NV][V], int64_t row,
                                           uint32_t t, uint32_t head, bool live, int tid, int lanes,
                                           float (*sh)[32]) {
  using Vt = Vec<E, V>;
  const auto at = [&](int64_t by_row, int64_t by_head) {
    return static_cast<int64_t>(t) * by_row + static_cast<int64_t>(head) * by_head;
  };
  const Vt* weight = static_cast<const Vt*>(a.weight);
  if (a.sum && live) {
    Vt* o = reinterpret_cast<Vt*>(static_cast<E*>(a.sum) + at(a.sum_row, a.sum_head));
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (tid + j * lanes < a.n) o[tid + j * lanes] = pack<E>(v[j]);
  }
  // weight + offset of the thread's j-th vector (0 past the row, where v is 0 too)
  const auto gains = [&](int j, float (&g)[V]) {
    if (a.weight) {
      Vt w{};
      if (tid + j * lanes < a.n) w = weight[tid + j * lanes];
      unpack(w, g);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) g[i] = 1.f;
    }
    if (a.offset != 0.f) {
#pragma unroll
      for (int i = 0; i < V; ++i) g[i] += a.offset;
    }
  };
  float ss = 0.f;
  uint32_t most = 0;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float g[V];
    if (CODES) gains(j, g);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      ss = fmaf(v[j][i], v[j][i], ss);
      if (CODES) most = max(most, magnitude(v[j][i] * g[i]));
    }
  }
  row_reduce<LANES, CODES>(ss, most, sh[0]);
  float by = __frsqrt_rn(fmaf(ss, a.inv_d, a.eps));
  // Squares that left fp32's range, above or (beside a small eps) below: again, on elements
  // scaled by a power of two. All lanes of a warp, or of the block, take part.
  const bool odd = !(ss < 1e37f) || ss < 1e-24f;
  if (LANES == 0 ? odd : __any_sync(kFull, odd)) {
    uint32_t m = 0;
    float s2 = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) m = max(m, magnitude(v[j][i]));
    row_reduce<LANES, true>(s2, m, sh[1]);
    const int e = m != 0 && m < 0x7F800000u ? ilogbf(__uint_as_float(m)) : 0;
    const float f0 = __int_as_float((127 - e / 2) << 23);            // 2^-e in two factors
    const float f1 = __int_as_float((127 - (e - e / 2)) << 23);
    s2 = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float z = v[j][i] * f0 * f1;
        s2 = fmaf(z, z, s2);
      }
    row_reduce<LANES, false>(s2, m, sh[2]);
    if (odd)
      by = static_cast<float>(1.0 / sqrt(ldexp(static_cast<double>(s2) / a.D, 2 * e) +
                                         static_cast<double>(a.eps)));
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float g[V];
    gains(j, g);
#pragma unroll
    for (int i = 0; i < V; ++i) v[j][i] = v[j][i] * by * g[i];
  }
  if (a.out && live) {
    Vt* o = reinterpret_cast<Vt*>(static_cast<E*>(a.out) + at(a.out_row, a.out_head));
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (tid + j * lanes < a.n) o[tid + j * lanes] = pack<E>(v[j]);
  }
  if constexpr (CODES) {
    // (the largest product may have left fp32's range where the result does not: from the
    // results then)
    const float product = __uint_as_float(most);
    const bool far = odd || most >= 0x7F800000u || (product < 1e-30f && most != 0);
    uint32_t m = __float_as_uint(product * by);
    if (LANES == 0 ? far : __any_sync(kFull, far)) {
      uint32_t again = 0;
      float none = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (tid + j * lanes < a.n) again = max(again, magnitude(v[j][i]));
      row_reduce<LANES, true>(none, again, sh[3]);
      if (far) m = again;
    }
    const float scale = m < 0x7F800000u
                            ? fmaxf(__uint_as_float(m) * (1.f / kCodeMax), kScaleMin)
                            : __uint_as_float(0x7FC00000u);
    const float inv = __frcp_rn(scale);
    if (live) {
      if (tid == 0) a.scales[row] = scale;
      Bytes<V>* o = reinterpret_cast<Bytes<V>*>(a.codes + at(a.c_row, a.c_head));
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        Bytes<V> w;
        if constexpr (V % 4 == 0) {
          uint32_t* words = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
          for (int i = 0; i < V; i += 4)
            words[i / 4] = __byte_perm(two_codes(v[j][i] * inv, v[j][i + 1] * inv),
                                       two_codes(v[j][i + 2] * inv, v[j][i + 3] * inv), 0x5410);
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i)
            w.e[i] = __nv_cvt_float_to_fp8(v[j][i] * inv, __NV_SATFINITE, __NV_E4M3);
        }
        if (tid + j * lanes < a.n) o[tid + j * lanes] = w;
      }
    }
  }
}

// A row per LANES lanes (LANES = 0: per block), NV vectors of V elements per thread.
template <typename E, int V, int NV, int LANES, bool CODES>
__global__ void __launch_bounds__(LANES == 0 ? 512 : 128, LANES == 0 && NV * V <= 16 ? 3 : 1)
    norm_kernel(NormArgs a) {
  __shared__ float sh[4][32];
  griddep_wait();
  griddep_launch_dependents();
  const int lanes = LANES == 0 ? static_cast<int>(blockDim.x) : LANES;
  const int tid = LANES == 0 ? static_cast<int>(threadIdx.x)
                             : static_cast<int>(threadIdx.x) % lanes;
  const int64_t row = LANES == 0 ? static_cast<int64_t>(blockIdx.x)
                                 : static_cast<int64_t>(blockIdx.x) * (blockDim.x / lanes) +
                                       threadIdx.x / lanes;
  const bool live = row < a.rows;        // (lanes of a dead row take part in the reductions)
  const uint32_t some = static_cast<uint32_t>(live ? row : 0);
  const uint32_t t = a.H == 1 ? some : some / static_cast<uint32_t>(a.H), h = some - t * a.H;
  using Vt = Vec<E, V>;
  float v[NV][V];
  {
    const Vt* x = reinterpret_cast<const Vt*>(static_cast<const E*>(a.x) + t * a.x_row + h * a.x_head);
    const Vt* add =
        reinterpret_cast<const Vt*>(static_cast<const E*>(a.add) + t * a.add_row + h * a.add_head);
    Vt p[NV], q[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int u = tid + j * lanes;
      p[j] = Vt{};
      q[j] = Vt{};
      if (live && u < a.n) {
        p[j] = x[u];
        if (a.add) q[j] = add[u];
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) unpack(p[j], v[j]);
    if (a.add) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float b[V];
        unpack(q[j], b);
#pragma unroll
        for (int i = 0; i < V; ++i) v[j][i] += b[i];
      }
    }
  }
  finish_row<E, V, NV, LANES, CODES>(a, v, row, t, h, live, tid, lanes, sh);
}

template <typename E, int V, int NV, int LANES>
cudaError_t launch_rows(const NormArgs& a, int threads, cudaStream_t s) {
  const int64_t per = LANES == 0 ? 1 : threads / LANES;
  const dim3 blocks(static_cast<unsigned>((a.rows + per - 1) / per)), block(threads);
  return a.codes ? launch_pdl(norm_kernel<E, V, NV, LANES, true>, blocks, block, 0, s, a)
                 : launch_pdl(norm_kernel<E, V, NV, LANES, false>, blocks, block, 0, s, a);
}

int round32(int n) { return (n + 31) / 32 * 32; }

template <typename E, int V>
cudaError_t launch_norm_v(NormArgs a, cudaStream_t s) {
  a.n = a.D / V;
  constexpr int kWarpRows = 128;         // threads of a block of several rows
  if (a.n <= 8) return launch_rows<E, V, 1, 8>(a, kWarpRows, s);
  if (a.n <= 16) return launch_rows<E, V, 2, 8>(a, kWarpRows, s);
  if (a.n <= 32) return launch_rows<E, V, 2, 16>(a, kWarpRows, s);
  if (a.n <= 64) return launch_rows<E, V, 2, 32>(a, kWarpRows, s);
  if (a.n <= 1024) return launch_rows<E, V, 2, 0>(a, round32((a.n + 1) / 2), s);
  if (a.n <= 2048) return launch_rows<E, V, 4, 0>(a, round32((a.n + 3) / 4), s);
  if constexpr (V * sizeof(E) < 16 || sizeof(E) == 4) {
    if (a.n <= 4096) return launch_rows<E, V, 8, 0>(a, round32((a.n + 7) / 8), s);
  }
  if constexpr (V <= 2 && V * sizeof(E) <= 4) {
    if (a.n <= 8192) return launch_rows<E, V, 16, 0>(a, round32((a.n + 15) / 16), s);
  }
  if constexpr (V == 1) return launch_rows<E, V, 32, 0>(a, round32((a.n + 31) / 32), s);
  return cudaErrorInvalidValue;
}

// Vectors of 16 bytes, of two 16-bit elements, or single elements.
template <typename E>
cudaError_t launch_norm(const NormArgs& a, cudaStream_t s) {
  const uint64_t strides =
      static_cast<uint64_t>(a.x_row | a.x_head | (a.add ? a.add_row | a.add_head : 0) |
                            (a.sum ? a.sum_row | a.sum_head : 0) |
                            (a.out ? a.out_row | a.out_head : 0) |
                            (a.codes ? a.c_row | a.c_head : 0));
  const uintptr_t p = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.add) |
                      reinterpret_cast<uintptr_t>(a.sum) | reinterpret_cast<uintptr_t>(a.out) |
                      reinterpret_cast<uintptr_t>(a.weight);
  const auto fits = [&](unsigned v) {
    return a.D % v == 0 && strides % v == 0 && p % (v * sizeof(E)) == 0 &&
           reinterpret_cast<uintptr_t>(a.codes) % v == 0;
  };
  constexpr int kWide = 16 / sizeof(E);
  if (fits(kWide)) return launch_norm_v<E, kWide>(a, s);
  if constexpr (sizeof(E) == 2) {
    if (fits(2)) return launch_norm_v<E, 2>(a, s);
  }
  return launch_norm_v<E, 1>(a, s);
}

bool bad_align(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

}  // namespace
}  // namespace moeq4

extern "C" moe_status moe_rms_norm(const moe_norm* n, void* stream) {
  using namespace moeq4;
  if (!n || n->T < 0 || n->H < 1 || n->D < 1 || n->dtype < MOE_BF16 || n->dtype > MOE_F32)
    return MOE_ERR_ARG;
  if (!(n->eps > 0.f) || !std::isfinite(n->eps) || !std::isfinite(n->offset)) return MOE_ERR_ARG;
  if (n->D > kMaxD || n->H > 65535 || static_cast<int64_t>(n->T) * n->H > 0x7FFFFFFF)
    return MOE_ERR_SHAPE;
  if (n->T == 0) return MOE_OK;
  if (!n->x || (!n->out && !n->codes) || (n->codes && !n->scales)) return MOE_ERR_ARG;
  if (n->x_row < 0 || n->x_head < 0 || (n->add && (n->add_row < 0 || n->add_head < 0)))
    return MOE_ERR_SHAPE;
  const struct {
    const void* p;
    int64_t row, head;
  } outs[3] = {{n->sum, n->sum_row, n->sum_head},
               {n->out, n->out_row, n->out_head},
               {n->codes, n->codes_row, n->codes_head}};
  for (int i = 0; i < 3; ++i) {
    if (!outs[i].p) continue;
    if (!rows_disjoint(outs[i].row, outs[i].head, n->T, n->H, n->D)) return MOE_ERR_SHAPE;
    for (int j = 0; j < i; ++j)
      if (outs[i].p == outs[j].p) return MOE_ERR_ARG;
    // in place: each thread overwrites the elements that it has read
    const bool as_x = outs[i].row == n->x_row && outs[i].head == n->x_head && i < 2;
    const bool as_add = outs[i].row == n->add_row && outs[i].head == n->add_head && i < 2;
    if ((outs[i].p == n->x && !as_x) || (n->add && outs[i].p == n->add && !as_add))
      return MOE_ERR_ARG;
  }
  const unsigned es = n->dtype == MOE_F32 ? 4 : 2;
  if (bad_align(n->x, es) || bad_align(n->add, es) || bad_align(n->sum, es) ||
      bad_align(n->out, es) || bad_align(n->weight, es) || (n->codes && bad_align(n->scales, 4)))
    return MOE_ERR_ALIGN;
  const moe_status st = check_device();
  if (st != MOE_OK) return st;
  NormArgs a{};
  a.x = n->x;
  a.add = n->add;
  a.weight = n->weight;
  a.sum = n->sum;
  a.out = n->out;
  a.codes = n->codes;
  a.scales = n->scales;
  a.x_row = n->x_row;
  a.x_head = n->x_head;
  a.add_row = n->add_row;
  a.add_head = n->add_head;
  a.sum_row = n->sum_row;
  a.sum_head = n->sum_head;
  a.out_row = n->out_row;
  a.out_head = n->out_head;
  a.c_row = n->codes_row;
  a.c_head = n->codes_head;
  a.rows = n->T * n->H;
  a.H = n->H;
  a.D = n->D;
  a.eps = n->eps;
  a.offset = n->offset;
  a.inv_d = static_cast<float>(1.0 / n->D);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = n->dtype == MOE_F32   ? launch_norm<float>(a, s)
                        : n->dtype == MOE_F16 ? launch_norm<__half>(a, s)
                                              : launch_norm<__nv_bfloat16>(a, s);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
