// attn.cu — attention over the paged, quantised key/value cache, with an
// optional prefix that every request of the batch shares (moe_kv_attention).
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "internal.h"
#include "kv.cuh"
#include "ptx.cuh"

namespace moeq4 {
namespace {

constexpr int kWarps = 4;

struct AttnArgs {
  const uint16_t* q;
  uint16_t* out;
  int64_t q_row, q_head, o_row, o_head;
  const int32_t *table, *lens, *prefix_table;
  int B, nq, Hq, table_stride, max_len, prefix_len, G;
  float scale;
  KvCache c;
};

// A context length as the kernels use it.
__device__ __forceinline__ int context_len(const AttnArgs& a, int b) {
  const int n = a.lens[b];
  if (n >= 0 && n <= a.max_len) return n;
  atomicOr(a.c.err, MOE_DEVERR_BAD_LENGTH);
  return n < 0 ? 0 : a.max_len;
}

// Block = one query row of one head; its warps share the tokens, each with its
// own running maximum and sum, joined through shared memory. Lane l holds
// elements l*E .. l*E+E-1 of the head.
template <int D, int BITS>
__global__ void __launch_bounds__(kWarps * 32) attn_row_kernel(AttnArgs a) {
  constexpr int E = D / 32;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int row = blockIdx.x, hq = blockIdx.y;
  const int b = row / a.nq, i = row % a.nq, hk = hq / a.G;
  const int len = context_len(a, b);
  const int seen = max(0, len - a.nq + 1 + i);
  float q[E], o[E] = {};
  const uint16_t* qp = a.q + row * a.q_row + hq * a.q_head + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e)
    q[e] = __uint_as_float(static_cast<uint32_t>(qp[e]) << 16) * a.scale;
  float m = -INFINITY, l = 0.f;
  for (int part = 0; part < 2; ++part) {
    const int32_t* pages =
        part == 0 ? a.prefix_table : a.table + static_cast<int64_t>(b) * a.table_stride;
    const int n = part == 0 ? a.prefix_len : seen;
    for (int t = warp; t < n; t += kWarps) {
      const int page = pages[t / a.c.page_size], r = t % a.c.page_size;
      if (page < 0 || page >= a.c.pages) {
        if (lane == 0) atomicOr(a.c.err, MOE_DEVERR_BAD_PAGE);
        continue;
      }
      float kv[2][E];
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint8_t* blk = kv_block(a.c, page, hk + w * a.c.Hkv);
        const uint32_t sb = *reinterpret_cast<const uint32_t*>(
            blk + a.c.code_bytes + (r * (D / kKvGroup) + lane * E / kKvGroup) * 4);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int d = lane * E + e;
          const uint32_t byte = blk[static_cast<int64_t>(r) * a.c.row_bytes + d * BITS / 8];
          const uint32_t code = BITS == 8 ? byte : (byte >> (d % 2 * 4)) & 15u;
          kv[w][e] = fmaf(bf16_lo(sb), static_cast<float>(code), bf16_hi(sb));
        }
      }
      float x = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) x = fmaf(q[e], kv[0][e], x);
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, s);
      const float top = fmaxf(m, x);
      const float base = top == -INFINITY ? 0.f : top;
      const float keep = __expf(m - base), p = __expf(x - base);
      m = top;
      l = fmaf(l, keep, p);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(o[e], keep, p * kv[1][e]);
    }
  }
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][D];
  if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
  for (int e = 0; e < E; ++e) so[warp][lane * E + e] = o[e];
  __syncthreads();
  float top = -INFINITY, sum = 0.f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w]);
  if (top == -INFINITY) top = 0.f;
  for (int w = 0; w < kWarps; ++w) sum += sl[w] * __expf(sm[w] - top);
  for (int d = threadIdx.x; d < D; d += kWarps * 32) {
    float y = 0.f;
    for (int w = 0; w < kWarps; ++w) y += so[w][d] * __expf(sm[w] - top);
    a.out[row * a.o_row + hq * a.o_head + d] =
        static_cast<uint16_t>(pack_bf16(sum == 0.f ? 0.f : y / sum, 0.f));
  }
}

template <int D>
cudaError_t launch_rows(const AttnArgs& a, cudaStream_t s) {
  const dim3 grid(a.B * a.nq, a.Hq);
  if (a.c.bits == 8)
    attn_row_kernel<D, 8><<<grid, kWarps * 32, 0, s>>>(a);
  else
    attn_row_kernel<D, 4><<<grid, kWarps * 32, 0, s>>>(a);
  return cudaGetLastError();
}

bool rows_disjoint(int64_t row, int64_t head, int64_t T, int64_t H, int64_t D) {
  const bool head_in = (H == 1 || head >= D) && (T == 1 || row >= (H - 1) * head + D);
  const bool row_in = (T == 1 || row >= D) && (H == 1 || head >= (T - 1) * row + D);
  return head_in || row_in;
}

bool bad16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool bad4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

}  // namespace
}  // namespace moeq4

extern "C" size_t moe_kv_attention_workspace_size(int32_t B, int32_t nq, int32_t Hq, int32_t Hkv,
                                                  int32_t D, int32_t max_len, int32_t prefix_len) {
  (void)B, (void)nq, (void)Hq, (void)Hkv, (void)D, (void)max_len, (void)prefix_len;
  return 256;
}

extern "C" moe_status moe_kv_attention(const moe_kv_attn* a, const moe_kv_cache* c, void* ws,
                                       size_t ws_bytes, void* stream) {
  using namespace moeq4;
  if (!a || a->B < 0 || a->nq < 1 || a->Hq < 1 || a->max_len < 0 || a->prefix_len < 0 ||
      a->table_stride < 0 || !std::isfinite(a->scale))
    return MOE_ERR_ARG;
  moe_status st = check_kv_cache(c);
  if (st != MOE_OK) return st;
  if (a->Hq % c->Hkv || a->Hq > 65535 || static_cast<int64_t>(a->B) * a->nq > (1 << 24))
    return MOE_ERR_SHAPE;
  if (a->B == 0) return MOE_OK;
  const int64_t pages = (static_cast<int64_t>(a->max_len) + c->page_size - 1) / c->page_size;
  if (!a->q || !a->out || !a->lens || (a->max_len > 0 && !a->table) ||
      (a->prefix_len > 0 && !a->prefix_table) || !ws)
    return MOE_ERR_ARG;
  if (a->table_stride < pages || a->q_row < 0 || a->q_head < 0 || a->out_row < 0 ||
      a->out_head < 0 ||
      !rows_disjoint(a->out_row, a->out_head, static_cast<int64_t>(a->B) * a->nq, a->Hq, c->D))
    return MOE_ERR_SHAPE;
  if (bad16(a->q) || bad16(a->out) || bad16(ws) || bad4(a->lens) || bad4(a->table) ||
      bad4(a->prefix_table) || a->q_row % 8 || a->q_head % 8 || a->out_row % 8 || a->out_head % 8)
    return MOE_ERR_ALIGN;
  if (ws_bytes < moe_kv_attention_workspace_size(a->B, a->nq, a->Hq, c->Hkv, c->D, a->max_len,
                                                 a->prefix_len))
    return MOE_ERR_WORKSPACE;
  AttnArgs k{};
  k.q = a->q;
  k.out = a->out;
  k.q_row = a->q_row;
  k.q_head = a->q_head;
  k.o_row = a->out_row;
  k.o_head = a->out_head;
  k.table = a->table;
  k.lens = a->lens;
  k.prefix_table = a->prefix_table;
  k.B = a->B;
  k.nq = a->nq;
  k.Hq = a->Hq;
  k.table_stride = a->table_stride;
  k.max_len = a->max_len;
  k.prefix_len = a->prefix_len;
  k.G = a->Hq / c->Hkv;
  k.scale = a->scale;
  k.c = kv_cache_args(*c);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = c->D == 64    ? launch_rows<64>(k, s)
                        : c->D == 128 ? launch_rows<128>(k, s)
                                      : launch_rows<256>(k, s);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
