// attn.cuh — arguments and helpers shared by the attention kernels.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "kv.cuh"
#include "ptx.cuh"

namespace moeq4 {

// A call's contexts: the prefix (all query rows of the batch see it whole) and the
// requests' own tokens. Each is worked on by the split kernel (few query rows per unit)
// or by the row kernel (128 or 256 query rows per unit). Both line up the token
// tiles of all their units and give every block an equal share of them.
struct AttnArgs {
  const uint16_t* q;
  uint16_t* out;
  int64_t q_row, q_head, o_row, o_head;
  const int32_t *table, *lens, *prefix_table;
  int B, nq, Hq, table_stride, max_len, prefix_len, G;
  float scale2;              // scale * log2(e)
  KvCache c;
  int skip_pages[2], skip_blocks[2];     // four blocks further, and eight
  // split kernel: units of 8 nt query rows
  int nt;
  int pre_blocks, pre_tiles;             // units of the prefix, and per key/value head (0: not here)
  int own_tiles;                         // units per request and key/value head (0: not here)
  int32_t* share_out;                    // tiles per block, found on the device
  int32_t* first;                        // [B] tiles per unit of the requests before b
  // row kernel: units of unit_rows query rows, tiles of row_tile tokens, by the largest length
  int unit_rows, row_tile;
  int pre_units, own_units;              // (0: not here)
  int pre_row_tiles, own_row_tiles;      // units per key/value head (and request)
  int own_T, share;                      // tiles per unit and per block
  int pre_T;                             // tiles of the prefix, either kernel
  // partial results, D values and (m, l) each: the prefix's at [part][row][head], the own
  // tokens' from own_whole on, the split kernel's slots [block][2][8 nt] from slots on
  int lone;                              // one context only: a unit in one piece gives the output
  int64_t own_whole, slots;
  float* part;
  float2* ml;
  uint64_t timeout_ns;
};

// A context length as the kernels use it.
__device__ __forceinline__ int context_len(const AttnArgs& a, int b, bool report) {
  const int n = a.lens[b];
  if (n >= 0 && n <= a.max_len) return n;
  if (report) atomicOr(a.c.err, MOE_DEVERR_BAD_LENGTH);
  return n < 0 ? 0 : a.max_len;
}

// Own tokens that row r (query token r / G) of a request with n tokens sees.
__device__ __forceinline__ int own_limit(const AttnArgs& a, int n, int r) {
  return max(0, n - a.nq + 1 + r / a.G);
}

// Place of row tile rt in the order of a request's units: first, last, second,
// last but one, ... so that a block's consecutive units see much and little in turn.
__host__ __device__ inline int unit_place(int rt, int tiles) {
  return rt < (tiles + 1) / 2 ? 2 * rt : 2 * (tiles - 1 - rt) + 1;
}
__host__ __device__ inline int unit_tile(int place, int tiles) {
  return place & 1 ? tiles - 1 - (place >> 1) : place >> 1;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t min_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// Row kernel (tcgen05): launches it over a.pre_units / a.own_units.
cudaError_t launch_attn_rows(const AttnArgs& a, unsigned blocks, cudaStream_t s);
int attn_unit_rows(int D);             // query rows of a unit
int attn_row_tile(int D);              // tokens of a tile

}  // namespace moeq4
