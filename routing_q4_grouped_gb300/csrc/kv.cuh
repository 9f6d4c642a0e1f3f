// kv.cuh — layout of the paged key/value cache (moe_kv_cache in moeq4.h) and the
// rotary angle, shared by the kernels that write, read and attend over it.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>

#include "../../include/moeq4.h"

namespace moeq4 {

constexpr int kKvGroup = 64;         // elements that share a scale and a bias

// One cache as the kernels see it; all offsets are 64-bit.
struct KvCache {
  uint8_t* data;
  int32_t* err;
  int pages, page_size, Hkv, D, bits;
  int row_bytes;                     // codes of one token of one head
  int code_bytes;                    // codes of one head of a page (words follow)
  int head_bytes;                    // one head of a page
  int64_t page_bytes;
  uint32_t page_blocks;              // 16-token blocks per page
  uint64_t page_magic;               // floor(2^37 / page_blocks) + 1
};

moe_status check_kv_cache(const moe_kv_cache* c);
KvCache kv_cache_args(const moe_kv_cache& c);

// Page of 16-token block blk < 2^27: blk / page_blocks by multiplication. The magic number is
// at most 2^37 + 1, so the product stays below 2^64, and its excess over 2^37 / page_blocks is
// at most 1, so the quotient is too large by at most blk * 2^-37 < 2^-10, less than the
// 1 / page_blocks >= 2^-8 that the next whole page needs.
__host__ __device__ inline int page_of_block(const KvCache& c, uint32_t blk) {
  return static_cast<int>((blk * c.page_magic) >> 37);
}

// The block of head h (key heads 0 .. Hkv-1, then value heads) of a page.
__device__ __forceinline__ uint8_t* kv_block(const KvCache& c, int page, int h) {
  return c.data + page * c.page_bytes + static_cast<int64_t>(h) * c.head_bytes;
}

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// cos and sin of pos * phase (a 64-bit fraction of a turn; the product wraps at
// whole turns). The top 32 bits of the wrapped product, as a signed half turn,
// give the angle in [-pi, pi) to 2^-24 of its size plus 2^-31 turns; in that range sinf and cosf need no
// long reduction.
__device__ __forceinline__ void rope_sincos(int32_t pos, uint64_t phase, float& c, float& s) {
  const uint64_t w = static_cast<uint64_t>(static_cast<int64_t>(pos)) * phase;
  const float a = __fmul_rn(static_cast<float>(static_cast<int32_t>(w >> 32)),
                            3.14159265358979323846f / 2147483648.0f);
  sincosf(a, &s, &c);
}

// (a, b) turned; products and sums rounded one by one so that every path that
// turns an element gives the same bits.
__device__ __forceinline__ float rope_first(float a, float b, float c, float s) {
  return __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
}
__device__ __forceinline__ float rope_second(float a, float b, float c, float s) {
  return __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}

}  // namespace moeq4
