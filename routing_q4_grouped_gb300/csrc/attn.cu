// attn.cu — attention over the paged, quantised key/value cache, with an
// optional prefix that every request of the batch shares (moe_kv_attention).
//
// Contexts are cut into splits; a block takes one split for a tile of query rows
// that share a key/value head (the heads of a group, a request's query tokens
// and, for the prefix, all requests of the batch), and writes a partial result:
// the largest logit m, the sum l of exp2(x - m) and the weighted sum of values.
// A second kernel joins the splits of a row.
//
// Few rows read many codes, so the work is bound by memory bandwidth as long as
// turning codes into tensor-core operands costs less than the bytes. Two choices
// keep it cheap:
//  * Codes go into the products as integers. Keys: a code c alone in the low bits of an
//    fp16 is the subnormal number c 2^-24, which the tensor cores take at full rate, so
//    one byte permutation or mask makes an operand pair. With value = s c + b,
//      q . k = sum over groups of  s sum c q + b sum q.
//    Values: c under the byte 0x64 is 1024 + c, and one subtraction centres it, c - z with
//    z = 128 or 8. (Uncentred, the sum of w c and the sum of w b / s nearly cancel over a
//    long context, and the tensor cores' truncating sums show: at 131071 tokens the
//    output's error against 64 bits was 0.0019 instead of 0.0017.) The values' scale is
//    taken into the weights, rounded to fp16 once, w = fp16(p s / u), and used for codes and
//    biases alike, so that the rounding stays relative to the value:
//      sum_t p_t v_t = u (sum_t w_t (c_t - z) + sum_t w_t (b_t / s_t + z)).
//    u is a power of two near the scales, one per group of the head, since a group has
//    its own sums: a small group beside a large one keeps its bits. It moves with the
//    scales (the sums are fp32 and move along). A step in which one group's scales differ
//    by more than 2^12, or that holds a scale that is 0, subnormal or not finite, takes
//    the same sums with w as two bf16 (16 bits and fp32's range) and biases in fp32, so
//    large values of little weight cost the others nothing.
//  * Tokens are the rows (M) of the products and queries the columns (N = 8), so
//    that 8 rows fill the tensor core: X^T = K Q^T, then O^T = V^T P^T. The
//    products' own register layouts let a thread read 16 (keys) or 8 (values)
//    neighbouring codes of a token at once; P is transposed between the two
//    products by one 8x8 register transpose per 8 tokens and group.
// q' and w are fp16: q' is the query scaled by a power of two so that its row's largest
// element is near 2^12; p <= 2^8 and s / u < 2^7, so neither leaves fp16's range (one
// rounding of 2^-11 for weights above 2^-14 units, less for smaller ones; bf16 queries
// are exact above 2^-26 of their row's largest element). Logits, maxima, sums and outputs
// are fp32.
//
// Measured (D = 128, 32 query heads on 8 key/value heads, join included): one request of
// 131071 tokens, 8 bits, 55 us, 5.2 TB/s, 76 % of the copy's bandwidth; 64 requests of
// mixed lengths, 4 bits, 95 us, 3.2 TB/s. There a byte holds twice the codes and the
// issue slots bind (54 % of them used over the whole kernel, 42 % at 8 bits, tensor
// cores at 16 to 19 %), not the memory.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/moeq4_debug.h"
#include "attn.cuh"
#include "internal.h"

namespace moeq4 {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr uint32_t kAll = 0xFFFFFFFFu;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// D += A B: A 16x16 fp16 (row), B 16x8 fp16 (col), D 16x8 fp32.
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same with bf16 operands.
__device__ __forceinline__ void mma16816_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two small whole numbers, exact in both types.
__device__ __forceinline__ uint32_t f16x2_to_bf16x2(uint32_t v) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v));
  return pack_bf16(f.x, f.y);
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}

__device__ __forceinline__ float max_over_rows8(float v) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
__device__ __forceinline__ float sum_over_rows8(float v) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// Geometry of the split kernel for head size D and code width BITS.
template <int D, int BITS>
struct Geo {
  static constexpr int J = D / kKvGroup;          // groups of a head
  static constexpr int RB = D * BITS / 8;         // code bytes of a token
  static constexpr int TB = D * BITS > 1024 ? 1 : 2;   // 16-token blocks per step
  static constexpr int kCodes = 16 * RB;          // one block's codes (keys or values)
  static constexpr int kWords = 16 * J * 4;
  static constexpr int kBlock = 2 * (kCodes + kWords);   // K codes, V codes, K words, V words
  static constexpr int kStage = TB * kBlock;
  static constexpr int kStages = TB == 1 ? 3 : 2;
  static constexpr int kWarpBytes = kStages * kStage;
  static constexpr int kRing = kWarps * kWarpBytes;
  // Shared memory is laid out in rows of RB bytes (a token) whose 32-byte units are
  // exchanged by the token's low bits, so that the lanes of one shared-memory access,
  // which read the same unit of several tokens, meet no bank twice (twice at most for
  // rows of one or two units). Keys are read for 4 or 2 neighbouring tokens at once,
  // values for tokens 0 2 4 6.
  static constexpr int kUnits = RB / 32;
  __device__ static int key_unit(int row) {
    return kUnits < 2 ? 0 : BITS == 8 ? (kUnits >= 4 ? (row & 1) << 1 : 0)
                                      : (kUnits >= 4 ? row & 3 : (row >> 1) & 1);
  }
  __device__ static int value_unit(int row) {
    return kUnits >= 4 ? (row >> 1) & 3 : kUnits == 2 ? (row >> 1) & 1 : 0;
  }
  // A lane's byte offset for its reads of group 0 (group j: key_at / value_at).
  __device__ static uint32_t key_lane(int g, int t) {
    return BITS == 8 ? g * RB + ((t >> 1) ^ key_unit(g)) * 32 + (t & 1) * 16
                     : g * RB + key_unit(g) * 32 + t * 8;
  }
  __device__ static uint32_t value_lane(int g, int t) {
    return BITS == 8 ? 2 * t * RB + ((g >> 2) ^ value_unit(2 * t)) * 32 + (g & 3) * 8
                     : 2 * t * RB + value_unit(2 * t) * 32 + g * 4;
  }
  __device__ static constexpr uint32_t group_bits(int j) { return j * (BITS == 8 ? 64u : 32u); }
  // A lane's destination of 16-byte chunk `lane` of a block; chunk 32 c + lane goes to
  // (it ^ copy_bits(c)) + 512 c: a copy instruction covers whole rows.
  static constexpr int kChunks = RB / 16;            // per row
  __device__ static uint32_t copy_lane(int lane, bool value) {
    const int row = lane / kChunks, at = lane % kChunks;
    return row * RB + ((at >> 1) ^ (value ? value_unit(row) : key_unit(row))) * 32 + (at & 1) * 16;
  }
  __device__ static constexpr uint32_t copy_bits(int c, bool value) {
    return !value ? 0u : RB == 128 ? (c & 1) * 64u : RB == 256 ? (c & 3) * 32u : 0u;
  }
};

// Blocks of the split kernel that share a multiprocessor, by registers and shared memory.
constexpr int split_blocks_per_sm(int D, int BITS, int NT) {
  return D == 256 ? 2 : D == 128 ? (NT == 2 ? 2 : BITS == 8 ? 3 : 4) : (NT == 2 ? 3 : 5);
}

template <int D, int BITS, int NT>
struct SplitSmem {
  static constexpr size_t kMerge = size_t(kWarps) * 8 * NT * (D + 4) * 4;   // rows padded by 4
  static constexpr size_t kBytes =
      (Geo<D, BITS>::kRing > kMerge ? size_t(Geo<D, BITS>::kRing) : kMerge) + kWarps * 8 * NT * 8;
};

// One step's operands and state of a warp.
template <int D, int BITS, int NT>
struct Warp {
  using G = Geo<D, BITS>;
  uint32_t q[NT][G::J][8];        // queries: B operand of X^T = K Q^T
  float qsum[NT][G::J][2];        // 2^-24 * sum of q' by group
  float row_scale[NT][2];         // scale2 * 2^(24 + row exponent)
  int lim[NT][2];                 // tokens seen by the row
  float m[NT][2], l[NT][2];
  float o[NT][G::J][4][4];        // O^T: group, tile of 16 elements
  float ob[NT][G::J][2];          // sum of w * (bias / scale + z)
  float top_x[NT][2];             // m + 8: the bound of a logit
  // o and ob of group j are in units of a power of two near the values' scales. Its bounds
  // as packed words (as of a value word: scale in the low half, bias in the high half, their
  // exponents alone), and the largest exponent so far. The same in all lanes.
  uint32_t low[G::J], high[G::J], seen[G::J];

  static constexpr uint32_t kWindow = 6;          // scales within 2^-6 .. 2^6 of the unit,
  static constexpr uint32_t kBias = 24;           // biases below 2^24 units (bf16 groups have 2^23)
  __device__ __forceinline__ void set_unit(int j, uint32_t field) {
    low[j] = (field - kWindow) << 7;
    high[j] = (field + kWindow) << 7 | min(field + kBias, 254u) << 23;
    seen[j] = max(seen[j], field + kBias);
  }
  __device__ __forceinline__ uint32_t unit_field(int j) const { return (low[j] >> 7) + kWindow; }
  __device__ __forceinline__ float unit(int j) const {
    return __uint_as_float((low[j] << 16) + (kWindow << 23));
  }
  __device__ __forceinline__ float per_unit(int j) const {
    return __uint_as_float(((254u - kWindow) << 23) - (low[j] << 16));
  }

  // Whether a value word of a token is not what the plain step takes: a normal scale and a
  // bias in the window of its group's unit.
  template <bool MASK>
  __device__ __forceinline__ bool outside(const uint32_t (&vw)[G::TB][2][G::J], int tok0,
                                          const int (&top)[G::TB], int g) const {
    bool odd = false;
#pragma unroll
    for (int j = 0; j < G::J; ++j) {
      uint32_t lo = low[j], hi = high[j];
#pragma unroll
      for (int b = 0; b < G::TB; ++b)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if (MASK && tok0 + 16 * b + 8 * r + g >= top[b]) continue;
          const uint32_t e = vw[b][r][j] & 0x7F807F80u;
          lo = min_u16x2(lo, e);
          hi = max_u16x2(hi, e);
        }
      odd |= lo != low[j] || hi != high[j];
    }
    return odd;
  }

  // Moves the units of the groups whose scales left the window, and what has been summed up
  // along with them. True if no units suit this step: a group's scales span more than the
  // window, or are 0, subnormal or not finite, or a bias is far above them.
  __device__ __forceinline__ bool refer(const uint32_t (&vw)[G::TB][2][G::J], int tok0,
                                        const int (&top)[G::TB], int g) {
    bool wide = false;
#pragma unroll
    for (int j = 0; j < G::J; ++j) {
      uint32_t hi = 0, lo = 255, bias = 0;
      bool odd = false;
#pragma unroll
      for (int b = 0; b < G::TB; ++b)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if (tok0 + 16 * b + 8 * r + g >= top[b]) continue;
          uint32_t s = vw[b][r][j] >> 7 & 255u, z = vw[b][r][j] >> 23 & 255u;
          odd |= s == 0 || s == 255u || z == 255u;
          if (vw[b][r][j] & 0x7Fu) s = max(s, 1u);            // (subnormal: below 2^-126)
          if (s < 255u) hi = max(hi, s);
          if (s > 0) lo = min(lo, s);
          if (z < 255u) bias = max(bias, z);
        }
      hi = __reduce_max_sync(kAll, hi);
      lo = __reduce_min_sync(kAll, lo);
      bias = __reduce_max_sync(kAll, bias);
      // what is summed up stays finite with a unit at most 2^60 below all it was made of
      seen[j] = max(seen[j], max(hi, bias));
      const uint32_t old = unit_field(j);
      uint32_t to = old;
      if (hi > 0 && (hi > to + kWindow || lo + kWindow < to)) to = min(hi, lo + kWindow);
      to = min(max(max(to, seen[j] > 61u ? seen[j] - 60u : 1u), 7u), 247u);
      odd |= lo + kWindow < to || hi > to + kWindow || bias > to + kBias;
      wide |= __any_sync(kAll, odd);
      if (to == old) continue;
      const int by = min(max(static_cast<int>(old) - static_cast<int>(to), -126), 127);
      const float f = __uint_as_float(static_cast<uint32_t>(127 + by) << 23);
      set_unit(j, to);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int c = 0; c < 2; ++c) ob[n][j][c] *= f;
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[n][j][u][i] *= f;
      }
    }
    return wide;
  }

  __device__ __forceinline__ static void load_words(const uint8_t* p, uint32_t (&w)[G::J]) {
    if constexpr (G::J == 1) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (G::J == 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x, w[1] = v.y;
    } else {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    }
  }

  // The value words of tokens g and g + 8 of each block.
  __device__ __forceinline__ static void load_value_words(const uint8_t* st, int g,
                                                          uint32_t (&vw)[G::TB][2][G::J]) {
#pragma unroll
    for (int b = 0; b < G::TB; ++b)
#pragma unroll
      for (int r = 0; r < 2; ++r)
        load_words(st + b * G::kBlock + 2 * G::kCodes + G::kWords + (8 * r + g) * (G::J * 4), vw[b][r]);
  }

  // Columns 2t, 2t+1 of this thread (queries); rows lane/4 and lane/4 + 8 (tokens).
  // `fresh`: the piece's first step of this warp.
  template <bool MASK>
  __device__ __forceinline__ void step(const uint8_t* st, int tok0, const int (&top)[G::TB], int g,
                                       uint32_t key_off, uint32_t value_off, bool fresh) {
    float x[G::TB][NT][4];
    uint32_t vw[G::TB][2][G::J];
    load_value_words(st, g, vw);
#pragma unroll
    for (int b = 0; b < G::TB; ++b) {
      const uint8_t* kc = st + b * G::kBlock;
      const uint8_t* words = kc + 2 * G::kCodes + g * (G::J * 4);
      uint32_t kw[2][G::J];
#pragma unroll
      for (int r = 0; r < 2; ++r) load_words(words + r * (8 * G::J * 4), kw[r]);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[b][n][i] = 0.f;
#pragma unroll
      for (int j = 0; j < G::J; ++j) {
        // 16 codes of tokens g and g + 8: elements 64 j + 16 t ..
        uint32_t w[2][4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint8_t* kp = kc + (key_off ^ G::group_bits(j)) + r * 8 * G::RB;
          if (BITS == 8) {
            const uint4 v = *reinterpret_cast<const uint4*>(kp);
            w[r][0] = v.x, w[r][1] = v.y, w[r][2] = v.z, w[r][3] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(kp);
            w[r][0] = v.x, w[r][1] = v.x >> 8, w[r][2] = v.y, w[r][3] = v.y >> 8;
          }
        }
        float acc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          uint32_t a[4];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            if (BITS == 8) {
              a[r] = prmt(w[r][s], 0u, 0x4140);
              a[2 + r] = prmt(w[r][s], 0u, 0x4342);
            } else {
              a[r] = w[r][s] & 0x000F000Fu;
              a[2 + r] = w[r][s] & 0x00F000F0u;        // 16 c
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816(acc[n], a, q[n][j][2 * s], q[n][j][2 * s + 1]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t sb = kw[i >> 1][j];
            x[b][n][i] = fmaf(bf16_lo(sb), acc[n][i],
                              fmaf(bf16_hi(sb), qsum[n][j][i & 1], x[b][n][i]));
          }
      }
    }
    // A row's reference m is any value near its largest logit, so that weights may
    // pass 1 by 2^8; it moves only when a logit leaves that bound.
    bool grow = false;
#pragma unroll
    for (int b = 0; b < G::TB; ++b) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int tok = tok0 + 16 * b + 8 * r + g;
        const bool any = !MASK || tok < top[b];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float& v = x[b][n][2 * r + c];
            v *= row_scale[n][c];
            if (MASK && !(any && tok < lim[n][c])) v = -INFINITY;
            grow |= v > top_x[n][c];
          }
      }
    }
    if (fresh) {
      // units from one token's scales, so that the search is seldom needed
#pragma unroll
      for (int j = 0; j < G::J; ++j) {
        const uint32_t s = __shfl_sync(kAll, vw[0][0][j], 0) >> 7 & 255u;
        if (tok0 < top[0] && s > 0 && s < 255u) set_unit(j, min(max(s, 7u), 247u));
      }
    }
    bool wide = false;
    const bool odd = outside<MASK>(vw, tok0, top, g);
    if (__any_sync(kAll, grow || odd)) {
      if (__any_sync(kAll, odd)) wide = refer(vw, tok0, top, g);
      rescale(x);
    }
    // weights
#pragma unroll
    for (int b = 0; b < G::TB; ++b)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float ref = m[n][i & 1] == -INFINITY ? 0.f : m[n][i & 1];
          const float p = exp2_approx(x[b][n][i] - ref);
          x[b][n][i] = p;
          l[n][i & 1] += p;
        }
    if (wide) {
      values<true>(st, vw, x, value_off);
      return;
    }
    if (MASK) {                                  // a scale of one unit for what is not there
#pragma unroll
      for (int b = 0; b < G::TB; ++b)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int j = 0; j < G::J; ++j)
            if (tok0 + 16 * b + 8 * r + g >= top[b]) vw[b][r][j] = unit_field(j) << 7;
    }
    values<false>(st, vw, x, value_off);
  }

  // O^T += V^T P^T
  template <bool WIDE>
  __device__ __forceinline__ void values(const uint8_t* st, const uint32_t (&vw)[G::TB][2][G::J],
                                         const float (&x)[G::TB][NT][4], uint32_t value_off) {
#pragma unroll
    for (int b = 0; b < G::TB; ++b) {
      const uint8_t* vc = st + b * G::kBlock + G::kCodes;
#pragma unroll
      for (int j = 0; j < G::J; ++j) {
        uint32_t pb[NT][2], pl[NT][2];
        const float inverse = per_unit(j);
        constexpr float kZ = BITS == 8 ? 128.f : 8.f;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float s = bf16_lo(vw[b][r][j]), bias = bf16_hi(vw[b][r][j]);
          const float su = s * inverse;
          if (!WIDE) {
            // bias / s with one correction step: exact where the quotient is a float
            float inv;
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
            float ratio = bias * inv;
            ratio = fmaf(fmaf(-ratio, s, bias), inv, ratio) + kZ;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const uint32_t w2 = pack_f16(x[b][n][2 * r] * su, x[b][n][2 * r + 1] * su);
              pb[n][r] = transpose8x8(w2);
              const float2 wf = __half22float2(*reinterpret_cast<const __half2*>(&w2));
              ob[n][j][0] = fmaf(wf.x, ratio, ob[n][j][0]);
              ob[n][j][1] = fmaf(wf.y, ratio, ob[n][j][1]);
            }
          } else {
            // any scale: weights as two bf16 each (16 bits, fp32's range), the rest in fp32;
            // nothing of a token reaches a row that gives it no weight
            const float rest = fmaf(s, kZ, bias) * inverse;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              float w[2], low[2];
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const float p = x[b][n][2 * r + c];
                const bool none = p == 0.f;
                w[c] = none ? 0.f : p * su;
                low[c] = w[c] - __bfloat162float(__float2bfloat16_rn(w[c]));
                if (!none) ob[n][j][c] = fmaf(p, rest, ob[n][j][c]);
              }
              pb[n][r] = transpose8x8(pack_bf16(w[0], w[1]));
              pl[n][r] = transpose8x8(pack_bf16(low[0], low[1]));
            }
          }
        }
        // 8 codes of tokens 2t, 2t+1, 2t+8, 2t+9: elements 64 j + 8 g ..
        uint32_t w[4][2];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint8_t* vp =
              vc + (value_off ^ G::group_bits(j)) + ((k & 1) + 8 * (k >> 1)) * G::RB;
          if (BITS == 8) {
            const uint2 v = *reinterpret_cast<const uint2*>(vp);
            w[k][0] = v.x, w[k][1] = v.y;
          } else {
            w[k][0] = *reinterpret_cast<const uint32_t*>(vp);
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {        // tiles 2h, 2h + 1: elements 4h .. 4h + 3 of the 8
          uint32_t a[2][4];
#pragma unroll
          for (int k = 0; k < 2; ++k) {      // token pairs (2t, 2t+1) and (2t+8, 2t+9)
            if (BITS == 8) {
              const uint32_t lo = prmt(w[2 * k][h], w[2 * k + 1][h], 0x5140);
              const uint32_t hi = prmt(w[2 * k][h], w[2 * k + 1][h], 0x7362);
              constexpr uint32_t kC = 0x64806480u;               // 1024 + 128
              a[0][2 * k] = sub_f16x2(prmt(lo, 0x64646464u, 0x4140), kC);
              a[0][2 * k + 1] = sub_f16x2(prmt(lo, 0x64646464u, 0x4342), kC);
              a[1][2 * k] = sub_f16x2(prmt(hi, 0x64646464u, 0x4140), kC);
              a[1][2 * k + 1] = sub_f16x2(prmt(hi, 0x64646464u, 0x4342), kC);
            } else {
              // odd elements stay multiplied by 16 until the end
              const uint32_t v = prmt(w[2 * k][0], w[2 * k + 1][0], h ? 0x7632 : 0x5410);
              constexpr uint32_t k1024 = 0x64006400u, kC = 0x64086408u, kC16 = 0x64806480u;
              a[0][2 * k] = sub_f16x2(lop3_and_or(v, 0x000F000Fu, k1024), kC);
              a[0][2 * k + 1] = sub_f16x2(lop3_and_or(v, 0x00F000F0u, k1024), kC16);
              a[1][2 * k] = sub_f16x2(lop3_and_or(v >> 8, 0x000F000Fu, k1024), kC);
              a[1][2 * k + 1] = sub_f16x2(lop3_and_or(v >> 8, 0x00F000F0u, k1024), kC16);
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (!WIDE) {
              mma16816(o[n][j][2 * h], a[0], pb[n][0], pb[n][1]);
              mma16816(o[n][j][2 * h + 1], a[1], pb[n][0], pb[n][1]);
            } else {
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                uint32_t c[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) c[i] = f16x2_to_bf16x2(a[k][i]);
                mma16816_bf16(o[n][j][2 * h + k], c, pb[n][0], pb[n][1]);
                mma16816_bf16(o[n][j][2 * h + k], c, pl[n][0], pl[n][1]);
              }
            }
          }
        }
      }
    }
  }

  // Moves the rows' m to their largest logit, and what has been summed up along with it.
  __device__ __forceinline__ void rescale(const float (&x)[G::TB][NT][4]) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float keep[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float mx = -INFINITY;
#pragma unroll
        for (int b = 0; b < G::TB; ++b)
#pragma unroll
          for (int r = 0; r < 2; ++r) mx = fmaxf(mx, x[b][n][2 * r + c]);
        mx = max_over_rows8(mx);
        keep[c] = 1.f;
        if (!(mx > m[n][c])) continue;
        keep[c] = exp2_approx(m[n][c] - mx);    // (0 from -inf on, where nothing is summed up)
        m[n][c] = mx;
        top_x[n][c] = mx + 8.f;
        l[n][c] *= keep[c];
      }
#pragma unroll
      for (int j = 0; j < G::J; ++j) {
        ob[n][j][0] *= keep[0];
        ob[n][j][1] *= keep[1];
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[n][j][u][i] *= keep[i & 1];
      }
    }
  }
};

constexpr int kSplitTile = kWarps * 32;          // tokens; shares are counted in these tiles

// Where a block's share of the split kernel's tiles begins. The tiles of all units
// are lined up (the prefix's units first, then request by request) and cut into
// equal shares, whatever the requests' lengths.
struct Share {
  int g, end;                                // tiles [g, end) of all
  int share;                                 // tiles per block
  int first;                                 // tiles per unit of the requests before b
  int b;
};

__device__ __forceinline__ int split_tiles(int tokens) {
  return (tokens + kSplitTile - 1) / kSplitTile;
}

// Sums up the requests' tiles (each thread a run of requests) and finds the request
// at which this block's share begins. Block 0 keeps the sums for the join.
__device__ __forceinline__ Share find_share(const AttnArgs& a) {
  __shared__ int sums[kWarps];
  __shared__ int found_first;
  __shared__ int found_b;
  const int pre_total = a.pre_blocks * a.pre_T;
  const int per = (a.B + kThreads - 1) / kThreads;
  const int lo = min(a.B, static_cast<int>(threadIdx.x) * per), hi = min(a.B, lo + per);
  int mine = 0;
  if (a.own_tiles)
    for (int r = lo; r < hi; ++r) mine += split_tiles(context_len(a, r, blockIdx.x == 0));
  int upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(kAll, upto, o);
    if ((threadIdx.x & 31) >= o) upto += x;
  }
  if ((threadIdx.x & 31) == 31) sums[threadIdx.x / 32] = upto;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < threadIdx.x / 32) upto += sums[w];
    total += sums[w];
  }
  const int units = a.c.Hkv * a.own_tiles;   // per request
  Share s;
  s.share = max(1, static_cast<int>((pre_total + total * units + gridDim.x - 1) / gridDim.x));
  s.g = blockIdx.x * s.share;
  s.end = min(s.g + s.share, pre_total + total * units);
  int first = upto - mine;
  const int want = max(0, s.g - pre_total);
  if (blockIdx.x == 0 || (want >= first * units && want < upto * units)) {
    for (int r = lo; r < hi; ++r) {
      const int n = split_tiles(context_len(a, r, false));
      if (blockIdx.x == 0) a.first[r] = first;
      if (want >= first * units && want < (first + n) * units) {
        found_first = first;
        found_b = r;
      }
      first += n;
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.share_out = s.share;
  __syncthreads();
  s.first = found_first;                         // (read only if the share has own tiles)
  s.b = found_b;
  return s;
}

// One block takes its share piece by piece: a run of tiles of one unit, i.e. of one
// context (a request's own tokens, or the prefix) for a tile of 8 NT query rows of one
// key/value head. Its warps take every fourth step of 16 TB tokens, each through a ring
// of asynchronous copies of its own (no block barrier until the join of the warps). A
// unit in one piece gives the output itself, or the row's one partial result of that
// context; the pieces of a cut unit go to the block's two slots.
template <int D, int BITS, int NT>
__global__ void __launch_bounds__(kThreads, split_blocks_per_sm(D, BITS, NT))
    attn_split_kernel(const AttnArgs a) {
  using G = Geo<D, BITS>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = __shfl_sync(kAll, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  const int g = lane >> 2, t = lane & 3;
  // After the row kernel this one depends on nothing that kernel writes, only on what it
  // waited for itself before it let this one start; it takes over multiprocessors as
  // they come free and waits at its end, for the join.
  if (!a.pre_units) griddep_wait();
  griddep_launch_dependents();
  Share sh = find_share(a);
  const int first_g = sh.g;
  const int pre_total = a.pre_blocks * a.pre_T;
  const int units = a.c.Hkv * a.own_tiles;
  while (sh.g < sh.end) {
  // ---- which work
  const bool pre = sh.g < pre_total;
  int b = 0, tile, hk, n_rows, ctx, T;
  int unit_g;
  const int32_t* pages;
  if (pre) {
    const int u = sh.g / a.pre_T;
    T = a.pre_T;
    unit_g = u * T;
    tile = u % a.pre_tiles;
    hk = u / a.pre_tiles;
    n_rows = a.B * a.nq * a.G;
    ctx = a.prefix_len;
    pages = a.prefix_table;
  } else {
    const int at = sh.g - pre_total;
    ctx = context_len(a, sh.b, false);
    T = split_tiles(ctx);
    while (at >= (sh.first + T) * units) {       // the next request with any tokens
      sh.first += T;
      ctx = context_len(a, ++sh.b, false);
      T = split_tiles(ctx);
    }
    b = sh.b;
    const int u = (at - sh.first * units) / T;
    unit_g = pre_total + sh.first * units + u * T;
    tile = u % a.own_tiles;
    hk = u / a.own_tiles;
    n_rows = a.nq * a.G;
    pages = a.table + static_cast<int64_t>(b) * a.table_stride;
  }
  const int stop = min(sh.end, unit_g + T);
  const bool whole = sh.g == unit_g && stop == unit_g + T;
  const int slot = 2 * blockIdx.x + (sh.g != first_g);
  const int row0 = tile * 8 * NT;
  // the tile's last row sees most
  const auto limit = [&](int r) {
    return pre ? ctx : own_limit(a, ctx, r);
  };
  const int t0 = (sh.g - unit_g) * kSplitTile;
  const int t1 = min(min((stop - unit_g) * kSplitTile, ctx),
                     limit(min(row0 + 8 * NT, n_rows) - 1));
  sh.g = stop;

  // ---- tokens: the first copies are on their way while the queries are prepared
  uint8_t* ring = smem + warp * G::kWarpBytes;
  constexpr int kStep = 16 * G::TB;
  const int steps = t1 > t0 ? (t1 - t0 + kStep - 1) / kStep : 0;
  const uint8_t* lane_src = a.c.data + static_cast<int64_t>(hk) * a.c.head_bytes + lane * 16;
  const int64_t to_values = static_cast<int64_t>(a.c.Hkv) * a.c.head_bytes;
  const uint32_t copy_k = smem_u32(ring) + G::copy_lane(lane, false);
  const uint32_t copy_v = smem_u32(ring) + G::kCodes + G::copy_lane(lane, true);
  const uint32_t copy_w = smem_u32(ring) + 2 * G::kCodes + lane * 16;
  // page and 16-token block within it of the step after the one last requested; a
  // warp's next step is kWarps TB blocks further
  int page[G::TB], in_page[G::TB], at_page[G::TB], tok_next = t0 + warp * kStep;
#pragma unroll
  for (int i = 0; i < G::TB; ++i) {
    const uint32_t blk = static_cast<uint32_t>(tok_next >> 4) + i;
    at_page[i] = page_of_block(a.c, blk);
    in_page[i] = static_cast<int>(blk - at_page[i] * a.c.page_blocks);
    page[i] = tok_next + 16 * i < t1 ? __ldg(pages + at_page[i]) : -1;
  }
  const auto look = [&]() {
    tok_next += kWarps * kStep;
#pragma unroll
    for (int i = 0; i < G::TB; ++i) {
      at_page[i] += a.skip_pages[G::TB - 1];
      in_page[i] += a.skip_blocks[G::TB - 1];
      if (in_page[i] >= static_cast<int>(a.c.page_blocks)) in_page[i] -= a.c.page_blocks, ++at_page[i];
      page[i] = tok_next + 16 * i < t1 ? __ldg(pages + at_page[i]) : -1;
    }
  };
  uint32_t absent = 0;                         // bit (stage, block): nothing was requested
  const auto request = [&](int stage) {
#pragma unroll
    for (int i = 0; i < G::TB; ++i) {
      const bool ok = static_cast<uint32_t>(page[i]) < static_cast<uint32_t>(a.c.pages);
      const uint32_t bit = 1u << (stage * G::TB + i);
      absent = ok ? absent & ~bit : absent | bit;
      if (ok) {
        const uint8_t* src = lane_src + page[i] * a.c.page_bytes;
        const uint8_t* codes = src + in_page[i] * G::kCodes;
        const uint8_t* words = src + (a.c.code_bytes + in_page[i] * G::kWords);
        const uint32_t at = stage * G::kStage + i * G::kBlock;
#pragma unroll
        for (int c = 0; c < G::RB / 32; ++c) {
          cp_async16(copy_k + at + 512 * c, codes + 512 * c);
          cp_async16((copy_v ^ G::copy_bits(c, true)) + at + 512 * c, codes + to_values + 512 * c);
        }
        if (lane < G::kWords / 16) {
          cp_async16(copy_w + at, words);
          cp_async16(copy_w + G::kWords + at, words + to_values);
        }
      } else if (tok_next + 16 * i < t1) {
        if (lane == 0) atomicOr(a.c.err, MOE_DEVERR_BAD_PAGE);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < G::kStages - 1; ++s) {
    request(s);
    look();
  }

  // ---- queries
  Warp<D, BITS, NT> w;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = row0 + 8 * n + g;
    float mx = 0.f;
    float qv[G::J][16];
    if (r < n_rows) {
      const int qrow = pre ? r / a.G : b * a.nq + r / a.G;
      const uint16_t* qp = a.q + qrow * a.q_row + (hk * a.G + r % a.G) * a.q_head;
#pragma unroll
      for (int j = 0; j < G::J; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 v = *reinterpret_cast<const uint4*>(qp + 64 * j + 16 * t + 8 * h);
          const uint32_t wd[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            qv[j][8 * h + 2 * i] = bf16_lo(wd[i]);
            qv[j][8 * h + 2 * i + 1] = bf16_hi(wd[i]);
          }
        }
    } else {
#pragma unroll
      for (int j = 0; j < G::J; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) qv[j][i] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < G::J; ++j)
#pragma unroll
      for (int i = 0; i < 16; ++i) mx = fmaxf(mx, fabsf(qv[j][i]));
    mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 2));
    const uint32_t e = min(max(__float_as_uint(mx) >> 23, 1u), 253u);
    // q' reaches 2^12 .. 2^13: subnormals only below 2^-26 of the row's largest element
    const float down = __uint_as_float((254u - e) << 23) * 4096.f;
    const float up = __uint_as_float(e << 23) * 4096.f;         // 2^-12 * 2^24
#pragma unroll
    for (int j = 0; j < G::J; ++j) {
      float all = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // operand pairs in the order the codes come out of a word: neighbours of a
        // byte pair, or nibbles 4 apart, the odd ones times 16 and so q' over 16
        const int e0 = BITS == 8 ? 2 * i : 8 * (i / 4) + i % 4;
        const int e1 = BITS == 8 ? e0 + 1 : e0 + 4;
        const float z = BITS == 4 && (i & 1) ? down * 0.0625f : down;
        const uint32_t p = pack_f16(qv[j][e0] * z, qv[j][e1] * z);
        w.q[n][j][i] = p;
        const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&p));
        all += (back.x + back.y) * (BITS == 4 && (i & 1) ? 16.f : 1.f);
      }
      all += __shfl_xor_sync(kAll, all, 1);
      all += __shfl_xor_sync(kAll, all, 2);
#pragma unroll
      for (int c = 0; c < 2; ++c) {            // of the columns this thread accumulates
        w.qsum[n][j][c] = __shfl_sync(kAll, all, (2 * t + c) * 4) * 0x1p-24f;
        w.ob[n][j][c] = 0.f;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) w.o[n][j][u][i] = 0.f;
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      w.row_scale[n][c] = a.scale2 * __shfl_sync(kAll, up, (2 * t + c) * 4);
      const int rc = row0 + 8 * n + 2 * t + c;
      w.lim[n][c] = rc < n_rows ? limit(rc) : t1;
      w.m[n][c] = -INFINITY;
      w.l[n][c] = 0.f;
      w.top_x[n][c] = -INFINITY;
    }
  }
#pragma unroll
  for (int j = 0; j < G::J; ++j) w.seen[j] = 0, w.set_unit(j, 127), w.seen[j] = 0;
  int low = t1;                                // tokens that every row of the tile sees
#pragma unroll
  for (int n = 0; n < NT; ++n) low = min(low, min(w.lim[n][0], w.lim[n][1]));
  low = __reduce_min_sync(kAll, low);

  const uint32_t key_off = G::key_lane(g, t), value_off = G::value_lane(g, t);
  int stage = 0;
  for (int s = warp; s < steps; s += kWarps) {
    {
      const int free = stage == 0 ? G::kStages - 1 : stage - 1;
      request(free);
      look();
    }
    cp_async_wait<G::kStages - 1>();
    __syncwarp();
    const int tok0 = t0 + s * kStep;
    const uint32_t gone = absent >> (stage * G::TB) & ((1u << G::TB) - 1);
    int top[G::TB];
#pragma unroll
    for (int i = 0; i < G::TB; ++i) top[i] = gone >> i & 1 ? 0 : t1;
    const uint8_t* st = ring + stage * G::kStage;
    if (tok0 + kStep <= low && gone == 0)
      w.template step<false>(st, tok0, top, g, key_off, value_off, s == warp);
    else
      w.template step<true>(st, tok0, top, g, key_off, value_off, s == warp);
    __syncwarp();                              // the stage may be overwritten
    stage = stage == G::kStages - 1 ? 0 : stage + 1;
  }
  cp_async_wait<0>();
  __syncthreads();                             // the ring becomes the join's buffer

  // ---- join the warps
  constexpr int kRow = D + 4;
  float* so = reinterpret_cast<float*>(smem);
  float2* sml = reinterpret_cast<float2*>(smem + SplitSmem<D, BITS, NT>::kBytes - kWarps * 8 * NT * 8);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int r = 8 * n + 2 * t + c;
      const float l = sum_over_rows8(w.l[n][c]);
      if (g == 0) sml[warp * 8 * NT + r] = make_float2(w.m[n][c], l);
#pragma unroll
      for (int j = 0; j < G::J; ++j) {
        const float ob = sum_over_rows8(w.ob[n][j][c]);
        const float up = w.unit(j);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          constexpr float kOdd = BITS == 4 ? 0.0625f : 1.f;
          *reinterpret_cast<float2*>(so + (warp * 8 * NT + r) * kRow + 64 * j + 8 * g + 2 * u) =
              make_float2((w.o[n][j][u][c] + ob) * up,
                          fmaf(w.o[n][j][u][2 + c], kOdd, ob) * up);
        }
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 8 * NT * D / 4; i += kThreads) {
    const int r = i / (D / 4), d = i % (D / 4) * 4;
    const int row = row0 + r;
    if (row >= n_rows) break;
    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) top = fmaxf(top, sml[k * 8 * NT + r].x);
    const float ref = top == -INFINITY ? 0.f : top;
    float l = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      const float2 ml = sml[k * 8 * NT + r];
      if (ml.x == -INFINITY && ml.y == 0.f) continue;
      const float keep = exp2_approx(ml.x - ref);
      const float4 v = *reinterpret_cast<const float4*>(so + (k * 8 * NT + r) * kRow + d);
      l = fmaf(ml.y, keep, l);
      y.x = fmaf(v.x, keep, y.x);
      y.y = fmaf(v.y, keep, y.y);
      y.z = fmaf(v.z, keep, y.z);
      y.w = fmaf(v.w, keep, y.w);
    }
    const int qrow = pre ? row / a.G : b * a.nq + row / a.G;
    const int head = hk * a.G + row % a.G;
    if (whole && a.lone) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      *reinterpret_cast<uint2*>(a.out + qrow * a.o_row + head * a.o_head + d) =
          make_uint2(pack_bf16(y.x * inv, y.y * inv), pack_bf16(y.z * inv, y.w * inv));
    } else {
      const int64_t at = whole ? (pre ? 0 : a.own_whole) + static_cast<int64_t>(qrow) * a.Hq + head
                               : a.slots + static_cast<int64_t>(slot) * (8 * NT) + r;
      *reinterpret_cast<float4*>(a.part + at * D + d) = y;
      if (d == 0) a.ml[at] = make_float2(top, l);
    }
  }
  __syncthreads();                             // the join's buffer becomes the ring again
  }
  if (a.pre_units) griddep_wait();
}

// Joins the parts of a query row and head: a warp per row, or W warps that share its parts.
// Bound by latency, so the loads come in as few dependent rounds as they can: where the
// row's parts are; then their (m, l), a part per lane, and their values, kJoinLoads parts
// at a time, beside each other.
constexpr int kJoinLoads = 8;
template <int W>
constexpr int kJoinThreads = W == 1 ? kThreads : 32 * W;

template <int D, int W>
__global__ void __launch_bounds__(kJoinThreads<W>) attn_join_kernel(const AttnArgs a) {
  griddep_wait();
  constexpr int E = D / 32;
  constexpr int kRows = kJoinThreads<W> / 32 / W;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t heads = static_cast<int64_t>(a.B) * a.nq * a.Hq;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * kRows + warp / W;
  if (at >= heads) return;                       // (W > 1: at is the block's)
  const int row = static_cast<int>(at / a.Hq), head = static_cast<int>(at % a.Hq);
  const int hk = head / a.G, b = row / a.nq;
  // (loads that do not wait for each other)
  // (with max_len = 0 no other kernel looks at the lengths)
  const bool own = a.own_units || a.own_tiles;
  const bool report = !own && row % a.nq == 0 && head == 0 && warp % W == 0 && lane == 0;
  const int len = own || report ? context_len(a, b, report) : 0;
  const int first = a.own_tiles ? a.first[b] : 0;
  const int share = a.pre_blocks || a.own_tiles ? *a.share_out : 1;
  // Parts of each context: `n` of them; the first at p0, the second at p1, then p1 + step, ...
  struct Parts {
    int n = 0;
    int64_t p0 = 0, p1 = 0, step = 0;
    __device__ int64_t at(int i) const { return i == 0 ? p0 : p1 + (i - 1) * step; }
  } parts[2];
  // row kernel: part k of the row at (k * heads + row); split kernel: tiles [g, g + T)
  const auto of_rows = [&](Parts& p, int64_t base, int g, int T) {
    p.n = T > 0 ? (g + T - 1) / a.share - g / a.share + 1 : 0;
    p.p0 = base + at;
    p.p1 = base + heads + at;
    p.step = heads;
  };
  const auto of_split = [&](Parts& p, int64_t whole, int g, int T, int r) {
    if (T == 0) return;
    const int k0 = g / share, k1 = (g + T - 1) / share;
    const int rows = 8 * a.nt;
    p.n = k1 - k0 + 1;
    // a unit that begins inside a block's share is that block's second kind of piece
    p.p0 = p.n == 1 ? whole + at : a.slots + static_cast<int64_t>(2 * k0 + (g != k0 * share)) * rows + r % rows;
    p.p1 = a.slots + static_cast<int64_t>(2 * (k0 + 1)) * rows + r % rows;
    p.step = 2 * rows;
  };
  if (a.pre_units) {
    const int u = hk * a.pre_row_tiles + (row * a.G + head % a.G) / a.unit_rows;
    of_rows(parts[0], 0, u * a.pre_T, (a.prefix_len + a.row_tile - 1) / a.row_tile);
  } else if (a.pre_blocks) {
    const int r = row * a.G + head % a.G;
    const int u = hk * a.pre_tiles + r / (8 * a.nt);
    of_split(parts[0], 0, u * a.pre_T, a.pre_T, r);
  }
  if (own) {
    const int r = row % a.nq * a.G + head % a.G;
    if (a.own_units) {
      const int rt = r / a.unit_rows;
      const int u = (b * a.c.Hkv + hk) * a.own_row_tiles + unit_place(rt, a.own_row_tiles);
      const int seen = own_limit(a, len, min((rt + 1) * a.unit_rows, a.nq * a.G) - 1);
      of_rows(parts[1], a.own_whole, a.pre_units * a.pre_T + u * a.own_T,
              (seen + a.row_tile - 1) / a.row_tile);
    } else {
      const int T = split_tiles(len);
      const int units = a.c.Hkv * a.own_tiles;
      of_split(parts[1], a.own_whole,
               a.pre_blocks * a.pre_T + first * units + (hk * a.own_tiles + r / (8 * a.nt)) * T, T, r);
    }
  }
  if (a.lone && parts[0].n + parts[1].n == 1) return;   // its kernel wrote the output
  const int n = parts[0].n + parts[1].n;
  float m = -INFINITY, l = 0.f, o[E] = {};
  for (int s0 = warp % W; s0 < n; s0 += 32 * W) {
    // lane i holds the (m, l) of part s0 + W i
    const int s = s0 + W * lane;
    const bool in = s < n;
    const int64_t i = s < parts[0].n ? parts[0].at(s) : parts[1].at(s - parts[0].n);
    const float2 ml = in ? a.ml[i] : make_float2(0.f, 0.f);
    const bool live = in && !(ml.x == -INFINITY && ml.y == 0.f);
    const int count = min(32, (n - s0 + W - 1) / W);
    float top = live ? ml.x : -INFINITY;
#pragma unroll
    for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, x));
    top = fmaxf(top, m);
    const float keep = m == top ? 1.f : exp2_approx(m - top);
    const float add = live ? exp2_approx(ml.x - (top == -INFINITY ? 0.f : top)) : 0.f;
    const uint32_t alive = __ballot_sync(kAll, live);
    m = top;
    float sum = live ? ml.y * add : 0.f;
#pragma unroll
    for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(kAll, sum, x);
    l = fmaf(l, keep, sum);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= keep;
    for (int k0 = 0; k0 < count; k0 += kJoinLoads) {
      float v[kJoinLoads][E];
#pragma unroll
      for (int k = 0; k < kJoinLoads; ++k) {       // (k0 + k < 32)
        const float* from = a.part + __shfl_sync(kAll, i, k0 + k) * D + lane * E;
        const bool use = alive >> (k0 + k) & 1;    // (the whole warp's)
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          float2 x = make_float2(0.f, 0.f);
          if (use) x = *reinterpret_cast<const float2*>(from + e);
          v[k][e] = x.x, v[k][e + 1] = x.y;
        }
      }
#pragma unroll
      for (int k = 0; k < kJoinLoads; ++k) {
        const float w = __shfl_sync(kAll, add, k0 + k);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(v[k][e], w, o[e]);
      }
    }
  }
  if constexpr (W > 1) {
    __shared__ float2 sml[W];
    __shared__ float so[W][D];
    if (lane == 0) sml[warp] = make_float2(m, l);
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][lane * E + e] = o[e];
    __syncthreads();
    if (warp) return;
    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < W; ++k) top = fmaxf(top, sml[k].x);
    const float ref = top == -INFINITY ? 0.f : top;
    l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      if (sml[k].x == -INFINITY && sml[k].y == 0.f) continue;
      const float keep = exp2_approx(sml[k].x - ref);
      l = fmaf(sml[k].y, keep, l);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(so[k][lane * E + e], keep, o[e]);
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<uint32_t*>(a.out + row * a.o_row + head * a.o_head + lane * E + e) =
        pack_bf16(o[e] * inv, o[e + 1] * inv);
}

// How a call is cut into blocks.
struct Plan {
  AttnArgs a;                // units, shares and partial results
  int64_t split_tiles;       // most tiles of the split kernel
  unsigned row_blocks;
  size_t ml, first, total;   // workspace: offsets of the (m, l) pairs and the tile sums, size
};

// Sizes shares and grids only: no block waits for another, so a device with fewer
// multiprocessors gives the same results.
constexpr int kSMs = 152;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The row kernel is taken from 64 query rows of a key/value head on, if there is enough to
// multiply: it takes longer to get going and then multiplies faster. Measured, one request, 8
// bits, 2 key/value heads (4 bits alike), split and row kernel, us:
//   GFLOP              0.25         0.5          1            2            4
//   D 64,   64 rows    11.6  14.6   13.9  16.8   20.4  21.0   23.1  29.9   36.2  48.8
//   D 64,  256 rows    15.6  15.1   14.4  15.6   17.6  16.4   25.4  18.9   36.3  21.9
//   D 128,  64 rows    13.3  17.0   14.8  17.5   18.0  19.4   27.2  24.1   36.9  34.0
//   D 128, 256 rows    13.5  19.8   20.4  19.9   23.0  20.3   27.5  20.7   36.7  24.1
//   D 256,  64 rows    13.8  18.8   16.2  19.2   21.1  20.8   29.9  23.3   42.8  30.9
//   D 256, 1024 rows                13.8  20.3   18.3  21.0   31.2  22.4   44.0  24.7
// At D = 64 a unit of 64 rows is a quarter full, and the split kernel stays ahead of it.
constexpr int64_t kRowKernelRows = 64;
constexpr double kRowKernelFlops = 1e9;
bool row_kernel_pays(int64_t rows, int64_t heads, int D, int64_t len) {
  return rows >= kRowKernelRows && 4.0 * D * rows * heads * len >= kRowKernelFlops;
}

// Tiles per block for `units` units of T tiles on `sms` blocks, and the tiles that a unit
// is taken to have. Equal shares of the lined-up tiles leave some blocks two pieces, and a
// piece costs about as much as 5 tiles to start and end; with fewer units than blocks a
// unit may instead be cut into equal parts of its own (T rounded up to whole shares).
void share_out(int64_t units, int64_t* T, int64_t* share) {
  constexpr int64_t kPieceTiles = 5;
  const int64_t lined = std::max<int64_t>(1, ceil_div(units * *T, kSMs));
  if (units <= kSMs) {
    const int64_t own = std::max<int64_t>(2, ceil_div(*T, kSMs / units));   // (each part costs a partial result)
    if (own + kPieceTiles <= lined + (lined < *T ? 2 * kPieceTiles : kPieceTiles)) {
      *share = own;
      *T = ceil_div(*T, own) * own;
      return;
    }
  }
  *share = lined;
}

// The sizes that a call takes; products of them stay below 2^63.
bool sizes_allowed(int64_t B, int64_t nq, int64_t Hq, int64_t Hkv, int D, int64_t max_len,
                   int64_t prefix_len) {
  return B >= 0 && nq >= 1 && Hq >= 1 && Hq <= 65535 && Hkv >= 1 && Hkv <= 1024 && Hq % Hkv == 0 &&
         (D == 64 || D == 128 || D == 256) && max_len >= 0 && max_len <= (1 << 30) &&
         prefix_len >= 0 && prefix_len <= (1 << 30) && B * nq <= (1 << 24) &&
         B * nq * Hq <= 0x7FFFFFFF;
}

// False if the sizes are not allowed or ask for too much work.
bool make_plan(int64_t B, int64_t nq, int64_t Hq, int64_t Hkv, int D, int max_len, int prefix_len,
               Plan* out) {
  if (!sizes_allowed(B, nq, Hq, Hkv, D, max_len, prefix_len)) return false;
  Plan p{};
  AttnArgs& a = p.a;
  const int64_t G = Hq / Hkv;
  const int64_t own_rows = nq * G, pre_rows = B * nq * G;
  const bool pre = prefix_len > 0, own = max_len > 0;
  const bool pre_tc = pre && row_kernel_pays(pre_rows, Hkv, D, prefix_len);
  const bool own_tc = own && row_kernel_pays(own_rows, B * Hkv, D, max_len);
  // two column tiles share the conversion of the codes; at D = 256 their state
  // would not fit the registers
  a.nt = D <= 128 && ((own && !own_tc && own_rows > 8) || (pre && !pre_tc && pre_rows > 8)) ? 2 : 1;
  int64_t split_tiles = 0, pre_T = 0, own_T = 0, pre_units = 0, own_units = 0;
  a.unit_rows = attn_unit_rows(D);
  a.row_tile = attn_row_tile(D);
  if (pre_tc) {
    a.pre_row_tiles = static_cast<int>(ceil_div(pre_rows, a.unit_rows));
    pre_T = ceil_div(prefix_len, a.row_tile);
    pre_units = Hkv * a.pre_row_tiles;
  } else if (pre) {
    a.pre_tiles = static_cast<int>(ceil_div(pre_rows, 8 * a.nt));
    a.pre_T = static_cast<int>(ceil_div(prefix_len, kSplitTile));
    a.pre_blocks = static_cast<int>(Hkv) * a.pre_tiles;
    split_tiles += static_cast<int64_t>(a.pre_blocks) * a.pre_T;
  }
  if (own_tc) {
    a.own_row_tiles = static_cast<int>(ceil_div(own_rows, a.unit_rows));
    own_T = ceil_div(max_len, a.row_tile);
    own_units = B * Hkv * a.own_row_tiles;
  } else if (own) {
    a.own_tiles = static_cast<int>(ceil_div(own_rows, 8 * a.nt));
    split_tiles += B * Hkv * a.own_tiles * ceil_div(max_len, kSplitTile);
  }
  // one wave of blocks, or fewer with a tile each
  int wave = 0;
  for (int bits : {4, 8}) wave = std::max(wave, kSMs * split_blocks_per_sm(D, bits, a.nt));
  p.split_tiles = split_tiles;
  int64_t share = 0;
  if (pre_units && own_units)
    share = std::max<int64_t>(1, ceil_div(pre_units * pre_T + own_units * own_T, kSMs));
  else if (pre_units)
    share_out(pre_units, &pre_T, &share);
  else if (own_units)
    share_out(own_units, &own_T, &share);
  const int64_t tiles = pre_units * pre_T + own_units * own_T;
  if (split_tiles > (1 << 30) || tiles > (1 << 30)) return false;   // the kernels count them in 32 bits
  const int64_t slots = 2 * std::min<int64_t>(wave, split_tiles);
  if (tiles > 0) {
    a.share = static_cast<int>(share);
    p.row_blocks = static_cast<unsigned>(ceil_div(tiles, share));
    a.pre_units = static_cast<int>(pre_units);
    a.own_units = static_cast<int>(own_units);
    if (pre_units) a.pre_T = static_cast<int>(pre_T);
    if (own_units) a.own_T = static_cast<int>(own_T);
  }
  // partial results: the prefix's per row, the own tokens' per row, the split kernel's slots
  const int64_t heads = B * nq * Hq;
  const int64_t pre_parts = a.pre_units ? (a.pre_T - 1) / a.share + 2 : pre ? 1 : 0;
  const int64_t own_parts = a.own_units ? (a.own_T - 1) / a.share + 2 : own && pre ? 1 : 0;
  a.lone = !(pre && own);
  a.own_whole = (a.lone && !a.pre_units ? 0 : pre_parts) * heads;
  a.slots = a.own_whole + own_parts * heads;
  if (a.lone && !a.pre_units && !a.own_units) a.slots = 0;   // whole pieces write the output
  const int64_t n = a.slots + slots * 8 * a.nt;
  p.ml = (static_cast<size_t>(n) * D * 4 + 255) / 256 * 256;
  p.first = (p.ml + static_cast<size_t>(n) * 8 + 255) / 256 * 256;
  p.total = p.first + (static_cast<size_t>(B) + 1) * 4;
  p.total = (p.total + 255) / 256 * 256;
  *out = p;
  return true;
}

template <int D, int BITS, int NT>
cudaError_t launch_split(const AttnArgs& a, int64_t tiles, cudaStream_t s) {
  const unsigned blocks = static_cast<unsigned>(
      std::min<int64_t>(tiles, kSMs * split_blocks_per_sm(D, BITS, NT)));
  constexpr size_t smem = SplitSmem<D, BITS, NT>::kBytes;
  const auto kernel = attn_split_kernel<D, BITS, NT>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(kernel, smem, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(blocks), dim3(kThreads), smem, s, a);
}

template <int D>
cudaError_t launch(const AttnArgs& a, const Plan& p, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (p.row_blocks) e = launch_attn_rows(a, p.row_blocks, s);
  if (e != cudaSuccess) return e;
  if (p.split_tiles) {
    if constexpr (D <= 128) {
      if (a.nt == 2)
        e = a.c.bits == 8 ? launch_split<D, 8, 2>(a, p.split_tiles, s)
                          : launch_split<D, 4, 2>(a, p.split_tiles, s);
    }
    if (a.nt == 1)
      e = a.c.bits == 8 ? launch_split<D, 8, 1>(a, p.split_tiles, s)
                        : launch_split<D, 4, 1>(a, p.split_tiles, s);
  }
  if (e != cudaSuccess) return e;
  const int64_t heads = static_cast<int64_t>(a.B) * a.nq * a.Hq;
  // Fewer rows have more parts each, and more warps to spare for them. Measured, whole
  // calls with 8, 4 and 1 warps per row: 32 rows and heads of 57 parts 53.4, 55.0, 61.3 us;
  // 1024 of 20 parts 69.2, 62.7, 63.6 us; 2048 of 2 parts (4 and 1) 100.0, 97.7 us.
  const auto join = [&](auto kernel, int warps, int64_t blocks) {
    return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(32 * warps), 0, s, a);
  };
  if (heads <= kSMs) return join(attn_join_kernel<D, 8>, 8, heads);
  if (heads <= kSMs * 8) return join(attn_join_kernel<D, 4>, 4, heads);
  return join(attn_join_kernel<D, 1>, kWarps, ceil_div(heads, kWarps));
}

bool bad16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool bad4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

}  // namespace
}  // namespace moeq4

extern "C" size_t moe_kv_attention_workspace_size(int32_t B, int32_t nq, int32_t Hq, int32_t Hkv,
                                                  int32_t D, int32_t max_len, int32_t prefix_len) {
  moeq4::Plan p;
  return moeq4::make_plan(B, nq, Hq, Hkv, D, max_len, prefix_len, &p) ? p.total : 0;
}

extern "C" int32_t moe_debug_kv_attention_rows(int32_t B, int32_t nq, int32_t Hq, int32_t Hkv,
                                               int32_t D, int32_t max_len, int32_t prefix_len) {
  moeq4::Plan p;
  if (!moeq4::make_plan(B, nq, Hq, Hkv, D, max_len, prefix_len, &p)) return -1;
  return (p.a.pre_units > 0 ? 1 : 0) | (p.a.own_units > 0 ? 2 : 0);
}

extern "C" moe_status moe_kv_attention(const moe_kv_attn* a, const moe_kv_cache* c, void* ws,
                                       size_t ws_bytes, void* stream) {
  using namespace moeq4;
  if (!a || a->B < 0 || a->nq < 1 || a->Hq < 1 || a->max_len < 0 || a->prefix_len < 0 ||
      a->table_stride < 0 || !std::isfinite(a->scale))
    return MOE_ERR_ARG;
  moe_status st = check_kv_cache(c);
  if (st != MOE_OK) return st;
  if (!sizes_allowed(a->B, a->nq, a->Hq, c->Hkv, c->D, a->max_len, a->prefix_len)) return MOE_ERR_SHAPE;
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
  Plan p;
  if (!make_plan(a->B, a->nq, a->Hq, c->Hkv, c->D, a->max_len, a->prefix_len, &p)) return MOE_ERR_SHAPE;
  if (ws_bytes < p.total) return MOE_ERR_WORKSPACE;
  if ((st = check_device()) != MOE_OK) return st;
  AttnArgs& k = p.a;
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
  k.scale2 = a->scale * 1.44269504088896340736f;
  k.c = kv_cache_args(*c);
  for (int tb = 1; tb <= 2; ++tb) {
    k.skip_pages[tb - 1] = kWarps * tb / static_cast<int>(k.c.page_blocks);
    k.skip_blocks[tb - 1] = kWarps * tb % static_cast<int>(k.c.page_blocks);
  }
  k.part = static_cast<float*>(ws);
  k.ml = reinterpret_cast<float2*>(static_cast<char*>(ws) + p.ml);
  k.share_out = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + p.first);
  k.first = k.share_out + 1;
  k.timeout_ns = wait_timeout_ns();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = c->D == 64    ? launch<64>(k, p, s)
                        : c->D == 128 ? launch<128>(k, p, s)
                                      : launch<256>(k, p, s);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
