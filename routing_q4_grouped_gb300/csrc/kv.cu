// kv.cu — rotary positions and the quantised key/value cache: moe_rope,
// moe_kv_append (turn, quantise, write) and moe_kv_read (read back).
//
// All three move each byte once and do little arithmetic per byte, so they are
// bound by memory bandwidth at many tokens and by launch latency at few. One
// launch each, no shared memory, no scratch. Bandwidths below are of a copy of 6.8 TB/s
// as measured on the same card, where a plain fill of memory reaches 4.0 TB/s: what
// writes more than it reads cannot come near the copy.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/moeq4_debug.h"
#include "internal.h"
#include "kv.cuh"
#include "ptx.cuh"

namespace moeq4 {

moe_status check_kv_cache(const moe_kv_cache* c) {
  if (!c || !c->data || !c->err) return MOE_ERR_ARG;
  if (moe_kv_cache_size(c->pages, c->page_size, c->Hkv, c->D, c->bits) == 0) return MOE_ERR_SHAPE;
  if ((reinterpret_cast<uintptr_t>(c->data) & 15u) || (reinterpret_cast<uintptr_t>(c->err) & 3u))
    return MOE_ERR_ALIGN;
  return MOE_OK;
}

KvCache kv_cache_args(const moe_kv_cache& c) {
  KvCache k{};
  k.data = static_cast<uint8_t*>(c.data);
  k.err = c.err;
  k.pages = c.pages;
  k.page_size = c.page_size;
  k.Hkv = c.Hkv;
  k.D = c.D;
  k.bits = c.bits;
  k.row_bytes = c.D * c.bits / 8;
  k.code_bytes = c.page_size * k.row_bytes;
  k.head_bytes = k.code_bytes + c.page_size * (c.D / kKvGroup) * 4;
  k.page_bytes = 2ll * c.Hkv * k.head_bytes;
  k.page_blocks = static_cast<uint32_t>(c.page_size / 16);
  k.page_magic = (1ull << 37) / k.page_blocks + 1;
  return k;
}

namespace {

constexpr int kThreads = 128;

bool bad_align(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// ------------------------------------------------------------------- rotary

struct RopeArgs {
  const void* x;
  void* out;
  const int32_t* pos;
  const uint64_t* phase;
  int64_t x_row, x_head, o_row, o_head;
  int T, H, D, rot;
  int units;                 // units of 2V elements per head, D / 2V
  int per;                   // heads per thread
  float mscale;
  int interleaved, backward, copy_tail;
};

template <typename E>
__device__ __forceinline__ float to_f(E v);
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f(float v) { return v; }
template <typename E>
__device__ __forceinline__ E from_f(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float from_f(float v) { return v; }

template <typename E, int V>
struct alignas(V * sizeof(E)) Vec {
  E e[V];
};

// Thread = (token, block of heads, unit): a unit is two vectors of V elements rot/2 apart,
// which hold V whole pairs in either layout (elements i and i + rot/2 meet across the two,
// elements 2i and 2i + 1 within one), so that neighbouring lanes always touch
// neighbouring vectors. The V angles are computed once and used for every head of the
// block; heads go two at a time, to keep more loads in flight. Units past rot / 2V copy.
// Measured: 2047 tokens of 40 fp32 heads of 128 elements (83.9 MB), 15.7 us, 79 % of the
// copy's bandwidth. One token: 2.4 us on the device, which is the launch.
template <typename E, int V>
__global__ void __launch_bounds__(kThreads) rope_kernel(RopeArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int tokens = max(1, kThreads / a.units);       // per block; (units above the block: several)
  const int u = threadIdx.x % a.units + blockIdx.z * kThreads;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * tokens + threadIdx.x / a.units;
  if (t >= a.T || u >= a.units || threadIdx.x >= tokens * a.units) return;
  const int h0 = blockIdx.y * a.per, h1 = min(a.H, h0 + a.per);
  const int turned = a.rot / (2 * V);
  const bool tail = u >= turned;
  if (tail && !a.copy_tail) return;
  const int first = tail ? a.rot + (u - turned) * 2 * V : u * V;
  const int second = tail ? first + V : first + a.rot / 2;
  const E* x = static_cast<const E*>(a.x) + t * a.x_row;
  E* o = static_cast<E*>(a.out) + t * a.o_row;
  using Vt = Vec<E, V>;
  float c[V], s[V];
  if (!tail) {
    const int32_t pos = a.pos[t];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      // pairs of the first vector, then (interleaved) those of the second
      const int pair = !a.interleaved ? first + i
                       : i < V / 2    ? first / 2 + i
                                      : second / 2 + i - V / 2;
      rope_sincos(pos, a.phase[pair], c[i], s[i]);
      c[i] *= a.mscale;
      s[i] *= a.backward ? -a.mscale : a.mscale;
    }
  }
  const auto turn = [&](Vt& p, Vt& q) {
    if (tail) return;
    if (a.interleaved) {
#pragma unroll
      for (int i = 0; i + 1 < V; i += 2) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          Vt& v = k ? q : p;
          const int at = i / 2 + k * (V / 2);
          const float fa = to_f(v.e[i]), fb = to_f(v.e[i + 1]);
          v.e[i] = from_f<E>(rope_first(fa, fb, c[at], s[at]));
          v.e[i + 1] = from_f<E>(rope_second(fa, fb, c[at], s[at]));
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float fa = to_f(p.e[i]), fb = to_f(q.e[i]);
        p.e[i] = from_f<E>(rope_first(fa, fb, c[i], s[i]));
        q.e[i] = from_f<E>(rope_second(fa, fb, c[i], s[i]));
      }
    }
  };
  for (int h = h0; h < h1; h += 2) {
    Vt p[2], q[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (h + k >= h1) break;
      p[k] = *reinterpret_cast<const Vt*>(x + (h + k) * a.x_head + first);
      q[k] = *reinterpret_cast<const Vt*>(x + (h + k) * a.x_head + second);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (h + k >= h1) break;
      turn(p[k], q[k]);
      *reinterpret_cast<Vt*>(o + (h + k) * a.o_head + first) = p[k];
      *reinterpret_cast<Vt*>(o + (h + k) * a.o_head + second) = q[k];
    }
  }
}

// One pair, or two elements to copy, per thread: any sizes, strides and alignment.
template <typename E>
__global__ void __launch_bounds__(kThreads) rope_pair_kernel(RopeArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int u = static_cast<int>(id % (a.D / 2));
  const int64_t th = id / (a.D / 2);
  const int64_t t = th / a.H, h = th % a.H;
  if (t >= a.T) return;
  const E* x = static_cast<const E*>(a.x) + t * a.x_row + h * a.x_head;
  E* o = static_cast<E*>(a.out) + t * a.o_row + h * a.o_head;
  if (2 * u >= a.rot) {
    if (a.copy_tail) {
      o[2 * u] = x[2 * u];
      o[2 * u + 1] = x[2 * u + 1];
    }
    return;
  }
  const int first = a.interleaved ? 2 * u : u, second = a.interleaved ? 2 * u + 1 : u + a.rot / 2;
  float c, s;
  rope_sincos(a.pos[t], a.phase[u], c, s);
  c *= a.mscale;
  s *= a.backward ? -a.mscale : a.mscale;
  const float fa = to_f(x[first]), fb = to_f(x[second]);
  o[first] = from_f<E>(rope_first(fa, fb, c, s));
  o[second] = from_f<E>(rope_second(fa, fb, c, s));
}

// Heads per thread: one while the call is small (latency), up to `most` that share their
// angles once there are threads enough to fill the multiprocessors several times. Measured
// back to back: an append of 4096 tokens of 32 + 8 + 8 heads with at most 16, 4 and 1 heads
// 29.9, 37.3 and 98.1 us; rope on 2047 tokens of 40 heads with 4, 2 and 1 heads 10.6, 10.8
// and 16.3 us (inputs partly in L2).
int heads_per_thread(int64_t T, int64_t units, int64_t H, int most) {
  int per = 1;
  while (per < most && T * units * H / (2 * per) >= 152 * 1024) per *= 2;
  return per;
}

template <typename E, int V>
cudaError_t launch_rope_v(RopeArgs a, cudaStream_t s) {
  a.units = a.D / (2 * V);
  a.per = heads_per_thread(a.T, a.units, a.H, 4);
  const int tokens = std::max(1, kThreads / a.units);
  const dim3 grid((a.T - 1) / tokens + 1, (a.H + a.per - 1) / a.per,
                  (a.units + kThreads - 1) / kThreads);
  return launch_pdl(rope_kernel<E, V>, grid, dim3(kThreads), 0, s, a);
}

template <typename E>
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s) {
  const uint64_t all = static_cast<uint64_t>(a.x_row | a.x_head | a.o_row | a.o_head);
  const uint64_t p = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.out);
  const auto fits = [&](int v) {
    return a.rot % (2 * v) == 0 && a.D % (2 * v) == 0 && all % v == 0 && p % (v * sizeof(E)) == 0;
  };
  constexpr int kWide = 16 / sizeof(E);
  if (fits(kWide)) return launch_rope_v<E, kWide>(a, s);
  if (fits(kWide / 2)) return launch_rope_v<E, kWide / 2>(a, s);
  const int64_t blocks = (static_cast<int64_t>(a.T) * a.H * (a.D / 2) + kThreads - 1) / kThreads;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  return launch_pdl(rope_pair_kernel<E>, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, s, a);
}

// ------------------------------------------------------------------- append

struct AppendArgs {
  const uint16_t *q, *k, *v;
  uint16_t* q_out;
  int64_t q_row, q_head, k_row, k_head, v_row, v_head, qo_row, qo_head;
  const int32_t *slots, *pos;
  const uint64_t* phase;     // nullptr: no rotation
  int T, Hq, rot, interleaved;
  float mscale;
  int per, turn_blocks;      // heads per thread; blocks of query and key heads
  KvCache c;
};

__device__ __forceinline__ void unpack8(uint4 w, float (&v)[8]) {
  const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(r[i]);
    v[2 * i + 1] = bf16_hi(r[i]);
  }
}

__device__ __forceinline__ float ld_bf16(const uint16_t* p) {
  return __uint_as_float(static_cast<uint32_t>(*p) << 16);
}

// Turns the 8 elements from e0 on of one head after another to one position. Element e
// becomes x cos -+ partner sin (- in the first of a pair), rounded to bf16.
struct Turner {
  float c[8], s[8];          // cos, and sin with its sign, of each element's pair
  int n;                     // elements below rot
  int mode;                  // 0: none of them; 1: partners are neighbours; 2: a run at `shift`;
  int shift;                 // 3: one by one, element i's at shift or (upper half) -shift
  int upper;

  __device__ __forceinline__ void prepare(const AppendArgs& a, int e0, int32_t pos) {
    n = a.phase ? min(max(a.rot - e0, 0), 8) : 0;
    mode = 0;
    shift = upper = 0;
    if (n == 0) return;
    const int half = a.rot / 2;
    mode = a.interleaved ? 1 : half % 8 == 0 ? 2 : 3;
    shift = mode == 2 && e0 >= half ? -half : half;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = e0 + i;
      const bool first = a.interleaved ? (e & 1) == 0 : e < half;
      const int pair = a.interleaved ? e >> 1 : first ? e : e - half;
      if (!first) upper |= 1 << i;
      c[i] = 1.f;
      s[i] = 0.f;
      if (i < n) {
        rope_sincos(pos, a.phase[pair], c[i], s[i]);
        c[i] *= a.mscale;
        s[i] *= first ? -a.mscale : a.mscale;
      }
    }
  }
  // The partner run, where it is one (mode 2).
  __device__ __forceinline__ uint4 partner(const uint16_t* head, int e0) const {
    return mode == 2 ? *reinterpret_cast<const uint4*>(head + e0 + shift) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ uint4 turn(const uint16_t* head, int e0, uint4 own, uint4 other) const {
    if (mode == 0) return own;
    float v[8], p[8];
    unpack8(own, v);
    if (mode == 1) {
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = v[i ^ 1];
    } else if (mode == 2) {
      unpack8(other, p);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        p[i] = i < n ? ld_bf16(head + e0 + i + (upper >> i & 1 ? -shift : shift)) : 0.f;
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      float y[2];
#pragma unroll
      for (int k = 0; k < 2; ++k)
        y[k] = i + k < n ? __fadd_rn(__fmul_rn(v[i + k], c[i + k]), __fmul_rn(p[i + k], s[i + k]))
                         : v[i + k];
      w[i / 2] = pack_bf16(y[0], y[1]);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// Quantises the 8 elements of each lane in groups of 8 lanes and writes codes and word.
template <int BITS>
__device__ __forceinline__ void store_codes(const AppendArgs& a, uint4 raw, int slot, int head,
                                            int run, bool write) {
  float v[8];
  unpack8(raw, v);
  float lo = v[0], hi = v[0];
  bool finite = true;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo = fminf(lo, v[i]);
    hi = fmaxf(hi, v[i]);
    finite &= fabsf(v[i]) < INFINITY;
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
  }
  finite = ((__ballot_sync(0xFFFFFFFFu, finite) >> (threadIdx.x & 24u)) & 0xFFu) == 0xFFu;
  if (!write) return;
  constexpr float kLevels = (1 << BITS) - 1;
  uint32_t words = 0x7FC00000u;            // scale 0, bias NaN
  uint32_t code[8] = {};
  if (finite) {
    // halves: max - min may pass the largest float; the constant is one rounding of 2 / levels
    const float range = __fsub_rn(0.5f * hi, 0.5f * lo);
    words = pack_bf16(__fmul_rn(range, 1.0f / (0.5f * kLevels)), lo);
    const float scale = bf16_lo(words);
    // (the reciprocal of a scale below 2^-126 may pass the largest float: differences and
    // scale are taken 2^64 times as large there, which is exact)
    const float up = scale < 0x1p-126f ? 0x1p64f : 1.f;
    const float per = scale > 0.f ? __fdiv_rn(1.0f, scale * up) : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      code[i] = static_cast<uint32_t>(
          fminf(fmaxf(rintf(__fmul_rn(__fsub_rn(v[i], lo) * up, per)), 0.f), kLevels));
  }
  const int page = page_of_block(a.c, static_cast<uint32_t>(slot) >> 4);
  const int row = slot - page * a.c.page_size;
  uint8_t* blk = kv_block(a.c, page, head);
  uint8_t* dst = blk + row * a.c.row_bytes + run * BITS;
  if (BITS == 8)
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(code[0] | code[1] << 8 | code[2] << 16 | code[3] << 24,
                   code[4] | code[5] << 8 | code[6] << 16 | code[7] << 24);
  else
    *reinterpret_cast<uint32_t*>(dst) = code[0] | code[1] << 4 | code[2] << 8 | code[3] << 12 |
                                        code[4] << 16 | code[5] << 20 | code[6] << 24 |
                                        code[7] << 28;
  if ((run & 7) == 0)
    *reinterpret_cast<uint32_t*>(blk + a.c.code_bytes +
                                 (row * (a.c.D / kKvGroup) + run / 8) * 4) = words;
}

// Thread = (token, block of heads, run of 8 elements). The blocks cover the query and key
// heads, whose angles a thread computes once for all of its heads, then the value heads.
// (q_out may be q only if no thread reads what another wrote: a turned run reads its
// partner run of the same head, whose D / 8 <= 32 threads are lanes of one warp;
// __syncwarp separates a head's reads from its writes.) Eight lanes hold a group of 64: its
// least and largest element take three exchanges each.
// Measured: 4096 tokens of 32 + 8 + 8 heads, D = 128, 4 bits (50 MB read, 38 MB written),
// 29.9 us, 43 % of the copy's bandwidth; issue slots are 53 % busy with turning, rounding
// and quantising, and the loads of a thread's few heads in flight bind beside them. 64
// tokens: 3.7 us on the device.
template <int BITS>
__global__ void __launch_bounds__(kThreads) append_kernel(AppendArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int runs = a.c.D / 8;              // 8, 16 or 32
  const int run = threadIdx.x & (runs - 1);
  const int hb = blockIdx.y;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads / runs) + threadIdx.x / runs;
  const bool live = t < a.T;               // whole groups of 8 lanes: D / 8 is a multiple of 8
  const int turned = a.Hq + a.c.Hkv;       // heads that turn
  const bool values = hb >= a.turn_blocks;
  const int h0 = (values ? hb - a.turn_blocks : hb) * a.per;
  const int h1 = min(values ? a.c.Hkv : turned, h0 + a.per);
  const int e0 = run * 8;
  int slot = -1;
  Turner turner;
  turner.mode = 0;
  if (live) {
    if (values || h1 > a.Hq) slot = a.slots[t];
    if (!values) turner.prepare(a, e0, a.phase ? a.pos[t] : 0);
  }
  const bool inside = slot >= 0 && slot < a.c.pages * a.c.page_size;
  if (slot != -1 && !inside && run == 0 && values && h0 == 0) atomicOr(a.c.err, MOE_DEVERR_BAD_SLOT);
  const auto head_at = [&](int h) {
    return values     ? a.v + t * a.v_row + h * a.v_head
           : h < a.Hq ? a.q + t * a.q_row + h * a.q_head
                      : a.k + t * a.k_row + (h - a.Hq) * a.k_head;
  };
  // Four heads' loads are in flight at a time: with one, the loop waits for memory.
  const uint4 none = make_uint4(0, 0, 0, 0);
  constexpr int kBatch = 4;
  for (int hh = h0; hh < h0 + a.per; hh += kBatch) {
    uint4 own[kBatch], other[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      own[k] = other[k] = none;
      if (live && hh + k < h1) {
        const uint16_t* head = head_at(hh + k);
        own[k] = *reinterpret_cast<const uint4*>(head + e0);
        other[k] = turner.partner(head, e0);
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (live && hh + k < h1) own[k] = turner.turn(head_at(hh + k), e0, own[k], other[k]);
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int h = hh + k;
      const bool here = live && h < h1;
      const bool query = here && !values && h < a.Hq;
      if (query) *reinterpret_cast<uint4*>(a.q_out + t * a.qo_row + h * a.qo_head + e0) = own[k];
      const bool code = here && !query;
      if (__any_sync(0xFFFFFFFFu, code))
        store_codes<BITS>(a, own[k], slot, values ? a.c.Hkv + h : h - a.Hq, run, code && inside);
    }
  }
}

// --------------------------------------------------------------------- read

// Thread = (run of 8 codes of a key or value head, four rows): lanes read neighbouring
// codes and write neighbouring 16 bytes of bf16, and a thread's four rows keep their
// loads in flight together. (Block = rows x one head; no division but by page.)
// Measured: 32768 rows of 8 heads, D = 128, 4 bits (38 MB read, 134 MB written), 42.0 us,
// 60 % of the copy's bandwidth; a plain fill of the 134 MB takes 34 us.
constexpr int kReadRows = 4;

template <int BITS>
__global__ void __launch_bounds__(kThreads) read_kernel(KvCache c, const int32_t* slots, int n,
                                                        uint16_t* k_out, uint16_t* v_out) {
  griddep_wait();
  griddep_launch_dependents();
  const int runs = c.D / 8, step = kThreads / runs;     // rows apart
  const int run = threadIdx.x & (runs - 1), h = blockIdx.y;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * step * kReadRows + threadIdx.x / runs;
  uint16_t* out = h < c.Hkv ? k_out : v_out;
  if (t0 >= n || !out) return;
  uint32_t q[kReadRows][2], w[kReadRows];
  bool in[kReadRows];
#pragma unroll
  for (int i = 0; i < kReadRows; ++i) {
    const int slot = t0 + i * step < n ? slots[t0 + i * step] : -1;
    in[i] = slot >= 0 && slot < c.pages * c.page_size;
    if (!in[i]) {
      if (slot != -1 && run == 0 && h % c.Hkv == 0) atomicOr(c.err, MOE_DEVERR_BAD_SLOT);
      continue;
    }
    const int page = page_of_block(c, static_cast<uint32_t>(slot) >> 4);
    const int row = slot - page * c.page_size;
    const uint8_t* blk = kv_block(c, page, h);
    w[i] = *reinterpret_cast<const uint32_t*>(blk + c.code_bytes +
                                              (row * (c.D / kKvGroup) + run / 8) * 4);
    const uint8_t* src = blk + row * c.row_bytes + run * BITS;
    if (BITS == 8) {
      const uint2 x = *reinterpret_cast<const uint2*>(src);
      q[i][0] = x.x, q[i][1] = x.y;
    } else {
      q[i][0] = *reinterpret_cast<const uint32_t*>(src);
    }
  }
#pragma unroll
  for (int i = 0; i < kReadRows; ++i) {
    if (t0 + i * step >= n) break;
    uint32_t r[4] = {};
    if (in[i]) {
      const float scale = bf16_lo(w[i]), bias = bf16_hi(w[i]);
      constexpr int kPer = 32 / BITS;
      constexpr uint32_t kMask = (1u << BITS) - 1;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t two = q[i][2 * k / kPer] >> (2 * k % kPer * BITS);
        r[k] = pack_bf16(fmaf(scale, static_cast<float>(two & kMask), bias),
                         fmaf(scale, static_cast<float>((two >> BITS) & kMask), bias));
      }
    }
    reinterpret_cast<uint4*>(out + ((t0 + i * step) * c.Hkv + h % c.Hkv) * c.D)[run] =
        make_uint4(r[0], r[1], r[2], r[3]);
  }
}

moe_status check_rope(const moe_rope_spec* r, int D) {
  if (!r || !r->phase) return MOE_ERR_ARG;
  if (r->interleaved < 0 || r->interleaved > 1 || !std::isfinite(r->mscale)) return MOE_ERR_ARG;
  if (r->rot < 2 || r->rot % 2 || r->rot > D) return MOE_ERR_SHAPE;
  if (bad_align(r->phase, 8)) return MOE_ERR_ALIGN;
  return MOE_OK;
}

// Strided bf16 rows that the vector path reads 16 bytes at a time.
moe_status check_rows(const void* p, int64_t row, int64_t head) {
  if (!p) return MOE_ERR_ARG;
  if (row < 0 || head < 0) return MOE_ERR_SHAPE;
  if (bad_align(p, 16) || row % 8 || head % 8) return MOE_ERR_ALIGN;
  return MOE_OK;
}

}  // namespace
}  // namespace moeq4

extern "C" size_t moe_kv_cache_size(int32_t pages, int32_t page_size, int32_t Hkv, int32_t D,
                                    int32_t bits) {
  if (pages < 1 || page_size < 16 || page_size % 16 || page_size > 4096 || Hkv < 1 ||
      Hkv > 1024 || (D != 64 && D != 128 && D != 256) || (bits != 4 && bits != 8) ||
      static_cast<int64_t>(pages) * page_size > 0x7FFFFFFF)
    return 0;
  return static_cast<size_t>(pages) * 2 * Hkv * page_size * (D * bits / 8 + D / moeq4::kKvGroup * 4);
}

extern "C" moe_status moe_rope_phases(uint64_t* phase, int32_t rot, double base, int32_t scaling,
                                      double factor, double trained, double fast, double slow) {
  if (!phase || !(base > 1.0) || !std::isfinite(base) || !(factor >= 1.0) ||
      !std::isfinite(factor) || scaling < MOE_ROPE_PLAIN || scaling > MOE_ROPE_BANDS)
    return MOE_ERR_ARG;
  if (rot < 2 || rot % 2) return MOE_ERR_SHAPE;
  if (scaling == MOE_ROPE_BANDS &&
      (!(trained > 0.0) || !(slow > 0.0) || !(fast > slow) || !std::isfinite(trained) ||
       !std::isfinite(fast)))
    return MOE_ERR_ARG;
  if (scaling == MOE_ROPE_BASE && rot == 2) return MOE_ERR_SHAPE;   // the exponent rot / (rot - 2)
  constexpr double kTurn = 6.283185307179586476925;
  if (scaling == MOE_ROPE_BASE) base *= std::pow(factor, rot / (rot - 2.0));
  // pair index whose frequency makes `turns` turns over the trained length
  const auto pair_of = [&](double turns) {
    return rot * std::log(trained / (turns * kTurn)) / (2.0 * std::log(base));
  };
  double lo = 0.0, hi = 0.0;
  if (scaling == MOE_ROPE_BANDS) {
    lo = std::max(0.0, std::floor(pair_of(fast)));
    hi = std::min(rot - 1.0, std::ceil(pair_of(slow)));   // (0 or less: every pair is slow)
  }
  for (int i = 0; i < rot / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot);
    if (scaling == MOE_ROPE_LINEAR) f /= factor;
    if (scaling == MOE_ROPE_BANDS) {
      const double slowed = i >= hi ? 1.0 : i <= lo ? 0.0 : (i - lo) / (hi - lo);
      f = f * (1.0 - slowed) + f / factor * slowed;
    }
    phase[i] = static_cast<uint64_t>(std::rint(std::ldexp(f / kTurn, 64)));
  }
  return MOE_OK;
}

extern "C" moe_status moe_rope(const void* x, int64_t x_row, int64_t x_head, void* out,
                               int64_t out_row, int64_t out_head, const int32_t* pos, int32_t T,
                               int32_t H, int32_t D, const moe_rope_spec* rope, int32_t backward,
                               int32_t dtype, void* stream) {
  using namespace moeq4;
  if (T < 0 || H < 1 || D < 2 || backward < 0 || backward > 1 || dtype < MOE_BF16 ||
      dtype > MOE_F32)
    return MOE_ERR_ARG;
  if (D % 2 || D > 65536 || H > 65535) return MOE_ERR_SHAPE;
  moe_status st = check_rope(rope, D);
  if (st != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  if (!x || !out || !pos) return MOE_ERR_ARG;
  if (x_row < 0 || x_head < 0 || !rows_disjoint(out_row, out_head, T, H, D)) return MOE_ERR_SHAPE;
  if (x == out && (x_row != out_row || x_head != out_head)) return MOE_ERR_ARG;
  const unsigned es = dtype == MOE_F32 ? 4 : 2;
  if (bad_align(x, es) || bad_align(out, es) || bad_align(pos, 4)) return MOE_ERR_ALIGN;
  if ((st = check_device()) != MOE_OK) return st;
  RopeArgs a{};
  a.x = x;
  a.out = out;
  a.pos = pos;
  a.phase = rope->phase;
  a.x_row = x_row;
  a.x_head = x_head;
  a.o_row = out_row;
  a.o_head = out_head;
  a.T = T;
  a.H = H;
  a.D = D;
  a.rot = rope->rot;
  a.mscale = rope->mscale;
  a.interleaved = rope->interleaved;
  a.backward = backward;
  a.copy_tail = x != out;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = dtype == MOE_F32   ? launch_rope<float>(a, s)
                  : dtype == MOE_F16 ? launch_rope<__half>(a, s)
                                     : launch_rope<__nv_bfloat16>(a, s);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" moe_status moe_kv_append(const moe_kv_new* n, const moe_kv_cache* c, void* stream) {
  using namespace moeq4;
  if (!n || n->T < 0 || n->Hq < 0) return MOE_ERR_ARG;
  moe_status st = check_kv_cache(c);
  if (st != MOE_OK) return st;
  if (n->rope && (st = check_rope(n->rope, c->D)) != MOE_OK) return st;
  if (!n->rope && n->q) return MOE_ERR_ARG;
  if (n->T == 0) return MOE_OK;
  if ((st = check_rows(n->k, n->k_row, n->k_head)) != MOE_OK ||
      (st = check_rows(n->v, n->v_row, n->v_head)) != MOE_OK)
    return st;
  if (!n->slots || (n->rope && !n->pos)) return MOE_ERR_ARG;
  if (bad_align(n->slots, 4) || bad_align(n->pos, 4)) return MOE_ERR_ALIGN;
  const int Hq = n->q ? n->Hq : 0;
  if (n->q) {
    if (n->Hq < 1) return MOE_ERR_ARG;
    if (n->Hq > 32768) return MOE_ERR_SHAPE;
    if ((st = check_rows(n->q, n->q_row, n->q_head)) != MOE_OK ||
        (st = check_rows(n->q_out, n->qo_row, n->qo_head)) != MOE_OK)
      return st;
    if (!rows_disjoint(n->qo_row, n->qo_head, n->T, Hq, c->D)) return MOE_ERR_SHAPE;
    if (n->q == n->q_out && (n->q_row != n->qo_row || n->q_head != n->qo_head)) return MOE_ERR_ARG;
  }
  AppendArgs a{};
  a.q = n->q;
  a.k = n->k;
  a.v = n->v;
  a.q_out = n->q_out;
  a.q_row = n->q_row;
  a.q_head = n->q_head;
  a.k_row = n->k_row;
  a.k_head = n->k_head;
  a.v_row = n->v_row;
  a.v_head = n->v_head;
  a.qo_row = n->qo_row;
  a.qo_head = n->qo_head;
  a.slots = n->slots;
  a.pos = n->pos;
  a.T = n->T;
  a.Hq = Hq;
  if (n->rope) {
    a.phase = n->rope->phase;
    a.rot = n->rope->rot;
    a.interleaved = n->rope->interleaved;
    a.mscale = n->rope->mscale;
  }
  a.c = kv_cache_args(*c);
  a.per = heads_per_thread(n->T, c->D / 8, Hq + 2 * c->Hkv, 16);
  a.turn_blocks = (Hq + c->Hkv + a.per - 1) / a.per;
  const int tokens = kThreads / (c->D / 8);      // per block
  const dim3 grid((n->T - 1) / tokens + 1, a.turn_blocks + (c->Hkv + a.per - 1) / a.per);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if ((st = check_device()) != MOE_OK) return st;
  const cudaError_t e = launch_pdl(c->bits == 8 ? append_kernel<8> : append_kernel<4>, grid,
                                   dim3(kThreads), 0, s, a);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" moe_status moe_kv_read(const moe_kv_cache* c, const int32_t* slots, int32_t n,
                                  uint16_t* k_out, uint16_t* v_out, void* stream) {
  using namespace moeq4;
  if (n < 0) return MOE_ERR_ARG;
  moe_status st = check_kv_cache(c);
  if (st != MOE_OK) return st;
  if (n == 0) return MOE_OK;
  if (!slots || (!k_out && !v_out)) return MOE_ERR_ARG;
  if (bad_align(slots, 4) || bad_align(k_out, 16) || bad_align(v_out, 16)) return MOE_ERR_ALIGN;
  const int rows = kThreads / (c->D / 8) * kReadRows;   // per block
  const dim3 grid((n - 1) / rows + 1, 2 * c->Hkv);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const KvCache k = kv_cache_args(*c);
  if ((st = check_device()) != MOE_OK) return st;
  const cudaError_t e =
      launch_pdl(c->bits == 8 ? read_kernel<8> : read_kernel<4>,
                 grid, dim3(kThreads), 0, s, k, slots, n, k_out, v_out);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" int32_t moe_debug_kv_page(int32_t page_size, int32_t slot) {
  if (slot < 0 || moe_kv_cache_size(1, page_size, 1, 64, 8) == 0) return -1;
  const moe_kv_cache c = {nullptr, nullptr, 1, page_size, 1, 64, 8};
  return moeq4::page_of_block(moeq4::kv_cache_args(c), static_cast<uint32_t>(slot) >> 4);
}
