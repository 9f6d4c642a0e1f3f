// attn_rows.cu — attention for many query rows of one key/value head (a chunk of a
// prompt, or a batch behind a shared prefix) on the 5th-generation tensor cores.
//
// With R rows a cached byte feeds 4 R operations, so from about a hundred rows on
// the products bound the work, not the bytes. A unit is 256 query rows (128 for
// D = 256) of one key/value head against a run of token tiles:
//   X[rows, tokens] = Q K^T     tcgen05.mma, M = 128 rows, N = 128 tokens (64 for
//                               D = 256), keys in shared memory (128-byte swizzle)
//   P = exp2(X - m)             tensor memory -> registers -> tensor memory, one
//                               thread per row, fp16, in place of X
//   O[rows, D] += P V           A = P from tensor memory, B = V^T in shared memory
// Codes are turned into fp16 operands once per tile, for all rows of the unit. A code
// c alone in the low bits of an fp16 is the subnormal c 2^-24, so value = s c + b is
// one fp16 fma with 2^24 s, with one rounding of 2^-11.
//
// fp16's range. Queries are divided by the power of two under their row's largest
// element, the keys of each 32 tokens by one over their largest magnitude, which goes into
// the logits' factor. A tile with keys that differ by more than 2^6 within 32 tokens takes
// one exponent per key (the same formulas with a factor per column).
// Values are divided by a power of two per group of the head and piece, since a group has
// its own columns of O: it is found from the piece's first tile and undone when the
// outputs are written, so groups of any ratio keep their bits. A tile in which a group of a
// token is outside the window in which fp16 rounds it by 2^-12 of its size or better is
// multiplied as bf16, weights and values (2^-8 each, fp32's range).
//
// The row maximum is not looked for tile by tile: m is only a reference, any value
// near the largest logit does. All weights are positive, so a row whose 32 columns sum to less
// than 2^15 held no weight near fp16's end and m stands; otherwise (and at a row's
// first tile) the tile's logits are read again for their maximum, m moves there and
// O and l follow. That leaves one fma, one exp2, one addition and half a conversion
// per element.
//
// Warps (one block per SM, persistent over its share of tiles):
//   0-3, 4-7  softmax of query tile 0 and 1 (warp % 4 = tensor-memory lane quarter),
//             their queries' load and their outputs' store (D = 256: 4-7 do half of both
//             for tile 0)
//   11        issues the products
//   15        finds the pages of the tiles ahead
//   8 9 10 12 13 14 16 17 (D = 64: the first four)  scales, and codes to operands
// D <= 128: two query tiles share each token tile and take turns, one in the tensor
// cores while the other is in its softmax. D = 256: one query tile, held in tensor
// memory, tiles of 64 tokens, and logits that alternate between two slots. Every wait on an
// mbarrier has a time limit; after one ran out, no thread waits again and the kernel ends
// with MOE_DEVERR_PIPE_TIMEOUT.
//
// Measured: the last 4096 query tokens of 32768 (16 query heads on 2, D = 128, 8 bits),
// 995 us, 1040 TFLOP/s, 53 % of the bf16 peak as measured. A tile of 128 tokens for 256
// rows takes about 4500 cycles, its products alone 2200. What binds is latency: the
// conversion of the next tile (codes from L2, fp16 arithmetic, shared memory) and the
// softmax (about 3400 cycles) leave each other hardly any slack. 512 rows behind a prefix
// of 16000 tokens (D = 256, 14 tiles a block) take 13 % of the peak: to load the queries
// (7 us, several dependent rounds of loads that queue behind the codes'), to come to the
// first weights (2 us) and to write partial results (4 us) costs as much as 8 tiles.
#include <cstdint>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "attn.cuh"
#include "internal.h"

namespace moeq4 {
namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kSoftWarps = 8;
constexpr int kMmaWarp = 11, kPageWarp = 15;
// Conversion warps: 8 9 10, 12 13 14, 16 17, i.e. none with warp % 4 == 3. A warp issues
// from sub-partition warp % 4, and the products' warp must not wait for busy neighbours
// there: alone on the multiprocessor it issues one product per 64 cycles (their full rate),
// beside four warps of fp32 arithmetic one per 128.
__host__ __device__ constexpr bool is_conv_warp(int warp) { return warp >= kSoftWarps && warp % 4 != 3; }
__host__ __device__ constexpr int conv_index(int warp) { return warp - 8 - (warp > 11) - (warp > 15); }
constexpr int kMetaRing = 4;
constexpr int kMaxSpread = 6;          // exponents of a tile's keys that share one power of two
constexpr uint32_t kTmemCols = 512;
constexpr uint8_t kDead = 0x80;        // token flag: its page is outside the cache

// Operands are divided so that the largest 2^24 scale is a finite fp16 (scale <= largest
// magnitude / 2^(BITS - 1)): keys by 2^kKeyRoom above the power of two under their largest,
// values by 2^kValueRoom above their group's.
template <int BITS>
constexpr int kKeyRoom = BITS == 8 ? 2 : 6;
template <int BITS>
constexpr uint32_t kValueRoom = BITS == 8 ? 1 : 5;
// A group's values may be up to 2^kAbove larger than the piece's first tokens suggested, and
// 2^kWindow smaller than that: there fp16's subnormals round them by 2^-12 of the group's size.
template <int BITS>
constexpr uint32_t kAbove = BITS == 8 ? 3 : 2;
template <int BITS>
constexpr uint32_t kWindow = BITS == 8 ? 11 : 7;

template <int D>
struct RowGeo {
  static constexpr int J = D / kKvGroup;
  static constexpr int QT = D == 256 ? 1 : 2;         // query tiles of a unit
  static constexpr int TT = D == 256 ? 64 : 128;      // tokens of a tile
  static constexpr int kConvWarps = D == 64 ? 4 : 8;
  static constexpr int kConvThreads = kConvWarps * 32;
  static constexpr int kThreads = (kConvWarps == 4 ? 16 : 18) * 32;
  static constexpr int KS = D == 256 ? 3 : 2;         // operand tiles in flight, keys and values each
  static constexpr bool kQTmem = D == 256;            // queries in tensor memory, not shared memory
  static constexpr int kStageRow = kQTmem ? 64 : 128;             // bytes of a row in a softmax warp's staging
  static constexpr uint32_t kQBytes = kQTmem ? 0 : 128 * D * 2;   // a query tile
  static constexpr uint32_t kTileBytes = TT * D * 2;  // a key or value tile
  static constexpr uint32_t kOffK = QT * kQBytes;
  static constexpr uint32_t kOffV = kOffK + KS * kTileBytes;
  static constexpr uint32_t kOffMeta = kOffV + KS * kTileBytes;
  static constexpr uint32_t kColO = 0;                // tensor memory: O of query tile q at D q,
  static constexpr uint32_t kColS = QT * D;           // then two logit slots of TT columns,
  static constexpr uint32_t kColQ = kColS + 2 * TT;   // then the queries
  static_assert(kColQ + (kQTmem ? D / 2 : 0) <= kTmemCols, "tensor memory");
  static_assert(KS < kMetaRing, "rings");
};

// Scales, biases and exponents of one tile, ready for use.
template <int D>
struct alignas(16) Meta {
  static constexpr int J = RowGeo<D>::J, TT = RowGeo<D>::TT;
  uint16_t vs[J][TT], vb[J][TT];       // values: scale * 2^24, bias (fp16, divided)
  uint32_t ksb[J][TT];                 // keys: as vs and vb, bias in the high half
  float kf[TT];                        // divisor of each token's key (slow tiles)
  uint8_t flag[TT];                    // bit j: value group j is NaN; kDead
  float run_kf[4];                     // of each run of 32 tokens (other tiles)
  // of each run: keys, values need the slow path; values outside the window of fp16
  alignas(8) uint8_t slow[2][4];
  alignas(4) uint8_t wide[4];
  uint32_t units;                      // exponent fields of the value groups' divisors
};

// Whether a tile's values are multiplied as bf16.
template <int D>
__device__ __forceinline__ bool is_wide(const Meta<D>& m) {
  return *reinterpret_cast<const uint32_t*>(m.wide) != 0;
}

struct Ctl {
  uint64_t q_full[2], k_full[3], k_empty[3], v_full[3];
  uint64_t s_full[2], p_full[2], pv_done[2], drain;
  // of tile t at t % 4: pages found; scales written; products done
  uint64_t base_full[kMetaRing], meta_full[kMetaRing], done[kMetaRing];
  int64_t base[kMetaRing][8];          // byte offset of a 16-token block's key codes
  const uint8_t* values;               // the cache's first value block
  int32_t words[kMetaRing][8];         // from there to its words; -1: no such block (its codes
                                       // are read from the cache's start and multiplied by 0)
  uint32_t run_top[2][4];              // of a piece's first tile: largest exponents of each run
  uint32_t units;                      // D = 256: the piece's, for the second warpgroup
  uint32_t tmem_base;
  int abort;
};

// Where the queries are in tensor memory, the softmax warps' staging has its own place,
// and after it 128 rows' ends.
template <int D>
constexpr uint32_t kOffStage =
    (RowGeo<D>::kOffMeta + kMetaRing * sizeof(Meta<D>) + sizeof(Ctl) + 127) / 128 * 128;

template <int D>
constexpr size_t row_smem() {
  return 1024 + kOffStage<D> +
         (RowGeo<D>::kQTmem ? kSoftWarps * 32 * RowGeo<D>::kStageRow + 128 * sizeof(float2) : 0);
}

// One block's piece of a unit: token tiles [kt0, kt1) for query rows row0 ...
struct Seg {
  bool pre;
  int b, hk, row0, n_rows, ctx, kt0, kt1, tiles, part;
  const int32_t* pages;
};

// Walks a block's share [g, end) of the tiles of all units.
struct Walk {
  int g, end;
  __device__ explicit Walk(const AttnArgs& a) {
    const int total = a.pre_units * a.pre_T + a.own_units * a.own_T;
    g = blockIdx.x * a.share;
    end = min(g + a.share, total);
  }
  // The next piece with any work; false at the end.
  __device__ bool next(const AttnArgs& a, Seg& s, bool report) {
    const int pre_total = a.pre_units * a.pre_T;
    while (g < end) {
      int base, T;
      if (g < pre_total) {
        const int u = g / a.pre_T;
        s.pre = true;
        T = a.pre_T;
        base = u * T;
        s.hk = u / a.pre_row_tiles;
        s.b = 0;
        s.row0 = u % a.pre_row_tiles * a.unit_rows;
        s.n_rows = a.B * a.nq * a.G;
        s.ctx = a.prefix_len;
        s.pages = a.prefix_table;
      } else {
        const int u = (g - pre_total) / a.own_T;
        s.pre = false;
        T = a.own_T;
        base = pre_total + u * T;
        const int place = u % a.own_row_tiles, bh = u / a.own_row_tiles;
        s.hk = bh % a.c.Hkv;
        s.b = bh / a.c.Hkv;
        s.row0 = unit_tile(place, a.own_row_tiles) * a.unit_rows;
        s.n_rows = a.nq * a.G;
        s.ctx = context_len(a, s.b, report && s.hk == 0 && place == 0);
        s.pages = a.table + static_cast<int64_t>(s.b) * a.table_stride;
      }
      const int last = min(s.row0 + a.unit_rows, s.n_rows) - 1;
      const int seen = s.pre ? s.ctx : own_limit(a, s.ctx, last);
      s.tiles = (seen + a.row_tile - 1) / a.row_tile;
      s.kt0 = g - base;
      const int stop = min(end, base + T);
      s.kt1 = min(stop - base, s.tiles);
      s.part = static_cast<int>(blockIdx.x) - base / a.share;
      g = stop;
      if (s.kt1 > s.kt0) return true;
    }
    return false;
  }
  __device__ static int seen(const AttnArgs& a, const Seg& s) {
    const int last = min(s.row0 + a.unit_rows, s.n_rows) - 1;
    return s.pre ? s.ctx : own_limit(a, s.ctx, last);
  }
};

// A bounded wait: after the first that runs out, none waits again.
struct Waiter {
  Ctl* ctl;
  int32_t* err;
  uint64_t limit;
  bool ok;
  __device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity) {
    if (!ok) return;
    if (mbar_wait(bar, parity, &ctl->abort, limit)) return;
    ok = false;
    if (atomicExch(&ctl->abort, 1) == 0) atomicOr(err, MOE_DEVERR_PIPE_TIMEOUT);
  }
};

// Instruction descriptor, kind::f16: fp16 A and B, fp32 D, both K-major, M = 128.
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t N) {
  return (1u << 4) | ((N >> 3) << 17) | ((128u >> 4) << 24);
}
constexpr uint32_t kBothBf16 = 1u << 7 | 1u << 10;     // added: bf16 A and B

// 64 of the reduction (4 steps of 16), issued by one elected lane: A and B in shared memory.
__device__ __forceinline__ void mma_ss_chunk(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\t"
      ".reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
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

// The same for 128 of the reduction: second operands at a + a_step and b + b_step.
__device__ __forceinline__ void mma_ss_pair(uint32_t d, uint64_t a, uint64_t b, uint64_t a_step,
                                            uint64_t b_step, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\t"
      ".reg .b64 a1, a2, a3, b1, b2, b3, c0, c1, c2, c3, f0, f1, f2, f3;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "add.u64 a1, %1, 2;\n\tadd.u64 a2, %1, 4;\n\tadd.u64 a3, %1, 6;\n\t"
      "add.u64 b1, %2, 2;\n\tadd.u64 b2, %2, 4;\n\tadd.u64 b3, %2, 6;\n\t"
      "add.u64 c0, %1, %3;\n\tadd.u64 f0, %2, %4;\n\t"
      "add.u64 c1, c0, 2;\n\tadd.u64 c2, c0, 4;\n\tadd.u64 c3, c0, 6;\n\t"
      "add.u64 f1, f0, 2;\n\tadd.u64 f2, f0, 4;\n\tadd.u64 f3, f0, 6;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %5, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %5, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %5, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %5, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], c0, f0, %5, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], c1, f1, %5, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], c2, f2, %5, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], c3, f3, %5, 1;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "l"(a_step), "l"(b_step), "r"(idesc), "r"(accumulate)
      : "memory");
}

// tcgen05.st: 32 lanes x 32-bit, 8 consecutive columns per thread.
__device__ __forceinline__ void tmem_st_32x32b_x8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
      : "memory");
}

// Of a word (scale and bias): whether both are finite; an exponent field above all magnitudes
// of its group, times 128 (that of 2^(BITS - 126) for zeros and subnormal scales).
__device__ __forceinline__ bool finite_word(uint32_t word) {
  return (((word & 0x7F807F80u) + 0x00800080u) & 0x80008000u) == 0;
}
__device__ __forceinline__ bool zero_word(uint32_t word) { return (word & 0x7FFF7FFFu) == 0; }
template <int BITS>
__device__ __forceinline__ uint32_t group_field(uint32_t word) {
  const uint32_t u = word & 0x7F807F80u;
  return max((u & 0xFFFFu) + (BITS << 7), u >> 16);
}
__device__ __forceinline__ float pow2_field(uint32_t e) { return __uint_as_float(e << 23); }

__device__ __forceinline__ void st_shared_v4(uint32_t at, uint32_t x, uint32_t y, uint32_t z,
                                             uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void unpack_f32x2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// -------------------------------------------------- pages of the tiles ahead

// One warp turns page numbers into the offsets of each tile's 16-token blocks, up to
// three tiles ahead of the products.
template <int D, int BITS>
struct Pages {
  using G = RowGeo<D>;
  static constexpr int J = G::J, TT = G::TT;
  static constexpr int RB = D * BITS / 8;
  const AttnArgs& a;
  Ctl& ctl;
  int lane;

  __device__ void run(const Seg& sg, int seen, uint32_t& tc, Waiter& w) {
    int tok = sg.kt0 * TT + 16 * lane;               // lane i has block i of a tile
    const auto look = [&](int t, int& page, uint32_t& in_page) {
      const uint32_t blk = static_cast<uint32_t>(t) >> 4;
      const uint32_t at = page_of_block(a.c, blk);
      in_page = blk - at * a.c.page_blocks;
      page = lane < TT / 16 && t < seen ? __ldg(sg.pages + at) : -1;
    };
    int page, next;
    uint32_t in_page, next_in;
    look(tok, page, in_page);
    for (int it = sg.kt0; it < sg.kt1; ++it, ++tc, tok += TT) {
      const int slot = tc % kMetaRing;
      look(tok + TT, next, next_in);
      if (tc >= kMetaRing) w.wait(&ctl.done[slot], (tc / kMetaRing - 1) & 1);
      if (lane < TT / 16) {
        int64_t off = 0;
        int wd = -1;
        if (page >= 0 && page < a.c.pages) {
          off = page * a.c.page_bytes + static_cast<int64_t>(sg.hk) * a.c.head_bytes +
                in_page * (16 * RB);
          wd = a.c.code_bytes + static_cast<int>(in_page) * (16 * J * 4 - 16 * RB);
        } else if (tok < seen) {
          atomicOr(a.c.err, MOE_DEVERR_BAD_PAGE);
        }
        ctl.base[slot][lane] = off;
        ctl.words[slot][lane] = wd;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.base_full[slot]);
      page = next;
      in_page = next_in;
    }
  }
};

// -------------------------------------------------------- codes to operands

template <int D, int BITS>
struct Converter {
  using G = RowGeo<D>;
  static constexpr int RB = D * BITS / 8;
  static constexpr int TT = G::TT;
  static constexpr int PR = D / 16;                  // 16-code pieces of a row
  static constexpr int KU = TT * PR / G::kConvThreads;    // key pieces per thread and tile
  static constexpr int VU = TT * D / 64 / G::kConvThreads;   // value pieces (8 tokens x 8 elements)
  static constexpr int KW = BITS / 2;                // words of a key piece (16 codes)
  static constexpr int J = G::J;
  // runs of 32 tokens, keys and values, per warp and tile (with fewer runs than warps the
  // last warps have none)
  static constexpr int kRuns = 2 * TT / 32;
  static constexpr int WU = kRuns > G::kConvWarps ? kRuns / G::kConvWarps : 1;

  const AttnArgs& a;
  Ctl& ctl;
  Meta<D>* metas;
  uint8_t* smem;
  int cw, lane;
  uint32_t units;                                    // of the piece's value groups, 8 bits each
  uint32_t words[WU][J];
  uint32_t kr[KU][KW];
  uint32_t vr[VU][8][BITS / 4];

  // Run i of this warp: tokens 32 r + lane of the keys (kv = 0) or of the values.
  __device__ __forceinline__ bool run_of(int i, int& kv, int& r) const {
    const int id = cw + G::kConvWarps * i;
    kv = id / (TT / 32);
    r = id % (TT / 32);
    return id < kRuns;
  }
  __device__ void load_words(int slot) {
#pragma unroll
    for (int i = 0; i < WU; ++i) {
      int kv, r;
      if (!run_of(i, kv, r)) return;
      const int tk = 32 * r + lane;
      const uint8_t* p = a.c.data + ctl.base[slot][tk >> 4] + max(ctl.words[slot][tk >> 4], 0) +
                         (tk & 15) * (J * 4);
      if (kv) p += static_cast<int64_t>(a.c.Hkv) * a.c.head_bytes;
      if constexpr (J == 1) {
        words[i][0] = ld_nc_u32(p);
      } else if constexpr (J == 2) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
        words[i][0] = v.x, words[i][1] = v.y;
      } else {
        const uint4 v = ld_nc_v4(p);
        words[i][0] = v.x, words[i][1] = v.y, words[i][2] = v.z, words[i][3] = v.w;
      }
    }
  }
  // The divisors of a piece's value groups from its first tile (`n` seen tokens): the least of
  // the runs' largest values, so that neither a few large nor a few small tokens decide.
  __device__ void find_units(int slot, int n, uint32_t parity) {
#pragma unroll
    for (int i = 0; i < WU; ++i) {
      int kv, r;
      if (!run_of(i, kv, r) || kv == 0) continue;
      const int tk = 32 * r + lane;
      const bool ok = tk < n && ctl.words[slot][tk >> 4] >= 0;
      uint32_t all = 0;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const bool use = ok && finite_word(words[i][j]) && !zero_word(words[i][j]);
        const uint32_t e = use ? group_field<BITS>(words[i][j]) >> 7 : 0u;
        all |= min(__reduce_max_sync(kAll, e), 255u) << (8 * j);
      }
      if (lane == 0) ctl.run_top[parity][r] = all;
    }
    named_bar_sync(4, G::kConvThreads);
    units = 0;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      uint32_t low = 255u;
#pragma unroll
      for (int r = 0; r < TT / 32; ++r) {
        const uint32_t e = ctl.run_top[parity][r] >> (8 * j) & 255u;
        if (e) low = min(low, e);
      }
      if (low == 255u) low = 127u;                   // (no values but 0)
      units |= min(low + kAbove<BITS>, 248u) << (8 * j);
    }
  }

  // Exponents, scales and biases of a tile of `n` seen tokens from the loaded words.
  __device__ void put_meta(Meta<D>& m, int slot, int n) const {
#pragma unroll
    for (int i = 0; i < WU; ++i) {
      int kv, r;
      if (!run_of(i, kv, r)) return;
      const int tk = 32 * r + lane;
      const bool ok = tk < n && ctl.words[slot][tk >> 4] >= 0;
      const bool dead = tk < n && !ok;               // a page outside the cache would hold it
      uint32_t bad = 0;
      if (kv == 0) {
        uint32_t big = 0;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          if (ok && !finite_word(words[i][j]))
            bad |= 1u << j;
          else if (ok && !zero_word(words[i][j]))
            big = max(big, group_field<BITS>(words[i][j]) >> 7);
        }
        const uint32_t top = __reduce_max_sync(kAll, big);
        const uint32_t low = __reduce_min_sync(kAll, big ? big : 255u);
        const bool slow = __any_sync(kAll, dead) || top > low + kMaxSpread;
        const uint32_t E = top == 0 ? 127u : min(top, 253u);
        const uint32_t eu = slow && big ? min(big, 253u) : E;
        constexpr float kRoom = 1 << kKeyRoom<BITS>;
        const float down = pow2_field(254u - eu) * (1.f / kRoom);
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const bool nan = bad >> j & 1;
          // (down may be 2^124: its product with 2^24 is no float)
          const float s = ok && !nan ? bf16_lo(words[i][j]) * down * 0x1p24f : 0.f;
          const float b = ok && !nan ? bf16_hi(words[i][j]) * down : 0.f;
          m.ksb[j][tk] = nan ? 0x7E000000u : pack_f16(s, b);      // a NaN key: NaN logits
        }
        m.kf[tk] = pow2_field(eu) * kRoom;
        if (lane == 0) m.run_kf[r] = pow2_field(E) * kRoom;
        if (lane == 0) m.slow[0][r] = slow;
      } else {
        bool out = false;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const uint32_t unit = units >> (8 * j) & 255u;
          uint32_t word = ok ? words[i][j] : 0u;
          if (!finite_word(word)) bad |= 1u << j, word = 0u;
          // (unsigned: too small, or above the unit)
          out |= !zero_word(word) && (unit << 7) - group_field<BITS>(word) > kWindow<BITS> << 7;
          const float down = pow2_field(254u - kValueRoom<BITS> - unit);
          const uint32_t sb = pack_f16(bf16_lo(word) * down * 0x1p24f, bf16_hi(word) * down);
          m.vs[j][tk] = static_cast<uint16_t>(sb);
          m.vb[j][tk] = static_cast<uint16_t>(sb >> 16);
        }
        m.flag[tk] = static_cast<uint8_t>(bad | (dead ? kDead : 0));
        const bool slow = __any_sync(kAll, bad != 0 || dead);
        const bool wide = __any_sync(kAll, out);
        if (lane == 0) {
          m.slow[1][r] = slow;
          m.wide[r] = wide;
          m.units = units;
        }
      }
    }
  }

  // Key piece u of a lane: 16 codes (group j, quarter of it) of token row. The rows of a
  // piece are RU, of a warp RW = KU * RU (8, 16 or 32); lanes are laid out so that the eight
  // lanes of a shared-memory store hit every bank once.
  static constexpr int RU = 32 / PR, RW = KU * RU;
  static constexpr int RB16 = RW < 16 ? RW : 16;         // of one 16-token block
  __device__ __forceinline__ int key_row() const {       // of piece 0, within the warp's rows
    return D == 64 ? lane >> 2 : D == 128 ? (lane >> 2 & 1) | (lane >> 3 & 2) : lane >> 2 & 1;
  }
  __device__ __forceinline__ int key_group() const {
    return D == 64 ? 0 : D == 128 ? lane >> 3 & 1 : lane >> 3;
  }
  __device__ void load_keys(int slot) {
    const int in_row = key_group() * (4 * 2 * BITS) + (lane & 3) * (2 * BITS);
#pragma unroll
    for (int b = 0; b < RW / RB16; ++b) {
      const uint8_t* p = a.c.data + ctl.base[slot][(cw * RW >> 4) + b] +
                         ((cw * RW & 15) + key_row()) * RB + in_row;
#pragma unroll
      for (int i = 0; i < RB16 / RU; ++i) {
        uint32_t(&k)[KW] = kr[b * (RB16 / RU) + i];
        if constexpr (BITS == 8) {
          const uint4 v = ld_nc_v4(p + i * RU * RB);
          k[0] = v.x, k[1] = v.y, k[2] = v.z, k[3] = v.w;
        } else {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(p + i * RU * RB));
          k[0] = v.x, k[1] = v.y;
        }
      }
    }
  }

  // Value piece u: tokens 64 th + 8 (lane % 8) .. of elements d0 + u * kPieceD ..; th is the
  // same for all pieces of a warp.
  static constexpr int TH = TT / 64;
  static constexpr int kPieceD = G::kConvWarps / TH * 32;
  __device__ __forceinline__ int value_half() const { return cw % TH; }
  __device__ __forceinline__ int value_d0() const { return cw / TH * 32 + (lane >> 3) * 8; }
  __device__ void load_values(int slot) {
    const int t0 = value_half() * 64 + (lane & 7) * 8;
    const uint8_t* p = a.c.data + ctl.base[slot][t0 >> 4] +
                       static_cast<int64_t>(a.c.Hkv) * a.c.head_bytes + (t0 & 15) * RB +
                       value_d0() * BITS / 8;
#pragma unroll
    for (int u = 0; u < VU; ++u) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if constexpr (BITS == 8) {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(p + k * RB + u * kPieceD));
          vr[u][k][0] = v.x, vr[u][k][1] = v.y;
        } else {
          vr[u][k][0] = ld_nc_u32(p + k * RB + u * (kPieceD / 2));
        }
      }
    }
  }

  // Keys: 16 codes of a token -> two 16-byte chunks of its row. 4-bit chunks hold
  // elements 0 4 1 5 2 6 3 7 (as they come out of a word); the queries' do too.
  __device__ void put_keys(const Meta<D>& m, uint32_t off) const {
    const int j = key_group(), row = cw * RW + key_row();
    const uint32_t dst = smem_u32(smem) + off + j * (TT * 128) + row * 128 +
                         (((lane & 3) * 2 ^ (row & 7)) << 4);
#pragma unroll
    for (int u = 0; u < KU; ++u) {
      const uint32_t sb = m.ksb[j][row + u * RU];
      const uint32_t s2 = prmt(sb, sb, 0x1010), b2 = prmt(sb, sb, 0x3232);
      uint32_t r[8];
      if constexpr (BITS == 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          r[2 * i] = fma_f16x2(s2, prmt(kr[u][i], 0u, 0x4140), b2);
          r[2 * i + 1] = fma_f16x2(s2, prmt(kr[u][i], 0u, 0x4342), b2);
        }
      } else {
        const uint32_t s16 = fma_f16x2(s2, 0x2C002C00u, 0u);      // scale / 16
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w = i & 1 ? kr[u][i >> 1] >> 8 : kr[u][i >> 1];
          r[2 * i] = fma_f16x2(s2, w & 0x000F000Fu, b2);
          r[2 * i + 1] = fma_f16x2(s16, w & 0x00F000F0u, b2);
        }
      }
      const uint32_t at = (dst ^ ((u * RU & 7) << 4)) + u * RU * 128;
      st_shared_v4(at, r[0], r[1], r[2], r[3]);
      st_shared_v4(at ^ 16u, r[4], r[5], r[6], r[7]);
    }
  }

  // Values, transposed: 8 tokens x 8 elements -> one 16-byte chunk in each of 8 rows.
  __device__ void put_values(const Meta<D>& m, uint32_t off) const {
    const int th = value_half(), tg = lane & 7;
    const uint32_t dst0 = smem_u32(smem) + off + th * (D * 128) + value_d0() * 128 + (tg << 4);
#pragma unroll
    for (int u = 0; u < VU; ++u) {
      const int j = (value_d0() + u * kPieceD) / kKvGroup;
      const uint4 sv = *reinterpret_cast<const uint4*>(&m.vs[j][th * 64 + tg * 8]);
      const uint4 bv = *reinterpret_cast<const uint4*>(&m.vb[j][th * 64 + tg * 8]);
      const uint32_t s[4] = {sv.x, sv.y, sv.z, sv.w}, b[4] = {bv.x, bv.y, bv.z, bv.w};
      const uint32_t dst = dst0 + u * (kPieceD * 128);
#pragma unroll
      for (int h = 0; h < 2; ++h) {                 // elements 4h .. 4h + 3
        uint32_t r[4][4];                           // [element][token pair]
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          if constexpr (BITS == 8) {
            const uint32_t x = vr[u][2 * p][h], y = vr[u][2 * p + 1][h];
            const uint32_t lo = prmt(x, y, 0x5140), hi = prmt(x, y, 0x7362);
            r[0][p] = fma_f16x2(s[p], prmt(lo, 0u, 0x4140), b[p]);
            r[1][p] = fma_f16x2(s[p], prmt(lo, 0u, 0x4342), b[p]);
            r[2][p] = fma_f16x2(s[p], prmt(hi, 0u, 0x4140), b[p]);
            r[3][p] = fma_f16x2(s[p], prmt(hi, 0u, 0x4342), b[p]);
          } else {
            const uint32_t v = prmt(vr[u][2 * p][0], vr[u][2 * p + 1][0], h ? 0x7632 : 0x5410);
            const uint32_t s16 = fma_f16x2(s[p], 0x2C002C00u, 0u);
            r[0][p] = fma_f16x2(s[p], v & 0x000F000Fu, b[p]);
            r[1][p] = fma_f16x2(s16, v & 0x00F000F0u, b[p]);
            r[2][p] = fma_f16x2(s[p], v >> 8 & 0x000F000Fu, b[p]);
            r[3][p] = fma_f16x2(s16, v >> 8 & 0x00F000F0u, b[p]);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = 4 * h + i;
          st_shared_v4((dst ^ (row << 4)) + row * 128, r[i][0], r[i][1], r[i][2], r[i][3]);
        }
      }
    }
  }

  // The same as bf16 from the cache, of a tile of `n` seen tokens. Seldom: not inlined, and
  // nothing is taken from the caller's registers, so that it costs the loop few of them.
  static __device__ __noinline__ void put_wide_values(uint8_t* smem, uint32_t tile, int slot, int n) {
    const Ctl& ctl = *reinterpret_cast<const Ctl*>(smem + G::kOffMeta + kMetaRing * sizeof(Meta<D>));
    const uint32_t units = reinterpret_cast<const Meta<D>*>(smem + G::kOffMeta)[slot].units;
    const int cw = conv_index(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int th = cw % TH, tg = lane & 7, d0 = cw / TH * 32 + (lane >> 3) * 8;
    const int t0 = th * 64 + tg * 8;
    const int to_words = ctl.words[slot][t0 >> 4];
    const uint8_t* block = ctl.values + ctl.base[slot][t0 >> 4];
#pragma unroll 1
    for (int u = 0; u < VU; ++u) {
      const int d = d0 + u * kPieceD, j = d / kKvGroup;
      const float down = pow2_field(254u - kValueRoom<BITS> - (units >> (8 * j) & 255u));
      const uint32_t dst = smem_u32(smem) + tile + th * (D * 128) + d * 128 + (tg << 4);
#pragma unroll 1
      for (int i = 0; i < 8; ++i) {
        uint32_t r[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float v[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int t = (t0 & 15) + 2 * k + x;
            uint32_t word = 0;
            if (to_words >= 0 && t0 + 2 * k + x < n)
              word = __ldg(reinterpret_cast<const uint32_t*>(block + to_words + t * (J * 4)) + j);
            if (!finite_word(word)) word = 0;
            const uint32_t byte = __ldg(block + t * RB + (d + i) * BITS / 8);
            const uint32_t code = BITS == 8 ? byte : byte >> (i & 1) * 4 & 15u;
            v[x] = fmaf(bf16_lo(word), static_cast<float>(code), bf16_hi(word)) * down;
          }
          r[k] = pack_bf16(v[0], v[1]);
        }
        st_shared_v4((dst ^ (i << 4)) + i * 128, r[0], r[1], r[2], r[3]);
      }
    }
  }

  // All tiles of one piece; `tc` counts this block's tiles. What a tile needs from memory
  // is requested as soon as its registers are free, half a tile and more ahead, and its
  // scales are ready before its keys are: no warp waits for another inside a tile.
  __device__ void run(const Seg& sg, int seen, uint32_t& tc, uint32_t piece, Waiter& w) {
    const auto pages_of = [&](uint32_t t) {
      w.wait(&ctl.base_full[t % kMetaRing], (t / kMetaRing) & 1);
    };
    const auto scales_for = [&](uint32_t t, int it) {   // (the ring slot was tile t - 4's)
      if (t >= kMetaRing) w.wait(&ctl.done[t % kMetaRing], (t / kMetaRing - 1) & 1);
      put_meta(metas[t % kMetaRing], t % kMetaRing, min(seen - it * TT, TT));
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.meta_full[t % kMetaRing]);
    };
    pages_of(tc);
    load_words(tc % kMetaRing);
    load_keys(tc % kMetaRing);
    load_values(tc % kMetaRing);
    find_units(tc % kMetaRing, min(seen - sg.kt0 * TT, TT), piece & 1);
    scales_for(tc, sg.kt0);
    if (sg.kt0 + 1 < sg.kt1) {
      pages_of(tc + 1);
      load_words((tc + 1) % kMetaRing);
    }
    for (int it = sg.kt0; it < sg.kt1; ++it, ++tc) {
      const int st = tc % G::KS;
      const Meta<D>& m = metas[tc % kMetaRing];
      w.wait(&ctl.meta_full[tc % kMetaRing], (tc / kMetaRing) & 1);
      if (tc >= G::KS) w.wait(&ctl.k_empty[st], (tc / G::KS - 1) & 1);
      put_keys(m, G::kOffK + st * G::kTileBytes);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.k_full[st]);
      if (it + 1 < sg.kt1) {
        load_keys((tc + 1) % kMetaRing);
        scales_for(tc + 1, it + 1);
        if (it + 2 < sg.kt1) {
          pages_of(tc + 2);
          load_words((tc + 2) % kMetaRing);
        }
      }
      if (tc >= G::KS) w.wait(&ctl.done[(tc - G::KS) % kMetaRing], ((tc - G::KS) / kMetaRing) & 1);
      if (is_wide(m))
        put_wide_values(smem, G::kOffV + st * G::kTileBytes, tc % kMetaRing, min(seen - it * TT, TT));
      else
        put_values(m, G::kOffV + st * G::kTileBytes);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.v_full[st]);
      if (it + 1 < sg.kt1) load_values((tc + 1) % kMetaRing);
    }
  }
};

// ------------------------------------------------------------------ softmax

template <int D, int BITS>
struct Softmax {
  using G = RowGeo<D>;
  const AttnArgs& a;
  Ctl& ctl;
  Meta<D>* metas;
  uint8_t* smem;
  uint32_t tmem;             // + lane quarter
  int wg, warp, lane;
  float m, l;                // reference of the logits (log2), sum
  float c;                   // scale2 * 2^(row exponent)
  uint32_t nan;              // value groups that are NaN for this row
  uint32_t units;            // divisors of the value groups

  // This warp's staging: 32 rows of SB bytes, 16-byte pieces permuted by their row, for
  // turning between a thread's own row and neighbouring lanes on one row (which memory
  // wants). Queries in shared memory lend it after their last product.
  static constexpr int SB = G::kStageRow;
  static constexpr int PC = SB / 16;              // pieces of a row,
  static constexpr int RL = 32 / PC;              // rows of a warp's access
  __device__ __forceinline__ uint8_t* stage() const {
    return smem + (G::kQTmem ? kOffStage<D> + warp * (32 * SB) : wg * G::kQBytes + (warp & 3) * (32 * SB));
  }
  static __device__ __forceinline__ int piece(int row, int k) {
    return row * SB + ((k ^ (SB == 128 ? row & 7 : row >> 1 & 3)) << 4);
  }

  // The rows' queries, each divided by the power of two under its largest element, as
  // fp16 in the key tiles' element order. `qp` is the thread's own row; lanes read
  // neighbouring pieces of a row. (D = 256: each warpgroup prepares half of the elements.)
  __device__ void load_query(const uint16_t* qp, bool live) {
    const uint32_t lives = __ballot_sync(kAll, live);
    const uint64_t base = reinterpret_cast<uint64_t>(qp);
    const auto at = [&](int row) { return reinterpret_cast<const uint8_t*>(__shfl_sync(kAll, base, row)); };
    // largest magnitude: bf16 bits without their sign order like the numbers
    constexpr int LW = D / 64;                    // words of a row per lane
    uint32_t mx = 0;
#pragma unroll 1
    for (int r0 = 0; r0 < 32; r0 += 8) {
      uint32_t w[8][LW];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const uint8_t* q = at(r0 + u) + lane * (4 * LW);
#pragma unroll
        for (int k = 0; k < LW; ++k) w[u][k] = 0;
        if (lives >> (r0 + u) & 1) {
          if constexpr (LW == 1) {
            w[u][0] = ld_nc_u32(q);
          } else if constexpr (LW == 2) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(q));
            w[u][0] = v.x, w[u][1] = v.y;
          } else {
            const uint4 v = ld_nc_v4(q);
            w[u][0] = v.x, w[u][1] = v.y, w[u][2] = v.z, w[u][3] = v.w;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        uint32_t x = w[u][0] & 0x7FFF7FFFu;
#pragma unroll
        for (int k = 1; k < LW; ++k) x = max_u16x2(x, w[u][k] & 0x7FFF7FFFu);
        x = __reduce_max_sync(kAll, max(x >> 16, x & 0xFFFFu));
        if (lane == r0 + u) mx = x;
      }
    }
    const uint32_t e = min(max(mx >> 7, 1u), 253u);
    const float down = pow2_field(254u - e);
    c = a.scale2 * pow2_field(e);
    constexpr int kChunks = D / 8 / PC, kMine = G::kQTmem ? kChunks / 2 : kChunks;
    constexpr int kBatch = 8 / PC;                // chunks of PC pieces loaded together
    const int first = G::kQTmem ? wg * kMine : 0;
#pragma unroll 1
    for (int j0 = first; j0 < first + kMine; j0 += kBatch) {
      uint4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int row = u % PC * RL + lane / PC;
        const uint4* q = reinterpret_cast<const uint4*>(at(row)) + (j0 + u / PC) * PC + lane % PC;
        v[u] = make_uint4(0, 0, 0, 0);
        if (lives >> row & 1) v[u] = __ldg(q);
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        uint8_t* dst = stage() + (G::kQTmem ? 0 : j0 * 16384);
#pragma unroll
        for (int u = 0; u < PC; ++u) {
          const uint4 x4 = v[b * PC + u];
          const int row = u * RL + lane / PC;
          const float f = __shfl_sync(kAll, down, row);
          const float x[8] = {bf16_lo(x4.x) * f, bf16_hi(x4.x) * f, bf16_lo(x4.y) * f, bf16_hi(x4.y) * f,
                              bf16_lo(x4.z) * f, bf16_hi(x4.z) * f, bf16_lo(x4.w) * f, bf16_hi(x4.w) * f};
          *reinterpret_cast<uint4*>(dst + piece(row, lane % PC)) =
              BITS == 8 ? make_uint4(pack_f16(x[0], x[1]), pack_f16(x[2], x[3]), pack_f16(x[4], x[5]),
                                     pack_f16(x[6], x[7]))
                        : make_uint4(pack_f16(x[0], x[4]), pack_f16(x[1], x[5]), pack_f16(x[2], x[6]),
                                     pack_f16(x[3], x[7]));
        }
        if constexpr (G::kQTmem) {
          __syncwarp();
          uint32_t q[4 * PC];
#pragma unroll
          for (int k = 0; k < PC; ++k) {
            const uint4 x4 = *reinterpret_cast<const uint4*>(dst + piece(lane, k));
            q[4 * k] = x4.x, q[4 * k + 1] = x4.y, q[4 * k + 2] = x4.z, q[4 * k + 3] = x4.w;
          }
          tmem_st_32x32b_x16(tmem + G::kColQ + 16 * (j0 + b), q);
          __syncwarp();
        }
      }
    }
    if (G::kQTmem) tmem_st_wait();
  }

  // This thread's row of O times `up` and the groups' units (NaN for the groups in
  // `nan_groups`) to memory at element `dst`, as the output or as a partial result. (D = 256: each warpgroup half of it.)
  __device__ void store(int64_t dst, bool live, bool output, float up, uint32_t nan_groups,
                        uint32_t group_units) {
    constexpr int kCols = SB / 4, kChunks = D / kCols, kMine = G::kQTmem ? kChunks / 2 : kChunks;
    const int first = G::kQTmem ? wg * kMine : 0;
    const uint32_t lives = __ballot_sync(kAll, live);
    uint8_t* st = stage();
#pragma unroll 1
    for (int h = first; h < first + kMine; ++h) {
      const int j = h * kCols / kKvGroup;
      const float unit = pow2_field((group_units >> (8 * j) & 255u) + kValueRoom<BITS>);
      const float f = nan_groups >> j & 1 ? NAN : up * unit;
#pragma unroll
      for (int k = 0; k < PC / 4; ++k) {
        uint32_t v[16];
        tmem_ld_32x32b_x16(tmem + G::kColO + (G::kQTmem ? 0 : wg * D) + kCols * h + 16 * k, v);
        tmem_ld_wait();
        tmem_regs_ready(v);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<float4*>(st + piece(lane, 4 * k + i)) =
              make_float4(__uint_as_float(v[4 * i]) * f, __uint_as_float(v[4 * i + 1]) * f,
                          __uint_as_float(v[4 * i + 2]) * f, __uint_as_float(v[4 * i + 3]) * f);
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < PC; ++i) {
        const int row = RL * i + lane / PC;
        const int64_t to = __shfl_sync(kAll, dst, row) + kCols * h + lane % PC * 4;
        const float4 y = *reinterpret_cast<const float4*>(st + piece(row, lane % PC));
        if (lives >> row & 1) {
          if (output)
            *reinterpret_cast<uint2*>(a.out + to) = make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
          else
            *reinterpret_cast<float4*>(a.part + to) = y;
        }
      }
      __syncwarp();
    }
  }

  // Logit (log2 units) of column k of a tile; -inf where the row does not see it.
  template <bool SLOW, bool MASK>
  __device__ __forceinline__ float logit(float s, float ck, const Meta<D>& t, int k, int lim) const {
    float x = SLOW ? s * (c * t.kf[k]) : s * ck;
    if (MASK && k >= lim) x = -INFINITY;
    if (SLOW && (t.flag[k] & kDead)) x = -INFINITY;
    return x;
  }

  // Weights of columns 64 H .. 64 H + 63 (runs 2H and 2H + 1, each with its factor) into
  // registers, and the runs' sums. The next 16 logits are on their way out of
  // tensor memory while these are worked on.
  template <bool MASK, int H>
  __device__ __forceinline__ void weights(uint32_t s_col, const float (&ck)[2], float off,
                                          int lim, uint32_t (&p)[32], float (&sum)[2]) {
    uint32_t v[2][16];
    tmem_ld_32x32b_x16(tmem + s_col + 64 * H, v[0]);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint64_t ck2 = pack_f32x2(ck[r], ck[r]), off2 = pack_f32x2(off, off);
      uint64_t part[2] = {0, 0};
#pragma unroll
      for (int h = 2 * r; h < 2 * r + 2; ++h) {
        uint32_t(&u)[16] = v[h & 1];
        tmem_ld_wait();
        tmem_regs_ready(u);
        if (h < 3) tmem_ld_32x32b_x16(tmem + s_col + 64 * H + 16 * (h + 1), v[(h + 1) & 1]);
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const int col = 64 * H + 16 * h + i;
          float x0, x1;
          unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(u[i]), __uint_as_float(u[i + 1])), ck2, off2),
                       x0, x1);
          if (MASK && col >= lim) x0 = -INFINITY;
          if (MASK && col + 1 >= lim) x1 = -INFINITY;
          const float w0 = exp2_approx(x0), w1 = exp2_approx(x1);
          part[(i >> 1) & 1] = add_f32x2(part[(i >> 1) & 1], pack_f32x2(w0, w1));
          p[8 * h + i / 2] = pack_f16(w0, w1);
        }
      }
      float s0, s1;
      unpack_f32x2(add_f32x2(part[0], part[1]), s0, s1);
      sum[r] = s0 + s1;
    }
  }

  // Moves m to the largest logit of columns 16 H0 .. (in the lanes that `need` it), and l, O
  // and the tile's weights already written (columns below 16 H0) along with it.
  template <bool SLOW, bool MASK, int H0>
  __device__ __forceinline__ void move(uint32_t s_col, const Meta<D>& t, int lim, bool need, bool first,
                                       uint64_t* pv, uint32_t pv_parity, Waiter& w) {
    float mx = -INFINITY;
#pragma unroll 1
    for (int h = H0; h < G::TT / 16; ++h) {
      uint32_t v[16];
      tmem_ld_32x32b_x16(tmem + s_col + 16 * h, v);
      tmem_ld_wait();
      tmem_regs_ready(v);
      const float ck = c * t.run_kf[h >> 1];
#pragma unroll
      for (int i = 0; i < 16; ++i)
        mx = fmaxf(mx, logit<SLOW, MASK>(__uint_as_float(v[i]), ck, t, 16 * h + i, lim));
    }
    float fo = 1.f;
    if (need && mx > m) {
      fo = exp2_approx(m - mx);                     // (0 from -inf on)
      l *= fo;
      m = mx;
    }
    if (!__any_sync(kAll, fo != 1.f)) return;
    if (H0 > 0) {
      const uint32_t f2 = pack_f16(fo, fo);
#pragma unroll 1
      for (int h = 0; h < H0 / 2; ++h) {
        uint32_t v[16];
        tmem_ld_32x32b_x16(tmem + s_col + 16 * h, v);
        tmem_ld_wait();
        tmem_regs_ready(v);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = fma_f16x2(v[i], f2, 0u);
        tmem_st_32x32b_x16(tmem + s_col + 16 * h, v);
      }
      tmem_st_wait();
    }
    if (first) return;
    w.wait(pv, pv_parity);                          // the last product into O is done
    tc_fence_after();
    const uint32_t o_col = tmem + G::kColO + wg * D;
#pragma unroll 1
    for (int h = 0; h < D / 16; ++h) {
      uint32_t v[16];
      tmem_ld_32x32b_x16(o_col + 16 * h, v);
      tmem_ld_wait();
      tmem_regs_ready(v);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * fo);
      tmem_st_32x32b_x16(o_col + 16 * h, v);
    }
    tmem_st_wait();
  }

  // Half H of a tile. Its 64 weights are packed into 32 columns that hold logits of
  // half 0, so a tile takes no tensor memory beside its logits.
  template <bool MASK, int H>
  __device__ __forceinline__ void half_tile(uint32_t s_col, const Meta<D>& t, int lim, bool first,
                                            uint64_t* pv, uint32_t pv_parity, Waiter& w) {
    uint32_t p[32];
    const float2 kf = *reinterpret_cast<const float2*>(&t.run_kf[2 * H]);
    float sum[2];
    const float ck[2] = {c * kf.x, c * kf.y};
    bool need = m == -INFINITY && lim > 64 * H;
#pragma unroll 1
    for (int round = 0;; ++round) {
      if (__any_sync(kAll, need)) move<false, MASK, 4 * H>(s_col, t, lim, need, first, pv, pv_parity, w);
      weights<MASK, H>(s_col, ck, m == -INFINITY ? 0.f : -m, lim, p, sum);
      need = fmaxf(sum[0], sum[1]) >= 32768.f;
      if (round || !__any_sync(kAll, need)) break;
    }
    l += sum[0] + sum[1];
    tmem_st_32x32b_x16(tmem + s_col + 32 * H, reinterpret_cast<uint32_t(&)[16]>(p[0]));
    tmem_st_32x32b_x16(tmem + s_col + 32 * H + 16, reinterpret_cast<uint32_t(&)[16]>(p[16]));
    tmem_st_wait();
  }
  template <bool MASK>
  __device__ __forceinline__ void tile(uint32_t s_col, const Meta<D>& t, int lim, bool first,
                                       uint64_t* pv, uint32_t pv_parity, Waiter& w) {
    half_tile<MASK, 0>(s_col, t, lim, first, pv, pv_parity, w);
    if constexpr (G::TT == 128) half_tile<MASK, 1>(s_col, t, lim, first, pv, pv_parity, w);
  }

  // A tile with an exponent per key, NaN groups, missing pages or values outside the window
  // (`wide`: weights as bf16): m always moves to the maximum, so no weight passes 1 and the
  // weights may overwrite the logits that have been read.
  __device__ __forceinline__ void slow_tile(uint32_t s_col, const Meta<D>& t, int lim, bool wide, bool first,
                                            uint64_t* pv, uint32_t pv_parity, Waiter& w) {
    move<true, true, 0>(s_col, t, lim, true, first, pv, pv_parity, w);
    const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll 1
    for (int h = 0; h < G::TT / 16; ++h) {
      uint32_t v[16], p[8];
      tmem_ld_32x32b_x16(tmem + s_col + 16 * h, v);
      tmem_ld_wait();
      tmem_regs_ready(v);
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        float wt[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int col = 16 * h + i + k;
          const float x = logit<true, true>(__uint_as_float(v[i + k]), 0.f, t, col, lim);
          wt[k] = exp2_approx(x - ref);
          l += wt[k];
          if (x != -INFINITY) nan |= t.flag[col];
        }
        p[i / 2] = wide ? pack_bf16(wt[0], wt[1]) : pack_f16(wt[0], wt[1]);
      }
      tmem_st_32x32b_x8(tmem + s_col + 8 * h, p);
    }
    tmem_st_wait();
  }

  // sp: parity of each logit slot's next phase (bit = slot); pc: products into O so far.
  __device__ void run(const Seg& sg, int nqt, uint32_t tc, uint32_t sp, uint32_t pc, Waiter& w) {
    const int r = sg.row0 + (G::kQTmem ? 0 : wg * 128) + (warp & 3) * 32 + lane;
    const bool live = r < sg.n_rows;
    const int qrow = live ? (sg.pre ? r / a.G : sg.b * a.nq + r / a.G) : 0;
    const int head = sg.hk * a.G + (live ? r % a.G : 0);
    load_query(a.q + qrow * a.q_row + head * a.q_head, live);
    if (G::kQTmem)
      tc_fence_before();
    else
      fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl.q_full[G::kQTmem ? 0 : wg]);
    const int nt = sg.kt1 - sg.kt0;
    const bool lone = a.lone && sg.kt0 == 0 && sg.kt1 == sg.tiles;
    const int64_t at = (sg.pre ? 0 : a.own_whole) +
                       static_cast<int64_t>(sg.part) * a.B * a.nq * a.Hq +
                       static_cast<int64_t>(qrow) * a.Hq + head;
    const int64_t dst = lone ? qrow * a.o_row + head * a.o_head : at * D;
    float2* ends = reinterpret_cast<float2*>(smem + kOffStage<D> + kSoftWarps * 32 * SB);
    if (G::kQTmem && wg == 1) {                    // helps with the row's ends only
      named_bar_sync(3, kSoftWarps * 32);
      w.wait(&ctl.pv_done[0], (pc + nt - 1) & 1);
      tc_fence_after();
      const float2 end = ends[(warp & 3) * 32 + lane];
      store(dst, live, lone, end.x, __float_as_uint(end.y), ctl.units);
      tc_fence_before();
      return;
    }
    m = -INFINITY;
    l = 0.f;
    nan = 0;
    units = 0;
    const int lim = !live ? 0 : sg.pre ? sg.ctx : own_limit(a, sg.ctx, r);
    for (int it = 0; it < nt; ++it) {
      const int slot = nqt == 2 ? wg : it & 1;
      const Meta<D>& t = metas[(tc + it) & 3];
      w.wait(&ctl.meta_full[(tc + it) & 3], ((tc + it) >> 2) & 1);
      w.wait(&ctl.s_full[slot], sp >> slot & 1);
      sp ^= 1u << slot;
      tc_fence_after();
      const int rel = lim - (sg.kt0 + it) * G::TT;
      const uint32_t s_col = G::kColS + G::TT * slot;
      const uint32_t pv_parity = (pc + it - 1) & 1;
      uint64_t* pv = &ctl.pv_done[wg];
      if (it == 0) units = t.units;
      const bool wide = is_wide(t);
      if (*reinterpret_cast<const uint64_t*>(t.slow) != 0 || wide)
        slow_tile(s_col, t, rel, wide, it == 0, pv, pv_parity, w);
      else if (__all_sync(kAll, rel >= G::TT))
        tile<false>(s_col, t, rel, it == 0, pv, pv_parity, w);
      else
        tile<true>(s_col, t, rel, it == 0, pv, pv_parity, w);
      // The end waits for the last product; with one query tile the last but one may still
      // run now (these logits were issued before it). A parity tells only neighbouring
      // phases apart, so that one is waited for while the last cannot have been issued.
      if (it > 0 && it == nt - 1) w.wait(pv, pv_parity);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.p_full[slot]);
    }
    // ---- outputs
    w.wait(&ctl.pv_done[wg], (pc + nt - 1) & 1);
    tc_fence_after();
    const float up = !lone ? 1.f : l == 0.f ? 0.f : 1.f / l;
    if (live && !lone) a.ml[at] = make_float2(m, l);
    if (G::kQTmem) {
      ends[(warp & 3) * 32 + lane] = make_float2(up, __uint_as_float(nan));
      if (lane == 0) ctl.units = units;
      named_bar_sync(3, kSoftWarps * 32);
    }
    store(dst, live, lone, up, nan, units);
    tc_fence_before();
  }
};

// ------------------------------------------------------------------- kernel

template <int D, int BITS>
__global__ void __launch_bounds__(RowGeo<D>::kThreads, 1) attn_rows_kernel(const AttnArgs a) {
  using G = RowGeo<D>;
  extern __shared__ uint8_t smem_raw[];
  // (an offset, not a rounded pointer: the compiler keeps seeing shared memory)
  uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
  Meta<D>* metas = reinterpret_cast<Meta<D>*>(smem + G::kOffMeta);
  Ctl& ctl = *reinterpret_cast<Ctl*>(smem + G::kOffMeta + kMetaRing * sizeof(Meta<D>));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 3; ++i) {
      mbar_init(&ctl.k_full[i], G::kConvWarps);
      mbar_init(&ctl.k_empty[i], 1);
      mbar_init(&ctl.v_full[i], G::kConvWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl.q_full[i], G::kQTmem ? 8 : 4);
      mbar_init(&ctl.s_full[i], 1);
      mbar_init(&ctl.p_full[i], 4);
      mbar_init(&ctl.pv_done[i], 1);
    }
    for (int i = 0; i < kMetaRing; ++i) {
      mbar_init(&ctl.base_full[i], 1);
      mbar_init(&ctl.meta_full[i], G::kConvWarps);
      mbar_init(&ctl.done[i], 1);
    }
    mbar_init(&ctl.drain, 1);
    for (int i = 0; i < kMetaRing; ++i)              // (D = 256 has two runs a tile)
      for (int r = 0; r < 4; ++r) metas[i].slow[0][r] = metas[i].slow[1][r] = metas[i].wide[r] = 0;
    ctl.values = a.c.data + static_cast<int64_t>(a.c.Hkv) * a.c.head_bytes;
    ctl.abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    // After a wait that ran out, conversion goes on with what the ring holds: offsets inside
    // the cache, whether or not a tile's pages were found.
    static_assert(kMetaRing * 8 == 32, "a lane each");
    ctl.base[lane / 8][lane % 8] = 0;
    ctl.words[lane / 8][lane % 8] = -1;
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&ctl.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem_base;
  griddep_wait();
  griddep_launch_dependents();
  Waiter w{&ctl, a.c.err, a.timeout_ns, true};

  uint32_t tc = 0;                               // this block's tiles so far
  Walk walk(a);
  Seg sg;
  const auto query_tiles = [](const Seg& g) { return G::QT == 2 && g.row0 + 128 < g.n_rows ? 2 : 1; };
  if (warp < kSoftWarps) {
    Softmax<D, BITS> sm{a, ctl, metas, smem, tmem + ((warp & 3) << 21), warp >> 2, warp, lane};
    uint32_t sp = 0, pc[2] = {0, 0};
    while (walk.next(a, sg, threadIdx.x == 0)) {
      const int nt = sg.kt1 - sg.kt0, nqt = query_tiles(sg);
      if (G::kQTmem || sm.wg < nqt) sm.run(sg, nqt, tc, sp, !G::kQTmem && sm.wg ? pc[1] : pc[0], w);
      // a warpgroup without a query tile may not run ahead: a wait tells only
      // neighbouring phases of its barrier apart
      named_bar_sync(2, kSoftWarps * 32);
      tc += nt;
      sp ^= nqt == 2 ? (nt & 1) * 3 : ((nt + 1) / 2 & 1) | (nt / 2 & 1) << 1;
      pc[0] += nt;
      pc[1] += nqt == 2 ? nt : 0;
    }
  } else if (is_conv_warp(warp) && conv_index(warp) < G::kConvWarps) {
    Converter<D, BITS> cv{a, ctl, metas, smem, conv_index(warp), lane};
    for (uint32_t piece = 0; walk.next(a, sg, false); ++piece)
      cv.run(sg, Walk::seen(a, sg), tc, piece, w);
  } else if (warp == kPageWarp) {
    Pages<D, BITS> pg{a, ctl, lane};
    while (walk.next(a, sg, false)) pg.run(sg, Walk::seen(a, sg), tc, w);
  } else if (warp == kMmaWarp) {
    // This warp's own instructions set the pace of the products if there are many between
    // them: the two orders of a piece are written out, ring positions and parities are
    // counters of their own, and what comes from memory is broadcast from lane 0, which
    // tells the compiler that it is the same in all lanes (uniform registers).
    const uint32_t idesc_x = idesc_f16(G::TT), idesc_o = idesc_f16(D);
    const uint32_t base = smem_u32(smem);
    const uint32_t tmem = __shfl_sync(kAll, ctl.tmem_base, 0);
    uint32_t ks = 0, kp = 0, vs = 0, vp = 0;       // next key and value tile: ring place, parity
    uint32_t dn = 0, mt = 0, qp[2] = {0, 0}, pp[2] = {0, 0};
    // whether the next tile's values are bf16 (known with its keys, used with its values)
    const auto look = [&]() {
      const bool wide = is_wide(metas[mt]);
      mt = (mt + 1) % kMetaRing;
      return wide;
    };
    const auto logits = [&](int q, int slot) {       // X of query tile q with key tile ks
      __syncwarp();
      const uint32_t x = tmem + G::kColS + G::TT * slot;
      const uint64_t kd = sdesc_k_sw128(base + G::kOffK + ks * G::kTileBytes);
      if constexpr (G::kQTmem) {
#pragma unroll
        for (int j = 0; j < G::J; j += 2)
          mma_ts_tile_pair_elect(x, tmem + G::kColQ + 32 * j, tmem + G::kColQ + 32 * (j + 1),
                                 kd + j * (G::TT * 8), kd + (j + 1) * (G::TT * 8), idesc_x, j > 0);
      } else {
        const uint64_t qd = sdesc_k_sw128(base + q * G::kQBytes);
        if constexpr (G::J == 2)
          mma_ss_pair(x, qd, kd, 1024, G::TT * 8, idesc_x, 0);
        else
          mma_ss_chunk(x, qd, kd, idesc_x, 0);
      }
      mma_commit_elect(&ctl.s_full[slot]);
    };
    const auto keys_done = [&]() {
      mma_commit_elect(&ctl.k_empty[ks]);
      if (++ks == G::KS) ks = 0, kp ^= 1;
    };
    const auto outputs = [&](int q, int slot, bool first, bool wide) {   // O of query tile q with value tile vs
      w.wait(&ctl.p_full[slot], slot ? pp[1] : pp[0]);
      (slot ? pp[1] : pp[0]) ^= 1;
      tc_fence_after();
      __syncwarp();
      const uint32_t p = tmem + G::kColS + G::TT * slot, o = tmem + G::kColO + q * D;
      const uint64_t v = sdesc_k_sw128(base + G::kOffV + vs * G::kTileBytes);
      const uint32_t idesc = __any_sync(kAll, wide) ? idesc_o | kBothBf16 : idesc_o;
      if constexpr (G::TT == 128)
        mma_ts_tile_pair_elect(o, p, p + 32, v, v + D * 128 / 16, idesc, !first);
      else
        mma_ts_tile_chunk_elect(o, p, v, idesc, !first);
      mma_commit_elect(&ctl.pv_done[q]);
    };
    const auto values_done = [&]() {
      mma_commit_elect(&ctl.done[dn]);
      dn = (dn + 1) % kMetaRing;
      if (++vs == G::KS) vs = 0, vp ^= 1;
    };
    while (walk.next(a, sg, false)) {
      const int nt = __shfl_sync(kAll, sg.kt1 - sg.kt0, 0);
      const int nqt = __shfl_sync(kAll, query_tiles(sg), 0);
      w.wait(&ctl.q_full[0], qp[0]);
      qp[0] ^= 1;
      if (nqt == 2) {
        w.wait(&ctl.q_full[1], qp[1]);
        qp[1] ^= 1;
        tc_fence_after();
        bool wide = false;
        for (int it = 0; it < nt; ++it) {
          w.wait(&ctl.k_full[ks], kp);
          tc_fence_after();
          logits(0, 0);
          const bool next = look();
          if (it > 0) {
            outputs(1, 1, it == 1, wide);
            values_done();
          }
          wide = next;
          logits(1, 1);
          keys_done();
          w.wait(&ctl.v_full[vs], vp);
          outputs(0, 0, it == 0, wide);
        }
        outputs(1, 1, nt == 1, wide);
        values_done();
      } else {
        tc_fence_after();
        bool wide = false;
        for (int it = 0; it < nt; ++it) {
          w.wait(&ctl.k_full[ks], kp);
          tc_fence_after();
          logits(0, it & 1);
          keys_done();
          const bool next = look();
          if (it > 0) {
            w.wait(&ctl.v_full[vs], vp);
            outputs(0, (it - 1) & 1, it == 1, wide);
            values_done();
          }
          wide = next;
        }
        w.wait(&ctl.v_full[vs], vp);
        outputs(0, (nt - 1) & 1, nt == 1, wide);
        values_done();
      }
    }
    // nothing issued may outlive the tensor memory
    mma_commit_elect(&ctl.drain);
    w.ok = true;
    w.wait(&ctl.drain, 0);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, int BITS>
cudaError_t launch_rows(const AttnArgs& a, unsigned blocks, cudaStream_t s) {
  constexpr size_t smem = row_smem<D>();
  static_assert(smem <= 227 * 1024, "shared memory");
  const auto kernel = attn_rows_kernel<D, BITS>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(kernel, smem, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(blocks), dim3(RowGeo<D>::kThreads), smem, s, a);
}

}  // namespace

int attn_unit_rows(int D) { return D == 256 ? 128 : 256; }
int attn_row_tile(int D) { return D == 256 ? RowGeo<256>::TT : RowGeo<128>::TT; }

cudaError_t launch_attn_rows(const AttnArgs& a, unsigned blocks, cudaStream_t s) {
  if (a.c.bits == 8)
    return a.c.D == 64    ? launch_rows<64, 8>(a, blocks, s)
           : a.c.D == 128 ? launch_rows<128, 8>(a, blocks, s)
                          : launch_rows<256, 8>(a, blocks, s);
  return a.c.D == 64    ? launch_rows<64, 4>(a, blocks, s)
         : a.c.D == 128 ? launch_rows<128, 4>(a, blocks, s)
                        : launch_rows<256, 4>(a, blocks, s);
}

}  // namespace moeq4
