/*
 * moeq4.h — C-ABI of the GB300 (sm_103a) prefill MoE expert layer with 4-bit
 * groupwise-affine weights.
 *
 * Sources, cited by page title and section:
 *  [A] "Perplexity Lily 오픈소스 공개 — Apple Silicon에서 Qwen3.6-35B-A3B를 더 빠르게 돌리는
 *      Rust + Metal 추론 엔진" (alltoptrend.co.kr), §5-1 and §5-2.
 *  [C] "Apple silicon용 Lily, Qwen 추론 최적화" (aitrends.kr), sections "Qwen 구조와
 *      Prefill 경로" and "GPU 상주와 메모리 절감", glossary.
 *
 * Conventions shared by every call
 *  - All array pointers are DEVICE pointers, 16-byte aligned, owned by the
 *    caller. The library never allocates, frees or synchronises (except
 *    moe_get_device_error, which says so), and keeps no state between calls
 *    besides per-device constants (SM count) and the GEMM kernels' dynamic
 *    shared-memory attribute, which is set once per device.
 *  - Every compute call is asynchronous on `stream` (a cudaStream_t passed as
 *    void*; NULL = legacy default stream). Outputs are valid in stream order.
 *  - bf16 values are passed as their uint16_t bit patterns.
 *  - Arguments are validated on the host; a failed check returns a negative
 *    status and enqueues nothing. A launch failure returns MOE_ERR_CUDA.
 *    Problems only the device can see (non-finite logits, a pipeline wait
 *    that ran out of time) set bits in the caller's device error word and
 *    never trap; read it with moe_get_device_error after synchronising.
 *  - Limits: 1 <= E <= 1024, 1 <= k <= min(E, 32), 1 <= block_m <= 128,
 *    T*k < 2^30, d % 256 == 0, f % 128 == 0, f_s % 128 == 0, d <= 16384,
 *    f, f_s <= 8192.
 */
#ifndef MOEQ4_H
#define MOEQ4_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t moe_status;
#define MOE_OK                0
#define MOE_ERR_ARG          -1  /* null pointer, negative size, k/E/block_m out of range */
#define MOE_ERR_SHAPE        -2  /* d, f, f_s not multiples of the tile quanta / too large */
#define MOE_ERR_WORKSPACE    -3  /* ws NULL or smaller than the *_workspace_size result */
#define MOE_ERR_CUDA         -4  /* a CUDA runtime/driver call or launch failed */
#define MOE_ERR_DEVICE       -5  /* device error word is non-zero (moe_get_device_error) */
#define MOE_ERR_UNSUPPORTED  -6  /* current device is not sm_103 */
#define MOE_ERR_ALIGN        -7  /* a pointer is not 16-byte aligned */
#define MOE_ERR_TOO_LARGE    -8  /* sizes exceed the fixed scratch of moe_route_noalloc */

/* Bits of the device error word. */
#define MOE_DEVERR_NONFINITE_LOGIT  1  /* a router logit was NaN/Inf (treated as -inf) */
#define MOE_DEVERR_SCAN_TIMEOUT     2  /* reserved (routing has no waits; never set) */
#define MOE_DEVERR_PIPE_TIMEOUT     4  /* a GEMM pipeline or grid barrier wait gave up */
#define MOE_DEVERR_BAD_TILE         8  /* a block-map entry was out of range */
#define MOE_DEVERR_BAD_WORKSPACE   16  /* the FFN scratch counters were not zero at launch,
                                          or the routing's count rows did not add up to
                                          T*k (a scratch shared by overlapping calls) and
                                          a row could not be placed (its write was
                                          skipped) */
#define MOE_DEVERR_BAD_SLOT        32  /* a cache slot was neither -1 nor inside the cache */
#define MOE_DEVERR_BAD_PAGE        64  /* a page of a context was outside the cache (its
                                          tokens were left out) */
#define MOE_DEVERR_BAD_LENGTH     128  /* a context length was negative or above max_len
                                          (taken as 0 or max_len) */

/* One 4-bit groupwise-affine matrix [R][K] ([A] §5-1; [C] glossary):
 *   qw    uint32 [R][K/8]   8 codes per word, code c of a row in word c/8 at bits 4*(c%8)
 *   scale bf16   [R][K/64]  one scale per 64 consecutive weights along K
 *   bias  bf16   [R][K/64]  one bias  per 64 consecutive weights along K
 * Dequantised weight: bf16(fp32(scale) * q + fp32(bias)). Stacked experts are
 * contiguous: expert e's rows start at row e*R. */
typedef struct moe_q4_mat {
  const uint32_t* qw;
  const uint16_t* scale;
  const uint16_t* bias;
} moe_q4_mat;

/* Weights of one MoE layer.
 *   gate_up    [E][2f][d]: rows 0..f-1 gate projection, rows f..2f-1 up projection
 *   down       [E][d][f]
 *   sh_gate_up [2f_s][d], sh_down [d][f_s]: the always-on shared expert ([C] "Qwen 구조와
 *              Prefill 경로": 8 of 256 experts plus one shared expert), added with
 *              weight 1; all pointers NULL and f_s = 0 when the layer has none. */
typedef struct moe_q4_weights {
  moe_q4_mat gate_up;
  moe_q4_mat down;
  moe_q4_mat sh_gate_up;
  moe_q4_mat sh_down;
  int32_t E, d, f, f_s;
} moe_q4_weights;

/* The same weights in the kernel-native order that moe_expert_ffn streams,
 * produced once by moe_q4_prepack (values unchanged; only their order differs).
 * Each matrix [R][K] is cut into units of 256 rows (two 128-row tiles) and
 * K-chunks of 64; chunk c of unit u is one contiguous 9216-byte block:
 *   bytes [0, 8192)     codes of tile 0 then tile 1; per tile, K 0-31 of its
 *                       128 rows (16 bytes each, row-major) then K 32-63;
 *                       nibbles of each word in the order k0 k2 k4 k6 k1 k3 k5 k7
 *   bytes [8192, 9216)  2 x 128 words: scale | bias << 16 (bf16 bits)
 * Row i of tile t of unit p of expert e is, for gate/up (F = f or f_s),
 *   e*2F + up*F + 64*(2p + t) + 8*(i >> 4) + (i & 7), up = (i >> 3) & 1
 * (gate and up rows of a feature interleaved in blocks of 8), and for down
 *   e*d + 256p + 128t + i.
 * Matrices follow each other: routed gate/up, routed down, shared gate/up,
 * shared down. */
typedef struct moe_q4_packed {
  const void* data;   /* device buffer of moe_q4_packed_size() bytes */
  int32_t E, d, f, f_s;
} moe_q4_packed;

/* Bytes of the kernel-native copy of one layer's weights (same as the inputs). */
size_t moe_q4_packed_size(int32_t E, int32_t d, int32_t f, int32_t f_s);

/* Reorders W into the kernel-native layout at dst (device, dst_bytes >=
 * moe_q4_packed_size). Run once when the weights are loaded. */
moe_status moe_q4_prepack(const moe_q4_weights* W, void* dst, size_t dst_bytes, void* stream);

/* Routing result, written by moe_route, read by moe_expert_ffn. Device arrays:
 *   ids     int32 [T][k]   chosen experts per token, descending logit, ties to lower index
 *   w       fp32  [T][k]   softmax over E restricted to the chosen experts (sums to 1)
 *   counts  int32 [E]      rows per expert (histogram of allocations)
 *   offsets int32 [E+1]    exclusive prefix sum of counts; offsets[E] = T*k
 *   perm    int32 [T*k]    perm[offsets[e] + r] = t*k + j, the r-th (t, j) of expert e
 *                          in ascending (t, j) order
 *   inv     int32 [T*k]    inv[t*k + j] = position of (t, j) in perm
 *   tiles   int32 [moe_route_max_tiles()][3]  block map: (expert, first row, rows),
 *                          experts ascending, at most block_m rows per tile
 *   n_tiles int32 [1]      number of valid block-map entries (device-resident)
 *   err     int32 [1]      device error word (MOE_DEVERR_* bits); zero it once
 *                          before first use, the library only ORs bits into it
 * T, E, k, block_m describe the arrays (host values). */
typedef struct moe_route_out {
  int32_t* ids;
  float*   w;
  int32_t* counts;
  int32_t* offsets;
  int32_t* perm;
  int32_t* inv;
  int32_t* tiles;
  int32_t* n_tiles;
  int32_t* err;
  int32_t T, E, k, block_m;
} moe_route_out;

/* Upper bound on the block-map length: T*k/block_m + min(E, T*k). */
int32_t moe_route_max_tiles(int32_t T, int32_t E, int32_t k, int32_t block_m);

/* Bytes of scratch for moe_route: one row of per-expert counts per routing
 * block. Its contents at launch do not matter (every call writes each row
 * before it reads it) and it needs no zero-filling; calls that overlap on the
 * GPU must not share it. */
size_t moe_route_workspace_size(int32_t T, int32_t E, int32_t k);

/* Bytes of scratch for moe_expert_ffn: two grid-barrier counters (256 bytes),
 * the SwiGLU activations of every routed row (tile-padded to 16 rows), those of
 * the shared expert, and the fp32 combine buffer [T][d]. Zero-fill it before
 * first use; every call leaves the counters zero again. */
size_t moe_ffn_workspace_size(int32_t T, int32_t E, int32_t k, int32_t d, int32_t f,
                              int32_t f_s, int32_t block_m);

/* Bytes of scratch for moe_layer: the routing part followed by the FFN part.
 * Zero-fill it before first use (the FFN part's counters must start zeroed).
 * The split between the two parts depends on T: a workspace serves calls with
 * the T it was sized for; for another T use another workspace, or zero-fill it
 * again before the first call with the new T. */
size_t moe_layer_workspace_size(int32_t T, int32_t E, int32_t k, int32_t d, int32_t f,
                                int32_t f_s, int32_t block_m);

/* Routing on the GPU, enqueued on one stream with no host synchronisation
 * ([A] §5-2: histogram, prefix scan, scatter and block map in one command
 * buffer; [C] "GPU 상주와 메모리 절감": per-token expert selection, histogram
 * of allocations, prefix scan for start offsets, scatter into expert groups).
 *   logits  fp32 [T][E] row-major router logits (device)
 *   out     result arrays and T, E, k, block_m (host struct, device arrays)
 *   ws      scratch of moe_route_workspace_size(T, E, k) bytes
 * T = 0 is allowed (counts/offsets zeroed, n_tiles = 0; logits, ids, w, perm
 * and inv may then be NULL). A batch of at most 8 tokens takes one kernel
 * launch, a larger one two (choose and count, then place), each launched with
 * programmatic stream serialization; no block waits on another, and inv holds
 * the rows' local ranks between the two. A launch the device refuses returns
 * MOE_ERR_CUDA. */
moe_status moe_route(const float* logits, const moe_route_out* out, void* ws, size_t ws_bytes,
                     void* stream);

/* How moe_route_scored chooses. Score of an expert: softmax over all E logits, or the
 * sigmoid of its own. key = score + bias; the bias (a balance term) takes part in the
 * choice only. The E experts form `groups` runs of E / groups; a group ranks by the sum
 * of its group_best largest keys, the top_groups best groups stay, and the k largest
 * keys among their experts are chosen, descending; equal ranks and equal keys go to the
 * lower index. Weight of a choice: factor * score, divided by the sum of the chosen
 * scores if renorm (0 where that sum is 0). */
#define MOE_SCORE_SOFTMAX 0
#define MOE_SCORE_SIGMOID 1

typedef struct moe_route_score {
  const float* bias;       /* device fp32 [E], or NULL: none. -inf: only where fewer than k
                              other experts are left; NaN counts as -inf */
  int32_t score;           /* MOE_SCORE_SOFTMAX or MOE_SCORE_SIGMOID */
  int32_t groups;          /* divides E, at most 32; 1: no groups */
  int32_t top_groups;      /* 1 <= top_groups <= groups, k <= top_groups * E / groups */
  int32_t group_best;      /* 1 or 2 (at most E / groups); not used without groups */
  int32_t renorm;          /* 0 or 1 */
  float   factor;
} moe_route_score;

/* moe_route with another choice: the same arrays, limits and scratch; one launch, two, or from
 * 2048 tokens on three. Keys are compared in 64-bit arithmetic, and without a bias (and with
 * group_best 1) as the exact scores, whose order is that of the logits (+0.0 and -0.0 are
 * equal). Sums that are equal on paper may differ there by a rounding (s(x) + s(-x) of two
 * groups, say), and then go by it. Weights are fp32 within a few units in the
 * last place. A NaN or -inf logit counts as the least finite number, +inf as the largest, and
 * either sets MOE_DEVERR_NONFINITE_LOGIT. */
moe_status moe_route_scored(const float* logits, const moe_route_score* score,
                            const moe_route_out* out, void* ws, size_t ws_bytes, void* stream);

/* moe_route for callers that cannot allocate device memory. The pages have no
 * counterpart; this entry exists for code that may not call cudaMalloc at all,
 * such as a serving process that reserves all device memory up front and hands
 * out fixed arenas, or a plugin that has no access to its host framework's
 * allocator. Same inputs, outputs and results as moe_route, but its scratch is
 * a fixed array inside the library (1 MB, held on every GPU that loads the
 * library until the process exits), so:
 *  - sizes are limited to T <= 8192, E <= 256, k <= 8; larger ones return
 *    MOE_ERR_TOO_LARGE and enqueue nothing;
 *  - the first call on a device looks up the array's device address (with
 *    that device current); make that first call before any stream capture;
 *  - every call shares the one array: whatever an earlier call left in it
 *    (even one that did not finish) is overwritten before it is read; calls
 *    whose work overlaps on the GPU (other streams, other host threads) race
 *    and must be serialised by the caller;
 *  - it calls no cudaMalloc, cudaFree or allocating library routine. */
moe_status moe_route_noalloc(const float* logits, const moe_route_out* out, void* stream);

/* Router projection with the top-k selection fused into its epilogue ([C] "Qwen
 * 구조와 Prefill 경로": the router picks 8 of 256 experts per token; "GPU 상주와 메모리
 * 절감": per-token expert selection stays on the GPU):
 *   logits[t][e] = sum_c x[t][c] * Wr[e][c]   (bf16 inputs, fp32 accumulation)
 *   out->ids[t][j] = the k largest logits of token t, descending, ties to the lower index
 *   out->w[t][j]   = exp(l_j - l_max) / sum over the chosen of exp(l - l_max), fp64 -> fp32
 *   x         bf16 [T][d] token activations (device)
 *   w_router  bf16 [E][d] router weights, E = out->E (device)
 *   logits    fp32 [T][E] (device) or NULL when only the choice is wanted
 *   out       only ids, w and err are written; T, E, k describe them
 * Limits: E % 16 == 0, E <= 256, k <= 8, d % 64 == 0. Non-finite logits rank as
 * -inf and set MOE_DEVERR_NONFINITE_LOGIT. One kernel launch (tcgen05; a cluster
 * of 4, 2 or 1 CTAs per 128 tokens, each with a share of the experts, merging
 * their lists through distributed shared memory). T = 0 launches nothing. */
moe_status moe_router_topk(const uint16_t* x, const uint16_t* w_router, int32_t T, int32_t d,
                           float* logits, const moe_route_out* out, void* stream);

/* The rest of the routing (histogram, prefix scan, scatter, block map, as in
 * moe_route) from chosen experts already in out->ids and out->w, e.g. written
 * by moe_router_topk. An id outside [0, E) sets MOE_DEVERR_BAD_TILE and counts
 * as expert 0. ws as for moe_route. */
moe_status moe_route_ids(const moe_route_out* out, void* ws, size_t ws_bytes, void* stream);

/* The layer from hidden states: moe_router_topk, moe_route_ids and
 * moe_expert_ffn on one stream, no host sync. logits may be NULL; ws of
 * moe_layer_workspace_size(...) bytes, zero-filled before first use. The
 * router limits above apply. Every host-side check of the three steps runs
 * before the first launch: a rejected call enqueues nothing. */
moe_status moe_layer_router(const uint16_t* x, const uint16_t* w_router, int32_t T,
                            const moe_q4_packed* W, float* logits, const moe_route_out* r,
                            uint16_t* y, void* ws, size_t ws_bytes, void* stream);

/* Grouped expert FFN with in-kernel 4-bit dequantisation ([A] §5-1: weights stay
 * packed, dequantised tile by tile on chip, FP32 accumulation; [C] "Qwen 구조와
 * Prefill 경로"):
 *   y[t] = bf16( sum_j w[t,j] * FFN_{ids[t,j]}(x[t]) + FFN_shared(x[t]) ),
 *   FFN_e(x) = Wd_e * bf16( silu(Wg_e x) * (Wu_e x) ).
 *   x   bf16 [T][d] token activations (device)
 *   W   layer weights in the kernel-native layout (moe_q4_prepack); W->d must equal d
 *   r   routing result of moe_route for the same T (device arrays)
 *   y   bf16 [T][d] output (device)
 *   ws  scratch of moe_ffn_workspace_size(T, E, k, d, f, f_s, block_m) bytes
 * T = 0 is allowed: nothing is launched, and x and y may be NULL. */
moe_status moe_expert_ffn(const uint16_t* x, int32_t T, int32_t d, const moe_q4_packed* W,
                          const moe_route_out* r, uint16_t* y, void* ws, size_t ws_bytes,
                          void* stream);

/* moe_expert_ffn for small batches (decode steps, short prompts: T <= 64).
 * With a few tokens per expert the layer streams 4-bit weights ([A] §6:
 * batch-1 decode is bound by memory bandwidth), so each touched expert's work
 * is split along K over many CTAs and multiplied on the CUDA cores with fp32
 * accumulation: three launches (gate/up partial sums, SwiGLU + down with the
 * weighted combine, bf16 output). Same arguments, result and workspace as
 * moe_expert_ffn, which takes this path by itself for T <= 2. T > 64 returns
 * MOE_ERR_SHAPE. */
moe_status moe_expert_ffn_decode(const uint16_t* x, int32_t T, int32_t d,
                                 const moe_q4_packed* W, const moe_route_out* r, uint16_t* y,
                                 void* ws, size_t ws_bytes, void* stream);

/* moe_route followed by moe_expert_ffn on the same stream, no host sync.
 *   x bf16 [T][d], logits fp32 [T][E]; r receives the routing result; y bf16 [T][d].
 *   ws of moe_layer_workspace_size(...) bytes, zero-filled before first use.
 * T = 0 is allowed (the routing result is the empty one; x, logits and y may
 * be NULL). Every host-side check of both steps runs before the first launch:
 * a rejected call enqueues nothing. */
moe_status moe_layer(const uint16_t* x, const float* logits, int32_t T, const moe_q4_packed* W,
                     const moe_route_out* r, uint16_t* y, void* ws, size_t ws_bytes,
                     void* stream);

/* moe_layer with the routing of moe_route_scored. Every host-side check of both steps
 * runs before the first launch. */
moe_status moe_layer_scored(const uint16_t* x, const float* logits, int32_t T,
                            const moe_q4_packed* W, const moe_route_score* score,
                            const moe_route_out* r, uint16_t* y, void* ws, size_t ws_bytes,
                            void* stream);

/* Input of the next stacked layer in the bounded-chunk prefill run ([A] §5-2:
 * long prompts run in bounded chunks; [C] "GPU 상주와 메모리 절감"):
 *   out[t] = bf16( v / sqrt(mean(v^2)) ),  v = y[t] + x[t]   (fp32, no epsilon)
 *   y, x, out bf16 [T][d] (device); out may alias x. d % 8 == 0. */
moe_status moe_residual_rms(const uint16_t* y, const uint16_t* x, uint16_t* out, int32_t T,
                            int32_t d, void* stream);

/* Asks the GPU to bring [ptr, ptr + bytes) of device memory into L2 (bulk
 * prefetch requests, no data returned), as one small kernel on `stream` that
 * may overlap the tail of the previous kernel (programmatic serialization).
 * In the bounded-chunk run ([A] §5-2) the caller issues it after layer l's FFN
 * with the first megabytes of layer l+1's packed weights: the gate/up weights
 * of the experts that layer's first units read. ptr and bytes 16-byte aligned. */
moe_status moe_l2_prefetch(const void* ptr, size_t bytes, void* stream);

/* ------------------------------------------------------------------------
 * Attention side of a decoder layer: rotary positions, a paged key/value cache
 * in the weights' number format, and attention over it.
 * ------------------------------------------------------------------------ */

#define MOE_BF16 0
#define MOE_F16  1
#define MOE_F32  2
#define MOE_E4M3 3   /* 8 bits: 4 of exponent, 3 of mantissa, largest value 448, no infinity */

/* Residual addition and root-mean-square norm of T tokens of H rows of D elements (H = 1:
 * hidden rows; H heads: per head):
 *   h = x + add,  y = h / sqrt(mean(h^2) + eps) * (weight + offset)
 * in fp32 (sums whose squares leave fp32's range are taken again on scaled elements).
 * Any of three results, each rounded once: sum = h, out = y, and y in 8 bits:
 *   scales = max(max|y| / 448, 2^-126) of a row, codes = e4m3(y / scale), ties to even.
 * A row whose y holds a NaN or an infinity has the scale NaN. */
typedef struct moe_norm {
  const void* x;   int64_t x_row, x_head;             /* dtype; token t, row h at t*row + h*head */
  const void* add; int64_t add_row, add_head;         /* dtype, or NULL: h = x */
  void* sum;       int64_t sum_row, sum_head;         /* dtype, or NULL */
  void* out;       int64_t out_row, out_head;         /* dtype, or NULL */
  uint8_t* codes;  int64_t codes_row, codes_head;     /* e4m3, or NULL */
  float* scales;                                      /* [T][H], with codes */
  const void* weight;                                 /* dtype [D], or NULL: 1 */
  int32_t T, H, D;
  int32_t dtype;                                      /* MOE_BF16, MOE_F16 or MOE_F32 */
  float eps;                                          /* > 0 */
  float offset;                                       /* added to the weight */
} moe_norm;

/* One launch. At least one of out and codes. sum or out may be x or add with the same
 * strides; any other overlap of arrays is not allowed, and rows of a result may not
 * overlap. D <= 16384, H <= 65535, T * H < 2^31. Elements aligned to their type; 16-byte
 * aligned pointers and strides (codes: 8 bytes, or 4 for MOE_F32) take the vector path,
 * anything else one element per load. T = 0 launches nothing. */
moe_status moe_rms_norm(const moe_norm* a, void* stream);

/* Dense projection of T tokens with its epilogue:
 *   y = act(x w^T + bias) + add,   e4m3: act(x_scale[t] w_scale[n] (x w^T) + bias) + add
 * fp32 accumulation on the tensor cores (for fp32 results in pieces of 1024 bytes of K, which
 * are added in fp32), everything after it in fp32, one rounding. Activations keep their value in
 * a negative tail: off by 2^-16 of it next to 16-bit results, by a few units in the last place
 * next to fp32 results, and by as much as the rounding of an exponential's argument makes. */
#define MOE_ACT_NONE      0
#define MOE_ACT_RELU      1
#define MOE_ACT_SILU      2  /* y / (1 + exp(-y)) */
#define MOE_ACT_GELU      3  /* y/2 (1 + erf(y / sqrt 2)) */
#define MOE_ACT_GELU_TANH 4  /* y/2 (1 + tanh(sqrt(2/pi) (y + 0.044715 y^3))) */

typedef struct moe_linear_args {
  const void* x;    int64_t x_row;       /* dtype [T][K], row t at t*x_row elements */
  const void* w;    int64_t w_row;       /* dtype [N][K] */
  const float* x_scale;                  /* [T], MOE_E4M3 only (the scales of moe_rms_norm) */
  const float* w_scale;                  /* [N], MOE_E4M3 only */
  const float* bias;                     /* [N], or NULL */
  const void* add;  int64_t add_row;     /* out_dtype [T][N], or NULL */
  void* out;        int64_t out_row;     /* out_dtype [T][N] */
  int32_t* err;                          /* device error word */
  int32_t T, N, K;
  int32_t dtype;                         /* MOE_BF16, MOE_F16 or MOE_E4M3 */
  int32_t out_dtype;                     /* dtype or MOE_F32; any 16- or 32-bit type from MOE_E4M3 */
  int32_t act;
} moe_linear_args;

/* One launch. x and w: 16-byte aligned, rows that do not overlap, strides and K multiples of
 * 16 bytes; out and add: aligned to their type, any stride (out's rows may not overlap).
 * K <= 65536; T, N <= 2^30. add may be out with the same stride; out overlaps nothing else.
 * T = 0 launches nothing. A token's result does not depend on the other tokens' values (an
 * infinity or NaN stays in its row), but a batch of another size may add a row's products in
 * another order. */
moe_status moe_linear(const moe_linear_args* a, void* stream);

/* Rotary positions. The first `rot` elements of a head form rot/2 pairs
 * (a_i, b_i): elements (i, i + rot/2), or (2i, 2i + 1) when interleaved. At
 * position p pair i is turned by angle 2 pi frac(p * phase[i] / 2^64):
 *   a' = mscale * (a cos - b sin),  b' = mscale * (b cos + a sin).
 * phase[i] is the turn per position as a 64-bit binary fraction, so the product
 * wraps at whole turns and the angle keeps its precision at any int32 position.
 * Elements from `rot` on pass through unscaled. */
typedef struct moe_rope_spec {
  const uint64_t* phase;   /* device, [rot/2]; fill it from moe_rope_phases */
  int32_t rot;             /* even, 2 <= rot <= head size */
  int32_t interleaved;     /* 0 or 1 */
  float   mscale;          /* factor of the turned elements (1 unless scaled for long contexts) */
} moe_rope_spec;

/* How the frequencies base^(-2i/rot) are changed for contexts beyond the
 * trained length. */
#define MOE_ROPE_PLAIN  0  /* as they are */
#define MOE_ROPE_LINEAR 1  /* all divided by `factor` (positions interpolated) */
#define MOE_ROPE_BASE   2  /* base * factor^(rot/(rot-2)): the lowest frequency divided by `factor` */
#define MOE_ROPE_BANDS  3  /* pairs with at least `fast` turns over `trained` positions stay, those
                              with at most `slow` turns are divided by `factor`, linear in the
                              pair index between (Peng et al., "YaRN: Efficient Context Window
                              Extension of Large Language Models", 2023, section 3.2) */

/* Host function: fills phase[rot/2] (host memory). base > 1, factor >= 1; trained
 * > 0 and fast > slow > 0 for MOE_ROPE_BANDS (ignored otherwise). */
moe_status moe_rope_phases(uint64_t* phase, int32_t rot, double base, int32_t scaling,
                           double factor, double trained, double fast, double slow);

/* out[t][h] = x[t][h] turned to position pos[t]; backward = 1: the transposed
 * rotation, which takes the gradient of out to that of x.
 *   x, out  device, `dtype` MOE_BF16, MOE_F16 or MOE_F32, T tokens of H heads of D
 *           elements (D even); token t, head h starts at element t*row + h*head.
 *           Strides in elements; out's rows may not overlap. out == x with the same
 *           strides is allowed, any other overlap of the two is not. H <= 65535,
 *           D <= 65536.
 *   pos     int32 [T] device (any value)
 * Angles, sines and products in fp32, one rounding to dtype. 16-byte aligned
 * pointers and strides take the vector path, anything else a scalar one. */
moe_status moe_rope(const void* x, int64_t x_row, int64_t x_head, void* out, int64_t out_row,
                    int64_t out_head, const int32_t* pos, int32_t T, int32_t H, int32_t D,
                    const moe_rope_spec* rope, int32_t backward, int32_t dtype, void* stream);

/* A paged cache of keys and values in groupwise-affine codes: each run of 64
 * elements of a head shares one bf16 scale and bias, value = scale * code + bias.
 * Slot s is token s % page_size of page s / page_size. A page holds, for the Hkv
 * key heads and then the Hkv value heads, one block each:
 *   codes  [page_size][D * bits / 8] bytes; 4-bit: element 2i of a row in the low
 *          nibble of byte i
 *   words  [page_size][D / 64] uint32, scale | bias << 16
 * bits 4 or 8, D 64, 128 or 256, page_size a multiple of 16 up to 4096,
 * pages * page_size < 2^31. Offsets into the cache are 64-bit. */
typedef struct moe_kv_cache {
  void*    data;           /* device, moe_kv_cache_size() bytes, 16-byte aligned */
  int32_t* err;            /* device error word (MOE_DEVERR_* bits are OR-ed into it) */
  int32_t  pages, page_size, Hkv, D, bits;
} moe_kv_cache;

/* Bytes of a cache; 0 if the sizes are not allowed. */
size_t moe_kv_cache_size(int32_t pages, int32_t page_size, int32_t Hkv, int32_t D, int32_t bits);

/* New tokens: bf16 queries, keys and values as they leave the projections
 * (token t, head h at element t*row + h*head; 16-byte aligned pointers, strides
 * multiples of 8). */
typedef struct moe_kv_new {
  const uint16_t* k;  int64_t k_row, k_head;          /* [T][Hkv][D] */
  const uint16_t* v;  int64_t v_row, v_head;          /* [T][Hkv][D] */
  const uint16_t* q;  int64_t q_row, q_head;          /* [T][Hq][D], or NULL: no queries */
  uint16_t* q_out;    int64_t qo_row, qo_head;        /* turned queries; may be q */
  const int32_t* slots;                               /* [T] distinct slots, -1: skip the token's row */
  const int32_t* pos;                                 /* [T]; NULL without rope */
  const moe_rope_spec* rope;                          /* NULL: keys are kept as given, q must be NULL */
  int32_t T, Hq;
} moe_kv_new;

/* Turns queries and keys to their positions, quantises keys and values and
 * writes them into the cache, in one launch. Turned queries and keys are rounded
 * to bf16; per group of 64: bias = min, scale = bf16((max - min) / (2^bits - 1)),
 * code = round((x - bias) * (1 / scale)), difference, reciprocal and product rounded to
 * fp32, ties to even; 0 where scale is 0 (the group is constant, or its range is below
 * bf16's smallest numbers).
 * A group that holds a NaN or an infinity reads back as NaN. Slots outside the
 * cache are skipped and set MOE_DEVERR_BAD_SLOT. q_out may be q with the same strides;
 * otherwise it overlaps no input. Hq <= 32768. T = 0 launches nothing. */
moe_status moe_kv_append(const moe_kv_new* a, const moe_kv_cache* c, void* stream);

/* Cache rows back as bf16(scale * code + bias): k_out, v_out [n][Hkv][D] dense,
 * 16-byte aligned, either may be NULL. A slot of -1 gives a row of zeros; one
 * outside the cache too, and sets MOE_DEVERR_BAD_SLOT. */
moe_status moe_kv_read(const moe_kv_cache* c, const int32_t* slots, int32_t n, uint16_t* k_out,
                       uint16_t* v_out, void* stream);

/* Attention of B requests with nq query tokens each over their cached contexts.
 * Request b attends first to the prefix that all requests share (prefix_len
 * tokens in the pages of prefix_table; read and multiplied once for the whole
 * batch), then to its own lens[b] tokens in the pages table[b][...], of which the
 * last nq are its query tokens: query i sees own tokens 0 .. lens[b] - nq + i.
 *   o = sum_t softmax_t(scale * q . k_t) v_t,  0 where nothing is seen.
 * Query head h reads key/value head h / (Hq / Hkv). Memory of slots that are not
 * seen is never used in arithmetic, whatever it holds. Results do not depend on max_len,
 * but many query tokens take longer with one far above the lengths. */
typedef struct moe_kv_attn {
  const uint16_t* q;  int64_t q_row, q_head;          /* bf16 [B*nq][Hq][D], row b*nq + i */
  uint16_t* out;      int64_t out_row, out_head;      /* bf16 [B*nq][Hq][D]; rows may not overlap */
  const int32_t* table;                               /* [B][table_stride] page numbers */
  const int32_t* lens;                                /* [B] */
  const int32_t* prefix_table;                        /* [ceil(prefix_len / page_size)], or NULL */
  int32_t B, nq, Hq, table_stride;
  int32_t max_len;                                    /* no lens[b] is above it */
  int32_t prefix_len;
  float scale;
} moe_kv_attn;

/* Bytes of scratch for moe_kv_attention (partial results of split contexts). It
 * needs no zero-filling; calls that overlap on the GPU must not share it. 0 if the
 * sizes are not allowed. */
size_t moe_kv_attention_workspace_size(int32_t B, int32_t nq, int32_t Hq, int32_t Hkv, int32_t D,
                                       int32_t max_len, int32_t prefix_len);

/* Limits: B * nq <= 2^24, Hq % Hkv == 0, Hq <= 65535, max_len and prefix_len <= 2^30.
 * Sizes whose work passes 2^30 tiles (8 query rows x 64 tokens at the least) are
 * MOE_ERR_SHAPE. B = 0 launches nothing. Page numbers are read only as far as lens and
 * prefix_len reach; a page outside the cache gives no tokens and sets
 * MOE_DEVERR_BAD_PAGE, a length outside 0 .. max_len is clamped and sets
 * MOE_DEVERR_BAD_LENGTH. q and out: 16-byte aligned, strides multiples of 8, no
 * overlap. */
moe_status moe_kv_attention(const moe_kv_attn* a, const moe_kv_cache* c, void* ws,
                            size_t ws_bytes, void* stream);

/* Synchronises `stream`, copies the device error word `err` to *code and
 * returns MOE_ERR_DEVICE if it is non-zero, MOE_OK otherwise. */
moe_status moe_get_device_error(const int32_t* err, int32_t* code, void* stream);

/* Static text for a status code. */
const char* moe_status_string(moe_status s);

#ifdef __cplusplus
}
#endif

#endif /* MOEQ4_H */
