// route_scored.cuh — the choice of moe_route_scored, included by route.cu inside its
// namespace: scores, a bias that takes part in the choice only, groups of experts, top-k
// and the weights of one token, by one warp.
//
//   s_e   = exp(l_e - max l) / sum_i exp(l_i - max l)   or   1 / (1 + exp(-l_e))
//   key_e = s_e + bias_e
//   a group's rank is the sum of its `group_best` largest keys; the top_groups groups of
//   the largest rank stay, and of their experts the k of the largest keys are chosen
//   w_j   = factor * s_j (/ sum of the chosen s)
// Equal ranks and equal keys go to the lower index. Scores grow with the logits, so without a
// bias (and with groups ranked by one key) the logits themselves are the keys: exact ones.

// What a router logit counts as: NaN and -inf as the least finite number, +inf as the
// largest, so that every score is a number.
__device__ __forceinline__ float finite_logit(float x, bool& bad) {
  constexpr float kMax = 3.402823466e38f;
  if (isfinite(x)) return x;
  bad = true;
  return x > 0.f ? kMax : -kMax;
}
// A bias of -inf (an expert taken out of use) or +inf keeps sums of two keys finite.
__device__ __forceinline__ float finite_bias(float b) {
  constexpr float kMax = 3.402823466e38f;
  return b > -kMax ? fminf(b, kMax) : -kMax;   // (NaN: the least)
}

__device__ __forceinline__ bool keys_are_scores(const RouteArgs& a) {
  return a.bias != nullptr || (a.groups > 1 && a.group_best == 2);
}

// Larger key first, then lower expert.
__device__ __forceinline__ bool before(double ka, int ea, double kb, int eb) {
  return ka > kb || (ka == kb && ea < eb);
}

// A score in fp64 (softmax: with the row's largest logit and sum). Not inlined: it is rare.
__device__ __noinline__ double score64(float x, bool softmax, float top, double sum) {
  if (softmax) return exp(static_cast<double>(x) - static_cast<double>(top)) / sum;
  const double z = exp(-fabs(static_cast<double>(x)));   // (never overflows)
  return (x < 0.f ? z : 1.0) / (1.0 + z);
}
__device__ __forceinline__ double bias64(const RouteArgs& a, int e) {
  return a.bias ? static_cast<double>(finite_bias(a.bias[e])) : 0.0;
}
// sum of exp(l - top) over token t's experts.
__device__ __noinline__ double softmax_sum64(const RouteArgs& a, int t, int lane, float top) {
  const float* row = a.logits + static_cast<size_t>(t) * a.E;
  double sum = 0.0;
  for (int e = lane; e < a.E; e += 32)
    sum += exp(static_cast<double>(row[e]) - static_cast<double>(top));
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(kFull, sum, off);
  return sum;
}
// Rank of group g (its largest key, or two keys' sum, from scores) in fp64.
__device__ __noinline__ double group_rank64(const RouteArgs& a, int t, int lane, int g, float top,
                                            double sum) {
  const float* row = a.logits + static_cast<size_t>(t) * a.E;
  const int n = a.E / a.groups;
  double b0 = -INFINITY, b1 = -INFINITY;
  for (int i = lane; i < n; i += 32) {
    const int e = g * n + i;
    const double key = score64(row[e], a.score == MOE_SCORE_SOFTMAX, top, sum) + bias64(a, e);
    b1 = fmax(b1, fmin(b0, key));
    b0 = fmax(b0, key);
  }
  for (int off = 16; off > 0; off >>= 1) {
    const double o0 = __shfl_xor_sync(kFull, b0, off), o1 = __shfl_xor_sync(kFull, b1, off);
    b1 = fmax(fmin(b0, o0), fmax(b1, o1));
    b0 = fmax(b0, o0);
  }
  return a.group_best == 2 ? b0 + b1 : b0;
}

// The whole choice of token t in fp64. Experts of a lane: lane + 32 s.
template <int S>
__device__ __noinline__ void select_scored_exact(const RouteArgs& a, int t, int lane, int* sE,
                                                 float* sV) {
  const int E = a.E, k = a.k;
  const float* row = a.logits + static_cast<size_t>(t) * E;
  float x[S];
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int e = lane + 32 * s;
    bool bad = false;                              // (reported by the caller)
    x[s] = e < E ? finite_logit(row[e], bad) : 0.f;
  }
  double score[S], key[S];
  double sum = 0.0;
  if (a.score == MOE_SCORE_SOFTMAX) {
    float m = -INFINITY;
#pragma unroll
    for (int s = 0; s < S; ++s)
      if (lane + 32 * s < E) m = fmaxf(m, x[s]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, off));
#pragma unroll
    for (int s = 0; s < S; ++s) {
      score[s] = lane + 32 * s < E ? exp(static_cast<double>(x[s]) - static_cast<double>(m)) : 0.0;
      sum += score[s];
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(kFull, sum, off);
#pragma unroll
    for (int s = 0; s < S; ++s) score[s] /= sum;
  } else {
#pragma unroll
    for (int s = 0; s < S; ++s) score[s] = score64(x[s], false, 0.f, 1.0);
  }
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int e = lane + 32 * s;
    key[s] = -INFINITY;                            // not a candidate
    if (e < E)
      key[s] = keys_are_scores(a)
                   ? score[s] + bias64(a, e)
                   : static_cast<double>(x[s]);
  }
  if (a.groups > 1) {
    const int n = E / a.groups;
    double rank = -INFINITY;                       // of group `lane`
    for (int g = 0; g < a.groups; ++g) {
      double b0 = -INFINITY, b1 = -INFINITY;       // the group's largest two keys
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const int e = lane + 32 * s;
        if (e >= g * n && e < g * n + n) {
          b1 = fmax(b1, fmin(b0, key[s]));
          b0 = fmax(b0, key[s]);
        }
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        const double o0 = __shfl_xor_sync(kFull, b0, off), o1 = __shfl_xor_sync(kFull, b1, off);
        b1 = fmax(fmin(b0, o0), fmax(b1, o1));
        b0 = fmax(b0, o0);
      }
      if (lane == g) rank = a.group_best == 2 ? b0 + b1 : b0;
    }
    int ahead = 0;                                 // groups that go before group `lane`
    for (int g = 0; g < a.groups; ++g) {
      const double o = __shfl_sync(kFull, rank, g);
      ahead += before(o, g, rank, lane) ? 1 : 0;
    }
    const uint32_t open = __ballot_sync(kFull, lane < a.groups && ahead < a.top_groups);
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int e = lane + 32 * s;
      if (e < E && !(open >> (e / n) & 1u)) key[s] = -INFINITY;
    }
  }
  double w = 0.0;                                  // lane j: score of the j-th choice
  int chosen = 0;
  uint32_t taken = 0;                              // of this lane's experts
  for (int j = 0; j < k; ++j) {
    double bk = -INFINITY, bs = 0.0;
    int be = INT_MAX;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int e = lane + 32 * s;
      if (!(taken >> s & 1u) && key[s] > -INFINITY && before(key[s], e, bk, be)) {
        bk = key[s];
        bs = score[s];
        be = e;
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const double ok = __shfl_xor_sync(kFull, bk, off), os = __shfl_xor_sync(kFull, bs, off);
      const int oe = __shfl_xor_sync(kFull, be, off);
      if (before(ok, oe, bk, be)) {
        bk = ok;
        bs = os;
        be = oe;
      }
    }
    if ((be & 31) == lane && be < E) taken |= 1u << (be >> 5);
    if (lane == j) {
      chosen = be;
      w = bs;
    }
  }
  double total = 1.0;
  if (a.renorm) {
    total = w;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(kFull, total, off);
  }
  if (lane < k) {
    sE[lane] = chosen;
    // every chosen score may be 0 (sigmoids of logits below -745)
    sV[lane] = total > 0.0 ? static_cast<float>(w / total * a.factor) : 0.f;
  }
}

// What is the same for every token of a call.
struct ScoreMode {
  bool by_score;             // keys are scores plus bias; else logits
  bool sum;                  // the softmax's sum over all experts is needed
  bool vec;                  // 16-byte loads of a lane's experts
  bool grouped;              // some groups fall out
  bool lanes_alike;          // a lane's experts are all in use, or none is
  int n;                     // experts per group
  int lanes_per_group;       // a power of two of lanes hold a group's experts; 0: they do not
  uint32_t inv_n;            // e / n = e * inv_n >> 20 (e < 1024, 2 <= groups)
};

template <int S>
__device__ __forceinline__ ScoreMode score_mode(const RouteArgs& a) {
  ScoreMode m;
  m.by_score = keys_are_scores(a);
  m.sum = a.score == MOE_SCORE_SOFTMAX && (m.by_score || !a.renorm);
  m.vec = S % 4 == 0 && a.E % S == 0;
  m.grouped = a.top_groups < a.groups;
  m.n = a.E / a.groups;
  const int l = m.n / S;
  m.lanes_per_group = l * S == m.n && (l & (l - 1)) == 0 ? l : 0;
  m.lanes_alike = a.E % S == 0 && (!m.grouped || m.lanes_per_group != 0);
  m.inv_n = ((1u << 20) + m.n - 1) / m.n;
  return m;
}

// Order-preserving signed integer of a float, and back.
__device__ __forceinline__ int signed_key(float x) {
  const int u = __float_as_int(x);
  return u ^ ((u >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float signed_float(int k) {
  return __int_as_float(k ^ ((k >> 31) & 0x7FFFFFFF));
}

// The choice of one token: experts into sE[0..k), weights into sV[0..k). Keys are fp32 with
// bounds on their errors; what these leave undecided (the last group that stays, the order of
// chosen experts, the last of them) is decided in fp64 by a few keys, one per lane. Returns
// false (and leaves sE and sV unset) for the whole choice in fp64: very many near-equal keys,
// scores near fp32's smallest numbers. Experts of a lane: lane * S + s.
//
// A candidate is one word: its key as an order-preserving integer, the low bits of which give
// way to the expert's number. One word sorts, reduces over the warp (in one instruction) and
// names its expert. Its order is certain where logits differ in the other bits, or keys by more
// than their errors' sum: a key in fp32 is off by at most
//   sigmoid   2^-21 (e^-x to 2 + 1.2 |x| units, one sum, one quotient, of numbers up to 1)
//   softmax   2^-17 of the largest score (a sum of up to 32 + 5 terms, each to 2 + 1.2 (max - x)
//             units, weighted with their size)
//   bias      2^-24 of the key
// and a word by 2^-23 of its magnitude for each number of the low bits. Candidates whose words
// are closer are compared by their fp32 keys, then by keys in fp64.
template <int S>
__device__ __forceinline__ bool select_scored_fast(const RouteArgs& a, const ScoreMode& m,
                                                   const float (&x)[S], const float (&bias)[S],
                                                   int t, int lane, int* sE, float* sV) {
  // the expert's number, complemented, and the size of the sorting network
  constexpr int kLow = (S <= 1 ? 32 : S <= 2 ? 64 : S <= 4 ? 128 : S <= 8 ? 256 : S <= 16 ? 512 : 1024) - 1;
  constexpr int P = S == 12 ? 16 : S;
  constexpr int kNone = INT_MIN;
  const int E = a.E, k = a.k;
  const bool softmax = a.score == MOE_SCORE_SOFTMAX;
  float top = 0.f, inv = 1.f, key[S];
  if (softmax && m.sum) {
    top = -INFINITY;
#pragma unroll
    for (int s = 0; s < S; ++s) top = fmaxf(top, lane * S + s < E ? x[s] : -INFINITY);
    top = signed_float(__reduce_max_sync(kFull, signed_key(top)));
    float sum = 0.f;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      key[s] = lane * S + s < E ? __expf(x[s] - top) : 0.f;
      sum += key[s];
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(kFull, sum, off);
    inv = 1.f / sum;
#pragma unroll
    for (int s = 0; s < S; ++s) key[s] *= inv;
  } else if (m.by_score) {
#pragma unroll
    for (int s = 0; s < S; ++s) key[s] = __fdividef(1.f, 1.f + __expf(-x[s]));
  }
#pragma unroll
  for (int s = 0; s < S; ++s) {
    if (!m.by_score) key[s] = x[s] + 0.f;          // (-0 is +0: words compare bits)
    else key[s] += bias[s];
  }
  // the errors of two fp32 keys add up to `fixed` and `per` of their magnitudes
  const float fixed = softmax ? inv * 0x1p-16f : 0x1p-20f;
  constexpr float per = 0x1p-23f, per_word = 0x1p-23f + (kLow + 1) * 0x1p-23f;
  double sum64 = 0.0;                              // once it is needed

  uint32_t open = kFull;                           // groups that stay
  if (m.grouped) {
    float g0 = -INFINITY, g1 = -INFINITY;          // lane g: the largest two keys of group g
    if (m.lanes_per_group != 0) {
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const float v = lane * S + s < E ? key[s] : -INFINITY;
        g1 = fmaxf(g1, fminf(g0, v));
        g0 = fmaxf(g0, v);
      }
      for (int off = m.lanes_per_group >> 1; off > 0; off >>= 1) {
        const float o0 = __shfl_xor_sync(kFull, g0, off), o1 = __shfl_xor_sync(kFull, g1, off);
        g1 = fmaxf(fminf(g0, o0), fmaxf(g1, o1));
        g0 = fmaxf(g0, o0);
      }
      g0 = __shfl_sync(kFull, g0, lane * m.lanes_per_group & 31);
      g1 = __shfl_sync(kFull, g1, lane * m.lanes_per_group & 31);
    } else {
      for (int g = 0; g < a.groups; ++g) {
        float b0 = -INFINITY, b1 = -INFINITY;
#pragma unroll
        for (int s = 0; s < S; ++s) {
          const int e = lane * S + s;
          const bool of = e < E && static_cast<int>(e * m.inv_n >> 20) == g;
          const float v = of ? key[s] : -INFINITY;
          b1 = fmaxf(b1, fminf(b0, v));
          b0 = fmaxf(b0, v);
        }
        // the largest of the warp, then the largest once that is taken away
        const int w0 = __reduce_max_sync(kFull, signed_key(b0));
        const int owner = __ffs(__ballot_sync(kFull, signed_key(b0) == w0)) - 1;
        const int w1 = __reduce_max_sync(kFull, signed_key(lane == owner ? b1 : b0));
        if (lane == g) {
          g0 = signed_float(w0);
          g1 = signed_float(w1);
        }
      }
    }
    const bool there = lane < a.groups;
    const float rank = !there ? -INFINITY : a.group_best == 2 ? fminf(fmaxf(g0 + g1, -3.402823466e38f), 3.402823466e38f)
                                     : g0;
    // the top_groups largest ranks, one after the other (equal ones together)
    const int rank_key = there ? signed_key(rank) : INT_MIN;
    int left_key = rank_key, low_key = INT_MIN;
    for (int got = 0; got < a.top_groups;) {
      low_key = __reduce_max_sync(kFull, left_key);
      got += __popc(__ballot_sync(kFull, left_key == low_key));
      if (left_key == low_key) left_key = INT_MIN;
    }
    const bool stays = there && rank_key >= low_key;       // (equal ranks: perhaps too many)
    // Groups whose rank is near the last that stays are compared in fp64; the others are sure.
    // Keys of experts out of use, or forced in, are beyond any rounding of the others.
    const float low = signed_float(low_key);
    float size = there ? fabsf(g0) + fabsf(g1) : 0.f;
    if (!(size < 1e30f)) size = 0.f;
    size = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(size)));
    const float gap = m.by_score ? 2.f * fixed + 4.f * per * size : 0.f;
    const uint32_t sure = __ballot_sync(kFull, there && rank - low > gap);
    const uint32_t near = __ballot_sync(kFull, there && fabsf(rank - low) <= gap);
    open = __ballot_sync(kFull, stays);
    if (__popc(near) > 1) {
      if (__popc(near) > 8) return false;
      double mine = rank;                          // (logits are exact)
      if (m.by_score) {
        if (softmax) sum64 = softmax_sum64(a, t, lane, top);
        for (uint32_t left = near; left != 0u; left &= left - 1u) {
          const int g = __ffs(left) - 1;
          const double r = group_rank64(a, t, lane, g, top, sum64);
          if (lane == g) mine = r;
        }
      }
      int before_me = 0;
      for (uint32_t left = near; left != 0u; left &= left - 1u) {
        const int g = __ffs(left) - 1;
        before_me += before(__shfl_sync(kFull, mine, g), g, mine, lane) ? 1 : 0;
      }
      open = sure | __ballot_sync(kFull, (near >> lane & 1u) && before_me < a.top_groups - __popc(sure));
    }
  }
  int v[P];
#pragma unroll
  for (int s = 0; s < P; ++s)
    v[s] = s < S ? (signed_key(key[s < S ? s : 0]) & ~kLow) | (kLow - s - lane * S) : kNone;
  if (m.lanes_alike) {
    const int e = lane * S;
    if (!(e < E && (!m.grouped || (open >> (e * m.inv_n >> 20) & 1u)))) {
#pragma unroll
      for (int s = 0; s < S; ++s) v[s] = kNone;
    }
  } else {
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int e = lane * S + s;
      if (!(e < E && (!m.grouped || (open >> (e * m.inv_n >> 20) & 1u)))) v[s] = kNone;
    }
  }
#pragma unroll
  for (int size = 2; size <= P; size <<= 1)
#pragma unroll
    for (int stride = size >> 1; stride > 0; stride >>= 1)
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int j = i ^ stride;
        if (j > i) {
          const int hi = max(v[i], v[j]), lo = min(v[i], v[j]);
          const bool desc = (i & size) == 0;
          v[i] = desc ? hi : lo;
          v[j] = desc ? lo : hi;
        }
      }
  // Lane j: the j-th candidate's word. They are drawn in order, the k first and those that the
  // k-th is not clear of.
  const auto clear_of = [&](int w0, int w1) {
    const float k0 = signed_float(w0), k1 = signed_float(w1);
    return m.by_score ? k0 - k1 > fixed + per_word * (fabsf(k0) + fabsf(k1))
                      : ((w0 ^ w1) & ~kLow) != 0;
  };
  int word = kNone, w = kNone;
  const auto draw = [&](int j) {
    if (lane == j) word = w;
    if (v[0] == w) {
#pragma unroll
      for (int s = 0; s + 1 < S; ++s) v[s] = v[s + 1];
      v[S - 1] = kNone;
    }
  };
  for (int j = 0; j < k; ++j) {
    w = __reduce_max_sync(kFull, v[0]);
    draw(j);
  }
  const int last = w;
  int drawn = k;
  for (;; ++drawn) {
    w = __reduce_max_sync(kFull, v[0]);
    if (w == kNone || clear_of(last, w)) break;
    if (drawn == 32) return false;
    draw(drawn);
  }
  const int above = __shfl_up_sync(kFull, word, 1);
  const bool sorted =
      drawn == k && __all_sync(kFull, lane == 0 || lane >= k || clear_of(above, word));
  const int chosen = kLow - (word & kLow);
  const bool held = lane < drawn;
  const float z = held ? a.logits[static_cast<size_t>(t) * E + chosen] : 0.f;
  int place = lane;
  if (!sorted) {
    // by their fp32 keys (logits: exact), where these are clear of each other
    float mine = z;
    if (m.by_score) {
      mine = softmax ? __expf(z - top) * inv : __fdividef(1.f, 1.f + __expf(-z));
      if (a.bias && held) mine += finite_bias(a.bias[chosen]);
    }
    place = 0;
    bool near = false;
    for (int j = 0; j < drawn; ++j) {
      const float o = __shfl_sync(kFull, mine, j);
      const int e = __shfl_sync(kFull, chosen, j);
      place += o > mine || (o == mine && e < chosen) ? 1 : 0;
      near |= j != lane && fabsf(o - mine) <= fixed + per * (fabsf(o) + fabsf(mine));
    }
    if (m.by_score && __any_sync(kFull, held && near)) {
      if (softmax && sum64 == 0.0) sum64 = softmax_sum64(a, t, lane, top);
      const double exact = score64(z, softmax, top, sum64) + (held ? bias64(a, chosen) : 0.0);
      place = 0;
      for (int j = 0; j < drawn; ++j)
        place += before(__shfl_sync(kFull, exact, j), __shfl_sync(kFull, chosen, j), exact, chosen) ? 1 : 0;
    }
  }
  // weights from the chosen logits
  const bool mine = held && place < k;
  if (softmax && !m.sum) top = __shfl_sync(kFull, z, 0);   // only ratios matter
  float s = 0.f;
  if (mine) s = softmax ? expf(z - top) * inv : __fdividef(1.f, 1.f + expf(-z));
  if (!__all_sync(kFull, !mine || (s > 1e-30f && s < 1e30f))) return false;
  float total = 1.f;
  if (a.renorm) {
    total = s;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(kFull, total, off);
  }
  if (mine) {
    sE[place] = chosen;
    sV[place] = __fdividef(s, total) * a.factor;
  }
  return true;
}

// The choice of the tokens t0 + first, t0 + first + stride, ... < t0 + nt by one warp.
template <int S>
__device__ __forceinline__ void select_scored(const RouteArgs& a, int t0, int first, int stride,
                                              int nt, int lane, int* sE, float* sV, bool& bad) {
  const ScoreMode m = score_mode<S>(a);
  float bias[S], next[S];
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int e = lane * S + s;
    bias[s] = a.bias && e < a.E ? finite_bias(a.bias[e]) : 0.f;
  }
  const auto load = [&](int i, float (&x)[S]) {
    if (i >= nt) return;
    const float* row = a.logits + static_cast<size_t>(t0 + i) * a.E + lane * S;
    if constexpr (S % 4 == 0) {
      if (m.vec) {
#pragma unroll
        for (int s = 0; s < S; s += 4) {
          const float4 q = lane * S < a.E ? *reinterpret_cast<const float4*>(row + s)
                                          : make_float4(0.f, 0.f, 0.f, 0.f);
          x[s] = q.x;
          x[s + 1] = q.y;
          x[s + 2] = q.z;
          x[s + 3] = q.w;
        }
        return;
      }
    }
#pragma unroll
    for (int s = 0; s < S; ++s) x[s] = lane * S + s < a.E ? row[s] : 0.f;
  };
  load(first, next);
  for (int i = first; i < nt; i += stride) {
    float x[S];
#pragma unroll
    for (int s = 0; s < S; ++s) x[s] = next[s];
    load(i + stride, next);                        // the next token's, beside this one's choice
    float zero = 0.f;                              // NaN once a logit is not finite
#pragma unroll
    for (int s = 0; s < S; ++s) zero = fmaf(x[s], 0.f, zero);
    const bool odd = __any_sync(kFull, zero != 0.f);
    bad |= odd;
    if (odd || !select_scored_fast<S>(a, m, x, bias, t0 + i, lane, sE + i * a.k, sV + i * a.k))
      select_scored_exact<S>(a, t0 + i, lane, sE + i * a.k, sV + i * a.k);
  }
}
