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

// The choice of token t in fp64: keys that differ in their 30th bit are still told apart.
// Experts of a lane: lane + 32 s.
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
    x[s] = e < E ? finite_logit(__ldg(row + e), bad) : 0.f;
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
    for (int s = 0; s < S; ++s) {
      const double z = exp(-fabs(static_cast<double>(x[s])));   // (never overflows)
      score[s] = (x[s] < 0.f ? z : 1.0) / (1.0 + z);
    }
  }
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int e = lane + 32 * s;
    key[s] = -INFINITY;                            // not a candidate
    if (e < E)
      key[s] = keys_are_scores(a)
                   ? score[s] + (a.bias ? static_cast<double>(finite_bias(a.bias[e])) : 0.0)
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
  int lanes_per_group;       // a power of two of lanes hold a group's experts; 0: they do not
};

template <int S>
__device__ __forceinline__ ScoreMode score_mode(const RouteArgs& a) {
  ScoreMode m;
  m.by_score = keys_are_scores(a);
  m.sum = a.score == MOE_SCORE_SOFTMAX && (m.by_score || !a.renorm);
  m.vec = S % 4 == 0 && a.E % S == 0;
  const int n = a.E / a.groups, l = n / S;
  m.lanes_per_group = a.groups > 1 && l * S == n && (l & (l - 1)) == 0 ? l : 0;
  return m;
}

// The choice of one token in fp32: experts into sE[0..k), weights into sV[0..k). Returns false
// (and leaves them unset) where fp32 cannot tell the order of keys that matter, for the exact
// form. Experts of a lane: lane * S + s.
//
// A key is held as an order-preserving integer whose low bits are its slot in the lane, so that
// one 32-bit word sorts, reduces over the warp and names the expert. Logits whose other bits
// differ are in their true order. An integer of a score's key is off by 2^-23 S of its
// magnitude, and the key in fp32 by at most
//   sigmoid   2^-21 (e^-x to 3 units, one sum, one quotient, of numbers up to 1)
//   softmax   2^-18 of the largest score (a sum of up to 32 + 5 terms, each to 3 units)
//   bias      2^-24 of the key.
// Two keys further apart than their errors' sum are in their true order.
template <int S>
__device__ __forceinline__ bool select_scored_fast(const RouteArgs& a, const ScoreMode& m,
                                                   const float (&x)[S], const float (&bias)[S],
                                                   int t, int lane, int* sE, float* sV) {
  const int E = a.E, k = a.k;
  const bool softmax = a.score == MOE_SCORE_SOFTMAX;
  float top = 0.f, inv = 1.f, key[S];
  if (softmax && m.sum) {
    top = -INFINITY;
#pragma unroll
    for (int s = 0; s < S; ++s)
      if (lane * S + s < E) top = fmaxf(top, x[s]);
    top = key_float(__reduce_max_sync(kFull, float_key(top)));
    float sum = 0.f;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      key[s] = lane * S + s < E ? expf(x[s] - top) : 0.f;
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
    if (!m.by_score) key[s] = x[s];
    else key[s] += bias[s];
  }
  // a key's error is at most half of `fixed` plus `per` of its magnitude
  const float fixed = softmax ? inv * 0x1p-17f : 0x1p-20f;
  constexpr float per = 0x1p-24f + S * 0x1p-23f;
  bool clear = true;
  uint32_t open = kFull;     // lanes whose group stays
  if (a.groups > 1 && a.top_groups < a.groups) {
    if (m.lanes_per_group == 0) return false;
    float b0 = -INFINITY, b1 = -INFINITY;          // the largest two keys of the lane's group
#pragma unroll
    for (int s = 0; s < S; ++s) {
      if (lane * S + s < E) {
        b1 = fmaxf(b1, fminf(b0, key[s]));
        b0 = fmaxf(b0, key[s]);
      }
    }
    for (int off = m.lanes_per_group >> 1; off > 0; off >>= 1) {
      const float o0 = __shfl_xor_sync(kFull, b0, off), o1 = __shfl_xor_sync(kFull, b1, off);
      b1 = fmaxf(fminf(b0, o0), fmaxf(b1, o1));
      b0 = fmaxf(b0, o0);
    }
    const float rank = a.group_best == 2 ? fmaxf(b0 + b1, -3.402823466e38f) : b0;
    int ahead = 0;
    for (int g = 0; g < a.groups; ++g)
      ahead += __shfl_sync(kFull, rank, g * m.lanes_per_group) > rank ? 1 : 0;
    const bool there = lane < a.groups * m.lanes_per_group, stays = there && ahead < a.top_groups;
    open = __ballot_sync(kFull, stays);
    // The last group that stays has to be clear of the first that does not. (Equal ranks are
    // ahead of neither, so that more groups would stay.) Keys of experts out of use, or forced
    // in, are beyond any rounding of the others.
    const float low = key_float(__reduce_min_sync(kFull, stays ? float_key(rank) : kFull));
    const uint32_t high = __reduce_max_sync(kFull, there && !stays ? float_key(rank) : 0u);
    float size = there ? fabsf(b0) + fabsf(b1) : 0.f;
    if (!(size < 1e30f)) size = 0.f;
    size = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(size)));
    clear = __popc(open) == a.top_groups * m.lanes_per_group &&
            low - key_float(high) > (m.by_score ? 2.f * fixed + 4.f * per * size : 0.f);
  }
  uint32_t v[S];
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const bool in = lane * S + s < E && (open >> lane & 1u);
    v[s] = in ? (float_key(key[s]) & ~static_cast<uint32_t>(S - 1)) | (S - 1 - s) : 0u;
  }
#pragma unroll
  for (int size = 2; size <= S; size <<= 1)
#pragma unroll
    for (int stride = size >> 1; stride > 0; stride >>= 1)
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const int j = i ^ stride;
        if (j > i) {
          const uint32_t hi = max(v[i], v[j]), lo = min(v[i], v[j]);
          const bool desc = (i & size) == 0;
          v[i] = desc ? hi : lo;
          v[j] = desc ? lo : hi;
        }
      }
  int chosen = 0;                                  // lane j: the j-th choice
  uint32_t prev = 0;
  for (int j = 0; j <= k; ++j) {
    const uint32_t w = __reduce_max_sync(kFull, v[0]);
    const uint32_t who = __ballot_sync(kFull, v[0] == w);
    if (w == 0u) break;                            // (only past the last expert, j = k)
    if (j > 0) {
      const float a0 = key_float(prev), a1 = key_float(w);
      clear = clear && (m.by_score ? a0 - a1 > fixed + per * (fabsf(a0) + fabsf(a1))
                                   : ((prev ^ w) & ~static_cast<uint32_t>(S - 1)) != 0u);
    }
    clear = clear && (who & (who - 1u)) == 0u;
    prev = w;
    if (j == k) break;
    const int owner = __ffs(who) - 1;
    if (lane == j) chosen = owner * S + (S - 1 - static_cast<int>(w & (S - 1)));
    if (lane == owner) {
#pragma unroll
      for (int s = 0; s + 1 < S; ++s) v[s] = v[s + 1];
      v[S - 1] = 0u;
    }
  }
  if (!clear) return false;
  // weights from the chosen logits
  const float z = lane < k ? __ldg(a.logits + static_cast<size_t>(t) * E + chosen) : 0.f;
  if (softmax && !m.sum) top = __shfl_sync(kFull, z, 0);   // only ratios matter
  float s = 0.f;
  if (lane < k) s = softmax ? expf(z - top) * inv : 1.f / (1.f + expf(-z));
  // (scores near fp32's smallest, or infinite ones that came from a bad logit: the exact form)
  if (!__all_sync(kFull, lane >= k || (s > 1e-30f && s < 1e30f))) return false;
  float total = 1.f;
  if (a.renorm) {
    total = s;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(kFull, total, off);
  }
  if (lane < k) {
    sE[lane] = chosen;
    sV[lane] = s / total * a.factor;
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
    bias[s] = a.bias && e < a.E ? finite_bias(__ldg(a.bias + e)) : 0.f;
  }
  const auto load = [&](int i, float (&x)[S]) {
    if (i >= nt) return;
    const float* row = a.logits + static_cast<size_t>(t0 + i) * a.E + lane * S;
    if constexpr (S % 4 == 0) {
      if (m.vec) {
#pragma unroll
        for (int s = 0; s < S; s += 4) {
          const float4 q = lane * S < a.E ? __ldg(reinterpret_cast<const float4*>(row + s))
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
    for (int s = 0; s < S; ++s) x[s] = lane * S + s < a.E ? __ldg(row + s) : 0.f;
  };
  load(first, next);
  for (int i = first; i < nt; i += stride) {
    float x[S];
#pragma unroll
    for (int s = 0; s < S; ++s) x[s] = next[s];
    load(i + stride, next);                        // the next token's, beside this one's choice
    bool odd = false;
#pragma unroll
    for (int s = 0; s < S; ++s) odd |= !isfinite(x[s]);
    odd = __any_sync(kFull, odd);
    bad |= odd;
    if (odd || !select_scored_fast<S>(a, m, x, bias, t0 + i, lane, sE + i * a.k, sV + i * a.k))
      select_scored_exact<S>(a, t0 + i, lane, sE + i * a.k, sV + i * a.k);
  }
}
