// route_scored.cuh — the choice of moe_route_scored, included by route.cu inside its
// namespace: scores, a bias that takes part in the choice only, groups of experts, top-k
// and the weights of one token, by one warp.
//
//   s_e   = exp(l_e - max l) / sum_i exp(l_i - max l)   or   1 / (1 + exp(-l_e))
//   key_e = s_e + bias_e
//   a group's rank is the sum of its `group_best` largest keys; the top_groups groups of
//   the largest rank stay, and of their experts the k of the largest keys are chosen
//   w_j   = factor * s_j (/ sum of the chosen s)
// Equal ranks and equal keys go to the lower index.

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

// Larger key first, then lower expert.
__device__ __forceinline__ bool before(double ka, int ea, double kb, int eb) {
  return ka > kb || (ka == kb && ea < eb);
}

// The choice in fp64: keys that differ in their 30th bit are still told apart. Experts of
// lane: lane + 32 s.
template <int S>
__device__ __noinline__ void select_scored_exact(const RouteArgs& a, const float (&x)[S], int lane,
                                                 int* sE, float* sV) {
  const int E = a.E, k = a.k;
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
    if (e < E) key[s] = score[s] + (a.bias ? static_cast<double>(finite_bias(a.bias[e])) : 0.0);
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

// The choice of token t: experts into sE[0..k), weights into sV[0..k).
template <int S>
__device__ __forceinline__ void select_scored(const RouteArgs& a, int t, int lane, int* sE,
                                              float* sV, bool& bad) {
  const float* row = a.logits + static_cast<size_t>(t) * a.E;
  float x[S];
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int e = lane + 32 * s;
    x[s] = e < a.E ? __ldg(row + e) : 0.f;
  }
#pragma unroll
  for (int s = 0; s < S; ++s) x[s] = finite_logit(x[s], bad);
  select_scored_exact<S>(a, x, lane, sE, sV);
}
