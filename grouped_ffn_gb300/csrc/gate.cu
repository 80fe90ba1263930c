// Router with a balance bias: scores, selection and weights for every token
// (moe_gate), the gradient of the logits (moe_gate_backward) and the bias
// update from expert loads (moe_gate_update_bias).
//
//   s_e = softmax(l)_e or sigmoid(l_e),   c_e = s_e + b_e
//   groups by the sum of their group_topn largest c, then the k largest c of
//   the kept groups (ties: lower id);   w = scale s  or  scale s / sum_k s.
//
// One warp per token, or (gate_many_kernel) four lanes.  GB300 issues fp64 at a
// small fraction of the fp32 rate and the choice needs more than fp32 only where
// two scores nearly meet, so the choice is made in fp32 with a bound on every
// score's error, and made again with scores to about 45 bits (the closest
// candidates one a lane, or the whole row in exact_token) when a gap that
// decides something is within the bounds: about one token in a thousand of a
// spread-out router with fp32 logits.  Of bf16 logits neighbours are often
// equal: without a bias the last choice ties with the first expert left out in
// about one row of twenty, which gate_many_kernel chooses again as well (65536
// such rows 74 us, with a bias 40 us).
//
// Layout: a group takes p = floor(32 / n_groups) neighbouring lanes and each
// of them V consecutive experts (without groups p = 32), so a lane never
// mixes groups and a row is read in order.  A score becomes a 32-bit key whose
// unsigned order is the scores' (the low log2 V bits give way to the element's
// position in its lane, which puts the lower of equal ones first).
// Each lane sorts its V keys once; a round of the top-k is then one warp
// reduction over the lanes' heads, and the winner moves up its list.
//
// 65536 rows of 256 fp32 logits take 11 us to read, the kernels 78 us with a warp
// a token (1100 instructions a token, 62% of the issue slots) and 39 us with four
// lanes a token (330).  The latter fills neither HBM (19%) nor the issue slots (54%
// while an SM has work, 38% of the launch): a third of a warp's time goes to its
// loads (a request of 16 bytes a lane touches 30 sectors, and none is in flight
// ahead), and rows chosen again hold up the end.  One token: 3.6 us, latency of
// the launch and of the warp's rounds.
#include <cuda_bf16.h>

#include <cfloat>

#include "common.cuh"

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kMaxTopn = 8;
constexpr float kBiasClamp = 1e30f;  // group sums of clamped biases stay finite
// below this logit sigmoid(l) is e^l to fp32 precision, and from -87 on it has fewer
// bits than a float or vanishes: where a chosen one is, renormalised weights are
// taken from scores relative to the largest (sigmoid_rel)
constexpr float kTinyLogit = -80.0f;

struct GateArgs {
  int32_t score_fn, k, n_groups, topk_groups, group_topn, renormalize;
  float scale;
};

__device__ __forceinline__ float load_logit(const float *p) { return __ldg(p); }
__device__ __forceinline__ float load_logit(const __nv_bfloat16 *p) {
  return __bfloat162float(__ldg(p));
}
__device__ __forceinline__ void store_grad(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_grad(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// A logit as the scores see it: -inf for -inf and NaN (a masked expert), and
// at most FLT_MAX.
__device__ __forceinline__ float usable(float x) { return fminf(fmaxf(x, -INFINITY), FLT_MAX); }

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
  return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, off));
  return v;
}

// (the maximum first: of a NaN and a number it is the number)
__device__ __forceinline__ float clamp_bias(float b) {
  return fminf(fmaxf(b, -kBiasClamp), kBiasClamp);
}

__device__ __forceinline__ float rcp_fast(float x) {  // within 1 ulp
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float exp2_fast(float x) {  // within 2 ulp, tiny results 0
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// e^(a - b) for a <= b, 0 for a = -inf: the difference is split error-free
// into hi + lo and e^(hi + lo) = e^hi (1 + lo).
__device__ __forceinline__ float exp_diff(float a, float b) {
  if (a == -INFINITY) return 0.0f;
  const float hi = __fsub_rn(a, b);
  const float bb = __fsub_rn(hi, a);
  const float lo = __fsub_rn(__fsub_rn(a, __fsub_rn(hi, bb)), __fadd_rn(b, bb));
  const float e = expf(hi);
  return hi > -FLT_MAX ? __fmaf_rn(e, lo, e) : 0.0f;
}

__device__ __forceinline__ float sigmoid32(float x) {
  // (far below zero 1 + e^-x overflows; the score is e^x there)
  const float e = expf(x < kTinyLogit ? x : -x);
  return x < kTinyLogit ? e : rcp_fast(__fadd_rn(1.0f, e));
}

// sigmoid(l) e^-ml for l <= ml < 0: e^(l - ml) / (1 + e^l).
__device__ __forceinline__ float sigmoid_rel(float l, float ml) {
  return exp_diff(l, ml) * sigmoid32(-l);
}
__device__ __forceinline__ bool tiny_logit(float l) { return l < kTinyLogit && l > -INFINITY; }

// Sum over lanes 0..15 (the others hold 0), in those lanes: four roundings.
__device__ __forceinline__ float sum16(float x) {
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) x += __shfl_xor_sync(kFull, x, off);
  return x;
}
__device__ __forceinline__ float max16(float x) {
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, off));
  return x;
}

// Float to an unsigned integer of the same order, and back.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ uint64_t ordered(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
  return u ^ ((uint64_t)((int64_t)u >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double unordered(uint64_t k) {
  return __longlong_as_double((int64_t)(k >> 63 ? k ^ 0x8000000000000000ull : ~k));
}

// What lane `lane` holds: experts [e0, e0 + n) of group grp, as part q of p.
template <int V>
struct Share {
  int p, grp, q, e0, n;
  uint32_t members;  // the lanes of this lane's group
  __device__ __forceinline__ Share(int E, int n_groups, int lane) {
    const int gsz = E / n_groups;
    p = 32 / n_groups;
    grp = lane / p;
    q = lane - grp * p;
    const bool has = grp < n_groups && q * V < gsz;
    e0 = has ? grp * gsz + q * V : 0;
    n = has ? min(V, gsz - q * V) : 0;
    members = (p == 32 ? kFull : ((1u << p) - 1u)) << (grp * p & 31);
  }
  // The largest x among the lanes of this lane's group.
  template <typename K>
  __device__ __forceinline__ K group_max(K x, int lane) const {
    K best = x;
    if ((p & (p - 1)) == 0) {
      for (int off = p >> 1; off > 0; off >>= 1) {
        const K o = __shfl_xor_sync(kFull, best, off);
        best = o > best ? o : best;
      }
    } else {
      for (int j = 1; j < p; ++j) {
        const K o = __shfl_sync(kFull, x, (q + j < p ? lane + j : lane + j - p) & 31);
        best = o > best ? o : best;
      }
    }
    return best;
  }
};

// The weight of this lane's chosen expert with logit l (lanes past k hold -inf);
// m and zinv: the row's largest logit and 1 / sum e^(l - m) (softmax scores).
__device__ __forceinline__ float chosen_weight(const GateArgs &a, float l, float m, float zinv) {
  float v;
  if (a.score_fn == MOE_SCORE_SOFTMAX) {
    // renormalised, the chosen experts may all be far below the row's largest
    if (a.renormalize) m = max16(l);
    v = exp_diff(l, m);
    if (!a.renormalize) v *= zinv;
  } else {
    v = sigmoid32(l);
    if (a.renormalize && __any_sync(kFull, tiny_logit(l))) {
      const float ml = max16(l);
      if (ml < 0.0f) v = sigmoid_rel(l, ml);
    }
  }
  if (a.renormalize) {
    const float den = sum16(v);
    v = den > 0.0f ? v * rcp_fast(den) : 0.0f;
  }
  return a.scale * v;
}

// ------------------------------------------------------------ two-float scores
// A value as the unevaluated sum h + l of two floats: about 48 bits at the
// fp32 rate (the fp64 exponential and division made a row cost 12 us).
struct Two {
  float h, l;
};

// e^(hi + lo) for -60 <= hi <= 0, |lo| <= ulp(hi): n = rint(hi / ln 2), r = hi +
// lo - n ln 2 in two floats (ln 2 in three: 16 bits, so that n times it is exact,
// 24 and 24), then Taylor's series, degrees 12 to 7 in fp32 and 6 to 0 in two
// floats.  Relative error below 2^-45.
__device__ __forceinline__ Two exp_two(float hi, float lo) {
  const float n = rintf(hi * 1.4426950409f);
  const float r1 = __fmaf_rn(-n, 0x1.62e4p-1f, hi);  // exact
  const float p = __fmul_rn(n, 0x1.7f7d1cp-20f), pe = __fmaf_rn(n, 0x1.7f7d1cp-20f, -p);
  float rh = __fsub_rn(r1, p);
  const float bb = __fsub_rn(rh, r1);
  const float e = __fsub_rn(__fsub_rn(r1, __fsub_rn(rh, bb)), __fadd_rn(p, bb));
  float rl = __fadd_rn(e, __fsub_rn(lo, __fmaf_rn(n, 0x1.ef357ap-45f, pe)));
  const float t = __fadd_rn(rh, rl);
  rl = __fsub_rn(rl, __fsub_rn(t, rh));
  rh = t;
  float q = 1.0f / 479001600.0f;
  q = __fmaf_rn(q, rh, 1.0f / 39916800.0f);
  q = __fmaf_rn(q, rh, 1.0f / 3628800.0f);
  q = __fmaf_rn(q, rh, 1.0f / 362880.0f);
  q = __fmaf_rn(q, rh, 1.0f / 40320.0f);
  q = __fmaf_rn(q, rh, 1.0f / 5040.0f);
  // 1/6!, ..., 1/0! as two floats each
  const float ch[7] = {0x1.6c16c2p-10f, 0x1.111112p-7f, 0x1.555556p-5f, 0x1.555556p-3f, 0.5f, 1.0f, 1.0f};
  const float cl[7] = {-0x1.27d27ep-35f, -0x1.ddddep-32f, -0x1.555556p-30f, -0x1.555556p-28f, 0.0f, 0.0f, 0.0f};
  Two a{q, 0.0f};
#pragma unroll
  for (int i = 0; i < 7; ++i) {  // a = c + r a
    const float ph = __fmul_rn(rh, a.h);
    float pl = __fmaf_rn(rh, a.h, -ph);
    pl = __fmaf_rn(rh, a.l, pl);
    pl = __fmaf_rn(rl, a.h, pl);
    const float sum = __fadd_rn(ch[i], ph);
    a.l = __fadd_rn(__fsub_rn(ph, __fsub_rn(sum, ch[i])), __fadd_rn(pl, cl[i]));
    a.h = sum;
  }
  const float scale = __int_as_float((127 + (int)n) << 23);
  return Two{a.h * scale, a.l * scale};
}

// Scores to about 45 bits; far from zero, where two floats would leave their
// range, in fp64.
__device__ __noinline__ double exp_64(float hi, float lo) {
  if (hi < -60.0f) return exp((double)hi + (double)lo);
  const Two e = exp_two(hi, lo);
  return (double)e.h + (double)e.l;
}
__device__ __noinline__ double sigmoid_64(float x) {
  if (fabsf(x) > 60.0f) return 1.0 / (1.0 + exp(-(double)x));
  const Two e = exp_two(-fabsf(x), 0.0f);
  const float dh = __fadd_rn(1.0f, e.h);
  const float dl = __fadd_rn(__fsub_rn(e.h, __fsub_rn(dh, 1.0f)), e.l);
  const float r = __frcp_rn(dh);
  const float rl = __fmul_rn(r, __fmaf_rn(-dl, r, __fmaf_rn(-dh, r, 1.0f)));  // 1 / d = r + rl
  if (x >= 0.0f) return (double)r + (double)rl;
  const float ph = __fmul_rn(e.h, r);
  const float pl = __fmaf_rn(e.l, r, __fmaf_rn(e.h, rl, __fmaf_rn(e.h, r, -ph)));
  return (double)ph + (double)pl;
}

// One row again: the scores to 45 bits as doubles (whose order as integers is theirs), the
// definition step by step; lane j < k writes the j-th choice.
template <typename L, int V>
__device__ __noinline__ void exact_token(const L *row, int E, const float *bias, const GateArgs &a,
                                         int32_t *ids, float *w) {
  const int lane = threadIdx.x & 31;
  const Share<V> sh(E, a.n_groups, lane);
  uint64_t key[V];  // 0: none, 1: masked
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (i < sh.n) m = fmaxf(m, usable(load_logit(row + sh.e0 + i)));
  double z = 0.0;
  const bool softmax = a.score_fn == MOE_SCORE_SOFTMAX;
  // as in gate_kernel: the logits' order, where scores would vanish in fp64 too
  const bool by_logit = bias == nullptr && a.n_groups == 1;
  auto exp_of = [&](float l) {  // e^(l - m)
    if (l == -INFINITY) return 0.0;
    const float d = __fsub_rn(l, m), bb = __fsub_rn(d, l);
    if (d < -800.0f) return 0.0;
    return exp_64(d, __fsub_rn(__fsub_rn(l, __fsub_rn(d, bb)), __fadd_rn(m, bb)));
  };
  if (softmax) {
    m = warp_max(m);
    for (int i = 0; i < sh.n; ++i) z += exp_of(usable(load_logit(row + sh.e0 + i)));
    z = warp_sum(z);
  }
  const double zinv = z > 0.0 ? 1.0 / z : 0.0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    key[i] = 0;
    if (i < sh.n) {
      key[i] = 1;
      const float l = usable(load_logit(row + sh.e0 + i));
      if (l > -INFINITY) {
        double c = by_logit ? (double)l : softmax ? exp_of(l) * zinv : sigmoid_64(l);
        if (bias) c += clamp_bias(__ldg(bias + sh.e0 + i));
        key[i] = ordered(c);
      }
    }
  }
  // the first of this lane's largest keys, those in `used` left out
  auto head = [&](uint32_t used, int &at) {
    uint64_t best = 0;
    at = 0;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (!((used >> i) & 1u) && key[i] > best) {
        best = key[i];
        at = i;
      }
    return best;
  };
  int at;
  if (a.n_groups > 1) {
    uint32_t used = 0;
    double gs = -INFINITY;
    for (int r = 0; r < a.group_topn; ++r) {
      const uint64_t mine = head(used, at);
      const uint64_t best = sh.group_max(mine, lane);
      if (best > 1) gs = r == 0 ? unordered(best) : gs + unordered(best);
      if (__ffs(__ballot_sync(kFull, mine == best) & sh.members) - 1 == lane) used |= 1u << at;
    }
    const uint64_t gk = ordered(gs);
    int rank = 0;
    for (int g = 0; g < a.n_groups; ++g) {
      const uint64_t o = __shfl_sync(kFull, gk, g * sh.p);
      if (o > gk || (o == gk && g < sh.grp)) ++rank;
    }
    if (rank >= a.topk_groups || sh.grp >= a.n_groups) {
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = 0;
    }
  }
  uint32_t used = 0;
  int my_id = 0;
  for (int j = 0; j < a.k; ++j) {
    const uint64_t mine = head(used, at);
    const uint32_t hi = (uint32_t)(mine >> 32), lo = (uint32_t)mine;
    const uint32_t top = __reduce_max_sync(kFull, hi);
    const uint32_t low = __reduce_max_sync(kFull, hi == top ? lo : 0u);
    const int src = __ffs(__ballot_sync(kFull, hi == top && lo == low)) - 1;
    const int id = __shfl_sync(kFull, sh.e0 + at, src);
    if (lane == j) my_id = id;
    if (lane == src) used |= 1u << at;
  }
  const float my_l = lane < a.k ? usable(load_logit(row + my_id)) : -INFINITY;
  const float v = chosen_weight(a, my_l, m, (float)zinv);
  if (lane < a.k) {
    ids[lane] = my_id;
    w[lane] = v;
  }
}

// ------------------------------------------------------------ fp32 selection
// Descending sort of V (a power of two) keys: Batcher's odd-even merge network.
template <int V, typename K>
__device__ __forceinline__ void sort_keys(K (&k)[V]) {
#pragma unroll
  for (int p = 1; p < V; p <<= 1)
#pragma unroll
    for (int q = p; q >= 1; q >>= 1)
#pragma unroll
      for (int j = q % p; j + q < V; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < V && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const K hi = max(k[i + j], k[i + j + q]);
            k[i + j + q] = min(k[i + j], k[i + j + q]);
            k[i + j] = hi;
          }
}

template <int V, typename K>
__device__ __forceinline__ void pop(K (&k)[V], bool yes, K none = 0) {
#pragma unroll
  for (int i = 0; i + 1 < V; ++i) k[i] = yes ? k[i + 1] : k[i];
  if (yes) k[V - 1] = none;
}

// V logits from p (16-byte pieces where the launch says that they line up).
template <int V, bool VEC>
__device__ __forceinline__ void load_row(const float *p, int n, float (&l)[V]) {
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      float4 f = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (n > 0) f = __ldg(reinterpret_cast<const float4 *>(p + i));
      l[i] = f.x;
      l[i + 1] = f.y;
      l[i + 2] = f.z;
      l[i + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = i < n ? __ldg(p + i) : -INFINITY;
  }
}
template <int V, bool VEC>
__device__ __forceinline__ void load_row(const __nv_bfloat16 *p, int n, float (&l)[V]) {
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      uint2 u = make_uint2(0xFF80FF80u, 0xFF80FF80u);
      if (n > 0) u = __ldg(reinterpret_cast<const uint2 *>(p + i));
      l[i] = __uint_as_float(u.x << 16);
      l[i + 1] = __uint_as_float(u.x & 0xFFFF0000u);
      l[i + 2] = __uint_as_float(u.y << 16);
      l[i + 3] = __uint_as_float(u.y & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = i < n ? load_logit(p + i) : -INFINITY;
  }
}

template <typename L, int V, bool VEC>
__global__ void __launch_bounds__(256, V <= 8 ? 4 : 2)
    gate_kernel(const L *__restrict__ logits, int64_t ld, int64_t T, int E,
                const float *__restrict__ bias, GateArgs a, int32_t *__restrict__ ids,
                float *__restrict__ w) {
  moe::pdl_wait();
  moe::pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t warp0 = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int64_t nwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
  const Share<V> sh(E, a.n_groups, lane);
  const int e0 = sh.e0, n = sh.n;
  const bool softmax = a.score_fn == MOE_SCORE_SOFTMAX;
  // without bias and groups the scores' order is the logits'
  const bool by_logit = bias == nullptr && a.n_groups == 1;
  const bool need_z = softmax && (!by_logit || !a.renormalize);
  float b[V];
  if (bias != nullptr) {
#pragma unroll
    for (int i = 0; i < V; ++i) b[i] = i < n ? clamp_bias(__ldg(bias + e0 + i)) : 0.0f;
  }
  // Error bounds of a key's score c: kScoreErr of the row's largest s (fast
  // exponential, reciprocal or sum), and of |c| the bits given to the position
  // and the rounding of the addition.
  const float key_err = by_logit ? (V - 1) * 0x1p-23f : V * 0x1p-23f;
  const float score_err = by_logit ? 0.0f : softmax ? 1.2e-6f : 3e-7f;

  // Rows in doubt that the candidates do not settle are noted and come again
  // after 32 rows, out of this loop.
  for (int64_t first = warp0; first < T; first += 32 * nwarps) {
    uint32_t doubtful = 0;
    int64_t t = first;
    for (int it = 0; it < 32 && t < T; ++it, t += nwarps) {
      const L *row = logits + t * ld;
      float l[V];
      load_row<V, VEC>(row + e0, n, l);
      float m = -INFINITY, zinv = 1.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) l[i] = usable(l[i]);
      uint32_t key[V];
      float c[V];
      if (need_z) {
#pragma unroll
        for (int i = 0; i < V; ++i) m = fmaxf(m, l[i]);
        m = warp_max(m);
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] = exp_diff(l[i], m);
        float part[V];
#pragma unroll
        for (int i = 0; i < V; ++i) part[i] = c[i];
#pragma unroll
        for (int s = V / 2; s > 0; s >>= 1)
#pragma unroll
          for (int i = 0; i < s; ++i) part[i] += part[i + s];
        float z = part[0];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) z += __shfl_xor_sync(kFull, z, off);
        zinv = z > 0.0f ? __fdiv_rn(1.0f, z) : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float x = l[i];
        if (!by_logit) {
          x = softmax ? c[i] * zinv : rcp_fast(1.0f + exp2_fast(l[i] * -1.442695041f));
          if (bias != nullptr) x += b[i];
        }
        // a masked expert's key lies below every score's, that of no expert is 0
        const uint32_t k = l[i] > -INFINITY ? ordered(x + 0.0f) & ~(uint32_t)(V - 1) : (uint32_t)V;
        key[i] = i < n ? k | (uint32_t)(V - 1 - i) : 0u;
      }
      sort_keys<V>(key);
      bool sure = true;
      const float s_err = score_err * (softmax ? zinv : 1.0f);

      if (a.n_groups > 1) {
        // the group's group_topn largest scores, one round each
        uint32_t k2[V];
#pragma unroll
        for (int i = 0; i < V; ++i) k2[i] = key[i];
        float gs = 0.0f, size = 0.0f;
        bool any = false;
        for (int r = 0; r < a.group_topn; ++r) {
          const uint32_t h = sh.group_max(k2[0], lane);
          const uint32_t same = __ballot_sync(kFull, k2[0] == h) & sh.members;
          if (h >= 2u * V) {
            const float x = unordered(h & ~(uint32_t)(V - 1));
            gs += x;
            size += fabsf(x);
            any = true;
          }
          pop<V>(k2, lane == __ffs(same) - 1);
        }
        const bool valid = sh.grp < a.n_groups;
        if (!any) gs = -INFINITY;
        int rank = 0;
        for (int g = 0; g < a.n_groups; ++g) {
          const float o = __shfl_sync(kFull, gs, g * sh.p);
          if (o > gs || (o == gs && g < sh.grp)) ++rank;
        }
        const bool keep = valid && rank < a.topk_groups;
        const float err = a.group_topn * s_err + (key_err + a.group_topn * 0x1p-23f) * size;
        // the kept groups' least possible score against the others' largest
        const uint32_t least = __reduce_min_sync(kFull, keep ? ordered(any ? gs - err : gs) : 0xFFFFFFFFu);
        const uint32_t most =
            __reduce_max_sync(kFull, valid && !keep ? ordered(any ? gs + err : gs) : 0u);
        // (groups without an unmasked expert are exact ties, taken by id)
        if (a.topk_groups < a.n_groups && least <= most && most != ordered(-INFINITY)) sure = false;
        if (!keep) {
#pragma unroll
          for (int i = 0; i < V; ++i) key[i] = 0;
        }
      }

      uint32_t my_key = 0;
      int my_src = 0;
      auto take = [&](int j) {  // lane j receives the best key left
        // equal scores of several lanes: the lowest lane holds the lowest id
        const uint32_t head = key[0] & ~(uint32_t)(V - 1);
        const uint32_t top = __reduce_max_sync(kFull, head);
        const int src = __ffs(__ballot_sync(kFull, head == top)) - 1;
        const uint32_t won = __shfl_sync(kFull, key[0], src);
        if (lane == j) {
          my_key = won;
          my_src = src;
        }
        pop<V>(key, lane == src);
      };
      // Lane j < n: its key and the one after it may be the other way round
      // (a call of the whole warp).
      auto in_doubt = [&](int n) {
        uint32_t next = __shfl_down_sync(kFull, my_key, 1);
        const uint32_t rest = __reduce_max_sync(kFull, key[0]);  // the best one left out
        if (lane == n - 1) next = rest;
        const float x = unordered(my_key & ~(uint32_t)(V - 1));
        const float y = unordered(next & ~(uint32_t)(V - 1));
        const bool apart = x - y > 2.0f * s_err + key_err * (fabsf(x) + fabsf(y));
        return lane < n && next >= 2u * V && !apart;
      };
      for (int j = 0; j < a.k; ++j) take(j);
      bool doubt = false;
      // bf16 logits keep all their bits in a key: their order is exact
      if (!(by_logit && sizeof(L) == 2)) doubt = __any_sync(kFull, in_doubt(a.k));
      int n_cand = a.k;
      if (doubt && (bias == nullptr || !softmax)) {
        // four more candidates; a clear gap after them leaves the rest out
        n_cand = min(a.k + 4, 32);
        for (int j = a.k; j < n_cand; ++j) take(j);
        const bool open = in_doubt(n_cand);  // (every lane takes part)
        if (__any_sync(kFull, open && lane == n_cand - 1)) sure = false;
      } else if (doubt) {
        sure = false;  // a softmax's score takes the whole row again
      }
      int my_id = __shfl_sync(kFull, e0, my_src) + (V - 1 - (int)(my_key & (V - 1)));
      float my_l = lane < n_cand && my_key != 0 ? usable(load_logit(row + my_id)) : -INFINITY;
      // scores that vanish in fp64 are exact ties, among experts left out too
      if (doubt && bias == nullptr && a.n_groups > 1 &&
          __any_sync(kFull, my_l > -INFINITY && my_l - (softmax ? m : 0.0f) < -700.0f))
        sure = false;
      if (doubt && sure) {
        // one candidate a lane: the logits in order (scores rise with them)
        // without a bias, else the scores to 45 bits; ties by id
        double c = my_l;
        if (bias != nullptr && my_l > -INFINITY)
          c = sigmoid_64(my_l) + clamp_bias(__ldg(bias + my_id));
        const int id = lane < n_cand && my_key != 0 ? my_id : 0x7FFFFFFF;
        int rank = 0;
        for (int j = 0; j < n_cand; ++j) {
          const double oc = __shfl_sync(kFull, c, j);
          const int oid = __shfl_sync(kFull, id, j);
          if (oc > c || (oc == c && oid < id)) ++rank;
        }
        const float l0 = my_l;
        for (int j = 0; j < n_cand; ++j) {
          const int r = __shfl_sync(kFull, rank, j), oid = __shfl_sync(kFull, id, j);
          const float ol = __shfl_sync(kFull, l0, j);
          if (lane == r) {
            my_id = oid;
            my_l = ol;
          }
        }
      }
      if (lane >= a.k) my_l = -INFINITY;
      if (!__all_sync(kFull, sure)) doubtful |= 1u << it;
      const float v = chosen_weight(a, my_l, m, zinv);
      if (lane < a.k) {
        ids[t * a.k + lane] = my_id;
        w[t * a.k + lane] = v;
      }
    }
    for (; doubtful != 0; doubtful &= doubtful - 1) {
      const int64_t u = first + (__ffs(doubtful) - 1) * nwarps;
      exact_token<L, V>(logits + u * ld, E, bias, a, ids + u * a.k, w + u * a.k);
    }
  }
}

// ------------------------------------------------------- many tokens at once
// Four lanes a token, eight tokens a warp: what a warp does once a token in
// gate_kernel (rounds, checks, weights) it does here once for eight.  Lane q
// of a token holds experts [q P, (q + 1) P), P = E / 4, as GL whole groups (or,
// without groups, a quarter of the row), and goes through them in batches of
// eight: sort the batch, keep the eight largest of it and the group's list.
// Where all eight choices are one lane's, its list is empty when the last of
// them is compared with the best expert left out, so the largest key that a
// list let go is kept beside it.
//
// Keys are fixed-point numbers, c 2^28 rounded down to 32 bits, the low bits
// that count to P given to the place in the lane: 2^-22 of |c| < 8 at P = 64,
// where a float key would lose 2^-17 of c.  Scores beyond that range stay at its ends: among
// themselves they count as ties, which are in doubt like any other, and a group
// whose score they enter puts its row in doubt.  Keys below kLow are masked
// experts (kMasked and a place) and none (kNone).
constexpr int kManyThreads = 256;

constexpr int kManyMaxP = 128;  // E <= 512
constexpr int32_t kNone = (int32_t)0x80000000, kMasked = kNone + kManyMaxP,
                  kLow = kNone + 4 * kManyMaxP;

// Descending bitonic merge of eight keys that first fall and then rise.
__device__ __forceinline__ void merge8(int32_t (&k)[8]) {
#pragma unroll
  for (int d = 4; d >= 1; d >>= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((i & d) == 0) {
        const int32_t hi = max(k[i], k[i + d]);
        k[i + d] = min(k[i], k[i + d]);
        k[i] = hi;
      }
}

// The eight largest of two descending lists, descending; ninth becomes the
// largest key left out where that is larger.
__device__ __forceinline__ void merge_top8(int32_t (&a)[8], const int32_t (&b)[8], int32_t &ninth) {
  int32_t out[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    out[i] = min(a[i], b[7 - i]);
    a[i] = max(a[i], b[7 - i]);
  }
  ninth = __vimax3_s32(__vimax3_s32(out[0], out[1], out[2]), __vimax3_s32(out[3], out[4], out[5]),
                       __vimax3_s32(out[6], out[7], ninth));
  merge8(a);
}

__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(kFull, x, 1));
  return fmaxf(x, __shfl_xor_sync(kFull, x, 2));
}
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(kFull, x, 1);
  return x + __shfl_xor_sync(kFull, x, 2);
}
__device__ __forceinline__ int32_t quad_max(int32_t x) {
  x = max(x, __shfl_xor_sync(kFull, x, 1));
  return max(x, __shfl_xor_sync(kFull, x, 2));
}
__device__ __forceinline__ int32_t quad_min(int32_t x) {
  x = min(x, __shfl_xor_sync(kFull, x, 1));
  return min(x, __shfl_xor_sync(kFull, x, 2));
}

__device__ __forceinline__ void load8(const float *p, float (&l)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4 *>(p));
  const float4 b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
  l[0] = a.x, l[1] = a.y, l[2] = a.z, l[3] = a.w;
  l[4] = b.x, l[5] = b.y, l[6] = b.z, l[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&l)[8]) {
  const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p));
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    l[2 * i] = __uint_as_float(w[i] << 16);
    l[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

template <typename L>
__device__ __forceinline__ void exact_token_of(const L *row, int E, const float *bias,
                                               const GateArgs &a, int32_t *ids, float *w) {
  if (E <= 32)
    exact_token<L, 1>(row, E, bias, a, ids, w);
  else if (E <= 64)
    exact_token<L, 2>(row, E, bias, a, ids, w);
  else if (E <= 128)
    exact_token<L, 4>(row, E, bias, a, ids, w);
  else if (E <= 256)
    exact_token<L, 8>(row, E, bias, a, ids, w);
  else
    exact_token<L, 16>(row, E, bias, a, ids, w);
}

template <typename L, int GL>
__global__ void __launch_bounds__(kManyThreads, 3)
    gate_many_kernel(const L *__restrict__ logits, int64_t ld, int64_t T, int E,
                     const float *__restrict__ bias, GateArgs a, int32_t *__restrict__ ids,
                     float *__restrict__ w) {
  const int P = E / 4, NB = P / 8, NBG = NB / GL;
  const int32_t place = (1 << (32 - __clz(P - 1))) - 1;  // the bits of a place
  const int pad = P + 4;  // a lane's biases (times 2^28), off the other lanes' banks
  __shared__ __align__(16) float bias_s[4 * (kManyMaxP + 4)];
  moe::pdl_wait();
  moe::pdl_trigger();
  for (int e = threadIdx.x; e < E; e += kManyThreads)
    bias_s[e / P * pad + e % P] = bias != nullptr ? clamp_bias(__ldg(bias + e)) * 0x1p28f : 0.0f;
  __syncthreads();
  const int lane = threadIdx.x & 31, q = lane & 3;
  const uint32_t quad = 0xFu << (lane & 28);
  const int64_t warp0 = ((int64_t)blockIdx.x * kManyThreads + threadIdx.x) >> 5;
  const int64_t nwarps = ((int64_t)gridDim.x * kManyThreads) >> 5;
  const bool softmax = a.score_fn == MOE_SCORE_SOFTMAX;
  const float *my_bias = bias_s + q * pad;

  for (int64_t first = warp0 * 8; first < T; first += nwarps * 32) {
    uint32_t doubtful = 0;  // a bit a token, eight a turn
    int64_t t8 = first;
    for (int turn = 0; turn < 4 && t8 < T; ++turn, t8 += nwarps * 8) {
      const bool real = t8 + (lane >> 2) < T;
      const int64_t t = real ? t8 + (lane >> 2) : T - 1;
      const L *row = logits + t * ld + q * P;
      float m = -INFINITY, zinv = 1.0f;
      if (softmax) {
#pragma unroll 2
        for (int b = 0; b < NB; ++b) {
          float l[8];
          load8(row + 8 * b, l);
#pragma unroll
          for (int i = 0; i < 8; ++i) m = fmaxf(m, usable(l[i]));
        }
        m = quad_max(m);
        float z = 0.0f;
#pragma unroll 1
        for (int b = 0; b < NB; ++b) {
          float l[8];
          load8(row + 8 * b, l);
#pragma unroll
          for (int i = 0; i < 8; ++i) l[i] = exp_diff(usable(l[i]), m);
          z += ((l[0] + l[1]) + (l[2] + l[3])) + ((l[4] + l[5]) + (l[6] + l[7]));
        }
        z = quad_sum(z);
        zinv = z > 0.0f ? __fdiv_rn(1.0f, z) : 0.0f;
      }
      int32_t list[GL][8], ninth[GL];  // (the largest key that the list let go)
#pragma unroll
      for (int g = 0; g < GL; ++g) {
        ninth[g] = kNone;
#pragma unroll
        for (int i = 0; i < 8; ++i) list[g][i] = kNone;
#pragma unroll 1
        for (int b = 0; b < NBG; ++b) {
          const int at = (g * NBG + b) * 8;
          float l[8], bb[8];
          load8(row + at, l);
          *reinterpret_cast<float4 *>(bb) = *reinterpret_cast<const float4 *>(my_bias + at);
          *reinterpret_cast<float4 *>(bb + 4) = *reinterpret_cast<const float4 *>(my_bias + at + 4);
          int32_t key[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float x = l[i];
            const float s = softmax ? exp2_fast((fminf(x, m) - m) * 1.442695041f) * zinv
                                    : rcp_fast(1.0f + exp2_fast(x * -1.442695041f));
            const int32_t k = max(__float2int_rd(__fmaf_rn(s, 0x1p28f, bb[i])), kLow);
            // (a NaN fails the comparison)
            key[i] = (x > -INFINITY ? k & ~place : kMasked) | (place - (at + i));
          }
          sort_keys<8>(key);
          merge_top8(list[g], key, ninth[g]);
        }
      }
      // What a key may be off by: its place and rounding, the score (see
      // gate_kernel; a softmax's are at most zinv) and the addition.
      const uint32_t err = place + (uint32_t)((softmax ? 1.2e-6f * zinv : 3e-7f) * 0x1p28f) + 130u;
      bool sure = true;

      if (a.n_groups > 1) {
        // a group's score, halved: c as in the keys, 0 for what is masked
        int32_t gs[GL];
        int rank[GL];
        const int32_t top = 0x7FFFFFFF - place;
        bool end = false;  // a score at an end of the range
#pragma unroll
        for (int g = 0; g < GL; ++g) {
          const int32_t k0 = list[g][0], k1 = list[g][1];
          gs[g] = k0 < kLow ? kNone : k0 >> 1;
          if (k0 >= kLow) end |= k0 <= kLow + place || k0 >= top;
          if (a.group_topn > 1 && k1 >= kLow) {
            gs[g] += k1 >> 1;
            end |= k1 <= kLow + place || k1 >= top;
          }
          rank[g] = 0;
        }
        if (end) sure = false;
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
          for (int h = 0; h < GL; ++h) {
            const int32_t o = __shfl_xor_sync(kFull, gs[h], d);
            const int id = (q ^ d) * GL + h;
#pragma unroll
            for (int g = 0; g < GL; ++g)
              if (o > gs[g] || (o == gs[g] && id < q * GL + g)) ++rank[g];
          }
        int32_t least = 0x7FFFFFFF, most = kNone;
#pragma unroll
        for (int g = 0; g < GL; ++g) {
          const bool keep = rank[g] < a.topk_groups;
          if (keep)
            least = min(least, gs[g]);
          else
            most = max(most, gs[g]);
          if (!keep) ninth[g] = kNone;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (!keep) list[g][i] = kNone;
        }
        least = quad_min(least);
        most = quad_max(most);
        // (groups without an unmasked expert are exact ties, taken by id)
        if (a.topk_groups < a.n_groups && most != kNone &&
            (uint32_t)least - (uint32_t)most <= 2 * err + 4)
          sure = false;
      }
#pragma unroll
      for (int g = 1; g < GL; ++g) {
        merge_top8(list[0], list[g], ninth[0]);
        ninth[0] = max(ninth[0], ninth[g]);
      }

      int32_t my_key[2] = {0, 0}, last = 0;
      uint32_t close = 0;  // bit j: entries j and j + 1
      int my_q[2] = {0, 0};
      for (int j = 0; j <= a.k; ++j) {
        // (at least what the list let go, unless all its eight entries are taken)
        const int32_t head = max(list[0][0], ninth[0]) & ~place;
        const int32_t best = quad_max(head);
        if (j > 0 && best >= kLow && (uint32_t)last - (uint32_t)best <= 2 * err)
          close |= 1u << (j - 1);
        if (j == a.k) break;
        last = best;
        const int src = __ffs(__ballot_sync(kFull, head == best) & quad) - 1;
        const int32_t won = __shfl_sync(kFull, list[0][0], src);
        if ((j & 3) == q) {
          if (j < 4) {
            my_key[0] = won;
            my_q[0] = src & 3;
          } else {
            my_key[1] = won;
            my_q[1] = src & 3;
          }
        }
        pop<8>(list[0], lane == src, kNone);
      }
      // entries q and q + 4
      int my_id[2];
      float my_l[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        my_id[s] = my_q[s] * P + (place - (my_key[s] & place));
        my_l[s] = 4 * s + q < a.k ? usable(load_logit(logits + t * ld + my_id[s])) : -INFINITY;
      }
      if (__any_sync(kFull, close != 0)) {
        // equal logits with equal biases are exact ties, already by id
        float my_b[2], nl[2], nb[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) my_b[s] = bias_s[my_id[s] + 4 * my_q[s]];
        const int next = (lane & 28) | ((q + 1) & 3);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          // entry q + 1 of the same four, or the first of the other four
          const float l0 = __shfl_sync(kFull, my_l[s], next), l1 = __shfl_sync(kFull, my_l[1], next);
          const float b0 = __shfl_sync(kFull, my_b[s], next), b1 = __shfl_sync(kFull, my_b[1], next);
          nl[s] = q < 3 ? l0 : l1;
          nb[s] = q < 3 ? b0 : b1;
        }
        uint32_t open = close;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int j = 4 * s + q;
          if (j < a.k - 1 && my_l[s] == nl[s] && my_b[s] == nb[s]) open &= ~(1u << j);
        }
        open &= __shfl_xor_sync(kFull, open, 1);
        open &= __shfl_xor_sync(kFull, open, 2);
        if (open != 0) sure = false;
      }
      // any lane of a token speaks for it: bits 4 i ... 4 i + 3 to bit i
      uint32_t bits = __ballot_sync(kFull, !sure && real);
      bits |= bits >> 1;
      bits = (bits | bits >> 2) & 0x11111111u;
      bits = (bits | bits >> 3) & 0x03030303u;
      bits = (bits | bits >> 6) & 0x000F000Fu;
      bits = (bits | bits >> 12) & 0xFFu;
      doubtful |= bits << (8 * turn);

      // weights, as chosen_weight
      float v[2];
      if (softmax) {
        const float ml = a.renormalize ? quad_max(fmaxf(my_l[0], my_l[1])) : m;
        v[0] = exp_diff(my_l[0], ml);
        v[1] = exp_diff(my_l[1], ml);
      } else {
        v[0] = sigmoid32(my_l[0]);
        v[1] = sigmoid32(my_l[1]);
        const uint32_t tiny = __ballot_sync(kFull, tiny_logit(my_l[0]) || tiny_logit(my_l[1]));
        if (a.renormalize && tiny != 0) {
          const float ml = quad_max(fmaxf(my_l[0], my_l[1]));
          if ((tiny & quad) != 0 && ml < 0.0f) {
            v[0] = sigmoid_rel(my_l[0], ml);
            v[1] = sigmoid_rel(my_l[1], ml);
          }
        }
      }
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (4 * s + q >= a.k) v[s] = 0.0f;
      float f = softmax ? zinv : 1.0f;
      if (a.renormalize) {
        const float den = quad_sum(v[0] + v[1]);
        f = den > 0.0f ? rcp_fast(den) : 0.0f;
      }
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (real && 4 * s + q < a.k) {
          ids[t * a.k + 4 * s + q] = my_id[s];
          w[t * a.k + 4 * s + q] = a.scale * (v[s] * f);
        }
    }
    __syncwarp();  // the rows' first results are written
    for (; doubtful != 0; doubtful &= doubtful - 1) {
      const int i = __ffs(doubtful) - 1;
      const int64_t u = first + (i >> 3) * nwarps * 8 + (i & 7);
      exact_token_of<L>(logits + u * ld, E, bias, a, ids + u * a.k, w + u * a.k);
    }
  }
}

// Gradient of the logits for a gradient g of the weights (the selection and
// the bias carry none).  With v the renormalised weights without scale:
//   sigmoid            dl_e = scale g_e s_e (1 - s_e)                selected e
//   sigmoid, renorm    dl_e = scale (g_e - sum g v) v_e (1 - s_e)    selected e
//   softmax            dl_e = s_e (scale g_e [selected] - scale sum g s)  all e
//   softmax, renorm    dl_e = scale (g_e - sum g v) v_e              selected e
// A warp takes TPW tokens at once, 32 / TPW lanes for the choices of each, so
// that the loads of ids, logits and gradients (one behind the other) of several
// tokens are in flight: 65536 fp32 rows of 256, renormalised, 20.6 us (30.6 us with
// one token at a time), every expert's score 44 us; 10 and 20 us are what the
// bytes take.  The zeros' stores wait for that chain, and the loads and stores of
// whole rows are 4 bytes a lane.  A row is first written whole (zeros, or -s_e
// scale sum g s), then lane j < k of its token overwrites the j-th chosen
// expert's entry.
template <int LPT>
__device__ __forceinline__ float part_sum(float x) {
#pragma unroll
  for (int off = LPT / 2; off > 0; off >>= 1) x += __shfl_xor_sync(kFull, x, off);
  return x;
}
template <int LPT>
__device__ __forceinline__ float part_max(float x) {
#pragma unroll
  for (int off = LPT / 2; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, off));
  return x;
}

template <typename L, int VPL, int TPW>
__global__ void __launch_bounds__(256)
    gate_backward_kernel(const L *__restrict__ logits, int64_t ld, int64_t T, int E,
                         const int32_t *__restrict__ ids, const float *__restrict__ grad_w,
                         GateArgs a, L *__restrict__ grad_logits, int32_t *status) {
  moe::pdl_wait();
  moe::pdl_trigger();
  constexpr int LPT = 32 / TPW;
  const int lane = threadIdx.x & 31, sub = lane / LPT, j = lane % LPT;
  const int64_t warp0 = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int64_t nwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
  const bool softmax = a.score_fn == MOE_SCORE_SOFTMAX;
  const bool dense = softmax && !a.renormalize;
  for (int64_t t0 = warp0 * TPW; t0 < T; t0 += nwarps * TPW) {
    const int64_t t = t0 + sub;
    const int n = (int)(T - t0 < TPW ? T - t0 : TPW);  // tokens of this turn
    int id = -1;
    float g = 0.0f, my_l = -INFINITY;
    if (sub < n && j < a.k) {
      id = __ldg(ids + t * a.k + j);
      g = a.scale * __ldg(grad_w + t * a.k + j);
      if (id < 0 || id >= E) {
        moe::report_error(status, MOE_ERR_DEVICE_INDEX, (int32_t)(t * a.k + j), moe::K_GATE);
        id = -1;
        g = 0.0f;
      } else {
        my_l = usable(load_logit(logits + t * ld + id));
      }
    }
    const bool live = my_l > -INFINITY;
    float mine = 0.0f;  // this lane's entry
    if (dense) {
      float x[TPW][VPL], zinv[TPW], my_m = 0.0f, my_zinv = 0.0f;
#pragma unroll
      for (int s = 0; s < TPW; ++s)
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          const int e = lane + 32 * i;
          x[s][i] = s < n && e < E ? usable(load_logit(logits + (t0 + s) * ld + e)) : -INFINITY;
        }
#pragma unroll
      for (int s = 0; s < TPW; ++s) {
        float m = -INFINITY, z = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) m = fmaxf(m, x[s][i]);
        m = warp_max(m);
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          x[s][i] = exp_diff(x[s][i], m);
          z += x[s][i];
        }
        z = part_sum<32>(z);
        zinv[s] = z > 0.0f ? __fdiv_rn(1.0f, z) : 0.0f;
        if (sub == s) {
          my_m = m;
          my_zinv = zinv[s];
        }
      }
      const float p = live ? exp_diff(my_l, my_m) * my_zinv : 0.0f;
      const float dot = part_sum<LPT>(g * p);
      mine = p * (g - dot);
#pragma unroll
      for (int s = 0; s < TPW; ++s) {
        const float f = zinv[s] * __shfl_sync(kFull, dot, s * LPT);
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          const int e = lane + 32 * i;
          if (s < n && e < E) store_grad(grad_logits + (t0 + s) * E + e, -x[s][i] * f);
        }
      }
    } else {
      float num = 0.0f, q = 1.0f;  // q = 1 - s
      if (!softmax && live) {
        num = sigmoid32(my_l);
        q = sigmoid32(-my_l);
      }
      if (a.renormalize) {
        const float ml = part_max<LPT>(my_l);
        const uint32_t tiny = __ballot_sync(kFull, tiny_logit(my_l));
        const uint32_t part = (LPT == 32 ? kFull : (1u << LPT) - 1u) << (sub * LPT);
        if (softmax)
          num = live ? exp_diff(my_l, ml) : 0.0f;
        else if ((tiny & part) != 0 && ml < 0.0f)
          num = live ? sigmoid_rel(my_l, ml) : 0.0f;
        const float den = part_sum<LPT>(num);
        const float v = den > 0.0f ? __fdiv_rn(num, den) : 0.0f;
        const float dot = part_sum<LPT>(g * v);
        mine = (g - dot) * v * q;
      } else {
        mine = g * num * q;
      }
      // zeros: the turn's rows lie one after the other
      L *out = grad_logits + t0 * E;
      const int64_t bytes = (int64_t)n * E * sizeof(L);
      if ((reinterpret_cast<uintptr_t>(out) | bytes) % 16 == 0) {
        for (int64_t i = lane; i < bytes / 16; i += 32)
          reinterpret_cast<uint4 *>(out)[i] = make_uint4(0, 0, 0, 0);
      } else {
        for (int64_t i = lane; i < (int64_t)n * E; i += 32) store_grad(out + i, 0.0f);
      }
    }
    __syncwarp();  // the rows' stores come before the overwriting ones
    if (id >= 0) store_grad(grad_logits + t * E + id, mine);
  }
}

// b_e + rate * sign(mean load - load_e): the mean is compared as total
// against E * load, in integers.
__global__ void __launch_bounds__(512) gate_update_bias_kernel(const int32_t *__restrict__ counts,
                                                               int E, const float *bias, float rate,
                                                               float *bias_out) {
  moe::pdl_wait();
  moe::pdl_trigger();
  __shared__ long long part[16];
  const int e = threadIdx.x;
  const long long n = e < E ? counts[e] : 0;
  long long total = n;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(kFull, total, off);
  if ((e & 31) == 0) part[e >> 5] = total;
  __syncthreads();
  if (e < E) {
    total = 0;
    for (int i = 0; i < 16; ++i) total += part[i];
    const long long d = total - (long long)E * n;
    bias_out[e] = bias[e] + (d > 0 ? rate : d < 0 ? -rate : 0.0f);
  }
}

// ------------------------------------------------------------------ host
moe_status check_cfg(const moe_gate_cfg *cfg, int32_t logits_type, int64_t T, int32_t E,
                     int64_t ld) {
  if (cfg == nullptr || T < 0 || E < 1 || ld < E) return MOE_ERR_INVALID_ARG;
  if (logits_type != MOE_F32 && logits_type != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (cfg->score_fn != MOE_SCORE_SOFTMAX && cfg->score_fn != MOE_SCORE_SIGMOID)
    return MOE_ERR_INVALID_ARG;
  if (cfg->k < 1 || cfg->k > E || cfg->n_groups < 1 || (cfg->renormalize & ~1))
    return MOE_ERR_INVALID_ARG;
  if (!(cfg->scale > 0.0f) || cfg->scale > FLT_MAX) return MOE_ERR_INVALID_ARG;
  if (cfg->k > 16 || E > 512 || cfg->n_groups > 32 || E % cfg->n_groups != 0)
    return MOE_ERR_UNSUPPORTED;
  const int gsz = E / cfg->n_groups;
  if (cfg->topk_groups < 1 || cfg->topk_groups > cfg->n_groups) return MOE_ERR_INVALID_ARG;
  if (cfg->group_topn < 1 || cfg->group_topn > gsz) return MOE_ERR_INVALID_ARG;
  if (cfg->group_topn > kMaxTopn) return MOE_ERR_UNSUPPORTED;
  if (cfg->k > cfg->topk_groups * gsz) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

GateArgs args_of(const moe_gate_cfg *c) {
  return GateArgs{c->score_fn,   c->k,           c->n_groups, c->topk_groups,
                  c->group_topn, c->renormalize, c->scale};
}

// Blocks of 8 warps, a token each at a time: at most as many as are resident
// together (per_sm of each SM), so that all warps take as many tokens.
unsigned gate_grid(int64_t T, int per_sm) {
  int64_t blocks = (T + 7) / 8;
  const int64_t cap = (int64_t)moe_host::sm_count() * per_sm;
  return (unsigned)(blocks > cap ? cap : blocks);
}

// Calls f with the smallest of 1, 2, 4, 8, 16, 32 that is at least n, as a type.
template <int N>
struct Int {
  static constexpr int value = N;
};
template <typename F>
moe_status by_size(int n, F &&f) {
  if (n <= 1) return f(Int<1>{});
  if (n <= 2) return f(Int<2>{});
  if (n <= 4) return f(Int<4>{});
  if (n <= 8) return f(Int<8>{});
  if (n <= 16) return f(Int<16>{});
  return f(Int<32>{});
}

// gate_many_kernel's cases: a row in four equal parts of whole batches and
// whole groups, 16-byte loads.  Fewer tokens than kManyTokens leave SMs idle
// and take a warp each: 256 experts in 8 groups, 4096 tokens 9.8 us with a warp
// a token against 14.9 us here, 8192 tokens 19 against 15 us, 65536 78 against
// 39 us; 32 experts 3.7 and 5.7, 7.1 and 5.8, 27 and 15 us.
constexpr int64_t kManyTokens = 8192;

template <typename L>
bool many_fits(const void *logits, int64_t ld, int64_t T, int E, const float *bias,
               const GateArgs &a) {
  const int G = a.n_groups;
  return T >= kManyTokens && E % 32 == 0 && a.k <= 8 && a.group_topn <= 2 &&
         (G == 1 ? bias != nullptr
                 : G % 4 == 0 && G <= 16 && G != 12 && E / G % 8 == 0) &&
         ld % 8 == 0 && reinterpret_cast<uintptr_t>(logits) % 16 == 0;
}

template <typename L, int GL>
moe_status launch_many_parts(const void *logits, int64_t ld, int64_t T, int E, const float *bias,
                             GateArgs a, int32_t *ids, float *w, cudaStream_t st) {
  constexpr int per_block = kManyThreads / 4;
  int64_t blocks = (T + per_block - 1) / per_block;
  // four times as many as are resident: a block that meets a row in doubt takes
  // longer, and others take its place (65536 tokens: 13% less than with three an SM)
  const int64_t cap = (int64_t)moe_host::sm_count() * 12;
  if (blocks > cap) blocks = cap;
  return moe_host::launch_pdl(gate_many_kernel<L, GL>, dim3((unsigned)blocks), dim3(kManyThreads),
                              0, st, static_cast<const L *>(logits), ld, T, E, bias, a, ids, w);
}

template <typename L>
moe_status launch_many(const void *logits, int64_t ld, int64_t T, int E, const float *bias,
                       GateArgs a, int32_t *ids, float *w, cudaStream_t st) {
  if (a.n_groups == 16) return launch_many_parts<L, 4>(logits, ld, T, E, bias, a, ids, w, st);
  if (a.n_groups == 8) return launch_many_parts<L, 2>(logits, ld, T, E, bias, a, ids, w, st);
  return launch_many_parts<L, 1>(logits, ld, T, E, bias, a, ids, w, st);
}

template <typename L>
moe_status launch_gate(const void *logits, int64_t ld, int64_t T, int E, const float *bias,
                       GateArgs a, int32_t *ids, float *w, cudaStream_t st) {
  if (many_fits<L>(logits, ld, T, E, bias, a))
    return launch_many<L>(logits, ld, T, E, bias, a, ids, w, st);
  const L *l = static_cast<const L *>(logits);
  const int gsz = E / a.n_groups, p = 32 / a.n_groups;
  return by_size((gsz + p - 1) / p, [&](auto v) {
    constexpr int V = decltype(v)::value;
    auto run = [&](auto kernel) {
      return moe_host::launch_pdl(kernel, dim3(gate_grid(T, V <= 8 ? 4 : 2)), dim3(256), 0, st, l,
                                  ld, T, E, bias, a,
                                  ids, w);
    };
    if constexpr (V >= 4) {
      // four logits a load: every lane's experts start on a multiple of four
      // in memory and none has a part of its V
      if (gsz % V == 0 && ld % 4 == 0 &&
          reinterpret_cast<uintptr_t>(logits) % (4 * sizeof(L)) == 0)
        return run(gate_kernel<L, V, true>);
    }
    return run(gate_kernel<L, V, false>);
  });
}

template <typename L>
moe_status launch_backward(const void *logits, int64_t ld, int64_t T, int E, const int32_t *ids,
                           const float *g, GateArgs a, void *out, int32_t *status,
                           cudaStream_t st) {
  return by_size((E + 31) / 32, [&](auto v) {
    constexpr int VPL = decltype(v)::value > 16 ? 16 : decltype(v)::value;
    constexpr int TPW = VPL > 8 ? 2 : 4;  // rows of up to 512 values in registers
    auto run = [&](auto kernel, int tpw) {
      return moe_host::launch_pdl(kernel, dim3(gate_grid((T + tpw - 1) / tpw, 8)), dim3(256), 0, st,
                                  static_cast<const L *>(logits), ld, T, E, ids, g, a,
                                  static_cast<L *>(out), status);
    };
    // two at once where a token's choices need 16 lanes, or where four rows in
    // registers cost more than they hide (256 experts, 65536 tokens: 47 us)
    const bool dense = a.score_fn == MOE_SCORE_SOFTMAX && !a.renormalize;
    return a.k <= 8 && !(dense && VPL >= 8) ? run(gate_backward_kernel<L, VPL, TPW>, TPW)
                                            : run(gate_backward_kernel<L, VPL, 2>, 2);
  });
}

}  // namespace

extern "C" moe_status moe_gate(const void *logits, int32_t logits_type, int64_t ld, int64_t T,
                               int32_t E, const float *bias, const moe_gate_cfg *cfg,
                               int32_t *topk_ids, float *topk_w, void *stream) {
  if (moe_status s = check_cfg(cfg, logits_type, T, E, ld)) return s;
  if (T == 0) return MOE_OK;
  if (!logits || !topk_ids || !topk_w) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return logits_type == MOE_F32
             ? launch_gate<float>(logits, ld, T, E, bias, args_of(cfg), topk_ids, topk_w, st)
             : launch_gate<__nv_bfloat16>(logits, ld, T, E, bias, args_of(cfg), topk_ids, topk_w, st);
}

extern "C" moe_status moe_gate_backward(const void *logits, int32_t logits_type, int64_t ld,
                                        int64_t T, int32_t E, const int32_t *topk_ids,
                                        const float *grad_w, const moe_gate_cfg *cfg,
                                        void *grad_logits, void *ws, size_t ws_bytes,
                                        void *stream) {
  if (moe_status s = check_cfg(cfg, logits_type, T, E, ld)) return s;
  if (moe_status s = moe_host::check_ws(ws, ws_bytes, moe::kStatusBytes)) return s;
  if (T == 0) return MOE_OK;
  if (!logits || !topk_ids || !grad_w || !grad_logits) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int32_t *status = moe_host::status_ptr(ws);
  return logits_type == MOE_F32
             ? launch_backward<float>(logits, ld, T, E, topk_ids, grad_w, args_of(cfg), grad_logits,
                                      status, st)
             : launch_backward<__nv_bfloat16>(logits, ld, T, E, topk_ids, grad_w, args_of(cfg),
                                              grad_logits, status, st);
}

extern "C" moe_status moe_gate_update_bias(const int32_t *counts, int32_t E, const float *bias,
                                           float rate, float *bias_out, void *stream) {
  if (E < 1 || !(rate >= 0.0f) || rate > FLT_MAX || !counts || !bias || !bias_out)
    return MOE_ERR_INVALID_ARG;
  if (E > 512) return MOE_ERR_UNSUPPORTED;
  return moe_host::launch_pdl(gate_update_bias_kernel, dim3(1), dim3(512), 0,
                              static_cast<cudaStream_t>(stream), counts, (int)E, bias, rate,
                              bias_out);
}
