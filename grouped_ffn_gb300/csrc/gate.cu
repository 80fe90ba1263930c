// Router with a balance bias: scores, selection and weights for every token
// (moe_gate), the gradient of the logits (moe_gate_backward) and the bias
// update from expert loads (moe_gate_update_bias).
//
//   s_e = softmax(l)_e or sigmoid(l_e),   c_e = s_e + b_e
//   groups by the sum of their group_topn largest c, then the k largest c of
//   the kept groups (ties: lower id);   w = scale s  or  scale s / sum_k s.
//
// One warp per token; lane L holds experts L, L + 32, ... (VPL each).
#include <cuda_bf16.h>

#include <cfloat>
#include <climits>

#include "common.cuh"

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kMaxTopn = 8;
constexpr float kBiasClamp = 1e30f;  // group sums of clamped biases stay finite
// below this largest selected logit, sigmoid(l) is e^l to fp32 precision and
// the renormalised weights are taken from e^(l - max l), which cannot vanish
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
__device__ __forceinline__ float usable(float x) { return x > -INFINITY ? fminf(x, FLT_MAX) : -INFINITY; }

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

// Arg-max over the warp of the values whose bit is set in mask (element i of
// this lane is id lane + 32 i): the largest value, ties to the lower id.
template <int VPL>
__device__ __forceinline__ void warp_argmax(const double (&v)[VPL], uint32_t mask, int lane,
                                            double &bv, int &bid) {
  bv = 0.0;
  bid = INT_MAX;
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    if (((mask >> i) & 1u) && (bid == INT_MAX || v[i] > bv)) {
      bv = v[i];
      bid = lane + 32 * i;
    }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const double ov = __shfl_xor_sync(kFull, bv, off);
    const int oid = __shfl_xor_sync(kFull, bid, off);
    if (oid != INT_MAX && (bid == INT_MAX || ov > bv || (ov == bv && oid < bid))) {
      bv = ov;
      bid = oid;
    }
  }
}

template <typename L, int VPL>
__global__ void __launch_bounds__(256) gate_kernel(const L *__restrict__ logits, int64_t ld,
                                                   int64_t T, int E,
                                                   const float *__restrict__ bias, GateArgs a,
                                                   int32_t *__restrict__ ids,
                                                   float *__restrict__ w) {
  moe::pdl_wait();
  moe::pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t warp0 = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int64_t nwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
  const int gsz = E / a.n_groups;
  for (int64_t t = warp0; t < T; t += nwarps) {
    float l[VPL];
    double c[VPL];
    uint32_t avail = 0, on = 0;  // experts, and those not masked
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + 32 * i;
      l[i] = -INFINITY;
      if (e < E) {
        l[i] = usable(load_logit(logits + t * ld + e));
        avail |= 1u << i;
        if (l[i] > -INFINITY) on |= 1u << i;
      }
    }
    float m = -INFINITY;
    double z = 0.0;
    if (a.score_fn == MOE_SCORE_SOFTMAX) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) m = fmaxf(m, l[i]);
      m = warp_max(m);
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if ((on >> i) & 1u) z += exp((double)l[i] - (double)m);
      z = warp_sum(z);
    }
    double s[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      s[i] = 0.0;
      c[i] = -INFINITY;
      if ((on >> i) & 1u) {
        s[i] = a.score_fn == MOE_SCORE_SOFTMAX ? exp((double)l[i] - (double)m) / z
                                               : 1.0 / (1.0 + exp(-(double)l[i]));
        double b = 0.0;
        if (bias) b = fmaxf(fminf(__ldg(bias + lane + 32 * i), kBiasClamp), -kBiasClamp);
        c[i] = s[i] + b;
      }
    }
    if (a.n_groups > 1) {
      double mine = -INFINITY;
      for (int g = 0; g < a.n_groups; ++g) {
        uint32_t mask = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (((on >> i) & 1u) && (lane + 32 * i) / gsz == g) mask |= 1u << i;
        for (int r = 0; r < a.group_topn; ++r) {
          double bv;
          int bid;
          warp_argmax<VPL>(c, mask, lane, bv, bid);
          if (bid == INT_MAX) break;
          if (lane == g) mine = r == 0 ? bv : mine + bv;
          if ((bid & 31) == lane) mask &= ~(1u << (bid >> 5));
        }
      }
      double gs[1] = {mine};
      uint32_t free_ = lane < a.n_groups ? 1u : 0u, kept = 0;
      for (int r = 0; r < a.topk_groups; ++r) {
        double bv;
        int bg;
        warp_argmax<1>(gs, free_, lane, bv, bg);
        kept |= 1u << bg;
        if (bg == lane) free_ = 0;
      }
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (((avail >> i) & 1u) && !((kept >> ((lane + 32 * i) / gsz)) & 1u)) avail &= ~(1u << i);
    }
    int my_id = 0;
    for (int j = 0; j < a.k; ++j) {
      double bv;
      int bid;
      warp_argmax<VPL>(c, avail, lane, bv, bid);
      if ((bid & 31) == lane) avail &= ~(1u << (bid >> 5));
      if (lane == j) my_id = bid;
    }
    // the selected experts' scores, from the lanes that hold them
    double my_s = 0.0;
    float my_l = -INFINITY;
    for (int j = 0; j < a.k; ++j) {
      const int id = __shfl_sync(kFull, my_id, j);
      double sv = 0.0;
      float lv = 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (i == (id >> 5)) {
          sv = s[i];
          lv = l[i];
        }
      sv = __shfl_sync(kFull, sv, id & 31);
      lv = __shfl_sync(kFull, lv, id & 31);
      if (lane == j) {
        my_s = sv;
        my_l = lv;
      }
    }
    if (a.renormalize) {
      const float ml = warp_max(my_l);
      // (softmax: the selected experts may all be far below the row's largest)
      const bool rel = a.score_fn == MOE_SCORE_SOFTMAX || ml < kTinyLogit;
      const double num = rel ? (my_l > -INFINITY ? exp((double)my_l - (double)ml) : 0.0) : my_s;
      const double den = warp_sum(lane < a.k ? num : 0.0);
      my_s = den > 0.0 ? num / den : 0.0;
    }
    if (lane < a.k) {
      ids[t * a.k + lane] = my_id;
      w[t * a.k + lane] = (float)((double)a.scale * my_s);
    }
  }
}

// Gradient of the logits for a gradient g of the weights (the selection and
// the bias carry none).  With v the renormalised weights without scale:
//   sigmoid            dl_e = scale g_e s_e (1 - s_e)                selected e
//   sigmoid, renorm    dl_e = scale (g_e - sum g v) v_e (1 - s_e)    selected e
//   softmax            dl_e = s_e (scale g_e [selected] - scale sum g s)  all e
//   softmax, renorm    dl_e = scale (g_e - sum g v) v_e              selected e
template <typename L, int VPL>
__global__ void __launch_bounds__(256)
    gate_backward_kernel(const L *__restrict__ logits, int64_t ld, int64_t T, int E,
                         const int32_t *__restrict__ ids, const float *__restrict__ grad_w,
                         GateArgs a, L *__restrict__ grad_logits, int32_t *status) {
  moe::pdl_wait();
  moe::pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t warp0 = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int64_t nwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
  const bool dense = a.score_fn == MOE_SCORE_SOFTMAX && !a.renormalize;
  for (int64_t t = warp0; t < T; t += nwarps) {
    int id = -1;
    float g = 0.0f, my_l = -INFINITY;
    if (lane < a.k) {
      id = __ldg(ids + t * a.k + lane);
      if (id < 0 || id >= E) {
        moe::report_error(status, MOE_ERR_DEVICE_INDEX, (int32_t)(t * a.k + lane), moe::K_GATE);
        id = -1;
      } else {
        g = __ldg(grad_w + t * a.k + lane);
        my_l = usable(load_logit(logits + t * ld + id));
      }
    }
    const bool live = my_l > -INFINITY;
    double mine = 0.0;  // this lane's assignment: its share of dl
    double p[VPL];      // dense: every expert's score
    double dot = 0.0;
    if (dense) {
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int e = lane + 32 * i;
        p[i] = e < E ? usable(load_logit(logits + t * ld + e)) : -INFINITY;
        m = fmaxf(m, (float)p[i]);
      }
      m = warp_max(m);
      double z = 0.0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        p[i] = p[i] > -INFINITY ? exp(p[i] - (double)m) : 0.0;
        z += p[i];
      }
      z = warp_sum(z);
#pragma unroll
      for (int i = 0; i < VPL; ++i) p[i] = z > 0.0 ? p[i] / z : 0.0;
      dot = warp_sum(live ? (double)g * (exp((double)my_l - (double)m) / z) : 0.0);
      mine = (double)a.scale * g;
    } else {
      const double s = a.score_fn == MOE_SCORE_SIGMOID && live ? 1.0 / (1.0 + exp(-(double)my_l)) : 0.0;
      if (a.renormalize) {
        const float ml = warp_max(my_l);
        const bool rel = a.score_fn == MOE_SCORE_SOFTMAX || ml < kTinyLogit;
        const double num = !live ? 0.0 : rel ? exp((double)my_l - (double)ml) : s;
        const double den = warp_sum(num);
        const double v = den > 0.0 ? num / den : 0.0;
        dot = warp_sum((double)g * v);
        mine = (double)a.scale * (g - dot) * v * (1.0 - s);
      } else {
        mine = (double)a.scale * g * s * (1.0 - s);
      }
    }
    double out[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) out[i] = 0.0;
    for (int j = 0; j < a.k; ++j) {
      const int e = __shfl_sync(kFull, id, j);
      const double v = __shfl_sync(kFull, mine, j);
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (e == lane + 32 * i) out[i] = v;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + 32 * i;
      if (e < E) {
        if (dense) out[i] = p[i] * (out[i] - (double)a.scale * dot);
        store_grad(grad_logits + t * E + e, (float)out[i]);
      }
    }
  }
}

// b_e + rate * sign(mean load - load_e): the mean is compared as total
// against E * load, in integers.
__global__ void __launch_bounds__(512) gate_update_bias_kernel(const int32_t *__restrict__ counts,
                                                               int E, const float *bias, float rate,
                                                               float *bias_out) {
  moe::pdl_wait();
  moe::pdl_trigger();
  __shared__ unsigned long long total;
  const int e = threadIdx.x;
  if (e == 0) total = 0;
  __syncthreads();
  const long long n = e < E ? counts[e] : 0;
  if (e < E) atomicAdd(&total, (unsigned long long)n);  // integers: the order does not matter
  __syncthreads();
  if (e < E) {
    const long long d = (long long)total - (long long)E * n;
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

unsigned gate_grid(int64_t T) {
  int64_t blocks = (T + 7) / 8;
  const int64_t cap = (int64_t)moe_host::sm_count() * 16;
  return (unsigned)(blocks > cap ? cap : blocks);
}

// Calls f with the experts a lane holds (1, 2, 4, 8 or 16) as a type.
template <int N>
struct Vpl {
  static constexpr int value = N;
};
template <typename F>
moe_status by_experts(int E, F &&f) {
  if (E <= 32) return f(Vpl<1>{});
  if (E <= 64) return f(Vpl<2>{});
  if (E <= 128) return f(Vpl<4>{});
  if (E <= 256) return f(Vpl<8>{});
  return f(Vpl<16>{});
}

template <typename L>
moe_status launch_gate(const void *logits, int64_t ld, int64_t T, int E, const float *bias,
                       GateArgs a, int32_t *ids, float *w, cudaStream_t st) {
  return by_experts(E, [&](auto v) {
    return moe_host::launch_pdl(gate_kernel<L, decltype(v)::value>, dim3(gate_grid(T)), dim3(256), 0,
                                st, static_cast<const L *>(logits), ld, T, E, bias, a, ids, w);
  });
}

template <typename L>
moe_status launch_backward(const void *logits, int64_t ld, int64_t T, int E, const int32_t *ids,
                           const float *g, GateArgs a, void *out, int32_t *status,
                           cudaStream_t st) {
  return by_experts(E, [&](auto v) {
    return moe_host::launch_pdl(gate_backward_kernel<L, decltype(v)::value>, dim3(gate_grid(T)),
                                dim3(256), 0, st, static_cast<const L *>(logits), ld, T, E, ids, g,
                                a, static_cast<L *>(out), status);
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
