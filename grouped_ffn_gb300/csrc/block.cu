// The block around the experts: RMS norms before and after them, the block's
// gate and residual scale, and the gradients of all but the experts' products.
//
// "14. Serving Mixture-of-Experts Models", "Follow one token", steps 2 and 4:
// rows are copied to their experts and come back as a weighted sum.  Here the
// sum goes on through the norm after the block, the gate and the residual in
// the same pass, and the two steps get their gradients: of the copies (a sum
// over a token's dispatched rows) and of the weighted sum (rows and weights).
//
// All are bound by HBM: a row is read once, kept in registers across the row's
// reductions, and each result is written once.
#include <cuda_bf16.h>
#include <float.h>
#include <math.h>

#include "common.cuh"

namespace {

// A row's CTA has up to 512 threads, each with U chunks of 8 elements: two for
// rows of up to 8192, four beyond (up to 128 registers a thread either way).
constexpr int kRowThreads = 512;
constexpr int kMaxH = kRowThreads * 4 * 8;
constexpr float kShrink = 0x1p-70f;

struct Rows {
  const int32_t *dest_row;
  int64_t n_rows;
  int32_t *status;
};

__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&p);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

// Eight elements of a row held as bf16 (one 16-byte access) or fp32 (two).
template <typename X>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
    a = *reinterpret_cast<const uint4 *>(p);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const { unpack8(a, f); }
  __device__ __forceinline__ void set(const float (&f)[8]) { a = pack8(f); }
  __device__ __forceinline__ void store(__nv_bfloat16 *p) const {
    *reinterpret_cast<uint4 *>(p) = a;
  }
};
template <>
struct Chunk<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = reinterpret_cast<const float4 *>(p)[0];
    b = reinterpret_cast<const float4 *>(p)[1];
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    a = make_float4(f[0], f[1], f[2], f[3]);
    b = make_float4(f[4], f[5], f[6], f[7]);
  }
  __device__ __forceinline__ void store(float *p) const {
    reinterpret_cast<float4 *>(p)[0] = a;
    reinterpret_cast<float4 *>(p)[1] = b;
  }
};

// Eight weights of a norm (ones without).
__device__ __forceinline__ void load_weight(const float *w, int c, float (&f)[8]) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 1.0f;
    return;
  }
  const float4 a = __ldg(reinterpret_cast<const float4 *>(w) + 2 * c);
  const float4 b = __ldg(reinterpret_cast<const float4 *>(w) + 2 * c + 1);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
  f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

// Sums over a warp of N values (a power of two) in N - 1 + log2(32 / N)
// shuffles: in each step half of the lanes go on with half of the values.
// Lane L ends with the sum of value L / (32 / N) in v[0].
template <int N>
__device__ __forceinline__ void warp_sums(float (&v)[N], int lane) {
  int step = 16;
#pragma unroll
  for (int n = N; n > 1; n >>= 1) {
    const bool up = lane & step;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const float keep = up ? v[i + n / 2] : v[i], send = up ? v[i] : v[i + n / 2];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, step);
    }
    step >>= 1;
  }
#pragma unroll
  for (int s = 16 / N; s > 0; s >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], s);
}

// A warp's sums to buf[value][warp], and a value's total from there: every
// warp adds the same numbers in the same order, so all threads agree.
template <int N>
__device__ __forceinline__ void put_sums(float (&v)[N], float *buf, int warp, int lane) {
  warp_sums(v, lane);
  if (lane % (32 / N) == 0) buf[lane / (32 / N) * 32 + warp] = v[0];
}
__device__ __forceinline__ float total(const float *buf, int value, int nw, int lane) {
  float x = lane < nw ? buf[value * 32 + lane] : 0.0f;
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
  return x;
}

__device__ __forceinline__ float inv_rms(float sum, int H, float eps) {
  return 1.0f / sqrtf(sum / (float)H + eps);
}

// The sum of squares of a row held in registers and 1 / its root mean square.
// Where the squares pass fp32's range, the row is brought down by 2^-70 first
// (eps vanishes next to such a row): rows of any finite values have a norm.
struct Norm {
  float pre, r;  // the row's factor, and 1 / rms of the row times it
};
template <int U>
__device__ __forceinline__ Norm row_norm(float (&x)[U][8], int H, float eps, float *buf, int warp,
                                         int nw, int lane) {
  float s[1] = {0.0f};
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < 8; ++i) s[0] = fmaf(x[u][i], x[u][i], s[0]);
  put_sums(s, buf, warp, lane);
  __syncthreads();
  float sum = total(buf, 0, nw, lane);
  Norm n{1.0f, 0.0f};
  if (!(sum <= FLT_MAX)) {
    n.pre = kShrink;
    s[0] = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[u][i] *= kShrink;
        s[0] = fmaf(x[u][i], x[u][i], s[0]);
      }
    __syncthreads();
    put_sums(s, buf, warp, lane);
    __syncthreads();
    sum = total(buf, 0, nw, lane);
    eps = 0.0f;
  }
  n.r = inv_rms(sum, H, eps);
  return n;
}

// The rows of a token's assignments: bit j of the result is set where row j
// takes part.  -1 is a dropped assignment; other rows outside are reported.
template <int KMAX>
__device__ __forceinline__ uint32_t token_rows(const Rows &p, int64_t t, int k, int32_t (&r)[KMAX]) {
  uint32_t live = 0;
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    if (j < k) {
      r[j] = __ldg(p.dest_row + t * k + j);
      if (r[j] >= 0 && r[j] < p.n_rows)
        live |= 1u << j;
      else if (r[j] != -1 && threadIdx.x == 0)
        moe::report_error(p.status, MOE_ERR_DEVICE_INDEX, (int32_t)(t * k + j), moe::K_BLOCK);
    }
  }
  return live;
}

// ------------------------------------------------------------------ forward
// out = x / rms(x) * weight.  One CTA a row.
template <int U, typename X>
__global__ void __launch_bounds__(kRowThreads)
    norm_kernel(const X *__restrict__ x, int64_t T, int H, const float *__restrict__ weight,
                            float eps, __nv_bfloat16 *__restrict__ out) {
  __shared__ float buf[2][32];
  moe::pdl_wait();
  moe::pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5, H8 = H / 8;
  int par = 0;
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x, par ^= 1) {
    float v[U][8] = {};
    Chunk<X> in[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = threadIdx.x + u * blockDim.x;
      if (c < H8) in[u].load(x + t * H + 8 * c);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if ((int)(threadIdx.x + u * blockDim.x) < H8) in[u].get(v[u]);
    const Norm n = row_norm(v, H, eps, buf[par], warp, nw, lane);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = threadIdx.x + u * blockDim.x;
      if (c >= H8) continue;
      float w[8], o[8];
      load_weight(weight, c, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = v[u][i] * n.r * w[i];
      *reinterpret_cast<uint4 *>(out + t * H + 8 * c) = pack8(o);
    }
  }
}

struct CombineNormParams {
  const uint4 *yp;
  Rows rows;
  const float *topk_w;
  int64_t T;
  int k, H;
  const uint4 *shared;
  const void *residual;
  const float *weight, *gate, *next_weight;
  int post;
  float eps, scale;
  void *y;
  uint4 *next;
};

// c = shared + sum_j w_j Y[row_j], y = scale x + gate norm(c), next = norm(y).
// One CTA a token; c and then y stay in registers across the two sums.
template <int KMAX, int U, typename X>
__global__ void __launch_bounds__(kRowThreads) combine_norm_kernel(const CombineNormParams p) {
  __shared__ float buf[2][2][32];
  moe::pdl_wait();
  moe::pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5, H8 = p.H / 8;
  int par = 0;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, par ^= 1) {
    int32_t r[KMAX];
    const uint32_t live = token_rows(p.rows, t, p.k, r);
    float w[KMAX];
#pragma unroll
    for (int j = 0; j < KMAX; ++j)
      if (j < p.k) w[j] = __ldg(p.topk_w + t * p.k + j);
    float acc[U][8] = {};
    Chunk<X> res[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = threadIdx.x + u * blockDim.x;
      if (c >= H8) continue;
      uint4 v[KMAX];
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if ((live >> j) & 1u) v[j] = moe::ld_stream_u4(p.yp + (int64_t)r[j] * H8 + c);
      if (p.shared) unpack8(moe::ld_stream_u4(p.shared + t * H8 + c), acc[u]);
      // (y may be the residual itself: no read-only load)
      res[u].load(static_cast<const X *>(p.residual) + t * p.H + 8 * c);
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if ((live >> j) & 1u) {
          float f[8];
          unpack8(v[j], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[u][i] = fmaf(w[j], f[i], acc[u][i]);
        }
    }
    float g = p.gate ? __ldg(p.gate + t) : 1.0f;
    float rc = 1.0f;
    if (p.post) rc = row_norm(acc, p.H, p.eps, buf[par][0], warp, nw, lane).r;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = threadIdx.x + u * blockDim.x;
      if (c >= H8) continue;
      float wt[8], x[8];
      load_weight(p.weight, c, wt);
      res[u].get(x);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[u][i] = fmaf(p.scale, x[i], g * (acc[u][i] * rc * wt[i]));
      res[u].set(acc[u]);
      res[u].store(static_cast<X *>(p.y) + t * p.H + 8 * c);
      res[u].get(acc[u]);  // as it is held
    }
    if (p.next) {
      const Norm n = row_norm(acc, p.H, p.eps, buf[par][1], warp, nw, lane);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = threadIdx.x + u * blockDim.x;
        if (c >= H8) continue;
        float wt[8], o[8];
        load_weight(p.next_weight, c, wt);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = acc[u][i] * n.r * wt[i];
        p.next[t * H8 + c] = pack8(o);
      }
    }
  }
}

// ------------------------------------------------------------------ backward
struct CombineBwdParams {
  const void *gy;
  const uint4 *yp;
  Rows rows;
  const float *topk_w;
  int64_t T;
  int k, H;
  const uint4 *shared;
  const float *weight, *gate;
  int post;
  float eps;
  uint4 *gyp;
  float *gw;
  uint4 *gshared;
  float *ggate;
  float *partial;  // [gridDim.x, H], or NULL
};

// y = sum_j w_j Y[row_j]: dY[row_j] = w_j dy, dw_j = dy . Y[row_j].  Nothing
// waits for the sums, so the row streams through in chunks.
template <int KMAX, typename X>
__global__ void __launch_bounds__(128) combine_bwd_kernel(const CombineBwdParams p) {
  __shared__ float buf[2][KMAX * 32];
  moe::pdl_wait();
  moe::pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5, H8 = p.H / 8;
  int par = 0;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, par ^= 1) {
    int32_t r[KMAX];
    const uint32_t live = token_rows(p.rows, t, p.k, r);
    float w[KMAX], dot[KMAX];
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
      if (j < p.k) w[j] = __ldg(p.topk_w + t * p.k + j);
      dot[j] = 0.0f;
    }
    for (int c = threadIdx.x; c < H8; c += blockDim.x) {
      uint4 v[KMAX];
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if ((live >> j) & 1u) v[j] = moe::ld_stream_u4(p.yp + (int64_t)r[j] * H8 + c);
      Chunk<X> in;
      in.load(static_cast<const X *>(p.gy) + t * p.H + 8 * c);
      float g[8];
      in.get(g);
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if ((live >> j) & 1u) {
          float f[8], o[8];
          unpack8(v[j], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dot[j] = fmaf(g[i], f[i], dot[j]);
            o[i] = w[j] * g[i];
          }
          p.gyp[(int64_t)r[j] * H8 + c] = pack8(o);
        }
    }
    put_sums(dot, buf[par], warp, lane);
    __syncthreads();
    for (int j = warp; j < p.k; j += nw) {
      const float d = total(buf[par], j, nw, lane);
      if (lane == 0) p.gw[t * p.k + j] = d;
    }
  }
}

// The gradient through norm and gate.  With e = gy weight, one pass over the
// rows gives c (the sum over j of a chunk is complete before the next chunk)
// and all of sum c^2, sum e c, e . Y_j and c . Y_j, so the expert rows are read
// once and need not be kept:
//   dc = gate r (e - c m),  m = r^2 mean(e c),  dw_j = gate r (e . Y_j - m c . Y_j).
// The weight's gradient is kept per thread over the CTA's tokens and added up
// by sum_partials_kernel in a fixed order.
template <int KMAX, int U, typename X>
__global__ void __launch_bounds__(kRowThreads) combine_norm_bwd_kernel(const CombineBwdParams p) {
  constexpr int kSums = 2 * KMAX;
  __shared__ float buf[2][(kSums + 2) * 32];
  moe::pdl_wait();
  moe::pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5, H8 = p.H / 8;
  float pw[U][8] = {};
  int par = 0;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, par ^= 1) {
    int32_t r[KMAX];
    const uint32_t live = token_rows(p.rows, t, p.k, r);
    float w[KMAX];
#pragma unroll
    for (int j = 0; j < KMAX; ++j)
      if (j < p.k) w[j] = __ldg(p.topk_w + t * p.k + j);
    float acc[U][8] = {};
    Chunk<X> in[U];
    float d[kSums], s[2] = {0.0f, 0.0f};  // e . Y_j, then c . Y_j
#pragma unroll
    for (int j = 0; j < kSums; ++j) d[j] = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = threadIdx.x + u * blockDim.x;
      if (c >= H8) continue;
      uint4 v[KMAX];
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if ((live >> j) & 1u) v[j] = moe::ld_stream_u4(p.yp + (int64_t)r[j] * H8 + c);
      if (p.shared) unpack8(moe::ld_stream_u4(p.shared + t * H8 + c), acc[u]);
      in[u].load(static_cast<const X *>(p.gy) + t * p.H + 8 * c);
      float e[8], wt[8], f[8];
      load_weight(p.weight, c, wt);
      in[u].get(e);
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] *= wt[i];
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if ((live >> j) & 1u) {
          unpack8(v[j], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            acc[u][i] = fmaf(w[j], f[i], acc[u][i]);
            d[j] = fmaf(e[i], f[i], d[j]);
          }
        }
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if ((live >> j) & 1u) {
          unpack8(v[j], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) d[KMAX + j] = fmaf(acc[u][i], f[i], d[KMAX + j]);
        }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s[0] = fmaf(acc[u][i], acc[u][i], s[0]);
        s[1] = fmaf(e[i], acc[u][i], s[1]);
      }
    }
    float *b = buf[par];
    put_sums(d, b, warp, lane);
    put_sums(s, b + kSums * 32, warp, lane);
    __syncthreads();
    const float g = p.gate ? __ldg(p.gate + t) : 1.0f;
    float s1 = total(b, kSums, nw, lane), s2 = total(b, kSums + 1, nw, lane);
    float pre = 1.0f, rc = 1.0f, m = 0.0f;
    if (p.post) {
      float eps = p.eps;
      if (!(s1 <= FLT_MAX)) {
        // squares beyond fp32's range: the same sums with c and Y_j times 2^-70
        pre = kShrink;
        eps = 0.0f;
        s[0] = s[1] = 0.0f;
#pragma unroll
        for (int j = 0; j < kSums; ++j) d[j] = 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int c = threadIdx.x + u * blockDim.x;
          if (c >= H8) continue;
          float e[8], wt[8], f[8];
          load_weight(p.weight, c, wt);
          in[u].get(e);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            e[i] *= wt[i];
            acc[u][i] *= kShrink;
            s[0] = fmaf(acc[u][i], acc[u][i], s[0]);
            s[1] = fmaf(e[i], acc[u][i], s[1]);
          }
#pragma unroll
          for (int j = 0; j < KMAX; ++j)
            if ((live >> j) & 1u) {
              unpack8(moe::ld_stream_u4(p.yp + (int64_t)r[j] * H8 + c), f);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                d[j] = fmaf(e[i], f[i] * kShrink, d[j]);
                d[KMAX + j] = fmaf(acc[u][i], f[i] * kShrink, d[KMAX + j]);
              }
            }
        }
        __syncthreads();
        put_sums(d, b, warp, lane);
        put_sums(s, b + kSums * 32, warp, lane);
        __syncthreads();
        s1 = total(b, kSums, nw, lane);
        s2 = total(b, kSums + 1, nw, lane);
      }
      rc = inv_rms(s1, p.H, eps);
      m = rc * rc * (s2 / (float)p.H);
    }
    for (int j = warp; j < p.k; j += nw) {
      const float ey = total(b, j, nw, lane), cy = total(b, KMAX + j, nw, lane);
      if (lane == 0) p.gw[t * p.k + j] = g * rc * (ey - m * cy);
    }
    if (p.ggate && threadIdx.x == 0) p.ggate[t] = s2 * rc;
    const float a = g * rc * pre;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = threadIdx.x + u * blockDim.x;
      if (c >= H8) continue;
      float gy[8], wt[8], o[8];
      load_weight(p.weight, c, wt);
      in[u].get(gy);
      if (p.partial) {
#pragma unroll
        for (int i = 0; i < 8; ++i) pw[u][i] = fmaf(g * gy[i], acc[u][i] * rc, pw[u][i]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) gy[i] = a * fmaf(-m, acc[u][i], gy[i] * wt[i]);
      if (p.gshared) p.gshared[t * H8 + c] = pack8(gy);
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if ((live >> j) & 1u) {
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = w[j] * gy[i];
          p.gyp[(int64_t)r[j] * H8 + c] = pack8(o);
        }
    }
  }
  if (p.partial) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = threadIdx.x + u * blockDim.x;
      if (c >= H8) continue;
      Chunk<float> o;
      o.set(pw[u]);
      o.store(p.partial + (int64_t)blockIdx.x * p.H + 8 * c);
    }
  }
}

struct NormBwdParams {
  const uint4 *grad;
  Rows rows;  // dest_row NULL: grad has a row a token
  const uint4 *add;
  const void *x;
  int64_t T;
  int k, H;
  const float *weight;
  float eps, scale;
  const void *rgrad;
  void *gx;
  float *partial;
};

// u = add + the sum of the copies' gradients (or grad's own row), e = u weight:
//   gx = scale rgrad + r (e - x r^2 mean(e x)),  weight's gradient sum_t u x r.
template <int KMAX, int U, typename X>
__global__ void __launch_bounds__(kRowThreads) norm_bwd_kernel(const NormBwdParams p) {
  __shared__ float buf[2][2 * 32];
  moe::pdl_wait();
  moe::pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5, H8 = p.H / 8;
  float pw[U][8] = {};
  int par = 0;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, par ^= 1) {
    int32_t r[KMAX];
    uint32_t live = 1;
    if (p.rows.dest_row) live = token_rows(p.rows, t, p.k, r);
    float acc[U][8] = {}, x[U][8] = {}, s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = threadIdx.x + u * blockDim.x;
      if (c >= H8) continue;
      uint4 v[KMAX];
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if ((live >> j) & 1u)
          v[j] = moe::ld_stream_u4(p.grad + (p.rows.dest_row ? (int64_t)r[j] : t) * H8 + c);
      if (p.add) unpack8(moe::ld_stream_u4(p.add + t * H8 + c), acc[u]);
      Chunk<X> in;
      in.load(static_cast<const X *>(p.x) + t * p.H + 8 * c);
      in.get(x[u]);
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if ((live >> j) & 1u) {
          float f[8];
          unpack8(v[j], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[u][i] += f[i];
        }
      float wt[8];
      load_weight(p.weight, c, wt);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s[0] = fmaf(x[u][i], x[u][i], s[0]);
        s[1] = fmaf(acc[u][i] * wt[i], x[u][i], s[1]);
      }
    }
    float *b = buf[par];
    put_sums(s, b, warp, lane);
    __syncthreads();
    float s1 = total(b, 0, nw, lane), s2 = total(b, 1, nw, lane), pre = 1.0f, eps = p.eps;
    if (!(s1 <= FLT_MAX)) {  // as in row_norm
      pre = kShrink;
      eps = 0.0f;
      s[0] = s[1] = 0.0f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = threadIdx.x + u * blockDim.x;
        if (c >= H8) continue;
        float wt[8];
        load_weight(p.weight, c, wt);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[u][i] *= kShrink;
          s[0] = fmaf(x[u][i], x[u][i], s[0]);
          s[1] = fmaf(acc[u][i] * wt[i], x[u][i], s[1]);
        }
      }
      __syncthreads();
      put_sums(s, b, warp, lane);
      __syncthreads();
      s1 = total(b, 0, nw, lane);
      s2 = total(b, 1, nw, lane);
    }
    const float rc = inv_rms(s1, p.H, eps), m = rc * rc * (s2 / (float)p.H), a = rc * pre;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = threadIdx.x + u * blockDim.x;
      if (c >= H8) continue;
      float wt[8], o[8] = {};
      load_weight(p.weight, c, wt);
      if (p.rgrad) {
        // (gx may be rgrad itself: no read-only load)
        Chunk<X> in;
        in.load(static_cast<const X *>(p.rgrad) + t * p.H + 8 * c);
        in.get(o);
      }
      if (p.partial) {
#pragma unroll
        for (int i = 0; i < 8; ++i) pw[u][i] = fmaf(acc[u][i], x[u][i] * rc, pw[u][i]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        o[i] = fmaf(p.scale, o[i], a * fmaf(-m, x[u][i], acc[u][i] * wt[i]));
      Chunk<X> out;
      out.set(o);
      out.store(static_cast<X *>(p.gx) + t * p.H + 8 * c);
    }
  }
  if (p.partial) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = threadIdx.x + u * blockDim.x;
      if (c >= H8) continue;
      Chunk<float> o;
      o.set(pw[u]);
      o.store(p.partial + (int64_t)blockIdx.x * p.H + 8 * c);
    }
  }
}

// grad_x[t] = add[t] + sum_j grad[row_j].
template <int KMAX, typename X>
__global__ void __launch_bounds__(128)
    permute_bwd_kernel(const uint4 *__restrict__ grad, Rows rows, const uint4 *__restrict__ add,
                       int64_t T, int k, int H, X *__restrict__ gx) {
  moe::pdl_wait();
  moe::pdl_trigger();
  const int H8 = H / 8;
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
    int32_t r[KMAX];
    const uint32_t live = token_rows(rows, t, k, r);
    for (int c = threadIdx.x; c < H8; c += blockDim.x) {
      uint4 v[KMAX];
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if ((live >> j) & 1u) v[j] = moe::ld_stream_u4(grad + (int64_t)r[j] * H8 + c);
      float acc[8] = {}, f[8];
      if (add) unpack8(moe::ld_stream_u4(add + t * H8 + c), acc);
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if ((live >> j) & 1u) {
          unpack8(v[j], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i] += f[i];
        }
      Chunk<X> out;
      out.set(acc);
      out.store(gx + t * H + 8 * c);
    }
  }
}

// The weight's gradient: the n partial rows added up in a fixed order.  A CTA
// takes 32 columns (a 128-byte line of each row), its 64 groups of 8 lanes every
// 64th row each.
constexpr int kSumThreads = 512, kSumGroups = kSumThreads / 8;
__global__ void __launch_bounds__(kSumThreads)
    sum_partials_kernel(const float *__restrict__ partial, int n, int H, float *__restrict__ out) {
  __shared__ float4 part[kSumGroups][8];
  moe::pdl_wait();
  moe::pdl_trigger();
  const int group = threadIdx.x >> 3, i8 = threadIdx.x & 7;
  const int col = blockIdx.x * 32 + 4 * i8;
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (col < H) {
#pragma unroll 4
    for (int i = group; i < n; i += kSumGroups) {
      const float4 v = *reinterpret_cast<const float4 *>(partial + (int64_t)i * H + col);
      a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
    }
  }
  part[group][i8] = a;
  __syncthreads();
  if (threadIdx.x >= 32) return;
  // lane L: column L of the 32
  const float *s = reinterpret_cast<const float *>(part) + threadIdx.x;
  float sum = 0.0f;
#pragma unroll 8
  for (int i = 0; i < kSumGroups; ++i) sum += s[i * 32];
  if (blockIdx.x * 32 + threadIdx.x < H) out[blockIdx.x * 32 + threadIdx.x] = sum;
}

// ------------------------------------------------------------------ host
constexpr int kStreamThreads = 128;

int row_chunks(int H) { return H <= kRowThreads * 2 * 8 ? 2 : 4; }
int row_threads(int H) {
  const int u = row_chunks(H);
  return ((H / 8 + u - 1) / u + 31) / 32 * 32;
}

unsigned row_grid(int64_t T) {
  const int64_t cap = (int64_t)moe_host::sm_count() * 32;
  return (unsigned)(T < cap ? T : cap);
}

// CTAs of the gradients: two an SM, or as many as hold 1024 threads.
unsigned bwd_grid(int64_t T, int H) {
  const int threads = row_threads(H);
  int per_sm = 1024 / threads;
  if (per_sm < 2) per_sm = 2;
  const int64_t cap = (int64_t)moe_host::sm_count() * per_sm;
  return (unsigned)(T < cap ? T : cap);
}

bool bad_type(int32_t type) { return type != MOE_F32 && type != MOE_BF16; }
bool odd(const void *p) { return !moe_host::aligned16(p); }
bool bad_eps(float eps) { return !(eps > 0.0f) || !isfinite(eps); }

moe_status check_sizes(int64_t T, int32_t k, int32_t H, int64_t n_rows) {
  if (T < 0 || H < 1 || k < 1 || n_rows < 0) return MOE_ERR_INVALID_ARG;
  if (H % 8 != 0 || H > kMaxH || k > 16 || n_rows >= ((int64_t)1 << 31) ||
      T >= ((int64_t)1 << 31) / k)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

template <typename P>
moe_status launch(void (*kernel)(P), unsigned grid, int threads, cudaStream_t st, const P &p) {
  return moe_host::launch_pdl(kernel, dim3(grid), dim3((unsigned)threads), 0, st, p);
}

template <int U, typename X>
moe_status run_combine_norm(const CombineNormParams &p, cudaStream_t st) {
  const unsigned g = row_grid(p.T);
  const int n = row_threads(p.H);
  if (p.k <= 2) return launch(combine_norm_kernel<2, U, X>, g, n, st, p);
  if (p.k <= 4) return launch(combine_norm_kernel<4, U, X>, g, n, st, p);
  if (p.k <= 8) return launch(combine_norm_kernel<8, U, X>, g, n, st, p);
  return launch(combine_norm_kernel<16, U, X>, g, n, st, p);
}

template <typename X>
moe_status run_combine_bwd(const CombineBwdParams &p, cudaStream_t st) {
  const unsigned g = row_grid(p.T);
  const int n = kStreamThreads;
  if (p.k <= 2) return launch(combine_bwd_kernel<2, X>, g, n, st, p);
  if (p.k <= 4) return launch(combine_bwd_kernel<4, X>, g, n, st, p);
  if (p.k <= 8) return launch(combine_bwd_kernel<8, X>, g, n, st, p);
  return launch(combine_bwd_kernel<16, X>, g, n, st, p);
}

template <int U, typename X>
moe_status run_combine_norm_bwd(const CombineBwdParams &p, cudaStream_t st) {
  const unsigned g = bwd_grid(p.T, p.H);
  const int n = row_threads(p.H);
  if (p.k <= 2) return launch(combine_norm_bwd_kernel<2, U, X>, g, n, st, p);
  if (p.k <= 4) return launch(combine_norm_bwd_kernel<4, U, X>, g, n, st, p);
  if (p.k <= 8) return launch(combine_norm_bwd_kernel<8, U, X>, g, n, st, p);
  return launch(combine_norm_bwd_kernel<16, U, X>, g, n, st, p);
}

template <int U, typename X>
moe_status run_norm_bwd(const NormBwdParams &p, cudaStream_t st) {
  const unsigned g = bwd_grid(p.T, p.H);
  const int n = row_threads(p.H);
  if (!p.rows.dest_row) return launch(norm_bwd_kernel<1, U, X>, g, n, st, p);
  if (p.k <= 2) return launch(norm_bwd_kernel<2, U, X>, g, n, st, p);
  if (p.k <= 4) return launch(norm_bwd_kernel<4, U, X>, g, n, st, p);
  if (p.k <= 8) return launch(norm_bwd_kernel<8, U, X>, g, n, st, p);
  return launch(norm_bwd_kernel<16, U, X>, g, n, st, p);
}

template <typename X>
moe_status run_permute_bwd(const uint16_t *grad, const Rows &rows, const uint16_t *add, int64_t T,
                           int32_t k, int32_t H, void *gx, cudaStream_t st) {
  const dim3 g(row_grid(T)), b(kStreamThreads);
  const uint4 *in = reinterpret_cast<const uint4 *>(grad), *ad = reinterpret_cast<const uint4 *>(add);
  X *out = static_cast<X *>(gx);
  if (k <= 2) return moe_host::launch_pdl(permute_bwd_kernel<2, X>, g, b, 0, st, in, rows, ad, T, k, H, out);
  if (k <= 4) return moe_host::launch_pdl(permute_bwd_kernel<4, X>, g, b, 0, st, in, rows, ad, T, k, H, out);
  if (k <= 8) return moe_host::launch_pdl(permute_bwd_kernel<8, X>, g, b, 0, st, in, rows, ad, T, k, H, out);
  return moe_host::launch_pdl(permute_bwd_kernel<16, X>, g, b, 0, st, in, rows, ad, T, k, H, out);
}

template <typename X>
moe_status run_norm(const void *x, int64_t T, int32_t H, const float *weight, float eps, uint16_t *out,
                    cudaStream_t st) {
  const dim3 g(row_grid(T)), b((unsigned)row_threads(H));
  return moe_host::launch_pdl(row_chunks(H) == 2 ? norm_kernel<2, X> : norm_kernel<4, X>, g, b, 0, st,
                              static_cast<const X *>(x), T, (int)H, weight, eps,
                              reinterpret_cast<__nv_bfloat16 *>(out));
}

moe_status sum_partials(const float *partial, unsigned n, int32_t H, float *out, cudaStream_t st) {
  return moe_host::launch_pdl(sum_partials_kernel, dim3((unsigned)(H + 31) / 32), dim3(kSumThreads), 0,
                              st, partial, (int)n, (int)H, out);
}

// The scratch of a weight's gradient, or an all-zero gradient for no tokens.
moe_status check_scratch(const float *grad_weight, int64_t T, int32_t H, void *scratch,
                         size_t scratch_bytes) {
  if (!grad_weight) return MOE_OK;
  if (odd(grad_weight)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!scratch || odd(scratch) || scratch_bytes < moe_norm_scratch_bytes(T, H))
    return MOE_ERR_WORKSPACE;
  return MOE_OK;
}
moe_status zero_gradient(float *grad_weight, int32_t H, cudaStream_t st) {
  if (!grad_weight) return MOE_OK;
  return cudaMemsetAsync(grad_weight, 0, (size_t)H * 4, st) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace

extern "C" size_t moe_norm_scratch_bytes(int64_t T, int32_t H) {
  if (T < 1 || H < 8 || H % 8 != 0 || H > kMaxH) return 0;
  return (size_t)bwd_grid(T, H) * (size_t)H * 4;
}

extern "C" moe_status moe_norm(const void *x, int32_t x_type, int64_t T, int32_t H,
                               const float *weight, float eps, uint16_t *out, void *stream) {
  if (bad_type(x_type) || bad_eps(eps)) return MOE_ERR_INVALID_ARG;
  if (moe_status s = check_sizes(T, 1, H, 0)) return s;
  if (T == 0) return MOE_OK;
  if (!x || !out || odd(x) || odd(out) || odd(weight)) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return x_type == MOE_F32 ? run_norm<float>(x, T, H, weight, eps, out, st)
                           : run_norm<__nv_bfloat16>(x, T, H, weight, eps, out, st);
}

extern "C" moe_status moe_norm_backward(const uint16_t *grad, int64_t n_rows,
                                        const int32_t *dest_row, int32_t k, const uint16_t *add,
                                        const void *x, int32_t x_type, int64_t T, int32_t H,
                                        const float *weight, float eps, const void *residual_grad,
                                        float residual_scale, void *grad_x, float *grad_weight,
                                        void *scratch, size_t scratch_bytes, void *ws,
                                        size_t ws_bytes, void *stream) {
  if (bad_type(x_type) || bad_eps(eps) || !isfinite(residual_scale)) return MOE_ERR_INVALID_ARG;
  if (moe_status s = check_sizes(T, dest_row ? k : 1, H, n_rows)) return s;
  if (!dest_row && T > 0 && n_rows != T) return MOE_ERR_INVALID_ARG;
  if (moe_status s = moe_host::check_ws(ws, ws_bytes, moe::kStatusBytes)) return s;
  if (moe_status s = check_scratch(grad_weight, T, H, scratch, scratch_bytes)) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0) return zero_gradient(grad_weight, H, st);
  if ((!grad && n_rows > 0) || !x || !grad_x || odd(grad) || odd(add) || odd(x) || odd(weight) ||
      odd(residual_grad) || odd(grad_x))
    return MOE_ERR_INVALID_ARG;
  NormBwdParams p{};
  p.grad = reinterpret_cast<const uint4 *>(grad);
  p.rows = Rows{dest_row, n_rows, moe_host::status_ptr(ws)};
  p.add = reinterpret_cast<const uint4 *>(add);
  p.x = x;
  p.T = T;
  p.k = k;
  p.H = H;
  p.weight = weight;
  p.eps = eps;
  p.scale = residual_scale;
  p.rgrad = residual_grad;
  p.gx = grad_x;
  p.partial = grad_weight ? static_cast<float *>(scratch) : nullptr;
  const bool f32 = x_type == MOE_F32;
  moe_status s;
  if (row_chunks(H) == 2)
    s = f32 ? run_norm_bwd<2, float>(p, st) : run_norm_bwd<2, __nv_bfloat16>(p, st);
  else
    s = f32 ? run_norm_bwd<4, float>(p, st) : run_norm_bwd<4, __nv_bfloat16>(p, st);
  if (s != MOE_OK || !grad_weight) return s;
  return sum_partials(p.partial, bwd_grid(T, H), H, grad_weight, st);
}

extern "C" moe_status moe_permute_backward(const uint16_t *grad, int64_t n_rows,
                                           const int32_t *dest_row, const uint16_t *add, int64_t T,
                                           int32_t k, int32_t H, void *grad_x, int32_t x_type,
                                           void *ws, size_t ws_bytes, void *stream) {
  if (bad_type(x_type)) return MOE_ERR_INVALID_ARG;
  if (moe_status s = check_sizes(T, k, H, n_rows)) return s;
  if (moe_status s = moe_host::check_ws(ws, ws_bytes, moe::kStatusBytes)) return s;
  if (T == 0) return MOE_OK;
  if ((!grad && n_rows > 0) || !dest_row || !grad_x || odd(grad) || odd(add) || odd(grad_x))
    return MOE_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const Rows rows{dest_row, n_rows, moe_host::status_ptr(ws)};
  return x_type == MOE_F32 ? run_permute_bwd<float>(grad, rows, add, T, k, H, grad_x, st)
                           : run_permute_bwd<__nv_bfloat16>(grad, rows, add, T, k, H, grad_x, st);
}

extern "C" moe_status moe_combine_norm(const uint16_t *y_perm, int64_t n_rows,
                                       const int32_t *dest_row, const float *topk_w, int64_t T,
                                       int32_t k, int32_t H, const uint16_t *shared,
                                       const void *residual, int32_t x_type, const float *weight,
                                       const float *gate, const moe_block_cfg *cfg, void *y,
                                       const float *next_weight, uint16_t *next_out, void *ws,
                                       size_t ws_bytes, void *stream) {
  if (bad_type(x_type) || !cfg || (cfg->post_norm != 0 && cfg->post_norm != 1) ||
      bad_eps(cfg->eps) || !isfinite(cfg->residual_scale) || (!cfg->post_norm && weight) ||
      (next_weight && !next_out))
    return MOE_ERR_INVALID_ARG;
  if (moe_status s = check_sizes(T, k, H, n_rows)) return s;
  if (moe_status s = moe_host::check_ws(ws, ws_bytes, moe::kStatusBytes)) return s;
  if (T == 0) return MOE_OK;
  if ((!y_perm && n_rows > 0) || !dest_row || !topk_w || !residual || !y || odd(y_perm) ||
      odd(shared) || odd(residual) || odd(weight) || odd(y) || odd(next_weight) || odd(next_out))
    return MOE_ERR_INVALID_ARG;
  CombineNormParams p{};
  p.yp = reinterpret_cast<const uint4 *>(y_perm);
  p.rows = Rows{dest_row, n_rows, moe_host::status_ptr(ws)};
  p.topk_w = topk_w;
  p.T = T;
  p.k = k;
  p.H = H;
  p.shared = reinterpret_cast<const uint4 *>(shared);
  p.residual = residual;
  p.weight = weight;
  p.gate = gate;
  p.next_weight = next_weight;
  p.post = cfg->post_norm;
  p.eps = cfg->eps;
  p.scale = cfg->residual_scale;
  p.y = y;
  p.next = reinterpret_cast<uint4 *>(next_out);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (row_chunks(H) == 2)
    return x_type == MOE_F32 ? run_combine_norm<2, float>(p, st)
                             : run_combine_norm<2, __nv_bfloat16>(p, st);
  return x_type == MOE_F32 ? run_combine_norm<4, float>(p, st)
                           : run_combine_norm<4, __nv_bfloat16>(p, st);
}

extern "C" moe_status moe_combine_norm_backward(
    const void *grad_y, int32_t x_type, const uint16_t *y_perm, int64_t n_rows,
    const int32_t *dest_row, const float *topk_w, int64_t T, int32_t k, int32_t H,
    const uint16_t *shared, const float *weight, const float *gate, const moe_block_cfg *cfg,
    uint16_t *grad_y_perm, float *grad_topk_w, uint16_t *grad_shared, float *grad_weight,
    float *grad_gate, void *scratch, size_t scratch_bytes, void *ws, size_t ws_bytes,
    void *stream) {
  if (bad_type(x_type) || !cfg || (cfg->post_norm != 0 && cfg->post_norm != 1) ||
      bad_eps(cfg->eps) || !isfinite(cfg->residual_scale) ||
      (!cfg->post_norm && (weight || grad_weight)))
    return MOE_ERR_INVALID_ARG;
  if (moe_status s = check_sizes(T, k, H, n_rows)) return s;
  if (moe_status s = moe_host::check_ws(ws, ws_bytes, moe::kStatusBytes)) return s;
  if (moe_status s = check_scratch(grad_weight, T, H, scratch, scratch_bytes)) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0) return zero_gradient(grad_weight, H, st);
  if (!grad_y || (n_rows > 0 && (!y_perm || !grad_y_perm)) || !dest_row || !topk_w ||
      !grad_topk_w || odd(grad_y) || odd(y_perm) || odd(shared) || odd(weight) ||
      odd(grad_y_perm) || odd(grad_shared))
    return MOE_ERR_INVALID_ARG;
  CombineBwdParams p{};
  p.gy = grad_y;
  p.yp = reinterpret_cast<const uint4 *>(y_perm);
  p.rows = Rows{dest_row, n_rows, moe_host::status_ptr(ws)};
  p.topk_w = topk_w;
  p.T = T;
  p.k = k;
  p.H = H;
  p.shared = reinterpret_cast<const uint4 *>(shared);
  p.weight = weight;
  p.gate = gate;
  p.post = cfg->post_norm;
  p.eps = cfg->eps;
  p.gyp = reinterpret_cast<uint4 *>(grad_y_perm);
  p.gw = grad_topk_w;
  p.gshared = reinterpret_cast<uint4 *>(grad_shared);
  p.ggate = grad_gate;
  p.partial = grad_weight ? static_cast<float *>(scratch) : nullptr;
  const bool f32 = x_type == MOE_F32;
  moe_status s;
  if (row_chunks(H) == 2)
    s = f32 ? run_combine_norm_bwd<2, float>(p, st) : run_combine_norm_bwd<2, __nv_bfloat16>(p, st);
  else
    s = f32 ? run_combine_norm_bwd<4, float>(p, st) : run_combine_norm_bwd<4, __nv_bfloat16>(p, st);
  if (s != MOE_OK || !grad_weight) return s;
  return sum_partials(p.partial, bwd_grid(T, H), H, grad_weight, st);
}

extern "C" moe_status moe_combine_backward(const void *grad_y, int32_t x_type,
                                           const uint16_t *y_perm, int64_t n_rows,
                                           const int32_t *dest_row, const float *topk_w, int64_t T,
                                           int32_t k, int32_t H, uint16_t *grad_y_perm,
                                           float *grad_topk_w, void *ws, size_t ws_bytes,
                                           void *stream) {
  if (bad_type(x_type)) return MOE_ERR_INVALID_ARG;
  if (moe_status s = check_sizes(T, k, H, n_rows)) return s;
  if (moe_status s = moe_host::check_ws(ws, ws_bytes, moe::kStatusBytes)) return s;
  if (T == 0) return MOE_OK;
  if (!grad_y || (n_rows > 0 && (!y_perm || !grad_y_perm)) || !dest_row || !topk_w ||
      !grad_topk_w || odd(grad_y) || odd(y_perm) || odd(grad_y_perm))
    return MOE_ERR_INVALID_ARG;
  CombineBwdParams p{};
  p.gy = grad_y;
  p.yp = reinterpret_cast<const uint4 *>(y_perm);
  p.rows = Rows{dest_row, n_rows, moe_host::status_ptr(ws)};
  p.topk_w = topk_w;
  p.T = T;
  p.k = k;
  p.H = H;
  p.gyp = reinterpret_cast<uint4 *>(grad_y_perm);
  p.gw = grad_topk_w;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return x_type == MOE_F32 ? run_combine_bwd<float>(p, st) : run_combine_bwd<__nv_bfloat16>(p, st);
}
