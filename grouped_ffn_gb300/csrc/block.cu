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
// reductions, and each result is written once.  A token takes a team of threads.
// Every thread copies its own 16-byte pieces of the token's rows to its own places
// in shared memory (cp.async, no barrier), and as soon as it has used a piece it
// asks for the next token's: the reads go on while a token's sums meet and its
// results are written.  With plain loads into registers instead, 4096 tokens of
// 7168 with eight rows each, shared expert and next norm took 165 us; now 108 us.
#include <cuda_bf16.h>
#include <float.h>
#include <math.h>

#include "block_shape.cuh"
#include "common.cuh"

namespace {

using namespace block_shape;

// Rows whose squares pass fp32's range are brought down by this first: 16384 squares
// of (2^128 2^-72) add up to 2^126, and the row's largest element is still above 2^-15.
constexpr float kShrink = 0x1p-72f;

struct Rows {
  const int32_t *dest_row;
  int64_t n_rows;
  int32_t *status;
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&p);
}

// 16 bytes to shared memory, or zeros where there are none to copy.
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src, bool some) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(some ? 16 : 0)
               : "memory");
}

// Two fp32 numbers for the instructions that take two at a time.
typedef unsigned long long Pair;
__device__ __forceinline__ Pair pair(float a, float b) {
  Pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ Pair both(float a) { return pair(a, a); }
__device__ __forceinline__ void split(Pair v, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ float sum(Pair v) {
  float a, b;
  split(v, a, b);
  return a + b;
}
__device__ __forceinline__ Pair fma(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ Pair mul(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Pair plus(Pair a, Pair b) {
  Pair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float dot(const Pair (&a)[4], const Pair (&b)[4]) {
  return sum(fma(a[3], b[3], fma(a[2], b[2], fma(a[1], b[1], mul(a[0], b[0])))));
}
__device__ __forceinline__ void unpack(const uint4 &v, Pair (&f)[4]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    f[i] = pair(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t pack_pair(Pair v) {
  float a, b;
  split(v, a, b);
  return pack2(a, b);
}
__device__ __forceinline__ uint4 pack(const Pair (&f)[4]) {
  return make_uint4(pack_pair(f[0]), pack_pair(f[1]), pack_pair(f[2]), pack_pair(f[3]));
}

// Eight elements of a row held as bf16 (16 bytes) or fp32 (32).  Two accesses of 16
// bytes a thread each touch every sector of a warp's fp32 piece, which then crosses
// from L2 twice; so there a warp's kilobyte is copied and stored in whole sectors.
//  copy   a warp's pieces to its place in shared memory (N times 512 bytes at s),
//         zeros from the row's end on;
//  take   the thread's piece from there;
//  store  to a row: the whole warp calls it.
template <typename X>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16> {
  static constexpr int N = 1;
  uint4 a;
  __device__ __forceinline__ static void copy(uint32_t s, const __nv_bfloat16 *row, int c, int H8,
                                              int lane) {
    copy_async(s + lane * 16, row + 8 * (int64_t)min(c, H8 - 1), c < H8);
  }
  __device__ __forceinline__ void take(const uint8_t *s, int lane) {
    a = *reinterpret_cast<const uint4 *>(s + lane * 16);
  }
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
    a = *reinterpret_cast<const uint4 *>(p);
  }
  __device__ __forceinline__ void get(Pair (&f)[4]) const { unpack(a, f); }
  __device__ __forceinline__ void set(const Pair (&f)[4]) { a = pack(f); }
  __device__ __forceinline__ void store(__nv_bfloat16 *row, int c, int H8, int) const {
    if (c < H8) reinterpret_cast<uint4 *>(row)[c] = a;
  }
};
template <>
struct Chunk<float> {
  static constexpr int N = 2;
  float4 a, b;
  // 16-byte place of a warp's i-th four elements: lanes read their two without
  // bank conflicts
  __device__ __forceinline__ static int place(int i) { return (i ^ (i >> 3 & 1)) * 16; }
  __device__ __forceinline__ static void copy(uint32_t s, const float *row, int c, int H8, int lane) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = h * 32 + lane, at = 8 * (c - lane) + 4 * i;
      copy_async(s + place(i), row + min(at, 8 * H8 - 4), at < 8 * H8);
    }
  }
  __device__ __forceinline__ void take(const uint8_t *s, int lane) {
    a = *reinterpret_cast<const float4 *>(s + place(2 * lane));
    b = *reinterpret_cast<const float4 *>(s + place(2 * lane + 1));
  }
  __device__ __forceinline__ void load(const float *p) {
    a = reinterpret_cast<const float4 *>(p)[0];
    b = reinterpret_cast<const float4 *>(p)[1];
  }
  __device__ __forceinline__ void get(Pair (&f)[4]) const {
    f[0] = pair(a.x, a.y), f[1] = pair(a.z, a.w), f[2] = pair(b.x, b.y), f[3] = pair(b.z, b.w);
  }
  __device__ __forceinline__ void set(const Pair (&f)[4]) {
    split(f[0], a.x, a.y);
    split(f[1], a.z, a.w);
    split(f[2], b.x, b.y);
    split(f[3], b.z, b.w);
  }
  __device__ __forceinline__ void put(float *p) const {
    reinterpret_cast<float4 *>(p)[0] = a;
    reinterpret_cast<float4 *>(p)[1] = b;
  }
  // An even lane's second half goes out with the odd one's number in the first
  // instruction, the odd lane's first half with the even one's in the second.
  __device__ __forceinline__ void store(float *row, int c, int H8, int lane) const {
    const bool odd = lane & 1;
    const float4 v = odd ? a : b;
    const float4 w = make_float4(
        __shfl_xor_sync(0xffffffffu, v.x, 1), __shfl_xor_sync(0xffffffffu, v.y, 1),
        __shfl_xor_sync(0xffffffffu, v.z, 1), __shfl_xor_sync(0xffffffffu, v.w, 1));
    const int even = c - odd;  // the pair's first piece
    float4 *p = reinterpret_cast<float4 *>(row) + 2 * even + odd;
    if (even < H8) p[0] = odd ? w : a;
    if (even + 1 < H8) p[2] = odd ? b : w;
  }
};

// Eight weights of a norm (ones without).
__device__ __forceinline__ void load_weight(const float *w, int c, Pair (&f)[4]) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = both(1.0f);
    return;
  }
  Chunk<float> v;
  v.a = __ldg(reinterpret_cast<const float4 *>(w) + 2 * c);
  v.b = __ldg(reinterpret_cast<const float4 *>(w) + 2 * c + 1);
  v.get(f);
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

// A warp's sums to buf[value][warp], and a value's total from there, warps that are
// not there counting zero (clear_sums): all threads add the same numbers in the
// same order.  v[0] is then a warp's sum, and small() says of it that a total of 16
// such is within fp32's range (false for NaN).
template <int N>
__device__ __forceinline__ void put_sums(float (&v)[N], float *buf, int warp, int lane) {
  warp_sums(v, lane);
  if (lane % (32 / N) == 0) buf[lane / (32 / N) * kLine + warp] = v[0];
}
__device__ __forceinline__ bool small(float warp_sum) { return fabsf(warp_sum) <= FLT_MAX / 32.0f; }
// of up to eight warps
__device__ __forceinline__ float total_few(const float *buf, int value) {
  const float4 *b = reinterpret_cast<const float4 *>(buf + value * kLine);
  const float4 v = b[0], w = b[1];
  return ((v.x + v.y) + (v.z + v.w)) + ((w.x + w.y) + (w.z + w.w));
}
__device__ __forceinline__ float total_many(const float *buf, int value, int nw, int lane) {
  float x = lane < nw ? buf[value * kLine + lane] : 0.0f;
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
  return x;
}
__device__ __forceinline__ float total(const float *buf, int value, int nw, int lane) {
  return nw <= 8 ? total_few(buf, value) : total_many(buf, value, nw, lane);
}
__device__ __forceinline__ void clear_sums(float *buf, int n, int tid, int threads) {
  for (int i = tid; i < n; i += threads) buf[i] = 0.0f;
}

// (rsqrtf is within two units of its last place)
__device__ __forceinline__ float inv_rms(float sum, float inv_h, float eps) {
  return rsqrtf(fmaf(sum, inv_h, eps));
}

// The threads of one token: a CTA's (ALONE), or some of its warps with a barrier of
// their own.  (A barrier whose number the compiler does not know reserves all 16,
// and an SM has them for four CTAs only.)
template <bool ALONE>
struct Team {
  int index, threads, tid, warp, nw, lane;
  __device__ __forceinline__ explicit Team(int threads_) : threads(threads_) {
    index = threadIdx.x / threads;
    tid = threadIdx.x - index * threads;
    warp = tid >> 5;
    nw = threads >> 5;
    lane = threadIdx.x & 31;
  }
  __device__ __forceinline__ void sync() const {
    if (ALONE)
      __syncthreads();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(1 + index), "r"(threads) : "memory");
  }
  // the barrier, and whether any thread came with true
  __device__ __forceinline__ bool any(bool mine) const {
    int r;
    asm volatile(
        "{ .reg .pred p, q; setp.ne.s32 p, %3, 0; bar.red.or.pred q, %1, %2, p; selp.s32 %0, 1, 0, q; }"
        : "=r"(r)
        : "r"(1 + index), "r"(threads), "r"((int)mine)
        : "memory");
    return r;
  }
};

__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t smem_u32(const void *p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// The sum of squares of a row held in registers and 1 / its root mean square.
// Where the squares pass fp32's range, the row is brought down by 2^-72 first and eps
// by 2^-144: rows of any finite values have a norm.
struct Norm {
  float pre, r;  // the row's factor, and 1 / rms of the row times it
};
template <int U>
__device__ __forceinline__ Norm row_norm(Pair (&x)[U][4], float inv_h, float eps, float *buf,
                                         const Team<true> &tm) {
  auto squares = [&]() {
    Pair s = mul(x[0][0], x[0][0]);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = u == 0; i < 4; ++i) s = fma(x[u][i], x[u][i], s);
    float v[1] = {sum(s)};
    put_sums(v, buf, tm.warp, tm.lane);
    tm.sync();
    // (a team of one piece a thread has at most four warps)
    return U == 1 ? total_few(buf, 0) : total_many(buf, 0, tm.nw, tm.lane);
  };
  float s = squares();
  Norm n{1.0f, 0.0f};
  if (!(s <= FLT_MAX)) {
    n.pre = kShrink;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) x[u][i] = mul(x[u][i], both(kShrink));
    tm.sync();
    s = squares();
    eps *= kShrink * kShrink;
  }
  n.r = inv_rms(s, inv_h, eps);
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

// What a token's assignments say, one a lane: its row (-1: none), its weight; and
// the token's gate.  Loaded two tokens ahead.
struct Meta {
  int32_t row;
  float w, g;
};
__device__ __forceinline__ Meta load_meta(const int32_t *dest_row, const float *topk_w,
                                          const float *gate, int64_t t, int64_t T, int k, int lane) {
  Meta m{-1, 0.0f, 1.0f};
  if (t < T) {
    if (lane < k) {
      m.row = __ldg(dest_row + t * k + lane);
      if (topk_w) m.w = __ldg(topk_w + t * k + lane);
    }
    if (gate) m.g = __ldg(gate + t);
  }
  return m;
}
// Rows outside are reported and dropped; a dropped assignment weighs nothing.
template <bool ALONE>
__device__ __forceinline__ void settle(Meta &m, const Rows &p, int64_t t, int k,
                                       const Team<ALONE> &tm) {
  if (m.row != -1 && (m.row < 0 || m.row >= p.n_rows)) {
    if (tm.warp == 0)
      moe::report_error(p.status, MOE_ERR_DEVICE_INDEX, (int32_t)(t * k + tm.lane), moe::K_BLOCK);
    m.row = -1;
  }
  if (m.row < 0) m.w = 0.0f;
}
// A token's rows to a thread's places, `step` bytes apart: zeros for dropped ones
// and for threads past the row's end (which take its last piece's address c).
__device__ __forceinline__ void copy_rows(uint32_t dst, int step, const uint4 *rows, const Meta &m,
                                          int k, int H8, int c, bool in) {
#pragma unroll 4
  for (int j = 0; j < k; ++j) {
    const int32_t r = __shfl_sync(0xffffffffu, m.row, j);
    copy_async(dst + j * step, rows + (int64_t)max(r, 0) * H8 + c, in && r >= 0);
  }
}

// out = x / rms(x) * weight.  R / U tokens are on their way.  Bound by HBM: 16384
// rows of 4096 in fp32 59 us, 6.8 TB/s; 4096 rows of 1024 in bf16 4.6 us.
template <int U, int R, typename X>
__global__ void __launch_bounds__(kRowThreads, U <= 2 ? 2 : 1)
    norm_kernel(const X *x, int64_t T, int H, const float *__restrict__ weight, float eps,
                __nv_bfloat16 *out) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) float buf[2][kLine];
  const Team<true> tm((int)blockDim.x);
  const int H8 = H / 8, slot = tm.threads * 16 * Chunk<X>::N;
  const float inv_h = 1.0f / (float)H;
  uint8_t *mine = smem + tm.warp * 512 * Chunk<X>::N;  // the warp's places
  const uint32_t dst = smem_u32(mine);
  if constexpr (U == 1) {
    clear_sums(buf[0], 2 * kLine, tm.tid, tm.threads);
    __syncthreads();
  }
  moe::pdl_wait();
  moe::pdl_trigger();
  auto fetch = [&](int64_t t, int u, int at) {
    if (t < T) Chunk<X>::copy(dst + at * slot, x + t * H, tm.tid + u * tm.threads, H8, tm.lane);
    copy_commit();
  };
  static_assert(R % U == 0, "whole tokens");
#pragma unroll
  for (int u = 0; u < R; ++u) fetch(blockIdx.x + u / U * (int64_t)gridDim.x, u % U, u);
  int par = 0, at = 0;
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x, par ^= 1) {
    Pair v[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      copy_wait<R - 1>();
      __syncwarp();  // the warp's copies are there
      Chunk<X> in;
      in.take(mine + (at + u) * slot, tm.lane);
      in.get(v[u]);
      __syncwarp();  // and used
      fetch(t + R / U * (int64_t)gridDim.x, u, at + u);
    }
    at = at + U == R ? 0 : at + U;
    const Norm n = row_norm(v, inv_h, eps, buf[par], tm);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = tm.tid + u * tm.threads;
      if (c >= H8) continue;
      Pair w[4];
      load_weight(weight, c, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = mul(mul(v[u][i], both(n.r)), w[i]);
      *reinterpret_cast<uint4 *>(out + t * H + 8 * c) = pack(w);
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
// One CTA a token at a time; c and then y stay in registers across the two sums.
// Bound by HBM where there are rows enough: 4096 tokens of 7168, eight experts, a
// shared one and next norm 108 us, 6.5 TB/s; 16384 of 4096 in fp32, four experts,
// 163 us, 6.6 TB/s.  A single token takes 4.2 us in a graph, most of it the launch.
template <int U, int R, typename X>
__global__ void __launch_bounds__(kRowThreads, U == 1 ? 2 : 1)
    combine_norm_kernel(const CombineNormParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) float buf[2][2][kLine];
  const Team<true> tm((int)blockDim.x);
  const int H8 = p.H / 8, step = tm.threads * 16;
  const float inv_h = 1.0f / (float)p.H;
  const int at_res = p.k * step, at_shared = at_res + Chunk<X>::N * step;
  const int slot = at_shared + (p.shared ? step : 0);
  uint8_t *mine = smem + tm.tid * 16;
  const uint32_t dst = smem_u32(mine);
  const int warp_res = at_res + (tm.warp * Chunk<X>::N * 32 - tm.tid) * 16;  // from `mine`
  if constexpr (U == 1) {
    clear_sums(buf[0][0], 4 * kLine, tm.tid, tm.threads);
    __syncthreads();
  }
  moe::pdl_wait();
  moe::pdl_trigger();
  auto meta = [&](int64_t t) {
    return load_meta(p.rows.dest_row, p.topk_w, p.gate, t, p.T, p.k, tm.lane);
  };
  auto fetch = [&](int64_t t, const Meta &m, int u) {
    if (t < p.T) {
      const int c = tm.tid + u * tm.threads, cl = min(c, H8 - 1);
      const bool in = c < H8;
      const uint32_t d = dst + (u % R) * slot;
      copy_rows(d, step, p.yp, m, p.k, H8, cl, in);
      // (y may be the residual itself: a token's row is read before it is written)
      Chunk<X>::copy(d + warp_res, static_cast<const X *>(p.residual) + t * p.H, c, H8, tm.lane);
      if (p.shared) copy_async(d + at_shared, p.shared + t * H8 + cl, in);
    }
    copy_commit();
  };
  const int64_t stride = gridDim.x;
  Meta now = meta(blockIdx.x), next = meta(blockIdx.x + stride);
  settle(now, p.rows, blockIdx.x, p.k, tm);
#pragma unroll
  for (int u = 0; u < R; ++u) fetch(blockIdx.x, now, u);
  int par = 0;
  for (int64_t t = blockIdx.x; t < p.T; t += stride, par ^= 1) {
    settle(next, p.rows, t + stride, p.k, tm);
    const Meta after = meta(t + 2 * stride);
    Pair acc[U][4];
    Chunk<X> res[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      copy_wait<R - 1>();
      __syncwarp();  // the warp's copies are there
      const uint8_t *s = mine + (u % R) * slot;
      res[u].take(s + warp_res, tm.lane);
      uint4 first = make_uint4(0, 0, 0, 0);
      if (p.shared) first = *reinterpret_cast<const uint4 *>(s + at_shared);
      unpack(first, acc[u]);
#pragma unroll 4
      for (int j = 0; j < p.k; ++j) {
        const Pair w = both(__shfl_sync(0xffffffffu, now.w, j));
        Pair f[4];
        unpack(*reinterpret_cast<const uint4 *>(s + j * step), f);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[u][i] = fma(w, f[i], acc[u][i]);
      }
      __syncwarp();  // and used
      if (u + R < U)
        fetch(t, now, u + R);
      else
        fetch(t + stride, next, (u + R) % U);
    }
    float rc = 1.0f;
    if (p.post) rc = row_norm(acc, inv_h, p.eps, buf[par][0], tm).r;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = tm.tid + u * tm.threads;
      Pair wt[4], x[4];
      load_weight(p.weight, min(c, H8 - 1), wt);
      res[u].get(x);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const Pair f = mul(mul(acc[u][i], both(rc)), wt[i]);
        acc[u][i] = fma(both(p.scale), x[i], mul(both(now.g), f));
      }
      res[u].set(acc[u]);
      res[u].store(static_cast<X *>(p.y) + t * p.H, c, H8, tm.lane);
      res[u].get(acc[u]);  // as it is held
      if (c >= H8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[u][i] = 0;
      }
    }
    if (p.next) {
      const Norm n = row_norm(acc, inv_h, p.eps, buf[par][1], tm);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = tm.tid + u * tm.threads;
        if (c >= H8) continue;
        Pair wt[4];
        load_weight(p.next_weight, c, wt);
#pragma unroll
        for (int i = 0; i < 4; ++i) wt[i] = mul(mul(acc[u][i], both(n.r)), wt[i]);
        p.next[t * H8 + c] = pack(wt);
      }
    }
    now = next;
    next = after;
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
// waits for the sums, so the row streams through in chunks.  Bound by HBM: 4096
// tokens of 7168, eight experts, 148 us, 6.7 TB/s.
template <int KMAX, typename X>
__global__ void __launch_bounds__(128) combine_bwd_kernel(const CombineBwdParams p) {
  __shared__ __align__(16) float buf[2][KMAX * kLine];
  clear_sums(buf[0], 2 * KMAX * kLine, threadIdx.x, blockDim.x);
  __syncthreads();
  moe::pdl_wait();
  moe::pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, H8 = p.H / 8;
  int par = 0;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, par ^= 1) {
    int32_t r[KMAX];
    const uint32_t live = token_rows(p.rows, t, p.k, r);
    float w[KMAX], sums[KMAX];
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
      if (j < p.k) w[j] = __ldg(p.topk_w + t * p.k + j);
      sums[j] = 0.0f;
    }
    for (int c = threadIdx.x; c < H8; c += blockDim.x) {
      uint4 v[KMAX];
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if ((live >> j) & 1u) v[j] = moe::ld_stream_u4(p.yp + (int64_t)r[j] * H8 + c);
      Chunk<X> in;
      in.load(static_cast<const X *>(p.gy) + t * p.H + 8 * c);
      Pair g[4];
      in.get(g);
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if ((live >> j) & 1u) {
          Pair f[4], o[4];
          unpack(v[j], f);
          sums[j] += dot(g, f);
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = mul(both(w[j]), g[i]);
          p.gyp[(int64_t)r[j] * H8 + c] = pack(o);
        }
    }
    put_sums(sums, buf[par], warp, lane);
    __syncthreads();
    if ((int)threadIdx.x < p.k) p.gw[t * p.k + threadIdx.x] = total_few(buf[par], threadIdx.x);
  }
}

// A norm weight's gradient over a CTA's tokens: the teams' sums, added in order,
// to the CTA's partial row.  Uses the CTA's shared memory from its start.
template <int U>
__device__ __forceinline__ void put_partial(const Pair (&pw)[U][4], float *partial, int H, int teams,
                                            float *smem, const Team<false> &tm) {
  __syncthreads();  // (all copies to shared memory have been waited for)
  const int H8 = H / 8;
  Chunk<float> o;
  if (tm.index > 0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = tm.tid + u * tm.threads;
      if (c >= H8) continue;
      o.set(pw[u]);
      o.put(smem + (tm.index - 1) * H + 8 * c);
    }
  }
  __syncthreads();
  if (tm.index > 0) return;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = tm.tid + u * tm.threads;
    if (c >= H8) continue;
    Pair a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = pw[u][i];
    for (int m = 1; m < teams; ++m) {
      o.load(smem + (m - 1) * H + 8 * c);
      o.get(b);
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = plus(a[i], b[i]);
    }
    o.set(a);
    o.put(partial + (int64_t)blockIdx.x * H + 8 * c);
  }
}

// The gradient through norm and gate.  With e = gy weight, one pass over the
// rows gives c (the sum over j of a piece is complete before the next piece)
// and all of sum c^2, sum e c, e . Y_j and c . Y_j, so the expert rows are read
// once and need not be kept:
//   dc = gate r (e - c m),  m = r^2 mean(e c),  dw_j = gate r (e . Y_j - m c . Y_j).
// The weight's gradient is kept per thread over the CTA's tokens and added up
// by sum_partials_kernel in a fixed order.  With that kernel, 16384 tokens of 4096 in
// fp32, four experts: 243 us, 5.5 TB/s; 4096 of 7168, eight experts and a shared one:
// 216 us, 6.0 TB/s; 4096 of 1440, six and a shared one: 46 us, 3.9 TB/s.  Bound by
// latency at 16 warps an SM (128 registers; at 80 they spill, 434 us): issue is at 60%,
// HBM at 61%, and of the 6.6 cycles from a warp's instruction to its next 1.7 wait for
// a result of fixed latency, 1.2 for shared memory and 0.6 for global memory.  Leaving
// out one of the two dots, the weight's gradient or the stores saves a tenth each.
// Rows beyond 8192, or more than eight experts, spill: 2048 tokens of 12288 with four
// experts 161 us (2.8 TB/s), with 16 experts 581 us (2.9 TB/s).
template <int KMAX, int U, int R, typename X>
__global__ void __launch_bounds__(kRowThreads)
    combine_norm_bwd_kernel(const CombineBwdParams p, const int team_threads) {
  constexpr int kSums = 2 * KMAX;
  constexpr int kBuf = sums_floats(kSums + 2);
  extern __shared__ __align__(128) uint8_t smem[];
  const Team<false> tm(team_threads);
  const int teams = blockDim.x / team_threads;
  const int H8 = p.H / 8, step = tm.threads * 16;
  const float inv_h = 1.0f / (float)p.H;
  const int at_gy = p.k * step, at_shared = at_gy + Chunk<X>::N * step;
  const int slot = at_shared + (p.shared ? step : 0);
  float *buf = reinterpret_cast<float *>(smem) + tm.index * 2 * kBuf;
  uint8_t *rings = smem + teams * 2 * kBuf * 4;
  uint8_t *mine = rings + tm.index * R * slot + tm.tid * 16;
  const uint32_t dst = smem_u32(mine);
  const int warp_gy = at_gy + (tm.warp * Chunk<X>::N * 32 - tm.tid) * 16;  // from `mine`
  clear_sums(buf, 2 * kBuf, tm.tid, tm.threads);
  __syncthreads();
  moe::pdl_wait();
  moe::pdl_trigger();
  auto meta = [&](int64_t t) {
    return load_meta(p.rows.dest_row, p.topk_w, p.gate, t, p.T, p.k, tm.lane);
  };
  auto fetch = [&](int64_t t, const Meta &m, int u) {
    if (t < p.T) {
      const int c = tm.tid + u * tm.threads, cl = min(c, H8 - 1);
      const bool in = c < H8;
      const uint32_t d = dst + (u % R) * slot;
      copy_rows(d, step, p.yp, m, p.k, H8, cl, in);
      Chunk<X>::copy(d + warp_gy, static_cast<const X *>(p.gy) + t * p.H, c, H8, tm.lane);
      if (p.shared) copy_async(d + at_shared, p.shared + t * H8 + cl, in);
    }
    copy_commit();
  };
  const int64_t first = (int64_t)blockIdx.x * teams + tm.index, stride = (int64_t)gridDim.x * teams;
  Meta now = meta(first), next = meta(first + stride);
  settle(now, p.rows, first, p.k, tm);
#pragma unroll
  for (int u = 0; u < R; ++u) fetch(first, now, u);
  Pair pw[U][4];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < 4; ++i) pw[u][i] = 0;
  int par = 0;
  for (int64_t t = first; t < p.T; t += stride, par ^= 1) {
    settle(next, p.rows, t + stride, p.k, tm);
    const Meta after = meta(t + 2 * stride);
    Pair acc[U][4];
    Chunk<X> gin[U];
    float d[kSums], s[2] = {0.0f, 0.0f};  // e . Y_j, then c . Y_j
    float w[KMAX];
#pragma unroll
    for (int j = 0; j < KMAX; ++j) w[j] = __shfl_sync(0xffffffffu, now.w, j);
#pragma unroll
    for (int j = 0; j < kSums; ++j) d[j] = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      copy_wait<R - 1>();
      __syncwarp();  // the warp's copies are there
      const uint8_t *sp = mine + (u % R) * slot;
      Pair e[4], f[4];
      load_weight(p.weight, min(tm.tid + u * tm.threads, H8 - 1), f);
      gin[u].take(sp + warp_gy, tm.lane);
      gin[u].get(e);
#pragma unroll
      for (int i = 0; i < 4; ++i) e[i] = mul(e[i], f[i]);
      uint4 v = make_uint4(0, 0, 0, 0);
      if (p.shared) v = *reinterpret_cast<const uint4 *>(sp + at_shared);
      unpack(v, acc[u]);
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if (j < p.k) {
          unpack(*reinterpret_cast<const uint4 *>(sp + j * step), f);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[u][i] = fma(both(w[j]), f[i], acc[u][i]);
          d[j] += dot(e, f);
        }
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if (j < p.k) {
          unpack(*reinterpret_cast<const uint4 *>(sp + j * step), f);
          d[KMAX + j] += dot(acc[u], f);
        }
      s[0] += dot(acc[u], acc[u]);
      s[1] += dot(e, acc[u]);
      __syncwarp();  // and used
      if (u + R < U)
        fetch(t, now, u + R);
      else
        fetch(t + stride, next, (u + R) % U);
    }
    float *b = buf + par * kBuf;
    put_sums(d, b, tm.warp, tm.lane);
    put_sums(s, b + kSums * kLine, tm.warp, tm.lane);
    const bool wide = tm.any(!(small(d[0]) && small(s[0])));
    const float g = now.g;
    float s1 = total(b, kSums, tm.nw, tm.lane), s2 = total(b, kSums + 1, tm.nw, tm.lane);
    float pre = 1.0f, rc = 1.0f, m = 0.0f;
    float hat, ec;  // c / rms(c) is acc * hat; the sum of e with it
    if (!wide) {
      if (p.post) {
        rc = inv_rms(s1, inv_h, p.eps);
        m = rc * rc * (s2 * inv_h);
      }
      hat = rc;
      ec = s2 * rc;
      for (int j = tm.warp; j < p.k; j += tm.nw) {
        const float ey = total(b, j, tm.nw, tm.lane), cy = total(b, KMAX + j, tm.nw, tm.lane);
        float dw = g * rc * (ey - m * cy);
        // (the product of two sums may pass the range where that with gate and r does not)
        if (!(fabsf(m * cy) <= FLT_MAX)) dw = g * rc * ey - g * rc * m * cy;
        if (tm.lane == j) p.gw[t * p.k + j] = now.row < 0 ? 0.0f : dw;
      }
    } else {
      // A sum is not within fp32's range: of c^2, e c, or products with rows far larger
      // than c.  c is brought to rms 1 first, after which e's mean with it is no larger
      // than e, and dw_j comes from a pass over o = e - c mean(e c) and Y_j, with Y_j as
      // it is and times 2^-72.  Without the norm c takes no part, and may be infinite or
      // NaN.  (Rare, but here and not in a function that is called, whose conventions
      // cost the other tokens registers: 16384 x 4096, four experts, 457 us.)
      ec = s2;
      if (p.post) {
        float eps = p.eps;
        auto sum_again = [&]() {
          tm.sync();
          put_sums(s, b + kSums * kLine, tm.warp, tm.lane);
          tm.sync();
        };
        s[0] = s[1] = 0.0f;
        if (!(s1 <= FLT_MAX)) {
          pre = kShrink;
          eps *= kShrink * kShrink;
#pragma unroll
          for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[u][i] = mul(acc[u][i], both(kShrink));
            s[0] += dot(acc[u], acc[u]);
          }
          sum_again();
          s1 = total(b, kSums, tm.nw, tm.lane);
        }
        rc = inv_rms(s1, inv_h, eps);
        s[0] = 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          Pair e[4], f[4];
          load_weight(p.weight, min(tm.tid + u * tm.threads, H8 - 1), f);
          gin[u].get(e);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            acc[u][i] = mul(acc[u][i], both(rc));
            e[i] = mul(e[i], f[i]);
            f[i] = mul(acc[u][i], both(inv_h));
          }
          s[0] += dot(e, f);
        }
        sum_again();
        m = total(b, kSums, tm.nw, tm.lane);
        ec = m * (float)p.H;
#pragma unroll
        for (int j = 0; j < kSums; ++j) d[j] = 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int c = tm.tid + u * tm.threads;
          Pair o[4], f[4];
          load_weight(p.weight, min(c, H8 - 1), f);
          gin[u].get(o);
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = fma(both(-m), acc[u][i], mul(o[i], f[i]));
#pragma unroll
          for (int j = 0; j < KMAX; ++j) {
            const int32_t r = __shfl_sync(0xffffffffu, now.row, j);
            if (c < H8 && r >= 0) {
              unpack(moe::ld_stream_u4(p.yp + (int64_t)r * H8 + c), f);
              d[j] += dot(o, f);
#pragma unroll
              for (int i = 0; i < 4; ++i) f[i] = mul(f[i], both(kShrink));
              d[KMAX + j] += dot(o, f);
            }
          }
        }
        put_sums(d, b, tm.warp, tm.lane);
        tm.sync();
        for (int j = tm.warp; j < p.k; j += tm.nw) {
          const float y = total(b, j, tm.nw, tm.lane), less = total(b, KMAX + j, tm.nw, tm.lane);
          const float dw = fabsf(y) <= FLT_MAX ? g * rc * y * pre : g * rc * less * (pre / kShrink);
          if (tm.lane == j) p.gw[t * p.k + j] = now.row < 0 ? 0.0f : dw;
        }
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[u][i] = 0;
        for (int j = tm.warp; j < p.k; j += tm.nw) {
          const float ey = total(b, j, tm.nw, tm.lane);
          if (tm.lane == j) p.gw[t * p.k + j] = now.row < 0 ? 0.0f : g * ey;
        }
      }
      hat = 1.0f;
    }
    if (p.ggate && tm.tid == 0) p.ggate[t] = ec;
    const Pair a = both(g * rc * pre), minus_m = both(-m);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = tm.tid + u * tm.threads;
      const bool in = c < H8;
      Pair gy[4], o[4];
      load_weight(p.weight, min(c, H8 - 1), o);
      gin[u].get(gy);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (p.partial)
          pw[u][i] = fma(mul(both(g), gy[i]), mul(acc[u][i], both(hat)), pw[u][i]);
        gy[i] = mul(a, fma(minus_m, acc[u][i], mul(gy[i], o[i])));
      }
      if (in && p.gshared) p.gshared[t * H8 + c] = pack(gy);
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if (j < p.k) {
          const int32_t r = __shfl_sync(0xffffffffu, now.row, j);
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = mul(both(w[j]), gy[i]);
          if (in && r >= 0) p.gyp[(int64_t)r * H8 + c] = pack(o);
        }
    }
    now = next;
    next = after;
  }
  copy_wait<0>();
  if (p.partial) put_partial(pw, p.partial, p.H, teams, reinterpret_cast<float *>(smem), tm);
}

struct NormBwdParams {
  const uint4 *grad;
  Rows rows;  // dest_row NULL: grad has a row a token, and k is 1
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
// With sum_partials_kernel, 16384 rows of 4096 in fp32, four copies each: 231 us,
// 6.4 TB/s; 2048 of 12288 (which spill) 100 us, 3.5 TB/s.
template <int U, int R, typename X>
__global__ void __launch_bounds__(kRowThreads)
    norm_bwd_kernel(const NormBwdParams p, const int team_threads) {
  constexpr int kBuf = sums_floats(2);
  extern __shared__ __align__(128) uint8_t smem[];
  const Team<false> tm(team_threads);
  const int teams = blockDim.x / team_threads;
  const int H8 = p.H / 8, step = tm.threads * 16;
  const float inv_h = 1.0f / (float)p.H;
  const int at_x = p.k * step, at_add = at_x + Chunk<X>::N * step;
  const int at_res = at_add + (p.add ? step : 0);
  const int slot = at_res + (p.rgrad ? Chunk<X>::N * step : 0);
  float *buf = reinterpret_cast<float *>(smem) + tm.index * 2 * kBuf;
  uint8_t *rings = smem + teams * 2 * kBuf * 4;
  uint8_t *mine = rings + tm.index * R * slot + tm.tid * 16;
  const uint32_t dst = smem_u32(mine);
  const int warp_at = (tm.warp * Chunk<X>::N * 32 - tm.tid) * 16;  // the warp's places, from `mine`
  clear_sums(buf, 2 * kBuf, tm.tid, tm.threads);
  __syncthreads();
  moe::pdl_wait();
  moe::pdl_trigger();
  auto meta = [&](int64_t t) {
    if (p.rows.dest_row)
      return load_meta(p.rows.dest_row, nullptr, nullptr, t, p.T, p.k, tm.lane);
    return Meta{tm.lane == 0 && t < p.T ? (int32_t)t : -1, 0.0f, 1.0f};
  };
  auto fetch = [&](int64_t t, const Meta &m, int u) {
    if (t < p.T) {
      const int c = tm.tid + u * tm.threads, cl = min(c, H8 - 1);
      const bool in = c < H8;
      const uint32_t d = dst + (u % R) * slot;
      copy_rows(d, step, p.grad, m, p.k, H8, cl, in);
      Chunk<X>::copy(d + at_x + warp_at, static_cast<const X *>(p.x) + t * p.H, c, H8, tm.lane);
      // (gx may be rgrad itself: a token's row is read before it is written)
      if (p.rgrad)
        Chunk<X>::copy(d + at_res + warp_at, static_cast<const X *>(p.rgrad) + t * p.H, c, H8, tm.lane);
      if (p.add) copy_async(d + at_add, p.add + t * H8 + cl, in);
    }
    copy_commit();
  };
  const int64_t first = (int64_t)blockIdx.x * teams + tm.index, stride = (int64_t)gridDim.x * teams;
  Meta now = meta(first), next = meta(first + stride);
  settle(now, p.rows, first, p.k, tm);
#pragma unroll
  for (int u = 0; u < R; ++u) fetch(first, now, u);
  Pair pw[U][4];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < 4; ++i) pw[u][i] = 0;
  int par = 0;
  for (int64_t t = first; t < p.T; t += stride, par ^= 1) {
    settle(next, p.rows, t + stride, p.k, tm);
    const Meta after = meta(t + 2 * stride);
    Pair acc[U][4], x[U][4];
    float s[2] = {0.0f, 0.0f};
    Chunk<X> res[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      copy_wait<R - 1>();
      __syncwarp();  // the warp's copies are there
      const uint8_t *sp = mine + (u % R) * slot;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (p.add) v = *reinterpret_cast<const uint4 *>(sp + at_add);
      unpack(v, acc[u]);
      Chunk<X> in;
      in.take(sp + at_x + warp_at, tm.lane);
      in.get(x[u]);
      if (p.rgrad) res[u].take(sp + at_res + warp_at, tm.lane);
#pragma unroll 4
      for (int j = 0; j < p.k; ++j) {
        Pair f[4];
        unpack(*reinterpret_cast<const uint4 *>(sp + j * step), f);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[u][i] = plus(acc[u][i], f[i]);
      }
      Pair e[4];
      load_weight(p.weight, min(tm.tid + u * tm.threads, H8 - 1), e);
#pragma unroll
      for (int i = 0; i < 4; ++i) e[i] = mul(acc[u][i], e[i]);
      s[0] += dot(x[u], x[u]);
      s[1] += dot(e, x[u]);
      __syncwarp();  // and used
      if (u + R < U)
        fetch(t, now, u + R);
      else
        fetch(t + stride, next, (u + R) % U);
    }
    float *b = buf + par * kBuf;
    put_sums(s, b, tm.warp, tm.lane);
    const bool wide = tm.any(!small(s[0]));
    float s1 = total(b, 0, tm.nw, tm.lane);
    const float s2 = total(b, 1, tm.nw, tm.lane);
    float pre = 1.0f, rc, m, hat;
    if (!wide) {
      rc = hat = inv_rms(s1, inv_h, p.eps);
      m = rc * rc * (s2 * inv_h);
    } else {
      // sums beyond fp32's range: x is brought to rms 1 first, and e's mean with it is
      // no larger than e
      float eps = p.eps;
      auto sum_again = [&]() {
        tm.sync();
        put_sums(s, b, tm.warp, tm.lane);
        tm.sync();
        return total(b, 0, tm.nw, tm.lane);
      };
      s[0] = s[1] = 0.0f;
      if (!(s1 <= FLT_MAX)) {  // as in row_norm
        pre = kShrink;
        eps *= kShrink * kShrink;
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
          for (int i = 0; i < 4; ++i) x[u][i] = mul(x[u][i], both(kShrink));
          s[0] += dot(x[u], x[u]);
        }
        s1 = sum_again();
      }
      rc = inv_rms(s1, inv_h, eps);
      s[0] = 0.0f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        Pair e[4], f[4];
        load_weight(p.weight, min(tm.tid + u * tm.threads, H8 - 1), e);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[u][i] = mul(x[u][i], both(rc));
          e[i] = mul(acc[u][i], e[i]);
          f[i] = mul(x[u][i], both(inv_h));
        }
        s[0] += dot(e, f);
      }
      m = sum_again();
      hat = 1.0f;
    }
    const Pair a = both(rc * pre), minus_m = both(-m);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = tm.tid + u * tm.threads;
      Pair wt[4], o[4];
      load_weight(p.weight, min(c, H8 - 1), wt);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (p.partial) pw[u][i] = fma(acc[u][i], mul(x[u][i], both(hat)), pw[u][i]);
        wt[i] = mul(a, fma(minus_m, x[u][i], mul(acc[u][i], wt[i])));
      }
      if (p.rgrad) {
        res[u].get(o);
#pragma unroll
        for (int i = 0; i < 4; ++i) wt[i] = fma(both(p.scale), o[i], wt[i]);
      }
      Chunk<X> out;
      out.set(wt);
      out.store(static_cast<X *>(p.gx) + t * p.H, c, H8, tm.lane);
    }
    now = next;
    next = after;
  }
  copy_wait<0>();
  if (p.partial) put_partial(pw, p.partial, p.H, teams, reinterpret_cast<float *>(smem), tm);
}

// grad_x[t] = add[t] + sum_j grad[row_j].  Bound by HBM: 4096 tokens of 7168, eight
// copies each, 84 us, 7.0 TB/s (results still in L2).
template <int KMAX, typename X>
__global__ void __launch_bounds__(128)
    permute_bwd_kernel(const uint4 *__restrict__ grad, Rows rows, const uint4 *__restrict__ add,
                       int64_t T, int k, int H, X *__restrict__ gx) {
  moe::pdl_wait();
  moe::pdl_trigger();
  const int H8 = H / 8, lane = threadIdx.x & 31;
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
    int32_t r[KMAX];
    const uint32_t live = token_rows(rows, t, k, r);
    for (int c0 = threadIdx.x - lane; c0 < H8; c0 += blockDim.x) {
      const int c = c0 + lane;
      const bool in = c < H8;
      uint4 v[KMAX];
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if (in && (live >> j & 1u)) v[j] = moe::ld_stream_u4(grad + (int64_t)r[j] * H8 + c);
      Pair acc[4], f[4];
      uint4 first = make_uint4(0, 0, 0, 0);
      if (in && add) first = moe::ld_stream_u4(add + t * H8 + c);
      unpack(first, acc);
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if (live >> j & 1u) {
          unpack(v[j], f);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[i] = plus(acc[i], f[i]);
        }
      Chunk<X> out;
      out.set(acc);
      out.store(gx + t * H, c, H8, lane);
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
// Dynamic shared memory that with the static passes 48 KB, asked for once a
// kernel and device.
template <auto KERNEL>
moe_status allow_smem(size_t bytes) {
  constexpr int kMaxDevices = 64;
  static bool done[kMaxDevices] = {false};
  if (bytes <= 40 * 1024) return MOE_OK;
  int dev = 0;
  if (moe_host::refused(cudaGetDevice(&dev))) return MOE_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices || !done[dev]) {
    if (moe_host::refused(cudaFuncSetAttribute(
            KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit)))
      return MOE_ERR_CUDA;
    if (dev >= 0 && dev < kMaxDevices) done[dev] = true;
  }
  return MOE_OK;
}

template <auto KERNEL, typename... A>
moe_status launch_rows(int64_t T, int threads, int sm_threads, size_t smem, cudaStream_t st,
                       A... args) {
  if (moe_status s = allow_smem<KERNEL>(smem)) return s;
  const unsigned grid = rows_grid(T, threads, sm_threads, smem, moe_host::sm_count());
  return moe_host::launch_pdl(KERNEL, dim3(grid), dim3((unsigned)threads), smem, st, args...);
}

template <auto KERNEL, typename P>
moe_status launch_teams(const P &p, const TeamShape &s, cudaStream_t st) {
  if (moe_status e = allow_smem<KERNEL>(s.smem)) return e;
  return moe_host::launch_pdl(KERNEL, dim3(s.grid), dim3((unsigned)(s.teams * s.threads)), s.smem, st,
                              p, s.threads);
}

bool bad_type(int32_t type) { return type != MOE_F32 && type != MOE_BF16; }
bool odd(const void *p) { return !moe_host::aligned16(p); }
// The gradients take 1 / eps (of rows of zeros), the norms mean(x^2) + eps with a mean of
// up to 2^125: both stay within fp32's range.
bool bad_eps(float eps) { return !(eps >= 0x1p-126f && eps <= 0x1p127f); }

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
  const int n = threads_of(p.H, U);
  const size_t ring = (size_t)n * 16 * (p.k + Chunk<X>::N + (p.shared ? 1 : 0));
  if constexpr (U > 1) {
    if (2 * ring <= kSmemLimit)
      return launch_rows<combine_norm_kernel<U, 2, X>>(p.T, n, 512, 2 * ring, st, p);
  }
  return launch_rows<combine_norm_kernel<U, 1, X>>(p.T, n, U == 1 ? 1024 : 512, ring, st, p);
}

template <typename X>
moe_status run_combine_bwd(const CombineBwdParams &p, cudaStream_t st) {
  const unsigned g = stream_grid(p.T, moe_host::sm_count());
  const int n = stream_threads(p.H);
  if (p.k <= 2) return launch(combine_bwd_kernel<2, X>, g, n, st, p);
  if (p.k <= 4) return launch(combine_bwd_kernel<4, X>, g, n, st, p);
  if (p.k <= 8) return launch(combine_bwd_kernel<8, X>, g, n, st, p);
  return launch(combine_bwd_kernel<16, X>, g, n, st, p);
}

template <int KMAX, int U, typename X>
moe_status run_combine_norm_bwd_k(const CombineBwdParams &p, unsigned &grid, cudaStream_t st) {
  const int n = p.k + Chunk<X>::N + (p.shared ? 1 : 0);
  const TeamShape s(p.T, p.H, n, 2 * KMAX + 2, p.partial != nullptr, moe_host::sm_count());
  grid = s.grid;
  return s.r == 2 ? launch_teams<combine_norm_bwd_kernel<KMAX, U, 2, X>>(p, s, st)
                  : launch_teams<combine_norm_bwd_kernel<KMAX, U, 1, X>>(p, s, st);
}
template <int U, typename X>
moe_status run_combine_norm_bwd(const CombineBwdParams &p, unsigned &grid, cudaStream_t st) {
  if (p.k <= 2) return run_combine_norm_bwd_k<2, U, X>(p, grid, st);
  if (p.k <= 4) return run_combine_norm_bwd_k<4, U, X>(p, grid, st);
  if (p.k <= 8) return run_combine_norm_bwd_k<8, U, X>(p, grid, st);
  return run_combine_norm_bwd_k<16, U, X>(p, grid, st);
}

template <int U, typename X>
moe_status run_norm_bwd(const NormBwdParams &p, unsigned &grid, cudaStream_t st) {
  const int n = p.k + Chunk<X>::N * (p.rgrad ? 2 : 1) + (p.add ? 1 : 0);
  const TeamShape s(p.T, p.H, n, 2, p.partial != nullptr, moe_host::sm_count());
  grid = s.grid;
  return s.r == 2 ? launch_teams<norm_bwd_kernel<U, 2, X>>(p, s, st)
                  : launch_teams<norm_bwd_kernel<U, 1, X>>(p, s, st);
}

template <typename X>
moe_status run_permute_bwd(const uint16_t *grad, const Rows &rows, const uint16_t *add, int64_t T,
                           int32_t k, int32_t H, void *gx, cudaStream_t st) {
  const dim3 g(stream_grid(T, moe_host::sm_count())), b((unsigned)stream_threads(H));
  const uint4 *in = reinterpret_cast<const uint4 *>(grad), *ad = reinterpret_cast<const uint4 *>(add);
  X *out = static_cast<X *>(gx);
  if (k <= 2) return moe_host::launch_pdl(permute_bwd_kernel<2, X>, g, b, 0, st, in, rows, ad, T, k, H, out);
  if (k <= 4) return moe_host::launch_pdl(permute_bwd_kernel<4, X>, g, b, 0, st, in, rows, ad, T, k, H, out);
  if (k <= 8) return moe_host::launch_pdl(permute_bwd_kernel<8, X>, g, b, 0, st, in, rows, ad, T, k, H, out);
  return moe_host::launch_pdl(permute_bwd_kernel<16, X>, g, b, 0, st, in, rows, ad, T, k, H, out);
}

template <int U, typename X>
moe_status run_norm(const void *x, int64_t T, int32_t H, const float *weight, float eps, uint16_t *out,
                    cudaStream_t st) {
  const int n = threads_of(H, U);
  constexpr int R = 2 * U;
  return launch_rows<norm_kernel<U, R, X>>(T, n, U <= 2 ? 1024 : 512, (size_t)n * 16 * R * Chunk<X>::N, st,
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
  return moe_host::refused(cudaMemsetAsync(grad_weight, 0, (size_t)H * 4, st)) ? MOE_ERR_CUDA : MOE_OK;
}

}  // namespace

extern "C" size_t moe_norm_scratch_bytes(int64_t T, int32_t H) {
  if (T < 1 || H < 8 || H % 8 != 0 || H > kMaxH) return 0;
  return (size_t)bwd_grid(T, H, moe_host::sm_count()) * (size_t)H * 4;
}

extern "C" moe_status moe_norm(const void *x, int32_t x_type, int64_t T, int32_t H,
                               const float *weight, float eps, uint16_t *out, void *stream) {
  if (bad_type(x_type) || bad_eps(eps)) return MOE_ERR_INVALID_ARG;
  if (moe_status s = check_sizes(T, 1, H, 0)) return s;
  if (T == 0) return MOE_OK;
  if (!x || !out || odd(x) || odd(out) || odd(weight)) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (fwd_pieces(H) == 1)
    return x_type == MOE_F32 ? run_norm<1, float>(x, T, H, weight, eps, out, st)
                             : run_norm<1, __nv_bfloat16>(x, T, H, weight, eps, out, st);
  if (fwd_pieces(H) == 2)
    return x_type == MOE_F32 ? run_norm<2, float>(x, T, H, weight, eps, out, st)
                             : run_norm<2, __nv_bfloat16>(x, T, H, weight, eps, out, st);
  return x_type == MOE_F32 ? run_norm<4, float>(x, T, H, weight, eps, out, st)
                           : run_norm<4, __nv_bfloat16>(x, T, H, weight, eps, out, st);
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
  p.grad = static_cast<const uint4 *>(n_rows > 0 ? grad : x);
  p.rows = Rows{dest_row, n_rows, moe_host::status_ptr(ws)};
  p.add = reinterpret_cast<const uint4 *>(add);
  p.x = x;
  p.T = T;
  p.k = dest_row ? k : 1;
  p.H = H;
  p.weight = weight;
  p.eps = eps;
  p.scale = residual_scale;
  p.rgrad = residual_grad;
  p.gx = grad_x;
  p.partial = grad_weight ? static_cast<float *>(scratch) : nullptr;
  const bool f32 = x_type == MOE_F32;
  unsigned grid = 0;
  moe_status s;
  if (row_chunks(H) == 2)
    s = f32 ? run_norm_bwd<2, float>(p, grid, st) : run_norm_bwd<2, __nv_bfloat16>(p, grid, st);
  else
    s = f32 ? run_norm_bwd<4, float>(p, grid, st) : run_norm_bwd<4, __nv_bfloat16>(p, grid, st);
  if (s != MOE_OK || !grad_weight) return s;
  return sum_partials(p.partial, grid, H, grad_weight, st);
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
  // (without rows nothing is read there, but addresses are formed)
  p.yp = static_cast<const uint4 *>(n_rows > 0 ? y_perm : residual);
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
  if (fwd_pieces(H) == 1)
    return x_type == MOE_F32 ? run_combine_norm<1, float>(p, st)
                             : run_combine_norm<1, __nv_bfloat16>(p, st);
  if (fwd_pieces(H) == 2)
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
  p.yp = static_cast<const uint4 *>(n_rows > 0 ? y_perm : grad_y);
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
  unsigned grid = 0;
  moe_status s;
  if (row_chunks(H) == 2)
    s = f32 ? run_combine_norm_bwd<2, float>(p, grid, st) : run_combine_norm_bwd<2, __nv_bfloat16>(p, grid, st);
  else
    s = f32 ? run_combine_norm_bwd<4, float>(p, grid, st) : run_combine_norm_bwd<4, __nv_bfloat16>(p, grid, st);
  if (s != MOE_OK || !grad_weight) return s;
  return sum_partials(p.partial, grid, H, grad_weight, st);
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
