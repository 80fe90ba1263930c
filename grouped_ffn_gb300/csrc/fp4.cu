// Rows in microscaled 4-bit floating point: quantization (plain, or straight
// into the dispatched rows), restoration, and the weight layout of the grouped
// product (fp4.cuh has the formats).
//
// Every step but the rounding to e2m1 (and, NV, the rounding of the scale to
// E4M3) is exact, so the codes are those of real arithmetic: an MX scale is a
// power of two; an NV quotient x / s is either exactly halfway between two
// codes or at least 2^-8 away in relative terms for bf16 x, which the bf16
// path uses, and fp32 x carries the sign of its division's remainder in the
// last bit (rounding to odd), so that a quotient next to a border never lands
// on it.
//
// Bound by HBM: 4096 rows of 7168 to eight dispatched rows each (184 MB) take
// 27 us, back to bf16 (595 MB) 95 us: 6.3 TB/s together, 0.95 of the measured
// copy bandwidth.  Flat over pieces of rows, since rows are of any length.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "fp4.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kVec = 32;  // elements a thread quantizes: one MX block, two NV blocks

// Pieces of rows, flat over (row, piece): thread i of a chunk of rows finds its
// row by a multiplication (a 64-bit division costs more than the rest of a
// piece).  Exact for i < 2^31; longer inputs take several chunks (grid.y).
struct Pieces {
  int64_t rows, chunk;  // all rows, rows a chunk
  uint32_t per_row, mul, shift;

  static Pieces of(int64_t rows, int per_row) {
    Pieces p;
    p.rows = rows;
    p.per_row = (uint32_t)per_row;
    p.chunk = ((int64_t)1 << 30) / per_row;
    if (p.chunk > rows) p.chunk = rows;
    // per_row in (2^(L-1), 2^L]: q = i * ceil(2^(31+L) / per_row) >> (31+L),
    // off by less than i * 2^-31 / per_row < 1 / per_row
    uint32_t L = 0;
    while (((uint64_t)1 << L) < (uint64_t)per_row) ++L;
    p.mul = (uint32_t)((((uint64_t)1 << (31 + L)) + per_row - 1) / per_row);
    p.shift = 31 + L;
    return p;
  }
  unsigned chunks() const { return (unsigned)((rows + chunk - 1) / chunk); }
  __device__ __forceinline__ uint32_t total() const {  // of this chunk
    const int64_t left = rows - blockIdx.y * chunk;
    return (uint32_t)(left < chunk ? left : chunk) * per_row;
  }
  __device__ __forceinline__ void at(uint32_t i, int64_t &row, int &piece) const {
    const uint32_t q = (uint32_t)((uint64_t)i * mul >> shift);
    row = blockIdx.y * chunk + q;
    piece = (int)(i - q * per_row);
  }
};

__device__ __forceinline__ float pow2f(int e) {  // e in [-127, 127]
  return e > -127 ? __int_as_float((127 + e) << 23) : __int_as_float(1 << 22);
}

// The quotient q = fl(a / b) of positive a, b with its last bit forced to 1
// unless it is exact: a border between two codes is then never hit by rounding.
__device__ __forceinline__ float div_to_odd(float a, float b) {
  const float q = __fdiv_rn(a, b);
  const float r = fmaf(-q, b, a);
  uint32_t u = __float_as_uint(q);
  if (r != 0.0f && !(u & 1u) && u > 0u && u < 0x7F800000u) u += r > 0.0f ? 1u : 0xFFFFFFFFu;
  return __uint_as_float(u);
}

__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 c;\n\tcvt.rn.satfinite.e2m1x2.f32 c, %2, %1;\n\tcvt.u32.u8 %0, c;\n\t}"
      : "=r"(r)
      : "f"(lo), "f"(hi));
  return r;
}

__device__ __forceinline__ float e4m3_value(uint32_t code) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)code, __NV_E4M3)));
}

// N consecutive elements of a row.
template <int N>
__device__ __forceinline__ void load_elems(const float *p, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const float4 f = __ldcs(reinterpret_cast<const float4 *>(p) + i);
    v[4 * i] = f.x;
    v[4 * i + 1] = f.y;
    v[4 * i + 2] = f.z;
    v[4 * i + 3] = f.w;
  }
}
template <int N>
__device__ __forceinline__ void load_elems(const __nv_bfloat16 *p, float (&v)[N]) {
  uint4 u[N / 8];
#pragma unroll
  for (int i = 0; i < N / 8; ++i) u[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
#pragma unroll
  for (int i = 0; i < N / 8; ++i) {
    const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      v[8 * i + 2 * c] = __uint_as_float(w[c] << 16);
      v[8 * i + 2 * c + 1] = __uint_as_float(w[c] & 0xFFFF0000u);
    }
  }
}

// Codes (N / 8 words) and the scale byte of a block of N elements.
template <int FMT, bool WIDE, int N>
__device__ __forceinline__ uint32_t quantize_block(const float *x, int scale_exp, uint32_t *w) {
  uint32_t m = 0;  // the largest magnitude, as fp32 bits
#pragma unroll
  for (int i = 0; i < N; ++i) m = max(m, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  uint32_t scale;
  float y[N];
  bool zero = false;
  if (FMT == 0) {
    // the smallest e in [-127, 127] with amax <= 6 * 2^e: amax = M 2^q gives
    // q - 2, plus one when M > 1.5
    const int e = max(-127, (int)(m >> 23) - 129 + ((m & 0x7FFFFFu) > 0x400000u ? 1 : 0));
    scale = (uint32_t)(e + 127);
    const float inv = pow2f(-e);
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = x[i] * inv;
  } else {
    const float down = pow2f(-scale_exp);
    const float a = __uint_as_float(m) * down;
    const float sixth = WIDE ? div_to_odd(a, 6.0f) : __fdiv_rn(a, 6.0f);
    scale = __nv_cvt_float_to_fp8(sixth, __NV_SATFINITE, __NV_E4M3);
    zero = scale == 0;
    const float s = e4m3_value(scale);
    if (WIDE) {
#pragma unroll
      for (int i = 0; i < N; ++i) y[i] = copysignf(div_to_odd(fabsf(x[i]) * down, s), x[i]);
    } else {
      // a multiple of 2^-18 nearest to x / s: codes' borders are such
      // multiples, and any other quotient is further from them than the
      // reciprocal's error and this rounding together (|y| > 6 saturates)
      const float inv = __frcp_rn(s) * down;
#pragma unroll
      for (int i = 0; i < N; ++i) y[i] = __fadd_rn(__fmaf_rn(x[i], inv, 48.0f), -48.0f);
    }
  }
#pragma unroll
  for (int i = 0; i < N / 8; ++i) {
    w[i] = 0;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      w[i] |= e2m1x2(y[8 * i + 2 * c], y[8 * i + 2 * c + 1]) << (8 * c);
  }
  const bool bad = m >= 0x7F800000u;  // an infinity or NaN: the block reads back as NaN
  if (bad) scale = fp4::Fmt<FMT>::kScaleBad;
  if (bad || zero) {
#pragma unroll
    for (int i = 0; i < N / 8; ++i) w[i] = 0;
  }
  return scale;
}

// Rows of x to codes and scales.  k == 0: row t to row t.  k > 0: row t once
// to each of its k dispatched rows dest_row[t*k + j] (-1: dropped).
// One thread per 32 elements, a 16-byte store of codes for each destination.
template <typename X, int FMT>
__global__ void __launch_bounds__(kThreads)
    quantize_kernel(const X *__restrict__ x, int64_t ldx, Pieces pieces, int K, int k,
                    const int32_t *__restrict__ dest_row, int64_t n_rows, int scale_exp,
                    uint8_t *__restrict__ codes, uint8_t *__restrict__ sf, int sf_ld,
                    int32_t *status) {
  moe::pdl_wait();
  moe::pdl_trigger();
  constexpr bool WIDE = sizeof(X) == 4;
  const uint32_t total = pieces.total(), stride = gridDim.x * kThreads;
  const int nsf = K / fp4::Fmt<FMT>::kBlock;
  for (uint32_t i = blockIdx.x * kThreads + threadIdx.x; i < total; i += stride) {
    int64_t t;
    int piece;
    pieces.at(i, t, piece);
    float v[kVec];
    load_elems<kVec>(x + t * ldx + (int64_t)piece * kVec, v);
    uint32_t w[4], scale;
    if constexpr (FMT == 0) {
      scale = quantize_block<FMT, WIDE, 32>(v, scale_exp, w);
    } else {
      scale = quantize_block<FMT, WIDE, 16>(v, scale_exp, w);
      scale |= quantize_block<FMT, WIDE, 16>(v + 16, scale_exp, w + 2) << 8;
    }
    const uint4 q = make_uint4(w[0], w[1], w[2], w[3]);
    const int n_dst = k == 0 ? 1 : k;
    for (int j = 0; j < n_dst; ++j) {
      int64_t r = t;
      if (k > 0) {
        r = __ldg(dest_row + t * k + j);
        if (r < 0 || r >= n_rows) {
          if (r != -1 && piece == 0)
            moe::report_error(status, MOE_ERR_DEVICE_INDEX, (int32_t)(t * k + j), moe::K_PERMUTE);
          continue;
        }
      }
      *reinterpret_cast<uint4 *>(codes + r * (K / 2) + piece * 16) = q;
      uint8_t *srow = sf + r * sf_ld;
      if (FMT == 1)
        reinterpret_cast<uint16_t *>(srow)[piece] = (uint16_t)scale;
      else
        srow[piece] = (uint8_t)scale;
      if (piece == (int)pieces.per_row - 1)
        for (int c = nsf; c < sf_ld; ++c) srow[c] = 0;
    }
  }
}

__device__ __forceinline__ float2 e2m1x2_value(uint32_t code) {
  uint32_t h;
  asm("{\n\t.reg .b8 c;\n\tcvt.u8.u32 c, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}"
      : "=r"(h)
      : "r"(code));
  return __half22float2(*reinterpret_cast<__half2 *>(&h));
}

// A 16-byte store a piece (8 bf16 or 4 fp32 values, 4 or 2 bytes of codes), so
// that a warp's stores cover whole lines; kDeqUnroll pieces in flight a thread.
constexpr int kDeqUnroll = 4;

template <typename Y, int FMT>
__global__ void __launch_bounds__(kThreads)
    dequant_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ sf, int sf_ld,
                   Pieces pieces, int K, int scale_exp, Y *__restrict__ out) {
  moe::pdl_wait();
  moe::pdl_trigger();
  constexpr int N = 16 / sizeof(Y);  // elements a piece
  const uint32_t total = pieces.total(), stride = gridDim.x * kThreads;
  for (uint32_t i0 = blockIdx.x * kThreads + threadIdx.x; i0 < total; i0 += stride * kDeqUnroll) {
    uint32_t q[kDeqUnroll], c[kDeqUnroll];
    Y *dst[kDeqUnroll];
#pragma unroll
    for (int u = 0; u < kDeqUnroll; ++u) {
      const uint32_t i = i0 + u * stride;
      dst[u] = nullptr;
      q[u] = c[u] = 0;
      if (i < total) {
        int64_t r;
        int piece;
        pieces.at(i, r, piece);
        const uint8_t *src = codes + r * (K / 2) + piece * (N / 2);
        q[u] = N == 8 ? __ldcs(reinterpret_cast<const uint32_t *>(src))
                      : __ldcs(reinterpret_cast<const uint16_t *>(src));
        c[u] = __ldg(sf + r * sf_ld + piece / (fp4::Fmt<FMT>::kBlock / N));
        dst[u] = out + r * K + piece * N;
      }
    }
#pragma unroll
    for (int u = 0; u < kDeqUnroll; ++u) {
      if (dst[u] == nullptr) continue;
      const float s = FMT == 1       ? e4m3_value(c[u]) * pow2f(scale_exp)
                      : c[u] == 255 ? __int_as_float(0x7FFFFFFF)
                                     : pow2f((int)c[u] - 127);
      uint32_t o[4];
#pragma unroll
      for (int b = 0; b < N / 2; ++b) {
        const float2 f = e2m1x2_value(q[u] >> (8 * b) & 0xFFu);
        if constexpr (N == 8) {
          __nv_bfloat162 p = __floats2bfloat162_rn(f.x * s, f.y * s);
          o[b] = *reinterpret_cast<uint32_t *>(&p);
        } else {
          o[2 * b] = __float_as_uint(f.x * s);
          o[2 * b + 1] = __float_as_uint(f.y * s);
        }
      }
      __stcs(reinterpret_cast<uint4 *>(dst[u]), make_uint4(o[0], o[1], o[2], o[3]));
    }
  }
}

// Weight rows into the grouped product's tiles, [e][nb][kb] of tile_bytes
// each: two halves of 128 rows x 128 bytes of codes, 16-byte chunk c of row r
// at chunk c ^ (r & 7) (the 128-byte swizzle of the tensor core's operand),
// then each half's scales as 512-byte groups of 4 scale bytes a row, row r's
// at 16 (r % 32) + 4 (r / 32).  Rows past N and elements past K are zero.
// One thread per 16 bytes of codes, then one per scale group row.
__global__ void __launch_bounds__(kThreads)
    pack_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ sf, int64_t n_tiles,
                int N, int K, int sf_ld, int scale_bytes, int nbn, int nkb, int swiglu,
                uint8_t *__restrict__ packed, int tbytes) {
  const int units = 2 * fp4::kHalfRows * 8;        // 16-byte code chunks of a tile
  const int groups = scale_bytes / 4;              // 512-byte scale groups of a half
  const int sunits = 2 * fp4::kHalfRows * groups;  // 4-byte scale words of a tile
  const int64_t total = n_tiles * (units + sunits);
  const int64_t stride = (int64_t)gridDim.x * kThreads;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += stride) {
    const int64_t tile = i / (units + sunits);
    int u = (int)(i - tile * (units + sunits));
    const int kb = (int)(tile % nkb);
    const int nb = (int)(tile / nkb % nbn);
    const int64_t e = tile / nkb / nbn;
    uint8_t *dst = packed + tile * tbytes;
    const bool is_sf = u >= units;
    if (is_sf) u -= units;
    const int per = is_sf ? groups : 8;
    const int c = u % per, r = u / per % fp4::kHalfRows, half = u / per / fp4::kHalfRows;
    const int in_half = (swiglu ? nb * 128 : nb * 256 + half * 128) + r;
    const bool row_ok = swiglu ? in_half < N / 2 : in_half < N;
    const int64_t row = e * N + (swiglu ? (int64_t)half * (N / 2) : 0) + in_half;
    if (!is_sf) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (row_ok && kb * 128 + c * 16 < K / 2)
        v = __ldg(reinterpret_cast<const uint4 *>(codes + row * (K / 2) + kb * 128 + c * 16));
      *reinterpret_cast<uint4 *>(dst + half * fp4::kHalfRows * 128 + r * 128 +
                                 ((c ^ (r & 7)) * 16)) = v;
    } else {
      uint32_t v = 0;
      if (row_ok) {
        v = __ldg(reinterpret_cast<const uint32_t *>(sf + row * sf_ld + kb * scale_bytes + c * 4));
        // scales past K belong to no element
        const int valid = K * scale_bytes / fp4::kStepElems - (kb * scale_bytes + c * 4);
        if (valid < 4) v = valid <= 0 ? 0 : v & ((1u << (8 * valid)) - 1u);
      }
      *reinterpret_cast<uint32_t *>(dst + fp4::kTileCodes + (half * groups + c) * 512 +
                                    (r % 32) * 16 + (r / 32) * 4) = v;
    }
  }
}

// ------------------------------------------------------------------ host
bool fmt_ok(int32_t fmt) { return fmt == MOE_FP4_MX || fmt == MOE_FP4_NV; }

moe_status check_shape(int64_t rows, int32_t K, int32_t fmt, int32_t scale_exp) {
  if (rows < 0 || K < 1 || !fmt_ok(fmt)) return MOE_ERR_INVALID_ARG;
  if (fmt == MOE_FP4_MX && scale_exp != 0) return MOE_ERR_INVALID_ARG;
  if (K % 32 != 0 || K > (1 << 24) || scale_exp < -100 || scale_exp > 100)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Blocks for the pieces of a chunk, unroll of them a thread and turn.
dim3 pieces_grid(const Pieces &p, int unroll) {
  const int64_t per = (int64_t)kThreads * unroll;
  int64_t blocks = (p.chunk * p.per_row + per - 1) / per;
  const int64_t lim = (int64_t)moe_host::sm_count() * 16;
  return dim3((unsigned)(blocks > lim ? lim : blocks), p.chunks());
}

template <typename X, int FMT>
moe_status launch_quantize(const void *x, int64_t ldx, int64_t T, int32_t K, int32_t k,
                           const int32_t *dest_row, int64_t n_rows, int32_t scale_exp,
                           uint8_t *codes, uint8_t *sf, int32_t *status, cudaStream_t st) {
  const Pieces p = Pieces::of(T, K / kVec);
  return moe_host::launch_pdl(quantize_kernel<X, FMT>, pieces_grid(p, 1), dim3(kThreads), 0, st,
                              static_cast<const X *>(x), ldx, p, (int)K, (int)k, dest_row, n_rows, (int)scale_exp, codes, sf,
                              (int)moe_fp4_scale_ld(K, FMT), status);
}

template <typename Y, int FMT>
moe_status launch_dequant(const uint8_t *codes, const uint8_t *sf, int64_t n_rows, int32_t K,
                          int32_t scale_exp, void *out, cudaStream_t st) {
  const Pieces p = Pieces::of(n_rows, K / (16 / (int)sizeof(Y)));
  return moe_host::launch_pdl(dequant_kernel<Y, FMT>, pieces_grid(p, kDeqUnroll), dim3(kThreads), 0,
                              st, codes, sf, (int)moe_fp4_scale_ld(K, FMT), p, (int)K,
                              (int)scale_exp, static_cast<Y *>(out));
}

}  // namespace

extern "C" int64_t moe_fp4_scale_ld(int32_t K, int32_t fmt) {
  if (K < 1 || K % 32 != 0 || !fmt_ok(fmt)) return 0;
  return ((int64_t)K + fp4::kStepElems - 1) / fp4::kStepElems * (fmt == MOE_FP4_NV ? 16 : 8);
}

extern "C" size_t moe_fp4_packed_bytes(int32_t E, int32_t N, int32_t K, int32_t fmt,
                                       int32_t epilogue) {
  if (E < 1 || N < 1 || K < 1 || K % 32 != 0 || !fmt_ok(fmt)) return 0;
  if (epilogue != MOE_EPI_NONE && epilogue != MOE_EPI_SWIGLU) return 0;
  const size_t nkb = ((size_t)K + fp4::kStepElems - 1) / fp4::kStepElems;
  const size_t nbn =
      epilogue == MOE_EPI_SWIGLU ? ((size_t)N / 2 + 127) / 128 : ((size_t)N + 255) / 256;
  return (size_t)E * nbn * nkb * fp4::tile_bytes(fmt);
}

extern "C" moe_status moe_quantize_fp4(const void *x, int32_t x_type, int64_t ldx, int64_t n_rows,
                                       int32_t K, int32_t fmt, int32_t scale_exp, uint8_t *codes,
                                       uint8_t *sf, void *stream) {
  if (moe_status s = check_shape(n_rows, K, fmt, scale_exp)) return s;
  if ((x_type != MOE_F32 && x_type != MOE_BF16) || ldx < K) return MOE_ERR_INVALID_ARG;
  if (n_rows == 0) return MOE_OK;
  if (!x || !codes || !sf) return MOE_ERR_INVALID_ARG;
  if (!moe_host::aligned16(x) || !moe_host::aligned16(codes) || !moe_host::aligned16(sf) ||
      ldx * (x_type == MOE_F32 ? 4 : 2) % 16 != 0)
    return MOE_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto run = fmt == MOE_FP4_MX
                 ? (x_type == MOE_F32 ? launch_quantize<float, 0> : launch_quantize<__nv_bfloat16, 0>)
                 : (x_type == MOE_F32 ? launch_quantize<float, 1> : launch_quantize<__nv_bfloat16, 1>);
  return run(x, ldx, n_rows, K, 0, nullptr, n_rows, scale_exp, codes, sf, nullptr, st);
}

extern "C" moe_status moe_permute_fp4(const uint16_t *x, int64_t T, int32_t K, int32_t k,
                                      const int32_t *dest_row, int64_t n_rows, int32_t fmt,
                                      int32_t scale_exp, uint8_t *codes, uint8_t *sf, void *ws,
                                      size_t ws_bytes, void *stream) {
  if (moe_status s = check_shape(T, K, fmt, scale_exp)) return s;
  if (k < 1 || n_rows < 0) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !dest_row || ((!codes || !sf) && n_rows > 0)) return MOE_ERR_INVALID_ARG;
  if (!moe_host::aligned16(x) || !moe_host::aligned16(codes) || !moe_host::aligned16(sf))
    return MOE_ERR_INVALID_ARG;
  if (moe_status s = moe_host::check_ws(ws, ws_bytes, moe::kStatusBytes)) return s;
  auto run = fmt == MOE_FP4_MX ? launch_quantize<__nv_bfloat16, 0> : launch_quantize<__nv_bfloat16, 1>;
  return run(x, K, T, K, k, dest_row, n_rows, scale_exp, codes, sf, moe_host::status_ptr(ws),
             static_cast<cudaStream_t>(stream));
}

extern "C" moe_status moe_dequant_fp4(const uint8_t *codes, const uint8_t *sf, int64_t n_rows,
                                      int32_t K, int32_t fmt, int32_t scale_exp, void *out,
                                      int32_t out_type, void *stream) {
  if (moe_status s = check_shape(n_rows, K, fmt, scale_exp)) return s;
  if (out_type != MOE_F32 && out_type != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (n_rows == 0) return MOE_OK;
  if (!codes || !sf || !out) return MOE_ERR_INVALID_ARG;
  if (!moe_host::aligned16(codes) || !moe_host::aligned16(sf) || !moe_host::aligned16(out))
    return MOE_ERR_INVALID_ARG;
  auto run = fmt == MOE_FP4_MX
                 ? (out_type == MOE_F32 ? launch_dequant<float, 0> : launch_dequant<__nv_bfloat16, 0>)
                 : (out_type == MOE_F32 ? launch_dequant<float, 1> : launch_dequant<__nv_bfloat16, 1>);
  return run(codes, sf, n_rows, K, scale_exp, out, static_cast<cudaStream_t>(stream));
}

extern "C" moe_status moe_pack_weights_fp4(const uint8_t *codes, const uint8_t *sf, int32_t E,
                                           int32_t N, int32_t K, int32_t fmt, int32_t epilogue,
                                           uint8_t *packed, void *stream) {
  if (E < 1 || N < 1) return MOE_ERR_INVALID_ARG;
  if (moe_status s = check_shape(E, K, fmt, 0)) return s;
  if (epilogue != MOE_EPI_NONE && epilogue != MOE_EPI_SWIGLU) return MOE_ERR_INVALID_ARG;
  const int swiglu = epilogue == MOE_EPI_SWIGLU;
  if (N % (swiglu ? 16 : 8) != 0) return MOE_ERR_UNSUPPORTED;
  if (!codes || !sf || !packed || packed == codes || packed == sf) return MOE_ERR_INVALID_ARG;
  if (!moe_host::aligned16(codes) || !moe_host::aligned16(sf) || !moe_host::aligned16(packed))
    return MOE_ERR_INVALID_ARG;
  const int nkb = (K + fp4::kStepElems - 1) / fp4::kStepElems;
  const int nbn = swiglu ? (N / 2 + 127) / 128 : (N + 255) / 256;
  const int64_t n_tiles = (int64_t)E * nbn * nkb;
  pack_kernel<<<(unsigned)moe_host::sm_count() * 16, kThreads, 0,
                static_cast<cudaStream_t>(stream)>>>(
      codes, sf, n_tiles, N, K, (int)moe_fp4_scale_ld(K, fmt), fmt == MOE_FP4_NV ? 16 : 8, nbn, nkb,
      swiglu, packed, fp4::tile_bytes(fmt));
  return moe_host::launch_status();
}
