// Grouped product of bf16 rows with 4-bit expert weights, for few rows a
// segment: decode steps, whose time is the weights' stream.
//
// "Mixture-of-Experts Inference", "Memory pressure" (a decode step is dominated
// by loading the expert weights); "14. Serving Mixture-of-Experts Models",
// "Follow one token", step 3 (one kernel for every expert's segment).
//
// A weight is (q - z) s with a 4-bit code q, and s and z shared by a group of
// 32, 64 or 128 along K.  q - z is a small integer, exact in bf16, so a group's
// products are those of matrix instructions on bf16 (16 weight rows x 16 of K x
// 8 rows of x) with fp32 sums, and s multiplies the group's fp32 sum: no weight
// is rounded.
//
// Packed weights: blocks of 32 weight rows (two tiles of 16; with SwiGLU a tile
// is 8 gate rows and their 8 up rows, so that both meet in a CTA) by steps of
// 128 along K, in three planes [e][block][step]: codes (2048 bytes), scales
// (64 bytes for each group of the step) and zeros (32).  A lane's 16 bytes of
// codes are its operands of four matrix instructions.
#include <cuda_bf16.h>

#include "common.cuh"
#include "umma.cuh"

namespace {

constexpr int kBlockRows = 32;   // weight rows of a block
constexpr int kStepK = 128;      // K of a step
constexpr int kStepCodes = kBlockRows * kStepK / 2;
constexpr int kMaxSegs = 1024;
constexpr int kPackThreads = 256;

__host__ __device__ constexpr int scale_bytes(int ng) { return 64 * ng; }
__host__ __device__ constexpr int zero_bytes(int ng) { return 32 * ng; }

// The weight row of row r of a block, or -1 past the end.
__device__ __forceinline__ int weight_row(int nb, int r, int N, int swiglu) {
  if (!swiglu) {
    const int n = nb * kBlockRows + r;
    return n < N ? n : -1;
  }
  const int j = nb * 16 + (r >> 4) * 8 + (r & 7);
  return j < N / 2 ? j + (r & 8 ? N / 2 : 0) : -1;
}

// Codes, scales and zeros to the three planes; a thread writes 16 bytes of
// codes, or one scale and zero.  Within a lane's 16 bytes (lane = 4 g + p) word
// 2 h + s holds K = 64 half + 32 h + 8 p + 4 s + {0, 1, 2, 3} of rows g and
// g + 8, nibbles in the order (g, 0) (g + 8, 0) (g, 2) (g + 8, 2) and the same
// of the odd elements: the four operands are nibble i of each 16-bit half.
__global__ void __launch_bounds__(kPackThreads)
    pack_int4_kernel(const uint8_t *__restrict__ codes, const uint16_t *__restrict__ scales,
                     const uint8_t *__restrict__ zeros, int64_t n_steps, int N, int K, int ng,
                     int nbn, int nst, int swiglu, uint8_t *__restrict__ out_codes,
                     uint8_t *__restrict__ out_scales, uint8_t *__restrict__ out_zeros) {
  const int units = kStepCodes / 16, sunits = kBlockRows * ng;
  const int64_t total = n_steps * (units + sunits);
  const int groups = K / (kStepK / ng);  // of a row
  for (int64_t i = (int64_t)blockIdx.x * kPackThreads + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * kPackThreads) {
    const int64_t step = i / (units + sunits);
    int u = (int)(i - step * (units + sunits));
    const int st = (int)(step % nst), nb = (int)(step / nst % nbn);
    const int64_t e = step / nst / nbn;
    if (u < units) {
      const int m = u >> 6, half = u >> 5 & 1, lane = u & 31, g = lane >> 2, p = lane & 3;
      uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
      for (int b = 0; b < 2; ++b) {  // rows g and g + 8
        const int row = weight_row(nb, m * 16 + g + 8 * b, N, swiglu);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int k = st * kStepK + half * 64 + h * 32 + p * 8;
          if (row < 0 || k >= K) continue;
          const uint32_t v = __ldg(reinterpret_cast<const uint32_t *>(
              codes + (e * N + row) * (int64_t)(K / 2) + k / 2));
#pragma unroll
          for (int j = 0; j < 8; ++j) {  // element k + j
            const uint32_t q = v >> (4 * j) & 15u;
            const int nibble = (j >> 1 & 1) * 2 + b + (j & 1) * 4;
            w[2 * h + (j >> 2)] |= q << (4 * nibble);
          }
        }
      }
      *reinterpret_cast<uint4 *>(out_codes + step * kStepCodes + u * 16) =
          make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      u -= units;
      // [g][tile][group][row g or g + 8]
      const int b = u & 1, gi = u / 2 % ng, m = u / 2 / ng & 1, g = u / 4 / ng;
      const int row = weight_row(nb, m * 16 + g + 8 * b, N, swiglu);
      const int grp = st * ng + gi;
      const bool ok = row >= 0 && grp < groups;
      const int64_t at = (e * N + row) * (int64_t)groups + grp;
      reinterpret_cast<uint16_t *>(out_scales + step * scale_bytes(ng))[u] = ok ? scales[at] : 0;
      if (zeros) (out_zeros + step * zero_bytes(ng))[u] = ok ? zeros[at] & 127u : 0;
    }
  }
}

struct Params {
  const __nv_bfloat16 *x;
  const int32_t *seg_offsets, *seg_expert;
  const uint8_t *codes, *scales, *zeros;  // the three planes
  void *out;
  int32_t *status;
  int64_t n_rows;
  int32_t S, E, K, nbn, nst;
  int32_t out_n;  // columns of out
  int32_t swiglu, out_f32;
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src) {
  if (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 128 + q of nibble I of both halves of a word, as bf16 (its unit is 1 there).
template <int I>
__device__ __forceinline__ uint32_t nibble(uint32_t w) {
  return ((w >> (4 * I)) & 0x000F000Fu) | 0x43004300u;
}
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&a),
                                   *reinterpret_cast<const __nv_bfloat162 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}

// One block of weights times up to 8 NT rows of a segment.
struct Task {
  int64_t row0;
  int e, nb, n;
};

template <int NT, int NG, bool ZEROS>
struct Cfg {
  static constexpr int kStages = 4;
  static constexpr int kStage = kStepCodes + scale_bytes(NG) + (ZEROS ? zero_bytes(NG) : 0);
  static constexpr int kRedLd = kBlockRows + 2;  // a row's 32 partial results, off the banks
  static constexpr int kRed = 8 * NT * kRedLd * 4;
  static size_t smem(int warps, int S) {
    return (size_t)warps * (kStages * kStage + 2 * kRed) + (size_t)(2 * S + 2) * 4;
  }
};

// Persistent CTAs take (segment, block, row tile) in turn; the warps of a CTA
// split K and their sums meet in shared memory, in a fixed order.  Each warp
// keeps its own weights flowing through a ring that only it reads and fills
// (cp.async, no barrier), on into its next task while a task ends.  Rows of x
// come from L1 and L2, one 32-element piece ahead.
template <int NT, int NG, bool ZEROS>
__global__ void __launch_bounds__(256, NT == 4 ? 1 : 2) int4_product_kernel(const Params p) {
  using C = Cfg<NT, NG, ZEROS>;
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int g = lane >> 2, pl = lane & 3;
  uint8_t *ring = smem + warp * (C::kStages * C::kStage);
  float *red = reinterpret_cast<float *>(smem + warps * (C::kStages * C::kStage));
  int32_t *off = reinterpret_cast<int32_t *>(red + warps * 2 * (C::kRed / 4));
  int32_t *pre = off + p.S + 1;  // row tiles before segment s
  const uint32_t ring_addr = umma::smem_u32(ring);
  moe::pdl_wait();
  moe::pdl_trigger();
  int decreasing = 0;  // offsets that go back name no segments at all
  for (int s = threadIdx.x; s < p.S; s += blockDim.x) {
    const int64_t a = p.seg_offsets[s], b = p.seg_offsets[s + 1];
    const int e = p.seg_expert[s];
    int tiles = 0;
    if (b < a) {
      moe::report_error(p.status, MOE_ERR_DEVICE_INDEX, s, moe::K_INT4_PRODUCT);
      decreasing = 1;
    }
    if (b > a) {
      if (a < 0 || b > p.n_rows || e < 0 || e >= p.E)
        moe::report_error(p.status, MOE_ERR_DEVICE_INDEX, s, moe::K_INT4_PRODUCT);
      else
        tiles = (int)((b - a + 8 * NT - 1) / (8 * NT));
    }
    off[s] = (int)a;
    if (s == p.S - 1) off[p.S] = (int)b;
    pre[s] = tiles;
  }
  if (__syncthreads_or(decreasing)) return;
  if (warp == 0) umma::warp_exclusive_scan(pre, p.S, lane);
  __syncthreads();
  const int64_t total = (int64_t)pre[p.S] * p.nbn;

  // Task t: a segment's tasks follow one another, a block's row tiles together.
  auto decode = [&](int64_t t) {
    const int unit = (int)(t / p.nbn);  // the segment holds row tile `unit`
    int lo = 0, hi = p.S;               // last s with pre[s] <= unit
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= unit) lo = mid; else hi = mid;
    }
    const int tiles = pre[lo + 1] - pre[lo];
    const int local = (int)(t - (int64_t)pre[lo] * p.nbn);
    const int nb = local / tiles, rt = local - nb * tiles;
    Task k;
    k.row0 = (int64_t)off[lo] + rt * (8 * NT);
    k.n = min(8 * NT, off[lo + 1] - (int)k.row0);
    k.e = __ldg(p.seg_expert + lo);
    k.nb = nb;
    return k;
  };
  const int sb0 = (int)((int64_t)p.nst * warp / warps);
  const int sb1 = (int)((int64_t)p.nst * (warp + 1) / warps);

  // the copies run kStages - 1 steps ahead of the products
  int64_t ct = blockIdx.x, cstep = 0;
  int csb = sb0, cslot = 0;
  auto next_copy = [&]() {
    if (ct < total) {
      const Task k = decode(ct);
      cstep = ((int64_t)k.e * p.nbn + k.nb) * p.nst;
    }
  };
  auto copy = [&]() {
    if (ct < total && sb0 < sb1) {
      const uint32_t dst = ring_addr + cslot * C::kStage;
      const int64_t step = cstep + csb;
      const uint8_t *src = p.codes + step * kStepCodes;
#pragma unroll
      for (int i = 0; i < kStepCodes / 512; ++i)
        copy_async<16>(dst + (i * 32 + lane) * 16, src + (i * 32 + lane) * 16);
      if (lane < scale_bytes(NG) / 16)
        copy_async<16>(dst + kStepCodes + lane * 16, p.scales + step * scale_bytes(NG) + lane * 16);
      if (ZEROS && lane >= 16 && lane < 16 + zero_bytes(NG) / 16)
        copy_async<16>(dst + kStepCodes + scale_bytes(NG) + (lane - 16) * 16,
                       p.zeros + step * zero_bytes(NG) + (lane - 16) * 16);
      if (++csb == sb1) {
        csb = sb0;
        ct += gridDim.x;
        next_copy();
      }
    }
    copy_commit();
    cslot = cslot + 1 == C::kStages ? 0 : cslot + 1;
  };
  next_copy();
#pragma unroll
  for (int i = 0; i < C::kStages - 1; ++i) copy();

  int slot = 0, par = 0;
  for (int64_t t = blockIdx.x; t < total; t += gridDim.x, par ^= 1) {
    const Task k = decode(t);
    float acc[2][NT][4] = {};
    const __nv_bfloat16 *xr[NT];
    bool have[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      have[nt] = nt * 8 + g < k.n;
      xr[nt] = p.x + (k.row0 + nt * 8 + g) * p.K + 8 * pl;
    }
    auto load_x = [&](int kk, uint4 (&v)[NT]) {  // kk: the piece's first element of K
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        v[nt] = make_uint4(0, 0, 0, 0);
        if (have[nt] && kk < p.K) v[nt] = __ldg(reinterpret_cast<const uint4 *>(xr[nt] + kk));
      }
    };
    uint4 xn[NT];
    load_x(sb0 < sb1 ? sb0 * kStepK : p.K, xn);
    for (int sb = sb0; sb < sb1; ++sb) {
      copy_wait<C::kStages - 2>();
      __syncwarp();
      copy();  // into the slot that the step before this one left
      const uint8_t *st = ring + slot * C::kStage;
      const uint32_t *sc = reinterpret_cast<const uint32_t *>(st + kStepCodes) + g * 2 * NG;
      const uint16_t *zs =
          reinterpret_cast<const uint16_t *>(st + kStepCodes + scale_bytes(NG)) + g * 2 * NG;
      float part[2][NT][4] = {};
      uint4 w[2];
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        uint4 xv[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) xv[nt] = xn[nt];
        if (h < 3 || sb + 1 < sb1) load_x(sb * kStepK + 32 * (h + 1), xn);
        constexpr int kPieces = 4 / NG;  // of a group
        const int gi = h / kPieces;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          if ((h & 1) == 0)
            w[m] = *reinterpret_cast<const uint4 *>(st + (m * 64 + (h >> 1) * 32 + lane) * 16);
          uint32_t z0 = 0x43084308u, z1 = 0x43084308u;  // 128 + 8
          if (ZEROS) {
            const uint32_t z = zs[m * NG + gi];
            z0 = 0x43004300u | (z & 0xFFu) * 0x00010001u;
            z1 = 0x43004300u | (z >> 8) * 0x00010001u;
          }
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const uint32_t word = (h & 1) ? (s ? w[m].w : w[m].z) : (s ? w[m].y : w[m].x);
            const uint32_t a[4] = {sub2(nibble<0>(word), z0), sub2(nibble<1>(word), z1),
                                   sub2(nibble<2>(word), z0), sub2(nibble<3>(word), z1)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              if (nt == 0 || k.n > nt * 8)
                mma_bf16(part[m][nt], a, s ? xv[nt].z : xv[nt].x, s ? xv[nt].w : xv[nt].y);
          }
          if (h % kPieces == kPieces - 1) {
            const uint32_t v = sc[m * NG + gi];
            const float s0 = __uint_as_float(v << 16), s1 = __uint_as_float(v & 0xFFFF0000u);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              acc[m][nt][0] = fmaf(s0, part[m][nt][0], acc[m][nt][0]);
              acc[m][nt][1] = fmaf(s0, part[m][nt][1], acc[m][nt][1]);
              acc[m][nt][2] = fmaf(s1, part[m][nt][2], acc[m][nt][2]);
              acc[m][nt][3] = fmaf(s1, part[m][nt][3], acc[m][nt][3]);
#pragma unroll
              for (int i = 0; i < 4; ++i) part[m][nt][i] = 0.0f;
            }
          }
        }
      }
      slot = slot + 1 == C::kStages ? 0 : slot + 1;
    }
    // the warps' sums, [row of x][weight row] each
    float *mine = red + (par * warps + warp) * (C::kRed / 4);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          mine[(nt * 8 + 2 * pl + (i & 1)) * C::kRedLd + m * 16 + g + (i >> 1) * 8] = acc[m][nt][i];
    __syncthreads();
    const float *all = red + par * warps * (C::kRed / 4);
    const int cols = p.swiglu ? 16 : 32, pairs = cols / 2;
    for (int i = threadIdx.x; i < k.n * pairs; i += blockDim.x) {
      const int r = i / pairs, c = i % pairs * 2, col = k.nb * cols + c;
      const int at = r * C::kRedLd + (p.swiglu ? (c >> 3) * 16 + (c & 7) : c);
      float2 a = make_float2(0.0f, 0.0f), b = a;
      for (int w = 0; w < warps; ++w) {
        const float2 v = *reinterpret_cast<const float2 *>(all + w * (C::kRed / 4) + at);
        a.x += v.x, a.y += v.y;
        if (p.swiglu) {
          const float2 u = *reinterpret_cast<const float2 *>(all + w * (C::kRed / 4) + at + 8);
          b.x += u.x, b.y += u.y;
        }
      }
      if (p.swiglu) {
        a.x = a.x / (1.0f + expf(-a.x)) * b.x;
        a.y = a.y / (1.0f + expf(-a.y)) * b.y;
      }
      if (col >= p.out_n) continue;
      const int64_t o = (k.row0 + r) * p.out_n + col;
      if (p.out_f32)
        *reinterpret_cast<float2 *>(static_cast<float *>(p.out) + o) = a;
      else
        *reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(p.out) + o) =
            __floats2bfloat162_rn(a.x, a.y);
    }
  }
}

// ------------------------------------------------------------------ host
int blocks_of(int32_t N, bool swiglu) { return swiglu ? (N / 2 + 15) / 16 : (N + 31) / 32; }
int steps_of(int32_t K) { return (K + kStepK - 1) / kStepK; }

moe_status check_weights(int32_t E, int32_t N, int32_t K, int32_t group, int32_t epilogue) {
  if (E < 1 || N < 1 || K < 1) return MOE_ERR_INVALID_ARG;
  if (group != 32 && group != 64 && group != 128) return MOE_ERR_INVALID_ARG;
  if (epilogue != MOE_EPI_NONE && epilogue != MOE_EPI_SWIGLU) return MOE_ERR_INVALID_ARG;
  if (K % group != 0 || K > (1 << 24) || N % (epilogue == MOE_EPI_SWIGLU ? 16 : 8) != 0)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Steps of all experts, and where the planes of scales and zeros begin.
struct Planes {
  int64_t steps;
  size_t scales, zeros, bytes;
};
Planes planes(int32_t E, int32_t N, int32_t K, int32_t group, int has_zeros, int32_t epilogue) {
  const int ng = kStepK / group;
  Planes p;
  p.steps = (int64_t)E * blocks_of(N, epilogue == MOE_EPI_SWIGLU) * steps_of(K);
  p.scales = (size_t)p.steps * kStepCodes;
  p.zeros = p.scales + (size_t)p.steps * scale_bytes(ng);
  p.bytes = p.zeros + (has_zeros ? (size_t)p.steps * zero_bytes(ng) : 0);
  return p;
}

template <int NT, int NG, bool ZEROS>
moe_status launch(const Params &p, cudaStream_t st) {
  using C = Cfg<NT, NG, ZEROS>;
  constexpr int kMaxDevices = 64;
  static bool done[kMaxDevices] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
  const int warps = 8;
  if (dev < 0 || dev >= kMaxDevices || !done[dev]) {
    if (cudaFuncSetAttribute(int4_product_kernel<NT, NG, ZEROS>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)C::smem(8, kMaxSegs)) != cudaSuccess)
      return MOE_ERR_CUDA;
    if (dev >= 0 && dev < kMaxDevices) done[dev] = true;
  }
  const size_t smem = C::smem(warps, p.S);
  const int per_sm = NT < 4 && smem <= 113 * 1024 ? 2 : 1;
  int64_t grid = (int64_t)moe_host::sm_count() * per_sm;
  const int64_t tiles = (p.n_rows + 8 * NT - 1) / (8 * NT) + p.S;
  if (tiles * p.nbn < grid) grid = tiles * p.nbn;
  return moe_host::launch_pdl(int4_product_kernel<NT, NG, ZEROS>, dim3((unsigned)grid),
                              dim3(32 * warps), smem, st, p);
}

template <int NG, bool ZEROS>
moe_status launch_rows(const Params &p, cudaStream_t st) {
  if (p.n_rows <= 8) return launch<1, NG, ZEROS>(p, st);
  if (p.n_rows <= (int64_t)p.S * 16) return launch<2, NG, ZEROS>(p, st);
  return launch<4, NG, ZEROS>(p, st);
}

}  // namespace

extern "C" size_t moe_int4_packed_bytes(int32_t E, int32_t N, int32_t K, int32_t group,
                                        int32_t has_zeros, int32_t epilogue) {
  if (check_weights(E, N, K, group, epilogue) != MOE_OK) return 0;
  return planes(E, N, K, group, has_zeros, epilogue).bytes;
}

extern "C" moe_status moe_pack_weights_int4(const uint8_t *codes, const uint16_t *scales,
                                            const uint8_t *zeros, int32_t E, int32_t N, int32_t K,
                                            int32_t group, int32_t epilogue, uint8_t *packed,
                                            void *stream) {
  if (moe_status s = check_weights(E, N, K, group, epilogue)) return s;
  if (!codes || !scales || !packed || packed == codes) return MOE_ERR_INVALID_ARG;
  if (!moe_host::aligned16(codes) || !moe_host::aligned16(packed) ||
      (reinterpret_cast<uintptr_t>(scales) & 1u))
    return MOE_ERR_INVALID_ARG;
  const Planes pl = planes(E, N, K, group, zeros != nullptr, epilogue);
  const bool swi = epilogue == MOE_EPI_SWIGLU;
  pack_int4_kernel<<<(unsigned)moe_host::sm_count() * 16, kPackThreads, 0,
                     static_cast<cudaStream_t>(stream)>>>(
      codes, scales, zeros, pl.steps, N, K, kStepK / group, blocks_of(N, swi), steps_of(K), swi,
      packed, packed + pl.scales, packed + pl.zeros);
  return moe_host::launch_status();
}

extern "C" moe_status moe_grouped_product_int4(const uint16_t *x, int64_t n_rows,
                                               const int32_t *seg_offsets,
                                               const int32_t *seg_expert, int32_t S, int32_t E,
                                               const uint8_t *w_packed, int32_t N, int32_t K,
                                               int32_t group, int32_t has_zeros, int32_t epilogue,
                                               void *out, int32_t out_type, void *ws,
                                               size_t ws_bytes, void *stream) {
  if (n_rows < 0 || S < 1) return MOE_ERR_INVALID_ARG;
  if (out_type != MOE_F32 && out_type != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (has_zeros != 0 && has_zeros != 1) return MOE_ERR_INVALID_ARG;
  if (moe_status s = check_weights(E, N, K, group, epilogue)) return s;
  if (S > kMaxSegs || n_rows >= ((int64_t)1 << 31) - 64) return MOE_ERR_UNSUPPORTED;
  const bool swi = epilogue == MOE_EPI_SWIGLU;
  if (((n_rows + 7) / 8 + S) * blocks_of(N, swi) >= ((int64_t)1 << 31) - 65536)
    return MOE_ERR_UNSUPPORTED;
  if (!seg_offsets || !seg_expert || !w_packed) return MOE_ERR_INVALID_ARG;
  if (moe_status s = moe_host::check_ws(ws, ws_bytes, moe::kStatusBytes)) return s;
  if (n_rows == 0) return MOE_OK;
  if (!x || !out || !moe_host::aligned16(x) || !moe_host::aligned16(w_packed) ||
      !moe_host::aligned16(out))
    return MOE_ERR_INVALID_ARG;
  const Planes pl = planes(E, N, K, group, has_zeros, epilogue);
  Params p{};
  p.x = reinterpret_cast<const __nv_bfloat16 *>(x);
  p.seg_offsets = seg_offsets;
  p.seg_expert = seg_expert;
  p.codes = w_packed;
  p.scales = w_packed + pl.scales;
  p.zeros = w_packed + pl.zeros;
  p.out = out;
  p.status = moe_host::status_ptr(ws);
  p.n_rows = n_rows;
  p.S = S;
  p.E = E;
  p.K = K;
  p.nbn = blocks_of(N, swi);
  p.nst = steps_of(K);
  p.out_n = swi ? N / 2 : N;
  p.swiglu = swi;
  p.out_f32 = out_type == MOE_F32;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (group == 128) return has_zeros ? launch_rows<1, true>(p, st) : launch_rows<1, false>(p, st);
  if (group == 64) return has_zeros ? launch_rows<2, true>(p, st) : launch_rows<2, false>(p, st);
  return has_zeros ? launch_rows<4, true>(p, st) : launch_rows<4, false>(p, st);
}
