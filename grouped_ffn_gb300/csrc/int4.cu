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
// 128 along K, [e][block][step]: 2048 bytes of codes, then for each group of the
// step 64 bytes of scales and, if there are any, 32 of zeros.  A lane's 16 bytes
// of codes are its operands of four matrix instructions.
#include <cuda_bf16.h>

#include "common.cuh"
#include "umma.cuh"

namespace {

constexpr int kBlockRows = 32;   // weight rows of a block
constexpr int kStepK = 128;      // K of a step
constexpr int kStepCodes = kBlockRows * kStepK / 2;
constexpr int kMaxSegs = 1024;
constexpr int kWarps = 8;       // of a CTA
constexpr int kCtasPerSm = 2;   // up to 128 registers a thread; three with 80 measured the same
constexpr int kPackThreads = 256;

__host__ __device__ constexpr int scale_bytes(int ng) { return 64 * ng; }
__host__ __device__ constexpr int zero_bytes(int ng) { return 32 * ng; }
__host__ __device__ constexpr int step_bytes(int ng, bool zeros) {
  return kStepCodes + scale_bytes(ng) + (zeros ? zero_bytes(ng) : 0);
}

// The weight row of row r of a block, or -1 past the end.
__device__ __forceinline__ int weight_row(int nb, int r, int N, int swiglu) {
  if (!swiglu) {
    const int n = nb * kBlockRows + r;
    return n < N ? n : -1;
  }
  const int j = nb * 16 + (r >> 4) * 8 + (r & 7);
  return j < N / 2 ? j + (r & 8 ? N / 2 : 0) : -1;
}

// Codes, scales and zeros to the packed steps.  A CTA takes a block of weight rows
// and walks along K, two steps at a time; a thread writes 16 bytes of codes, then
// its share of the scales and zeros.  Within a lane's 16 bytes (lane = 4 g + p)
// word 2 h + s holds K = 64 half + 32 h + 8 p + 4 s + {0, 1, 2, 3} of rows g and
// g + 8, nibbles in the order (g, 0) (g + 8, 0) (g, 2) (g + 8, 2) and the same of
// the odd elements: the four operands are nibble i of each 16-bit half.
__global__ void __launch_bounds__(kPackThreads)
    pack_int4_kernel(const uint8_t *__restrict__ codes, const uint16_t *__restrict__ scales,
                     const uint8_t *__restrict__ zeros, int N, int K, int ng, int nbn, int nst,
                     int swiglu, uint8_t *__restrict__ packed) {
  constexpr int kUnits = kStepCodes / 16, kSteps = kPackThreads / kUnits;
  const int bytes = step_bytes(ng, zeros != nullptr);
  const int groups = K / (kStepK / ng);  // of a row
  const int64_t e = blockIdx.x / nbn;
  const int nb = (int)(blockIdx.x - e * nbn);
  uint8_t *out = packed + (int64_t)blockIdx.x * nst * bytes;
  const int u = threadIdx.x % kUnits, s0 = threadIdx.x / kUnits;
  const int m = u >> 6, half = u >> 5 & 1, lane = u & 31, g = lane >> 2, p = lane & 3;
  const uint8_t *src[2];
  bool row_ok[2];
#pragma unroll
  for (int b = 0; b < 2; ++b) {  // rows g and g + 8
    const int row = weight_row(nb, m * 16 + g + 8 * b, N, swiglu);
    row_ok[b] = row >= 0;
    src[b] = codes + (e * N + max(row, 0)) * (int64_t)(K / 2);
  }
  for (int st = s0; st < nst; st += kSteps) {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = st * kStepK + half * 64 + h * 32 + p * 8;
        if (!row_ok[b] || k >= K) continue;
        const uint32_t v = __ldg(reinterpret_cast<const uint32_t *>(src[b] + k / 2));
#pragma unroll
        for (int j = 0; j < 8; ++j) {  // element k + j
          const uint32_t q = v >> (4 * j) & 15u;
          const int nibble = (j >> 1 & 1) * 2 + b + (j & 1) * 4;
          w[2 * h + (j >> 2)] |= q << (4 * nibble);
        }
      }
    *reinterpret_cast<uint4 *>(out + (int64_t)st * bytes + u * 16) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  const int sunits = kBlockRows * ng;
  for (int64_t i = threadIdx.x; i < (int64_t)nst * sunits; i += kPackThreads) {
    const int st = (int)(i / sunits), v = (int)(i - (int64_t)st * sunits);
    // [g][tile][group][row g or g + 8]
    const int b = v & 1, gi = v / 2 % ng, tile = v / 2 / ng & 1, gr = v / 4 / ng;
    const int row = weight_row(nb, tile * 16 + gr + 8 * b, N, swiglu);
    const int grp = st * ng + gi;
    const bool ok = row >= 0 && grp < groups;
    const int64_t at = (e * N + row) * (int64_t)groups + grp;
    uint8_t *o = out + (int64_t)st * bytes + kStepCodes;
    reinterpret_cast<uint16_t *>(o)[v] = ok ? scales[at] : 0;
    if (zeros) o[scale_bytes(ng) + v] = ok ? zeros[at] & 127u : 0;
  }
}

struct Params {
  const __nv_bfloat16 *x;
  const int32_t *seg_offsets, *seg_expert;
  const uint8_t *w;  // packed steps
  void *out;
  int32_t *status;
  int64_t n_rows;
  int32_t S, E, K, nbn, nst;
  int32_t out_n;  // columns of out
  int32_t swiglu, out_f32;
};

// d = A B + d, or A B for the first of a group.
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1, bool first) {
  if (first) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
    return;
  }
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void copy_async(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 128 + q of nibble I of both halves of a word, as bf16 (its unit is 1 there).
// `one28` is 0x43004300 in a register that the compiler does not see through:
// one instruction for and and or, which takes one immediate only.
template <int I>
__device__ __forceinline__ uint32_t nibble(uint32_t w, uint32_t one28) {
  uint32_t r;
  asm("lop3.b32 %0, %1, 0x000F000F, %2, 0xEA;" : "=r"(r) : "r"(w >> (4 * I)), "r"(one28));
  return r;
}
// q - z as bf16 pairs, from 128 + q and -(128 + z): exact, one instruction.
__device__ __forceinline__ uint32_t add2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(0x3F803F80u), "r"(b));
  return r;
}

// One block of weights times up to 8 NT rows of a segment.
struct Task {
  int row0, e, nb, n;
};

template <int N>
struct Int {
  static constexpr int value = N;
};

template <int NT, int NG, bool ZEROS>
struct Cfg {
  static constexpr int kStages = 4;
  static constexpr int kStage = step_bytes(NG, ZEROS);
  static constexpr int kRedLd = kBlockRows + 2;  // a row's 32 partial results, off the banks
  static constexpr int kRed = 8 * NT * kRedLd * 4;
  static size_t smem(int S) {
    return (size_t)kWarps * (kStages * kStage + kRed) + (size_t)(2 * S + 3) * 4;
  }
};

// A lane's N words of shared memory, in as few loads as they allow.
template <int N>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t (&v)[N]) {
  if constexpr (N == 1) {
    v[0] = *reinterpret_cast<const uint32_t *>(p);
  } else if constexpr (N == 2) {
    const uint2 a = *reinterpret_cast<const uint2 *>(p);
    v[0] = a.x, v[1] = a.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint4 a = *reinterpret_cast<const uint4 *>(p + 4 * i);
      v[i] = a.x, v[i + 1] = a.y, v[i + 2] = a.z, v[i + 3] = a.w;
    }
  }
}

// One step of K (128) of a block: the products of NA tiles of 8 rows, scaled.
// The first product of a group starts from zero, the group's sum is added with
// its scale.  x holds the step's four pieces of 32 elements; each is replaced by
// that of the next step as soon as it is used, where the next step has one
// (32 h < next).  TAIL: only `left` < 128 elements of K remain in this step;
// pieces beyond them count as zeros.
template <int NA, int NG, bool ZEROS, bool TAIL>
__device__ __forceinline__ void step_products(const uint8_t *st, int g, int lane, uint32_t one28, int left,
                                              int next, const __nv_bfloat16 *const (&xp)[NA],
                                              uint4 (&x)[4][NA], float (&acc)[2][NA][4]) {
  constexpr int kPieces = 4 / NG;  // pieces of a group
  uint32_t sc[2 * NG], zs[NG];  // of [tile][group], two rows each
  load_words(st + kStepCodes + g * 8 * NG, sc);
  if (ZEROS) load_words(st + kStepCodes + scale_bytes(NG) + g * 4 * NG, zs);
  float part[2][NA][4];
  uint4 w[2];
  uint32_t z[2][2];
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    if (TAIL && 32 * h >= left) {
#pragma unroll
      for (int nt = 0; nt < NA; ++nt) x[h][nt] = make_uint4(0, 0, 0, 0);
    }
    const int gi = h / kPieces;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      if ((h & 1) == 0)
        w[m] = *reinterpret_cast<const uint4 *>(st + (m * 64 + (h >> 1) * 32 + lane) * 16);
      if (h % kPieces == 0) {
        z[m][0] = z[m][1] = 0xC308C308u;  // -(128 + 8)
        if (ZEROS) {
          const int at = m * NG + gi;  // two bytes each
          z[m][0] = __byte_perm(zs[at / 2], 0xC3u, at % 2 ? 0x4242 : 0x4040);
          z[m][1] = __byte_perm(zs[at / 2], 0xC3u, at % 2 ? 0x4343 : 0x4141);
        }
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint32_t word = (h & 1) ? (s ? w[m].w : w[m].z) : (s ? w[m].y : w[m].x);
        const uint32_t a[4] = {add2(nibble<0>(word, one28), z[m][0]), add2(nibble<1>(word, one28), z[m][1]),
                               add2(nibble<2>(word, one28), z[m][0]), add2(nibble<3>(word, one28), z[m][1])};
#pragma unroll
        for (int nt = 0; nt < NA; ++nt)
          mma_bf16(part[m][nt], a, s ? x[h][nt].z : x[h][nt].x, s ? x[h][nt].w : x[h][nt].y,
                   h % kPieces == 0 && s == 0);
      }
      if (h % kPieces == kPieces - 1) {
        const uint32_t v = sc[m * NG + gi];
        const float s0 = __uint_as_float(v << 16), s1 = __uint_as_float(v & 0xFFFF0000u);
#pragma unroll
        for (int nt = 0; nt < NA; ++nt) {
          acc[m][nt][0] = fmaf(s0, part[m][nt][0], acc[m][nt][0]);
          acc[m][nt][1] = fmaf(s0, part[m][nt][1], acc[m][nt][1]);
          acc[m][nt][2] = fmaf(s1, part[m][nt][2], acc[m][nt][2]);
          acc[m][nt][3] = fmaf(s1, part[m][nt][3], acc[m][nt][3]);
        }
      }
    }
    if (!TAIL && next >= kStepK) {
#pragma unroll
      for (int nt = 0; nt < NA; ++nt)
        x[h][nt] = __ldg(reinterpret_cast<const uint4 *>(xp[nt] + kStepK + 32 * h));
    }
  }
  if (!TAIL && next < kStepK) {
#pragma unroll
    for (int h = 0; h < 4; ++h)
#pragma unroll
      for (int nt = 0; nt < NA; ++nt)
        if (32 * h < next)
          x[h][nt] = __ldg(reinterpret_cast<const uint4 *>(xp[nt] + kStepK + 32 * h));
  }
}

// log2 of the warps that split a task's K: those for which the slowest warp has
// least to do, a task's end counting as a step; where warps have eight tasks and
// more of 16 steps at least, the larger of almost equal ones (within 5%), whose tasks
// spread better.
// With 1, 2, 4, 8 warps: 128 rows over 64 experts, 8192 -> 2 x 2048, 191, 189, 183,
// 202 us; 8 rows over 8 experts, 7168 -> 2 x 2048, 51, 30, 32, 34 us; 512 rows over
// 256 experts, 2048 -> 7168, 363, 403, 479, 654 us; 333 rows over 5 experts, 1440 ->
// 712, 20.6, 13.4, 9.4, 11.5 us.
__device__ __forceinline__ int team_log(int total, int steps, int warps) {
  int best = 0;
  float least = 0.0f;
#pragma unroll
  for (int l = 0; 1 << l <= kWarps; ++l) {
    const float turns = ceilf((float)total * (float)(1 << l) / (float)warps);
    const float cost = turns * ((float)((steps + (1 << l) - 1) >> l) + 1.0f);
    if (l == 0 || cost < least ||
        (turns >= 8.0f && steps >> l >= 16 && cost <= 1.05f * least))
      best = l;
    if (l == 0 || cost < least) least = cost;
  }
  return best;
}

// Persistent CTAs of eight warps.  Teams of ks warps take (segment, block, row
// tile) in turn; the warps of a team split K and their sums meet in shared
// memory, in a fixed order.  Each warp keeps its own weights flowing through a
// ring that only it reads and fills (cp.async, no barrier), on into its next
// task while a task ends.  Rows of x come from L1 and L2, a step ahead in registers.
// A lane whose row lies past the tile reads the tile's last row instead: a column of
// the product does not reach the others, and is not stored.
// Bound by the length of a warp's chain of instructions at 16 warps an SM, not by one
// unit: 289 instructions for 2 KB of codes (112 shifts and and-ors, 64 subtractions), and
// issue is at 63%, the ALU at 60%, HBM at 63%, tensor cores at 27%.  Of 6.2 cycles from a
// warp's instruction to its next 1.2 wait for a result of fixed latency, 1.1 for a busy
// unit, 1.1 for other warps to issue and 0.7 for loads.  128 rows over 64 experts, 8192
// -> 2 x 2048, 184 us, 5.1 TB/s; 512 rows over 256 experts, 2048 -> 7168, 361 us, 5.1
// TB/s; one token's eight rows over eight experts, 7168 -> 2 x 2048, 29.4 us, 4.1 TB/s
// (2048 of 2432 warps have one task's half each, 28 steps, and start and end are
// exposed).  Many rows expand the weights again for each 16 of a segment: 32768 rows over
// 256 experts, 7168 -> 2 x 2048, 6.8 ms, 282 TFLOP/s.
template <int NT, int NG, bool ZEROS>
__global__ void __launch_bounds__(32 * kWarps, kCtasPerSm)
    int4_product_kernel(const Params p) {
  using C = Cfg<NT, NG, ZEROS>;
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, pl = lane & 3;
  uint8_t *ring = smem + warp * (C::kStages * C::kStage);
  float *red = reinterpret_cast<float *>(smem + kWarps * (C::kStages * C::kStage));
  int32_t *off = reinterpret_cast<int32_t *>(red + kWarps * (C::kRed / 4));
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
  const int total = pre[p.S] * p.nbn;  // below 2^31 by the host's check

  // Task t: a segment's tasks follow one another, a block's row tiles together.
  // Tasks are asked for in ascending order; s is the last one's segment.  (Most
  // segments may be empty: the next one is found by halves.)
  auto decode = [&](int t, int &s) {
    if (pre[s + 1] * p.nbn <= t) {
      int hi = p.S;  // the last segment that begins at t or before
      for (++s; hi - s > 1;) {
        const int mid = (s + hi) >> 1;
        if (pre[mid] * p.nbn <= t) s = mid; else hi = mid;
      }
    }
    const int tiles = pre[s + 1] - pre[s], local = t - pre[s] * p.nbn;
    const int nb = tiles == 1 ? local : local / tiles, rt = local - nb * tiles;
    Task k;
    k.row0 = off[s] + rt * (8 * NT);
    k.n = min(8 * NT, off[s + 1] - k.row0);
    k.e = __ldg(p.seg_expert + s);
    k.nb = nb;
    return k;
  };
  // (what a task's end alone needs is read back from shared memory there: the
  // loop over steps has no registers to spare)
  volatile int32_t *log_ks_at = pre + p.S + 1;
  if (threadIdx.x == 0) *log_ks_at = team_log(total, p.nst, (int)gridDim.x * kWarps);
  __syncthreads();
  int sb0, sb1, first, stride;
  {
    const int log_ks = *log_ks_at, member = warp & ((1 << log_ks) - 1);
    sb0 = (int)((int64_t)p.nst * member >> log_ks);
    sb1 = (int)((int64_t)p.nst * (member + 1) >> log_ks);
    first = (int)((blockIdx.x * kWarps + warp) >> log_ks);
    stride = (int)(gridDim.x * kWarps >> log_ks);
  }

  // the copies run kStages - 1 steps ahead of the products
  int ct = first;
  int cseg = 0, seg = 0;
  int cleft = 0;  // steps of the task still to be copied
  uint32_t cdst = 0;
  const uint8_t *csrc = nullptr;
  auto next_copy = [&]() {
    if (ct < total && sb0 < sb1) {
      const Task k = decode(ct, cseg);
      csrc = p.w + (((int64_t)k.e * p.nbn + k.nb) * p.nst + sb0) * C::kStage + lane * 16;
      cleft = sb1 - sb0;
      ct += stride;
    }
  };
  auto copy = [&]() {
    if (cleft > 0) {
      const uint32_t dst = ring_addr + cdst + lane * 16;
#pragma unroll
      for (int i = 0; i < C::kStage / 512; ++i) copy_async(dst + i * 512, csrc + i * 512);
      constexpr int kWhole = C::kStage / 512 * 512;
      if (lane < (C::kStage - kWhole) / 16) copy_async(dst + kWhole, csrc + kWhole);
      csrc += C::kStage;
      if (--cleft == 0) next_copy();
    }
    copy_commit();
    cdst = cdst == (C::kStages - 1) * C::kStage ? 0 : cdst + C::kStage;
  };
  next_copy();
#pragma unroll
  for (int i = 0; i < C::kStages - 1; ++i) copy();

  auto team_sync = [&](int log_ks) {
    if (log_ks == 0)
      __syncwarp();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(1 + (warp >> log_ks)), "r"(32 << log_ks) : "memory");
  };
  uint32_t one28;
  asm volatile("mov.b32 %0, 0x43004300;" : "=r"(one28));
  for (int t = first; t < total; t += stride) {
    const Task k = decode(t, seg);
    float *mine = red + warp * (C::kRed / 4);
    auto products = [&](auto na) {
      constexpr int NA = decltype(na)::value;
      float acc[2][NA][4] = {};
      const __nv_bfloat16 *xp[NA];
      uint4 x[4][NA];
#pragma unroll
      for (int nt = 0; nt < NA; ++nt) {
        const int r = min(nt * 8 + g, k.n - 1);
        xp[nt] = p.x + ((int64_t)k.row0 + r) * p.K + (sb0 * kStepK + 8 * pl);
#pragma unroll
        for (int h = 0; h < 4; ++h)
          if (sb0 < sb1 && sb0 * kStepK + 32 * h < p.K)
            x[h][nt] = __ldg(reinterpret_cast<const uint4 *>(xp[nt] + 32 * h));
      }
      auto begin = [&]() {
        copy_wait<C::kStages - 2>();
        __syncwarp();
        copy();  // into the slot that the step before this one left
        return ring + cdst;  // the slot after it is the oldest
      };
      const int full = min(sb1, p.K / kStepK);
      for (int sb = sb0; sb < full; ++sb) {
        const int next = sb + 1 < sb1 ? p.K - (sb + 1) * kStepK : 0;
        step_products<NA, NG, ZEROS, false>(begin(), g, lane, one28, 0, next, xp, x, acc);
#pragma unroll
        for (int nt = 0; nt < NA; ++nt) xp[nt] += kStepK;
      }
      if (full < sb1)
        step_products<NA, NG, ZEROS, true>(begin(), g, lane, one28, p.K - full * kStepK, 0, xp, x,
                                           acc);
      // the warps' sums, [row of x][weight row] each
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int nt = 0; nt < NA; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mine[(nt * 8 + 2 * pl + (i & 1)) * C::kRedLd + m * 16 + g + (i >> 1) * 8] =
                acc[m][nt][i];
    };
    if (NT > 1 && k.n > 8)
      products(Int<NT>());
    else
      products(Int<1>());
    const int log_ks = *log_ks_at, ks = 1 << log_ks, leader = warp >> log_ks << log_ks;
    team_sync(log_ks);
    const float *all = red + leader * (C::kRed / 4);
    const int cols = p.swiglu ? 16 : 32, log_pairs = p.swiglu ? 3 : 4;
    for (int i = threadIdx.x - leader * 32; i < k.n << log_pairs; i += 32 * ks) {
      const int r = i >> log_pairs, c = 2 * (i - (r << log_pairs)), col = k.nb * cols + c;
      const int at = r * C::kRedLd + (p.swiglu ? (c >> 3) * 16 + (c & 7) : c);
      float2 a = make_float2(0.0f, 0.0f), b = a;
      for (int w = 0; w < ks; ++w) {
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
      const int64_t o = (int64_t)(k.row0 + r) * p.out_n + col;
      if (p.out_f32)
        *reinterpret_cast<float2 *>(static_cast<float *>(p.out) + o) = a;
      else
        *reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(p.out) + o) =
            __floats2bfloat162_rn(a.x, a.y);
    }
    team_sync(log_ks);
  }
}

// ------------------------------------------------------------------ host
int blocks_of(int32_t N, bool swiglu) { return swiglu ? (N / 2 + 15) / 16 : (N + 31) / 32; }
int steps_of(int32_t K) { return (K + kStepK - 1) / kStepK; }

moe_status check_weights(int32_t E, int32_t N, int32_t K, int32_t group, int32_t epilogue) {
  if (E < 1 || N < 1 || K < 1) return MOE_ERR_INVALID_ARG;
  if (group != 32 && group != 64 && group != 128) return MOE_ERR_INVALID_ARG;
  if (epilogue != MOE_EPI_NONE && epilogue != MOE_EPI_SWIGLU) return MOE_ERR_INVALID_ARG;
  const bool swi = epilogue == MOE_EPI_SWIGLU;
  if (K % group != 0 || K > (1 << 24) || N % (swi ? 16 : 8) != 0 ||
      (int64_t)E * blocks_of(N, swi) >= (int64_t)1 << 31)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int64_t all_steps(int32_t E, int32_t N, int32_t K, int32_t epilogue) {
  return (int64_t)E * blocks_of(N, epilogue == MOE_EPI_SWIGLU) * steps_of(K);
}

template <int NT, int NG, bool ZEROS>
moe_status launch(const Params &p, cudaStream_t st) {
  using C = Cfg<NT, NG, ZEROS>;
  constexpr int kMaxDevices = 64;
  static bool done[kMaxDevices] = {false};
  int dev = 0;
  if (moe_host::refused(cudaGetDevice(&dev))) return MOE_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices || !done[dev]) {
    if (moe_host::refused(cudaFuncSetAttribute(int4_product_kernel<NT, NG, ZEROS>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)C::smem(kMaxSegs))))
      return MOE_ERR_CUDA;
    if (dev >= 0 && dev < kMaxDevices) done[dev] = true;
  }
  int64_t grid = (int64_t)moe_host::sm_count() * kCtasPerSm;
  const int64_t tasks = ((p.n_rows + 8 * NT - 1) / (8 * NT) + p.S) * p.nbn;
  if (tasks < grid) grid = tasks;
  return moe_host::launch_pdl(int4_product_kernel<NT, NG, ZEROS>, dim3((unsigned)grid),
                              dim3(32 * kWarps), C::smem(p.S), st, p);
}

// Tiles of 8 rows where no segment can have more, else of 16 (with the second
// half left out where a tile has no more than 8): one row, 7168 -> 4096, 8.8 us
// against 10.0; 512 rows in Zipf segments of 64 experts, 4096 -> 2048, 90 against
// 84 us; tiles of 32 rows need a whole SM's registers for one CTA: 103 us.
template <int NG, bool ZEROS>
moe_status launch_rows(const Params &p, cudaStream_t st) {
  return p.n_rows <= 8 ? launch<1, NG, ZEROS>(p, st) : launch<2, NG, ZEROS>(p, st);
}

}  // namespace

extern "C" size_t moe_int4_packed_bytes(int32_t E, int32_t N, int32_t K, int32_t group,
                                        int32_t has_zeros, int32_t epilogue) {
  if (check_weights(E, N, K, group, epilogue) != MOE_OK) return 0;
  return (size_t)all_steps(E, N, K, epilogue) * step_bytes(kStepK / group, has_zeros != 0);
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
  const bool swi = epilogue == MOE_EPI_SWIGLU;
  pack_int4_kernel<<<(unsigned)((int64_t)E * blocks_of(N, swi)), kPackThreads, 0,
                     static_cast<cudaStream_t>(stream)>>>(
      codes, scales, zeros, N, K, kStepK / group, blocks_of(N, swi), steps_of(K), swi, packed);
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
  Params p{};
  p.x = reinterpret_cast<const __nv_bfloat16 *>(x);
  p.seg_offsets = seg_offsets;
  p.seg_expert = seg_expert;
  p.w = w_packed;
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
