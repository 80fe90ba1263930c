// Grouped product of FP4 rows with the experts' FP4 weights on block-scaled
// tcgen05 (formats and the weight tiles: fp4.cuh).
//
//   out[r, n] = alpha_e sum_K x[r, K] w_e[n, K]     rows r of segment s, e = seg_expert[s]
//   with SwiGLU: out = silu(alpha_e g) * (alpha_e u), g and u the two halves of N.
//
// The weights are the tensor core's M side (tiles of 2 x 128 weight rows, in
// shared memory exactly as they lie in memory, so one bulk copy a step), the
// rows its N side: N is the number of rows in the tile, rounded up to 16, so
// a segment of a few rows moves few bytes and wastes little of the tensor
// core.  A segment of n rows is cut into ceil(n / ROWS) tiles of equal size.
//
// Per CTA (one per SM), a ring of stages of 256 elements of K:
//   warp 0     weights (one bulk copy) and rows (TMA boxes of 16 rows)
//   warp 1     copies the stage's scales into TMEM (tcgen05.cp) and issues 8
//              block-scaled MMAs of K = 64 (4 steps x 2 weight halves)
//   warps 2-5  epilogue: TMEM lane = weight row, column = row of x (ROWS = 224:
//              warps 8-11 too)
//   warp 6     takes tiles from a counter (workspace) and hands them to the others
//   warp 7     the rows' scales into the layout that tcgen05.cp reads, loaded
//              as many stages ahead as there are, in registers
// TMEM: two accumulator slots of 2 x 112 columns, up to 64 columns of scales.
//
// ROWS = 112 (4 stages): a slot a tile, the epilogue of one under the products
// of the next.  Bound by the weight stream: 64 experts of one row each, 4096 x
// 4096, 85 us, 7.1 TB/s of weights; 128 rows over 64 experts, 8192 -> 2 x 2048,
// 130 us, 6.9 TB/s.
// ROWS = 224 (3 stages), where segments average more than 64 rows: a tile takes
// both slots, so that a stage of weights meets twice the rows, and the epilogue
// is not hidden.  Bound by what an SM takes in from L2 (68 KB a stage at about 96
// bytes a ns) and by the epilogue (2 to 3 us of 14 us a tile at K = 4096): 7448
// rows over 4 experts, 4096 x 4096, 57 us, 4.4 PFLOP/s, the tensor pipe busy 45%
// of the time (this kernel's 128 x 224 x 64 MMAs run at 9.6 PFLOP/s alone).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <mutex>

#include "common.cuh"
#include "fp4.cuh"
#include "tile_order.cuh"
#include "umma.cuh"

namespace {

using namespace umma;

constexpr int kSlotRows = 112;  // rows of x that one accumulator slot holds
constexpr int kBoxRows = 16;
constexpr int kMaxSegs = 1024;
constexpr uint32_t kTmemCols = 512;
constexpr int kSlotCols = 2 * kSlotRows;
constexpr int kScaleCol = 2 * kSlotCols;  // 32 columns of weight scales, up to 32 of row scales
constexpr int kOutWarpBytes = 16 * 64;    // an epilogue warp's 16 rows of 32 bf16

// Shared memory of tiles of up to ROWS rows (112 or 224).
template <int ROWS>
struct Cfg {
  static constexpr int kStages = ROWS == 112 ? 4 : 3;
  static constexpr int kBlocks = (ROWS + 127) / 128;  // 128-row blocks of row scales
  static constexpr int kEpiWarps = ROWS == 112 ? 4 : 8;
  static constexpr int kThreads = 128 + 32 * kEpiWarps;
  static constexpr int kXOff = fp4::kTileCodes + 4096;  // rows' codes within a stage
  static constexpr int kXsOff = kXOff + ROWS * 128;     // rows' scales, 4 groups a block
  static constexpr int kStageBytes = kXsOff + kBlocks * 4 * 512;
  struct __align__(8) Bars {
    uint64_t full[kStages];
    uint64_t empty[kStages];
    uint64_t tfull[2];
    uint64_t tempty[2];
    uint64_t sfull[4];
    uint64_t sempty[4];
    uint64_t drain;
  };
  static constexpr size_t kBarsOff = (size_t)kStages * kStageBytes;
  static constexpr size_t kMiscOff = kBarsOff + sizeof(Bars);
  static constexpr size_t kSlotsOff = (kMiscOff + 16 + 15) / 16 * 16;  // four tiles
  static constexpr size_t kEpiOff = kSlotsOff + 64;                     // the epilogue's tile, twice
  static constexpr size_t kSegOff = kEpiOff + 32;
  static constexpr size_t kOutOff = (kSegOff + (size_t)(3 * kMaxSegs + 3) * 4 + 15) / 16 * 16;
  static constexpr size_t kSmemBytes = kOutOff + kEpiWarps * kOutWarpBytes + 1024;
  static_assert(kStageBytes % 1024 == 0 && kXOff % 1024 == 0, "swizzle atoms are 1024 bytes");
  static_assert(kSmemBytes <= 232448, "shared memory of one SM");
};

struct Params {
  const int32_t *seg_offsets, *seg_expert;
  const uint8_t *w;    // packed tiles
  const uint8_t *sf;   // rows' scales
  const float *alpha;  // per expert, or NULL
  void *out;
  int32_t *status;
  int32_t *counter;  // tiles taken beyond the first of each CTA; finished CTAs
  int64_t n_rows;
  int32_t S, E, nkb, nbn, sf_ld;
  int32_t out_n;  // columns of out
};

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar,
                                          uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1], %2, [%3], %4;" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

__device__ __forceinline__ void fence_proxy_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// One lane of a whole warp.  TMA, tcgen05.cp and tcgen05.mma take their operands
// from uniform registers: behind elect.sync the compiler knows that one thread
// runs and issues them at once, behind a comparison of the lane it loops over
// the active threads for each (8 MMAs and 12 copies: 1501 cycles against 584).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(p));
  return p != 0;
}

// 512 bytes of scales (32 rows of 16 bytes) to 4 TMEM columns, repeated in
// the four lane quadrants: no swizzle, 8-row groups 128 bytes apart.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t saddr) {
  const uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(128 >> 4) << 32 |
                     (uint64_t)1 << 46;
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}

template <int FMT>
__device__ __forceinline__ void mma_fp4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                        uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        uint32_t accumulate) {
  if (FMT == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X"
        " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::2X"
        " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// 16 TMEM lanes x 16 columns as four 8 x 8 pieces: lane L of the warp gets
// lane L / 4 (r[0..1], r[4..5]) and L / 4 + 8 (r[2..3], r[6..7]), columns
// 2 (L % 4) and the next (r[4..7]: 8 further on).
__device__ __forceinline__ void tmem_ld_16x16(uint32_t taddr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr));
}

// Four 8 x 8 bf16 pieces, transposed on the way: row i of a piece (its lane
// 8 piece + i names the address) takes column i of the fragment.
__device__ __forceinline__ void stmatrix_t(uint32_t saddr, uint32_t a, uint32_t b, uint32_t c,
                                           uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared::cta.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                   saddr),
               "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// silu(g) u for fp32 results.
__device__ __forceinline__ float swiglu_accurate(float g, float u) {
  return g / (1.0f + expf(-g)) * u;
}

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// silu(alpha g) (alpha u) for two pairs g, u, as bf16 (two fp32 operations an
// instruction), by the approximate exponential and reciprocal: the errors, 2^-17
// and less, are far below the rounding of the result.  1 / (1 + e^-g) is 0 from
// e^-g = 2^126 on, as the result then is to fp32's range.  silu(g) is formed
// before the product with u, for g u alone may overflow.  (One reciprocal for two
// values, 1 / a = b / (a b), needs both e^-g below 2^62: with a branch for the
// others it measured 543 us where this takes 537, 65536 rows over 32 experts,
// 4096 -> 2 x 2048.)
__device__ __forceinline__ uint32_t swiglu_fast2(uint32_t g0, uint32_t g1, uint32_t u0, uint32_t u1,
                                                 uint64_t alpha2) {
  constexpr float kLog2e = 1.4426950409f;
  const uint64_t g = mul2(pack2(__uint_as_float(g0), __uint_as_float(g1)), alpha2);
  const uint64_t u = mul2(pack2(__uint_as_float(u0), __uint_as_float(u1)), alpha2);
  float x0, x1, d0, d1, r0, r1, y0, y1;
  unpack2(mul2(g, pack2(-kLog2e, -kLog2e)), x0, x1);
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d0) : "f"(x0));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d1) : "f"(x1));
  unpack2(add2(pack2(d0, d1), pack2(1.0f, 1.0f)), d0, d1);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(d0));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(d1));
  unpack2(mul2(mul2(g, pack2(r0, r1)), u), y0, y1);
  return pack_bf16x2(y0, y1);
}

// One tile: weight tile nb of expert e times rows [row0, row0 + n) of x; n = 0
// ends the tiles of a CTA.  kShared in nb: other tiles read these weights too.
constexpr int kShared = 1 << 30;
struct Tile {
  int e, nb, n, row0;
};

// The CTA's tiles in turn, decoded and handed out by the scheduling warp through
// two slots (log_slots 1): tiles differ in cost by a factor of ten and more (rows
// in the tile, weights in L2 or not), so each CTA takes the next one when it has
// room for it.  Warp 7 reads up to four stages ahead: where those reach beyond
// the next tile it takes four slots, or the epilogue, which frees the slots last,
// would wait for a stage that warp 7 stores only once it has its next tile.
struct Feed {
  uint64_t *full, *empty;
  const volatile int4 *slots;
  volatile int32_t *abort_flag;
  int32_t *status;
  uint32_t log_slots, n;

  // One thread: the next tile (n = 0 after an abort too).
  __device__ __forceinline__ Tile next() {
    const uint32_t i = n & ((1u << log_slots) - 1u);
    if (!mbar_wait(full + i, (n >> log_slots) & 1u, abort_flag, status, moe::K_FP4_PRODUCT))
      return Tile{0, 0, 0, 0};
    const Tile t{slots[i].x, slots[i].y, slots[i].z, slots[i].w};
    mbar_arrive(empty + i);
    ++n;
    return t;
  }
  // A whole warp.
  __device__ __forceinline__ Tile next_warp(int lane) {
    Tile t{0, 0, 0, 0};
    if (lane == 0) t = next();
    t.e = __shfl_sync(0xffffffffu, t.e, 0);
    t.nb = __shfl_sync(0xffffffffu, t.nb, 0);
    t.n = __shfl_sync(0xffffffffu, t.n, 0);
    t.row0 = __shfl_sync(0xffffffffu, t.row0, 0);
    return t;
  }
};

template <int FMT, bool SWIGLU, typename Y, int ROWS>
__global__ void __launch_bounds__(Cfg<ROWS>::kThreads, 1)
    product_kernel(const __grid_constant__ CUtensorMap tmap_x, const Params p) {
  using C = Cfg<ROWS>;
  using Bars = typename C::Bars;
  constexpr int kStages = C::kStages, kStageBytes = C::kStageBytes, kXOff = C::kXOff,
                kXsOff = C::kXsOff, kThreads = C::kThreads, kBlocks = C::kBlocks,
                kEpiThreads = 32 * C::kEpiWarps;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Bars *bars = reinterpret_cast<Bars *>(smem + C::kBarsOff);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kMiscOff);
  volatile int32_t *abort_flag = reinterpret_cast<int32_t *>(smem + C::kMiscOff + 4);
  volatile int4 *epi_tile = reinterpret_cast<int4 *>(smem + C::kEpiOff);
  int32_t *off = reinterpret_cast<int32_t *>(smem + C::kSegOff);  // [S + 1] first rows
  // [S + 1] row tiles before s, of segments of several and of one row tile
  int32_t *pre_h = off + kMaxSegs + 1;
  int32_t *pre_c = pre_h + kMaxSegs + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int32_t kid = moe::K_FP4_PRODUCT;
  constexpr int kScaleBytes = fp4::Fmt<FMT>::kScaleBytes;
  constexpr int kGroups = kScaleBytes / 4;  // 512-byte scale groups of 128 rows per stage
  constexpr uint32_t kTileBytes = fp4::tile_bytes(FMT);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bars->full[i], 2);  // the producer and the rows' scales
      mbar_init(&bars->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->tfull[i], 1);
      mbar_init(&bars->tempty[i], kEpiThreads);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bars->sfull[i], 1);
      mbar_init(&bars->sempty[i], 4);  // producer, MMA, row scales, epilogue
    }
    mbar_init(&bars->drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  moe::pdl_wait();
  moe::pdl_trigger();
  int decreasing = 0;  // offsets that go back name no segments at all
  for (int s = threadIdx.x; s < p.S; s += kThreads) {
    const int64_t a = p.seg_offsets[s], b = p.seg_offsets[s + 1];
    const int e = p.seg_expert[s];
    int mt = 0;
    if (b < a) {
      moe::report_error(p.status, MOE_ERR_DEVICE_INDEX, s, kid);
      decreasing = 1;
    }
    if (b > a) {
      if (a < 0 || b > p.n_rows || e < 0 || e >= p.E)
        moe::report_error(p.status, MOE_ERR_DEVICE_INDEX, s, kid);
      else
        mt = (int)((b - a + ROWS - 1) / ROWS);
    }
    off[s] = (int)a;
    if (s == p.S - 1) off[p.S] = (int)b;
    pre_h[s] = mt > 1 ? mt : 0;
    pre_c[s] = mt > 1 ? 0 : mt;
  }
  const bool none = __syncthreads_or(decreasing) != 0;
  if (warp == 0) warp_exclusive_scan(pre_h, p.S, lane);
  if (warp == 2) warp_exclusive_scan(pre_c, p.S, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  volatile int4 *slots = reinterpret_cast<int4 *>(smem + C::kSlotsOff);
  const uint32_t log_slots = p.nkb >= 4 ? 1 : 2;
  Feed feed{bars->sfull, bars->sempty, slots, abort_flag, p.status, log_slots, 0};

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (elect_one()) {
      prefetch_tmap(&tmap_x);
      // weights of several row tiles are kept in L2, others make room at once:
      // 32768 rows over 256 experts in Zipf segments 487 -> 464 us, 65536 over 32
      // 557 -> 539 us
      const uint64_t pol_once = policy_evict_first(), pol_keep = policy_evict_last();
      int stage = 0;
      uint32_t phase = 0, armed = 0, armed_par = 0;
      bool ok = true;
      for (Tile ti; ok && (ti = feed.next()).n > 0;) {
        const int boxes = (ti.n + kBoxRows - 1) / kBoxRows;
        const uint64_t pol = ti.nb & kShared ? pol_keep : pol_once;
        const uint8_t *w =
            p.w + ((int64_t)ti.e * p.nbn + (ti.nb & ~kShared)) * p.nkb * (int64_t)kTileBytes;
        for (int kb = 0; kb < p.nkb; ++kb) {
          if (!mbar_wait(&bars->empty[stage], phase ^ 1u, abort_flag, p.status, kid)) {
            ok = false;
            break;
          }
          uint8_t *st = smem + (size_t)stage * kStageBytes;
          mbar_arrive_expect_tx(&bars->full[stage], kTileBytes + boxes * kBoxRows * 128);
          bulk_load(st, w + (int64_t)kb * kTileBytes, kTileBytes, &bars->full[stage], pol);
          for (int b = 0; b < boxes; ++b)
            tma_load_2d(st + kXOff + b * kBoxRows * 128, &tmap_x, kb * 128, ti.row0 + b * kBoxRows,
                        &bars->full[stage]);
          armed |= 1u << stage;
          armed_par = (armed_par & ~(1u << stage)) | (phase << stage);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // Own copies land before the CTA exits.  After an abort the scales'
      // arrival of a stage may never come, so it is made here; where it did
      // come, the extra one counts towards a phase that nobody waits for.
      if (!ok)
        for (int i = 0; i < kStages; ++i)
          if ((armed >> i) & 1u) mbar_arrive(&bars->full[i]);
      for (int i = 0; i < kStages; ++i)
        if ((armed >> i) & 1u) mbar_wait_drain(&bars->full[i], (armed_par >> i) & 1u);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (elect_one()) {
      int stage = 0, acc = 0;
      uint32_t phase = 0, pe = 0;  // bit i: slot i's phase
      bool ok = true;
      for (Tile ti; ok && (ti = feed.next()).n > 0;) {
        const uint32_t nmma = (uint32_t)((ti.n + 15) & ~15);
        // e2m1 operands (bits 7-9, 10-11), N / 8 at 17, scales E8M0 (1) or
        // E4M3 (0) at 23, M = 128 at 27
        const uint32_t idesc = (1u << 7) | (1u << 10) | ((nmma >> 3) << 17) |
                               ((FMT == 0 ? 1u : 0u) << 23) | (1u << 27);
        // a tile of more than 112 rows takes both slots
        const bool big = ROWS > kSlotRows && ti.n > kSlotRows;
        if (big) acc = 0;
        const int slot = acc, rows = big ? ROWS : kSlotRows;
        if (!mbar_wait(&bars->tempty[slot], (pe >> slot & 1u) ^ 1u, abort_flag, p.status, kid)) break;
        pe ^= 1u << slot;
        if (big) {
          if (!mbar_wait(&bars->tempty[1], (pe >> 1) ^ 1u, abort_flag, p.status, kid)) break;
          pe ^= 2u;
        }
        tc_fence_after();
        const uint32_t d = tmem_base + (uint32_t)(slot * kSlotCols);
        const uint32_t sfa = tmem_base + kScaleCol, sfb = sfa + 32;
        for (int kb = 0; kb < p.nkb; ++kb) {
          if (!mbar_wait(&bars->full[stage], phase, abort_flag, p.status, kid)) {
            ok = false;
            break;
          }
          tc_fence_after();
          // warp 7's stores before the copies below.  (Here, not in warp 7: the
          // fence would wait for its loads in flight.)
          fence_proxy_async_shared();
          const uint32_t sw = smem_u32(smem + (size_t)stage * kStageBytes);
          const uint32_t sx = sw + kXOff;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int g = 0; g < kGroups; ++g)
              copy_scales(sfa + (h * kGroups + g) * 4,
                          sw + fp4::kTileCodes + (h * kGroups + g) * 512);
#pragma unroll
          for (int g = 0; g < kGroups; ++g)
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
              copy_scales(sfb + (g * kBlocks + b) * 4, sw + kXsOff + (g * kBlocks + b) * 512);
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            // NV: a group a step; MX: two steps share a group's 4 bytes
            const int g = FMT == 1 ? s : s / 2;
            const uint32_t id = FMT == 1 ? 0u : (uint32_t)(s & 1) * 2u;
            const uint32_t idesc_s = idesc | (id << 4) | (id << 29);
#pragma unroll
            for (int h = 0; h < 2; ++h)
              mma_fp4<FMT>(d + h * rows, sw128_desc(sw + h * 16384 + s * 32),
                           sw128_desc(sx + s * 32), idesc_s, sfa + (h * kGroups + g) * 4,
                           sfb + g * kBlocks * 4, (kb | s) != 0 ? 1u : 0u);
          }
          umma_commit(&bars->empty[stage]);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        umma_commit(&bars->tfull[slot]);
        acc = big ? 0 : acc ^ 1;
      }
      umma_commit(&bars->drain);
      mbar_wait_drain(&bars->drain, 0);
    }
  } else if (warp == 7) {
    // ------------------------------------------- the rows' scales, per stage
    constexpr int kPer = 4 * kBlocks;  // rows of a lane
    uint32_t v[kStages][kPer][kGroups];
    bool have[kStages];  // which of v hold a stage
    int kb = 0;
    Tile ti = feed.next_warp(lane);
    bool more = ti.n > 0;
    auto load = [&](uint32_t (&u)[kPer][kGroups]) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {  // rows lane, lane + 32, ...
#pragma unroll
        for (int g = 0; g < kGroups; ++g) u[j][g] = 0;
        const int r = lane + 32 * j;
        if (more && r < ti.n) {
          const uint8_t *src = p.sf + (int64_t)(ti.row0 + r) * p.sf_ld + kb * kScaleBytes;
          if constexpr (FMT == 1) {
            const uint4 x = __ldg(reinterpret_cast<const uint4 *>(src));
            u[j][0] = x.x;
            u[j][1] = x.y;
            u[j][2] = x.z;
            u[j][3] = x.w;
          } else {
            const uint2 x = __ldg(reinterpret_cast<const uint2 *>(src));
            u[j][0] = x.x;
            u[j][1] = x.y;
          }
        }
      }
      const bool got = more;
      if (more && ++kb == p.nkb) {
        kb = 0;
        ti = feed.next_warp(lane);
        more = ti.n > 0;
      }
      return got;
    };
#pragma unroll
    for (int d = 0; d < kStages; ++d) have[d] = load(v[d]);
    uint32_t phase = 0;
    bool ok = true;
    for (; ok; phase ^= 1u) {
#pragma unroll
      for (int d = 0; d < kStages; ++d) {
        if (!ok || !have[d]) {
          ok = false;
          break;
        }
        int got = 0;
        if (lane == 0)
          got = mbar_wait(&bars->empty[d], phase ^ 1u, abort_flag, p.status, kid) ? 1 : 0;
        ok = __shfl_sync(0xffffffffu, got, 0) != 0;
        if (!ok) break;
        uint8_t *dst = smem + (size_t)d * kStageBytes + kXsOff + lane * 16;
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
#pragma unroll
          for (int b = 0; b < kBlocks; ++b)
            *reinterpret_cast<uint4 *>(dst + (g * kBlocks + b) * 512) = make_uint4(
                v[d][4 * b][g], v[d][4 * b + 1][g], v[d][4 * b + 2][g], v[d][4 * b + 3][g]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->full[d]);
        have[d] = load(v[d]);
      }
    }
  } else if (warp == 6) {
    // ------------------------------------------------------------ scheduler
    // Tiles in order (segment, weight tile, row tile), so that CTAs side by side
    // read the same weight tile; those of segments of several row tiles (bound
    // by what SMs take in from L2) and of one (bound by HBM) merged in
    // proportion to their numbers.
    if (lane == 0) {
      const int64_t Mh = none ? 0 : pre_h[p.S], Mc = none ? 0 : pre_c[p.S];
      const int64_t total = (Mh + Mc) * p.nbn;
      int64_t t = blockIdx.x;
      for (uint32_t n = 0;; ++n) {
        Tile x{0, 0, 0, 0};
        if (t < total) {
          int s, m;
          if (Mh > 0 && Mc > 0)  // (the merge costs two 64-bit divisions)
            tile_order::merged(t, pre_h, pre_c, p.S, p.nbn, Mh, Mc, s, x.nb, m);
          else
            tile_order::in_stream(t, Mh > 0 ? pre_h : pre_c, p.S, p.nbn, s, x.nb, m);
          const int mt = pre_h[s + 1] - pre_h[s] + pre_c[s + 1] - pre_c[s];
          x.e = __ldg(p.seg_expert + s);
          tile_order::row_tile(off[s + 1] - off[s], mt, m, x.row0, x.n);
          x.row0 += off[s];
          if (mt > 1) x.nb |= kShared;
        }
        const uint32_t i = n & ((1u << log_slots) - 1u);
        if (!mbar_wait(&bars->sempty[i], ((n >> log_slots) & 1u) ^ 1u, abort_flag, p.status, kid))
          break;
        slots[i].x = x.e;
        slots[i].y = x.nb;
        slots[i].z = x.n;
        slots[i].w = x.row0;
        mbar_arrive(&bars->sfull[i]);
        if (x.n == 0) break;
        t = (int64_t)gridDim.x + atomicAdd(p.counter, 1);
      }
    }
  } else {
    // ------------------------------------------- epilogue warps 2..5 (8..11)
    const int q = warp & 3;          // TMEM lane quadrant this warp may access
    const int part = warp >= 8;      // which of the quadrant's warps
    constexpr int kStep = 16 * (C::kEpiWarps / 4);  // they take 16 rows in turn
    int acc = 0, turn = 0;
    uint32_t pf = 0;  // bit i: slot i's phase
    for (;; turn ^= 1) {
      // One thread takes the tile and waits for its products; all act on what it
      // leaves in one of two places in turn, so that the barrier is always
      // reached by every epilogue warp or, after an abort, by none.
      auto is_big = [](const Tile &t) { return ROWS > kSlotRows && t.n > kSlotRows; };
      if (warp == 2 && lane == 0) {
        Tile t = feed.next();
        const int slot = is_big(t) ? 0 : acc;
        if (t.n > 0 && !mbar_wait(&bars->tfull[slot], pf >> slot & 1u, abort_flag, p.status, kid))
          t.n = 0;
        epi_tile[turn].x = t.e;
        epi_tile[turn].y = t.nb;
        epi_tile[turn].z = t.n;
        epi_tile[turn].w = t.row0;
      }
      asm volatile("bar.sync 1, %0;" ::"n"(kEpiThreads) : "memory");
      const Tile ti{epi_tile[turn].x, epi_tile[turn].y & ~kShared, epi_tile[turn].z,
                    epi_tile[turn].w};
      if (ti.n == 0) break;
      const bool big = is_big(ti);
      if (big) acc = 0;
      const int slot = acc, rows = big ? ROWS : kSlotRows;
      pf ^= 1u << slot;
      tc_fence_after();
      const float alpha = p.alpha ? __ldg(p.alpha + ti.e) : 1.0f;
      const uint32_t tbase = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(slot * kSlotCols);
      const int colw = ti.nb * (SWIGLU ? 128 : 256) + q * 32;  // the warp's first column
      if constexpr (sizeof(Y) == 4) {
        // fp32: a lane's weight row is a column of out, 128 bytes a store
        const int col0 = colw + lane;
        Y *out = static_cast<Y *>(p.out) + (int64_t)ti.row0 * p.out_n + col0;
#pragma unroll 1
        for (int c = 16 * part; c < ti.n; c += kStep) {
          uint32_t a[16], b[16];
          tmem_ld16(tbase + c, a);
          tmem_ld16(tbase + rows + c, b);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (c + i >= ti.n) break;
            const float va = __uint_as_float(a[i]) * alpha, vb = __uint_as_float(b[i]) * alpha;
            Y *o = out + (int64_t)(c + i) * p.out_n;
            if (SWIGLU) {
              if (col0 < p.out_n) *o = swiglu_accurate(va, vb);
            } else {
              if (col0 < p.out_n) *o = va;
              if (col0 + 128 < p.out_n) o[128] = vb;
            }
          }
        }
      } else {
        // bf16: 32 weight rows x 16 rows of x at a time, transposed through
        // the warp's kilobyte of shared memory (row t in 64 bytes, 16-byte
        // chunk c at c ^ (t / 2 % 4)), out in 16-byte stores
        uint8_t *buf = smem + C::kOutOff + (4 * part + q) * kOutWarpBytes;
        const int piece = lane >> 3, st_row = (lane & 7) + (piece >> 1) * 8;
        const uint32_t st = smem_u32(buf) + st_row * 64;
        const int st_sw = (st_row >> 1) & 3;
        const uint64_t alpha2 = pack2(alpha, alpha);
        Y *out = static_cast<Y *>(p.out) + (int64_t)ti.row0 * p.out_n;
#pragma unroll 1
        for (int c = 16 * part; c < ti.n; c += kStep) {
          uint32_t v[2][2][8];  // [weight half][16 lanes][8]
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int r = 0; r < 2; ++r)
              tmem_ld_16x16(tbase + ((uint32_t)(16 * r) << 16) + h * rows + c, v[h][r]);
          tmem_wait_ld();
#pragma unroll
          for (int h = 0; h < (SWIGLU ? 1 : 2); ++h) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              uint32_t pk[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if (SWIGLU)
                  pk[i] = swiglu_fast2(v[0][r][2 * i], v[0][r][2 * i + 1], v[1][r][2 * i],
                                       v[1][r][2 * i + 1], alpha2);
                else
                  pk[i] = pack_bf16x2(__uint_as_float(v[h][r][2 * i]) * alpha,
                                      __uint_as_float(v[h][r][2 * i + 1]) * alpha);
              }
              stmatrix_t(st + (((2 * r + (piece & 1)) ^ st_sw) << 4), pk[0], pk[1], pk[2], pk[3]);
            }
            __syncwarp();
            const int col = colw + h * 128 + (lane & 3) * 8;
#pragma unroll
            for (int it = 0; it < 2; ++it) {
              const int t = it * 8 + (lane >> 2);
              const uint4 x = *reinterpret_cast<const uint4 *>(
                  buf + t * 64 + (((lane & 3) ^ ((t >> 1) & 3)) << 4));
              if (c + t < ti.n && col < p.out_n)
                *reinterpret_cast<uint4 *>(out + (int64_t)(c + t) * p.out_n + col) = x;
            }
            __syncwarp();
          }
        }
      }
      tc_fence_before();
      mbar_arrive(&bars->tempty[slot]);
      if (big) mbar_arrive(&bars->tempty[1]);
      acc = big ? 0 : acc ^ 1;
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmemCols);
  }
  // The last CTA to finish (no tile is taken any more) clears the counters for
  // the next launch on this workspace.
  if (threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(p.counter + 1, 1) == (int)gridDim.x - 1) {
      p.counter[0] = 0;
      p.counter[1] = 0;
    }
  }
}

// ------------------------------------------------------------------ host
// Above this many rows a segment on average, tiles of up to 224 rows.  (Empty
// segments count: how many there are is known on the device only, so a few long
// segments among many empty ones take the smaller tiles.)  Equal segments, 4096 x
// 4096: 64 experts of 64 rows 93 us either way, of 128 rows 106 us (a segment one
// tile instead of two, its weights read once), 4 experts of 2048 rows 68 us
// against 74 us.  Fewer rows a segment fill one slot, and four stages keep more
// of the weight stream in flight.
constexpr int kBigRows = 64;

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

template <int FMT, bool SWIGLU, typename Y, int ROWS>
moe_status launch(const CUtensorMap &m, const Params &p, cudaStream_t st) {
  constexpr int kMaxDevices = 64;
  static bool done[kMaxDevices] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices || !done[dev]) {
    if (cudaFuncSetAttribute(product_kernel<FMT, SWIGLU, Y, ROWS>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)Cfg<ROWS>::kSmemBytes) != cudaSuccess)
      return MOE_ERR_CUDA;
    if (dev >= 0 && dev < kMaxDevices) done[dev] = true;
  }
  int64_t grid = moe_host::sm_count();
  const int64_t max_tiles = ((p.n_rows + ROWS - 1) / ROWS + p.S) * p.nbn;
  if (max_tiles < grid) grid = max_tiles;
  return moe_host::launch_pdl(product_kernel<FMT, SWIGLU, Y, ROWS>, dim3((unsigned)grid),
                              dim3(Cfg<ROWS>::kThreads), Cfg<ROWS>::kSmemBytes, st, m, p);
}

template <int FMT, bool SWIGLU>
moe_status launch_type(const CUtensorMap &m, const Params &p, int32_t out_type, cudaStream_t st) {
  const bool big = p.n_rows > (int64_t)p.S * kBigRows;
  if (out_type == MOE_F32)
    return big ? launch<FMT, SWIGLU, float, 224>(m, p, st) : launch<FMT, SWIGLU, float, 112>(m, p, st);
  return big ? launch<FMT, SWIGLU, __nv_bfloat16, 224>(m, p, st)
             : launch<FMT, SWIGLU, __nv_bfloat16, 112>(m, p, st);
}

}  // namespace

extern "C" moe_status moe_grouped_product_fp4(const uint8_t *codes, const uint8_t *sf,
                                              int64_t n_rows, const int32_t *seg_offsets,
                                              const int32_t *seg_expert, int32_t S, int32_t E,
                                              const uint8_t *w_packed, int32_t N, int32_t K,
                                              int32_t fmt, int32_t epilogue, const float *alpha,
                                              void *out, int32_t out_type, void *ws,
                                              size_t ws_bytes, void *stream) {
  if (n_rows < 0 || S < 1 || E < 1 || N < 1 || K < 1) return MOE_ERR_INVALID_ARG;
  if (fmt != MOE_FP4_MX && fmt != MOE_FP4_NV) return MOE_ERR_INVALID_ARG;
  if (epilogue != MOE_EPI_NONE && epilogue != MOE_EPI_SWIGLU) return MOE_ERR_INVALID_ARG;
  if (out_type != MOE_F32 && out_type != MOE_BF16) return MOE_ERR_INVALID_ARG;
  const bool swi = epilogue == MOE_EPI_SWIGLU;
  if (S > kMaxSegs || K % 32 != 0 || K > (1 << 24) || N % (swi ? 16 : 8) != 0 ||
      n_rows >= ((int64_t)1 << 31) - kBoxRows)
    return MOE_ERR_UNSUPPORTED;
  Params p{};
  p.nkb = (K + fp4::kStepElems - 1) / fp4::kStepElems;
  p.nbn = swi ? (N / 2 + 127) / 128 : (N + 255) / 256;
  const int64_t max_tiles = ((n_rows + kSlotRows - 1) / kSlotRows + S) * p.nbn;
  if (max_tiles >= ((int64_t)1 << 31) - 65536) return MOE_ERR_UNSUPPORTED;
  if (!seg_offsets || !seg_expert || !w_packed) return MOE_ERR_INVALID_ARG;
  if (moe_status s = moe_host::check_ws(ws, ws_bytes, moe::kStatusBytes)) return s;
  if (n_rows == 0) return MOE_OK;
  if (!codes || !sf || !out) return MOE_ERR_INVALID_ARG;
  if (!moe_host::aligned16(codes) || !moe_host::aligned16(sf) || !moe_host::aligned16(w_packed) ||
      !moe_host::aligned16(out))
    return MOE_ERR_INVALID_ARG;
  PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
  if (!fn) return MOE_ERR_CUDA;
  // rows' codes: [n_rows, K / 2] bytes, boxes of 128 bytes x 16 rows
  CUtensorMap m;
  cuuint64_t dims[2] = {(cuuint64_t)K / 2, (cuuint64_t)n_rows};
  cuuint64_t strides[1] = {(cuuint64_t)K / 2};
  cuuint32_t box[2] = {128, kBoxRows};
  cuuint32_t estr[2] = {1, 1};
  if (fn(&m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(codes), dims, strides, box,
         estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return MOE_ERR_CUDA;
  p.seg_offsets = seg_offsets;
  p.seg_expert = seg_expert;
  p.w = w_packed;
  p.sf = sf;
  p.alpha = alpha;
  p.out = out;
  p.status = moe_host::status_ptr(ws);
  p.counter = p.status + moe::kFp4CounterWord;
  p.n_rows = n_rows;
  p.S = S;
  p.E = E;
  p.sf_ld = (int32_t)moe_fp4_scale_ld(K, fmt);
  p.out_n = swi ? N / 2 : N;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (fmt == MOE_FP4_MX)
    return swi ? launch_type<0, true>(m, p, out_type, st)
               : launch_type<0, false>(m, p, out_type, st);
  return swi ? launch_type<1, true>(m, p, out_type, st)
             : launch_type<1, false>(m, p, out_type, st);
}
