// Launch shapes of the block's kernels (block.cu): threads, CTAs and shared memory
// from the sizes of a call.  Host arithmetic alone, so that it can be checked for
// every size without a GPU.
#pragma once
#include <cstddef>
#include <cstdint>

namespace block_shape {

// A token's team has up to 512 threads, each with U pieces of 8 elements: two for
// rows of up to 8192, four beyond; in the forward pass one for rows of up to 1024,
// with 64 registers and twice the threads an SM (4096 tokens of 1024, six experts,
// combine with norms: 13.4 us against 16 with two pieces).
// R of the U pieces have a place in shared memory.
constexpr int kRowThreads = 512;
constexpr int kMaxH = kRowThreads * 4 * 8;
// Dynamic shared memory of a CTA, of the 227 KB that one may have.
constexpr int kSmemLimit = 225 * 1024;

// A warp's sums, a line a value (a team has at most 16 warps; lines of 20 floats let
// lanes read 16 bytes of lines of their own without bank conflicts).
constexpr int kLine = 20;
// Floats of n values' lines, whole 128-byte lines: a warp's 512 bytes of a ring after
// them then lie in four (not aligned, 4096 x 7168 with eight experts took 114 us
// instead of 109).
#ifdef __CUDACC__
__host__ __device__
#endif
constexpr int sums_floats(int n) { return (n * kLine + 31) / 32 * 32; }

// Threads of the streaming kernels: at most 128, and such that their turns over a
// row are full (H = 1416: 96 in two turns instead of 128 of which half the second
// turn's idle).
inline int stream_threads(int H) {
  const int pieces = H / 8, turns = (pieces + 127) / 128;
  return ((pieces + turns - 1) / turns + 31) / 32 * 32;
}
// CTAs of the streaming kernels, at most 32 an SM.
inline unsigned stream_grid(int64_t T, int sms) {
  const int64_t cap = (int64_t)sms * 32;
  return (unsigned)(T < cap ? T : cap);
}

inline int row_chunks(int H) { return H <= kRowThreads * 2 * 8 ? 2 : 4; }
inline int fwd_pieces(int H) { return H <= 1024 ? 1 : row_chunks(H); }
inline int threads_of(int H, int u) { return ((H / 8 + u - 1) / u + 31) / 32 * 32; }
inline int row_threads(int H) { return threads_of(H, row_chunks(H)); }

// CTAs of a kernel with one token a CTA at a time: as many an SM as shared memory and
// `sm_threads` threads allow (512 with up to 128 registers).  All run at once, each
// with its share of the tokens.
inline unsigned rows_grid(int64_t T, int threads, int sm_threads, size_t smem, int sms) {
  int64_t per_sm = (int64_t)(kSmemLimit / (smem + 1280));
  if (per_sm > sm_threads / threads) per_sm = sm_threads / threads;
  if (per_sm > 30) per_sm = 30;
  if (per_sm < 1) per_sm = 1;
  const int64_t grid = per_sm * sms;
  return (unsigned)(grid < T ? grid : T);
}

// Teams of a CTA of the gradients: what 512 threads hold, at most 8.
inline int bwd_teams(int H) {
  const int n = kRowThreads / row_threads(H);
  return n < 1 ? 1 : n > 8 ? 8 : n;
}
// and the most CTAs that they run: 512 threads an SM with up to 128 registers (the
// norm weights' gradients have as many partial rows).
inline unsigned bwd_grid(int64_t T, int H, int sms) {
  const int teams = bwd_teams(H);
  const int64_t cap = (int64_t)sms * (kRowThreads / (teams * row_threads(H)));
  const int64_t need = (T + teams - 1) / teams;
  return (unsigned)(need < cap ? need : cap);
}

// A CTA of teams: for each, its sums twice and R pieces of all rows of a token
// (`ring` bytes each), and together at least the norm weight's partial sums.
// (No CTA waits for another to end: each has its share of the tokens.)
struct TeamShape {
  int threads, teams, r;
  unsigned grid;
  size_t smem;
  // rows: pieces of 16 bytes that a thread copies of each of its U places
  TeamShape(int64_t T, int H, int rows, int sum_values, bool partial_sums, int sms)
      : threads(row_threads(H)) {
    const size_t ring = (size_t)threads * 16 * rows;
    const size_t sums = (size_t)sums_floats(sum_values) * 2 * 4;
    teams = bwd_teams(H);
    while (teams > 1 && teams * (sums + 2 * ring) > kSmemLimit) --teams;
    r = teams * (sums + 2 * ring) <= kSmemLimit ? 2 : 1;
    smem = teams * (sums + r * ring);
    const size_t partial = (size_t)(teams - 1) * H * 4;
    if (partial_sums && smem < partial) smem = partial;
    grid = bwd_grid(T, H, sms);
    // (an SM has 228 KB, so a CTA of any size up to the limit fits once)
    const size_t per_sm = kSmemLimit / (smem + 1024);
    const int64_t fit = (int64_t)(per_sm < 1 ? 1 : per_sm) * sms;
    if (grid > fit) grid = (unsigned)fit;
  }
};

}  // namespace block_shape
