// Host-side check of the launch shapes of the block's kernels (block_shape.cuh): for
// every row width, number of experts, type and set of optional rows that the calls
// take, a launch has CTAs, threads and shared memory within a CTA's limits, and no
// more CTAs than the norm weight's gradient has partial rows.  Built with nvcc as a
// host program; needs no GPU.  Exit code 0 = all cases pass.
#include <cstdio>

#include "block_shape.cuh"

using namespace block_shape;

constexpr size_t kCtaSmem = 227 * 1024, kStaticSmem = 1024, kSmSmem = 228 * 1024;

static long long bad = 0, cases = 0;

static void rows(const char *what, int H, int k, int T, int sms, int threads, int sm_threads, size_t smem) {
  const unsigned grid = rows_grid(T, threads, sm_threads, smem, sms);
  ++cases;
  if (grid >= 1 && grid <= (unsigned)T && threads >= 32 && threads <= kRowThreads && threads % 32 == 0 &&
      smem + kStaticSmem <= kCtaSmem)
    return;
  if (bad++ < 20) std::printf("%s: H %d k %d T %d: grid %u threads %d smem %zu\n", what, H, k, T, grid, threads, smem);
}

static void teams(const char *what, int H, int k, int T, int sms, int n, int values, bool partial) {
  const TeamShape s(T, H, n, values, partial, sms);
  ++cases;
  const size_t ring = (size_t)s.threads * 16 * n, sums = (size_t)sums_floats(values) * 2 * 4;
  if (s.grid >= 1 && s.grid <= bwd_grid(T, H, sms) && s.teams >= 1 && s.teams <= 8 && (s.r == 1 || s.r == 2) &&
      s.threads * row_chunks(H) * 8 >= H && s.teams * s.threads <= kRowThreads &&
      s.smem >= s.teams * (sums + s.r * ring) && (!partial || s.smem >= (size_t)(s.teams - 1) * H * 4) &&
      s.smem + kStaticSmem <= kCtaSmem && s.smem + 1024 <= kSmSmem)
    return;
  if (bad++ < 20)
    std::printf("%s: H %d k %d T %d rows %d: grid %u teams %d of %d smem %zu\n", what, H, k, T, n, s.grid, s.teams,
                s.threads, s.smem);
}

int main() {
  for (int H = 8; H <= kMaxH; H += 8)
    for (int sms : {1, 152})
      for (int T : {1, 5, 100000}) {
        const int u = fwd_pieces(H);
        for (int x = 1; x <= 2; ++x) {  // 16-byte pieces of 8 elements of the type: bf16, fp32
          rows("norm", H, 1, T, sms, threads_of(H, u), u <= 2 ? 1024 : 512, (size_t)threads_of(H, u) * 16 * 2 * u * x);
          for (int k = 1; k <= 16; ++k) {
            const int kmax = k <= 2 ? 2 : k <= 4 ? 4 : k <= 8 ? 8 : 16;
            for (int shared = 0; shared < 2; ++shared) {
              const size_t ring = (size_t)threads_of(H, u) * 16 * (k + x + shared);
              const bool two = u > 1 && 2 * ring <= kSmemLimit;
              rows("combine", H, k, T, sms, threads_of(H, u), u == 1 ? 1024 : 512, two ? 2 * ring : ring);
              for (bool partial : {false, true}) {
                teams("after the experts", H, k, T, sms, k + x + shared, 2 * kmax + 2, partial);
                for (int res = 0; res < 2; ++res)  // shared: add
                  teams("before the experts", H, k, T, sms, k + x * (1 + res) + shared, 2, partial);
              }
            }
          }
        }
      }
  std::printf("%s: %lld of %lld shapes are wrong\n", bad ? "block shapes" : "block shapes ok", bad, cases);
  return bad != 0;
}
