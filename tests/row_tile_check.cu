// Host-side check of the FP4 product's row tiles (tile_order.cuh): for segments
// of every small size and of sizes up to the largest that the product takes,
// the tiles of a segment follow one another without a gap, are multiples of 16
// but for the last, at most R rows and never empty.  Built with nvcc as a host
// program; needs no GPU.  Exit code 0 = all cases pass.
#include <cstdint>
#include <cstdio>

#include "tile_order.cuh"

static bool one(int64_t rows, int R) {
  const int mt = (int)((rows + R - 1) / R);  // as the kernel counts them
  // every tile of a short segment; of a long one both ends and some between
  const int step = mt > 5000 ? mt / 1000 : 1;
  int64_t next = 0;
  for (int m = 0; m < mt; m += (m + 4 < mt && m > 4) ? step : 1) {
    if (m >= mt) break;
    int first = -1, n = -1;
    tile_order::row_tile((int)rows, mt, m, first, n);
    if (step == 1 || m <= 5) {
      if (first != next) return false;
      next = (int64_t)first + n;
    }
    if (first < 0 || n < 1 || n > R || (int64_t)first + n > rows) return false;
    if (m + 1 < mt && n % 16 != 0) return false;
  }
  int first = -1, n = -1;
  tile_order::row_tile((int)rows, mt, mt - 1, first, n);
  return n >= 1 && n <= R && (int64_t)first + n == rows;
}

int main() {
  const int64_t top = ((int64_t)1 << 31) - 17;
  int64_t cases = 0;
  for (int R : {112, 224}) {
    for (int64_t rows = 1; rows < 60000; ++rows, ++cases)
      if (!one(rows, R)) {
        std::printf("%lld rows in tiles of %d\n", (long long)rows, R);
        return 1;
      }
    for (int64_t rows = top; rows > 60000; rows -= rows > top - 2000 ? 1 : rows / 50, ++cases)
      if (!one(rows, R)) {
        std::printf("%lld rows in tiles of %d\n", (long long)rows, R);
        return 1;
      }
  }
  std::printf("row tiles ok: %lld segments\n", (long long)cases);
  return 0;
}
