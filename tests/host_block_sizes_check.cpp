// Sizes that the host works out for the kernels between a block's linear
// layers, at the largest row counts; built for the CPU with AddressSanitizer
// and UndefinedBehaviorSanitizer by tests/test_block_abi_edges.py.  Prints
// "host block size checks passed" and returns 0 when every check holds.
#include <cstdint>
#include <cstdio>

#include "fp8q_internal.h"

int main() {
  int failures = 0;
  for (int64_t rows : {int64_t(1), int64_t(33), int64_t(129), int64_t(16385), (int64_t(1) << 31) - 512, (int64_t(1) << 31) - 1})
    for (int n : {8193, 16385, 1 << 29})
      for (bool f32 : {false, true}) {
        const fp8q::NormBwdShape s = fp8q::norm_bwd_shape((int)rows, n, f32);
        if (s.chunks != 0) continue;  // (a row in registers)
        const int64_t per = fp8q::norm_dw_rows((int)rows, s.blocks);
        // the blocks' rows are all there are, and no block begins before the one ahead of it
        if (!(per >= 1 && per * s.blocks >= rows && (per - 1) * s.blocks < rows)) {
          std::printf("rows %lld, %d columns, %d blocks: %lld rows each\n", (long long)rows, n, s.blocks, (long long)per);
          ++failures;
        }
      }
  // the forward pass: every width is held by the threads, and few rows' have what many rows' have in half as many with twice the chunks
  for (int n : {0, 1, 512, 1024, 1025, 1030, 1536, 2048, 2049, 4096, 4097, 7168, 8193, 16384})
    for (int rows : {1, 2047, 2048, 4095, 4096, 1 << 21, 2147483647}) {
      const fp8q::NormShape s = fp8q::norm_shape(rows, n), many = fp8q::norm_shape(2147483647, n);
      const bool holds = (int64_t)s.threads * s.chunks * 8 >= n && s.threads % 64 == 0 && s.threads >= 64 && s.threads <= (s.chunks == 4 ? 512 : 1024);
      const bool halves = s.threads == 2 * many.threads || (s.threads == 192 && many.threads == 128 && s.chunks == 1 && n <= 192 * 8);
      const bool same = s.split ? s.chunks <= 2 && many.threads % 64 == 0 && halves && 2 * s.chunks == many.chunks
                                : s.threads == many.threads && s.chunks == many.chunks;
      if (!holds || !same || many.split) {
        std::printf("%d rows, %d columns: %d chunks of %d threads, many rows %d of %d\n", rows, n, s.chunks, s.threads, many.chunks, many.threads);
        ++failures;
      }
    }
  if (failures == 0) std::printf("host block size checks passed\n");
  return failures != 0;
}
