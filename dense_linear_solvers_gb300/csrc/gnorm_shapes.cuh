// Shapes of the norms' kernels and the sums over rows (bs_gnorm calls).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "kernels.h"

namespace bsolve {

constexpr int kLong = 1024;  // threads of the looped kernels

// Threads of a row, vectors a thread and rows a turn; threads == 0: the looped kernels.
struct Shape {
  int threads, vectors, rows;
};

// Forward, with 16-byte vectors: the fewest threads with one each, 8 at least, two rows a turn; one row
// for blocks of 1024 threads, two vectors each for the longest rows.
inline Shape forward_shape(int width, int es) {
  const int n = (width * es + 15) / 16;
  for (int threads = 8; threads <= 512; threads *= 2)
    if (n <= threads) return {threads, 1, 2};
  if (n <= 1024) return {1024, 1, 1};
  return n <= 2048 ? Shape{1024, 2, 1} : Shape{0, 0, 1};
}

// Backward. 16 bits: 16-byte vectors, two rows a turn, which 128 registers a thread hold, 16 warps an
// SM: what a turn costs beside its elements is then spread over 16 of them. FP32: one row a turn
// with 64 registers and 32 warps, for which shared memory has room. Rows of more than 4096
// elements: 1024 threads, in 16 bits with two vectors of four elements each.
inline Shape backward_shape(int width, int es) {
  const int n = (width * es + 15) / 16, rows = es == 2 ? 2 : 1;
  for (int threads = 8; threads <= 512; threads *= 2)
    if (n <= threads) return {threads, 1, rows};
  return n <= 1024 ? Shape{1024, es == 2 ? 2 : 1, 1} : Shape{0, 0, 1};
}

inline int block_of(const Shape& s) { return s.threads == 0 ? kLong : (s.threads <= 32 ? 128 : s.threads); }

// Persistent blocks: what the GPU holds with 1024 threads an SM, or what the rows need.
inline int blocks_for(const Shape& s, int64_t rows, int threads = 1024) {
  const int64_t turn = s.threads == 0 ? 1 : s.rows * (block_of(s) / s.threads);
  const int64_t need = (rows + turn - 1) / turn;
  const int64_t held = static_cast<int64_t>(kSms) * (threads / block_of(s));
  return static_cast<int>(need < held ? need : held);
}

inline int backward_blocks(int width, int es, int64_t rows) {
  const Shape s = backward_shape(width, es);
  // looped: two blocks of 1024 threads with 32 registers each (4,096 x 8,192 FP32 training pass: 851 us,
  // with one block 1,093)
  return blocks_for(s, rows, s.threads == 0 ? 2 * kLong : (s.rows == 2 ? 512 : 1024));
}

// dw_post, dscale, dw_pre (null: not wanted) from `parts` partial sums, [parts][3][width].
cudaError_t launch_gnorm_sums(int width, int parts, const float* partial, float* dw_post,
                              float* dscale, float* dw_pre, cudaStream_t stream);

}  // namespace bsolve
