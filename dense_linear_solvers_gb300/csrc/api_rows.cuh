// Argument checks that the row operators' calls share.
#pragma once

#include <cstdint>
#include <initializer_list>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "bsolve.h"
#include "kernels.h"

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 30;  // a row's number, and a step beyond, fits 32 bits
constexpr int64_t kMaxLd = int64_t(1) << 21;

int element_size(bs_dtype dtype) {
  switch (dtype) {
    case BS_FP32: return 4;
    case BS_BF16:
    case BS_FP16: return 2;
    default: return 0;
  }
}

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// An operand of a call: `rows` pieces of `width` bytes, `pitch` bytes apart (null: absent).
struct Operand {
  const void* base;
  int64_t rows, width, pitch;
};

// Whether two operands share a byte. Operands of one pitch may interleave as column windows
// of one matrix: their windows are then compared within a row.
bool share(const Operand& a, const Operand& b) {
  if (!a.base || !b.base || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0)
    return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.base), y = reinterpret_cast<uintptr_t>(b.base);
  const uintptr_t xe = x + static_cast<uintptr_t>((a.rows - 1) * a.pitch + a.width);
  const uintptr_t ye = y + static_cast<uintptr_t>((b.rows - 1) * b.pitch + b.width);
  if (xe <= y || ye <= x) return false;
  if (a.pitch != b.pitch) return true;
  const int64_t pitch = a.pitch;
  const int64_t d = x <= y ? static_cast<int64_t>((y - x) % pitch)      // b's window starts d
                           : (pitch - static_cast<int64_t>((x - y) % pitch)) % pitch;  // after a's
  return d < a.width || d + b.width > pitch;
}

// Whether no output shares a byte with an input or another output.
bool apart(std::initializer_list<Operand> outs, std::initializer_list<Operand> ins) {
  for (auto a = outs.begin(); a != outs.end(); ++a) {
    for (auto b = a + 1; b != outs.end(); ++b)
      if (share(*a, *b)) return false;
    for (const Operand& b : ins)
      if (share(*a, b)) return false;
  }
  return true;
}

bs_status done(cudaError_t e) {
  if (e == cudaSuccess) return BS_OK;
  bsolve::record_cuda_error(e);
  return BS_ERR_CUDA;
}

// Calls f with a value of the row type.
template <typename F>
cudaError_t with_type(bs_dtype dtype, F&& f) {
  switch (dtype) {
    case BS_FP32: return f(float());
    case BS_BF16: return f(__nv_bfloat16());
    default: return f(__half());
  }
}

}  // namespace
