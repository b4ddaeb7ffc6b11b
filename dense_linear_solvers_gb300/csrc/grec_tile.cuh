// Staging of row tiles for the recurrence kernels (bs_grec calls): every warp copies the rows that
// it will itself read, 64 channels wide, into its own part of shared memory with cp.async, so
// that a copy needs no barrier but the warp's own.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "common.cuh"
#include "row_types.cuh"

namespace bsolve {

constexpr int kTileC = 64;   // channels of a tile: two a lane

// One row operand as the kernels see it. ALIGNED: 16-byte base and row distance; a row of a tile
// is then staged as it lies. Otherwise every row is staged from the 16-byte boundary at or
// below its first element, and read at its own shift (the boundary's bytes in front of the
// operand's first element are never read).
template <typename T, bool ALIGNED>
struct Tile {
  static constexpr int kRowBytes = kTileC * sizeof(T) + (ALIGNED ? 0 : 16);
  static constexpr int kPieces = kRowBytes / 16;
};

__device__ __forceinline__ void cp_async_16(void* smem, const void* gmem, int bytes) {
  const unsigned d = static_cast<unsigned>(__cvta_generic_to_shared(smem));
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(d), "l"(gmem), "r"(bytes)
               : "memory");
}

// Copies `rows` rows of `valid` elements (valid <= 64) into smem; `first` the first row's first
// element, `pitch` the rows' distance in bytes, `base` the operand's first byte. All lanes of
// the warp take part. Nothing outside the operand is read; what lies behind a row's valid
// elements in shared memory is unspecified.
template <typename T, bool ALIGNED, int R>
__device__ __forceinline__ void stage_rows(char* smem, const T* first, unsigned pitch, int rows,
                                           int valid, const T* base) {
  using G = Tile<T, ALIGNED>;
  const int lane = threadIdx.x & 31;
  const char* row0 = reinterpret_cast<const char*>(first);
  const int bytes = valid * static_cast<int>(sizeof(T));
  if constexpr (ALIGNED) {
    constexpr int kPer = 32 / G::kPieces;  // rows the warp copies at once
    static_assert(R % kPer == 0, "whole copies");
    const int piece = lane % G::kPieces, sub = lane / G::kPieces;
    const int left = bytes - piece * 16;
    const char* src = row0 + sub * static_cast<uint64_t>(pitch) + piece * 16;
    char* to = smem + sub * G::kRowBytes + piece * 16;
    if (rows == R && valid == kTileC) {
#pragma unroll
      for (int j = 0; j < R; j += kPer)
        cp_async_16(to + j * G::kRowBytes, src + j * static_cast<uint64_t>(pitch), 16);
    } else if (left > 0) {
      for (int j = 0; j + sub < rows; j += kPer)
        cp_async_16(to + j * G::kRowBytes, src + j * static_cast<uint64_t>(pitch),
                    left < 16 ? left : 16);
    }
  } else {
    for (int q = lane; q < rows * G::kPieces; q += 32) {
      const int k = q / G::kPieces, piece = q - k * G::kPieces;
      const char* src = row0 + k * static_cast<uint64_t>(pitch);
      const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15);
      const char* from = src - shift + piece * 16;
      const int left = bytes + shift - piece * 16;
      if (left <= 0) continue;
      char* to = smem + k * G::kRowBytes + piece * 16;
      if (from >= reinterpret_cast<const char*>(base)) {
        cp_async_16(to, from, left < 16 ? left : 16);
      } else {  // the boundary lies in front of the operand: its first elements one by one
        for (int b = shift; b < 16 && b < shift + bytes; b += static_cast<int>(sizeof(T)))
          *reinterpret_cast<T*>(to + b) = *reinterpret_cast<const T*>(from + b);
      }
    }
  }
}

// The lane's two channels of staged row k; `low` the low address bits of the first row.
template <typename T, bool ALIGNED>
__device__ __forceinline__ float2 staged_pair(const char* smem, int k, unsigned low,
                                              unsigned pitch) {
  using G = Tile<T, ALIGNED>;
  const int lane = threadIdx.x & 31;
  if constexpr (ALIGNED) {
    return to_f32(*reinterpret_cast<const typename Pair<T>::type*>(
        smem + k * G::kRowBytes + lane * 2 * static_cast<int>(sizeof(T))));
  } else {
    const unsigned shift = (low + k * pitch) & 15u;
    const T* at = reinterpret_cast<const T*>(smem + k * G::kRowBytes + shift) + 2 * lane;
    return make_float2(to_f32(at[0]), to_f32(at[1]));
  }
}

}  // namespace bsolve
