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

// Copies `rows` rows of `valid` elements (valid <= 64) into smem; `row0` the first row's first
// element, `pitch` the rows' distance in bytes, `base` the operand's first byte. All lanes of
// the warp take part. Nothing outside the operand is read; what lies behind a row's valid
// elements in shared memory is unspecified.
template <typename T>
__device__ __forceinline__ void stage_rows_unaligned(char* smem, const char* row0, unsigned pitch,
                                                     int rows, int valid, const char* base) {
  using G = Tile<T, false>;
  const int lane = threadIdx.x & 31;
  const int bytes = valid * static_cast<int>(sizeof(T));
  for (int q = lane; q < rows * G::kPieces; q += 32) {
    const int k = q / G::kPieces, piece = q - k * G::kPieces;
    const char* src = row0 + k * static_cast<uint64_t>(pitch);
    const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15);
    const char* from = src - shift + piece * 16;
    const int left = bytes + shift - piece * 16;
    if (left <= 0) continue;
    char* to = smem + k * G::kRowBytes + piece * 16;
    if (from >= base) {
      cp_async_16(to, from, left < 16 ? left : 16);
    } else {  // the boundary lies in front of the operand: its first elements one by one
      for (int b = shift; b < 16 && b < shift + bytes; b += static_cast<int>(sizeof(T)))
        *reinterpret_cast<T*>(to + b) = *reinterpret_cast<const T*>(from + b);
    }
  }
}

// Copies `rows` rows from row `row` of an operand, columns from c0, into smem (whole: R rows of 64
// elements). Addresses are worked out anew each time: a few instructions a step instead of registers
// over all of it.
template <typename T, bool ALIGNED, int R>
__device__ __forceinline__ void stage_tile(char* smem, const T* base, unsigned row, int64_t ld,
                                           int c0, int rows, bool whole, int valid) {
  const unsigned pitch = static_cast<unsigned>(ld) * static_cast<unsigned>(sizeof(T));
  if constexpr (ALIGNED) {
    constexpr int kPieces = Tile<T, true>::kPieces, kPer = 32 / kPieces;  // rows copied at once
    static_assert(R % kPer == 0, "whole copies");
    const int lane = threadIdx.x & 31, piece = lane % kPieces, sub = lane / kPieces;
    char* to = smem + sub * Tile<T, true>::kRowBytes + piece * 16;
    const char* from = reinterpret_cast<const char*>(base + c0) + piece * 16 +
                       static_cast<uint64_t>(row + sub) * pitch;
    if (whole) {
#pragma unroll
      for (int j = 0; j < R; j += kPer)
        cp_async_16(to + j * Tile<T, true>::kRowBytes, from + j * static_cast<uint64_t>(pitch), 16);
    } else {
      const int left = valid * static_cast<int>(sizeof(T)) - piece * 16;
      if (left > 0)
        for (int j = 0; j + sub < rows; j += kPer)
          cp_async_16(to + j * Tile<T, true>::kRowBytes, from + j * static_cast<uint64_t>(pitch),
                      left < 16 ? left : 16);
    }
  } else {
    stage_rows_unaligned<T>(
        smem, reinterpret_cast<const char*>(base + c0) + static_cast<uint64_t>(row) * pitch, pitch,
        rows, valid, reinterpret_cast<const char*>(base));
  }
}

// What staged_pair() needs to know of an operand's rows from row `row` where they are not aligned.
struct Shift {
  unsigned low, pitch;
};
template <typename T, bool ALIGNED>
__device__ __forceinline__ Shift shift_of(const T* base, unsigned row, int64_t ld) {
  if (ALIGNED) return {0, 0};
  const unsigned pitch = static_cast<unsigned>(ld) * static_cast<unsigned>(sizeof(T));
  return {static_cast<unsigned>(reinterpret_cast<uintptr_t>(base)) + row * pitch, pitch};
}

// The lane's two channels of staged row k (a tile's column 0 lies on a multiple of 64 elements, so
// that the shift of a row is that of its operand's row).
template <typename T, bool ALIGNED>
__device__ __forceinline__ float2 staged_pair(const char* smem, int k, Shift at_row) {
  using G = Tile<T, ALIGNED>;
  const int lane = threadIdx.x & 31;
  if constexpr (ALIGNED) {
    return to_f32(*reinterpret_cast<const typename Pair<T>::type*>(
        smem + k * G::kRowBytes + lane * 2 * static_cast<int>(sizeof(T))));
  } else {
    const unsigned shift = (at_row.low + k * at_row.pitch) & 15u;
    const T* at = reinterpret_cast<const T*>(smem + k * G::kRowBytes + shift) + 2 * lane;
    return make_float2(to_f32(at[0]), to_f32(at[1]));
  }
}

}  // namespace bsolve
