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
// is staged in 16-byte pieces. Otherwise FP32 rows are staged element by element, every lane its own
// two; 16-bit rows, whose elements are smaller than any asynchronous copy, in 16-byte pieces from
// the boundary at or below their first element, and read at their own shift (bytes in front of the
// operand's first element are never read).
template <typename T, bool ALIGNED>
struct Tile {
  static constexpr bool kShifted = !ALIGNED && sizeof(T) == 2;
  static constexpr int kRowBytes = kTileC * sizeof(T) + (kShifted ? 16 : 0);
};

// Copies `rows` rows from row `row` of an operand, columns from c0 (`valid` of them are there), into
// smem (whole: R rows of 64 elements). All lanes of the warp take part. Nothing outside the
// operand is read; what lies behind a row's valid elements in shared memory is unspecified.
// Addresses are worked out anew each time: a few instructions a step instead of registers over all
// of it.
template <typename T, bool ALIGNED, int R>
__device__ __forceinline__ void stage_tile(char* smem, const T* base, unsigned row, int64_t ld,
                                           int c0, int rows, bool whole, int valid) {
  using G = Tile<T, ALIGNED>;
  constexpr int kPieces = kTileC * static_cast<int>(sizeof(T)) / 16, kPer = 32 / kPieces;
  static_assert(R % kPer == 0, "whole copies");
  const unsigned pitch = static_cast<unsigned>(ld) * static_cast<unsigned>(sizeof(T));
  const int lane = threadIdx.x & 31;
  const int bytes = valid * static_cast<int>(sizeof(T));
  const char* row0 = reinterpret_cast<const char*>(base + c0) + static_cast<uint64_t>(row) * pitch;
  if constexpr (ALIGNED) {
    const int piece = lane % kPieces, sub = lane / kPieces;  // kPer rows copied at once
    char* to = smem + sub * G::kRowBytes + piece * 16;
    const char* from = row0 + piece * 16 + sub * static_cast<uint64_t>(pitch);
    if (whole) {
#pragma unroll
      for (int j = 0; j < R; j += kPer)
        cp_async_16(to + j * G::kRowBytes, from + j * static_cast<uint64_t>(pitch), 16);
    } else {
      const int left = bytes - piece * 16;
      if (left > 0)
        for (int j = 0; j + sub < rows; j += kPer)
          cp_async_16(to + j * G::kRowBytes, from + j * static_cast<uint64_t>(pitch),
                      left < 16 ? left : 16);
    }
  } else if constexpr (!G::kShifted) {
    char* to = smem + lane * 8;
    const char* from = row0 + lane * 8;
    if (2 * lane < valid) {
      const bool second = 2 * lane + 1 < valid;
#pragma unroll 4
      for (int j = 0; j < rows; ++j) {
        const char* src = from + j * static_cast<uint64_t>(pitch);
        cp_async_elem(reinterpret_cast<float*>(to + j * G::kRowBytes),
                      reinterpret_cast<const float*>(src));
        if (second)
          cp_async_elem(reinterpret_cast<float*>(to + j * G::kRowBytes + 4),
                        reinterpret_cast<const float*>(src + 4));
      }
    }
  } else {
    const int piece = lane % kPieces, sub = lane / kPieces;
#pragma unroll 2
    for (int j = 0; j + sub < rows; j += kPer) {
      const char* src = row0 + (j + sub) * static_cast<uint64_t>(pitch);
      const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15);
      const char* from = src - shift + piece * 16;
      char* to = smem + (j + sub) * G::kRowBytes + piece * 16;
      const int left = bytes + shift - piece * 16;
      // the boundary lies in front of the operand: its first elements one by one
      if (from < reinterpret_cast<const char*>(base)) {
        for (int b = shift; b < 16 && b < shift + bytes; b += 2)
          *reinterpret_cast<T*>(to + b) = *reinterpret_cast<const T*>(from + b);
      } else if (left > 0) {
        cp_async_16(to, from, left < 16 ? left : 16);
      }
      if (piece == 0 && bytes + shift > 16 * kPieces)  // one piece more
        cp_async_16(to + 16 * kPieces, from + 16 * kPieces, bytes + shift - 16 * kPieces);
    }
  }
}

// What staged_pair() needs to know of an operand's rows from row `row` where they are not aligned.
struct Shift {
  unsigned low, pitch;
};
template <typename T, bool ALIGNED>
__device__ __forceinline__ Shift shift_of(const T* base, unsigned row, int64_t ld) {
  if (!Tile<T, ALIGNED>::kShifted) return {0, 0};
  const unsigned pitch = static_cast<unsigned>(ld) * static_cast<unsigned>(sizeof(T));
  return {static_cast<unsigned>(reinterpret_cast<uintptr_t>(base)) + row * pitch, pitch};
}

// The lane's two channels of staged row k (a tile's column 0 lies on a multiple of 64 elements, so
// that the shift of a row is that of its operand's row).
template <typename T, bool ALIGNED>
__device__ __forceinline__ float2 staged_pair(const char* smem, int k, Shift at_row) {
  using G = Tile<T, ALIGNED>;
  const int lane = threadIdx.x & 31;
  if constexpr (!G::kShifted) {
    return to_f32(*reinterpret_cast<const typename Pair<T>::type*>(
        smem + k * G::kRowBytes + lane * 2 * static_cast<int>(sizeof(T))));
  } else {
    const unsigned shift = (at_row.low + k * at_row.pitch) & 15u;
    const T* at = reinterpret_cast<const T*>(smem + k * G::kRowBytes + shift) + 2 * lane;
    return make_float2(to_f32(at[0]), to_f32(at[1]));
  }
}

}  // namespace bsolve
