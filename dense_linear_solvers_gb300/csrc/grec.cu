// Gated linear recurrence (bs_grec calls of bsolve.h): forward over sequences, and one row from kept
// states.
#include <algorithm>
#include <type_traits>

#include "cluster.cuh"
#include "grec_math.cuh"
#include "grec_order.cuh"
#include "grec_tile.cuh"
#include "kernels.h"
#include "row_types.cuh"

namespace bsolve {
namespace {

// ------------------------------------------------------------------ forward
//
// A block takes a tile of 64 channels, a lane two of them, and W * kR consecutive rows at a time,
// a warp kR of them; a cluster of blocks takes consecutive such pieces of one sequence. One step:
//   every warp turns its rows into compositions h_j = A_j h_in + H_j from its first row on (A the
//     product of the a_t, H the state from zero), kept in registers;
//   the warps' last compositions meet in shared memory, the blocks' in every block's shared
//     memory over the cluster, while the copies of a later step are issued; each warp composes
//     those in front of it, in order, with the state at the step's start, which every block
//     carries along;
//   every warp applies its compositions to its own true state, one product-sum an element, and
//     stores the states.
// Each element is read and written once. The order of every sum follows from the sizes alone.
// 65,536 x 4,096 BF16 take 445 us (4.8 TB/s; 256 blocks on 128 of the 152 SMs, whose schedulers issue
// on half of their cycles, 28 instructions an element: between them the 16 warps wait for each
// other and for their own results), 64 x 512 x 2,048 85 us (6.3 TB/s), 4 x 4,096 x 2,048 FP32 83 us (6.5).
constexpr int kStages = 2;  // steps staged ahead

struct Composition {  // of two channels
  float2 A, H;
};

__device__ __forceinline__ float2 apply(const Composition& m, float2 h) { return fma2(m.A, h, m.H); }

// `second` after `first`.
__device__ __forceinline__ Composition compose(const Composition& second, const Composition& first) {
  return {second.A * first.A, apply(second, first.H)};
}

template <typename T, int W, int kR, bool ALIGNED>
struct GrecForwardShared {
  static constexpr int kOperand = kR * Tile<T, ALIGNED>::kRowBytes;  // one warp's rows
  static constexpr int kStage = 3 * kOperand;
  static constexpr int kWarp = kStages * kStage;
  static constexpr int kSegments = 2 * W * 32 * sizeof(Composition);
  // four-warp blocks run without clusters; an SM then holds four of them
  static constexpr int kBlocks = W == 4 ? 0 : 2 * kMaxCluster * 32 * sizeof(Composition);
  static constexpr int kBytes = kSegments + kBlocks + W * kWarp;
};

template <typename T, int W, int kR, bool ALIGNED>
__global__ void __launch_bounds__(32 * W, (sizeof(T) == 2 || kR == 8 ? 16 : 8) / W)
grec_forward_kernel(GrecRows<T> p, const float* __restrict__ lam, float kappa, const float* h0,
                    T* __restrict__ h, int64_t ldh, bool pairs, float* hT,
                    float* __restrict__ tape) {
  using S = GrecForwardShared<T, W, kR, ALIGNED>;
  extern __shared__ __align__(16) char shared[];
  Composition* segments = reinterpret_cast<Composition*>(shared);
  Composition* blocks = reinterpret_cast<Composition*>(shared + S::kSegments);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  char* mine = shared + S::kSegments + S::kBlocks + warp * S::kWarp;
  const int peers = W == 4 ? 1 : cluster_size(), rank = W == 4 ? 0 : cluster_rank();
  const int c0 = static_cast<int>(blockIdx.x) / peers * kTileC;
  const int valid = p.channels - c0 < kTileC ? p.channels - c0 : kTileC;
  const int c = c0 + 2 * lane;
  const bool first = c < p.channels, second = c + 1 < p.channels;
  const float2 rate = make_float2(first ? grec_rate(lam[c], kappa) : 0.f,
                                  second ? grec_rate(lam[c + 1], kappa) : 0.f);
  const bool small = __all_sync(0xFFFFFFFFu, rate.x <= kSmallRate && rate.y <= kSmallRate);
  const unsigned ph = static_cast<unsigned>(ldh * sizeof(T));
  const bool wide = valid == kTileC, whole = pairs && wide;
  const int step_rows = peers * W * kR;
  const int ahead = (rank * W + warp) * kR;  // the warp's first row of a step
  int parity = 0;
  if (peers > 1) cluster_sync();  // every block runs before one writes to another

  for (int64_t y = blockIdx.y; y < p.batch; y += gridDim.y) {
    const int64_t s = p.offsets != nullptr && p.batch <= kSortedBatch
                          ? nth_longest(p.offsets, static_cast<int>(p.batch), static_cast<int>(y),
                                        reinterpret_cast<int64_t*>(shared))
                          : y;
    int64_t start, end;
    sequence_rows(p.offsets, s, p.length, p.rows, &start, &end);
    float2 state = make_float2(0.f, 0.f);
    if (h0) {
      if (first) state.x = h0[s * p.channels + c];
      if (second) state.y = h0[s * p.channels + c + 1];
    }
    const int length = static_cast<int>(end - start);
    unsigned row = static_cast<unsigned>(start) + ahead;  // the warp's first row of this step
    int left = length - ahead;                            // from there to the sequence's end
    // a warp whose rows start at a multiple of 32 puts its state on the tape
    float* tape_at = tape == nullptr || ahead % kTapeRows != 0
                         ? nullptr
                         : tape + (tape_base(start, s) + ahead / kTapeRows) * p.channels + c;

    auto stage = [&](int slot, int k) {  // the rows of the k-th step from this one
      const int n = left - k * step_rows;
      if (n > 0) {
        const bool all = n >= kR && wide;
        const unsigned at = row + k * step_rows;
        char* to = mine + slot * S::kStage;
        stage_tile<T, ALIGNED, kR>(to, p.x, at, p.ldx, c0, n < kR ? n : kR, all, valid);
        stage_tile<T, ALIGNED, kR>(to + S::kOperand, p.r, at, p.ldr, c0, n < kR ? n : kR, all, valid);
        stage_tile<T, ALIGNED, kR>(to + 2 * S::kOperand, p.i, at, p.ldi, c0, n < kR ? n : kR, all,
                                  valid);
      }
      cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < kStages; ++k) stage(k, k);

    int slot = 0;
    for (int done = 0; done < length; done += step_rows, left -= step_rows, row += step_rows) {
      const int n = left < kR ? left : kR;  // may be negative: none
      cp_async_wait_group<kStages - 1>();
      __syncwarp();
      const char* in = mine + slot * S::kStage;
      const Shift lx = shift_of<T, ALIGNED>(p.x, row, p.ldx),
                  lr = shift_of<T, ALIGNED>(p.r, row, p.ldr),
                  li = shift_of<T, ALIGNED>(p.i, row, p.ldi);
      // of row j: the product of a up to it and the state from zero, in the end h_j = A_j h + H_j
      Composition m[kR];
      auto element = [&](int j, auto kind) {
        const float2 x = staged_pair<T, ALIGNED>(in, j, lx);
        const float2 r = staged_pair<T, ALIGNED>(in + S::kOperand, j, lr);
        const float2 i = staged_pair<T, ALIGNED>(in + 2 * S::kOperand, j, li);
        const Gates g =
            grec_gates<decltype(kind)::value>(grec_exp_neg<false>(r), grec_exp_neg<false>(i), rate);
        const float2 u = g.s * g.si * x;
        const Composition own{g.a, u};
        m[j] = j == 0 ? own : compose(own, m[j > 0 ? j - 1 : 0]);
      };
      if (n == kR && small) {  // no branch between the rows: their instructions interleave
#pragma unroll
        for (int j = 0; j < kR; ++j) element(j, std::true_type());
      } else if (n == kR) {
#pragma unroll
        for (int j = 0; j < kR; ++j) element(j, std::false_type());
      } else {
#pragma unroll
        for (int j = 0; j < kR; ++j) {
          if (j < n) {
            element(j, std::false_type());
          } else {  // past the sequence's end a row hands on what it gets
            m[j] = j == 0 ? Composition{both(1.f), both(0.f)} : m[j > 0 ? j - 1 : 0];
          }
        }
      }
      Composition* seg = segments + parity * W * 32 + lane;
      seg[warp * 32] = m[kR - 1];
      __syncthreads();
      // the composition of the block's rows in front of the warp's
      Composition front{both(1.f), both(0.f)};
#pragma unroll
      for (int w = 0; w < W - 1; ++w)
        if (w < warp) front = compose(seg[w * 32], front);
      Composition* blk = blocks + parity * kMaxCluster * 32 + lane;
      if (peers > 1) {
        if (warp == W - 1) {
          const Composition all = compose(m[kR - 1], front);
          for (int q = 0; q < peers; ++q) store_remote(blk + rank * 32, q, all);
          cluster_publish();
        }
        cluster_arrive();
      }
      stage(slot, kStages);
      slot = slot + 1 == kStages ? 0 : slot + 1;

      float2 before = state;  // the state in front of the block's, then of the warp's rows
      if (peers > 1) {
        cluster_wait();
#pragma unroll
        for (int q = 0; q < kMaxCluster; ++q) {
          if (q == peers) break;
          if (q == rank) before = state;
          state = apply(blk[q * 32], state);
        }
      } else {
#pragma unroll
        for (int w = 0; w < W; ++w) state = apply(seg[w * 32], state);
      }
      before = apply(front, before);
      parity ^= 1;

      if (tape_at != nullptr) {
        if (n > 0) {
          if (first) tape_at[0] = before.x;
          if (second) tape_at[1] = before.y;
        }
        tape_at += step_rows / kTapeRows * static_cast<int64_t>(p.channels);
      }
      T* out = h + c + row * ldh;
      auto emit = [&](int j, auto kind) {
        store_pair<T, decltype(kind)::value>(row_at(out, j, ph), apply(m[j], before), pairs, first,
                                             second);
      };
      if (n == kR && whole) {
#pragma unroll
        for (int j = 0; j < kR; ++j) emit(j, std::true_type());
      } else {
#pragma unroll
        for (int j = 0; j < kR; ++j)
          if (j < n) emit(j, std::false_type());
      }
    }
    cp_async_wait_all();
    if (hT && rank == 0 && warp == 0) {
      if (first) hT[s * p.channels + c] = state.x;
      if (second) hT[s * p.channels + c + 1] = state.y;
    }
  }
  if (peers > 1) cluster_sync();  // no block leaves while another may still write to it
}

// ------------------------------------------------------------------ one row
//
// A thread takes two neighbouring channels of the rows that its block walks (every gridDim.y-th), so that
// their rate is worked out once. 256 rows of 4,096 BF16 channels take 6.9 us cold (2.4 TB/s), one row
// of 2,048 4.4, most of it launch and the latency of one load after another. PAIRS: every row of every operand starts on a pair of elements.
constexpr int kStepThreads = 64;

template <typename T, bool PAIRS>
__device__ __forceinline__ float2 load_pair(const T* at, bool second) {
  if constexpr (PAIRS) {
    return to_f32(*reinterpret_cast<const typename Pair<T>::type*>(at));
  } else {
    return make_float2(to_f32(at[0]), second ? to_f32(at[1]) : 0.f);
  }
}

template <typename T, bool PAIRS>
__global__ void __launch_bounds__(kStepThreads)
grec_step_kernel(GrecRows<T> p, const float* __restrict__ lam, float kappa,
                 float* __restrict__ state, int64_t num_slots, const int32_t* __restrict__ slots,
                 T* __restrict__ y, int64_t ldy) {
  const int c = 2 * (blockIdx.x * kStepThreads + threadIdx.x);
  if (c >= p.channels) return;
  const bool second = c + 1 < p.channels;
  const float2 rate = make_float2(grec_rate(lam[c], kappa),
                                  second ? grec_rate(lam[c + 1], kappa) : 0.f);
#pragma unroll 2
  for (int64_t j = blockIdx.y; j < p.batch; j += gridDim.y) {
    const int64_t slot = slots ? slots[j] : j;
    const bool live = slot >= 0 && slot < num_slots;
    const float2 r = load_pair<T, PAIRS>(p.r + j * p.ldr + c, second),
                 i = load_pair<T, PAIRS>(p.i + j * p.ldi + c, second),
                 x = load_pair<T, PAIRS>(p.x + j * p.ldx + c, second);
    float2 h = make_float2(0.f, 0.f);
    if (live) {
      float* at = state + slot * p.channels + c;
      h = load_pair<float, PAIRS>(at, second);
      const Gates g = grec_gates<false>(grec_exp_neg<false>(r), grec_exp_neg<false>(i), rate);
      h = fma2(g.a, h, g.s * g.si * x);
      store_pair<float, PAIRS>(at, h, false, true, second);
    }
    store_pair<T, PAIRS>(y + j * ldy + c, h, false, true, second);
  }
}

template <typename T, int W, int kR, bool ALIGNED>
cudaError_t launch_forward(const GrecRows<T>& p, const float* lam, float kappa, const float* h0,
                           T* h, int64_t ldh, float* hT, float* tape, cudaStream_t stream) {
  using S = GrecForwardShared<T, W, kR, ALIGNED>;
  auto* kernel = grec_forward_kernel<T, W, kR, ALIGNED>;
  static HeldClusters known;
  Held held;
  const cudaError_t e = known.of(kernel, 32 * W, S::kBytes, &held);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (p.channels + kTileC - 1) / kTileC;
  const int64_t length = p.offsets ? p.rows / p.batch + 1 : p.length;
  const int cluster =
      W == 4 ? 1 : grec_cluster(held, tiles, p.batch, length, p.offsets != nullptr, W * kR);
  return launch_clusters(kernel, dim3(static_cast<unsigned>(tiles * cluster),
                                      static_cast<unsigned>(p.batch < 65535 ? p.batch : 65535)),
                         32 * W, S::kBytes, cluster, stream, p, lam, kappa, h0, h, ldh,
                         pair_stores(h, ldh), hT, tape);
}

// Blocks of four warps, without clusters, on 16-bit rows while there is a pair of a sequence and a tile
// for every SM: 64 x 512 rows x 2,048 channels BF16 take 85 us, with eight warps 100; 8 x 4,096 rows
// 103 and 111. Otherwise eight, which meet less often and share a sequence in clusters: one of
// 65,536 x 4,096 takes 445 us, with four warps 1,053; 4 x 4,096 x 2,048 FP32 86 and 90. Packed
// sequences end with their longest, which more warps and clusters shorten (60 of 670 rows on average
// x 1,024: 74 us with eight, 83 with four), until there are so many that it does not show (128 of
// 470: 100 with four, 115).
constexpr int64_t kFourWarpUnits = kSms, kFourWarpUnitsPacked = 10 * kSms;

}  // namespace

template <typename T>
cudaError_t launch_grec(const GrecRows<T>& p, const float* lam, float kappa, const float* h0,
                        T* h, int64_t ldh, float* hT, float* tape, cudaStream_t stream) {
  const bool aligned = rows_aligned(p.x, p.ldx) && rows_aligned(p.r, p.ldr) &&
                       rows_aligned(p.i, p.ldi);
  if constexpr (sizeof(T) == 2) {
    const int64_t units = (p.channels + kTileC - 1) / kTileC * p.batch;
    if (units >= (p.offsets ? kFourWarpUnitsPacked : kFourWarpUnits)) {
      auto* launch = aligned ? launch_forward<T, 4, 16, true> : launch_forward<T, 4, 16, false>;
      return launch(p, lam, kappa, h0, h, ldh, hT, tape, stream);
    }
  }
  // Rows that are not aligned take more shared memory and instructions to stage: eight rows a warp, so that
  // an SM holds two blocks (5 x 777 x 523 FP16 27 to 17 us; aligned rows lose 5 to 25%).
  auto* launch = aligned ? launch_forward<T, 8, 16, true> : launch_forward<T, 8, 8, false>;
  return launch(p, lam, kappa, h0, h, ldh, hT, tape, stream);
}

template <typename T>
cudaError_t launch_grec_step(const GrecRows<T>& p, const float* lam, float kappa, float* state,
                             int64_t num_slots, const int32_t* slots, T* y, int64_t ldy,
                             cudaStream_t stream) {
  const unsigned across = (p.channels + 2 * kStepThreads - 1) / (2 * kStepThreads);
  // 16 blocks an SM; more rows a block beyond that
  const int64_t down = std::max<int64_t>(1, 16 * kSms / across);
  const dim3 grid(across, static_cast<unsigned>(p.batch < down ? p.batch : down));
  const bool pairs = p.channels % 2 == 0 && pair_stores(p.x, p.ldx) && pair_stores(p.r, p.ldr) &&
                     pair_stores(p.i, p.ldi) && pair_stores(y, ldy) &&
                     pair_stores(state, p.channels);
  auto* kernel = pairs ? grec_step_kernel<T, true> : grec_step_kernel<T, false>;
  kernel<<<grid, kStepThreads, 0, stream>>>(p, lam, kappa, state, num_slots, slots, y, ldy);
  return cudaGetLastError();
}

#define BSOLVE_GREC(T)                                                                          \
  template cudaError_t launch_grec<T>(const GrecRows<T>&, const float*, float, const float*,    \
                                      T*, int64_t, float*, float*, cudaStream_t);               \
  template cudaError_t launch_grec_step<T>(const GrecRows<T>&, const float*, float, float*,     \
                                           int64_t, const int32_t*, T*, int64_t, cudaStream_t);
BSOLVE_GREC(float)
BSOLVE_GREC(__nv_bfloat16)
BSOLVE_GREC(__half)
#undef BSOLVE_GREC

}  // namespace bsolve
