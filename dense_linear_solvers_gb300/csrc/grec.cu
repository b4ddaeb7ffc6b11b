// Gated linear recurrence (bs_grec calls of bsolve.h): forward over sequences, and one row from kept
// states.
#include <type_traits>

#include "cluster.cuh"
#include "grec_math.cuh"
#include "grec_tile.cuh"
#include "kernels.h"
#include "row_types.cuh"

namespace bsolve {
namespace {

// ------------------------------------------------------------------ forward
//
// A block takes a tile of 64 channels, a lane two of them, and 8 * R consecutive rows at a time,
// a warp R of them; a cluster of blocks takes consecutive such pieces of one sequence. One step:
//   every warp turns its rows into (a_t, u_t), kept in registers, and their composition
//     h_out = A h_in + H (A the product of the a_t, H the state from zero);
//   the warps' compositions meet in shared memory, the blocks' in every block's shared memory
//     over the cluster; each warp composes those in front of it, in order, with the state
//     at the step's start, which every block carries along;
//   every warp runs its rows again from its own true state, one product-sum an element, and
//     stores them.
// Each element is read and written once. The order of every sum follows from the sizes alone.
constexpr int kWarps = 8;

struct Composition {  // of two channels
  float2 A, H;
};

__device__ __forceinline__ float2 apply(const Composition& m, float2 h) { return fma2(m.A, h, m.H); }

// `second` after `first`.
__device__ __forceinline__ Composition compose(const Composition& second, const Composition& first) {
  return {second.A * first.A, apply(second, first.H)};
}

template <typename T, int R, bool ALIGNED, int STAGES>
struct GrecForwardShared {
  static constexpr int kOperand = R * Tile<T, ALIGNED>::kRowBytes;  // one warp's rows
  static constexpr int kStage = 3 * kOperand;
  static constexpr int kWarp = STAGES * kStage;
  static constexpr int kSegments = 2 * kWarps * 32 * sizeof(Composition);
  static constexpr int kBlocks = 2 * kMaxCluster * 32 * sizeof(Composition);
  static constexpr int kBytes = kSegments + kBlocks + kWarps * kWarp;
};

template <typename T, int R, bool ALIGNED, int STAGES>
__global__ void __launch_bounds__(32 * kWarps, sizeof(T) == 2 ? 2 : 1)
grec_forward_kernel(GrecRows<T> p, const float* __restrict__ lam, float kappa, const float* h0,
                    T* __restrict__ h, int64_t ldh, bool pairs, float* hT,
                    float* __restrict__ tape) {
  using S = GrecForwardShared<T, R, ALIGNED, STAGES>;
  extern __shared__ __align__(16) char shared[];
  Composition* segments = reinterpret_cast<Composition*>(shared);
  Composition* blocks = reinterpret_cast<Composition*>(shared + S::kSegments);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  char* mine = shared + S::kSegments + S::kBlocks + warp * S::kWarp;
  const int peers = cluster_size(), rank = cluster_rank();
  const int c0 = static_cast<int>(blockIdx.x) / peers * kTileC;
  const int valid = p.channels - c0 < kTileC ? p.channels - c0 : kTileC;
  const int c = c0 + 2 * lane;
  const bool first = c < p.channels, second = c + 1 < p.channels;
  const float2 rate = make_float2(first ? grec_rate(lam[c], kappa) : 0.f,
                                  second ? grec_rate(lam[c + 1], kappa) : 0.f);
  const bool small = __all_sync(0xFFFFFFFFu, rate.x <= kSmallRate && rate.y <= kSmallRate);
  const unsigned px = static_cast<unsigned>(p.ldx * sizeof(T)),
                 pr = static_cast<unsigned>(p.ldr * sizeof(T)),
                 pi = static_cast<unsigned>(p.ldi * sizeof(T)),
                 ph = static_cast<unsigned>(ldh * sizeof(T));
  const bool whole = pairs && valid == kTileC;
  const int step_rows = peers * kWarps * R;
  int parity = 0;
  if (peers > 1) cluster_sync();  // every block runs before one writes to another

  for (int64_t s = blockIdx.y; s < p.batch; s += gridDim.y) {
    int64_t start, end;
    sequence_rows(p.offsets, s, p.length, p.rows, &start, &end);
    float2 state = make_float2(0.f, 0.f);
    if (h0) {
      if (first) state.x = h0[s * p.channels + c];
      if (second) state.y = h0[s * p.channels + c + 1];
    }
    const int64_t tb = tape_base(start, s);
    const int64_t steps = (end - start + step_rows - 1) / step_rows;
    int64_t row = start + (rank * kWarps + warp) * R;  // the warp's first row of this step

    auto stage = [&](int64_t at, int slot) {
      const int n = at >= end ? 0 : (end - at < R ? static_cast<int>(end - at) : R);
      char* to = mine + slot * S::kStage;
      if (n > 0) {
        stage_rows<T, ALIGNED, R>(to, p.x + at * p.ldx + c0, px, n, valid, p.x);
        stage_rows<T, ALIGNED, R>(to + S::kOperand, p.r + at * p.ldr + c0, pr, n, valid, p.r);
        stage_rows<T, ALIGNED, R>(to + 2 * S::kOperand, p.i + at * p.ldi + c0, pi, n, valid, p.i);
      }
      cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < STAGES; ++k) stage(row + static_cast<int64_t>(k) * step_rows, k);

    int slot = 0;
    for (int64_t step = 0; step < steps; ++step, row += step_rows) {
      const int n = row >= end ? 0 : (end - row < R ? static_cast<int>(end - row) : R);
      cp_async_wait_group<STAGES - 1>();
      __syncwarp();
      const char* in = mine + slot * S::kStage;
      const unsigned lx = low_bits(p.x + row * p.ldx), lr = low_bits(p.r + row * p.ldr),
                     li = low_bits(p.i + row * p.ldi);
      float2 a[R], u[R];
      Composition m{both(1.f), both(0.f)};
      auto element = [&](int j, auto kind) {
        const float2 x = staged_pair<T, ALIGNED>(in, j, lx, px);
        const float2 r =
            staged_pair<T, ALIGNED>(in + S::kOperand, j, lr, pr);
        const float2 i =
            staged_pair<T, ALIGNED>(in + 2 * S::kOperand, j, li, pi);
        const Gates g =
            grec_gates<decltype(kind)::value>(grec_exp_neg<false>(r), grec_exp_neg<false>(i), rate);
        a[j] = g.a;
        u[j] = g.s * g.si * x;
        m.A = m.A * a[j];
        m.H = fma2(a[j], m.H, u[j]);
      };
      if (n == R && small) {  // no branch between the rows: their instructions interleave
#pragma unroll
        for (int j = 0; j < R; ++j) element(j, std::true_type());
      } else if (n == R) {
#pragma unroll
        for (int j = 0; j < R; ++j) element(j, std::false_type());
      } else {
#pragma unroll
        for (int j = 0; j < R; ++j)
          if (j < n) element(j, std::false_type());
      }
      __syncwarp();
      stage(row + static_cast<int64_t>(STAGES) * step_rows, slot);
      slot = slot + 1 == STAGES ? 0 : slot + 1;

      // the composition of the block's rows in front of the warp's
      Composition* seg = segments + parity * kWarps * 32;
      seg[warp * 32 + lane] = m;
      __syncthreads();
      Composition front{both(1.f), both(0.f)};
#pragma unroll
      for (int w = 0; w < kWarps - 1; ++w)
        if (w < warp) front = compose(seg[w * 32 + lane], front);
      float2 before = state;  // the state in front of the block's, then of the warp's rows
      if (peers > 1) {
        Composition* blk = blocks + parity * kMaxCluster * 32;
        if (warp == kWarps - 1) {
          const Composition all = compose(m, front);
          for (int q = 0; q < peers; ++q) store_remote(blk + rank * 32 + lane, q, all);
          cluster_publish();
        }
        cluster_sync();
        for (int q = 0; q < peers; ++q) {
          if (q == rank) before = state;
          state = apply(blk[q * 32 + lane], state);
        }
      } else {
#pragma unroll
        for (int w = 0; w < kWarps; ++w) state = apply(seg[w * 32 + lane], state);
      }
      before = apply(front, before);
      parity ^= 1;

      if (tape && n > 0 && (row - start) % kTapeRows == 0) {
        float* at = tape + (tb + (row - start) / kTapeRows) * p.channels + c;
        if (first) at[0] = before.x;
        if (second) at[1] = before.y;
      }
      T* out = h + row * ldh + c;
      auto emit = [&](int j, auto kind) {
        before = fma2(a[j], before, u[j]);
        store_pair<T, decltype(kind)::value>(row_at(out, j, ph), before, pairs, first, second);
      };
      if (n == R && whole) {
#pragma unroll
        for (int j = 0; j < R; ++j) emit(j, std::true_type());
      } else {
#pragma unroll
        for (int j = 0; j < R; ++j)
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

template <typename T>
__global__ void __launch_bounds__(128)
grec_step_kernel(GrecRows<T> p, const float* __restrict__ lam, float kappa,
                 float* __restrict__ state, int64_t num_slots, const int32_t* __restrict__ slots,
                 T* __restrict__ y, int64_t ldy) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= p.channels) return;
  const float rate = grec_rate(lam[c], kappa);
  for (int64_t j = blockIdx.y; j < p.batch; j += gridDim.y) {
    const int64_t slot = slots ? slots[j] : j;
    float h = 0.f;
    if (slot >= 0 && slot < num_slots) {
      const Gates g = grec_gates<false>(grec_exp_neg<false>(both(to_f32(p.r[j * p.ldr + c]))),
                                        grec_exp_neg<false>(both(to_f32(p.i[j * p.ldi + c]))),
                                        both(rate));
      float* at = state + slot * p.channels + c;
      h = fmaf(g.a.x, *at, g.s.x * g.si.x * to_f32(p.x[j * p.ldx + c]));
      *at = h;
    }
    y[j * ldy + c] = from_f32<T>(h);
  }
}

dim3 grid_of(int channels, int64_t batch) {
  return dim3((channels + 127) / 128, static_cast<unsigned>(batch < 65535 ? batch : 65535));
}

}  // namespace

namespace {

template <typename T, int R, bool ALIGNED, int STAGES>
cudaError_t launch_forward(const GrecRows<T>& p, const float* lam, float kappa, const float* h0,
                           T* h, int64_t ldh, float* hT, float* tape, cudaStream_t stream) {
  using S = GrecForwardShared<T, R, ALIGNED, STAGES>;
  auto* kernel = grec_forward_kernel<T, R, ALIGNED, STAGES>;
  const int64_t tiles = (p.channels + kTileC - 1) / kTileC;
  const int64_t length = p.offsets ? p.rows / p.batch + 1 : p.length;
  const int cluster = grec_cluster(tiles * p.batch, length, kWarps * R);
  return launch_clusters(kernel, dim3(static_cast<unsigned>(tiles * cluster),
                                      static_cast<unsigned>(p.batch < 65535 ? p.batch : 65535)),
                         32 * kWarps, S::kBytes, cluster, stream, p, lam, kappa, h0, h, ldh,
                         pair_stores(h, ldh), hT, tape);
}

}  // namespace

template <typename T>
cudaError_t launch_grec(const GrecRows<T>& p, const float* lam, float kappa, const float* h0,
                        T* h, int64_t ldh, float* hT, float* tape, cudaStream_t stream) {
  const bool aligned = rows_aligned(p.x, p.ldx) && rows_aligned(p.r, p.ldr) &&
                       rows_aligned(p.i, p.ldi);
  return aligned ? launch_forward<T, 16, true, 2>(p, lam, kappa, h0, h, ldh, hT, tape, stream)
                 : launch_forward<T, 16, false, 2>(p, lam, kappa, h0, h, ldh, hT, tape, stream);
}

template <typename T>
cudaError_t launch_grec_step(const GrecRows<T>& p, const float* lam, float kappa, float* state,
                             int64_t num_slots, const int32_t* slots, T* y, int64_t ldy,
                             cudaStream_t stream) {
  grec_step_kernel<T><<<grid_of(p.channels, p.batch), 128, 0, stream>>>(p, lam, kappa, state,
                                                                       num_slots, slots, y, ldy);
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
