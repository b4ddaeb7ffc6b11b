// Backward pass of the gated linear recurrence (bs_grec_backward_batched of bsolve.h).
//
// The gradient g_t of the state after row t solves the transposed system,
//   g_t = dh_t + a_{t+1} g_{t+1},
// a scan from the last row to the first; every input's gradient is a product of g_t with factors
// of row t and of the state h_{t-1} before it. The states are not read back (h was rounded when it
// was stored) but solved again in FP32 from the tape, in the same pass over x, r and i that
// the gradients need: four reads and three writes an element.
//
// The mapping is the forward pass's: 64 channels a block, two a lane, eight rows a warp, pieces of
// 64 rows, which start at a state on the tape, so that the states need no exchange between blocks;
// consecutive pieces lie on the blocks of a cluster, which walk the sequence from its end.
// One step:
//   each warp turns its rows into running compositions, A the product of the a_t and H the state from
//     zero, kept in registers, and P = sum of A_t dh_t, the gradient a_t g_t handed on from zero;
//   the warps meet in shared memory, the blocks' (A, P) in every block's over the cluster;
//   each warp walks its rows backward from its true gradient, each with the state that its
//     composition gives from the warp's true one, writing the three gradients.
// The gradient of lam: every lane sums D = dL/dl * l over its rows, the block's warps are added at
// the end and each block writes one partial sum a channel; a second kernel adds those in order.
//
// 8 x 4,096 x 2,048 BF16 take 244 us, 3.9 TB/s of the seven operands; FP32 rows reach 5.5. What bounds
// it is how little the 16 warps that 128 registers leave can overlap: the schedulers issue on half of their
// cycles, 74 instructions an element, of which the gates' second evaluation is a good part; the
// bytes alone would take 140 us. Measured without gain: blocks of four warps (257 us), the
// exponentials of the gates worked out twice instead of kept (284).
#include <type_traits>

#include "cluster.cuh"
#include "grec_math.cuh"
#include "grec_order.cuh"
#include "grec_tile.cuh"
#include "kernels.h"
#include "row_types.cuh"

namespace bsolve {
namespace {

constexpr int W = 8;        // warps of a block
constexpr int kR = 8;       // rows a warp keeps in registers
constexpr int kStages = 2;  // steps staged ahead

struct Exchange {  // of two channels
  float2 A, P;
};
__device__ __forceinline__ float2 apply(const Exchange& m, float2 g) { return fma2(m.A, g, m.P); }
// `second` after `first`, towards the sequence's start.
__device__ __forceinline__ Exchange compose(const Exchange& second, const Exchange& first) {
  return {second.A * first.A, apply(second, first.P)};
}

template <typename T, bool ALIGNED>
struct GrecBackwardShared {
  static constexpr int kOperand = kR * Tile<T, ALIGNED>::kRowBytes;  // one warp's rows
  static constexpr int kStage = 4 * kOperand;
  static constexpr int kWarp = kStages * kStage;
  static constexpr int kSegments = 2 * W * 32 * sizeof(Exchange);
  static constexpr int kStates = 2 * W * 32 * sizeof(float2);
  static constexpr int kBlocks = 2 * kMaxCluster * 32 * sizeof(Exchange);
  static constexpr int kBytes = kSegments + kStates + kBlocks + W * kWarp;
};

template <typename T>
struct GrecGradRows {
  const T* dh;
  T *dx, *dr, *di;
  int64_t lddh, lddx, lddr, lddi;
  bool px, pr, pi;  // pairs of elements stored as one value
};

template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(32 * W, sizeof(T) == 2 ? 2 : 1)
grec_backward_kernel(GrecRows<T> p, GrecGradRows<T> g, const float* __restrict__ lam, float kappa,
                     const float* __restrict__ tape, const float* dhT, float* dh0,
                     float* __restrict__ partial) {
  using S = GrecBackwardShared<T, ALIGNED>;
  constexpr int kPiece = W * kR;  // rows of a block in a step
  static_assert(kPiece % kTapeRows == 0, "a block's piece starts at a state on the tape");
  extern __shared__ __align__(16) char shared[];
  Exchange* segments = reinterpret_cast<Exchange*>(shared);
  Exchange* blocks = reinterpret_cast<Exchange*>(shared + S::kSegments);
  float2* states = reinterpret_cast<float2*>(shared + S::kSegments + S::kBlocks);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  char* mine = shared + S::kSegments + S::kBlocks + S::kStates + warp * S::kWarp;
  const int peers = cluster_size(), rank = cluster_rank();
  const int c0 = static_cast<int>(blockIdx.x) / peers * kTileC;
  const int valid = p.channels - c0 < kTileC ? p.channels - c0 : kTileC;
  const int c = c0 + 2 * lane;
  const bool first = c < p.channels, second = c + 1 < p.channels;
  const float2 rate = make_float2(first ? grec_rate(lam[c], kappa) : 0.f,
                                  second ? grec_rate(lam[c + 1], kappa) : 0.f);
  const bool small = __all_sync(0xFFFFFFFFu, rate.x <= kSmallRate && rate.y <= kSmallRate);
  const unsigned es = sizeof(T);
  const unsigned pdx = g.lddx * es, pdr = g.lddr * es, pdi = g.lddi * es;
  const bool wide = valid == kTileC, whole = g.px && g.pr && g.pi && wide;
  const int step_rows = peers * kPiece;
  float2 dlam = make_float2(0.f, 0.f);
  int parity = 0;
  if (peers > 1) cluster_sync();  // every block runs before one writes to another

  for (int64_t y = blockIdx.y; y < p.batch; y += gridDim.y) {
    const int64_t s = p.offsets != nullptr && p.batch <= kSortedBatch
                          ? nth_longest(p.offsets, static_cast<int>(p.batch), static_cast<int>(y),
                                        reinterpret_cast<int64_t*>(shared))
                          : y;
    int64_t start, end;
    sequence_rows(p.offsets, s, p.length, p.rows, &start, &end);
    float2 carry = make_float2(0.f, 0.f);  // a_{t+1} g_{t+1} at the end of the step's rows
    if (dhT) {
      if (first) carry.x = dhT[s * p.channels + c];
      if (second) carry.y = dhT[s * p.channels + c + 1];
    }
    const int length = static_cast<int>(end - start);
    const int steps = (length + step_rows - 1) / step_rows;
    // the block's first row of this step, counted from the sequence's; the last step first
    int piece = (steps - 1) * step_rows + rank * kPiece;
    unsigned row = static_cast<unsigned>(start) + piece + warp * kR;  // the warp's first
    const float* tape_at = tape + (tape_base(start, s) + piece / kTapeRows) * p.channels + c;

    auto stage = [&](int slot, int k) {  // the rows of the k-th step from this one
      const int ahead = piece + warp * kR - k * step_rows;  // counted from the sequence's first row
      if (ahead >= 0) {
        const int n = length - ahead < kR ? length - ahead : kR;
        const bool all = n == kR && wide;
        const unsigned at = row - k * step_rows;
        char* to = mine + slot * S::kStage;
        stage_tile<T, ALIGNED, kR>(to, p.x, at, p.ldx, c0, n, all, valid);
        stage_tile<T, ALIGNED, kR>(to + S::kOperand, p.r, at, p.ldr, c0, n, all, valid);
        stage_tile<T, ALIGNED, kR>(to + 2 * S::kOperand, p.i, at, p.ldi, c0, n, all, valid);
        stage_tile<T, ALIGNED, kR>(to + 3 * S::kOperand, g.dh, at, g.lddh, c0, n, all, valid);
      }
      cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < kStages; ++k) stage(k, k);

    int slot = 0;
    for (; piece >= 0; piece -= step_rows, row -= step_rows) {
      const int left = length - piece - warp * kR;
      const int n = left < kR ? left : kR;    // may be negative: none
      float2 before = make_float2(0.f, 0.f);  // the state in front of the block's rows
      if (piece < length) {
        if (first) before.x = tape_at[0];
        if (second) before.y = tape_at[1];
      }
      tape_at -= step_rows / kTapeRows * static_cast<int64_t>(p.channels);
      cp_async_wait_group<kStages - 1>();
      __syncwarp();
      const char* in = mine + slot * S::kStage;
      const Shift lx = shift_of<T, ALIGNED>(p.x, row, p.ldx),
                  lr = shift_of<T, ALIGNED>(p.r, row, p.ldr),
                  li = shift_of<T, ALIGNED>(p.i, row, p.ldi),
                  lh = shift_of<T, ALIGNED>(g.dh, row, g.lddh);
      auto read = [&](int operand, int j, Shift at) {
        return staged_pair<T, ALIGNED>(in + operand * S::kOperand, j, at);
      };

      // of row j: e^-r, e^-i; from the warp's first row to it the product of a and the state from zero
      float2 er[kR], ei[kR], A[kR] = {}, H[kR] = {};
      Exchange m{both(1.f), both(0.f)};
      auto element = [&](int j, auto kind) {
        er[j] = grec_exp_neg<true>(read(1, j, lr));
        ei[j] = grec_exp_neg<true>(read(2, j, li));
        const Gates q = grec_gates<decltype(kind)::value>(er[j], ei[j], rate);
        const float2 u = q.s * q.si * read(0, j, lx);
        A[j] = j == 0 ? q.a : q.a * A[j > 0 ? j - 1 : 0];
        H[j] = j == 0 ? u : fma2(q.a, H[j > 0 ? j - 1 : 0], u);
        m.P = fma2(A[j], read(3, j, lh), m.P);
      };
      if (n == kR) {
        if (small) {
#pragma unroll
          for (int j = 0; j < kR; ++j) element(j, std::true_type());
        } else {
#pragma unroll
          for (int j = 0; j < kR; ++j) element(j, std::false_type());
        }
      } else {
#pragma unroll
        for (int j = 0; j < kR; ++j) {
          if (j < n) {
            element(j, std::false_type());
          } else {  // past the sequence's end a row hands on what it gets
            A[j] = j == 0 ? both(1.f) : A[j > 0 ? j - 1 : 0];
            H[j] = j == 0 ? both(0.f) : H[j > 0 ? j - 1 : 0];
          }
        }
      }
      m.A = A[kR - 1];

      Exchange* seg = segments + parity * W * 32 + lane;
      float2* st = states + parity * W * 32 + lane;
      seg[warp * 32] = m;
      st[warp * 32] = H[kR - 1];
      __syncthreads();
      Exchange behind{both(1.f), both(0.f)};  // the block's rows behind the warp's
#pragma unroll
      for (int w = W - 1; w > 0; --w)
        if (w > warp) behind = compose(seg[w * 32], behind);
      Exchange* blk = blocks + parity * kMaxCluster * 32 + lane;
      if (peers > 1) {
        if (warp == 0) {
          const Exchange all = compose(m, behind);
          for (int q = 0; q < peers; ++q) store_remote(blk + rank * 32, q, all);
          cluster_publish();
        }
        cluster_arrive();
      }
#pragma unroll
      for (int w = 0; w < W - 1; ++w)
        if (w < warp) before = fma2(seg[w * 32].A, before, st[w * 32]);
      float2 after = carry;  // what comes from behind the block's, then the warp's rows
      if (peers > 1) {
        cluster_wait();
#pragma unroll
        for (int q = kMaxCluster - 1; q >= 0; --q) {
          if (q >= peers) continue;
          if (q == rank) after = carry;
          carry = apply(blk[q * 32], carry);
        }
      } else {
#pragma unroll
        for (int w = W - 1; w >= 0; --w) carry = apply(seg[w * 32], carry);
      }
      after = apply(behind, after);
      parity ^= 1;

      T* dx = g.dx + c + row * g.lddx;
      T* dr = g.dr + c + row * g.lddr;
      T* di = g.di + c + row * g.lddi;
      auto emit = [&](int j, auto kind, auto all) {
        constexpr bool kWhole = decltype(all)::value;
        const float2 x = read(0, j, lx);
        const float2 gt = read(3, j, lh) + after;
        // the gates again from their exponentials: fewer registers than keeping them all
        const Gates q = grec_gates<decltype(kind)::value>(er[j], ei[j], rate);
        after = q.a * gt;
        const float2 y = q.si * x, gs = gt * q.s;
        // the state before the row, and D = g a t (sigma(i) x a / s - h)
        const float2 h = j == 0 ? before : fma2(A[j > 0 ? j - 1 : 0], before, H[j > 0 ? j - 1 : 0]);
        const float2 d = after * q.t * fma2(y * q.a, q.rs, h * both(-1.f));
        dlam = dlam + d;
        store_pair<T, kWhole>(row_at(dx, j, pdx), gs * q.si, g.px, first, second);
        store_pair<T, kWhole>(row_at(di, j, pdi), gs * y * (ei[j] * q.si), g.pi, first, second);
        store_pair<T, kWhole>(row_at(dr, j, pdr), d * (er[j] * q.sr), g.pr, first, second);
      };
      if (n == kR) {
        if (small && whole) {
#pragma unroll
          for (int j = kR - 1; j >= 0; --j) emit(j, std::true_type(), std::true_type());
        } else if (!ALIGNED && small) {
#pragma unroll
          for (int j = kR - 1; j >= 0; --j) emit(j, std::true_type(), std::false_type());
        } else if (whole) {
#pragma unroll
          for (int j = kR - 1; j >= 0; --j) emit(j, std::false_type(), std::true_type());
        } else {
#pragma unroll
          for (int j = kR - 1; j >= 0; --j) emit(j, std::false_type(), std::false_type());
        }
      } else {
#pragma unroll
        for (int j = kR - 1; j >= 0; --j)
          if (j < n) emit(j, std::false_type(), std::false_type());
      }
      __syncwarp();
      stage(slot, kStages);
      slot = slot + 1 == kStages ? 0 : slot + 1;
    }
    cp_async_wait_all();
    if (dh0 && rank == 0 && warp == 0) {
      if (first) dh0[s * p.channels + c] = carry.x;
      if (second) dh0[s * p.channels + c + 1] = carry.y;
    }
  }

  // the block's sum of D a channel, warps in order
  float2* sums = reinterpret_cast<float2*>(mine - warp * S::kWarp);
  __syncthreads();
  sums[warp * 32 + lane] = dlam;
  __syncthreads();
  if (warp == 0) {
    float2 sum = sums[lane];
#pragma unroll
    for (int w = 1; w < W; ++w) sum = sum + sums[w * 32 + lane];
    float* at = partial + (static_cast<int64_t>(blockIdx.y) * peers + rank) * p.channels + c;
    if (first) at[0] = sum.x;
    if (second) at[1] = sum.y;
  }
  if (peers > 1) cluster_sync();  // no block leaves while another may still write to it
}

// dlam[c] = slope(lam_c) * the sum of the blocks' parts: 32 channels a block, each of its 16
// warps every sixteenth part in order, then the warps' sums in order.
constexpr int kSumWarps = 16;

__global__ void __launch_bounds__(32 * kSumWarps)
grec_dlam_kernel(int channels, int64_t parts, const float* __restrict__ lam,
                 const float* __restrict__ partial, float* __restrict__ dlam) {
  __shared__ float sums[kSumWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x * 32 + lane;
  float sum = 0.f;
  if (c < channels) {
#pragma unroll 8
    for (int64_t k = warp; k < parts; k += kSumWarps) sum += partial[k * channels + c];
  }
  sums[warp][lane] = sum;
  __syncthreads();
  if (warp != 0 || c >= channels) return;
  sum = 0.f;
  for (int w = 0; w < kSumWarps; ++w) sum += sums[w][lane];
  dlam[c] = sum * grec_rate_slope(lam[c]);
}

int64_t tiles_of(int channels) { return (channels + kTileC - 1) / kTileC; }
int64_t grid_y(int64_t batch) { return batch < 65535 ? batch : 65535; }

template <typename T, bool ALIGNED>
cudaError_t launch_backward(const GrecRows<T>& p, const GrecGradRows<T>& g, const float* lam,
                            float kappa, const float* tape, const float* dhT, float* dh0,
                            float* partial, int64_t* parts, cudaStream_t stream) {
  using S = GrecBackwardShared<T, ALIGNED>;
  auto* kernel = grec_backward_kernel<T, ALIGNED>;
  static HeldClusters known;
  Held held;
  const cudaError_t e = known.of(kernel, 32 * W, S::kBytes, &held);
  if (e != cudaSuccess) return e;
  const int64_t length = p.offsets ? p.rows / p.batch + 1 : p.length;
  const int cluster = grec_cluster(held, tiles_of(p.channels), p.batch, length,
                                   p.offsets != nullptr, W * kR);
  *parts = grid_y(p.batch) * cluster;
  return launch_clusters(kernel,
                         dim3(static_cast<unsigned>(tiles_of(p.channels) * cluster),
                              static_cast<unsigned>(grid_y(p.batch))),
                         32 * W, S::kBytes, cluster, stream, p, g, lam, kappa, tape, dhT, dh0,
                         partial);
}

}  // namespace

size_t grec_backward_workspace(int channels, int64_t batch, int64_t) {
  if (batch == 0) return 0;
  const bool many = tiles_of(channels) * batch > kManyUnits;
  const int64_t parts = grid_y(batch) * (many ? 1 : kMaxCluster);
  return static_cast<size_t>(parts) * channels * sizeof(float);
}

template <typename T>
cudaError_t launch_grec_backward(const GrecRows<T>& p, const float* lam, float kappa,
                                 const float* tape, const T* dh, int64_t lddh, const float* dhT,
                                 T* dx, int64_t lddx, T* dr, int64_t lddr, T* di, int64_t lddi,
                                 float* dlam, float* dh0, void* work, cudaStream_t stream) {
  float* partial = static_cast<float*>(work);
  int64_t parts = 0;
  if (p.batch > 0) {
    const GrecGradRows<T> g{dh, dx, dr, di, lddh, lddx, lddr, lddi,
                            pair_stores(dx, lddx), pair_stores(dr, lddr), pair_stores(di, lddi)};
    const bool aligned = rows_aligned(p.x, p.ldx) && rows_aligned(p.r, p.ldr) &&
                         rows_aligned(p.i, p.ldi) && rows_aligned(dh, lddh);
    auto* launch = aligned ? launch_backward<T, true> : launch_backward<T, false>;
    const cudaError_t e = launch(p, g, lam, kappa, tape, dhT, dh0, partial, &parts, stream);
    if (e != cudaSuccess) return e;
  }
  grec_dlam_kernel<<<(p.channels + 31) / 32, 32 * kSumWarps, 0, stream>>>(p.channels, parts, lam,
                                                                         partial, dlam);
  return cudaGetLastError();
}

#define BSOLVE_GREC_BACKWARD(T)                                                                 \
  template cudaError_t launch_grec_backward<T>(                                                 \
      const GrecRows<T>&, const float*, float, const float*, const T*, int64_t, const float*,   \
      T*, int64_t, T*, int64_t, T*, int64_t, float*, float*, void*, cudaStream_t);
BSOLVE_GREC_BACKWARD(float)
BSOLVE_GREC_BACKWARD(__nv_bfloat16)
BSOLVE_GREC_BACKWARD(__half)
#undef BSOLVE_GREC_BACKWARD

}  // namespace bsolve
