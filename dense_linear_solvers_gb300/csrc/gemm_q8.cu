// Matrix product of 8-bit operands under block scales (bs_gemm_q8):
//   y[t][f] = sum over blocks b of 128 of  sa[t][b] sw[f / 128][b] sum over k in b of a[t][k] w[f][k].
//
// For few tokens tcgen05.mma (e4m3, FP32 sums in tensor memory) takes the features as its 128 rows and TOKENS tokens as
// its columns: a tile's 128 features share one weight scale a block, one token costs 16 columns at
// least instead of 128 rows, and a lane of the result is a feature, so that a warp's stores of one token are
// contiguous. Each block of 128 is a result of its own (four instructions of depth 32), which eight warps
// read back, multiply by its two scales and add up in FP32 registers while the next ones are computed
// into other columns of tensor memory. One thread keeps TMA copies of both operands several blocks ahead, one
// issues the products. Persistent blocks, one an SM; where tiles are fewer than SMs, clusters of 2 to
// 8 blocks share a tile's blocks of k and add their parts through distributed shared memory in order.
//
// Every wait is limited (kPatience); a block whose wait ran out stores NaN.
#include <algorithm>
#include <atomic>

#include <cuda.h>

#include "barrier.cuh"
#include "cluster.cuh"
#include "common.cuh"
#include "grec_math.cuh"
#include "kernels.h"
#include "row_types.cuh"

namespace bsolve {
namespace {

constexpr int kBlock = 128;       // elements under one scale, features of a tile
constexpr int kSumWarps = 8;      // warps that scale and add
constexpr int kThreads = (kSumWarps + 2) * 32;
constexpr int kMaxSplit = 8;

template <int TOKENS>
struct Config {
  static constexpr int kStage = (kBlock + TOKENS) * kBlock;  // bytes of both operands' block
  static constexpr int kStages = TOKENS == 128 ? 6 : 8;
  static constexpr int kResults = 4;                         // results in tensor memory
  static constexpr int kColumns = TOKENS * kResults < 32 ? 32 : TOKENS * kResults;
  static constexpr int kOwn = TOKENS / 2;                    // columns of a summing thread
  static constexpr int kPiece = kOwn < 32 ? kOwn : 32;       // columns read at once
  static constexpr int kShared = kStages * kStage + 1024;    // the stages start on 1024 bytes
};

struct Problem {
  int64_t m, n, k;
  const float *sa, *sw;
  int64_t ldsa, ldsw, ldy;
};

// ---------------------------------------------------------------------------- copies
__device__ __forceinline__ void copy_tile(void* to, const CUtensorMap* map, int x, int y, uint64_t* b) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%2, %3}], [%4];" ::"r"(smem_address(to)),
      "l"(map), "r"(x), "r"(y), "r"(smem_address(b))
      : "memory");
}

// ---------------------------------------------------------------------------- tensor memory
// A tile of rows of 128 bytes in shared memory as TMA's 128-byte swizzle leaves it: eight rows (1024 bytes)
// a group.
__device__ __forceinline__ uint64_t operand_at(unsigned at) {
  return static_cast<uint64_t>((at & 0x3FFFF) >> 4) | uint64_t(1) << 16 | uint64_t(1024 >> 4) << 32 |
         uint64_t(1) << 46 | uint64_t(2) << 61;
}
// e4m3 by e4m3 into FP32, both along k, 128 rows, so many columns.
__host__ __device__ constexpr unsigned instruction(int columns) {
  return 1u << 4 | static_cast<unsigned>(columns >> 3) << 17 | static_cast<unsigned>(kBlock >> 4) << 24;
}
__device__ __forceinline__ void product(unsigned result, uint64_t a, uint64_t b, unsigned kind,
                                        bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(result),
      "l"(a), "l"(b), "r"(kind), "r"(static_cast<unsigned>(add))
      : "memory");
}
__device__ __forceinline__ void commit(uint64_t* b) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   smem_address(b)) : "memory");
}
template <int N>
__device__ __forceinline__ void read_columns(unsigned at, float (&v)[N]);
template <>
__device__ __forceinline__ void read_columns<8>(unsigned at, float (&v)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
                 "=f"(v[7]) : "r"(at));
}
template <>
__device__ __forceinline__ void read_columns<16>(unsigned at, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, "
      "[%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]),
        "=f"(v[15]) : "r"(at));
}
template <>
__device__ __forceinline__ void read_columns<32>(unsigned at, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]),
        "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]),
        "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]),
        "=f"(v[29]), "=f"(v[30]), "=f"(v[31]) : "r"(at));
}

// ---------------------------------------------------------------------------- kernel
template <typename T, int TOKENS>
__global__ void __launch_bounds__(kThreads, 1)
gemm_q8_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a,
               Problem p, T* __restrict__ y) {
  using C = Config<TOKENS>;
  extern __shared__ unsigned char raw[];
  __shared__ __align__(16) float factors[2][TOKENS];
  __shared__ uint64_t full[C::kStages], empty[C::kStages], ready[C::kResults], taken[C::kResults];
  __shared__ unsigned columns;
  __shared__ volatile int failed;
  unsigned char* stages = raw + (1024 - (smem_address(raw) & 1023)) % 1024;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int split = cluster_size(), rank = cluster_rank();
  const int features = static_cast<int>((p.n + kBlock - 1) / kBlock);
  const int64_t tiles = features * ((p.m + TOKENS - 1) / TOKENS);
  const int blocks = static_cast<int>((p.k + kBlock - 1) / kBlock);
  const int first = static_cast<int>(int64_t(blocks) * rank / split),
            last = static_cast<int>(int64_t(blocks) * (rank + 1) / split);

  if (threadIdx.x == 0) {
    failed = 0;
    for (int s = 0; s < C::kStages; ++s) barrier_init(&full[s], 1), barrier_init(&empty[s], 1);
    for (int r = 0; r < C::kResults; ++r) barrier_init(&ready[r], 1), barrier_init(&taken[r], kSumWarps);
    barriers_ready();
  }
  if (warp == kSumWarps) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_address(&columns)),
                 "n"(C::kColumns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const unsigned memory = columns;
  const int64_t turn = gridDim.x / split;

  if (warp == kSumWarps) {
    if (lane == 0) {  // copies
      unsigned it = 0;
      bool ok = true;
      for (int64_t tile = blockIdx.x / split; ok && tile < tiles; tile += turn) {
        const int f0 = static_cast<int>(tile % features) * kBlock;
        const int t0 = static_cast<int>(tile / features) * TOKENS;
        for (int b = first; b < last; ++b, ++it) {
          const unsigned s = it % C::kStages;
          if (!(ok = wait_for(&empty[s], ((it / C::kStages) & 1) ^ 1, &failed))) break;
          barrier_expect(&full[s], C::kStage);
          unsigned char* at = stages + s * C::kStage;
          copy_tile(at, &map_w, b * kBlock, f0, &full[s]);
          copy_tile(at + kBlock * kBlock, &map_a, b * kBlock, t0, &full[s]);
        }
      }
      // nothing may be in flight when the block ends
      for (unsigned back = it > C::kStages ? it - C::kStages : 0; back < it; ++back)
        for (int n = 0; n < 1000000 && !barrier_passed(&full[back % C::kStages], (back / C::kStages) & 1);
             ++n) {
        }
    }
  } else if (warp == kSumWarps + 1) {
    if (lane == 0) {  // products
      unsigned it = 0;
      bool ok = true;
      for (int64_t tile = blockIdx.x / split; ok && tile < tiles; tile += turn)
        for (int b = first; b < last; ++b, ++it) {
          const unsigned s = it % C::kStages, r = it % C::kResults;
          if (!(ok = wait_for(&taken[r], ((it / C::kResults) & 1) ^ 1, &failed) &&
                     wait_for(&full[s], (it / C::kStages) & 1, &failed)))
            break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const unsigned at = smem_address(stages + s * C::kStage);
#pragma unroll
          for (int k = 0; k < kBlock; k += 32)
            product(memory + r * TOKENS, operand_at(at + k), operand_at(at + kBlock * kBlock + k),
                    instruction(TOKENS), k > 0);
          commit(&empty[s]);
          commit(&ready[r]);
        }
      for (int n = 0; it > 0 && n < 1000000; ++n)  // none may be in flight when the block ends
        if (barrier_passed(&ready[(it - 1) % C::kResults], ((it - 1) / C::kResults) & 1)) break;
    }
  } else {
    // warp w: lanes (features) 32 (w % 4) .., columns (tokens) of half w / 4
    const int half = warp / 4 * C::kOwn;
    const unsigned lanes = static_cast<unsigned>(warp % 4 * 32) << 16;
    unsigned it = 0;
    bool ok = true;
    for (int64_t tile = blockIdx.x / split; tile < tiles; tile += turn) {
      const int64_t f0 = tile % features, t0 = tile / features * TOKENS;
      const int64_t token = t0 + threadIdx.x;
      const bool scales = threadIdx.x < TOKENS && token < p.m;
      const float* sa = p.sa + token * p.ldsa;
      const float* sw = p.sw + f0 * p.ldsw;
      float sum[C::kOwn];
#pragma unroll
      for (int j = 0; j < C::kOwn; ++j) sum[j] = 0.f;
      float next_a = scales && first < last ? sa[first] : 0.f, next_w = first < last ? sw[first] : 0.f;
      for (int b = first; b < last; ++b, ++it) {  // with `ok` gone too: all warps meet
        float* f = factors[it & 1];
        if (threadIdx.x < TOKENS) f[threadIdx.x] = __fmul_rn(next_a, next_w);
        if (b + 1 < last) {
          next_a = scales ? sa[b + 1] : 0.f;
          next_w = sw[b + 1];
        }
        asm volatile("bar.sync 1, %0;" ::"n"(kSumWarps * 32) : "memory");
        const unsigned r = it % C::kResults;
        ok = __all_sync(0xFFFFFFFFu, ok && wait_for(&ready[r], (it / C::kResults) & 1, &failed));
        if (ok) {
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
          for (int c = 0; c < C::kOwn; c += C::kPiece) {
            float v[C::kPiece];
            read_columns<C::kPiece>(memory + lanes + r * TOKENS + half + c, v);
            asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
            for (int j = 0; j < C::kPiece; j += 4) {
              const float4 q = *reinterpret_cast<const float4*>(&f[half + c + j]);
              const float2 x = fma2(make_float2(v[j], v[j + 1]), make_float2(q.x, q.y),
                                    make_float2(sum[c + j], sum[c + j + 1]));
              const float2 z = fma2(make_float2(v[j + 2], v[j + 3]), make_float2(q.z, q.w),
                                    make_float2(sum[c + j + 2], sum[c + j + 3]));
              sum[c + j] = x.x, sum[c + j + 1] = x.y, sum[c + j + 2] = z.x, sum[c + j + 3] = z.y;
            }
          }
          asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
          __syncwarp();
          if (lane == 0) barrier_arrive(&taken[r]);
        }
      }
      const int64_t feature = f0 * kBlock + warp % 4 * 32 + lane;
      if (split == 1) {
        if (feature < p.n) {
          T* to = y + t0 * p.ldy + feature;
          const int64_t left = p.m - t0 - half;
#pragma unroll
          for (int j = 0; j < C::kOwn; ++j)
            if (j < left) to[(half + j) * p.ldy] = from_f32<T>(ok ? sum[j] : __int_as_float(0x7FC00000));
        }
      } else {
        // the parts of a tile (one a cluster): [token][feature] in the stages, whose copies are all used
        float* part = reinterpret_cast<float*>(stages);
#pragma unroll
        for (int j = 0; j < C::kOwn; ++j)
          part[(half + j) * kBlock + warp % 4 * 32 + lane] = ok ? sum[j] : __int_as_float(0x7FC00000);
      }
    }
  }
  __syncwarp();
  if (split > 1) {
    cluster_publish();
    cluster_sync();
    const int64_t tile = blockIdx.x / split;
    const int64_t f0 = tile % features * kBlock, t0 = tile / features * TOKENS;
    const unsigned part = smem_address(stages);
    for (int j = rank * kThreads + threadIdx.x; j < TOKENS * kBlock; j += split * kThreads) {
      const int64_t t = t0 + j / kBlock, f = f0 + j % kBlock;
      if (t >= p.m || f >= p.n) continue;
      float sum = 0.f;
      for (int r = 0; r < split; ++r) {
        unsigned at;
        float v;
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(part + 4 * j), "r"(r));
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
        sum = __fadd_rn(sum, v);
      }
      y[t * p.ldy + f] = from_f32<T>(sum);
    }
    cluster_sync();
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (warp == kSumWarps)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(memory), "n"(C::kColumns));
}

// ---------------------------------------------------------------------------- many tokens
// The same product with the tokens as the tensor core's rows and FEATURES features as its columns: a thread's token has
// one scale a block for all of the thread's columns, so that scaling and adding takes one instruction for two
// results and no shared memory; sixteen warps have a quarter of the columns each. Rows of y take 16 bytes at once.
// 16,384 x 8,192 x 4,096: 565 to 585 us (1.88 to 1.95 PFLOP/s); the copies alone, 48 KB a block of k and SM, need 422.
// Shared between the blocks of a cluster (multicast) they gain nothing: an SM takes in no more; two SMs on one tile of
// 256 x 256 (cta_group::2) would take in two thirds, but wait longer for each other (1.04 ms).
constexpr int kRowWarps = 16;
constexpr int kRowThreads = (kRowWarps + 2) * 32;

template <int FEATURES>
struct RowConfig {
  static constexpr int kStage = (kBlock + FEATURES) * kBlock;
  static constexpr int kStages = FEATURES == 256 ? 4 : 6;
  static constexpr int kResults = 512 / FEATURES;
  static constexpr int kOwn = FEATURES / 4;  // columns of a summing thread
  static constexpr int kShared = kStages * kStage + 1024;
};

template <typename T, int FEATURES>
__global__ void __launch_bounds__(kRowThreads, 1)
gemm_q8_rows_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_w,
                    Problem p, T* __restrict__ y) {
  using C = RowConfig<FEATURES>;
  extern __shared__ unsigned char raw[];
  __shared__ uint64_t full[C::kStages], empty[C::kStages], ready[C::kResults], taken[C::kResults];
  __shared__ unsigned columns;
  __shared__ volatile int failed;
  unsigned char* stages = raw + (1024 - (smem_address(raw) & 1023)) % 1024;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int across = static_cast<int>((p.n + FEATURES - 1) / FEATURES);
  const int64_t tiles = across * ((p.m + kBlock - 1) / kBlock);
  const int blocks = static_cast<int>((p.k + kBlock - 1) / kBlock);

  if (threadIdx.x == 0) {
    failed = 0;
    for (int s = 0; s < C::kStages; ++s) barrier_init(&full[s], 1), barrier_init(&empty[s], 1);
    for (int r = 0; r < C::kResults; ++r) barrier_init(&ready[r], 1), barrier_init(&taken[r], kRowWarps);
    barriers_ready();
  }
  if (warp == kRowWarps) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_address(&columns)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const unsigned memory = columns;

  if (warp == kRowWarps) {
    if (lane == 0) {  // copies
      unsigned it = 0;
      bool ok = true;
      for (int64_t tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x) {
        const int f0 = static_cast<int>(tile % across) * FEATURES;
        const int t0 = static_cast<int>(tile / across) * kBlock;
        for (int b = 0; b < blocks; ++b, ++it) {
          const unsigned s = it % C::kStages;
          if (!(ok = wait_for(&empty[s], ((it / C::kStages) & 1) ^ 1, &failed))) break;
          barrier_expect(&full[s], C::kStage);
          unsigned char* at = stages + s * C::kStage;
          copy_tile(at, &map_a, b * kBlock, t0, &full[s]);
          copy_tile(at + kBlock * kBlock, &map_w, b * kBlock, f0, &full[s]);
        }
      }
      // nothing may be in flight when the block ends
      for (unsigned back = it > C::kStages ? it - C::kStages : 0; back < it; ++back)
        for (int n = 0; n < 1000000 && !barrier_passed(&full[back % C::kStages], (back / C::kStages) & 1);
             ++n) {
        }
    }
  } else if (warp == kRowWarps + 1) {
    if (lane == 0) {  // products
      unsigned it = 0;
      bool ok = true;
      for (int64_t tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x)
        for (int b = 0; b < blocks; ++b, ++it) {
          const unsigned s = it % C::kStages, r = it % C::kResults;
          if (!(ok = wait_for(&taken[r], ((it / C::kResults) & 1) ^ 1, &failed) &&
                     wait_for(&full[s], (it / C::kStages) & 1, &failed)))
            break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const unsigned at = smem_address(stages + s * C::kStage);
#pragma unroll
          for (int k = 0; k < kBlock; k += 32)
            product(memory + r * FEATURES, operand_at(at + k), operand_at(at + kBlock * kBlock + k),
                    instruction(FEATURES), k > 0);
          commit(&empty[s]);
          commit(&ready[r]);
        }
      for (int n = 0; it > 0 && n < 1000000; ++n)  // none may be in flight when the block ends
        if (barrier_passed(&ready[(it - 1) % C::kResults], ((it - 1) / C::kResults) & 1)) break;
    }
  } else {
    // warp w: lanes (tokens) 32 (w % 4) .., columns (features) of quarter w / 4
    const int quarter = warp / 4 * C::kOwn;
    const unsigned at = memory + (static_cast<unsigned>(warp % 4 * 32) << 16) + quarter;
    unsigned it = 0;
    bool ok = true;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
      // (worked out again behind the loop, which has no registers for them)
      const float *sa, *sw;
      {
        const int64_t f0 = tile % across * FEATURES + quarter, token = tile / across * kBlock + warp % 4 * 32 + lane;
        // a token behind m: its operands are zeros; columns behind n: zeros either way
        sa = p.sa + min(token, p.m - 1) * p.ldsa;
        sw = p.sw + min(f0, p.n - 1) / kBlock * p.ldsw;
      }
      float2 sum[C::kOwn / 2];
#pragma unroll
      for (int j = 0; j < C::kOwn / 2; ++j) sum[j] = make_float2(0.f, 0.f);
      float next_a = sa[0], next_w = sw[0];
      for (int b = 0; b < blocks; ++b, ++it) {
        const float f = __fmul_rn(next_a, next_w);
        if (b + 1 < blocks) {
          next_a = sa[b + 1];
          next_w = sw[b + 1];
        }
        const unsigned r = it % C::kResults;
        ok = __all_sync(0xFFFFFFFFu, ok && wait_for(&ready[r], (it / C::kResults) & 1, &failed));
        if (!ok) continue;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
        for (int c = 0; c < C::kOwn; c += 16) {
          float v[16];
          read_columns<16>(at + r * FEATURES + c, v);
          asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
          if (c + 16 == C::kOwn) {  // read to the end: the next result may come
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) barrier_arrive(&taken[r]);
          }
#pragma unroll
          for (int j = 0; j < 16; j += 2)
            sum[(c + j) / 2] = fma2(make_float2(v[j], v[j + 1]), both(f), sum[(c + j) / 2]);
        }
      }
      const int64_t f0 = tile % across * FEATURES + quarter, token = tile / across * kBlock + warp % 4 * 32 + lane;
      if (token >= p.m) continue;
      T* to = y + token * p.ldy + f0;
      const float bad = __int_as_float(0x7FC00000);
      constexpr int kV = 16 / static_cast<int>(sizeof(T));
#pragma unroll
      for (int j = 0; j < C::kOwn; j += kV) {
        alignas(16) T w[kV];
#pragma unroll
        for (int e = 0; e < kV; e += 2)
          *reinterpret_cast<typename Pair<T>::type*>(w + e) = pair_from_f32<T>(ok ? sum[(j + e) / 2] : both(bad));
        if (f0 + j < p.n) *reinterpret_cast<uint4*>(to + j) = *reinterpret_cast<const uint4*>(w);
      }
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (warp == kRowWarps)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(memory));
}

// ---------------------------------------------------------------------------- launch
using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                            const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                            CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                            CUtensorMapFloatOOBfill);

cudaError_t encoder(Encode* out) {
  static std::atomic<Encode> kept{nullptr};  // the driver's function, the same for the whole process
  Encode known = kept.load();
  if (!known) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e =
        cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess) return e;
    if (q != cudaDriverEntryPointSuccess || !f) return cudaErrorNotSupported;
    kept.store(known = reinterpret_cast<Encode>(f));
  }
  *out = known;
  return cudaSuccess;
}

cudaError_t tile_map(Encode encode, CUtensorMap* map, const uint8_t* base, int64_t rows, int64_t width,
                     int64_t ld, int box) {
  const cuuint64_t dims[] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(rows)};
  // a single row's distance to the next may be any; a map's is a multiple of 16 bytes
  const cuuint64_t strides[] = {static_cast<cuuint64_t>(rows > 1 ? ld : (width + 15) / 16 * 16)};
  const cuuint32_t tile[] = {kBlock, static_cast<cuuint32_t>(box)}, steps[] = {1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(base), dims, strides,
                            tile, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// A tile's blocks of k over a cluster while that leaves no SM with two parts, nor a part without two blocks.
int split_of(int64_t tiles, int64_t blocks) {
  int split = 1;
  while (2 * split <= kMaxSplit && tiles * 2 * split <= kSms && blocks >= 4 * split) split *= 2;
  return split;
}

template <typename T, int TOKENS>
cudaError_t run(Encode encode, const GemmQ8<T>& g, cudaStream_t stream) {
  using C = Config<TOKENS>;
  CUtensorMap w, a;
  cudaError_t e = tile_map(encode, &w, g.w, g.n, g.k, g.ldw, kBlock);
  if (e == cudaSuccess) e = tile_map(encode, &a, g.a, g.m, g.k, g.lda, TOKENS);
  auto* kernel = gemm_q8_kernel<T, TOKENS>;
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kShared);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (g.n + kBlock - 1) / kBlock * ((g.m + TOKENS - 1) / TOKENS);
  const int64_t blocks = (g.k + kBlock - 1) / kBlock;
  const int split = split_of(tiles, blocks);
  const int64_t grid = split > 1 ? tiles * split : std::min<int64_t>(tiles, kSms);
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t config = cluster_config(&attr, dim3(static_cast<unsigned>(grid)), kThreads,
                                                   C::kShared, split, stream);
  return cudaLaunchKernelEx(&config, kernel, w, a,
                            Problem{g.m, g.n, g.k, g.sa, g.sw, g.ldsa, g.ldsw, g.ldy}, g.y);
}

template <typename T, int FEATURES>
cudaError_t run_rows(Encode encode, const GemmQ8<T>& g, cudaStream_t stream) {
  using C = RowConfig<FEATURES>;
  CUtensorMap w, a;
  cudaError_t e = tile_map(encode, &w, g.w, g.n, g.k, g.ldw, FEATURES);
  if (e == cudaSuccess) e = tile_map(encode, &a, g.a, g.m, g.k, g.lda, kBlock);
  auto* kernel = gemm_q8_rows_kernel<T, FEATURES>;
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kShared);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (g.n + FEATURES - 1) / FEATURES * ((g.m + kBlock - 1) / kBlock);
  kernel<<<static_cast<unsigned>(std::min<int64_t>(tiles, kSms)), kRowThreads, C::kShared, stream>>>(
      a, w, Problem{g.m, g.n, g.k, g.sa, g.sw, g.ldsa, g.ldsw, g.ldy}, g.y);
  return cudaGetLastError();
}

// y = 0: no block of k.
template <typename T>
__global__ void zero_kernel(int64_t m, int64_t n, int64_t ldy, T* y) {
  for (int64_t j = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; j < m * n;
       j += int64_t(gridDim.x) * blockDim.x)
    y[j / n * ldy + j % n] = from_f32<T>(0.f);
}

}  // namespace

template <typename T>
cudaError_t launch_gemm_q8(const GemmQ8<T>& g, cudaStream_t stream) {
  if (g.k == 0) {
    zero_kernel<<<kSms, 256, 0, stream>>>(g.m, g.n, g.ldy, g.y);
    return cudaGetLastError();
  }
  Encode encode;
  const cudaError_t e = encoder(&encode);
  if (e != cudaSuccess) return e;
  if (g.m <= 16) return run<T, 16>(encode, g, stream);
  if (g.m <= 32) return run<T, 32>(encode, g, stream);
  // The least (turns of all SMs) x (a tile's time: its blocks of k, and its start and end), in cycles, from 4,096 x 4,096
  // x 512 and 16,384 x 8,192 x 4,096 in BF16 (64 tokens 49 and 1,535 us, 128 tokens 39 and 917, rows by 128 features
  // 25 and 769, by 256 features 27 and 565; on 40 drawn sizes the choice is the best one or within 13%, but for a few
  // of 7 to 11 us). Rows of y that do not take 16 bytes at once are for the kernel whose lanes are features: a row
  // kernel's lanes would store elements of 32 rows (4,096 x 4,095 x 512: 128 tokens 40 us, rows 146 and 157;
  // 16,384 x 8,191 x 4,096: 919, 1,802 and 1,590).
  const int64_t blocks = (g.k + kBlock - 1) / kBlock;
  auto cost = [&](int features, int tokens, int block, int ends, bool splits) {
    const int64_t tiles = (g.n + features - 1) / features * ((g.m + tokens - 1) / tokens);
    const int split = splits ? split_of(tiles, blocks) : 1;
    return (tiles * split + kSms - 1) / kSms * ((blocks + split - 1) / split * block + ends);
  };
  const int64_t costs[] = {cost(kBlock, 64, 725, 3800, true), cost(kBlock, 128, 770, 7600, true),
                           cost(128, kBlock, 725, 3900, false), cost(256, kBlock, 960, 9200, false)};
  const bool vectors = ((reinterpret_cast<uintptr_t>(g.y) | static_cast<uintptr_t>(g.ldy * sizeof(T)) |
                         static_cast<uintptr_t>(g.n * sizeof(T))) & 15) == 0;
  switch (std::min_element(costs, costs + (vectors ? 4 : 2)) - costs) {
    case 0: return run<T, 64>(encode, g, stream);
    case 1: return run<T, 128>(encode, g, stream);
    case 2: return run_rows<T, 128>(encode, g, stream);
    default: return run_rows<T, 256>(encode, g, stream);
  }
}
template cudaError_t launch_gemm_q8(const GemmQ8<float>&, cudaStream_t);
template cudaError_t launch_gemm_q8(const GemmQ8<__nv_bfloat16>&, cudaStream_t);
template cudaError_t launch_gemm_q8(const GemmQ8<__half>&, cudaStream_t);

}  // namespace bsolve
