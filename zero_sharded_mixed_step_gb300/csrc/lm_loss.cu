// Softmax cross entropy of a language model's head over a large vocabulary,
// and its gradient, without ever keeping the logits.
//
//   l = h T^T           h: N tokens x d, T: V x d, both 16-bit
//   lse_i  = log sum_v exp(l_iv)          loss_i = lse_i - l_{i,t_i}
//   D_iv   = exp(l_iv - lse_i) - [v = t_i]     (0 for a token without target)
//   dh     = s D T      dT = s D^T h (+ what was there)
//
// Four matrix products of 2 N V d operations each: l for the loss, l again
// for D (keeping l would be N V values), and the two gradients.  All four run
// through one persistent tensor-core kernel, lm_gemm, with an epilogue each:
//   kStats    keeps the maximum and the sum of exponentials of each row over
//             the tile's columns, and the target's logit; lm_combine joins
//             them over the vocabulary;
//   kProbs    forms D of one piece of the vocabulary, 16-bit, in workspace;
//   kDHidden  D T over the piece, added to fp32 sums in workspace;
//   kDTable   D^T h of the piece's rows, complete over the tokens, rounded
//             once into the table's gradient.
// D is rounded to the inputs' 16-bit type, because the matrix instructions
// take two operands of one type; in fp16 it is scaled by 2^14 first (|D| <= 1,
// and a probability of 1 / V would lose bits as a subnormal), undone in the
// fp32 epilogues.  Everything else is fp32 until the outputs are rounded.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "step_math.cuh"
#include "umma.cuh"
#include "zero_context.h"
#include "zero_internal.h"
#include "zero_step.h"

namespace zero {

// Bounded device-side waits of lm_gemm that gave up.
__device__ unsigned int g_lm_timeouts;

namespace {

using namespace umma;
using dev::Fmt;

constexpr int kTileM = 256;          // rows of a tile: 128 in each CTA of the pair
constexpr int kTileN = 256;          // most columns of a tile (one fp32 accumulator; TMEM holds two)
constexpr int kTileK = 64;           // 128 bytes of a 16-bit operand: one swizzle row
constexpr int kStages = 6;
constexpr int kOperandBytes = 128 * kTileK * 2;      // one operand's half tile in one CTA
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kThreads = 192;        // warp 0 loads, warp 1 issues the products, warps 2-5 are the epilogue
constexpr int kGemmSmem = kStages * kStageBytes + 1024;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

enum Kind : int { kStats = 0, kProbs = 1, kDHidden = 2, kDTable = 3 };

// What fp16 scales D by (see above); bf16 has fp32's range.
template <typename T>
__host__ __device__ constexpr float d_scale() {
  return sizeof(T) == 2 && std::is_same<T, __half>::value ? 16384.f : 1.f;
}

struct GemmArgs {
  CUtensorMap a, b;
  int m_tiles, n_tiles, splits, kb_total;
  int M, N;                  // rows and columns of the product that exist
  int bn;                    // columns of a tile, a multiple of 32
  int b_boxes;               // boxes of an MN-major B half tile
  int b_half;                // columns of B that each CTA of the pair holds: bn / 2
  uint32_t stage_tx;         // bytes that land per stage, both CTAs together
  int b_row0;                // first row of the table that B starts from (kStats, kProbs: N; kDHidden: K)
  int tokens;
  int vocab0;                // vocabulary index of column 0 (kProbs)
  int vocab;
  const void* targets;
  int id_bytes;
  const float* lse;
  float2* part;              // kStats: [row][n tile] maximum and sum, in powers of 2
  float* target_logit;
  void* out16;               // kProbs: D; kDTable: the table's gradient
  int64_t out_stride;
  float* acc;                // kDHidden: [split][row][N]
  int add;                   // kDHidden: add to acc; kDTable: add to the gradient
  float scale;
};

// The target of token i, or -1 where it has none.
__device__ __forceinline__ int load_target(const void* ids, int id_bytes, int64_t i, int vocab) {
  const int64_t t = id_bytes == 8 ? static_cast<const int64_t*>(ids)[i] : static_cast<const int32_t*>(ids)[i];
  return t >= 0 && t < vocab ? static_cast<int>(t) : -1;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// One fp32 row of a tile of the accumulator, 32 columns at a time.
template <typename F>
__device__ __forceinline__ void for_columns(uint32_t tmem, int bn, F f) {
  float v[32];
  for (int c = 0; c < bn; c += 32) {
    tmem_ld32(tmem + c, v);
    tmem_ld_wait();
    f(c, v);
  }
}

template <typename T, int KIND>
__device__ __forceinline__ void epilogue(const GemmArgs& g, uint32_t tmem, int row, int mt, int nt, int split) {
  const int n0 = nt * g.bn;
  const bool row_ok = row < g.M;
  if constexpr (KIND == kStats) {
    const int target = row_ok ? load_target(g.targets, g.id_bytes, row, g.vocab) - n0 : -1;
    float top = -INFINITY, sum = 0.f;
    for_columns(tmem, g.bn, [&](int c, float (&v)[32]) {
      if (n0 + c + 32 > g.N) {
#pragma unroll
        for (int k = 0; k < 32; ++k)
          if (n0 + c + k >= g.N) v[k] = -INFINITY;
      }
      if (target >= c && target < c + 32) {
#pragma unroll
        for (int k = 0; k < 32; ++k)
          if (target == c + k) g.target_logit[row] = v[k];
      }
      float m = v[0];
#pragma unroll
      for (int k = 1; k < 32; ++k) m = fmaxf(m, v[k]);
      m *= kLog2e;
      if (m > top) {
        sum *= exp2_fast(top - m);
        top = m;
      }
      // a row of -inf so far: keep the reference finite, the sum stays 0
      const float ref = top == -INFINITY ? 0.f : top;
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int k = 0; k < 32; k += 2) {
        s0 += exp2_fast(fmaf(v[k], kLog2e, -ref));
        s1 += exp2_fast(fmaf(v[k + 1], kLog2e, -ref));
      }
      sum += s0 + s1;
    });
    if (row_ok) g.part[static_cast<int64_t>(row) * g.n_tiles + nt] = make_float2(top, sum);
  } else if constexpr (KIND == kProbs) {
    const int target = row_ok ? load_target(g.targets, g.id_bytes, row, g.vocab) : -1;
    const int local = target - g.vocab0 - n0;
    const float ref = row_ok ? g.lse[row] * kLog2e : 0.f;
    T* out = static_cast<T*>(g.out16) + static_cast<int64_t>(row) * g.out_stride + n0;
    for_columns(tmem, g.bn, [&](int c, float (&v)[32]) {
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        float p = exp2_fast(fmaf(v[k], kLog2e, -ref));
        if (local == c + k) p -= 1.f;
        v[k] = target >= 0 && n0 + c + k < g.N ? p * d_scale<T>() : 0.f;
      }
      if (row_ok) {
#pragma unroll
        for (int k = 0; k < 32; k += 8) {
          float w[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) w[q] = v[k + q];
          dev::st_16B(out + c + k, Fmt<T>::pack8(w));
        }
      }
    });
  } else if constexpr (KIND == kDHidden) {
    float* out = g.acc + (static_cast<int64_t>(split) * g.M + row) * g.N + n0;
    for_columns(tmem, g.bn, [&](int c, float (&v)[32]) {
#pragma unroll
      for (int k = 0; k < 32; k += 8) {
        if (!row_ok || n0 + c + k >= g.N) continue;
        float w[8];
        if (g.add) dev::ld_32B(out + c + k, w);
#pragma unroll
        for (int q = 0; q < 8; ++q) w[q] = g.add ? w[q] + v[k + q] : v[k + q];
        dev::st_32B(out + c + k, w);
      }
    });
  } else {
    T* out = static_cast<T*>(g.out16) + static_cast<int64_t>(row) * g.out_stride + n0;
    for_columns(tmem, g.bn, [&](int c, float (&v)[32]) {
#pragma unroll
      for (int k = 0; k < 32; k += 8) {
        if (!row_ok || n0 + c + k >= g.N) continue;
        float w[8];
        if (g.add) Fmt<T>::unpack8(dev::ld_16B(out + c + k), w);
#pragma unroll
        for (int q = 0; q < 8; ++q) w[q] = g.add ? fmaf(v[k + q], g.scale, w[q]) : v[k + q] * g.scale;
        dev::st_16B(out + c + k, Fmt<T>::pack8(w));
      }
    });
  }
}

// The persistent product kernel: pairs of CTAs, each pair one 256-row tile at
// a time, operands through a ring of TMA stages, two accumulators in TMEM so
// that one tile's epilogue runs beside the next one's products.
template <typename T, int KIND>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) lm_gemm(const __grid_constant__ GemmArgs g) {
  constexpr bool kAMn = KIND == kDTable;                        // A = D^T: rows of vocabulary are contiguous in D
  constexpr bool kBMn = KIND == kDTable || KIND == kDHidden;    // B = h or T with K the row index
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) uint64_t bars[2 * kStages + 5];
  __shared__ uint32_t tmem_slot;
  __shared__ int failed;
  const uint32_t ring = (smem_addr(raw) + 1023u) & ~1023u;
  const uint32_t bar0 = smem_addr(bars);
  auto full = [&](int s) { return bar0 + 8 * s; };
  auto empty = [&](int s) { return bar0 + 8 * (kStages + s); };
  auto done = [&](int a) { return bar0 + 8 * (2 * kStages + a); };        // accumulator a is complete
  auto taken = [&](int a) { return bar0 + 8 * (2 * kStages + 2 + a); };   // accumulator a has been read
  const uint32_t drained = bar0 + 8 * (2 * kStages + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int total = g.m_tiles * g.n_tiles * g.splits;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      bar_init(full(s), 1);
      bar_init(empty(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      bar_init(done(a), 1);
      bar_init(taken(a), 8);
    }
    bar_init(drained, 1);
    failed = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_map(&g.a);
    tma_prefetch_map(&g.b);
  }
  if (warp == 1) tmem_alloc(smem_addr(&tmem_slot), 512);
  __syncthreads();
  fence_before();
  cluster_sync();
  fence_after();
  const uint32_t tmem = tmem_slot;

  int issued = 0;      // stages loaded by this CTA (warp 0)
  bool ok = true;
  if (warp == 0) {
    if (lane == 0) {
      for (int t = pair; t < total && ok; t += pairs) {
        const int mt = t % g.m_tiles, rest = t / g.m_tiles, nt = rest % g.n_tiles, sp = rest / g.n_tiles;
        const int k0 = static_cast<int>(static_cast<int64_t>(g.kb_total) * sp / g.splits);
        const int k1 = static_cast<int>(static_cast<int64_t>(g.kb_total) * (sp + 1) / g.splits);
        const int am = mt * kTileM + static_cast<int>(rank) * 128;
        const int bn = nt * g.bn + static_cast<int>(rank) * g.b_half;
        for (int kb = k0; kb < k1; ++kb, ++issued) {
          const int s = issued % kStages;
          if (!(ok = bar_wait(empty(s), ((issued / kStages) & 1) ^ 1))) break;
          if (rank == 0) bar_expect(full(s), g.stage_tx);
          const uint32_t bar = in_cta(full(s), 0);
          const uint32_t sa = ring + s * kStageBytes, sb = sa + kOperandBytes;
          const int k = kb * kTileK;
          if (kAMn) {
            tma_load(sa, &g.a, am, k, bar);
            tma_load(sa + 8192, &g.a, am + 64, k, bar);
          } else {
            tma_load(sa, &g.a, k, am, bar);
          }
          if (kBMn) {
            const int row = k + (KIND == kDHidden ? g.b_row0 : 0);
            for (int j = 0; j < g.b_boxes; ++j) tma_load(sb + j * 8192, &g.b, bn + 64 * j, row, bar);
          } else {
            tma_load(sb, &g.b, k, bn + g.b_row0, bar);
          }
        }
      }
      if (!ok) failed = 1;
    }
  } else if (warp == 1) {
    if (rank == 0 && lane == 0) {
      const uint32_t idesc = instr_desc(std::is_same<T, __nv_bfloat16>::value, kAMn, kBMn, kTileM, g.bn);
      int stage = 0, tile = 0;
      for (int t = pair; t < total && ok; t += pairs, ++tile) {
        const int sp = t / g.m_tiles / g.n_tiles;
        const int k0 = static_cast<int>(static_cast<int64_t>(g.kb_total) * sp / g.splits);
        const int k1 = static_cast<int>(static_cast<int64_t>(g.kb_total) * (sp + 1) / g.splits);
        const int a = tile & 1;
        if (!(ok = bar_wait(taken(a), ((tile >> 1) & 1) ^ 1))) break;
        fence_after();
        const uint32_t d = tmem + a * kTileN;
        for (int kb = k0; kb < k1; ++kb, ++stage) {
          const int s = stage % kStages;
          if (!(ok = bar_wait(full(s), (stage / kStages) & 1))) break;
          fence_after();
          const uint32_t sa = ring + s * kStageBytes, sb = sa + kOperandBytes;
          const uint64_t da = operand_desc(sa, kAMn ? 8192 : 0), db = operand_desc(sb, kBMn ? 8192 : 0);
#pragma unroll
          for (int q = 0; q < kTileK / 16; ++q) {
            // 16 values of K further: 32 bytes within a K-major row, 16 rows of an MN-major tile
            const uint64_t ka = (kAMn ? 2048 : 32) * q >> 4, kb16 = (kBMn ? 2048 : 32) * q >> 4;
            mma(d, da + ka, db + kb16, idesc, kb > k0 || q > 0);
          }
          mma_commit(empty(s));
        }
        if (ok) mma_commit(done(a));
      }
      if (!ok) {
        // leave no product in flight behind
        failed = 1;
        mma_commit(drained);
        bar_wait(drained, 0);
      }
    }
  } else {
    int tile = 0;
    const int quad = warp & 3;
    for (int t = pair; t < total; t += pairs, ++tile) {
      const int mt = t % g.m_tiles, rest = t / g.m_tiles, nt = rest % g.n_tiles, sp = rest / g.n_tiles;
      const int a = tile & 1;
      if (!__all_sync(0xffffffffu, bar_wait(done(a), (tile >> 1) & 1))) {
        if (lane == 0) failed = 1;
        break;
      }
      fence_after();
      epilogue<T, KIND>(g, tmem + a * kTileN + (static_cast<uint32_t>(quad) << 21),
                        mt * kTileM + static_cast<int>(rank) * 128 + quad * 32 + lane, mt, nt, sp);
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive_cluster(in_cta(taken(a), 0));
    }
  }
  __syncthreads();
  if (failed) {
    if (threadIdx.x == 0) {
      atomicAdd(&g_lm_timeouts, 1u);
      // the copies in flight land on the leader's barriers: both CTAs stay until they have
      if (rank == 0)
        for (int j = max(0, issued - kStages); j < issued; ++j) bar_wait(full(j % kStages), (j / kStages) & 1);
    }
    __syncthreads();
  }
  fence_before();
  cluster_sync();
  fence_after();
  if (warp == 1) tmem_free(tmem, 512);
}

// ---- the small kernels around the products ---------------------------------------

constexpr int kSmallThreads = 256;

// One warp per token: joins the tiles' maxima and sums, writes lse and loss.
__global__ void __launch_bounds__(kSmallThreads) lm_combine(const float2* part, int tiles, const float* target_logit,
                                                            const void* targets, int id_bytes, int vocab, int tokens,
                                                            float* loss, float* lse) {
  const int row = (blockIdx.x * kSmallThreads + threadIdx.x) >> 5, lane = threadIdx.x & 31;
  if (row >= tokens) return;
  const float2* p = part + static_cast<int64_t>(row) * tiles;
  float top = -INFINITY, sum = 0.f;
  for (int k = lane; k < tiles; k += 32) {
    const float2 x = p[k];
    const float m = fmaxf(top, x.x);
    const float ref = m == -INFINITY ? 0.f : m;
    sum = sum * exp2_fast(top - ref) + x.y * exp2_fast(x.x - ref);
    top = m;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float t2 = __shfl_xor_sync(0xffffffffu, top, o), s2 = __shfl_xor_sync(0xffffffffu, sum, o);
    const float m = fmaxf(top, t2);
    const float ref = m == -INFINITY ? 0.f : m;
    sum = sum * exp2_fast(top - ref) + s2 * exp2_fast(t2 - ref);
    top = m;
  }
  if (lane == 0) {
    const float l = fmaf(top, kLn2, logf(sum));
    lse[row] = l;
    loss[row] = load_target(targets, id_bytes, row, vocab) >= 0 ? l - target_logit[row] : 0.f;
  }
}

// The hidden vectors with the rows of tokens without target set to 0: such a
// row times D's zeros must add nothing to the table's gradient even where it
// holds an infinity or a NaN.
__global__ void __launch_bounds__(kSmallThreads) lm_masked_hidden(const uint16_t* hidden, int64_t stride, int width8,
                                                                  const void* targets, int id_bytes, int vocab,
                                                                  int tokens, uint16_t* out) {
  const int64_t total = static_cast<int64_t>(tokens) * width8;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * kSmallThreads + threadIdx.x; e < total;
       e += static_cast<int64_t>(gridDim.x) * kSmallThreads) {
    const int64_t row = e / width8, c = e - row * width8;
    uint4 x = make_uint4(0, 0, 0, 0);
    if (load_target(targets, id_bytes, row, vocab) >= 0) x = dev::ld_16B(hidden + row * stride + c * 8);
    dev::st_16B(out + e * 8, x);
  }
}

// dh = scale * the sum of the splits' fp32 sums, in the splits' order.
template <typename T>
__global__ void __launch_bounds__(kSmallThreads) lm_finish_dhidden(const float* acc, int splits, int64_t tokens,
                                                                   int width8, float scale, T* out, int64_t stride) {
  const int64_t total = tokens * width8;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * kSmallThreads + threadIdx.x; e < total;
       e += static_cast<int64_t>(gridDim.x) * kSmallThreads) {
    const int64_t row = e / width8, c = e - row * width8;
    float s[8];
    dev::ld_32B(acc + e * 8, s);
    for (int k = 1; k < splits; ++k) {
      float x[8];
      dev::ld_32B(acc + (k * total + e) * 8, x);
#pragma unroll
      for (int q = 0; q < 8; ++q) s[q] += x[q];
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) s[q] *= scale;
    dev::st_16B(out + row * stride + c * 8, Fmt<T>::pack8(s));
  }
}

// ---- host -------------------------------------------------------------------------

using host::ceil_div;
using host::cuda_fail;
using host::fail;
using host::round_up;

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder (looked up once; nullptr if there is none).
EncodeFn encoder() {
  static EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult st;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &st) != cudaSuccess ||
        st != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// A matrix of `rows` x `cols` 16-bit values with a row stride, in boxes of
// box_rows x 64 under the 128-byte swizzle; what lies outside reads as 0.
int make_map(CUtensorMap* map, int dtype, const void* base, int64_t rows, int64_t cols, int64_t stride, int box_rows) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride) * 2};
  const cuuint32_t box[2] = {kTileK, static_cast<cuuint32_t>(box_rows)}, ones[2] = {1, 1};
  EncodeFn fn = encoder();
  if (!fn) return fail(ZERO_E_CUDA, "the driver offers no tensor-map encoder");
  const CUresult r = fn(map, dtype == ZERO_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                        const_cast<void*>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? ZERO_OK : fail(ZERO_E_CUDA, "encoding a tensor map failed (%d)", static_cast<int>(r));
}

using GemmFn = void (*)(const GemmArgs);

template <int KIND>
int launch_gemm(const GemmArgs& g, int dtype, cudaStream_t s) {
  const GemmFn fn = dtype == ZERO_FP16 ? static_cast<GemmFn>(lm_gemm<__half, KIND>)
                                       : static_cast<GemmFn>(lm_gemm<__nv_bfloat16, KIND>);
  ZERO_CUDA(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kGemmSmem));
  const int64_t tiles = static_cast<int64_t>(g.m_tiles) * g.n_tiles * g.splits;
  const int pairs = static_cast<int>(std::min<int64_t>(std::max(1, sm_count() / 2), tiles));
  fn<<<2 * pairs, kThreads, kGemmSmem, s>>>(g);
  ZERO_CUDA(cudaGetLastError());
  return ZERO_OK;
}

unsigned small_grid(int64_t items) {
  return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(ceil_div(items, kSmallThreads), sm_count() * 8)));
}

// How one gradient call is cut up, from the sizes alone.
struct GradPlan {
  int64_t piece;        // vocabulary rows per piece, a multiple of 256
  int bn;               // columns of a gradient tile
  int splits;           // of the vocabulary within kDHidden
};

// Tile width for `width` columns: the multiple of 32 that wastes least, counting
// what a tile costs besides its columns as 32 more.
int tile_width(int64_t width) {
  int best = kTileN;
  int64_t cost = INT64_MAX;
  for (int bn = kTileN; bn >= 32; bn -= 32) {
    const int64_t c = ceil_div(width, bn) * (bn + 32);
    if (c < cost) {
      cost = c;
      best = bn;
    }
  }
  return best;
}

constexpr int64_t kPieceBytes = int64_t(64) << 20;   // of D: stays in L2 between its three uses
constexpr int64_t kMinPiece = 2048;
constexpr int kMaxSplits = 64;

GradPlan plan_grad(int64_t tokens, int64_t vocab, int64_t width) {
  GradPlan p;
  const int64_t by_bytes = kPieceBytes / (2 * std::max<int64_t>(tokens, 1)) / 256 * 256;
  p.piece = std::min(round_up(vocab, 256), std::max(kMinPiece, by_bytes));
  p.bn = tile_width(width);
  const int64_t tiles = ceil_div(tokens, kTileM) * ceil_div(width, p.bn);
  const int64_t kb = ceil_div(std::min(p.piece, vocab), kTileK);
  p.splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({76 / tiles, kb / 4, kMaxSplits})));
  return p;
}

struct GradSpace {
  int64_t hidden, probs, acc, total;   // byte offsets of the parts
};

GradSpace grad_space(int64_t tokens, int64_t width, const GradPlan& p) {
  GradSpace s;
  s.hidden = 0;
  s.probs = round_up(tokens * width * 2, 256);
  s.acc = s.probs + round_up(tokens * p.piece * 2, 256);
  s.total = s.acc + round_up(p.splits * tokens * width * 4, 256);
  return s;
}

int64_t loss_tiles(int64_t vocab) { return ceil_div(vocab, kTileN); }

int64_t loss_space(int64_t tokens, int64_t vocab) {
  return round_up(tokens * loss_tiles(vocab) * 8, 256) + round_up(tokens * 4, 256);
}

constexpr int64_t kMaxTokens = int64_t(1) << 24, kMaxVocab = int64_t(1) << 24, kMaxWidth = int64_t(1) << 16;

int check_sizes(int64_t tokens, int64_t vocab, int64_t width) {
  if (tokens < 0 || tokens > kMaxTokens) return fail(ZERO_E_ARG, "tokens=%lld outside [0, 2^24]", (long long)tokens);
  if (vocab < 1 || vocab > kMaxVocab) return fail(ZERO_E_ARG, "vocab=%lld outside [1, 2^24]", (long long)vocab);
  if (width < 8 || width > kMaxWidth || width % 8)
    return fail(ZERO_E_ARG, "width=%lld must be a multiple of 8 in [8, 65536]", (long long)width);
  return ZERO_OK;
}

// A matrix of 16-bit rows: present, on 16-byte boundaries, rows apart by at least their width.
int check_matrix(const char* what, const void* p, int64_t stride, int64_t rows, int64_t width) {
  if (rows > 0 && p == nullptr) return fail(ZERO_E_ARG, "%s is NULL", what);
  if (stride < width || stride > (int64_t(1) << 32)) return fail(ZERO_E_ARG, "%s: row stride %lld is below the width or too large", what, (long long)stride);
  if (!host::aligned16(p) || stride % 8) return fail(ZERO_E_ALIGN, "%s: rows must start on 16-byte boundaries", what);
  return ZERO_OK;
}

int check_common(int64_t tokens, int64_t vocab, int64_t width, int dtype, const void* hidden, int64_t hidden_stride,
                 const void* table, int64_t table_stride, const void* targets, int id_bytes, const void* workspace) {
  int rc = check_sizes(tokens, vocab, width);
  if (rc) return rc;
  if (!host::valid_dtype(dtype)) return fail(ZERO_E_ARG, "the 16-bit format must be ZERO_FP16 or ZERO_BF16");
  if (id_bytes != 4 && id_bytes != 8) return fail(ZERO_E_ARG, "ids of %d bytes: 4 or 8 are supported", id_bytes);
  if ((rc = check_matrix("hidden", hidden, hidden_stride, tokens, width))) return rc;
  if ((rc = check_matrix("table", table, table_stride, vocab, width))) return rc;
  if (tokens > 0 && targets == nullptr) return fail(ZERO_E_ARG, "targets is NULL");
  if (reinterpret_cast<uintptr_t>(targets) % id_bytes) return fail(ZERO_E_ALIGN, "targets is not aligned to its ids");
  if (tokens > 0 && workspace == nullptr) return fail(ZERO_E_ARG, "workspace is NULL");
  if (reinterpret_cast<uintptr_t>(workspace) % 256) return fail(ZERO_E_ALIGN, "workspace must be 256-byte aligned");
  return ZERO_OK;
}

}  // namespace
}  // namespace zero

using namespace zero;

extern "C" int64_t zero_lm_workspace_bytes(int64_t tokens, int64_t vocab, int64_t width, int with_grad) {
  int rc = check_sizes(tokens, vocab, width);
  if (rc) return rc;
  int64_t bytes = std::max<int64_t>(256, loss_space(tokens, vocab));
  if (!with_grad) return bytes;
  // any smaller count of tokens has to fit too: its sums may be split more often, and its pieces be wider
  const int64_t wide = round_up(vocab, 256);
  const int64_t probs = std::max(std::min(tokens * wide * 2, kPieceBytes), tokens * std::min(kMinPiece, wide) * 2);
  const int64_t sums = std::max(tokens, std::min<int64_t>(tokens * kMaxSplits, 76 * kTileM)) * (round_up(width, 256)) * 4;
  return std::max(bytes, round_up(tokens * width * 2, 256) + round_up(probs, 256) + round_up(sums, 256));
}

extern "C" int zero_lm_loss(int64_t tokens, int64_t vocab, int64_t width, int dtype, const void* hidden,
                            int64_t hidden_stride, const void* table, int64_t table_stride, const void* targets,
                            int id_bytes, float* loss, float* lse, void* workspace, int64_t workspace_bytes,
                            void* stream) {
  int rc = check_common(tokens, vocab, width, dtype, hidden, hidden_stride, table, table_stride, targets, id_bytes,
                        workspace);
  if (rc) return rc;
  if (tokens > 0 && (!loss || !lse)) return fail(ZERO_E_ARG, "loss and lse are required");
  if (reinterpret_cast<uintptr_t>(loss) % 4 || reinterpret_cast<uintptr_t>(lse) % 4)
    return fail(ZERO_E_ALIGN, "loss and lse must be 4-byte aligned");
  if (tokens == 0) return ZERO_OK;
  if (workspace_bytes < loss_space(tokens, vocab))
    return fail(ZERO_E_ARG, "workspace of %lld bytes: %lld are needed", (long long)workspace_bytes,
                (long long)loss_space(tokens, vocab));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  GemmArgs g;
  std::memset(&g, 0, sizeof g);
  if ((rc = make_map(&g.a, dtype, hidden, tokens, width, hidden_stride, 128))) return rc;
  if ((rc = make_map(&g.b, dtype, table, vocab, width, table_stride, kTileN / 2))) return rc;
  g.m_tiles = static_cast<int>(ceil_div(tokens, kTileM));
  g.n_tiles = static_cast<int>(loss_tiles(vocab));
  g.splits = 1;
  g.kb_total = static_cast<int>(ceil_div(width, kTileK));
  g.M = g.tokens = static_cast<int>(tokens);
  g.N = g.vocab = static_cast<int>(vocab);
  g.bn = kTileN;
  g.b_half = kTileN / 2;
  g.stage_tx = 2 * kStageBytes;
  g.targets = targets;
  g.id_bytes = id_bytes;
  g.part = static_cast<float2*>(workspace);
  g.target_logit = reinterpret_cast<float*>(static_cast<char*>(workspace) + round_up(tokens * g.n_tiles * 8, 256));
  if ((rc = launch_gemm<kStats>(g, dtype, s))) return rc;
  lm_combine<<<static_cast<unsigned>(ceil_div(tokens * 32, kSmallThreads)), kSmallThreads, 0, s>>>(
      g.part, g.n_tiles, g.target_logit, targets, id_bytes, g.vocab, g.tokens, loss, lse);
  ZERO_CUDA(cudaGetLastError());
  return ZERO_OK;
}

extern "C" int zero_lm_loss_grad(int64_t tokens, int64_t vocab, int64_t width, int dtype, const void* hidden,
                                 int64_t hidden_stride, const void* table, int64_t table_stride, const void* targets,
                                 int id_bytes, const float* lse, double scale, void* dhidden, int64_t dhidden_stride,
                                 void* dtable, int64_t dtable_stride, int accumulate, void* workspace,
                                 int64_t workspace_bytes, void* stream) {
  int rc = check_common(tokens, vocab, width, dtype, hidden, hidden_stride, table, table_stride, targets, id_bytes,
                        workspace);
  if (rc) return rc;
  if (tokens > 0 && lse == nullptr) return fail(ZERO_E_ARG, "lse is NULL");
  if (reinterpret_cast<uintptr_t>(lse) % 4) return fail(ZERO_E_ALIGN, "lse must be 4-byte aligned");
  if (!std::isfinite(static_cast<float>(scale))) return fail(ZERO_E_ARG, "scale %g is not a finite fp32 value", scale);
  if ((rc = check_matrix("dhidden", dhidden, dhidden_stride, tokens, width))) return rc;
  if ((rc = check_matrix("dtable", dtable, dtable_stride, vocab, width))) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (tokens == 0) {
    // no token: the table's gradient is 0
    if (!accumulate)
      ZERO_CUDA(cudaMemset2DAsync(dtable, dtable_stride * 2, 0, width * 2, vocab, s));
    return ZERO_OK;
  }
  const GradPlan p = plan_grad(tokens, vocab, width);
  const GradSpace sp = grad_space(tokens, width, p);
  if (workspace_bytes < sp.total)
    return fail(ZERO_E_ARG, "workspace of %lld bytes: %lld are needed", (long long)workspace_bytes,
                (long long)sp.total);
  char* ws = static_cast<char*>(workspace);
  uint16_t* masked = reinterpret_cast<uint16_t*>(ws + sp.hidden);
  void* probs = ws + sp.probs;
  float* acc = reinterpret_cast<float*>(ws + sp.acc);
  const int width8 = static_cast<int>(width / 8);
  lm_masked_hidden<<<small_grid(tokens * width8), kSmallThreads, 0, s>>>(
      static_cast<const uint16_t*>(hidden), hidden_stride, width8, targets, id_bytes, static_cast<int>(vocab),
      static_cast<int>(tokens), masked);
  ZERO_CUDA(cudaGetLastError());

  GemmArgs g;
  std::memset(&g, 0, sizeof g);
  g.tokens = static_cast<int>(tokens);
  g.vocab = static_cast<int>(vocab);
  g.targets = targets;
  g.id_bytes = id_bytes;
  g.lse = lse;
  const float unscale = static_cast<float>(scale) / (dtype == ZERO_FP16 ? d_scale<__half>() : d_scale<__nv_bfloat16>());
  for (int64_t v0 = 0; v0 < vocab; v0 += p.piece) {
    const int64_t w = std::min(p.piece, vocab - v0);
    // D of the piece
    GemmArgs a = g;
    if ((rc = make_map(&a.a, dtype, masked, tokens, width, width, 128))) return rc;
    if ((rc = make_map(&a.b, dtype, table, vocab, width, table_stride, kTileN / 2))) return rc;
    a.m_tiles = static_cast<int>(ceil_div(tokens, kTileM));
    a.n_tiles = static_cast<int>(ceil_div(w, kTileN));
    a.splits = 1;
    a.kb_total = static_cast<int>(ceil_div(width, kTileK));
    a.M = g.tokens;
    a.N = static_cast<int>(w);
    a.bn = kTileN;
    a.b_half = kTileN / 2;
    a.stage_tx = 2 * kStageBytes;
    a.b_row0 = static_cast<int>(v0);
    a.vocab0 = static_cast<int>(v0);
    a.out16 = probs;
    a.out_stride = p.piece;
    if ((rc = launch_gemm<kProbs>(a, dtype, s))) return rc;
    // its share of dh
    GemmArgs b = g;
    if ((rc = make_map(&b.a, dtype, probs, tokens, w, p.piece, 128))) return rc;
    if ((rc = make_map(&b.b, dtype, table, vocab, width, table_stride, 64))) return rc;
    b.m_tiles = a.m_tiles;
    b.n_tiles = static_cast<int>(ceil_div(width, p.bn));
    b.kb_total = static_cast<int>(ceil_div(w, kTileK));
    b.splits = std::min(p.splits, b.kb_total);
    b.M = g.tokens;
    b.N = static_cast<int>(width);
    b.bn = p.bn;
    b.b_half = p.bn / 2;
    b.b_boxes = static_cast<int>(ceil_div(b.b_half, 64));
    b.stage_tx = 2 * (kOperandBytes + b.b_boxes * 8192);
    b.b_row0 = static_cast<int>(v0);
    b.acc = acc;
    b.add = v0 > 0;
    if ((rc = launch_gemm<kDHidden>(b, dtype, s))) return rc;
    // its rows of the table's gradient
    GemmArgs c = g;
    if ((rc = make_map(&c.a, dtype, probs, tokens, w, p.piece, 64))) return rc;
    if ((rc = make_map(&c.b, dtype, masked, tokens, width, width, 64))) return rc;
    c.m_tiles = static_cast<int>(ceil_div(w, kTileM));
    c.n_tiles = b.n_tiles;
    c.splits = 1;
    c.kb_total = static_cast<int>(ceil_div(tokens, kTileK));
    c.M = static_cast<int>(w);
    c.N = static_cast<int>(width);
    c.bn = p.bn;
    c.b_half = b.b_half;
    c.b_boxes = b.b_boxes;
    c.stage_tx = b.stage_tx;
    c.out16 = static_cast<uint16_t*>(dtable) + v0 * dtable_stride;
    c.out_stride = dtable_stride;
    c.add = accumulate != 0;
    c.scale = unscale;
    if ((rc = launch_gemm<kDTable>(c, dtype, s))) return rc;
  }
  const int64_t items = tokens * width8;
  if (dtype == ZERO_FP16)
    lm_finish_dhidden<__half><<<small_grid(items), kSmallThreads, 0, s>>>(acc, p.splits, tokens, width8, unscale,
                                                                          static_cast<__half*>(dhidden), dhidden_stride);
  else
    lm_finish_dhidden<__nv_bfloat16><<<small_grid(items), kSmallThreads, 0, s>>>(
        acc, p.splits, tokens, width8, unscale, static_cast<__nv_bfloat16*>(dhidden), dhidden_stride);
  ZERO_CUDA(cudaGetLastError());
  return ZERO_OK;
}

extern "C" int zero_lm_status(void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  unsigned int n = 0;
  ZERO_CUDA(cudaStreamSynchronize(s));
  ZERO_CUDA(cudaMemcpyFromSymbol(&n, g_lm_timeouts, sizeof n));
  if (n == 0) return ZERO_OK;
  const unsigned int zero_count = 0;
  ZERO_CUDA(cudaMemcpyToSymbol(g_lm_timeouts, &zero_count, sizeof zero_count));
  return fail(ZERO_E_STATE, "%u bounded device waits gave up; the losses or gradients they belonged to are incomplete", n);
}
