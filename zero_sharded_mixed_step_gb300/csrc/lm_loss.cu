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
//             them over the vocabulary (kFew: the same with the operands
//             exchanged, for a few tokens);
//   kProbs    forms D of one piece of the vocabulary, 16-bit, in workspace;
//   kDHidden  D T over the piece, added to fp32 sums in workspace;
//   kDTable   D^T h of the piece's rows, complete over the tokens, rounded
//             once into the table's gradient.
// D is rounded to the inputs' 16-bit type, because the matrix instructions
// take two operands of one type; in fp16 it is scaled by 2^14 first (|D| <= 1,
// and a probability of 1 / V would lose bits as a subnormal), undone in the
// fp32 epilogues.  Everything else is fp32 until the outputs are rounded.
//
// What bounds it.  A 256 x 256 tile takes 512 cycles of products for each 64
// of K, and 64 KB of operands, 64 bytes a cycle for each of the pair's SMs;
// measured, a block of K takes about 555 cycles however many pairs run.  On a
// rested GB300 the loss of 8192 tokens x 50257 x 768 runs its products at 0.95
// of the tensor pipe's cycles (307 us) and the gradient's launches at 0.81 to
// 0.84 (D is written at 0.7 TB/s beside them); loss and gradient together take
// 1.43 ms, 1.77 PFLOP/s over the four products.  Called without a pause the
// power limit brings the clock to about 1.45 GHz and the pair to 1.6 to 1.7 ms.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <type_traits>
#include <utility>

#include "launch.cuh"
#include "step_math.cuh"
#include "umma.cuh"
#include "zero_context.h"
#include "zero_internal.h"
#include "zero_step.h"

namespace zero {

// Bounded device-side waits of lm_gemm that gave up, over all calls; never set back (see zero_lm_status).
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
// warp 0 loads (warp 3 takes B from it where B is not K-major), warp 1 issues
// the products, warp 2 hands out the gradient's tiles, warps 4-11 are the
// epilogue: two for each quarter of the TMEM lanes, taking turns over the
// columns (one each measured the same at 768 in K, where its epilogue takes
// about half as long as a tile's products; narrower models have fewer)
constexpr int kThreads = 384;
constexpr int kEpilogueWarps = 8;
constexpr int kQueue = 4;            // tiles handed out ahead
constexpr int kGemmSmem = kStages * kStageBytes + 1024;
constexpr int kMaxJobs = 3;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

enum Kind : int { kFew = -1, kStats = 0, kProbs = 1, kDHidden = 2, kDTable = 3 };

// What fp16 scales D by (see above); bf16 has fp32's range.
template <typename T>
__host__ __device__ constexpr float d_scale() {
  return std::is_same<T, __half>::value ? 16384.f : 1.f;
}

// One matrix product of a launch, cut into tiles of kTileM x bn (x splits of K).
struct Job {
  int kind;
  int tiles;                 // m_tiles * n_tiles * splits
  int m_tiles, n_tiles, splits, kb_total;
  int M, N;                  // rows and columns of the product that exist
  int bn;                    // columns of a tile, a multiple of 32
  int b_boxes;               // boxes of an MN-major B half tile
  uint32_t stage_tx;         // bytes that land per stage, both CTAs together
  int b_row0;                // first row of the table that B starts from (kStats, kProbs: N; kDHidden: K)
  int vocab0;                // vocabulary index of column 0 (kProbs)
  void* out16;               // kProbs: D; kDTable: the table's gradient
  int64_t out_stride;
  float* acc;                // kDHidden: [split][row][N]
  int add;                   // kDHidden: add to acc; kDTable: add to the gradient
  int wide;                  // kDTable: rows allow 32-byte stores (100 x 50257 x 768: 105 us, 120 with 16-byte ones)
  float scale;
};

struct GemmArgs {
  CUtensorMap a[kMaxJobs], b[kMaxJobs];
  Job job[kMaxJobs];         // the longest tiles first, and kProbs last (see the loads)
  int jobs;
  int stall;                 // testing the bounded waits: the first pair's first block of K never arrives
  unsigned int* next;        // tiles handed out beyond one per pair (0 at the launch)
  unsigned int* failures;    // the workspace's count of waits that gave up
  unsigned int* lost;        // gradient: set where tiles of this call were not computed
  int vocab;
  const void* targets;
  int id_bytes;
  const float* lse;
  float2* part;              // maximum and sum, in powers of 2: kStats [row][n tile][half of its columns],
                             // kFew [token][32 rows of the vocabulary]
  float* target_logit;
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

__device__ __forceinline__ void st_32B_words(void* p, const uint4& a, const uint4& b) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w),
               "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

// A tile of a launch: which job, where, which blocks of K.  job < 0: no more.
struct alignas(16) Tile {
  int job, mt, nt, split, k0, k1, unused[2];
};

__device__ __forceinline__ Tile locate(const GemmArgs& g, int t) {
  Tile x{};
  while (x.job < g.jobs && t >= g.job[x.job].tiles) t -= g.job[x.job++].tiles;
  if (x.job == g.jobs) {
    x.job = -1;
    return x;
  }
  const Job& j = g.job[x.job];
  const unsigned m_tiles = j.m_tiles, rest = static_cast<unsigned>(t) / m_tiles;
  x.mt = t - static_cast<int>(rest * m_tiles);
  x.nt = static_cast<int>(rest);
  x.k1 = j.kb_total;
  if (j.splits > 1) {   // at most 2^18 blocks of K and 64 splits
    x.split = static_cast<int>(rest / static_cast<unsigned>(j.n_tiles));
    x.nt = static_cast<int>(rest) - x.split * j.n_tiles;
    x.k0 = static_cast<int>(static_cast<unsigned>(j.kb_total * x.split) / static_cast<unsigned>(j.splits));
    x.k1 = static_cast<int>(static_cast<unsigned>(j.kb_total * (x.split + 1)) / static_cast<unsigned>(j.splits));
  }
  return x;
}

// 32 values of each lane, joined over the lanes by op; lane l receives the
// l-th.  Each step exchanges half of what is left: 31 exchanges in all.
template <typename Op>
__device__ __forceinline__ float join_lanes(float (&x)[32], int lane, Op op) {
#pragma unroll
  for (int w = 16; w > 0; w /= 2) {
    const bool up = (lane & w) != 0;
#pragma unroll
    for (int k = 0; k < w; ++k) {
      const float give = up ? x[k] : x[k + w], keep = up ? x[k + w] : x[k];
      x[k] = op(keep, __shfl_xor_sync(0xffffffffu, give, w));
    }
  }
  return x[0];
}

// What the epilogue needs to know of its row, read before the tile is complete.
struct RowInfo {
  int target;      // -1: none
  float lse;
};

template <bool GRAD>
__device__ __forceinline__ RowInfo row_info(const GemmArgs& g, const Job& j, int row) {
  RowInfo r{-1, 0.f};
  if ((GRAD ? j.kind != kProbs : j.kind != kStats) || row >= j.M) return r;
  r.target = load_target(g.targets, g.id_bytes, row, g.vocab);
  if (GRAD) r.lse = g.lse[row];
  return r;
}

// This thread's row of the accumulator, 32 columns at a time from column
// `first` in steps of 64 (the quarter's other warp takes those between); the
// next columns are on their way while f works on these.  `release` runs as
// soon as the last columns are in registers.
template <typename F, typename R>
__device__ __forceinline__ void for_columns(uint32_t tmem, int first, int bn, F f, R release) {
  if (first >= bn) {
    release();
    return;
  }
  float va[32], vb[32];
  int c = first;
  tmem_ld32(tmem + c, va);
  tmem_ld_wait(va);
  for (;;) {
    if (c + 64 < bn) tmem_ld32(tmem + c + 64, vb);
    else release();
    f(c, va);
    c += 64;
    if (c >= bn) return;
    tmem_ld_wait(vb);
    if (c + 64 < bn) tmem_ld32(tmem + c + 64, va);
    else release();
    f(c, vb);
    c += 64;
    if (c >= bn) return;
    tmem_ld_wait(va);
  }
}

// The same without loads ahead, for the epilogues whose tiles take long anyway
// and which read what they add to.
template <typename F, typename R>
__device__ __forceinline__ void for_columns_plain(uint32_t tmem, int first, int bn, F f, R release) {
#pragma unroll 1
  for (int c = first; c < bn; c += 64) {
    float v[32];
    tmem_ld32(tmem + c, v);
    tmem_ld_wait(v);
    f(c, v);
  }
  release();
}

template <typename T, bool GRAD, typename R>
__device__ __forceinline__ void epilogue(const GemmArgs& g, const Job& j, const Tile& x, const RowInfo& info,
                                         uint32_t tmem, int row, int half, R release) {
  const int n0 = x.nt * j.bn;
  const bool row_ok = row < j.M;
  if (!GRAD && j.kind == kFew) {
    // a thread holds one row of the vocabulary, its columns are the tokens
    const int lane = threadIdx.x & 31;
    for_columns(tmem, half * 32, j.bn, [&](int c, float (&v)[32]) {
      const int token = n0 + c + lane;
      const int target = token < j.N ? load_target(g.targets, g.id_bytes, token, g.vocab) : -1;
      float m[32];
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        if (__shfl_sync(0xffffffffu, target, k) == row) g.target_logit[n0 + c + k] = v[k];
        v[k] = row_ok ? v[k] * kLog2e : -INFINITY;
        m[k] = v[k];
      }
      const float top = join_lanes(m, lane, [](float a, float b) { return fmaxf(a, b); });
      const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int k = 0; k < 32; ++k) v[k] = exp2_fast(v[k] - __shfl_sync(0xffffffffu, ref, k));
      const float sum = join_lanes(v, lane, [](float a, float b) { return a + b; });
      if (token < j.N) g.part[static_cast<int64_t>(token) * (j.m_tiles * 8) + row / 32] = make_float2(top, sum);
    }, release);
    return;
  }
  if (!GRAD) {
    const int target = info.target - n0;
    float top = -INFINITY, sum = 0.f;
    for_columns(tmem, half * 32, j.bn, [&](int c, float (&v)[32]) {
      if (n0 + c + 32 > j.N) {
#pragma unroll
        for (int k = 0; k < 32; ++k)
          if (n0 + c + k >= j.N) v[k] = -INFINITY;
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
    }, release);
    if (row_ok) g.part[(static_cast<int64_t>(row) * j.n_tiles + x.nt) * 2 + half] = make_float2(top, sum);
    return;
  }
  if (j.kind == kProbs) {
    const int local = info.target - j.vocab0 - n0;
    // a token without target: exp2(-inf) = 0 in every column
    const float ref = info.target >= 0 ? info.lse * kLog2e : INFINITY;
    T* out = static_cast<T*>(j.out16) + static_cast<int64_t>(row) * j.out_stride + n0;
    for_columns(tmem, half * 32, j.bn, [&](int c, float (&v)[32]) {
#pragma unroll
      for (int k = 0; k < 32; ++k) v[k] = exp2_fast(fmaf(v[k], kLog2e, -ref)) * d_scale<T>();
      if (local >= c && local < c + 32) {
#pragma unroll
        for (int k = 0; k < 32; ++k)
          if (local == c + k) v[k] -= d_scale<T>();
      }
      if (row_ok) {
#pragma unroll
        for (int k = 0; k < 32; k += 16) {
          float lo[8], hi[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            lo[q] = v[k + q];
            hi[q] = v[k + 8 + q];
          }
          st_32B_words(out + c + k, Fmt<T>::pack8(lo), Fmt<T>::pack8(hi));
        }
      }
    }, release);
  } else if (j.kind == kDHidden) {
    float* out = j.acc + (static_cast<int64_t>(x.split) * j.M + row) * j.N + n0;
    for_columns_plain(tmem, half * 32, j.bn, [&](int c, float (&v)[32]) {
      float w[4][8];
      if (j.add) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (row_ok && n0 + c + 8 * k < j.N) dev::ld_32B(out + c + 8 * k, w[k]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (!row_ok || n0 + c + 8 * k >= j.N) continue;
#pragma unroll
        for (int q = 0; q < 8; ++q) w[k][q] = j.add ? w[k][q] + v[8 * k + q] : v[8 * k + q];
        dev::st_32B(out + c + 8 * k, w[k]);
      }
    }, release);
  } else {
    T* out = static_cast<T*>(j.out16) + static_cast<int64_t>(row) * j.out_stride + n0;
    for_columns_plain(tmem, half * 32, j.bn, [&](int c, float (&v)[32]) {
      uint4 old[4];
      if (j.add) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (row_ok && n0 + c + 8 * k < j.N) old[k] = dev::ld_16B(out + c + 8 * k);
      }
#pragma unroll
      for (int k = 0; k < 4; k += 2) {
        uint4 packed[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int at = c + 8 * (k + h);
          if (!row_ok || n0 + at >= j.N) continue;
          float w[8];
          if (j.add) Fmt<T>::unpack8(old[k + h], w);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const float p = v[8 * (k + h) + q];
            w[q] = j.add ? fmaf(p, j.scale, w[q]) : p * j.scale;
          }
          packed[h] = Fmt<T>::pack8(w);
          if (!j.wide) dev::st_16B(out + at, packed[h]);
        }
        if (j.wide && row_ok && n0 + c + 8 * k < j.N) st_32B_words(out + c + 8 * k, packed[0], packed[1]);
      }
    }, release);
  }
}

// The loss's partial sums of a tile whose products never came: no number, so
// that the losses that lack it are none either.
__device__ __forceinline__ void spoil_parts(const GemmArgs& g, const Job& j, const Tile& x, int row, int half) {
  const float2 none = make_float2(-INFINITY, NAN);
  if (j.kind == kStats) {
    if (row < j.M) g.part[(static_cast<int64_t>(row) * j.n_tiles + x.nt) * 2 + half] = none;
    return;
  }
  for (int c = half * 32; c < j.bn; c += 64) {
    const int token = x.nt * j.bn + c + static_cast<int>(threadIdx.x & 31);
    if (token < j.N) g.part[static_cast<int64_t>(token) * (j.m_tiles * 8) + row / 32] = none;
  }
}

// The persistent product kernel: pairs of CTAs, each pair one 256-row tile at
// a time, operands through a ring of TMA stages, two accumulators in TMEM so
// that one tile's epilogue runs beside the next one's products.  The loss's
// tiles are all alike and are dealt out in turn.  The gradient's differ: one
// thread of the pair takes them from a counter, in the order of the jobs, the
// longest tiles first, so that the short ones fill the gaps at the end, and
// hands them to the roles of both CTAs through a short queue in shared memory.
template <typename T, bool GRAD>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) lm_gemm(const __grid_constant__ GemmArgs g) {
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) uint64_t bars[2 * kStages + 2 * kQueue + 5];
  __shared__ Tile queue[kQueue];
  __shared__ Job jobs[kMaxJobs];
  __shared__ uint32_t tmem_slot;
  __shared__ int failed;
  const uint32_t ring = (smem_addr(raw) + 1023u) & ~1023u;
  const uint32_t bar0 = smem_addr(bars);
  auto full = [&](int s) { return bar0 + 8 * s; };
  auto empty = [&](int s) { return bar0 + 8 * (kStages + s); };
  auto done = [&](int a) { return bar0 + 8 * (2 * kStages + a); };        // accumulator a is complete
  auto taken = [&](int a) { return bar0 + 8 * (2 * kStages + 2 + a); };   // accumulator a has been read
  const uint32_t drained = bar0 + 8 * (2 * kStages + 4);
  auto told = [&](int q) { return bar0 + 8 * (2 * kStages + 5 + q); };             // queue[q] holds a tile
  auto heard = [&](int q) { return bar0 + 8 * (2 * kStages + 5 + kQueue + q); };   // everyone has read it
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  allow_next();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      bar_init(full(s), 1);
      bar_init(empty(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      bar_init(done(a), 1);
      bar_init(taken(a), 2 * kEpilogueWarps);
    }
    for (int q = 0; q < kQueue; ++q) {
      bar_init(told(q), 1);
      bar_init(heard(q), 5 + 2 * kEpilogueWarps);   // in both CTAs two loaders and the epilogue, and the issuer
    }
    bar_init(drained, 1);
    failed = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    for (int k = 0; k < g.jobs; ++k) {
      tma_prefetch_map(&g.a[k]);
      tma_prefetch_map(&g.b[k]);
    }
  }
  if (warp == 1) tmem_alloc(smem_addr(&tmem_slot), 512);
  if (warp == 2 && lane < g.jobs) jobs[lane] = g.job[lane];
  __syncthreads();
  fence_before();
  cluster_sync();
  fence_after();
  const uint32_t tmem = tmem_slot;
  await_previous();

  // Every role runs as a whole warp with uniform control flow, one elected
  // lane issuing: what the loads and products take then sits in uniform
  // registers, and the issuing keeps up with the products (from a single
  // lane's branch, the products ran 10% slower).
  const bool lead = elect_one();
  bool ok = true;
  auto wait_all = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, bar_wait(bar, parity)) != 0; };
  // The i-th tile of this pair.  The one who hands out the gradient's runs in
  // the leader, so only the other CTA has to acquire from the cluster.
  auto tile_of = [&](int i) {
    if (!GRAD) return locate(g, pair + i * pairs);
    Tile x{};
    x.job = -1;
    const int q = i % kQueue;
    const uint32_t parity = (i / kQueue) & 1;
    ok = __all_sync(0xffffffffu, rank == 0 ? bar_wait(told(q), parity) : bar_wait<true>(told(q), parity)) != 0;
    if (!ok) return x;
    x = queue[q];
    __syncwarp();
    if (lead) bar_arrive(in_cta(heard(q), 0));
    return x;
  };

  int issued = 0;      // stages loaded by this warp
  if (warp == 0 || (GRAD && warp == 3)) {
    int s = 0;
    uint32_t phase = 1;
    for (int i = 0;; ++i) {
      const Tile x = tile_of(i);
      if (!ok || x.job < 0) break;
      const Job& j = jobs[x.job];
      const CUtensorMap *ma = &g.a[x.job], *mb = &g.b[x.job];
      const int kind = GRAD ? j.kind : static_cast<int>(kStats);   // kFew loads alike
      const int am = x.mt * kTileM + static_cast<int>(rank) * 128;
      const int bn = x.nt * j.bn + static_cast<int>(rank) * (j.bn / 2);
      // an MN-major operand comes as boxes of 64 columns, with K the row index
      const bool a_mn = kind == kDTable, b_mn = kind >= kDHidden;
      // One warp loads both operands where each is one box; four boxes a stage are too many for it.  The second
      // warp does not wait where it does not load, so it must not load again after that: products with an MN-major
      // B come first among a launch's jobs.
      const bool load_a = warp == 0, load_b = (warp == 0) != b_mn;
      const int row0 = b_mn ? (kind == kDHidden ? j.b_row0 : 0) : bn + j.b_row0;
      const bool two = j.b_boxes > 1, expect = load_a && rank == 0;
      const uint32_t tx = j.stage_tx;
      for (int kb = x.k0; kb < x.k1; ++kb, ++issued) {
        if (load_a || load_b) {
          ok = wait_all(empty(s), phase);
          if (!ok) break;
          const uint32_t bar = in_cta(full(s), 0);
          const uint32_t sa = ring + s * kStageBytes, sb = sa + kOperandBytes;
          const int k = kb * kTileK;
          if (lead) {
            if (expect) bar_expect(full(s), tx);
            if (load_a && !(g.stall && pair == 0 && issued == 0)) {
              if (a_mn) {
                tma_load(sa, ma, am, k, bar);
                tma_load(sa + 8192, ma, am + 64, k, bar);
              } else {
                tma_load(sa, ma, k, am, bar);
              }
            }
            if (load_b) {
              if (b_mn) {
                tma_load(sb, mb, bn, row0 + k, bar);
                if (two) tma_load(sb + 8192, mb, bn + 64, row0 + k, bar);
              } else {
                tma_load(sb, mb, k, row0, bar);
              }
            }
          }
          __syncwarp();
        }
        if (++s == kStages) {
          s = 0;
          phase ^= 1;
        }
      }
      if (!ok) break;
    }
    if (!ok && lead) failed = 1;
  } else if (warp == 1) {
    if (rank == 0) {
      int s = 0;
      uint32_t phase = 0;
      for (int i = 0;; ++i) {
        const Tile x = tile_of(i);
        if (!ok || x.job < 0) break;
        const Job& j = jobs[x.job];
        const bool a_mn = GRAD && j.kind == kDTable;      // A = D^T: rows of vocabulary are contiguous in D
        const bool b_mn = GRAD && j.kind >= kDHidden;     // B = h or T with K the row index
        const uint32_t idesc = instr_desc(std::is_same<T, __nv_bfloat16>::value, a_mn, b_mn, kTileM, j.bn);
        // 16 values of K further: 32 bytes within a K-major row, 16 rows of an MN-major tile
        const uint64_t a_step = (a_mn ? 2048 : 32) >> 4, b_step = (b_mn ? 2048 : 32) >> 4;
        const uint64_t a0 = operand_desc(ring, a_mn ? 8192 : 0), b0 = operand_desc(ring + kOperandBytes, b_mn ? 8192 : 0);
        const int a = i & 1;
        ok = wait_all(taken(a), ((i >> 1) & 1) ^ 1);
        if (!ok) break;
        fence_after();
        const uint32_t d = tmem + a * kTileN;
        for (int kb = x.k0; kb < x.k1; ++kb) {
          ok = wait_all(full(s), phase);
          if (!ok) break;
          fence_after();
          const uint64_t da = a0 + s * (kStageBytes >> 4), db = b0 + s * (kStageBytes >> 4);
          if (lead) {
#pragma unroll
            for (int q = 0; q < kTileK / 16; ++q) mma(d, da + q * a_step, db + q * b_step, idesc, kb > x.k0 || q > 0);
            mma_commit(empty(s));
          }
          __syncwarp();
          if (++s == kStages) {
            s = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        if (lead) mma_commit(done(a));
        __syncwarp();
      }
      if (!ok && lead) {
        // leave no product in flight behind
        failed = 1;
        mma_commit(drained);
        bar_wait(drained, 0);
      }
    }
  } else if (warp == 2) {
    if (GRAD && rank == 0 && lead) {
      for (int i = 0;; ++i) {
        const int q = i % kQueue;
        ok = bar_wait(heard(q), ((i / kQueue) & 1) ^ 1);
        if (!ok) break;
        const int t = i == 0 ? pair : pairs + static_cast<int>(atomicAdd(g.next, 1u));
        const Tile x = locate(g, t);
        for (uint32_t r = 0; r < 2; ++r) {
          const uint32_t at = in_cta(smem_addr(&queue[q]), r);
          st_cluster(at, x.job, x.mt, x.nt, x.split);
          st_cluster(at + 16, x.k0, x.k1, 0, 0);
          bar_arrive_written(in_cta(told(q), r));
        }
        if (x.job < 0) break;
      }
      if (!ok) failed = 1;
    }
  } else if (warp >= 4) {
    const int quad = warp & 3, half = (warp - 4) >> 2;
    auto row_of = [&](const Tile& x) { return x.mt * kTileM + static_cast<int>(rank) * 128 + quad * 32 + lane; };
    int i = 0;
    for (;; ++i) {
      const int a = i & 1;
      const Tile x = tile_of(i);
      if (!ok || x.job < 0) break;
      const Job& j = jobs[x.job];
      const int row = row_of(x);
      const RowInfo info = row_info<GRAD>(g, j, row);
      ok = wait_all(done(a), (i >> 1) & 1);
      if (!ok) break;
      fence_after();
      epilogue<T, GRAD>(g, j, x, info, tmem + a * kTileN + (static_cast<uint32_t>(quad) << 21), row, half, [&] {
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(in_cta(taken(a), 0));
      });
    }
    if (!ok) {
      if (lane == 0) failed = 1;
      if (!GRAD) {
        // this tile and the pair's others
        for (;; ++i) {
          const Tile x = tile_of(i);
          if (x.job < 0) break;
          spoil_parts(g, jobs[x.job], x, row_of(x), half);
        }
      }
    }
  }
  __syncthreads();
  if (failed) {
    if (threadIdx.x == 0) {
      atomicAdd(&g_lm_timeouts, 1u);
      atomicAdd(g.failures, 1u);
      if (GRAD) *g.lost = 1;
      // the copies in flight land on the leader's barriers: both CTAs stay until they have
      if (rank == 0)
        for (int k = max(0, issued - kStages); k < issued; ++k) bar_wait(full(k % kStages), (k / kStages) & 1);
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

// A maximum and a sum joined with another pair: sums of exponentials relative
// to their maxima.
__device__ __forceinline__ void join_pair(float& top, float& sum, float top2, float sum2) {
  const float m = fmaxf(top, top2), ref = m == -INFINITY ? 0.f : m;
  sum = sum * exp2_fast(top - ref) + sum2 * exp2_fast(top2 - ref);
  top = m;
}

// Joins the tiles' maxima and sums of each token and writes lse and loss: TEAM
// threads a token, a warp for many tokens, a block for kFew's few, whose parts
// are more (16 tokens of 1,576 parts: 8 us with a warp each).
template <int TEAM>
__global__ void __launch_bounds__(kSmallThreads) lm_combine(const float2* part, int tiles, const float* target_logit,
                                                            const void* targets, int id_bytes, int vocab, int tokens,
                                                            float* loss, float* lse) {
  __shared__ float2 of_warp[kSmallThreads / 32];
  allow_next();
  await_previous();
  const int row = (blockIdx.x * kSmallThreads + threadIdx.x) / TEAM, at = threadIdx.x % TEAM;
  if (row >= tokens) return;   // whole teams
  const float2* p = part + static_cast<int64_t>(row) * tiles;
  float top = -INFINITY, sum = 0.f;
  for (int k0 = at; k0 < tiles; k0 += TEAM * 4) {
    float2 x[4];
    float m = top;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[k] = k0 + TEAM * k < tiles ? p[k0 + TEAM * k] : make_float2(-INFINITY, 0.f);
      m = fmaxf(m, x[k].x);
    }
    const float ref = m == -INFINITY ? 0.f : m;
    sum *= exp2_fast(top - ref);
#pragma unroll
    for (int k = 0; k < 4; ++k) sum += x[k].y * exp2_fast(x[k].x - ref);
    top = m;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float t2 = __shfl_xor_sync(0xffffffffu, top, o), s2 = __shfl_xor_sync(0xffffffffu, sum, o);
    join_pair(top, sum, t2, s2);
  }
  if (TEAM > 32) {
    if (at % 32 == 0) of_warp[at / 32] = make_float2(top, sum);
    __syncthreads();
    if (at == 0)
      for (int k = 1; k < TEAM / 32; ++k) join_pair(top, sum, of_warp[k].x, of_warp[k].y);
  }
  if (at == 0) {
    const float l = fmaf(top, kLn2, logf(sum));
    lse[row] = l;
    loss[row] = load_target(targets, id_bytes, row, vocab) >= 0 ? l - target_logit[row] : 0.f;
  }
}

// The hidden vectors with the rows of tokens without target set to 0: such a
// row times D's zeros must add nothing to the table's gradient even where it
// holds an infinity or a NaN.  Also sets the products' tile counters, and the
// word after them that says whether a tile was lost, to 0.
__global__ void __launch_bounds__(kSmallThreads) lm_masked_hidden(const uint16_t* hidden, int64_t stride, int width8,
                                                                  const void* targets, int id_bytes, int vocab,
                                                                  int tokens, uint16_t* out, unsigned int* counters,
                                                                  int n_counters) {
  allow_next();
  await_previous();
  if (blockIdx.x == 0)
    for (int k = threadIdx.x; k < n_counters; k += kSmallThreads) counters[k] = 0;
  const int64_t total = static_cast<int64_t>(tokens) * width8;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * kSmallThreads + threadIdx.x; e < total;
       e += static_cast<int64_t>(gridDim.x) * kSmallThreads) {
    const int64_t row = e / width8, c = e - row * width8;
    uint4 x = make_uint4(0, 0, 0, 0);
    if (load_target(targets, id_bytes, row, vocab) >= 0) x = dev::ld_16B(hidden + row * stride + c * 8);
    dev::st_16B(out + e * 8, x);
  }
}

// dh = scale * the sum of the splits' fp32 sums, in the splits' order, BATCH
// loads at a time: several splits, of few tokens, kFinishBatch (one by one, 38
// splits of 30 tokens took 12 us), one split one, for the registers that a
// batch takes leave too few threads (8192 x 768 by batches: 14.8 us).  Where
// tiles were lost it is not known which: both gradients become NaN.
constexpr int kFinishBatch = 8;

template <typename T, int BATCH>
__global__ void __launch_bounds__(kSmallThreads) lm_finish_dhidden(const float* acc, int splits, int64_t tokens,
                                                                   int width8, float scale, T* out, int64_t stride,
                                                                   const unsigned int* lost, T* dtable, int64_t vocab,
                                                                   int64_t dtable_stride) {
  allow_next();
  await_previous();
  const bool spoiled = *lost != 0;
  const int64_t total = tokens * width8;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * kSmallThreads + threadIdx.x; e < total;
       e += static_cast<int64_t>(gridDim.x) * kSmallThreads) {
    const int64_t row = e / width8, c = e - row * width8;
    float s[8] = {};
    for (int k0 = 0; k0 < splits; k0 += BATCH) {
      float x[BATCH][8];
#pragma unroll
      for (int k = 0; k < BATCH; ++k)
        if (k0 + k < splits) dev::ld_32B(acc + ((k0 + k) * total + e) * 8, x[k]);
#pragma unroll
      for (int k = 0; k < BATCH; ++k)
        if (k0 + k < splits) {
#pragma unroll
          for (int q = 0; q < 8; ++q) s[q] += x[k][q];
        }
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) s[q] = spoiled ? NAN : s[q] * scale;
    dev::st_16B(out + row * stride + c * 8, Fmt<T>::pack8(s));
  }
  if (!spoiled) return;
  const float none[8] = {NAN, NAN, NAN, NAN, NAN, NAN, NAN, NAN};
  for (int64_t row = blockIdx.x; row < vocab; row += gridDim.x)
    for (int c = threadIdx.x; c < width8; c += kSmallThreads)
      dev::st_16B(dtable + row * dtable_stride + c * 8, Fmt<T>::pack8(none));
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

thread_local bool g_stall_next = false;

// Whether this call, the thread's next one, was to lose a block of operands.
bool take_stall() { return std::exchange(g_stall_next, false); }

// Launch the products; `stall` is handed to the first launch of a call alone.
template <bool GRAD>
int launch_gemm(GemmArgs& g, int dtype, cudaStream_t s, bool& stall) {
  g.stall = std::exchange(stall, false);
  const auto fn = dtype == ZERO_FP16 ? lm_gemm<__half, GRAD> : lm_gemm<__nv_bfloat16, GRAD>;
  ZERO_CUDA(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kGemmSmem));
  int64_t tiles = 0;
  for (int k = 0; k < g.jobs; ++k) tiles += g.job[k].tiles;
  const int pairs = static_cast<int>(std::min<int64_t>(std::max(1, sm_count() / 2), tiles));
  ZERO_CUDA(launch_chained(fn, dim3(2 * pairs), kThreads, kGemmSmem, s, g));
  return ZERO_OK;
}

unsigned small_grid(int64_t items) {
  return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(ceil_div(items, kSmallThreads), sm_count() * 8)));
}

// What the cutting up reckons with: the pairs among GB300's 152 SMs.
constexpr int64_t kPairs = 76;

// How one gradient call is cut up, from the sizes alone.
struct GradPlan {
  int64_t piece;        // vocabulary rows per piece, a multiple of 256
  int bn;               // columns of a gradient tile
  int splits;           // of the vocabulary within kDHidden
};

// Tile width for `width` columns of a gradient.  A block of K costs a pair
// 2 bn cycles of products, or the time its operands take from L2: about 600
// cycles for the 256 rows and 256 columns of the largest tile, in proportion
// to what is loaded (whole boxes of 64 columns for each CTA).
int tile_width(int64_t width) {
  int best = kTileN;
  int64_t cost = INT64_MAX;
  for (int bn = kTileN; bn >= 32; bn -= 32) {
    const int64_t loaded = kTileM + 2 * round_up(bn / 2, 64);
    const int64_t c = ceil_div(width, bn) * std::max<int64_t>(2 * bn, loaded * 600 / 512);
    if (c <= cost) {
      cost = c;
      best = bn;
    }
  }
  return best;
}

// Bytes of D at a time.  8192 tokens x 50257 x 768 take 1.66 ms with 64 MB, 1.61
// with 96 and 128, 1.60 with 192, 1.62 with 256 and 1.65 with 448 (two pieces).
constexpr int64_t kPieceBytes = int64_t(128) << 20;
// At least so many rows of the vocabulary at a time (the table's gradient is
// complete over the tokens, so its tiles take 256), while D of them stays
// below kMostPieceBytes.
constexpr int64_t kMinPiece = 2048, kLeastPiece = 256;
constexpr int64_t kMostPieceBytes = int64_t(1) << 30;
constexpr int kMaxSplits = 64;

int64_t piece_rows(int64_t tokens) {
  const int64_t row = 2 * std::max<int64_t>(tokens, 1);   // bytes of D per row of the vocabulary
  const int64_t least = std::max(kLeastPiece, std::min(kMinPiece, kMostPieceBytes / row / 256 * 256));
  return std::max(least, kPieceBytes / row / 256 * 256);
}

GradPlan plan_grad(int64_t tokens, int64_t vocab, int64_t width) {
  GradPlan p;
  // pieces of one size: a short last one has too few tiles for the SMs and the longest ones all the same
  const int64_t pieces = ceil_div(vocab, piece_rows(tokens));
  p.piece = round_up(ceil_div(vocab, pieces), 256);
  p.bn = tile_width(width);
  // With fewer tiles of dh than pairs of SMs, the vocabulary is split over them, at least 4 blocks of K each: 100
  // tokens x 50257 x 768 take 105 us so and 285 in one split, 1500 x 20000 x 512 104 and 157; twice as many splits
  // took 120 and 107.
  const int64_t tiles = ceil_div(tokens, kTileM) * ceil_div(width, p.bn);
  const int64_t kb = ceil_div(std::min(p.piece, vocab), kTileK);
  p.splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({kPairs / tiles, kb / 4, kMaxSplits})));
  return p;
}

// The workspace begins with its count of waits that gave up, which the calls
// add to and zero_lm_workspace_status reads and clears.
constexpr int64_t kStatusBytes = 256;

// Byte offsets of the workspace's parts: the masked hidden vectors, D of two
// pieces (one is formed while the other is used), dh's fp32 sums, and a tile
// counter for each launch with a word for lost tiles after them.
struct GradSpace {
  int64_t hidden, probs[2], acc, counters, total;
};

GradSpace grad_space(int64_t tokens, int64_t vocab, int64_t width, const GradPlan& p) {
  const int64_t pieces = ceil_div(vocab, p.piece);
  GradSpace s;
  s.hidden = kStatusBytes;
  s.probs[0] = s.hidden + round_up(tokens * width * 2, 256);
  s.probs[1] = s.probs[0] + round_up(tokens * p.piece * 2, 256);
  s.acc = s.probs[1] + (pieces > 1 ? s.probs[1] - s.probs[0] : 0);
  s.counters = s.acc + round_up(p.splits * tokens * width * 4, 256);
  s.total = s.counters + round_up((pieces + 2) * 4, 256);
  return s;
}

// Up to so many tokens the loss's operands change places: the vocabulary takes
// the 256 rows of a tile and the tokens its columns, so that the products take
// no time for rows that are not there; joining the columns over the lanes takes
// time for each 32 tokens instead, whatever the width.  Exchanged and with the
// tokens as rows, us, the same tables call after call (bf16):
//            50257 x 768  50257 x 1600  32000 x 2048  50257 x 128  8000 x 256
//   64       15.3  22.5   32.7  35.7    28.6  30.7    11.3  13.3   7.2  8.0
//   96       18.3  20.1   34.3  35.9    30.4  30.8    15.5  13.6   9.0  8.1
//   128      19.3  20.2   34.7  36.0    30.9  31.0    16.5  13.6   9.0  8.1
// Models of usual widths gain a little up to 128 tokens, the narrowest lose
// from about 96 on; one limit for all widths lies between.
constexpr int64_t kFewTokens = 96;

// The loss goes over the tokens in slabs: its partial sums take 16 bytes for
// each token and 256 columns, which must not grow with the batch.
constexpr int64_t kSlab = 32768;

int64_t loss_space(int64_t tokens, int64_t vocab) {
  tokens = std::min(tokens, kSlab);
  const int64_t tiles = ceil_div(vocab, kTileN);
  const int64_t parts = std::max(tokens * tiles, std::min(tokens, kFewTokens) * tiles * 4);
  return kStatusBytes + round_up(parts * 16, 256) + round_up(tokens * 4, 256);
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
  // any smaller count of tokens has to fit too: its pieces may be wider and its sums split more often.  With
  // fewer tokens D of a piece takes at most kPieceBytes, or less than kMinPiece rows of all the tokens would
  const int64_t wide = round_up(vocab, 256);
  const int64_t piece = std::max(std::min(tokens * std::min(wide, kMinPiece) * 2, std::max(kMostPieceBytes, tokens * kLeastPiece * 2)),
                                 std::min(tokens * wide * 2, kPieceBytes));
  const int64_t probs = 2 * piece;
  const int64_t sums = std::max(tokens, std::min<int64_t>(tokens * kMaxSplits, kPairs * kTileM)) * round_up(width, 256) * 4;
  const int64_t counters = (ceil_div(vocab, kLeastPiece) + 2) * 4;
  return std::max(bytes, kStatusBytes + round_up(tokens * width * 2, 256) + round_up(probs, 512) + round_up(sums, 256) +
                             round_up(counters, 256));
}

extern "C" int zero_lm_loss(int64_t tokens, int64_t vocab, int64_t width, int dtype, const void* hidden,
                            int64_t hidden_stride, const void* table, int64_t table_stride, const void* targets,
                            int id_bytes, float* loss, float* lse, void* workspace, int64_t workspace_bytes,
                            void* stream) {
  bool stall = take_stall();
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
  for (int64_t t0 = 0; t0 < tokens; t0 += kSlab) {
    const int64_t count = std::min(kSlab, tokens - t0);
    const void* slab_targets = static_cast<const char*>(targets) + t0 * id_bytes;
    GemmArgs g;
    std::memset(&g, 0, sizeof g);
    Job& j = g.job[0];
    // rows and columns of the product: tokens and vocabulary, or for a few tokens the other way round
    const bool few = count <= kFewTokens;
    j.kind = few ? kFew : kStats;
    j.M = static_cast<int>(few ? vocab : count);
    j.N = static_cast<int>(few ? count : vocab);
    j.bn = few ? static_cast<int>(round_up(count, 32)) : kTileN;
    j.m_tiles = static_cast<int>(ceil_div(j.M, kTileM));
    j.n_tiles = static_cast<int>(ceil_div(j.N, j.bn));
    j.splits = 1;
    j.tiles = j.m_tiles * j.n_tiles;
    j.kb_total = static_cast<int>(ceil_div(width, kTileK));
    j.stage_tx = 2 * (kOperandBytes + j.bn / 2 * kTileK * 2);
    const int parts = few ? j.m_tiles * 8 : j.n_tiles * 2;   // of a token
    g.jobs = 1;
    g.vocab = static_cast<int>(vocab);
    g.targets = slab_targets;
    g.id_bytes = id_bytes;
    g.failures = static_cast<unsigned int*>(workspace);
    char* space = static_cast<char*>(workspace) + kStatusBytes;
    g.part = reinterpret_cast<float2*>(space);
    g.target_logit = reinterpret_cast<float*>(space + round_up(count * parts * 8, 256));
    const uint16_t* rows = static_cast<const uint16_t*>(hidden) + t0 * hidden_stride;
    CUtensorMap *of_tokens = few ? &g.b[0] : &g.a[0], *of_vocab = few ? &g.a[0] : &g.b[0];
    if ((rc = make_map(of_tokens, dtype, rows, count, width, hidden_stride, few ? j.bn / 2 : 128))) return rc;
    if ((rc = make_map(of_vocab, dtype, table, vocab, width, table_stride, few ? 128 : j.bn / 2))) return rc;
    if ((rc = launch_gemm<false>(g, dtype, s, stall))) return rc;
    const int team = few ? kSmallThreads : 32;
    const dim3 grid(static_cast<unsigned>(ceil_div(count * team, kSmallThreads)));
    ZERO_CUDA(launch_chained(few ? lm_combine<kSmallThreads> : lm_combine<32>, grid, kSmallThreads, 0, s, g.part, parts,
                             g.target_logit, slab_targets, id_bytes, g.vocab, static_cast<int>(count), loss + t0,
                             lse + t0));
  }
  return ZERO_OK;
}

extern "C" int zero_lm_loss_grad(int64_t tokens, int64_t vocab, int64_t width, int dtype, const void* hidden,
                                 int64_t hidden_stride, const void* table, int64_t table_stride, const void* targets,
                                 int id_bytes, const float* lse, double scale, void* dhidden, int64_t dhidden_stride,
                                 void* dtable, int64_t dtable_stride, int accumulate, void* workspace,
                                 int64_t workspace_bytes, void* stream) {
  bool stall = take_stall();
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
  const GradSpace sp = grad_space(tokens, vocab, width, p);
  if (workspace_bytes < sp.total)
    return fail(ZERO_E_ARG, "workspace of %lld bytes: %lld are needed", (long long)workspace_bytes,
                (long long)sp.total);
  char* ws = static_cast<char*>(workspace);
  uint16_t* masked = reinterpret_cast<uint16_t*>(ws + sp.hidden);
  float* acc = reinterpret_cast<float*>(ws + sp.acc);
  unsigned int* counters = reinterpret_cast<unsigned int*>(ws + sp.counters);
  const int width8 = static_cast<int>(width / 8);
  const int64_t pieces = ceil_div(vocab, p.piece), items = tokens * width8;
  unsigned int* lost = counters + pieces + 1;
  ZERO_CUDA(launch_chained(lm_masked_hidden, dim3(small_grid(items)), kSmallThreads, 0, s,
                           static_cast<const uint16_t*>(hidden), hidden_stride, width8, targets, id_bytes,
                           static_cast<int>(vocab), static_cast<int>(tokens), masked, counters,
                           static_cast<int>(pieces + 2)));
  const float unscale = static_cast<float>(scale) / (dtype == ZERO_FP16 ? d_scale<__half>() : d_scale<__nv_bfloat16>());

  // Launch k forms D of piece k and multiplies with D of piece k - 1.
  for (int64_t k = 0; k <= pieces; ++k) {
    GemmArgs g;
    std::memset(&g, 0, sizeof g);
    g.next = counters + k;
    g.lost = lost;
    g.failures = static_cast<unsigned int*>(workspace);
    g.vocab = static_cast<int>(vocab);
    g.targets = targets;
    g.id_bytes = id_bytes;
    g.lse = lse;
    if (k > 0) {
      const int64_t v0 = (k - 1) * p.piece, w = std::min(p.piece, vocab - v0);
      const void* probs = ws + sp.probs[(k - 1) & 1];
      // the piece's share of dh, and its rows of the table's gradient: the longer tiles first
      Job dh{}, dt{};
      dh.kind = kDHidden;
      dh.bn = dt.bn = p.bn;
      dh.b_boxes = dt.b_boxes = static_cast<int>(ceil_div(p.bn / 2, 64));
      dh.stage_tx = dt.stage_tx = 2 * (kOperandBytes + dh.b_boxes * 8192);
      dh.n_tiles = dt.n_tiles = static_cast<int>(ceil_div(width, p.bn));
      dh.N = dt.N = static_cast<int>(width);
      dh.m_tiles = static_cast<int>(ceil_div(tokens, kTileM));
      dh.kb_total = static_cast<int>(ceil_div(w, kTileK));
      dh.splits = std::min(p.splits, dh.kb_total);
      dh.M = static_cast<int>(tokens);
      dh.b_row0 = static_cast<int>(v0);
      dh.acc = acc;
      dh.add = v0 > 0;
      dt.kind = kDTable;
      dt.m_tiles = static_cast<int>(ceil_div(w, kTileM));
      dt.kb_total = static_cast<int>(ceil_div(tokens, kTileK));
      dt.splits = 1;
      dt.M = static_cast<int>(w);
      dt.out16 = static_cast<uint16_t*>(dtable) + v0 * dtable_stride;
      dt.out_stride = dtable_stride;
      dt.add = accumulate != 0;
      dt.wide = width % 16 == 0 && dtable_stride % 16 == 0 && host::aligned32(dtable);
      dt.scale = unscale;
      const bool table_first = dt.kb_total >= dh.kb_total / dh.splits;
      const int at_h = table_first ? 1 : 0, at_t = 1 - at_h;
      dh.tiles = dh.m_tiles * dh.n_tiles * dh.splits;
      dt.tiles = dt.m_tiles * dt.n_tiles;
      g.job[at_h] = dh;
      g.job[at_t] = dt;
      if ((rc = make_map(&g.a[at_h], dtype, probs, tokens, w, p.piece, 128))) return rc;
      if ((rc = make_map(&g.b[at_h], dtype, table, vocab, width, table_stride, 64))) return rc;
      if ((rc = make_map(&g.a[at_t], dtype, probs, tokens, w, p.piece, 64))) return rc;
      if ((rc = make_map(&g.b[at_t], dtype, masked, tokens, width, width, 64))) return rc;
      g.jobs = 2;
    }
    if (k < pieces) {
      const int64_t v0 = k * p.piece, w = std::min(p.piece, vocab - v0);
      Job& j = g.job[g.jobs];
      j.kind = kProbs;
      j.bn = kTileN;
      j.m_tiles = static_cast<int>(ceil_div(tokens, kTileM));
      j.n_tiles = static_cast<int>(ceil_div(w, kTileN));
      j.splits = 1;
      j.tiles = j.m_tiles * j.n_tiles;
      j.kb_total = static_cast<int>(ceil_div(width, kTileK));
      j.M = static_cast<int>(tokens);
      j.N = static_cast<int>(w);
      j.stage_tx = 2 * kStageBytes;
      j.b_row0 = j.vocab0 = static_cast<int>(v0);
      j.out16 = ws + sp.probs[k & 1];
      j.out_stride = p.piece;
      if ((rc = make_map(&g.a[g.jobs], dtype, masked, tokens, width, width, 128))) return rc;
      if ((rc = make_map(&g.b[g.jobs], dtype, table, vocab, width, table_stride, kTileN / 2))) return rc;
      ++g.jobs;
    }
    if ((rc = launch_gemm<true>(g, dtype, s, stall))) return rc;
  }
  const auto finish = [&](auto* dh, auto* dt) {
    using T = std::remove_pointer_t<decltype(dh)>;
    const auto fn = p.splits > 1 ? lm_finish_dhidden<T, kFinishBatch> : lm_finish_dhidden<T, 1>;
    return launch_chained(fn, dim3(small_grid(items)), kSmallThreads, 0, s, acc, p.splits, tokens, width8, unscale, dh,
                          dhidden_stride, lost, dt, vocab, dtable_stride);
  };
  ZERO_CUDA(dtype == ZERO_FP16 ? finish(static_cast<__half*>(dhidden), static_cast<__half*>(dtable))
                               : finish(static_cast<__nv_bfloat16*>(dhidden), static_cast<__nv_bfloat16*>(dtable)));
  return ZERO_OK;
}

extern "C" int zero_lm_workspace_status(void* workspace, void* stream) {
  if (workspace == nullptr) return fail(ZERO_E_ARG, "workspace is NULL");
  if (reinterpret_cast<uintptr_t>(workspace) % 256) return fail(ZERO_E_ALIGN, "workspace must be 256-byte aligned");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  unsigned int n = 0;
  ZERO_CUDA(cudaMemcpyAsync(&n, workspace, sizeof n, cudaMemcpyDeviceToHost, s));
  ZERO_CUDA(cudaStreamSynchronize(s));
  if (n == 0) return ZERO_OK;
  ZERO_CUDA(cudaMemsetAsync(workspace, 0, sizeof n, s));
  return fail(ZERO_E_STATE, "%u bounded device waits gave up; the losses or gradients they belonged to are incomplete", n);
}

extern "C" int zero_lm_status(void* stream) {
  // The device's count only grows: what one call reports cannot be lost to another's clearing of it.
  constexpr int kDevices = 64;
  static std::mutex mutex;
  static unsigned int seen[kDevices];
  int device = 0;
  ZERO_CUDA(cudaGetDevice(&device));
  if (device >= kDevices) return fail(ZERO_E_ARG, "device %d: %d are supported", device, kDevices);
  ZERO_CUDA(cudaStreamSynchronize(static_cast<cudaStream_t>(stream)));
  std::lock_guard<std::mutex> lock(mutex);
  unsigned int n = 0;
  ZERO_CUDA(cudaMemcpyFromSymbol(&n, g_lm_timeouts, sizeof n));
  const unsigned int fresh = n - seen[device];
  seen[device] = n;
  if (fresh == 0) return ZERO_OK;
  return fail(ZERO_E_STATE, "%u bounded device waits gave up on the device; what they belonged to is incomplete", fresh);
}

extern "C" int zero_lm_inject_stall(void) {
  g_stall_next = true;
  return ZERO_OK;
}
