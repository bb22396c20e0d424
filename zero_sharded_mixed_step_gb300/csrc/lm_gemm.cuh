// The products of a language model's head with a large vocabulary, shared by the
// cross entropy (lm_loss.cu) and the log probabilities (lm_logprobs.cu): the
// tensor-core kernel with its epilogues, what a gradient's launches need around
// it, and how a call is cut up.  lm_loss.cu says what is computed and what
// bounds it.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cstdint>
#include <cmath>
#include <cstring>
#include <type_traits>
#include <utility>

#include "launch.cuh"
#include "step_math.cuh"
#include "tensor_map.h"
#include "umma.cuh"
#include "zero_context.h"
#include "zero_internal.h"
#include "zero_step.h"

namespace zero {

namespace {

// Bounded device-side waits of this file's lm_gemm that gave up, over all calls; never set back (see zero_lm_status).
__device__ unsigned int g_lm_timeouts;

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
constexpr int kStashBytes = kEpilogueWarps * 32 * 32 * 4;   // kLogprobs: 32 columns of each row of a warp

// What a launch computes: the loss's partial sums, its gradient's products, the
// same for log probabilities with entropy and alternatives, and for their
// gradients, where every token has weights of its own.
enum Mode : int { kLoss, kGrad, kLogprobs, kWeighted };
constexpr int kFewK = -1;
__host__ __device__ constexpr bool is_grad(int mode) { return mode == kGrad || mode == kWeighted; }

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
  // kLogprobs: partial sums (maximum of the plain logits, sum of exponentials, and of exponentials times exponents)
  // at [pair + row tile][row][half of its columns] or, kFew, [token][32 rows of the vocabulary], and the K largest
  // logits with their columns beside them, or, kFew, the logits as [token][logit_stride]
  float4* sums;
  int2* best;
  float* logits;
  int64_t logit_stride;
  float scale2;                // the logits' scale times log2(e); kWeighted too
  // kWeighted: what comes back for each token, its entropy, and the bits of the largest bound of D (NULL: bf16)
  const float *dlogp, *dentropy, *entropy;
  const unsigned int* largest;
};

// What fp16 scales the weighted D by: a power of two that keeps |D|, at most
// `largest`, below 2^14 and as far above the subnormals as that allows.
__device__ __forceinline__ int weighted_exponent(const unsigned int* largest) {
  if (largest == nullptr) return 0;
  const float most = __uint_as_float(*largest);
  return most > 0.f ? min(max(13 - ilogbf(most), -100), 100) : 0;
}

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

// Tile t of a launch of one job, neighbours along a row one after another, up to `end`.
__device__ __forceinline__ Tile along_row(const GemmArgs& g, int t, int end) {
  Tile x{};
  const unsigned n_tiles = g.job[0].n_tiles;
  x.job = t < end ? 0 : -1;
  x.mt = static_cast<int>(static_cast<unsigned>(t) / n_tiles);
  x.nt = t - x.mt * static_cast<int>(n_tiles);
  x.k1 = g.job[0].kb_total;
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
  float weight, tilt, at_target;   // kWeighted: D = p (weight + tilt log2 p) + at_target [v = target]
};

// Whether token i takes part in a weighted gradient: it has a target and a weight.
__device__ __forceinline__ bool has_weight(const float* dlogp, const float* dentropy, int64_t i) {
  return dlogp[i] != 0.f || (dentropy != nullptr && dentropy[i] != 0.f);
}

template <int MODE>
__device__ __forceinline__ RowInfo row_info(const GemmArgs& g, const Job& j, int row) {
  constexpr bool GRAD = is_grad(MODE);
  RowInfo r{-1, 0.f, 0.f, 0.f, 0.f};
  if ((GRAD ? j.kind != kProbs : j.kind != kStats) || row >= j.M) return r;
  r.target = load_target(g.targets, g.id_bytes, row, g.vocab);
  if (GRAD) r.lse = g.lse[row];
  if (MODE == kWeighted) {
    // d logp / d z = onehot - p,  d entropy / d z = -p (log p + entropy)
    const float a = g.dlogp[row], b = g.dentropy ? g.dentropy[row] : 0.f;
    const float unit = exp2f(static_cast<float>(weighted_exponent(g.largest)));
    if (r.target >= 0 && !has_weight(g.dlogp, g.dentropy, row)) r.target = -1;
    if (r.target >= 0) {
      r.weight = b == 0.f ? -a * unit : -fmaf(b, g.entropy[row], a) * unit;
      r.tilt = -b * kLn2 * unit;
      r.at_target = a * unit;
    }
  }
  return r;
}

// A row's running sums over the columns that a thread has seen: the maximum of
// the logits, and with x = z - z_max in powers of 2 (z the scaled logits)
//   sum = sum of 2^x,   tilt = sum of 2^x x,
// so that lse = ln 2 (z_max + log2 sum) and the entropy is ln 2 (log2 sum -
// tilt / sum), two terms of one sign.  And the K largest logits, the first of
// equal ones first, since a thread's columns come in ascending order.
template <int K>
struct RowState {
  float top, sum, tilt;
  float best[K > 0 ? K : 1];
  int id[K > 0 ? K : 1];

  __device__ __forceinline__ void clear() {
    top = -INFINITY;
    sum = tilt = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      best[k] = -INFINITY;
      id[k] = -1;
    }
  }
  __device__ __forceinline__ void insert(float v, int at) {
#pragma unroll
    for (int k = K - 1; k >= 0; --k) {
      const bool here = v > best[k], before = k > 0 && v > best[k > 0 ? k - 1 : 0];
      if (here) {
        best[k] = before ? best[k > 0 ? k - 1 : 0] : v;
        id[k] = before ? id[k > 0 ? k - 1 : 0] : at;
      }
    }
  }
};

// Exponents below this are taken as this where they multiply their power of 2,
// which is 0 by then: a logit of -infinity adds 0 to the entropy.
constexpr float kLeastExponent = -200.f;

// The reference that sums of exponentials are relative to, from the plain maximum.
__device__ __forceinline__ float reference(float top, float scale2) { return top == -INFINITY ? 0.f : top * scale2; }

// sum and tilt, relative to `from`, made relative to `to` (-infinity: of no
// column yet, both 0, or none at all, both NaN).
__device__ __forceinline__ void rebase(float& sum, float& tilt, float from, float to) {
  const float d = from - to, f = exp2_fast(d);
  tilt = f * fmaf(fmaxf(d, kLeastExponent), sum, tilt);
  sum *= f;
}

// One tile's columns of this thread's row joined to its running sums.  `stash`
// is 32 x 32 floats of this warp's shared memory: where a column of some row
// may enter its list, the 32 columns go there, since which registers do is
// known at run time alone.  That is rare: a row's chance is K / (columns seen).
template <int K, typename R>
__device__ __forceinline__ void scan_logprobs(const GemmArgs& g, const Job& j, const Tile& x, RowState<K>& st,
                                              int target, uint32_t tmem, int row, int half, float* stash, R release) {
  const int n0 = x.nt * j.bn, lane = threadIdx.x & 31;
  const float scale2 = g.scale2;
  target -= n0;
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
    if (m > st.top) {
      rebase(st.sum, st.tilt, st.top * scale2, m * scale2);
      st.top = m;
    }
    if (K > 0 && __any_sync(0xffffffffu, m > st.best[K - 1])) {
      unsigned some = 0;
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        stash[k * 32 + lane] = v[k];
        some |= (v[k] > st.best[K - 1] ? 1u : 0u) << k;
      }
      // each lane its own columns, from left to right; it reads what it wrote itself
      while (__any_sync(0xffffffffu, some != 0)) {
        const int k = __ffs(static_cast<int>(some)) - 1;
        if (some != 0) st.insert(stash[k * 32 + lane], n0 + c + k);
        some &= some - 1;
      }
    }
    const float ref = reference(st.top, scale2);
    float s0 = 0.f, s1 = 0.f, t0 = 0.f, t1 = 0.f;
#pragma unroll
    for (int k = 0; k < 32; k += 2) {
      const float x0 = fmaf(v[k], scale2, -ref), x1 = fmaf(v[k + 1], scale2, -ref);
      const float e0 = exp2_fast(x0), e1 = exp2_fast(x1);
      s0 += e0;
      s1 += e1;
      t0 = fmaf(e0, fmaxf(x0, kLeastExponent), t0);
      t1 = fmaf(e1, fmaxf(x1, kLeastExponent), t1);
    }
    st.sum += s0 + s1;
    st.tilt += t0 + t1;
  }, release);
}

template <int K>
__device__ __forceinline__ void store_state(const GemmArgs& g, const RowState<K>& st, int64_t at) {
  g.sums[at] = make_float4(st.top, st.sum, st.tilt, 0.f);
#pragma unroll
  for (int k = 0; k < K; ++k) g.best[at * K + k] = make_int2(__float_as_int(st.best[k]), st.id[k]);
}

// kFew's sums: a thread holds one row of the vocabulary, its columns are the
// tokens, each joined over the 32 rows of the warp.
template <typename R>
__device__ __forceinline__ void few_logprobs(const GemmArgs& g, const Job& j, const Tile& x, uint32_t tmem, int row,
                                             int half, R release) {
  const int lane = threadIdx.x & 31, n0 = x.nt * j.bn;
  const bool row_ok = row < j.M;
  for_columns_plain(tmem, half * 32, j.bn, [&](int c, float (&v)[32]) {
    const int token = n0 + c + lane;
    const int target = token < j.N ? load_target(g.targets, g.id_bytes, token, g.vocab) : -1;
    float y[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      if (__shfl_sync(0xffffffffu, target, k) == row) g.target_logit[n0 + c + k] = v[k];
      if (!row_ok) v[k] = -INFINITY;
      if (g.logits != nullptr && n0 + c + k < j.N) g.logits[(n0 + c + k) * g.logit_stride + row] = v[k];
      y[k] = v[k];
    }
    const float top = join_lanes(y, lane, [](float a, float b) { return fmaxf(a, b); });
    const float ref = reference(top, g.scale2);
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const float e = fmaf(v[k], g.scale2, -__shfl_sync(0xffffffffu, ref, k));
      v[k] = exp2_fast(e);
      y[k] = v[k] * fmaxf(e, kLeastExponent);
    }
    const float sum = join_lanes(v, lane, [](float a, float b) { return a + b; });
    const float tilt = join_lanes(y, lane, [](float a, float b) { return a + b; });
    if (token < j.N) g.sums[static_cast<int64_t>(token) * (j.m_tiles * 8) + row / 32] = make_float4(top, sum, tilt, 0.f);
  }, release);
}

template <typename T, int MODE, typename R>
__device__ __forceinline__ void epilogue(const GemmArgs& g, const Job& j, const Tile& x, const RowInfo& info,
                                         uint32_t tmem, int row, int half, R release) {
  constexpr bool GRAD = is_grad(MODE);
  const int n0 = x.nt * j.bn;
  const bool row_ok = row < j.M;
  if (MODE == kLogprobs) {
    few_logprobs(g, j, x, tmem, row, half, release);
    return;
  }
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
    const float to2 = MODE == kWeighted ? g.scale2 : kLog2e;
    T* out = static_cast<T*>(j.out16) + static_cast<int64_t>(row) * j.out_stride + n0;
    for_columns(tmem, half * 32, j.bn, [&](int c, float (&v)[32]) {
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        const float y = fmaf(v[k], to2, -ref);     // log2 of the probability
        // a probability of 0 counts as 2^-200 in the entropy's term, so that 0 times infinity is 0
        v[k] = MODE == kWeighted ? exp2_fast(y) * fmaf(info.tilt, fmaxf(y, -200.f), info.weight)
                                 : exp2_fast(y) * d_scale<T>();
      }
      if (local >= c && local < c + 32) {
#pragma unroll
        for (int k = 0; k < 32; ++k)
          if (local == c + k) v[k] += MODE == kWeighted ? info.at_target : -d_scale<T>();
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
    const float scale = MODE == kWeighted ? j.scale * exp2f(static_cast<float>(-weighted_exponent(g.largest))) : j.scale;
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
            w[q] = j.add ? fmaf(p, scale, w[q]) : p * scale;
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
template <int MODE>
__device__ __forceinline__ void spoil_parts(const GemmArgs& g, const Job& j, const Tile& x, int row, int half) {
  const float2 none = make_float2(-INFINITY, NAN);
  if (j.kind == kStats) {
    if (row < j.M) g.part[(static_cast<int64_t>(row) * j.n_tiles + x.nt) * 2 + half] = none;
    return;
  }
  for (int c = half * 32; c < j.bn; c += 64) {
    const int token = x.nt * j.bn + c + static_cast<int>(threadIdx.x & 31);
    if (token >= j.N) continue;
    const int64_t at = static_cast<int64_t>(token) * (j.m_tiles * 8) + row / 32;
    if (MODE == kLogprobs) g.sums[at] = make_float4(-INFINITY, NAN, NAN, 0.f);
    else g.part[at] = none;
  }
}

// The persistent product kernel: pairs of CTAs, each pair one 256-row tile at
// a time, operands through a ring of TMA stages, two accumulators in TMEM so
// that one tile's epilogue runs beside the next one's products.  The loss's
// tiles are all alike and are dealt out in turn.  The gradient's differ: one
// thread of the pair takes them from a counter, in the order of the jobs, the
// longest tiles first, so that the short ones fill the gaps at the end, and
// hands them to the roles of both CTAs through a short queue in shared memory.
// Log probabilities go over each row's columns in stretches, a pair's tiles
// being neighbours along a row, so that a thread's running sums and list pass
// from tile to tile and are written once for each stretch of a row.
// K: the length of their lists, or kFewK for a few tokens as columns.
template <typename T, int MODE, int K = 0>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) lm_gemm(const __grid_constant__ GemmArgs g) {
  constexpr bool GRAD = is_grad(MODE), kStretches = MODE == kLogprobs && K != kFewK;
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
  const int stretch0 = kStretches ? static_cast<int>(int64_t{g.job[0].tiles} * pair / pairs) : 0;
  const int stretch1 = kStretches ? static_cast<int>(int64_t{g.job[0].tiles} * (pair + 1) / pairs) : 0;
  auto tile_of = [&](int i) {
    if (kStretches) return along_row(g, stretch0 + i, stretch1);
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
    // kLogprobs: the row tile that the running sums belong to, and where they go
    RowState<(K > 0 ? K : 0)> st;
    int group = -1, target = -1;
    auto place = [&](int mt) {
      return (static_cast<int64_t>(pair + mt) * kTileM + static_cast<int>(rank) * 128 + quad * 32 + lane) * 2 + half;
    };
    int i = 0;
    for (;; ++i) {
      const int a = i & 1;
      const Tile x = tile_of(i);
      if (!ok || x.job < 0) break;
      const Job& j = jobs[x.job];
      const int row = row_of(x);
      const RowInfo info = row_info<MODE>(g, j, row);
      if (kStretches && x.mt != group) {
        if (group >= 0) store_state(g, st, place(group));
        st.clear();
        group = x.mt;
        target = info.target;
      }
      ok = wait_all(done(a), (i >> 1) & 1);
      if (!ok) break;
      fence_after();
      const uint32_t at = tmem + a * kTileN + (static_cast<uint32_t>(quad) << 21);
      auto release = [&] {
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(in_cta(taken(a), 0));
      };
      if constexpr (kStretches)
        scan_logprobs(g, j, x, st, target, at, row, half,
                      reinterpret_cast<float*>(raw + (ring - smem_addr(raw)) + kStages * kStageBytes) + (warp - 4) * 1024,
                      release);
      else
        epilogue<T, MODE>(g, j, x, info, at, row, half, release);
    }
    if (kStretches && ok && group >= 0) store_state(g, st, place(group));
    if (!ok) {
      if (lane == 0) failed = 1;
      if (kStretches) {
        // this stretch of the row, whatever it holds so far, and the pair's others
        st.clear();
        st.sum = st.tilt = NAN;
        for (int mt = group; mt <= (stretch1 - 1) / g.job[0].n_tiles; ++mt) store_state(g, st, place(mt));
      } else if (!GRAD) {
        // this tile and the pair's others
        for (;; ++i) {
          const Tile x = tile_of(i);
          if (x.job < 0) break;
          spoil_parts<MODE>(g, jobs[x.job], x, row_of(x), half);
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

// The largest bound of |D| over the tokens first, first + step, ... of a weighted
// gradient, as the bits of a float: |a| + |b| (entropy + 1/e) for the weights a
// and b, since |p log p| <= 1/e.  Weights that are not finite leave no bound; their
// D is none either.
__device__ __forceinline__ unsigned int largest_weight(const void* targets, int id_bytes, int vocab, int tokens,
                                                       const float* dlogp, const float* dentropy, const float* entropy,
                                                       int64_t first, int64_t step) {
  float most = 0.f;
  for (int64_t i = first; i < tokens; i += step) {
    if (load_target(targets, id_bytes, i, vocab) < 0) continue;
    const float b = dentropy ? dentropy[i] : 0.f;
    const float bound = fabsf(dlogp[i]) + (b == 0.f ? 0.f : fabsf(b) * (fabsf(entropy[i]) + 0.36788f));
    if (isfinite(bound)) most = fmaxf(most, bound);
  }
  return __float_as_uint(most);
}

// The hidden vectors with the rows of tokens without target set to 0: such a
// row times D's zeros must add nothing to the table's gradient even where it
// holds an infinity or a NaN.  WEIGHTED: a token whose weights are 0 counts as one
// without target.  Also sets the products' tile counters, and the words after
// them (whether a tile was lost; WEIGHTED: the largest bound of D), to 0.
template <bool WEIGHTED>
__global__ void __launch_bounds__(kSmallThreads) lm_masked_hidden(const uint16_t* hidden, int64_t stride, int width8,
                                                                  const void* targets, int id_bytes, int vocab,
                                                                  int tokens, uint16_t* out, unsigned int* counters,
                                                                  int n_counters, const float* dlogp,
                                                                  const float* dentropy, const float* entropy,
                                                                  unsigned int* largest) {
  allow_next();
  await_previous();
  if (blockIdx.x == 0)
    for (int k = threadIdx.x; k < n_counters; k += kSmallThreads)
      if (!WEIGHTED || counters + k != largest) counters[k] = 0;
  if (WEIGHTED && largest != nullptr && blockIdx.x == gridDim.x - 1) {
    // few tokens: the largest bound of D too, by one block
    __shared__ unsigned int most;
    if (threadIdx.x == 0) most = 0;
    __syncthreads();
    const unsigned int mine = __reduce_max_sync(
        0xffffffffu, largest_weight(targets, id_bytes, vocab, tokens, dlogp, dentropy, entropy, threadIdx.x, kSmallThreads));
    if ((threadIdx.x & 31) == 0) atomicMax(&most, mine);
    __syncthreads();
    if (threadIdx.x == 0) *largest = most;
  }
  const int64_t total = static_cast<int64_t>(tokens) * width8;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * kSmallThreads + threadIdx.x; e < total;
       e += static_cast<int64_t>(gridDim.x) * kSmallThreads) {
    const int64_t row = e / width8, c = e - row * width8;
    uint4 x = make_uint4(0, 0, 0, 0);
    if (load_target(targets, id_bytes, row, vocab) >= 0 && (!WEIGHTED || has_weight(dlogp, dentropy, row)))
      x = dev::ld_16B(hidden + row * stride + c * 8);
    dev::st_16B(out + e * 8, x);
  }
}

// The same by a launch of its own, for many tokens; `largest` is 0 before.
__global__ void __launch_bounds__(kSmallThreads) lm_largest_weight(const void* targets, int id_bytes, int vocab,
                                                                   int tokens, const float* dlogp,
                                                                   const float* dentropy, const float* entropy,
                                                                   unsigned int* largest) {
  allow_next();
  await_previous();
  const unsigned int of_warp = __reduce_max_sync(
      0xffffffffu, largest_weight(targets, id_bytes, vocab, tokens, dlogp, dentropy, entropy,
                                  static_cast<int64_t>(blockIdx.x) * kSmallThreads + threadIdx.x,
                                  static_cast<int64_t>(gridDim.x) * kSmallThreads));
  if ((threadIdx.x & 31) == 0 && of_warp != 0) atomicMax(largest, of_warp);
}
// Up to so many tokens it is found beside the hidden vectors' copy, by one block, which saves a launch.  Beside it and
// in a launch of its own, us a gradient: 129 x 2000 x 256 22.6 and 24.7, 1024 26.7 and 26.7, 4096 49.3 and 45.2, 16384
// 178 and 121; 129 x 8000 x 768 34.9 and 36.7, 1024 51.2 and 51.3, 4096 131 and 119, 16384 526 and 489.
constexpr int64_t kFewWeights = 1024;

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
                                                                   int64_t dtable_stride, const unsigned int* largest) {
  allow_next();
  await_previous();
  scale *= exp2f(static_cast<float>(-weighted_exponent(largest)));
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
using host::encoder;
using host::EncodeFn;
using host::fail;
using host::round_up;

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

// Whether this call, the thread's next one, was to lose a block of operands.
bool take_stall() { return std::exchange(g_stall_next, false); }

// What the cutting up reckons with: the pairs among GB300's 152 SMs.
constexpr int64_t kPairs = 76;

// Pairs of CTAs for so many tiles.
int pairs_for(int64_t tiles) {
  return static_cast<int>(std::min({std::max<int64_t>(1, sm_count() / 2), kPairs, tiles}));
}

// Launch the products; `stall` is handed to the first launch of a call alone.
template <int MODE, int K = 0>
int launch_gemm(GemmArgs& g, int dtype, cudaStream_t s, bool& stall) {
  g.stall = std::exchange(stall, false);
  const auto fn = dtype == ZERO_FP16 ? lm_gemm<__half, MODE, K> : lm_gemm<__nv_bfloat16, MODE, K>;
  constexpr int kSmem = kGemmSmem + (K > 0 ? kStashBytes : 0);
  ZERO_CUDA(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem));
  int64_t tiles = 0;
  for (int k = 0; k < g.jobs; ++k) tiles += g.job[k].tiles;
  ZERO_CUDA(launch_chained(fn, dim3(2 * pairs_for(tiles)), kThreads, kSmem, s, g));
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
// counter for each launch with `words` words after the last piece's: its own, one
// for lost tiles and, of a weighted gradient, one for the largest bound of D.
struct GradSpace {
  int64_t hidden, probs[2], acc, counters, total;
};

GradSpace grad_space(int64_t tokens, int64_t vocab, int64_t width, const GradPlan& p, int64_t words = 2) {
  const int64_t pieces = ceil_div(vocab, p.piece);
  GradSpace s;
  s.hidden = kStatusBytes;
  s.probs[0] = s.hidden + round_up(tokens * width * 2, 256);
  s.probs[1] = s.probs[0] + round_up(tokens * p.piece * 2, 256);
  s.acc = s.probs[1] + (pieces > 1 ? s.probs[1] - s.probs[0] : 0);
  s.counters = s.acc + round_up(p.splits * tokens * width * 4, 256);
  s.total = s.counters + round_up((pieces + words) * 4, 256);
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

// Bytes with which any count of up to `tokens` tokens has its gradient.
int64_t grad_bytes(int64_t tokens, int64_t vocab, int64_t width, int64_t words = 2) {
  // any smaller count of tokens has to fit too: its pieces may be wider and its sums split more often.  With
  // fewer tokens D of a piece takes at most kPieceBytes, or less than kMinPiece rows of all the tokens would
  const int64_t wide = round_up(vocab, 256);
  const int64_t piece = std::max(std::min(tokens * std::min(wide, kMinPiece) * 2, std::max(kMostPieceBytes, tokens * kLeastPiece * 2)),
                                 std::min(tokens * wide * 2, kPieceBytes));
  const int64_t probs = 2 * piece;
  const int64_t sums = std::max(tokens, std::min<int64_t>(tokens * kMaxSplits, kPairs * kTileM)) * round_up(width, 256) * 4;
  const int64_t counters = (ceil_div(vocab, kLeastPiece) + words) * 4;
  return kStatusBytes + round_up(tokens * width * 2, 256) + round_up(probs, 512) + round_up(sums, 256) +
         round_up(counters, 256);
}

// One gradient call's arguments, and what a weighted one has beside them.
struct GradCall {
  int64_t tokens, vocab, width;
  int dtype;
  const void* hidden;
  int64_t hidden_stride;
  const void* table;
  int64_t table_stride;
  const void* targets;
  int id_bytes;
  const float* lse;
  double scale;
  void* dhidden;
  int64_t dhidden_stride;
  void* dtable;
  int64_t dtable_stride;
  int accumulate;
  void* workspace;
  int64_t workspace_bytes;
  cudaStream_t stream;
  const float *dlogp = nullptr, *dentropy = nullptr, *entropy = nullptr;
  double logit_scale = 1.0;
};

// The launches of a gradient; its arguments have been checked.
template <int MODE>
int run_grad(const GradCall& c, bool& stall) {
  const int64_t tokens = c.tokens, vocab = c.vocab, width = c.width, table_stride = c.table_stride;
  const int64_t hidden_stride = c.hidden_stride, dhidden_stride = c.dhidden_stride, dtable_stride = c.dtable_stride;
  const int dtype = c.dtype, id_bytes = c.id_bytes, accumulate = c.accumulate;
  const void *hidden = c.hidden, *table = c.table, *targets = c.targets;
  void *dhidden = c.dhidden, *dtable = c.dtable, *workspace = c.workspace;
  const float *lse = c.lse, *dlogp = c.dlogp, *dentropy = c.dentropy, *entropy = c.entropy;
  const cudaStream_t s = c.stream;
  int rc;
  if (tokens == 0) {
    // no token: the table's gradient is 0
    if (!accumulate)
      ZERO_CUDA(cudaMemset2DAsync(dtable, dtable_stride * 2, 0, width * 2, vocab, s));
    return ZERO_OK;
  }
  constexpr bool kOwnWeights = MODE == kWeighted;
  constexpr int64_t kWords = kOwnWeights ? 3 : 2;
  const GradPlan p = plan_grad(tokens, vocab, width);
  const GradSpace sp = grad_space(tokens, vocab, width, p, kWords);
  if (c.workspace_bytes < sp.total)
    return fail(ZERO_E_ARG, "workspace of %lld bytes: %lld are needed", (long long)c.workspace_bytes,
                (long long)sp.total);
  char* ws = static_cast<char*>(workspace);
  uint16_t* masked = reinterpret_cast<uint16_t*>(ws + sp.hidden);
  float* acc = reinterpret_cast<float*>(ws + sp.acc);
  unsigned int* counters = reinterpret_cast<unsigned int*>(ws + sp.counters);
  const int width8 = static_cast<int>(width / 8);
  const int64_t pieces = ceil_div(vocab, p.piece), items = tokens * width8;
  unsigned int* lost = counters + pieces + 1;
  unsigned int* largest = kOwnWeights && dtype == ZERO_FP16 ? lost + 1 : nullptr;
  const bool few_weights = tokens <= kFewWeights;
  ZERO_CUDA(launch_chained(lm_masked_hidden<kOwnWeights>, dim3(small_grid(items)), kSmallThreads, 0, s,
                           static_cast<const uint16_t*>(hidden), hidden_stride, width8, targets, id_bytes,
                           static_cast<int>(vocab), static_cast<int>(tokens), masked, counters,
                           static_cast<int>(pieces + kWords), dlogp, dentropy, entropy, few_weights ? largest : nullptr));
  float unscale = static_cast<float>(c.scale);
  if (kOwnWeights) {
    if (largest != nullptr && !few_weights) {
      ZERO_CUDA(launch_chained(lm_largest_weight, dim3(small_grid(tokens)), kSmallThreads, 0, s, targets, id_bytes,
                               static_cast<int>(vocab), static_cast<int>(tokens), dlogp, dentropy, entropy, largest));
    }
  } else {
    unscale /= dtype == ZERO_FP16 ? d_scale<__half>() : d_scale<__nv_bfloat16>();
  }

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
    g.dlogp = dlogp;
    g.dentropy = dentropy;
    g.entropy = entropy;
    g.largest = largest;
    g.scale2 = static_cast<float>(c.logit_scale) * kLog2e;
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
    if ((rc = launch_gemm<MODE>(g, dtype, s, stall))) return rc;
  }
  const auto finish = [&](auto* dh, auto* dt) {
    using T = std::remove_pointer_t<decltype(dh)>;
    const auto fn = p.splits > 1 ? lm_finish_dhidden<T, kFinishBatch> : lm_finish_dhidden<T, 1>;
    return launch_chained(fn, dim3(small_grid(items)), kSmallThreads, 0, s, acc, p.splits, tokens, width8, unscale, dh,
                          dhidden_stride, lost, dt, vocab, dtable_stride, largest);
  };
  ZERO_CUDA(dtype == ZERO_FP16 ? finish(static_cast<__half*>(dhidden), static_cast<__half*>(dtable))
                               : finish(static_cast<__nv_bfloat16*>(dhidden), static_cast<__nv_bfloat16*>(dtable)));
  return ZERO_OK;
}

}  // namespace
}  // namespace zero
