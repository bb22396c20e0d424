// Orthogonalising a matrix by Newton-Schulz products, and the optimizer step
// that takes its direction from it (Muon).
//
//   X_0 = G / |G|_F, taken over its shorter side (m x n, m <= n)
//   A = X X^T,   P = a I + b A + c A^2,   X <- P X      for each step's (a, b, c)
//
// Every step maps the singular values by s -> a s + b s^3 + c s^5; the usual
// coefficients bring them near 1.  The step is, for each matrix of many,
//   g = (G_0 + ... + G_{W-1}) / W,   M <- mu M + g,   U = g + mu M or M,
//   theta <- theta (1 - lr wd) - lr s X(U),   16-bit copy <- theta
//
// Small matrices run in shared memory (muon_small.cu).  The others take three
// launches: two passes over the input, which find the norm and write X_0, and one
// persistent tensor-core kernel, ns_run, for all the steps.  Matrices of one
// shape (or its transpose) lie one after another in the workspace, X as m x n
// always, so that a 3-D tensor map loads any of them.  The work is a list of
// tiles of 256 rows, one product after another:
//   kGram   A, the blocks of 256 x 256 on and below the diagonal; what lies
//           above is read from there, rows and columns exchanged
//   kPoly   A A likewise, with P formed in its epilogue
//   kApply  P X; of the last step its epilogue writes the caller's matrix or
//           updates the master and the 16-bit copy in place.
//   kMultiply  of wide matrices (n >= 2 m), whose steps go by twos: with P_0 of A
//           the second A is P_0 A P_0, the second P, P_1, of that, and X <- P_1 P_0 X:
//           3 n / m + 5 units of work for two steps instead of 6 n / m + 2
// Pairs of CTAs take tiles from a counter in the list's order; a tile waits until
// every tile of its matrix's product before has been written, which another
// counter for each matrix says.  What a tile waits for has a lower number, so
// some running pair has it or has done it, and no wait can last for ever.  With
// several matrices a pair finds tiles that are ready; one product's tail runs
// beside the next one's start (with two steps in two parts, whose products' own
// time is about 226 us, 24 matrices of 768 x 768 took 490 us as 15 launches and
// take 368).
// Precision.  A singular value far below 1 grows by `a` (3.4) a step, and with
// it the noise that rounding X, A and P to 16 bits leaves in its direction:
// with fp16 operands throughout, a matrix whose largest singular values stand
// 20 times above the rest comes out 1.4e-2 off (Frobenius norm of the difference
// over the result's), with bf16 11e-2.  So in the first `fine` steps every
// operand is a sum of two fp16 parts (22 bits) and a product three products of
// parts.  A bf16 result takes them in all steps but the last, after which nothing
// grows: what that one leaves, 3e-4 to 9e-4 over the spectra of zero_step.h,
// stays below the result's own rounding of 1.7e-3 (two such steps leave up to
// 4e-3).  fp16 results, whose own rounding is 2.1e-4, fp32 results and the step,
// which writes an fp32 master, take all steps in two parts.
// X and A are stored times 2^12, P times 2^9: entries of fp16's normal range.
// The first X is the input times a power of two, the rest of 1 / |G| (between
// 1/2 and 1) being applied in the epilogues: a 16-bit input is then exact in
// one part.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <map>
#include <new>
#include <type_traits>
#include <utility>
#include <vector>

#include "launch.cuh"
#include "ns_common.cuh"
#include "step_math.cuh"
#include "tensor_map.h"
#include "umma.cuh"
#include "zero_context.h"
#include "zero_internal.h"
#include "zero_step.h"

namespace zero {
namespace {

using namespace umma;
using namespace ns;
using dev::Fmt;
using host::ceil_div;
using host::cuda_fail;
using host::fail;
using host::round_up;

// Bounded device-side waits of ns_run that gave up, over all calls; never set back (see zero_lm_status).
__device__ unsigned int g_ns_timeouts;

constexpr int kTileM = 256;          // rows of a tile: 128 in each CTA of the pair
constexpr int kTileN = 256;          // most columns of a tile
constexpr int kTileK = 64;
constexpr int kSlotBytes = 128 * kTileK * 2;     // one part of one operand's half tile in one CTA
// A stage of the operands' ring: one part of A and of B for one block of K.  A
// block in two parts takes two stages, the high parts first.
constexpr int kStages = 7, kStageBytes = 2 * kSlotBytes;
// warp 0 loads A, warp 3 loads B, warp 1 issues the products, warps 4-19 are the
// epilogue, four for each quarter of the TMEM lanes taking 16 columns in turn
// (two for each, 32 columns at a time, took twice as long for a tile, which the
// next product waits for), warp 2 says what they have written, and in the leader
// warp 20 takes the tiles
constexpr int kThreads = 672;
constexpr int kEpilogueWarps = 16, kTakerWarp = 20;
constexpr int kCols = 16;            // of a row that an epilogue thread holds at a time
constexpr int kQueue = 4;            // tiles on their way through a pair
constexpr int kRunSmem = kStages * kStageBytes + 1024;
constexpr int kMaxGroups = 12;       // shapes of one launch, whose parameters hold no more than 32,764 bytes
constexpr int64_t kPairs = 76;       // pairs of CTAs among GB300's 152 SMs
// Blocks of K that one accumulator takes in the steps in two parts of an fp32 result.  The tensor core cuts its sums
// to 24 bits at every instruction, always towards 0: 430 x 1321 came out 2.6e-5 off, growing with the size.  The
// epilogue adds up the accumulators of a tile, rounding to nearest, in TMEM beside them.  Whole tiles, 4, 2 blocks and
// 1 leave 24 matrices of 768 x 768 2.8e-5, 1.1e-5, 6.3e-6 and 3.9e-6 off (plain fp32 2.6e-6) in 527, 609, 669 and 757
// us; 2048 x 2048 takes 443, 479, 498 and 536.
constexpr int kSegment = 1;
// Columns of every tile of such a launch at most: an accumulator's neighbour in TMEM takes the sums, which are read
// while the next tile's first products run.
constexpr int kSegmentTile = 128, kSumsAt = 128;
static_assert(kSumsAt >= kSegmentTile && kSumsAt + kSegmentTile <= kTileN);

enum Kind : int { kGram, kPoly, kMultiply, kApply };
enum Final : int { kLast, kUpdate };       // what the last product does
enum Buffer : int { kX0, kX1, kA, kP, kT, kBuffers };
constexpr float kScaleT = 2048.f;          // of P A while two steps are joined
constexpr int kMaxPhases = 7 * kMaxSteps / 2;

// A product of a shape's list.
struct Phase {
  int8_t kind, a, b, out;            // its operands' and result's buffers
  int8_t step, parts_a, parts_b, two;   // kPoly: whose coefficients; the operands' parts; whether a low part is written
  int8_t units, fine, last, unused;  // powers of what the first X lacks of the norm; two parts in this step; the last
  float factor;                      // from the sums to what is written
};
// What the width of the tiles goes by.
__host__ __device__ constexpr int class_of(int kind) { return kind == kGram ? 0 : kind == kApply ? 2 : 1; }

// The matrices of one shape.
struct Shape {
  CUtensorMap box128[kBuffers], box64[kBuffers], box32[kBuffers];   // loads of so many rows x 64
  uint16_t* at[kBuffers];
  int matrices, first;               // how many, the first one's entry
  int m, n;
  int joined;                        // which list
  int bn[2][3];                      // columns of a tile by class: 64, 128 or 256; of one part, of two
  int tiles[2][3];                   // of one matrix
  int64_t ldx, lda, apart_x, apart_a, part_x, part_a;    // rows, matrices, parts
};

struct RunArgs {
  Shape shape[kMaxGroups];
  Phase phase[2][kMaxPhases];  // steps one by one, and by twos
  int phases[2];
  int shapes;
  int dtype;                   // kLast: of the results; kUpdate: of the 16-bit copies
  int stall;                   // testing the bounded waits: the first tile's first block of K never arrives
  int segment;                 // blocks of K for one accumulator in fine steps; 0: a tile's
  const Entry* entries;
  const Norm* norms;
  unsigned int* next;          // tiles taken so far (0 at the launch)
  unsigned int* exits;         // CTAs that have ended (0)
  unsigned int* written;       // for each matrix: halves of tiles written (0)
  unsigned int* failures;      // the workspace's count of waits that gave up
  unsigned int* lost;          // set where tiles of this call were not computed (0)
  int entries_here;            // of these shapes, from shape[0].first on
  float coefficients[3 * kMaxSteps];
};
static_assert(sizeof(RunArgs) <= 32764);

// What the roles of a pair need to know of a tile.
struct alignas(16) Tile {
  int kind;                    // -1: no more
  int shape, matrix, mt;
  int nt, phase, kb, bn;       // kb: blocks of K
};

// Tiles of a row of tiles that hold something on or below the diagonal.
__host__ __device__ inline int tiles_of_row(int mt, int bn, int n_tiles) {
  const int reach = (mt + 1) * (kTileM / bn);
  return reach < n_tiles ? reach : n_tiles;
}

// Where in the list a pair is: its tiles come in rising order.
struct Cursor {
  int phase = 0, shape = 0;
  unsigned start = 0;          // the first tile of this phase and shape
};

// Tile t of the list, at or after the cursor.  before[h]: the tiles of one
// matrix's products before, for each shape up to the cursor.
__device__ __forceinline__ Tile locate(const RunArgs& g, unsigned t, Cursor& c, unsigned* before) {
  Tile x = {};
  unsigned each = 0;
  for (;;) {
    const Shape& h = g.shape[c.shape];
    each = 0;
    if (c.phase < g.phases[h.joined]) {
      const Phase& f = g.phase[h.joined][c.phase];
      each = h.tiles[f.fine][class_of(f.kind)];
    }
    const unsigned count = each * h.matrices;
    if (t < c.start + count) break;
    c.start += count;
    __syncwarp();
    if ((threadIdx.x & 31) == 0) before[c.shape] += each;
    __syncwarp();
    if (++c.shape < g.shapes) continue;
    c.shape = 0;
    if (++c.phase < max(g.phases[0], g.phases[1])) continue;
    x.kind = -1;
    return x;
  }
  const Shape& h = g.shape[c.shape];
  const Phase& f = g.phase[h.joined][c.phase];
  x.kind = f.kind;
  x.shape = c.shape;
  x.phase = c.phase;
  unsigned r = t - c.start;
  x.matrix = static_cast<int>(r / each);
  r -= x.matrix * each;
  const int bn = x.bn = h.bn[f.fine][class_of(f.kind)];
  if (f.kind == kApply) {
    const unsigned m_tiles = (h.m + kTileM - 1) / kTileM;
    x.nt = static_cast<int>(r / m_tiles);
    x.mt = static_cast<int>(r - x.nt * m_tiles);
  } else {
    const int n_tiles = (h.m + bn - 1) / bn;
    for (;;) {
      const unsigned n = tiles_of_row(x.mt, bn, n_tiles);
      if (r < n) break;
      r -= n;
      ++x.mt;
    }
    x.nt = static_cast<int>(r);
  }
  x.kb = ((f.kind == kGram ? h.n : h.m) + kTileK - 1) / kTileK;
  return x;
}

// Blocks of K of one accumulator of a tile.
__device__ __forceinline__ int segment_of(const RunArgs& g, const Phase& f, const Tile& x) {
  return f.parts_a > 1 && g.segment > 0 ? g.segment : x.kb;
}

__device__ __forceinline__ const Phase& phase_of(const RunArgs& g, const Tile& x) {
  return g.phase[g.shape[x.shape].joined][x.phase];
}

// Of the symmetric matrices the blocks above the diagonal are not there: block kb of K of the
// operand whose rows begin at `row` is read with rows and columns exchanged
// where its columns lie in a later block of 256 than its rows.
__device__ __forceinline__ bool exchanged(int row, int kb) { return kb * kTileK / kTileM > row / kTileM; }

// Whether block kb of K of a tile's B has K as its row index, and the bytes of B's
// half tile for one CTA: rows of K-major, or whole boxes of 64 columns.
__device__ __forceinline__ bool b_is_mn(const Tile& x, int kb) {
  return x.kind == kApply || (x.kind != kGram && exchanged(x.nt * x.bn, kb));
}
__device__ __forceinline__ uint32_t b_bytes(const Tile& x, int kb) {
  const int half = x.bn / 2;
  return (b_is_mn(x, kb) ? (half + 63) / 64 * 64 : half) * kTileK * 2;
}

// ---- the epilogues -------------------------------------------------------------------

// 16 columns from col0 of this thread's row, v, in one or two parts, in rows of
// multiples of 16 values from a 32-byte boundary.
__device__ __forceinline__ void store_block(uint16_t* out, int64_t ld, int64_t part, int rows, int cols, int row, int col0,
                                            const float (&v)[kCols], bool two) {
  if (row >= rows || col0 >= cols) return;
  uint4 hi[2], lo[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float w[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) w[q] = v[8 * k + q];
    split8(w, hi[k], lo[k]);
  }
  uint16_t* to = out + row * ld + col0;
  st_32B_words(to, hi[0], hi[1]);
  if (two) st_32B_words(to + part, lo[0], lo[1]);
}

// 16 bytes that another SM wrote while this kernel ran: past L1.
__device__ __forceinline__ uint4 ld_fresh(const void* p) {
  uint4 r;
  asm volatile("ld.global.cg.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
  return r;
}

// What the epilogue reads beside the sums for 16 columns of a row, fetched
// before the sums are there: A's values of both parts (kPoly), or the master's.
struct Beside {
  uint4 w[4];
};

template <int FINAL>
__device__ __forceinline__ void fetch(const RunArgs& g, const Tile& x, int row, int c, Beside& b) {
  const Shape& h = g.shape[x.shape];
  const int col0 = x.nt * x.bn + c;
  const Phase& f = phase_of(g, x);
  if (x.kind == kPoly) {
    if (row >= h.m || col0 >= h.m) return;
    // A's rows are padded to 16 values: what is read past the last column is not used
    const uint16_t* a = h.at[f.a] + x.matrix * h.apart_a + row * h.lda + col0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      b.w[k] = ld_fresh(a + 8 * k);
      if (f.fine) b.w[2 + k] = ld_fresh(a + h.part_a + 8 * k);
    }
  } else if (FINAL == kUpdate && f.last) {
    if (row >= h.m || col0 >= h.n) return;
    read_master<kCols>(g.entries[h.first + x.matrix], h.n, row, col0, b.w);
  }
}

// A tile's columns of this thread's row: the accumulator's, and the sums of
// those before it, if any.
struct Sums {
  uint32_t tmem, before;
  bool some;                   // there are sums of accumulators before

  __device__ __forceinline__ void load(int c, float (&v)[kCols]) const {
    tmem_ld16(tmem + c, v);
    tmem_ld_wait(v);
    if (!some) return;
    float w[kCols];
    tmem_ld16(before + c, w);
    tmem_ld_wait(w);
#pragma unroll
    for (int k = 0; k < kCols; ++k) v[k] += w[k];
  }
  // The accumulator joins the sums.
  __device__ __forceinline__ void keep(int first, int bn) const {
#pragma unroll 1
    for (int c = first; c < bn; c += 64) {
      float v[kCols];
      load(c, v);
      tmem_st16(before + c, v);
    }
    tmem_st_wait();
  }
};

// 16 columns at a time from `first` in steps of 64; `release` runs when the
// last ones are in registers.
template <typename F, typename R>
__device__ __forceinline__ void each_16(const Sums& sums, int first, int bn, F f, R release) {
#pragma unroll 1
  for (int c = first; c < bn; c += 64) {
    float v[kCols];
    sums.load(c, v);
    if (c + 64 >= bn) release();
    f(c, v);
  }
}

template <int FINAL, typename R>
__device__ __forceinline__ void epilogue(const RunArgs& g, const Tile& x, const Sums& sums, Beside& b, int row,
                                         int share, R release) {
  const Shape& h = g.shape[x.shape];
  const int bn = x.bn, n0 = x.nt * bn;
  const int which = h.first + x.matrix;
  const Phase& f = phase_of(g, x);
  float scale = f.factor;
  if (f.units > 0) {
    const float unit = g.norms[which].unit;
    scale *= f.units > 1 ? unit * unit : unit;
  }
  const bool two = f.two;
  if (x.kind == kGram || x.kind == kMultiply) {
    uint16_t* out = h.at[f.out] + x.matrix * h.apart_a;
    each_16(sums, share * kCols, bn, [&](int c, float (&v)[kCols]) {
#pragma unroll
      for (int k = 0; k < kCols; ++k) v[k] *= scale;
      store_block(out, h.lda, h.part_a, h.m, h.m, row, n0 + c, v, two);
    }, release);
  } else if (x.kind == kPoly) {
    uint16_t* out = h.at[f.out] + x.matrix * h.apart_a;
    const float a = g.coefficients[3 * f.step] * kScaleP, once = g.coefficients[3 * f.step + 1] * (kScaleP / kScaleA);
    const float square = g.coefficients[3 * f.step + 2] * (kScaleP / (kScaleA * kScaleA));
    each_16(sums, share * kCols, bn, [&](int c, float (&v)[kCols]) {
      const int col0 = n0 + c;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float u[8], l[8] = {};
        Fmt<__half>::unpack8(b.w[k], u);
        if (f.fine) Fmt<__half>::unpack8(b.w[2 + k], l);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          v[8 * k + q] = fmaf(once, u[q] + l[q], square * v[8 * k + q]);
          if (row == col0 + 8 * k + q) v[8 * k + q] += a;
        }
      }
      if (c + 64 < bn) fetch<FINAL>(g, x, row, c + 64, b);
      store_block(out, h.lda, h.part_a, h.m, h.m, row, col0, v, two);
    }, release);
  } else if (!f.last) {
    uint16_t* out = h.at[f.out] + x.matrix * h.apart_x;
    each_16(sums, share * kCols, bn, [&](int c, float (&v)[kCols]) {
#pragma unroll
      for (int k = 0; k < kCols; ++k) v[k] *= scale;
      store_block(out, h.ldx, h.part_x, h.m, h.n, row, n0 + c, v, two);
    }, release);
  } else {
    const Entry& e = g.entries[which];
    const bool finite = g.norms[which].finite;
    if (!finite) scale = NAN;
    each_16(sums, share * kCols, bn, [&](int c, float (&v)[kCols]) {
      // a norm that is not finite leaves the state as it was
      if (row >= h.m || n0 + c >= h.n || (FINAL == kUpdate && !finite)) return;
#pragma unroll
      for (int k = 0; k < kCols; ++k) v[k] *= scale;
      if (FINAL == kUpdate) {
        step_master<kCols>(e, b.w, v);
        if (c + 64 < bn) fetch<FINAL>(g, x, row, c + 64, b);
      }
      write_columns<FINAL == kUpdate>(h.n, e, g.dtype, row, n0 + c, v);
    }, release);
  }
}

__device__ __forceinline__ unsigned ld_acquire(const unsigned* p) {
  unsigned v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void add_release(unsigned* p, unsigned v) {
  asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// All the steps of the matrices of a launch: see above.  Operands through a ring
// of TMA stages, two accumulators in TMEM so that one tile's epilogue runs beside
// the next one's products.
template <int FINAL>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) ns_run(const __grid_constant__ RunArgs g) {
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) uint64_t bars[2 * kStages + 3 * kQueue + 6];
  __shared__ Tile queue[kQueue];
  __shared__ uint32_t tmem_slot;
  __shared__ unsigned before[kMaxGroups];
  __shared__ int failed, last_out;
  const uint32_t ring = (smem_addr(raw) + 1023u) & ~1023u;
  const uint32_t bar0 = smem_addr(bars);
  auto full = [&](int s) { return bar0 + 8 * s; };
  auto empty = [&](int s) { return bar0 + 8 * (kStages + s); };
  auto done = [&](int a) { return bar0 + 8 * (2 * kStages + a); };        // accumulator a is complete
  auto taken = [&](int a) { return bar0 + 8 * (2 * kStages + 2 + a); };   // accumulator a has been read
  const uint32_t drained = bar0 + 8 * (2 * kStages + 4);
  auto told = [&](int q) { return bar0 + 8 * (2 * kStages + 5 + q); };             // queue[q] holds a tile
  auto heard = [&](int q) { return bar0 + 8 * (2 * kStages + 5 + kQueue + q); };   // everyone has read it
  auto stored = [&](int q) { return bar0 + 8 * (2 * kStages + 5 + 2 * kQueue + q); };  // this CTA's half of the tile is
  const uint32_t began = bar0 + 8 * (2 * kStages + 5 + 3 * kQueue);                    // the leader loads the next tile
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();

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
    bar_init(began, 1);
    for (int q = 0; q < kQueue; ++q) {
      bar_init(told(q), 1);
      bar_init(heard(q), 7 + 2 * kEpilogueWarps);   // the loaders, the issuer, the warps 2, the epilogue
      bar_init(stored(q), kEpilogueWarps);
    }
    bar_init(drained, 1);
    failed = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc(smem_addr(&tmem_slot), 512);
  __syncthreads();
  fence_before();
  cluster_sync();
  fence_after();
  const uint32_t tmem = tmem_slot;
  await_previous();

  const bool lead = elect_one();
  bool ok = true;
  auto wait_all = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, bar_wait(bar, parity)) != 0; };
  // The i-th tile of this pair, from the leader's last warp.
  auto tile_of = [&](int i) {
    Tile x{};
    x.kind = -1;
    const int q = i % kQueue;
    ok = __all_sync(0xffffffffu, bar_wait<true>(told(q), (i / kQueue) & 1)) != 0;
    if (!ok) return x;
    x = queue[q];
    __syncwarp();
    if (lead) bar_arrive(in_cta(heard(q), 0));
    return x;
  };

  int issued = 0;      // stages loaded by this warp
  if (warp == 0 || warp == 3) {
    int s = 0;
    uint32_t phase = 1;
    const bool first = warp == 0, stall = g.stall && blockIdx.x < 2;
    for (int i = 0;; ++i) {
      const Tile x = tile_of(i);
      if (!ok || x.kind < 0) break;
      if (first && rank == 0 && lead) bar_arrive_own(began);
      // what other CTAs' threads wrote is loaded through the async proxy
      fence_async_global();
      const Shape& h = g.shape[x.shape];
      const Phase& f = phase_of(g, x);
      const int bn = x.bn, depth = h.matrices, blocks = x.kb, parts_a = f.parts_a, parts_b = f.parts_b;
      // K-major, and boxes of 64 columns with K as the row index
      const int buffer = first ? f.a : f.b;
      const CUtensorMap* map = first || bn == 256 ? &h.box128[buffer] : bn == 128 ? &h.box64[buffer] : &h.box32[buffer];
      const CUtensorMap* map64 = &h.box64[buffer];
      // this CTA's rows (or columns) of the operand
      const int at = first ? x.mt * kTileM + static_cast<int>(rank) * 128 : x.nt * bn + static_cast<int>(rank) * (bn / 2);
      const bool second_box = first || bn == kTileN, counts = first && rank == 0;
      for (int kb = 0; kb < blocks; ++kb) {
        const bool mn = first ? x.kind != kGram && exchanged(x.mt * kTileM, kb) : b_is_mn(x, kb);
        const uint32_t of_b = 2 * b_bytes(x, kb);
        const int k = kb * kTileK;
        for (int part = 0; part < parts_a; ++part, ++issued) {
          // A stage without B is none of the second warp's: it may be used, and emptied, before that warp comes by,
          // and a wait for a phase that is two back never ends.
          const bool with_b = part < parts_b;
          if (first || with_b) ok = wait_all(empty(s), phase);
          if (!ok) break;
          if (lead && (first || with_b)) {
            const uint32_t bar = in_cta(full(s), 0), to = ring + s * kStageBytes + (first ? 0 : kSlotBytes);
            const int z = x.matrix + part * depth;
            if (counts) bar_expect(full(s), 2 * kSlotBytes + (with_b ? of_b : 0));
            if (first && stall && issued == 0) {
            } else if (mn) {
              tma_load3(to, map64, at, k, z, bar);
              if (second_box) tma_load3(to + 8192, map64, at + 64, k, z, bar);
            } else {
              tma_load3(to, map, k, at, z, bar);
            }
          }
          __syncwarp();
          if (++s == kStages) {
            s = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
      }
      if (!ok) break;
    }
    if (!ok && lead) failed = 1;
  } else if (warp == 1) {
    if (rank == 0) {
      int s = 0, turn = 0;     // accumulators begun
      uint32_t phase = 0;
      for (int i = 0;; ++i) {
        const Tile x = tile_of(i);
        if (!ok || x.kind < 0) break;
        const Phase& f = phase_of(g, x);
        const uint32_t idesc = instr_desc(false, false, false, kTileM, x.bn);
        const int blocks = x.kb, a_row = x.mt * kTileM, segment = segment_of(g, f, x);
        uint32_t d = 0;
        int a = 0;
        auto begin = [&] {
          a = turn & 1;
          ok = wait_all(taken(a), ((turn >> 1) & 1) ^ 1);
          if (!ok) return;
          fence_after();
          d = tmem + a * kTileN;
          ++turn;
        };
        begin();
        if (!ok) break;
        // 16 values of K further: 32 bytes within a K-major row, 16 rows of an MN-major tile
        const uint64_t a_k = operand_desc(ring, 0), a_mn = operand_desc(ring, 8192);
        const uint64_t b_k = operand_desc(ring + kSlotBytes, 0), b_mn = operand_desc(ring + kSlotBytes, 8192);
        // the tile's blocks of K in PA and PB parts, known here for the instructions to follow one another closely
        auto run = [&](auto pa, auto pb) {
          constexpr int PA = decltype(pa)::value, PB = decltype(pb)::value;
          int first = 0;       // block of this accumulator
          for (int kb = 0; kb < blocks; ++kb) {
            if (PA > 1 && kb == first + segment) {
              if (lead) mma_commit(done(a));
              __syncwarp();
              begin();
              if (!ok) break;
              first = kb;
            }
            const bool of_a = x.kind != kGram && exchanged(a_row, kb), of_b = b_is_mn(x, kb);
            const uint64_t a_step = of_a ? 128 : 2, b_step = of_b ? 128 : 2;
            const uint32_t id = idesc | (of_a ? 1u << 15 : 0u) | (of_b ? 1u << 16 : 0u);
            ok = wait_all(full(s), phase);
            if (!ok) break;
            fence_after();
            const int high = s;
            const uint64_t da = (of_a ? a_mn : a_k) + s * (kStageBytes >> 4), db = (of_b ? b_mn : b_k) + s * (kStageBytes >> 4);
            if (lead) {
#pragma unroll
              for (int q = 0; q < kTileK / 16; ++q) mma(d, da + q * a_step, db + q * b_step, id, kb > first || q > 0);
              if (PA == 1) mma_commit(empty(s));
            }
            __syncwarp();
            if (++s == kStages) {
              s = 0;
              phase ^= 1;
            }
            if (PA == 1) continue;
            ok = wait_all(full(s), phase);
            if (!ok) break;
            fence_after();
            const uint64_t la = (of_a ? a_mn : a_k) + s * (kStageBytes >> 4), lb = (of_b ? b_mn : b_k) + s * (kStageBytes >> 4);
            if (lead) {
              // of two parts each, the product of the low ones is left out: 2^-22 of the whole
#pragma unroll
              for (int q = 0; q < kTileK / 16; ++q) {
                mma(d, la + q * a_step, db + q * b_step, id, true);
                if (PB > 1) mma(d, da + q * a_step, lb + q * b_step, id, true);
              }
              mma_commit(empty(high));
              mma_commit(empty(s));
            }
            __syncwarp();
            if (++s == kStages) {
              s = 0;
              phase ^= 1;
            }
          }
        };
        using One = std::integral_constant<int, 1>;
        using Two = std::integral_constant<int, 2>;
        if (f.parts_a == 1) run(One{}, One{});
        else if (f.parts_b == 1) run(Two{}, One{});
        else run(Two{}, Two{});
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
    // A tile's stores are on their way when the epilogue is done with it; saying so takes until they have arrived.
    for (int i = 0;; ++i) {
      const Tile x = tile_of(i);
      if (!ok || x.kind < 0) break;
      ok = wait_all(stored(i % kQueue), (i / kQueue) & 1);
      if (!ok) break;
      if (lead) {
        add_release(g.written + g.shape[x.shape].first + x.matrix, 1u);
      }
      __syncwarp();
    }
    if (!ok && lead) failed = 1;
  } else if (warp == kTakerWarp) {
    // Takes the next tile when the leader begins to load the one before, waits for what it needs, and tells the roles.
    Cursor cursor;
    if (lane < kMaxGroups) before[lane] = 0;
    __syncwarp();
    for (int i = 0; rank == 0; ++i) {
      const int q = i % kQueue;
      ok = wait_all(heard(q), ((i / kQueue) & 1) ^ 1);
      if (ok && i > 0) ok = wait_all(began, (i - 1) & 1);
      if (!ok) break;
      unsigned t = 0;
      if (lead) t = atomicAdd(g.next, 1u);
      t = __reduce_max_sync(0xffffffffu, t);
      const Tile x = locate(g, t, cursor, before);
      if (x.kind >= 0 && before[x.shape] > 0) {
        const unsigned* p = g.written + g.shape[x.shape].first + x.matrix;
        const unsigned want = before[x.shape] * 2;
        bool there = true;
        if (lead) {
          const long long t0 = clock64();
          while (there && ld_acquire(p) < want) there = clock64() - t0 <= kWaitCycles;
        }
        ok = __all_sync(0xffffffffu, there) != 0;
        if (!ok) break;
      }
      if (lead) {
        for (uint32_t r = 0; r < 2; ++r) {
          const uint32_t at = in_cta(smem_addr(&queue[q]), r);
          st_cluster(at, x.kind, x.shape, x.matrix, x.mt);
          st_cluster(at + 16, x.nt, x.phase, x.kb, x.bn);
          bar_arrive_written(in_cta(told(q), r));
        }
      }
      __syncwarp();
      if (x.kind < 0) break;
    }
    if (!ok && lead) failed = 1;
  } else if (warp >= 4) {
    const int quad = warp & 3, share = (warp - 4) >> 2;
    const uint32_t my_lanes = tmem + (static_cast<uint32_t>(quad) << 21);
    Beside beside = {};
    int turn = 0;              // accumulators read
    for (int i = 0;; ++i) {
      const Tile x = tile_of(i);
      if (!ok || x.kind < 0) break;
      const int row = x.mt * kTileM + static_cast<int>(rank) * 128 + quad * 32 + lane;
      fetch<FINAL>(g, x, row, share * kCols, beside);
      const int segment = segment_of(g, phase_of(g, x), x);
      Sums sums = {0, my_lanes + kSumsAt, false};
      int a = 0;
      auto next = [&] {
        a = turn & 1;
        ok = wait_all(done(a), (turn >> 1) & 1);
        fence_after();
        sums.tmem = my_lanes + a * kTileN;
        ++turn;
      };
      auto release = [&] {
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(in_cta(taken(a), 0));
      };
      next();
      for (int k = segment; ok && k < x.kb; k += segment) {
        sums.keep(share * kCols, x.bn);
        sums.some = true;
        release();
        next();
      }
      if (!ok) break;
      epilogue<FINAL>(g, x, sums, beside, row, share, release);
      __syncwarp();
      // Warps may be a tile or two apart, not as many as there are barriers: of two tiles' products, at most, some warp
      // has not read the sums.
      if (lane == 0) bar_arrive_own(stored(i % kQueue));
    }
    if (!ok && lane == 0) failed = 1;
  }
  __syncthreads();
  if (failed) {
    if (threadIdx.x == 0) {
      atomicAdd(&g_ns_timeouts, 1u);
      atomicAdd(g.failures, 1u);
      *g.lost = 1;
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
  if (FINAL == kUpdate) return;
  // where tiles were lost it is not known which: the last CTA to end makes every result of the launch no number
  if (threadIdx.x == 0) {
    __threadfence();
    last_out = atomicAdd(g.exits, 1u) == gridDim.x - 1;
    __threadfence();
  }
  __syncthreads();
  if (!last_out || ld_acquire(g.lost) == 0) return;
  for (int k = 0; k < g.entries_here; ++k) {
    const Entry& e = g.entries[g.shape[0].first + k];
    const int64_t count = static_cast<int64_t>(e.rows) * e.cols;
    for (int64_t i = threadIdx.x; i < count; i += kThreads) {
      const int64_t r = i / e.cols, at = r * e.out_stride + (i - r * e.cols);
      if (g.dtype == ZERO_FP32) static_cast<float*>(e.out)[at] = NAN;
      else static_cast<uint16_t*>(e.out)[at] = pack1(g.dtype, NAN);
    }
  }
}

// ---- the passes before the products ------------------------------------------------------
//
// Both go over tiles of 32 rows x 256 columns of the caller's matrices.

constexpr int kPassBlocksPerSm = 8;
// Up to this many ranks the second pass reads the gradients again (2 W bytes an
// element) instead of their fp32 mean, which costs 8.
constexpr int kDirectRanks = 2;

template <int BYTES>
__global__ void __launch_bounds__(kPassThreads) copy_table(const __grid_constant__ TablePart<BYTES> part, int words,
                                                           uint64_t* to, unsigned int* counters, int n_counters) {
  allow_next();
  await_previous();
  for (int k = threadIdx.x; k < words; k += kPassThreads) to[k] = reinterpret_cast<const uint64_t*>(part.data)[k];
  for (int k = threadIdx.x; k < n_counters; k += kPassThreads) counters[k] = 0;
}

// The entry that tile t belongs to, found by a whole warp: 32 of the entries
// left are looked at together.
__device__ __forceinline__ int entry_of(const Entry* entries, int count, unsigned t) {
  int first = 0;
  while (count > 1) {
    const int apart = (count + 31) / 32, at = static_cast<int>(threadIdx.x & 31) * apart;
    const bool reached = at < count && entries[first + at].tile0 <= t;
    const int found = (__popc(__ballot_sync(0xffffffffu, reached)) - 1) * apart;
    first += found;
    count = min(apart, count - found);
  }
  return first;
}

// The tiles of one block of a pass: a stretch of all of them.
__device__ __forceinline__ unsigned stretch(unsigned tiles, unsigned block) {
  return static_cast<unsigned>(static_cast<uint64_t>(tiles) * block / gridDim.x);
}

// The first tile past those of entry `which`.
__device__ __forceinline__ unsigned end_of(const PassArgs& p, int which) {
  return which + 1 < p.count ? p.entries[which + 1].tile0 : p.tiles;
}

// The first pass: sums of squares, in fp32 within a thread (see Squares) and in fp64 beyond
// (and the mean gradient, kept where that pays).  A block goes over a stretch of
// the tiles and leaves a sum for each matrix that it meets, at [block + entry].
// WC > 0: so many ranks, known at compile time; 0: any number (8 ranks, whose
// loads are many anyway, took 120 us so for 28M elements, and 139 to 161 with
// WC = 8).
template <typename T, bool MUON, int WC>
__global__ void __launch_bounds__(kPassThreads) sum_squares(const __grid_constant__ PassArgs p) {
  allow_next();
  await_previous();
  const unsigned t1 = stretch(p.tiles, blockIdx.x + 1);
  for (unsigned t = stretch(p.tiles, blockIdx.x); t < t1;) {
    const int which = entry_of(p.entries, p.count, t);
    const Entry& e = p.entries[which];
    const int across = (e.cols + kPassCols - 1) / kPassCols;
    const unsigned tile0 = e.tile0, end = min(t1, end_of(p, which));
    double all = 0.0;
    for (; t < end; ++t) {
      const int tile = static_cast<int>(t - tile0), ty = tile / across;
      const int col = (tile - ty * across) * kPassCols + static_cast<int>(threadIdx.x & 31) * 8;
      const int n = e.cols - col;
      Squares squares;          // of a step's direction
      float held = 0.f;         // of an input
      const int first_row = ty * kPassRows + static_cast<int>(threadIdx.x >> 5);
      if (MUON && WC > 0 && e.wide) {
        // two rows' loads at a time, before the first store
        constexpr int kAtOnce = 2;
        const uint64_t* ranks = p.grads + static_cast<int64_t>(which) * p.W;
#pragma unroll
        for (int r = 0; r < kPassRows / 8; r += kAtOnce) {
          uint4 raw[kAtOnce][WC > 0 ? WC : 1];
          float m[kAtOnce][8];
          bool here[kAtOnce];
          int64_t at[kAtOnce];
#pragma unroll
          for (int j = 0; j < kAtOnce; ++j) {
            const int row = first_row + (r + j) * 8;
            here[j] = row < e.rows && n > 0;
            at[j] = static_cast<int64_t>(row) * e.cols + col;
            if (!here[j]) continue;
#pragma unroll
            for (int w = 0; w < WC; ++w) raw[j][w] = dev::ld_16B(reinterpret_cast<const T*>(ranks[w]) + at[j]);
            dev::ld_32B(e.momentum + at[j], m[j]);
          }
#pragma unroll
          for (int j = 0; j < kAtOnce; ++j) {
            if (!here[j]) continue;
            float g[8];
            if constexpr (!std::is_same<T, float>::value) mean_of<T, (WC > 0 ? WC : 1)>(raw[j], g);
            if (e.mean != nullptr) dev::st_32B(e.mean + at[j], g);
            float u[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float now = __fmaf_rn(p.mu, m[j][k], g[k]);
              u[k] = p.nesterov ? __fmaf_rn(p.mu, now, g[k]) : now;
            }
            squares.add(u, 8);
          }
        }
      } else {
#pragma unroll
        for (int r = 0; r < kPassRows / 8; ++r) {
          const int row = first_row + r * 8;
          if (row >= e.rows || n <= 0) continue;
          float u[8], m[8];
          direction8<T, MUON>(p, e, which, row, col, n, true, u, m);
          if (MUON) {
            squares.add(u, n);
            continue;
          }
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < n) held = fmaf(u[k], u[k], held);
        }
        if (!MUON && !std::is_same<T, __half>::value && !squares_held(held)) {
          held = 0.f;
#pragma unroll 1
          for (int row = first_row; row < min(e.rows, first_row + kPassRows) && n > 0; row += 8) {
            float u[8], m[8];
            direction8<T, MUON>(p, e, which, row, col, n, true, u, m);
            squares.add(u, n);
          }
        }
      }
      all += MUON || held == 0.f ? squares.total() : held;
    }
    all = block_sum(all);
    if (threadIdx.x == 0) p.part[blockIdx.x + which] = all;
  }
}

constexpr int kTurnBytes = kPassCols * (kPassRows + 1) * 4;

// A row's values on their way to X: times the power of two, in their parts, to
// their place or to be turned.
__device__ __forceinline__ void to_first(const PassArgs& p, const Entry& e, int row, int col, int in_tile,
                                         const First& x0, float (&u)[8], uint32_t* turned) {
#pragma unroll
  for (int k = 0; k < 8; ++k) u[k] = x0(u[k]);
  uint4 hi, lo;
  split8(u, hi, lo);
  if (!e.transposed) {
    // columns past the last, up to the boundary of 8, are not read again
    uint16_t* to = e.x + row * e.ld + col;
    dev::st_16B(to, hi);
    if (p.two) dev::st_16B(to + e.x_part, lo);
  } else {
    const uint16_t *h = reinterpret_cast<const uint16_t*>(&hi), *l = reinterpret_cast<const uint16_t*>(&lo);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      turned[((threadIdx.x & 31) * 8 + k) * (kPassRows + 1) + in_tile] = h[k] | static_cast<uint32_t>(l[k]) << 16;
  }
}

// The second pass: X = the matrix times a power of two that brings its norm
// to [2^12, 2^13), in one or two fp16 parts, transposed where it has more rows
// than columns; the new momentum, unless the norm is not finite.
template <typename T, bool MUON>
__global__ void __launch_bounds__(kPassThreads) make_first(const __grid_constant__ PassArgs p) {
  extern __shared__ uint32_t turned[];      // kTurnBytes, where matrices are turned
  allow_next();
  await_previous();
  const unsigned t1 = stretch(p.tiles, blockIdx.x + 1);
  for (unsigned t = stretch(p.tiles, blockIdx.x); t < t1;) {
    const int which = entry_of(p.entries, p.count, t);
    const Entry& e = p.entries[which];
    const int across = (e.cols + kPassCols - 1) / kPassCols;
    const unsigned tile0 = e.tile0, past = end_of(p, which), end = min(t1, past);
    // the blocks of the first pass, of which there were as many, that met this matrix
    unsigned first = static_cast<unsigned>(static_cast<uint64_t>(tile0) * gridDim.x / p.tiles);
    while (stretch(p.tiles, first + 1) <= tile0) ++first;
    double s = 0.0;
    for (unsigned b = first + threadIdx.x; b < gridDim.x && stretch(p.tiles, b) < past; b += kPassThreads)
      if (stretch(p.tiles, b + 1) > stretch(p.tiles, b)) s += p.part[b + which];
    const First x0(block_sum(s));
    if (t == tile0 && threadIdx.x == 0) p.norms[which] = {x0.unit, x0.finite};
    for (; t < end; ++t) {
      const int tile = static_cast<int>(t - tile0), ty = tile / across, col0 = (tile - ty * across) * kPassCols;
      const int col = col0 + static_cast<int>(threadIdx.x & 31) * 8, n = e.cols - col;
      if (e.transposed) __syncthreads();   // the tile before has been written
      const int warp_row = static_cast<int>(threadIdx.x >> 5), first_row = ty * kPassRows + warp_row;
      if (MUON && e.mean != nullptr && e.wide) {
        // two rows' loads at a time, before the first store
#pragma unroll
        for (int r = 0; r < kPassRows / 8; r += 2) {
          float g[2][8], m[2][8];
          bool here[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int row = first_row + (r + j) * 8;
            const int64_t at = static_cast<int64_t>(row) * e.cols + col;
            here[j] = row < e.rows && n > 0;
            if (!here[j]) continue;
            dev::ld_32B(e.mean + at, g[j]);
            dev::ld_32B(e.momentum + at, m[j]);
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (!here[j]) continue;
            const int in_tile = warp_row + (r + j) * 8, row = ty * kPassRows + in_tile;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              m[j][k] = __fmaf_rn(p.mu, m[j][k], g[j][k]);
              g[j][k] = p.nesterov ? __fmaf_rn(p.mu, m[j][k], g[j][k]) : m[j][k];
            }
            if (x0.finite) dev::st_32B(e.momentum + static_cast<int64_t>(row) * e.cols + col, m[j]);
            to_first(p, e, row, col, in_tile, x0, g[j], turned);
          }
        }
      } else {
#pragma unroll
        for (int r = 0; r < kPassRows / 8; ++r) {
          const int in_tile = r * 8 + warp_row, row = ty * kPassRows + in_tile;
          if (row >= e.rows || n <= 0) continue;
          float u[8], m[8];
          direction8<T, MUON>(p, e, which, row, col, n, false, u, m);
          if (MUON && x0.finite) store_some(e.momentum + static_cast<int64_t>(row) * e.cols + col, e.wide, n, m);
          to_first(p, e, row, col, in_tile, x0, u, turned);
        }
      }
      if (e.transposed) {
        __syncthreads();
        // half a warp writes a column of the tile, two rows a lane; a row past the last one lies in the padding
        const int pair = static_cast<int>(threadIdx.x & 15) * 2, row = ty * kPassRows + pair;
        if (row >= e.rows) continue;
        for (int c = static_cast<int>(threadIdx.x >> 4); c < min(kPassCols, e.cols - col0); c += kPassThreads / 16) {
          const uint32_t a = turned[c * (kPassRows + 1) + pair], b = turned[c * (kPassRows + 1) + pair + 1];
          uint16_t* to = e.x + (col0 + c) * e.ld + row;
          *reinterpret_cast<uint32_t*>(to) = __byte_perm(a, b, 0x5410);
          if (p.two) *reinterpret_cast<uint32_t*>(to + e.x_part) = __byte_perm(a, b, 0x7632);
        }
      }
    }
  }
}

// ---- host -------------------------------------------------------------------------------

constexpr int64_t kMaxSide = 32768, kMaxMatrices = 65536;
constexpr int64_t kStatusBytes = 256;
constexpr int64_t kMostPassBlocks = 2 * kPairs * kPassBlocksPerSm;

// The matrices of one shape, or of its transpose.
struct Group {
  int64_t m, n;
  std::vector<int64_t> members;
  int64_t first;               // of its entries
  int64_t ldx, lda;
  int64_t at[kBuffers];        // byte offsets of the buffers: high parts, then low parts
  // See kMultiply; T is theirs alone.  By twos and one by one, us (bf16): eight of 1024 x 1536 453 and 454, of 1024 x
  // 2048 494 and 547, of 1024 x 4096 715 and 999; one of them 241 and 226, 249 and 240, 294 and 330.
  bool joined() const { return n >= 2 * m; }
  int64_t x_part() const { return static_cast<int64_t>(members.size()) * m * ldx; }
  int64_t a_part() const { return static_cast<int64_t>(members.size()) * m * lda; }
};

// How a call's matrices are laid out in the workspace.
struct Plan {
  std::vector<Group> groups;
  std::vector<int64_t> small;  // the matrices that one cluster of CTAs takes whole
  int64_t count = 0, tiles = 0;
  int64_t table, table_words, counters, norms, part, mean, total;
  // tiles lost, then for each launch its tiles taken and CTAs ended, then for each matrix its tiles written
  int64_t launches() const { return ceil_div(static_cast<int64_t>(groups.size()), kMaxGroups); }
  int64_t counter_words() const { return 1 + 2 * launches() + count; }
};

int64_t pass_tiles(int64_t rows, int64_t cols) { return ceil_div(rows, kPassRows) * ceil_div(cols, kPassCols); }

int make_plan(Plan& plan, int64_t n_matrices, const int64_t* rows, const int64_t* cols, int W, bool muon) {
  if (n_matrices < 0 || n_matrices > kMaxMatrices)
    return fail(ZERO_E_ARG, "n_matrices=%lld outside [0, %lld]", (long long)n_matrices, (long long)kMaxMatrices);
  if (n_matrices > 0 && (!rows || !cols)) return fail(ZERO_E_ARG, "rows and cols are required");
  int64_t numel = 0;
  std::map<std::pair<int64_t, int64_t>, size_t> known;
  for (int64_t i = 0; i < n_matrices; ++i) {
    if (rows[i] < 1 || rows[i] > kMaxSide || cols[i] < 1 || cols[i] > kMaxSide)
      return fail(ZERO_E_ARG, "matrix %lld: %lld x %lld, sides outside [1, %lld]", (long long)i, (long long)rows[i],
                  (long long)cols[i], (long long)kMaxSide);
    if (small_fits(rows[i], cols[i])) {
      plan.small.push_back(i);
      continue;
    }
    const int64_t m = std::min(rows[i], cols[i]), n = std::max(rows[i], cols[i]);
    ++plan.count;
    const auto [it, fresh] = known.try_emplace({m, n}, plan.groups.size());
    if (fresh) {
      plan.groups.emplace_back();
      plan.groups.back().m = m;
      plan.groups.back().n = n;
    }
    plan.groups[it->second].members.push_back(i);
    plan.tiles += pass_tiles(rows[i], cols[i]);
    numel += round_up(rows[i] * cols[i], 8);
  }
  if (plan.tiles > INT32_MAX) return fail(ZERO_E_ARG, "too many elements");
  // the longest products first
  std::sort(plan.groups.begin(), plan.groups.end(),
            [](const Group& a, const Group& b) { return a.n != b.n ? a.n > b.n : a.m > b.m; });
  plan.table = kStatusBytes;
  plan.table_words = plan.count * (static_cast<int64_t>(sizeof(Entry)) / 8 + (muon ? W : 0));
  plan.counters = plan.table + round_up(plan.table_words * 8, 256);
  plan.norms = plan.counters + round_up(plan.counter_words() * 4, 256);
  plan.part = plan.norms + round_up(plan.count * static_cast<int64_t>(sizeof(Norm)), 256);
  plan.mean = plan.part + round_up((kMostPassBlocks + plan.count) * 8, 256);
  int64_t at = plan.mean + (muon && W > kDirectRanks ? round_up(numel * 4, 256) : 0);
  int64_t first = 0;
  for (Group& g : plan.groups) {
    g.first = first;
    first += static_cast<int64_t>(g.members.size());
    g.ldx = round_up(g.n, 16);
    g.lda = round_up(g.m, 16);
    for (int k = 0; k < kBuffers; ++k) {
      g.at[k] = at;
      if (k != kT || g.joined()) at += round_up((k <= kX1 ? g.x_part() : g.a_part()) * 4, 256);
    }
  }
  plan.total = std::max<int64_t>(at, 512);
  return ZERO_OK;
}

// A stack of `depth` row-major fp16 matrices, in boxes of box_rows x 64 under the
// 128-byte swizzle; what lies outside a matrix reads as 0.
int make_map3(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t ld, int64_t depth, int box_rows) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(depth)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2, static_cast<cuuint64_t>(ld) * rows * 2};
  const cuuint32_t box[3] = {kTileK, static_cast<cuuint32_t>(box_rows), 1}, ones[3] = {1, 1, 1};
  const host::EncodeFn fn = host::encoder();
  if (!fn) return fail(ZERO_E_CUDA, "the driver offers no tensor-map encoder");
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base), dims, strides, box, ones,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? ZERO_OK : fail(ZERO_E_CUDA, "encoding a tensor map failed (%d)", static_cast<int>(r));
}

// Tiles of one matrix's product of a class.
int tiles_of(int of, int64_t m, int64_t n, int bn) {
  const int kind = of == 2 ? kApply : kGram;
  const int m_tiles = static_cast<int>(ceil_div(m, kTileM)), n_tiles = static_cast<int>(ceil_div(kind == kApply ? n : m, bn));
  if (kind == kApply) return m_tiles * n_tiles;
  int t = 0;
  for (int mt = 0; mt < m_tiles; ++mt) t += tiles_of_row(mt, bn, n_tiles);
  return t;
}

// The width of a product's tiles.  A block of K takes 2 bn cycles for each of
// the products of parts, or the time its operands take to load (48 bytes a
// cycle); a tile has some 2000 cycles besides, and the tiles of a product that
// are one more than the pairs take as long as two each.
int width_of(int of, int64_t m, int64_t n, int matrices, bool fine, int most) {
  const int products = fine ? 3 : 1, parts = fine ? 2 : 1;
  const int64_t kb = ceil_div(of == 0 ? n : m, kTileK);
  int best = most;
  double least = 0;
  for (int bn = most; bn >= 64; bn /= 2) {
    const double tiles = static_cast<double>(tiles_of(of, m, n, bn)) * matrices;
    const double block = std::max<double>(2 * bn * products, (128 + bn / 2) * kTileK * 2 * parts / 48.0);
    const double cost = (kb * block + 2000) * (matrices > 1 ? std::max(1.0, tiles / kPairs) : std::ceil(tiles / kPairs));
    if (bn == most || cost < least) {
      least = cost;
      best = bn;
    }
  }
  return best;
}

struct Recurrence {
  int steps, fine;
  const double* coefficients;
  int first_parts;             // of the first X
  int last;                    // Final
  int dtype;                   // of what it writes
};

// The list of a shape's products, steps one by one or by twos; its length.
int make_phases(Phase* to, const Recurrence& r, bool joined) {
  int count = 0, x = kX0;
  auto add = [&](int kind, int a, int b, int out, int step, bool fine, int parts_a, int parts_b, bool two, int units,
                 float factor) {
    const Phase f = {static_cast<int8_t>(kind), static_cast<int8_t>(a), static_cast<int8_t>(b), static_cast<int8_t>(out),
                     static_cast<int8_t>(step), static_cast<int8_t>(parts_a), static_cast<int8_t>(parts_b),
                     static_cast<int8_t>(two), static_cast<int8_t>(units), static_cast<int8_t>(fine), 0, 0, factor};
    to[count++] = f;
  };
  for (int s = 0; s < r.steps;) {
    const bool fine = s < r.fine;
    const int parts = fine ? 2 : 1, of_x = s == 0 ? std::min(parts, r.first_parts) : parts;
    // the joined P's entries, up to the product of both a, have to fit fp16
    const bool two = joined && s + 1 < (fine ? r.fine : r.steps) &&
                     std::fabs(r.coefficients[3 * s] * r.coefficients[3 * s + 3]) <= 64.0;
    const int past = s + (two ? 2 : 1);
    add(kGram, x, x, kA, s, fine, of_x, of_x, fine, s == 0 ? 2 : 0, kScaleA / (kScaleX * kScaleX));
    add(kPoly, kA, kA, kP, s, fine, parts, parts, fine, 0, 0.f);
    if (two) {
      add(kMultiply, kP, kA, kT, s, fine, parts, parts, fine, 0, kScaleT / (kScaleP * kScaleA));
      add(kMultiply, kT, kP, kA, s, fine, parts, parts, fine, 0, kScaleA / (kScaleT * kScaleP));
      add(kPoly, kA, kA, kT, s + 1, fine, parts, parts, fine, 0, 0.f);
      add(kMultiply, kT, kP, kA, s, fine, parts, parts, fine, 0, 1.f / kScaleP);
    }
    const bool last = past == r.steps;
    add(kApply, two ? kA : kP, x, x ^ 1, s, fine, parts, of_x, past < r.fine, s == 0 ? 1 : 0,
        last ? 1.f / (kScaleP * kScaleX) : 1.f / kScaleP);
    to[count - 1].last = last;
    x ^= 1;
    s = past;
  }
  return count;
}

// The steps of plan.groups[from, to).
template <int FINAL>
int run_groups(const Plan& plan, size_t from, size_t to, const Recurrence& r, char* ws, cudaStream_t s, bool& stall) {
  static thread_local RunArgs g;
  std::memset(&g, 0, sizeof g);
  g.dtype = r.dtype;
  g.segment = FINAL == kLast && r.dtype == ZERO_FP32 && r.fine > 0 ? kSegment : 0;
  g.stall = std::exchange(stall, false);
  g.entries = reinterpret_cast<const Entry*>(ws + plan.table);
  g.norms = reinterpret_cast<const Norm*>(ws + plan.norms);
  g.failures = reinterpret_cast<unsigned int*>(ws);
  unsigned int* counters = reinterpret_cast<unsigned int*>(ws + plan.counters);
  g.lost = counters;
  g.next = counters + 1 + 2 * (from / kMaxGroups);
  g.exits = g.next + 1;
  g.written = counters + 1 + 2 * plan.launches();
  for (int k = 0; k < 3 * r.steps; ++k) g.coefficients[k] = static_cast<float>(r.coefficients[k]);
  for (int joined = 0; joined < 2; ++joined) g.phases[joined] = make_phases(g.phase[joined], r, joined);
  int64_t all = 0, most = 1;
  for (size_t i = from; i < to; ++i) {
    const Group& group = plan.groups[i];
    Shape& h = g.shape[g.shapes++];
    const int c = static_cast<int>(group.members.size());
    const int64_t m = group.m, n = group.n;
    h.matrices = c;
    h.first = static_cast<int>(group.first);
    h.m = static_cast<int>(m);
    h.n = static_cast<int>(n);
    h.joined = group.joined();
    g.entries_here += c;
    for (int fine = 0; fine < 2; ++fine)
      for (int of = 0; of < 3; ++of) {
        h.bn[fine][of] = width_of(of, m, n, c, fine, g.segment > 0 ? kSegmentTile : kTileN);
        h.tiles[fine][of] = tiles_of(of, m, n, h.bn[fine][of]);
        most = std::max(most, static_cast<int64_t>(c) * h.tiles[fine][of]);
        all += 4 * static_cast<int64_t>(r.steps) * c * h.tiles[fine][of];
      }
    h.ldx = group.ldx;
    h.lda = group.lda;
    h.apart_x = m * group.ldx;
    h.apart_a = m * group.lda;
    h.part_x = group.x_part();
    h.part_a = group.a_part();
    for (int k = 0; k < kBuffers; ++k) {
      if (k == kT && !h.joined) continue;
      const bool of_x = k <= kX1;
      char* at = ws + group.at[k];
      h.at[k] = reinterpret_cast<uint16_t*>(at);
      CUtensorMap* maps[3] = {&h.box128[k], &h.box64[k], &h.box32[k]};
      for (int b = 0; b < 3; ++b)
        if (const int rc = make_map3(maps[b], at, m, of_x ? n : m, of_x ? group.ldx : group.lda, 2 * c, 128 >> b)) return rc;
    }
  }
  if (all > INT32_MAX) return fail(ZERO_E_ARG, "too many tiles");
  const auto fn = ns_run<FINAL>;
  ZERO_CUDA(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kRunSmem));
  const int pairs = static_cast<int>(std::min({std::max<int64_t>(1, sm_count() / 2), kPairs, most * static_cast<int64_t>(to - from)}));
  ZERO_CUDA(launch_chained(fn, dim3(2 * pairs), kThreads, kRunSmem, s, g));
  return ZERO_OK;
}

template <int BYTES>
int send_table_of(const std::vector<uint64_t>& words, char* to, unsigned int* counters, int n_counters, cudaStream_t s) {
  static thread_local TablePart<BYTES> part;
  constexpr size_t kWords = BYTES / 8;
  for (size_t at = 0; at < words.size(); at += kWords) {
    const size_t count = std::min(kWords, words.size() - at);
    std::memcpy(part.data, words.data() + at, count * 8);
    ZERO_CUDA(launch_chained(copy_table<BYTES>, dim3(1), kPassThreads, 0, s, part, static_cast<int>(count),
                             reinterpret_cast<uint64_t*>(to) + at, counters, n_counters));
  }
  return ZERO_OK;
}

int send_table(const Plan& plan, const std::vector<uint64_t>& words, char* ws, cudaStream_t s) {
  unsigned int* counters = reinterpret_cast<unsigned int*>(ws + plan.counters);
  const int n = static_cast<int>(plan.counter_words());
  return words.size() * 8 <= kSmallTable ? send_table_of<kSmallTable>(words, ws + plan.table, counters, n, s)
                                         : send_table_of<kLargeTable>(words, ws + plan.table, counters, n, s);
}

template <typename T, bool MUON>
int launch_passes(const PassArgs& p, cudaStream_t s) {
  const int64_t most = std::min(static_cast<int64_t>(sm_count()) * kPassBlocksPerSm, kMostPassBlocks);
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(p.tiles, most)));
  auto first = sum_squares<T, MUON, 0>;
  if constexpr (MUON) {
    if (p.W == 1) first = sum_squares<T, MUON, 1>;
    if (p.W == 2) first = sum_squares<T, MUON, 2>;
    if (p.W == 4) first = sum_squares<T, MUON, 4>;
  }
  ZERO_CUDA(launch_chained(first, grid, kPassThreads, 0, s, p));
  ZERO_CUDA(launch_chained(make_first<T, MUON>, grid, kPassThreads, p.turns ? kTurnBytes : 0, s, p));
  return ZERO_OK;
}

// Every group, kMaxGroups of them at a time.
int run_all(const Plan& plan, const Recurrence& r, char* ws, cudaStream_t s, bool& stall) {
  const size_t groups = plan.groups.size();
  for (size_t from = 0; from < groups; from += kMaxGroups) {
    const size_t to = std::min(groups, from + kMaxGroups);
    const int rc = r.last == kUpdate ? run_groups<kUpdate>(plan, from, to, r, ws, s, stall)
                                     : run_groups<kLast>(plan, from, to, r, ws, s, stall);
    if (rc) return rc;
  }
  return ZERO_OK;
}

int check_recurrence(int steps, const double* coefficients, int fine) {
  if (steps < 1 || steps > kMaxSteps) return fail(ZERO_E_ARG, "steps=%d outside [1, %d]", steps, kMaxSteps);
  if (!coefficients) return fail(ZERO_E_ARG, "coefficients is NULL");
  for (int k = 0; k < 3 * steps; ++k)
    if (!(std::fabs(coefficients[k]) <= 64.0))
      return fail(ZERO_E_ARG, "coefficient %d is %g: at most 64 in size is supported", k, coefficients[k]);
  if (fine < -1 || fine > steps) return fail(ZERO_E_ARG, "fine_steps=%d outside [-1, %d]", fine, steps);
  return ZERO_OK;
}

int check_workspace(const void* workspace, int64_t bytes, int64_t needed) {
  if (workspace == nullptr) return fail(ZERO_E_ARG, "workspace is NULL");
  if (reinterpret_cast<uintptr_t>(workspace) % 256) return fail(ZERO_E_ALIGN, "workspace must be 256-byte aligned");
  if (bytes < needed)
    return fail(ZERO_E_ARG, "workspace of %lld bytes: %lld are needed", (long long)bytes, (long long)needed);
  return ZERO_OK;
}

// The steps that carry two parts where the caller leaves it open: all, for bf16
// results all but the last (see above).
int fine_steps(int fine, int steps, bool bf16) { return fine >= 0 ? fine : bf16 ? steps - 1 : steps; }

// Fills an entry's place in the workspace.
void place(Entry& e, const Group& g, int64_t member, char* ws) {
  e.ld = g.ldx;
  e.x = reinterpret_cast<uint16_t*>(ws + g.at[kX0]) + member * g.m * g.ldx;
  e.x_part = g.x_part();
}

// The lists of matrices are kept on the host while a call is cut up.
int out_of_memory() { return fail(ZERO_E_NOMEM, "no host memory for the list of matrices"); }

}  // namespace

cudaError_t ns_timeouts(unsigned int* out) {
  unsigned int small = 0;
  const cudaError_t e = ns::small_timeouts(&small);
  if (e != cudaSuccess) return e;
  const cudaError_t e2 = cudaMemcpyFromSymbol(out, g_ns_timeouts, sizeof *out);
  *out += small;
  return e2;
}

}  // namespace zero

using namespace zero;

extern "C" int64_t zero_orthogonalize_workspace_bytes(int64_t n_matrices, const int64_t* rows, const int64_t* cols) try {
  Plan plan;
  const int rc = make_plan(plan, n_matrices, rows, cols, 0, false);
  return rc ? rc : plan.total;
} catch (const std::bad_alloc&) {
  return out_of_memory();
}

extern "C" int zero_orthogonalize(int64_t n_matrices, const int64_t* rows, const int64_t* cols, int dtype,
                                  const void* const* in, const int64_t* in_strides, void* const* out,
                                  const int64_t* out_strides, int steps, const double* coefficients, int fine,
                                  void* workspace, int64_t workspace_bytes, void* stream) try {
  bool stall = std::exchange(g_stall_next, false);
  Plan plan;
  int rc = make_plan(plan, n_matrices, rows, cols, 0, false);
  if (rc || (rc = check_recurrence(steps, coefficients, fine))) return rc;
  if (dtype != ZERO_FP16 && dtype != ZERO_BF16 && dtype != ZERO_FP32)
    return fail(ZERO_E_ARG, "the format must be ZERO_FP16, ZERO_BF16 or ZERO_FP32");
  if (n_matrices > 0 && (!in || !out)) return fail(ZERO_E_ARG, "in and out are required");
  const int item = dtype == ZERO_FP32 ? 4 : 2;
  for (int64_t i = 0; i < n_matrices; ++i) {
    const int64_t si = in_strides ? in_strides[i] : cols[i], so = out_strides ? out_strides[i] : cols[i];
    if (!in[i] || !out[i]) return fail(ZERO_E_ARG, "matrix %lld: a NULL pointer", (long long)i);
    if (reinterpret_cast<uintptr_t>(in[i]) % item || reinterpret_cast<uintptr_t>(out[i]) % item)
      return fail(ZERO_E_ALIGN, "matrix %lld: not aligned to its elements", (long long)i);
    if (si < cols[i] || so < cols[i] || si > (int64_t(1) << 32) || so > (int64_t(1) << 32))
      return fail(ZERO_E_ARG, "matrix %lld: a row stride is below its columns or too large", (long long)i);
  }
  if (n_matrices == 0) return ZERO_OK;
  if ((rc = check_workspace(workspace, workspace_bytes, plan.total))) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  auto entry = [&](int64_t i) {
    Entry e;
    std::memset(&e, 0, sizeof e);
    e.rows = static_cast<int>(rows[i]);
    e.cols = static_cast<int>(cols[i]);
    e.transposed = rows[i] > cols[i];
    e.in = in[i];
    e.out = out[i];
    e.in_stride = in_strides ? in_strides[i] : cols[i];
    e.out_stride = out_strides ? out_strides[i] : cols[i];
    const uintptr_t both = reinterpret_cast<uintptr_t>(e.in) | reinterpret_cast<uintptr_t>(e.out);
    e.wide = both % (8 * item) == 0 && (e.cols | e.in_stride | e.out_stride) % 8 == 0;
    return e;
  };
  Recurrence r = {steps, fine_steps(fine, steps, dtype == ZERO_BF16), coefficients, dtype == ZERO_FP32 ? 2 : 1,
                  kLast, dtype};
  std::vector<Entry> small;
  for (int64_t i : plan.small) small.push_back(entry(i));
  SmallCall c = {small.data(), nullptr, static_cast<int>(small.size()), false, dtype, dtype, 0, 0.f, 0, steps, r.fine,
                 r.first_parts, coefficients, static_cast<unsigned int*>(workspace), s};
  if ((rc = run_small(c, stall))) return rc;
  if (plan.count == 0) return ZERO_OK;
  constexpr size_t kEntryWords = sizeof(Entry) / 8;
  std::vector<uint64_t> words(plan.table_words);
  unsigned tile = 0;
  bool turns = false;
  for (const Group& g : plan.groups)
    for (size_t k = 0; k < g.members.size(); ++k) {
      Entry e = entry(g.members[k]);
      e.tile0 = tile;
      turns = turns || e.transposed;
      tile += static_cast<unsigned>(pass_tiles(e.rows, e.cols));
      place(e, g, static_cast<int64_t>(k), ws);
      std::memcpy(&words[(g.first + k) * kEntryWords], &e, sizeof e);
    }
  if ((rc = send_table(plan, words, ws, s))) return rc;
  PassArgs p;
  std::memset(&p, 0, sizeof p);
  p.entries = reinterpret_cast<const Entry*>(ws + plan.table);
  p.count = static_cast<int>(plan.count);
  p.tiles = tile;
  p.turns = turns;
  p.two = r.first_parts > 1 && r.fine > 0;
  p.part = reinterpret_cast<double*>(ws + plan.part);
  p.norms = reinterpret_cast<Norm*>(ws + plan.norms);
  rc = dtype == ZERO_FP16   ? launch_passes<__half, false>(p, s)
       : dtype == ZERO_BF16 ? launch_passes<__nv_bfloat16, false>(p, s)
                            : launch_passes<float, false>(p, s);
  return rc ? rc : run_all(plan, r, ws, s, stall);
} catch (const std::bad_alloc&) {
  return out_of_memory();
}

extern "C" int64_t zero_muon_workspace_bytes(int W, int64_t n_matrices, const int64_t* rows, const int64_t* cols) try {
  if (W < 1 || W > ZERO_MAX_RANKS) return fail(ZERO_E_ARG, "W=%d outside [1, %d]", W, ZERO_MAX_RANKS);
  Plan plan;
  const int rc = make_plan(plan, n_matrices, rows, cols, W, true);
  return rc ? rc : plan.total;
} catch (const std::bad_alloc&) {
  return out_of_memory();
}

extern "C" int zero_muon_step(int W, int64_t n_matrices, const int64_t* rows, const int64_t* cols, int grad_dtype,
                              int work_dtype, const void* const* grads, float* const* master, float* const* momentum,
                              void* const* p16, double lr, double mu, int nesterov, double weight_decay,
                              const double* scales, int steps, const double* coefficients, int fine, void* workspace,
                              int64_t workspace_bytes, void* stream) try {
  bool stall = std::exchange(g_stall_next, false);
  if (W < 1 || W > ZERO_MAX_RANKS) return fail(ZERO_E_ARG, "W=%d outside [1, %d]", W, ZERO_MAX_RANKS);
  Plan plan;
  int rc = make_plan(plan, n_matrices, rows, cols, W, true);
  if (rc || (rc = check_recurrence(steps, coefficients, fine))) return rc;
  if (!host::valid_dtype(grad_dtype) || !host::valid_dtype(work_dtype))
    return fail(ZERO_E_ARG, "the 16-bit formats must be ZERO_FP16 or ZERO_BF16");
  if (!std::isfinite(static_cast<float>(lr))) return fail(ZERO_E_ARG, "lr %g is not a finite fp32 value", lr);
  if (!(mu >= 0.0 && mu < 1.0)) return fail(ZERO_E_ARG, "mu %g outside [0, 1)", mu);
  if (!std::isfinite(static_cast<float>(1.0 - lr * weight_decay)))
    return fail(ZERO_E_ARG, "weight_decay %g: 1 - lr * weight_decay is not a finite fp32 value", weight_decay);
  if (n_matrices > 0 && (!grads || !master || !momentum || !p16))
    return fail(ZERO_E_ARG, "grads, master, momentum and p16 are required");
  for (int64_t i = 0; i < n_matrices; ++i) {
    if (!master[i] || !momentum[i] || !p16[i]) return fail(ZERO_E_ARG, "matrix %lld: a NULL pointer", (long long)i);
    if (reinterpret_cast<uintptr_t>(master[i]) % 4 || reinterpret_cast<uintptr_t>(momentum[i]) % 4 ||
        reinterpret_cast<uintptr_t>(p16[i]) % 2)
      return fail(ZERO_E_ALIGN, "matrix %lld: not aligned to its elements", (long long)i);
    if (scales && !std::isfinite(static_cast<float>(lr * scales[i])))
      return fail(ZERO_E_ARG, "scales[%lld] %g: lr * scale is not a finite fp32 value", (long long)i, scales[i]);
    for (int w = 0; w < W; ++w) {
      const void* g = grads[w * n_matrices + i];
      if (!g) return fail(ZERO_E_ARG, "matrix %lld: rank %d's gradient is NULL", (long long)i, w);
      if (reinterpret_cast<uintptr_t>(g) % 2)
        return fail(ZERO_E_ALIGN, "matrix %lld: rank %d's gradient is not aligned to its elements", (long long)i, w);
    }
  }
  if (n_matrices == 0) return ZERO_OK;
  if ((rc = check_workspace(workspace, workspace_bytes, plan.total))) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  auto entry = [&](int64_t i, uint64_t* ranks) {
    Entry e;
    std::memset(&e, 0, sizeof e);
    e.rows = static_cast<int>(rows[i]);
    e.cols = static_cast<int>(cols[i]);
    e.transposed = rows[i] > cols[i];
    e.master = master[i];
    e.momentum = momentum[i];
    e.p16 = p16[i];
    e.step = static_cast<float>(lr * (scales ? scales[i] : 1.0));
    e.keep = static_cast<float>(1.0 - lr * weight_decay);
    const uintptr_t fp32 = reinterpret_cast<uintptr_t>(e.master) | reinterpret_cast<uintptr_t>(e.momentum);
    uintptr_t b16 = reinterpret_cast<uintptr_t>(e.p16);
    for (int w = 0; w < W; ++w) {
      ranks[w] = reinterpret_cast<uint64_t>(grads[w * n_matrices + i]);
      b16 |= reinterpret_cast<uintptr_t>(grads[w * n_matrices + i]);
    }
    e.wide = fp32 % 32 == 0 && b16 % 16 == 0 && e.cols % 8 == 0;
    return e;
  };
  Recurrence r = {steps, fine_steps(fine, steps, false), coefficients, 2, kUpdate, work_dtype};
  std::vector<Entry> small;
  std::vector<uint64_t> small_ranks(plan.small.size() * W);
  for (int64_t i : plan.small) small.push_back(entry(i, &small_ranks[small.size() * W]));
  SmallCall c = {small.data(), small_ranks.data(), static_cast<int>(small.size()), true, grad_dtype, work_dtype, W,
                 static_cast<float>(mu), nesterov != 0, steps, r.fine, r.first_parts, coefficients,
                 static_cast<unsigned int*>(workspace), s};
  if ((rc = run_small(c, stall))) return rc;
  if (plan.count == 0) return ZERO_OK;
  constexpr size_t kEntryWords = sizeof(Entry) / 8;
  std::vector<uint64_t> words(plan.table_words);
  uint64_t* ranks = words.data() + plan.count * kEntryWords;
  unsigned tile = 0;
  bool turns = false;
  int64_t mean_at = plan.mean;
  for (const Group& g : plan.groups)
    for (size_t k = 0; k < g.members.size(); ++k) {
      const int64_t to = g.first + static_cast<int64_t>(k);
      Entry e = entry(g.members[k], ranks + to * W);
      if (W > kDirectRanks) {
        e.mean = reinterpret_cast<float*>(ws + mean_at);
        mean_at += round_up(static_cast<int64_t>(e.rows) * e.cols, 8) * 4;
      }
      e.tile0 = tile;
      turns = turns || e.transposed;
      tile += static_cast<unsigned>(pass_tiles(e.rows, e.cols));
      place(e, g, static_cast<int64_t>(k), ws);
      std::memcpy(&words[to * kEntryWords], &e, sizeof e);
    }
  if ((rc = send_table(plan, words, ws, s))) return rc;
  PassArgs p;
  std::memset(&p, 0, sizeof p);
  p.entries = reinterpret_cast<const Entry*>(ws + plan.table);
  p.grads = reinterpret_cast<const uint64_t*>(ws + plan.table) + plan.count * kEntryWords;
  p.count = static_cast<int>(plan.count);
  p.tiles = tile;
  p.turns = turns;
  p.W = W;
  p.mu = static_cast<float>(mu);
  p.nesterov = nesterov != 0;
  p.two = r.fine > 0;
  p.part = reinterpret_cast<double*>(ws + plan.part);
  p.norms = reinterpret_cast<Norm*>(ws + plan.norms);
  rc = grad_dtype == ZERO_FP16 ? launch_passes<__half, true>(p, s) : launch_passes<__nv_bfloat16, true>(p, s);
  return rc ? rc : run_all(plan, r, ws, s, stall);
} catch (const std::bad_alloc&) {
  return out_of_memory();
}
