// Orthogonalisation of small matrices: everything in one launch.
//
// The recurrence (muon.cu) on a matrix of up to 128 rows is a chain of short
// products, each of which depends on all of the one before: as launches of
// their own, 15 of them take some 7 us each whatever the size.  Here one CTA, or
// a cluster of up to 8, keeps a matrix in shared memory from its input to its
// result: X (m x n, m <= 128) in slices of up to 256 columns, a slice for each
// CTA, in two fp16 parts; A and P (m x m) whole in every CTA, P in A's place.
// The products run on the tensor core from there, their sums come back from
// TMEM:
//   A = X X^T      each CTA over its columns; the CTAs of a cluster then add
//                  up: every one a share of A's columns over all, in the CTAs'
//                  order, and hands the result to all of them
//   P = a I + b A + c A^2   in every CTA alike
//   X <- P X       each CTA its columns
// X's tiles of 64 columns, rows of 128 bytes in the 128-byte swizzle, serve as
// operands both ways: K-major for X X^T, with K the row index for P X.
//
// What bounds it: latency.  A step of a 64 x 64 matrix issues 12 to 36 matrix
// instructions of 32 to 64 cycles each; what takes the time is the way from one
// product to the next (issue, TMEM, registers, shared memory, a barrier).

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <utility>
#include <vector>

#include "launch.cuh"
#include "ns_common.cuh"
#include "umma.cuh"
#include "zero_context.h"

namespace zero {
namespace {

using namespace umma;
using namespace ns;
using host::ceil_div;
using host::cuda_fail;
using host::round_up;

// Bounded device-side waits of ns_small that gave up, over all calls; never set back (see zero_lm_status).
__device__ unsigned int g_small_timeouts;

// Four warps for each quarter of the TMEM lanes, 16 columns in turn (with two steps of five in two parts eight matrices
// of 128 x 256 take 49.6 us, with two warps of 32 columns 55.7; by default, with four, 53).
constexpr int kThreads = 512, kCols = 16;
constexpr int kMostRows = 128, kMostSlice = 256, kMostCtas = 8;

template <int BYTES>
struct SmallArgs {
  int steps, fine, first_parts;
  int out_dtype;
  int W;
  float mu;
  int nesterov;
  int grads_at;                // word of the table where the gradients' addresses begin
  int stall;                   // testing the bounded waits: the first matrix's first product is never reported done
  unsigned int* failures;
  float coefficients[3 * kMaxSteps];
  TablePart<BYTES> table;      // Entry after Entry, then W addresses for each
};

// The CTAs that a matrix takes.
__host__ __device__ inline int ctas_for(const Entry& e) {
  const int n = e.rows > e.cols ? e.rows : e.cols;
  return (n + kMostSlice - 1) / kMostSlice;
}

// ---- products by one CTA ------------------------------------------------------------------

__device__ __forceinline__ void alloc_one(uint32_t slot, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(columns) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void free_one(uint32_t addr, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
}
__device__ __forceinline__ void mma_one(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(
          d),
      "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add))
      : "memory");
}
__device__ __forceinline__ void commit_one(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// ---- shared memory of this CTA and of the others of its cluster --------------------------------

__device__ __forceinline__ uint4 ld_shared(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ void st_shared(uint32_t a, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void st_shared1(uint32_t a, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
__device__ __forceinline__ void st_shared16(uint32_t a, uint16_t v) {
  asm volatile("st.shared.b16 [%0], %1;" ::"r"(a), "h"(v) : "memory");
}
__device__ __forceinline__ float ld_there(uint32_t a) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ double ld_there64(uint32_t a) {
  double v;
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t cluster_ctas() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void meet_cluster() {
  __syncwarp();
  cluster_sync();
}

// One matrix of this launch; blocks of a cluster's size follow one another.
template <typename T, bool MUON, int BYTES>
__global__ void __launch_bounds__(kThreads, 1) ns_small(const __grid_constant__ SmallArgs<BYTES> g) {
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) uint64_t bars[2];
  __shared__ double squares_here;
  __shared__ uint32_t tmem_slot;
  __shared__ float ok_here;
  const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
  const uint32_t bar = smem_addr(bars), drained = bar + 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());
  const int which = static_cast<int>(blockIdx.x) / static_cast<int>(cluster_ctas());
  const Entry& e = reinterpret_cast<const Entry*>(g.table.data)[which];
  // How a matrix is cut goes by its own shape: its sums are then the same whatever else is in the call.  In a cluster
  // that is larger the CTAs left over end here; barriers of a cluster wait for those that have not ended.
  const int ctas = ctas_for(e);
  if (rank >= ctas) return;

  // X is m x n; this CTA has its columns [c0, c0 + nl).  Rows and columns are
  // padded to 16, which is what a matrix instruction takes of K.
  const bool turned = e.transposed;
  const int m = turned ? e.cols : e.rows, n = turned ? e.rows : e.cols;
  const int mp = (m + 15) & ~15, slice = ((n + ctas - 1) / ctas + 15) & ~15;
  const int c0 = rank * slice, nl = min(max(n - c0, 0), slice), nk = (nl + 15) & ~15;
  const uint32_t tile = mp * 128, x_part = (slice + 63) / 64 * tile, a_part = (mp + 63) / 64 * tile;
  const uint32_t xs = base, as = base + 2 * x_part;
  auto at = [&](uint32_t from, int row, int col) {      // a group of 8 columns
    return from + (col >> 6) * tile + row * 128 + ((((col & 63) >> 3) ^ (row & 7)) << 4);
  };
  int columns = 32;
  while (columns < max(mp, nk)) columns *= 2;

  allow_next();
  if (threadIdx.x == 0) {
    bar_init(bar, 1);
    bar_init(drained, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) alloc_one(smem_addr(&tmem_slot), columns);
  for (uint32_t k = threadIdx.x * 16; k < 2 * x_part; k += kThreads * 16) st_shared(xs + k, make_uint4(0, 0, 0, 0));
  await_previous();

  // ---- the norm, and X as a power of two times the matrix (as make_first in muon.cu) ----
  PassArgs p = {};
  p.grads = reinterpret_cast<const uint64_t*>(g.table.data) + g.grads_at;
  p.W = g.W;
  p.mu = g.mu;
  p.nesterov = g.nesterov;
  // items of 8 columns of the caller's: along its rows, or, turned, the rows first, which are X's columns
  const int groups = ((turned ? m : nl) + 7) / 8, items = groups * (turned ? nl : m);
  auto item = [&](int i, int& row, int& col, int& count) {
    if (turned) {
      row = c0 + i % nl;
      col = i / nl * 8;
      count = m - col;
    } else {
      row = i / groups;
      col = c0 + (i - row * groups) * 8;
      count = c0 + nl - col;
    }
  };
  float mine = 0.f;
  for (int i = threadIdx.x; i < items; i += kThreads) {
    int row, col, count;
    item(i, row, col, count);
    float u[8], mom[8];
    direction8<T, MUON>(p, e, which, row, col, count, true, u, mom);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < count) mine = fmaf(u[k], u[k], mine);
  }
  double all = mine;
  if (!squares_held(mine)) {
    Squares again;
#pragma unroll 1
    for (int i = threadIdx.x; i < items; i += kThreads) {
      int row, col, count;
      item(i, row, col, count);
      float u[8], mom[8];
      direction8<T, MUON>(p, e, which, row, col, count, true, u, mom);
      again.add(u, count);
    }
    all = again.total();
  }
  all = block_sum<kThreads>(all);
  if (ctas > 1) {
    if (threadIdx.x == 0) squares_here = all;
    meet_cluster();
    all = 0.0;
    for (int k = 0; k < ctas; ++k) all += ld_there64(in_cta(smem_addr(&squares_here), k));
  }
  const First x0(all);
  const bool finite = x0.finite;
  for (int i = threadIdx.x; i < items; i += kThreads) {
    int row, col, count;
    item(i, row, col, count);
    float u[8], mom[8];
    direction8<T, MUON>(p, e, which, row, col, count, false, u, mom);
    if (MUON && finite) store_some(e.momentum + static_cast<int64_t>(row) * e.cols + col, e.wide, count, mom);
#pragma unroll
    for (int k = 0; k < 8; ++k) u[k] = k < count ? x0(u[k]) : 0.f;
    uint4 hi, lo;
    split8(u, hi, lo);
    if (!turned) {
      const uint32_t to = at(xs, row, col - c0);
      st_shared(to, hi);
      if (g.first_parts > 1) st_shared(to + x_part, lo);
    } else {
      const uint16_t *h = reinterpret_cast<const uint16_t*>(&hi), *l = reinterpret_cast<const uint16_t*>(&lo);
      const int j = row - c0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (k >= count) break;
        const uint32_t to = at(xs, col + k, j & ~7) + (j & 7) * 2;
        st_shared16(to, h[k]);
        if (g.first_parts > 1) st_shared16(to + x_part, l[k]);
      }
    }
  }
  fence_all_async();
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_slot;

  // ---- the steps ----
  const int quad = warp & 3, share = warp >> 2, row = quad * 32 + lane;
  const uint32_t my_lanes = tmem + (static_cast<uint32_t>(quad) << 21);
  const bool rows_here = quad * 32 < mp;
  bool ok = true, issuer = false;
  uint32_t phase = 0;
  if (warp == 0) issuer = elect_one();
  // the products issued so far, waited for by everyone
  auto finish = [&](bool report) {
    if (ok && issuer && report) commit_one(bar);
    if (ok) ok = bar_wait(bar, phase);
    phase ^= 1;
    fence_after();
  };
  // before the next product: what was written to shared memory is seen, what is in TMEM has been read
  auto ready = [&] {
    fence_async();
    fence_before();
    __syncthreads();
    fence_after();
  };
  // sums over K of products of operands in one or two parts; steps of K of a K-major operand lie 32 bytes apart within
  // a tile of 64, those of X as P's partner 16 rows.  The products of low parts come first: the tensor core cuts its
  // sums to 24 bits at every instruction, which costs nothing while they are small.
  auto multiply = [&](uint32_t a, uint32_t a_low, int a_parts, uint32_t b, uint32_t b_low, int b_parts, int K, int N,
                      bool b_mn) {
    if (!ok || !issuer) return;
    const uint32_t idesc = instr_desc(false, false, b_mn, 128, N);
    bool some = false;
    auto each = [&](auto f) {
      for (int k = 0; k < K / 16; ++k) {
        const uint32_t k_off = (k >> 2) * tile + (k & 3) * 32;
        f(operand_desc(a + k_off, 0), b_mn ? operand_desc(b + k * 2048, tile) : operand_desc(b + k_off, 0));
      }
    };
    auto add = [&](uint64_t da, uint64_t db) {
      mma_one(tmem, da, db, idesc, some);
      some = true;
    };
    if (a_parts > 1 || b_parts > 1)
      each([&](uint64_t da, uint64_t db) {
        if (a_parts > 1) add(da + (a_low >> 4), db);
        if (b_parts > 1) add(da, db + (b_low >> 4));
      });
    each(add);
  };
  // 16 sums of this thread's row, from column c
  auto load = [&](int c, float (&v)[kCols]) {
    __syncwarp();
    tmem_ld16(my_lanes + c, v);
    tmem_ld_wait(v);
  };
  // 8 values of a row in one or two parts
  auto put = [&](uint32_t from, uint32_t part, int r, int c, const float (&w)[8], bool two) {
    uint4 hi, lo;
    split8(w, hi, lo);
    const uint32_t to = at(from, r, c);
    st_shared(to, hi);
    if (two) st_shared(to + part, lo);
  };

  for (int step = 0; step < g.steps; ++step) {
    const int parts = step < g.fine ? 2 : 1, x_parts = step == 0 ? min(parts, g.first_parts) : parts;
    const bool last = step + 1 == g.steps;
    const float rest = step == 0 ? x0.unit : 1.f;       // what the first X lacks of the norm
    const float gram = rest * rest * (kScaleA / (kScaleX * kScaleX));

    // A = X X^T
    if (nk > 0) multiply(xs, x_part, x_parts, xs, x_part, x_parts, nk, mp, false);
    finish(!(g.stall && which == 0 && rank == 0 && step == 0));
    if (ctas == 1) {
      for (int c = share * kCols; c < mp && rows_here; c += 64) {
        float v[kCols];
        load(c, v);
#pragma unroll
        for (int k = 0; k < kCols; k += 8) {
          float w[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) w[q] = v[k + q] * gram;
          if (row < mp && c + k < mp) put(as, a_part, row, c + k, w, parts > 1);
        }
      }
    } else {
      // this CTA's sums in A's place, column after column
      for (int c = share * kCols; c < mp && rows_here; c += 64) {
        float v[kCols];
        load(c, v);
#pragma unroll
        for (int k = 0; k < kCols; ++k)
          if (row < mp && c + k < mp) st_shared1(as + ((c + k) * mp + row) * 4, v[k]);
      }
      meet_cluster();
      // a share of the groups of 8 columns over all the CTAs: at most 128 x 16 / 2 of them, 2 a thread
      constexpr int kShare = 128 * 16 / 2 / kThreads;
      float sum[kShare][8];
#pragma unroll
      for (int s = 0; s < kShare; ++s) {
        const int i = s * kThreads + static_cast<int>(threadIdx.x);
#pragma unroll
        for (int q = 0; q < 8; ++q) sum[s][q] = 0.f;
        const int g8 = i / mp, r = i - g8 * mp, col = (g8 * ctas + rank) * 8;
        if (col >= mp) continue;
        for (int k = 0; k < ctas; ++k) {
          const uint32_t from = in_cta(as + (col * mp + r) * 4, k);
#pragma unroll
          for (int q = 0; q < 8; ++q) sum[s][q] += ld_there(from + q * mp * 4);
        }
      }
      meet_cluster();
#pragma unroll
      for (int s = 0; s < kShare; ++s) {
        const int i = s * kThreads + static_cast<int>(threadIdx.x);
        const int g8 = i / mp, r = i - g8 * mp, col = (g8 * ctas + rank) * 8;
        if (col >= mp) continue;
        uint4 hi, lo;
#pragma unroll
        for (int q = 0; q < 8; ++q) sum[s][q] *= gram;
        split8(sum[s], hi, lo);
        for (int k = 0; k < ctas; ++k) {
          const uint32_t to = in_cta(at(as, r, col), k);
          st_cluster(to, hi.x, hi.y, hi.z, hi.w);
          if (parts > 1) st_cluster(to + a_part, lo.x, lo.y, lo.z, lo.w);
        }
      }
      fence_all_async();
      meet_cluster();
    }
    ready();

    // P = a I + b A + c A^2, in A's place
    multiply(as, a_part, parts, as, a_part, parts, mp, mp, false);
    finish(true);
    const float pa = g.coefficients[3 * step] * kScaleP, pb = g.coefficients[3 * step + 1] * (kScaleP / kScaleA);
    const float pc = g.coefficients[3 * step + 2] * (kScaleP / (kScaleA * kScaleA));
    for (int c = share * kCols; c < mp && rows_here; c += 64) {
      float v[kCols];
      load(c, v);
#pragma unroll
      for (int k = 0; k < kCols; k += 8) {
        if (row >= mp || c + k >= mp) continue;
        float h[8], l[8] = {}, w[8];
        const uint32_t from = at(as, row, c + k);
        Fmt<__half>::unpack8(ld_shared(from), h);
        if (parts > 1) Fmt<__half>::unpack8(ld_shared(from + a_part), l);
#pragma unroll
        for (int q = 0; q < 8; ++q) w[q] = fmaf(pb, h[q] + l[q], pc * v[k + q]) + (row == c + k + q ? pa : 0.f);
        put(as, a_part, row, c + k, w, parts > 1);
      }
    }
    ready();

    // X <- P X
    if (nk > 0) multiply(as, a_part, parts, xs, x_part, x_parts, mp, nk, true);
    finish(true);
    if (!last) {
      for (int c = share * kCols; c < nk && rows_here; c += 64) {
        float v[kCols];
        load(c, v);
#pragma unroll
        for (int k = 0; k < kCols; k += 8) {
          float w[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) w[q] = v[k + q] * (rest / kScaleP);
          if (row < mp && c + k < nk) put(xs, x_part, row, c + k, w, step + 1 < g.fine);
        }
      }
      ready();
      continue;
    }
    ok = __syncthreads_and(ok);
    bool good = ok;
    if (ctas > 1) {
      if (threadIdx.x == 0) ok_here = ok ? 1.f : 0.f;
      meet_cluster();
      for (int k = 0; k < ctas; ++k) good = good && ld_there(in_cta(smem_addr(&ok_here), k)) != 0.f;
    }
    const float out = finite && good ? rest / (kScaleP * kScaleX) : NAN;
    for (int c = share * kCols; c < nk && rows_here; c += 64) {
      float v[kCols];
      load(c, v);
      // a norm that is not finite leaves the state as it was
      if (row >= m || c >= nl || (MUON && !(finite && good))) continue;
#pragma unroll
      for (int k = 0; k < kCols; ++k) v[k] *= out;
      if (MUON) {
        uint4 theta[kCols / 4];
        read_master<kCols>(e, c0 + nl, row, c0 + c, theta);
        step_master<kCols>(e, theta, v);
      }
      write_columns<MUON>(c0 + nl, e, g.out_dtype, row, c0 + c, v);
    }
  }
  if (!ok && threadIdx.x == 0) {
    atomicAdd(&g_small_timeouts, 1u);
    atomicAdd(g.failures, 1u);
  }
  if (!ok && issuer) {
    // leave no product in flight behind
    commit_one(drained);
    bar_wait(drained, 0);
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 0) free_one(tmem, columns);
  if (ctas > 1) meet_cluster();    // the others may still look at this CTA's shared memory
}

// ---- host -------------------------------------------------------------------------

// Bytes of shared memory of a matrix in each of its CTAs.  A product takes 128
// rows of its first operand whatever there are: what it reads past the last part
// of A, rows whose sums nobody looks at, is there as well.
int64_t space_for(const Entry& e) {
  const int64_t m = std::min(e.rows, e.cols), n = std::max(e.rows, e.cols);
  const int64_t mp = round_up(m, 16), slice = round_up(ceil_div(n, ctas_for(e)), 16);
  return 2 * mp * 128 * (ceil_div(slice, 64) + ceil_div(mp, 64)) + (kMostRows - mp) * 128 + 1024;
}

// So much shared memory at least: more than half of an SM's, so that no other CTA
// that takes TMEM, of this launch or of another stream's, shares the SM.  CTAs of
// two clusters that had TMEM on one SM each and waited for it on the other's would
// wait for ever.
constexpr int64_t kAloneBytes = 116 * 1024;

template <typename T, bool MUON, int BYTES>
int launch_small(SmallArgs<BYTES>& a, int count, int ctas, int64_t space, cudaStream_t s) {
  space = std::max(space, kAloneBytes);
  const auto fn = ns_small<T, MUON, BYTES>;
  ZERO_CUDA(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(space)));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(count) * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(space);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  ZERO_CUDA(cudaLaunchKernelEx(&cfg, fn, a));
  return ZERO_OK;
}

template <int BYTES>
int launch_type(const SmallCall& c, SmallArgs<BYTES>& a, int count, int ctas, int64_t space) {
  if (c.muon)
    return c.in_dtype == ZERO_FP16 ? launch_small<__half, true>(a, count, ctas, space, c.stream)
                                   : launch_small<__nv_bfloat16, true>(a, count, ctas, space, c.stream);
  return c.in_dtype == ZERO_FP16   ? launch_small<__half, false>(a, count, ctas, space, c.stream)
         : c.in_dtype == ZERO_BF16 ? launch_small<__nv_bfloat16, false>(a, count, ctas, space, c.stream)
                                   : launch_small<float, false>(a, count, ctas, space, c.stream);
}

// The entries pick[0, count), as many launches as their table takes.
template <int BYTES>
int run_table(const SmallCall& c, const int* pick, int count, int ctas, bool& stall) {
  static thread_local SmallArgs<BYTES> a;
  const int each = static_cast<int>(sizeof(Entry)) + 8 * c.W, most = BYTES / each;
  a.steps = c.steps;
  a.fine = c.fine;
  a.first_parts = c.first_parts;
  a.out_dtype = c.out_dtype;
  a.W = c.W;
  a.mu = c.mu;
  a.nesterov = c.nesterov;
  a.failures = c.failures;
  for (int k = 0; k < 3 * c.steps; ++k) a.coefficients[k] = static_cast<float>(c.coefficients[k]);
  for (int from = 0; from < count; from += most) {
    const int here = std::min(most, count - from);
    int64_t space = 0;
    a.grads_at = here * static_cast<int>(sizeof(Entry) / 8);
    for (int k = 0; k < here; ++k) {
      const Entry& e = c.entries[pick[from + k]];
      space = std::max(space, space_for(e));
      std::memcpy(a.table.data + k * sizeof(Entry), &e, sizeof e);
      if (c.W > 0)
        std::memcpy(a.table.data + here * sizeof(Entry) + static_cast<size_t>(k) * 8 * c.W,
                    c.grads + static_cast<int64_t>(pick[from + k]) * c.W, 8 * static_cast<size_t>(c.W));
    }
    a.stall = std::exchange(stall, false);
    const int rc = launch_type(c, a, here, ctas, space);
    if (rc) return rc;
  }
  return ZERO_OK;
}

}  // namespace

namespace ns {

bool small_fits(int64_t rows, int64_t cols) {
  return std::min(rows, cols) <= kMostRows && std::max(rows, cols) <= kMostSlice * kMostCtas;
}

int run_small(const SmallCall& c, bool& stall) {
  std::vector<int> order(c.count);
  for (int k = 0; k < c.count; ++k) order[k] = k;
  std::stable_sort(order.begin(), order.end(),
                   [&](int a, int b) { return ctas_for(c.entries[a]) > ctas_for(c.entries[b]); });
  for (int from = 0; from < c.count;) {
    // matrices that take as many CTAs go together; where there are SMs for it, those that take fewer go with them
    const int ctas = ctas_for(c.entries[order[from]]);
    int to = from;
    while (to < c.count && (ctas_for(c.entries[order[to]]) == ctas || (c.count - from) * ctas <= sm_count())) ++to;
    const int64_t bytes = static_cast<int64_t>(to - from) * (static_cast<int64_t>(sizeof(Entry)) + 8 * c.W);
    const int rc = bytes <= kSmallTable ? run_table<kSmallTable>(c, &order[from], to - from, ctas, stall)
                                        : run_table<kLargeTable>(c, &order[from], to - from, ctas, stall);
    if (rc) return rc;
    from = to;
  }
  return ZERO_OK;
}

cudaError_t small_timeouts(unsigned int* out) { return cudaMemcpyFromSymbol(out, g_small_timeouts, sizeof *out); }

}  // namespace ns
}  // namespace zero
