// The global gradient norm over many tensors, and clipping by it.
//
//   g_e  = (G_0[e] + ... + G_{W-1}[e]) / W        (ranks in order, fp32)
//   norm = sqrt(sum over every tensor's elements e of g_e^2)
//   coef = min(1, max_norm / (norm + 1e-6))
//
// zero_grad_norm computes norm, zero_grad_clip writes round(coef g), and
// zero_step_clipped runs the step on coef g: its first pass reads the W
// gradient vectors once, keeps g in fp32 and sums the squares, its second
// runs Adam on coef g.  The fp32 mean costs 8 bytes an element (written and
// read) where reading the W gradients again would cost 2 W, which is faster
// for 1 and 2 ranks.
//
// What bounds them: HBM.  The clipped step of 124M elements of 8 ranks moves 2 W
// + 4 bytes an element in its first pass (2.49 GB in 358 us, 6.95 TB/s) and 30
// in its second (3.73 GB in 548 us, 6.8 TB/s), 912 to 918 us in all; the same
// bytes at the measured copy rate take 917.  The norm and the clipped mean of
// 148 tensors of 4 ranks, 20M elements, take 34 + 36 us on the device (160 and
// 200 MB); a Python caller spends 220 us on 592 tensor objects.
//
// Squares are summed in fp32 by each thread and in fp64 from there on: within
// a block, and over the blocks in their order by the last block to finish, so
// the norm does not depend on the order in which blocks run.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "launch.cuh"
#include "step_math.cuh"
#include "zero_context.h"
#include "zero_internal.h"
#include "zero_step.h"

namespace zero {
namespace {

using namespace dev;
using host::ceil_div;
using host::fail;

constexpr int kThreads = 256;
// Blocks of the mean pass on each SM: 2 took 918 us for the whole clipped step of
// 124M elements of 8 ranks, 3 took 927 and 4 took 936.
constexpr int kMeanBlocksPerSm = 2;
constexpr int kMaxBlocks = 1024;           // partial sums of one launch
constexpr double kClipEps = 1e-6;
// Up to this many ranks the clipped step reads the gradients twice (4 W bytes an
// element) instead of writing and reading their fp32 mean (2 W + 8).  At 60M
// elements: 1 rank 312 us, 2 ranks 312, 3 ranks 388 against 381 for 4 through
// the mean.
constexpr int kDirectRanks = 2;

// Workspace: the number of blocks that have finished (0 between calls), then
// a partial sum of squares for each block.
struct NormSpace {
  unsigned int* done;
  double* part;
};
constexpr int64_t kNormBytes = 256 + kMaxBlocks * 8;

NormSpace norm_space(void* ws) {
  return {static_cast<unsigned int*>(ws), reinterpret_cast<double*>(static_cast<char*>(ws) + 256)};
}

// ---- element types -------------------------------------------------------------

// 8 consecutive elements of T, read and written in one access, as floats.
template <typename T>
struct Eight {
  using Raw = uint4;
  static __device__ __forceinline__ Raw raw(const T* p) { return ld_16B(p); }
  static __device__ __forceinline__ void unpack(const Raw& r, float (&f)[8]) { Fmt<T>::unpack8(r, f); }
  static __device__ __forceinline__ void store(T* p, const float (&f)[8]) { st_16B(p, Fmt<T>::pack8(f)); }
  static __device__ __forceinline__ float load1(const T* p) { return Fmt<T>::load1(p, 0); }
  static __device__ __forceinline__ void store1(T* p, float x) { Fmt<T>::store1(p, 0, x); }
};

template <>
struct Eight<float> {
  struct Raw {
    float f[8];
  };
  static __device__ __forceinline__ Raw raw(const float* p) {
    Raw r;
    ld_32B(p, r.f);
    return r;
  }
  static __device__ __forceinline__ void unpack(const Raw& r, float (&f)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = r.f[k];
  }
  static __device__ __forceinline__ void store(float* p, const float (&f)[8]) { st_32B(p, f); }
  static __device__ __forceinline__ float load1(const float* p) { return *p; }
  static __device__ __forceinline__ void store1(float* p, float x) { *p = x; }
};

__device__ __forceinline__ void ld_32B_words(const void* p, uint4& a, uint4& b) {
  asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
               : "l"(p));
}

// ---- sums over the blocks ---------------------------------------------------------

// Adds the block's sum of squares to its slot; the last block of the launch
// adds all the slots [0, blocks) in order and, with `norm`, writes the root.
__device__ __forceinline__ void finish_sum(float mine, const NormSpace& ws, unsigned int first, unsigned int blocks,
                                           float* norm) {
  __shared__ double warp_sum[kThreads / 32];
  __shared__ bool last;
  double s = mine;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    double t = 0.0;
    for (int k = 0; k < kThreads / 32; ++k) t += warp_sum[k];
    ws.part[first + blockIdx.x] = t;
    __threadfence();
    last = norm != nullptr && atomicAdd(ws.done, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  double t = 0.0;
  for (unsigned int k = threadIdx.x; k < blocks; k += kThreads) t += __ldcg(ws.part + k);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = t;
  __syncthreads();
  if (threadIdx.x == 0) {
    double all = 0.0;
    for (int k = 0; k < kThreads / 32; ++k) all += warp_sum[k];
    *norm = static_cast<float>(sqrt(all));
    *ws.done = 0;
  }
}

__device__ __forceinline__ float clip_coef(float norm, float max_norm) {
  return fminf(1.f, __fdiv_rn(max_norm, __fadd_rn(norm, static_cast<float>(kClipEps))));
}

// ---- many tensors ------------------------------------------------------------------
//
// The tensors' sizes and addresses travel as the kernel's parameters, so a
// call needs no copy to the device; a list that does not fit one launch takes
// several.  Work is cut into chunks of kChunk elements of one tensor.  There
// are two sizes of parameters: a launch with the large one takes the host 17
// us, with the small one 6, whatever it holds.

constexpr int kChunk = 8192;
constexpr int kSmallTable = 9 * 1024, kLargeTable = 28 * 1024;   // a launch's parameters may hold 32,764 bytes

template <int BYTES>
struct Table {
  int tensors, W;
  unsigned int chunks;
  int want_out;
  // follows: chunk_start[tensors + 1], then per tensor its element count,
  // W gradient addresses and, with want_out, an output address
  alignas(8) unsigned char data[BYTES];

  __host__ __device__ int64_t words() const { return 1 + W + want_out; }
  __host__ __device__ const unsigned int* starts() const { return reinterpret_cast<const unsigned int*>(data); }
  __host__ __device__ const int64_t* row(int t) const {
    return reinterpret_cast<const int64_t*>(data + (tensors + 2) / 2 * 8) + t * words();
  }
};

// 8 elements of every rank at element i, summed in rank order in fp32.  WC > 0:
// W known at compile time, all its loads in flight at once; WC == 0: any W,
// 8 ranks at a time.  `rank` gives rank w's vector.
template <typename T, int WC, typename F>
__device__ __forceinline__ void sum_ranks8(F rank, int64_t i, int W, float (&sum)[8]) {
  constexpr int kAtOnce = WC > 0 ? WC : 8;
  for (int w0 = 0; w0 < (WC > 0 ? 1 : W); w0 += kAtOnce) {
    typename Eight<T>::Raw raw[kAtOnce];
#pragma unroll
    for (int w = 0; w < kAtOnce; ++w)
      if (WC > 0 || w0 + w < W) raw[w] = Eight<T>::raw(rank(w0 + w) + i);
#pragma unroll
    for (int w = 0; w < kAtOnce; ++w) {
      if (WC == 0 && w0 + w >= W) break;
      float f[8];
      Eight<T>::unpack(raw[w], f);
#pragma unroll
      for (int k = 0; k < 8; ++k) sum[k] = w0 + w == 0 ? f[k] : __fadd_rn(sum[k], f[k]);
    }
  }
}

// The same for 16 elements, in 32-byte loads where `wide` says that every
// rank's vector allows them.
template <typename T, int WC, typename F>
__device__ __forceinline__ void sum_ranks16(F rank, int64_t i, int W, bool wide, float (&sum)[2][8]) {
  constexpr int kAtOnce = WC > 0 && WC <= 8 ? WC : 8;
  for (int w0 = 0; w0 < (WC > 0 ? WC : W); w0 += kAtOnce) {
    uint4 raw[kAtOnce][2];
#pragma unroll
    for (int w = 0; w < kAtOnce; ++w) {
      if (WC > 0 || w0 + w < W) {
        if (wide) {
          ld_32B_words(rank(w0 + w) + i, raw[w][0], raw[w][1]);
        } else {
          raw[w][0] = ld_16B(rank(w0 + w) + i);
          raw[w][1] = ld_16B(rank(w0 + w) + i + 8);
        }
      }
    }
#pragma unroll
    for (int w = 0; w < kAtOnce; ++w) {
      if (WC == 0 && w0 + w >= W) break;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float f[8];
        Fmt<T>::unpack8(raw[w][h], f);
#pragma unroll
        for (int k = 0; k < 8; ++k) sum[h][k] = w0 + w == 0 ? f[k] : __fadd_rn(sum[h][k], f[k]);
      }
    }
  }
}

template <typename T, typename F>
__device__ __forceinline__ float mean1(F rank, int64_t i, int W, bool pow2, float inv_w) {
  float g = Eight<T>::load1(rank(0) + i);
  for (int w = 1; w < W; ++w) g = __fadd_rn(g, Eight<T>::load1(rank(w) + i));
  return rank_mean(g, W, inv_w, pow2);
}

// The warp's 32 x 8 values v, lane after lane, to out, which lies `shift`
// elements (1..7) before a boundary of 8: every lane but the last stores one
// whole group made of its own tail and the next lane's head; the first
// lane's head and the last lane's tail go element by element.
template <typename T>
__device__ __forceinline__ void store_shifted(T* out, int shift, const float (&v)[8], int lane) {
  float x[16];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    x[k] = v[k];
    x[8 + k] = __shfl_down_sync(0xffffffffu, v[k], 1);
  }
  if (lane == 0) {
#pragma unroll
    for (int k = 0; k < 7; ++k)
      if (k < shift) Eight<T>::store1(out + k, v[k]);
  }
  if (lane == 31) {
#pragma unroll
    for (int k = 1; k < 8; ++k)
      if (k >= shift) Eight<T>::store1(out + k, v[k]);
  }
  // x moved down by `shift` places, one bit of it at a time
#pragma unroll
  for (int bit = 1; bit < 8; bit *= 2) {
    if (shift & bit) {
#pragma unroll
      for (int k = 0; k + bit < 16; ++k) x[k] = x[k + bit];
    }
  }
  if (lane < 31) {
    float y[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = x[k];
    Eight<T>::store(out + shift, y);
  }
}

// One pass over a table's tensors: the sum of squares of the mean (CLIP
// false), or the clipped mean (CLIP true).  Tensors whose W gradients lie
// alike relative to a group of 8 elements are read a group at a time; the
// output may lie anywhere.  The clipping pass walks the chunks backwards:
// what the norm's pass read last is what L2 still holds.
template <typename T, int WC, bool CLIP, int BYTES>
__global__ void __launch_bounds__(kThreads) tensors_pass(const __grid_constant__ Table<BYTES> t, NormSpace ws,
                                                         unsigned int first, unsigned int blocks, float* norm,
                                                         float max_norm) {
  await_previous();
  const int W = WC > 0 ? WC : t.W;
  const bool pow2 = (W & (W - 1)) == 0;
  const float inv_w = 1.f / W;
  const int lane = threadIdx.x & 31;
  float coef = 1.f;
  if (CLIP) {
    const float n = *norm;
    coef = isfinite(n) ? clip_coef(n, max_norm) : 1.f;
  }
  float squares = 0.f;
  for (unsigned int at = blockIdx.x; at < t.chunks; at += gridDim.x) {
    const unsigned int chunk = CLIP ? t.chunks - 1 - at : at;
    // the last tensor that starts at or before this chunk
    int lo = 0, hi = t.tensors - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (t.starts()[mid] <= chunk) lo = mid;
      else hi = mid - 1;
    }
    const int64_t* row = t.row(lo);
    const int64_t numel = row[0], begin = static_cast<int64_t>(chunk - t.starts()[lo]) * kChunk;
    const int64_t end = min(numel, begin + kChunk);
    auto rank = [&](int w) { return reinterpret_cast<const T*>(row[1 + w]); };
    T* out = CLIP ? reinterpret_cast<T*>(row[1 + W]) : nullptr;
    // elements from a pointer to the next boundary of 8 elements
    auto to_boundary = [](int64_t p) { return static_cast<int>((-p & (8 * static_cast<int64_t>(sizeof(T)) - 1)) / sizeof(T)); };
    const int head = to_boundary(row[1]);
    bool alike = true;
    for (int w = 1; w < W; ++w) alike = alike && to_boundary(row[1 + w]) == head;
    int64_t v0 = min(begin + head, end), v1 = v0;       // [v0, v1): whole groups of 8
    if (alike) v1 = v0 + (end - v0) / 8 * 8;
    const int shift = CLIP ? to_boundary(row[1 + W] + v0 * static_cast<int64_t>(sizeof(T))) : 0;
    // whole warps of groups, then the groups left over
    const int64_t vw = v0 + (v1 - v0) / 256 * 256;
    for (int64_t i = v0 + threadIdx.x * 8; i < v1; i += kThreads * 8) {
      float g[8];
      sum_ranks8<T, WC>(rank, i, W, g);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        g[k] = rank_mean(g[k], W, inv_w, pow2);
        if (CLIP) g[k] *= coef;
        else squares = fmaf(g[k], g[k], squares);
      }
      if (CLIP) {
        if (shift == 0) {
          Eight<T>::store(out + i, g);
        } else if (i - lane * 8 < vw) {
          store_shifted<T>(out + i, shift, g, lane);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) Eight<T>::store1(out + i + k, g[k]);
        }
      }
    }
    // what is left: the head (or everything, where the gradients lie unlike) and the tail
    auto one = [&](int64_t i) {
      const float g = mean1<T>(rank, i, W, pow2, inv_w);
      if (CLIP) Eight<T>::store1(out + i, g * coef);
      else squares = fmaf(g, g, squares);
    };
    for (int64_t i = begin + threadIdx.x; i < v0; i += kThreads) one(i);
    for (int64_t i = v1 + threadIdx.x; i < end; i += kThreads) one(i);
  }
  if (!CLIP) finish_sum(squares, ws, first, blocks, norm);
}

// ---- the step's two passes --------------------------------------------------------------

struct MeanNormArgs {
  int W;
  const void* grads[kMaxRanks];
  int64_t n;
  float* mean;               // NULL: the update will read the gradients again
  int wide;                  // every gradient vector is 32-byte aligned
  float inv_w;
  NormSpace ws;
  float* norm;
};

// 16 elements of each rank at a time in one 32-byte load (as 8, at twice the
// threads, the pass ran at 0.94 of this rate).
template <typename GT, int WC>
__global__ void __launch_bounds__(kThreads) mean_norm_pass(const __grid_constant__ MeanNormArgs a) {
  await_previous();
  const int W = WC > 0 ? WC : a.W;
  const bool pow2 = (W & (W - 1)) == 0;
  auto rank = [&](int w) { return static_cast<const GT*>(a.grads[w]); };
  float squares = 0.f;
  const int64_t groups = a.n >> 4;
  const bool wide = a.wide;
  for (int64_t gi = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; gi < groups;
       gi += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t i = gi << 4;
    float sum[2][8];
    sum_ranks16<GT, WC>(rank, i, W, wide, sum);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        sum[h][k] = rank_mean(sum[h][k], W, a.inv_w, pow2);
        squares = fmaf(sum[h][k], sum[h][k], squares);
      }
      if (a.mean) st_32B(a.mean + i + 8 * h, sum[h]);
    }
  }
  if (blockIdx.x == 0) {
    for (int64_t e = (groups << 4) + threadIdx.x; e < a.n; e += kThreads) {
      const float g = mean1<GT>(rank, e, W, pow2, a.inv_w);
      if (a.mean) a.mean[e] = g;
      squares = fmaf(g, g, squares);
    }
  }
  finish_sum(squares, a.ws, 0, gridDim.x, a.norm);
}

struct ClippedArgs {
  const float* mean;
  const void* grads[kDirectRanks];
  float* master;
  float* m;
  float* v;
  Seg segs[kMaxSegs];
  AdamCoef coef;
  const float* norm;
  float max_norm;
};

// Adam on coef * g over a segment; the ZeRO-3 gather of its old 16-bit values
// (pre_out) as in the fused step.  g comes from the fp32 mean (WC == 0) or
// again from the WC ranks' gradients.  A norm that is not finite leaves the
// state as it was.  The groups run from the segment's end to its start: the
// end of the mean is what L2 still holds of the pass before.
template <typename GT, typename OT, int WC>
__global__ void __launch_bounds__(kThreads) clipped_update(const __grid_constant__ ClippedArgs a) {
  await_previous();
  constexpr bool pow2 = (WC & (WC - 1)) == 0;
  const Seg& seg = a.segs[blockIdx.y];
  const float norm = *a.norm;
  const bool update = isfinite(norm);
  const float coef = update ? clip_coef(norm, a.max_norm) : 0.f;
  auto rank = [&](int w) { return static_cast<const GT*>(a.grads[w]); };
  OT* out = static_cast<OT*>(seg.out);
  OT* pre = static_cast<OT*>(seg.pre_out);
  if (!update && !pre) return;
  const int64_t lo = seg.lo, hi = seg.lo + seg.len;
  const int64_t g0 = (lo + 7) >> 3, g1 = hi >> 3;
  const bool out_vec = ((reinterpret_cast<uintptr_t>(out) - static_cast<uintptr_t>(lo) * 2u) & 15u) == 0;
  const bool pre_vec = out_vec && ((reinterpret_cast<uintptr_t>(pre) - static_cast<uintptr_t>(lo) * 2u) & 15u) == 0;
  auto one = [&](int64_t e) {
    const int64_t j = e - lo;
    if (pre) pre[j] = out[j];
    if (!update) return;
    float g;
    if constexpr (WC > 0) g = mean1<GT>(rank, e, WC, pow2, a.coef.inv_w);
    else g = a.mean[e];
    float th = a.master[e], m = a.m[e], v = a.v[e];
    adam_element(__fmul_rn(g, coef), th, m, v, a.coef);
    a.master[e] = th;
    a.m[e] = m;
    a.v[e] = v;
    Fmt<OT>::store1(out, j, th);
  };
  for (int64_t g = g1 - 1 - (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x); g >= g0;
       g -= static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t i = g << 3, j = i - lo;
    if (pre) {
      if (pre_vec) {
        st_16B(pre + j, ld_16B(out + j));
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) pre[j + k] = out[j + k];
      }
    }
    if (!update) continue;
    float x[8], th[8], m[8], v[8];
    typename Eight<GT>::Raw raw[WC > 0 ? WC : 1];
    if constexpr (WC > 0) {
#pragma unroll
      for (int w = 0; w < WC; ++w) raw[w] = Eight<GT>::raw(rank(w) + i);
    } else {
      ld_32B(a.mean + i, x);
    }
    ld_32B(a.master + i, th);
    ld_32B(a.m + i, m);
    ld_32B(a.v + i, v);
    if constexpr (WC > 0) {
#pragma unroll
      for (int w = 0; w < WC; ++w) {
        float f[8];
        Eight<GT>::unpack(raw[w], f);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = w == 0 ? f[k] : __fadd_rn(x[k], f[k]);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = rank_mean(x[k], WC, a.coef.inv_w, pow2);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) adam_element(__fmul_rn(x[k], coef), th[k], m[k], v[k], a.coef);
    st_32B(a.master + i, th);
    st_32B(a.m + i, m);
    st_32B(a.v + i, v);
    if (out_vec) {
      st_16B(out + j, Fmt<OT>::pack8(th));
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) Fmt<OT>::store1(out, j + k, th[k]);
    }
  }
  if (blockIdx.x == 0) {
    const int64_t head = g0 < g1 ? g0 << 3 : hi, tail = g0 < g1 ? g1 << 3 : hi;
    for (int64_t e = lo + threadIdx.x; e < head; e += kThreads) one(e);
    for (int64_t e = tail + threadIdx.x; e < hi; e += kThreads) one(e);
  }
}

using ClippedFn = void (*)(const ClippedArgs);

template <typename GT, typename OT>
ClippedFn pick_clipped_w(int direct) {
  switch (direct) {
    case 1: return clipped_update<GT, OT, 1>;
    case 2: return clipped_update<GT, OT, 2>;
    default: return clipped_update<float, OT, 0>;
  }
}

ClippedFn pick_clipped(int gdt, int wdt, int direct) {
  if (gdt == kF16) return wdt == kF16 ? pick_clipped_w<__half, __half>(direct) : pick_clipped_w<__half, __nv_bfloat16>(direct);
  return wdt == kF16 ? pick_clipped_w<__nv_bfloat16, __half>(direct) : pick_clipped_w<__nv_bfloat16, __nv_bfloat16>(direct);
}

using MeanNormFn = void (*)(const MeanNormArgs);

template <typename GT>
MeanNormFn pick_mean_norm(int W) {
  switch (W) {
    case 1: return mean_norm_pass<GT, 1>;
    case 2: return mean_norm_pass<GT, 2>;
    case 4: return mean_norm_pass<GT, 4>;
    case 8: return mean_norm_pass<GT, 8>;
    case 16: return mean_norm_pass<GT, 16>;
    default: return mean_norm_pass<GT, 0>;
  }
}

// ---- host -------------------------------------------------------------------------------

int check_tensors(int W, int64_t n_tensors, const int64_t* numels, int dtype, const void* const* grads,
                  void* const* out) {
  if (W < 1 || W > kMaxRanks) return fail(ZERO_E_ARG, "W=%d outside [1, %d]", W, kMaxRanks);
  if (n_tensors < 0 || n_tensors > (int64_t(1) << 24)) return fail(ZERO_E_ARG, "%lld tensors", (long long)n_tensors);
  if (dtype != ZERO_FP16 && dtype != ZERO_BF16 && dtype != ZERO_FP32)
    return fail(ZERO_E_ARG, "the gradients' format must be ZERO_FP16, ZERO_BF16 or ZERO_FP32");
  if (n_tensors > 0 && (numels == nullptr || grads == nullptr)) return fail(ZERO_E_ARG, "numels and grads are required");
  const uintptr_t size = dtype == ZERO_FP32 ? 4 : 2;
  for (int64_t t = 0; t < n_tensors; ++t) {
    if (numels[t] < 0 || numels[t] > (int64_t(1) << 46))
      return fail(ZERO_E_ARG, "tensor %lld has %lld elements", (long long)t, (long long)numels[t]);
    if (numels[t] == 0) continue;
    for (int w = 0; w <= W; ++w) {
      if (w == W && out == nullptr) break;
      const void* p = w < W ? grads[w * n_tensors + t] : out[t];
      if (p == nullptr) return fail(ZERO_E_ARG, "tensor %lld: a pointer is NULL", (long long)t);
      if (reinterpret_cast<uintptr_t>(p) % size) return fail(ZERO_E_ALIGN, "tensor %lld is not aligned to its elements", (long long)t);
    }
  }
  return ZERO_OK;
}

// Tensors that a table of `bytes` holds.
int64_t table_tensors(int bytes, int W, bool out) { return (bytes - 16) / (8 * (1 + W + (out ? 1 : 0)) + 4); }

// Fill tables from the list and call launch(table, last) for each.
template <int BYTES, typename F>
int for_tables_of(int W, int64_t n_tensors, const int64_t* numels, const void* const* grads, void* const* out,
                  F launch) {
  static thread_local Table<BYTES> t;
  static thread_local int64_t pick[BYTES / 16];   // the tensors of one launch
  const int64_t most = table_tensors(BYTES, W, out != nullptr);
  int64_t k = 0;
  do {
    int64_t chunks = 0;
    int count = 0;
    while (k < n_tensors && count < most) {
      const int64_t c = ceil_div(numels[k], kChunk);
      if (c > INT32_MAX) return fail(ZERO_E_ARG, "tensor %lld has too many elements", (long long)k);
      if (count > 0 && chunks + c > INT32_MAX) break;
      if (c > 0) {
        pick[count++] = k;
        chunks += c;
      }
      ++k;
    }
    t.tensors = count;
    t.W = W;
    t.want_out = out ? 1 : 0;
    t.chunks = static_cast<unsigned int>(chunks);
    unsigned int* starts = const_cast<unsigned int*>(t.starts());
    unsigned int at = 0;
    for (int j = 0; j < t.tensors; ++j) {
      starts[j] = at;
      at += static_cast<unsigned int>(ceil_div(numels[pick[j]], kChunk));
      int64_t* row = const_cast<int64_t*>(t.row(j));
      row[0] = numels[pick[j]];
      for (int w = 0; w < W; ++w) row[1 + w] = reinterpret_cast<int64_t>(grads[w * n_tensors + pick[j]]);
      if (out) row[1 + W] = reinterpret_cast<int64_t>(out[pick[j]]);
    }
    starts[t.tensors] = at;
    const int rc = launch(t, k >= n_tensors);
    if (rc) return rc;
  } while (k < n_tensors);
  return ZERO_OK;
}

template <typename F>
int for_tables(int W, int64_t n_tensors, const int64_t* numels, const void* const* grads, void* const* out, F launch) {
  return n_tensors <= table_tensors(kSmallTable, W, out != nullptr)
             ? for_tables_of<kSmallTable>(W, n_tensors, numels, grads, out, launch)
             : for_tables_of<kLargeTable>(W, n_tensors, numels, grads, out, launch);
}

unsigned pass_blocks(int64_t chunks, int64_t most) {
  return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>({chunks, static_cast<int64_t>(sm_count()) * 4, most})));
}

int check_norm_args(const float* norm, const void* workspace, int64_t workspace_bytes) {
  if (norm == nullptr) return fail(ZERO_E_ARG, "norm is NULL");
  if (reinterpret_cast<uintptr_t>(norm) % 4) return fail(ZERO_E_ALIGN, "norm must be 4-byte aligned");
  if (workspace == nullptr) return fail(ZERO_E_ARG, "workspace is NULL");
  if (reinterpret_cast<uintptr_t>(workspace) % 256) return fail(ZERO_E_ALIGN, "workspace must be 256-byte aligned");
  if (workspace_bytes < kNormBytes)
    return fail(ZERO_E_ARG, "workspace of %lld bytes: %lld are needed", (long long)workspace_bytes, (long long)kNormBytes);
  return ZERO_OK;
}

// One launch over a list that fits its table.
template <typename T, int WC, bool CLIP, int BYTES>
cudaError_t launch_table(const Table<BYTES>& t, unsigned blocks, const NormSpace& ws, unsigned first, float* norm,
                         float max_norm, cudaStream_t s) {
  return launch_chained(tensors_pass<T, WC, CLIP, BYTES>, dim3(blocks), kThreads, 0, s, t, ws, first, first + blocks,
                        norm, max_norm);
}

template <typename T, bool CLIP, int BYTES>
cudaError_t launch_tensors_w(const Table<BYTES>& t, unsigned blocks, const NormSpace& ws, unsigned first, float* norm,
                             float max_norm, cudaStream_t s) {
  switch (t.W) {
    case 1: return launch_table<T, 1, CLIP>(t, blocks, ws, first, norm, max_norm, s);
    case 2: return launch_table<T, 2, CLIP>(t, blocks, ws, first, norm, max_norm, s);
    case 4: return launch_table<T, 4, CLIP>(t, blocks, ws, first, norm, max_norm, s);
    case 8: return launch_table<T, 8, CLIP>(t, blocks, ws, first, norm, max_norm, s);
    default: return launch_table<T, 0, CLIP>(t, blocks, ws, first, norm, max_norm, s);
  }
}

template <bool CLIP, int BYTES>
cudaError_t launch_tensors(const Table<BYTES>& t, int dtype, unsigned blocks, const NormSpace& ws, unsigned first,
                           float* norm, float max_norm, cudaStream_t s) {
  if (dtype == ZERO_FP16) return launch_tensors_w<__half, CLIP>(t, blocks, ws, first, norm, max_norm, s);
  if (dtype == ZERO_BF16) return launch_tensors_w<__nv_bfloat16, CLIP>(t, blocks, ws, first, norm, max_norm, s);
  return launch_tensors_w<float, CLIP>(t, blocks, ws, first, norm, max_norm, s);
}

}  // namespace

int64_t clip_workspace_bytes(int W, int64_t n_pad) {
  return kNormBytes + (W <= kDirectRanks ? 0 : host::round_up(n_pad * 4, 256));
}

float* clip_mean(void* workspace) { return reinterpret_cast<float*>(static_cast<char*>(workspace) + kNormBytes); }

cudaError_t launch_mean_norm(int W, int grad_dtype, const void* const* grads, int64_t n_pad, void* workspace,
                             float* norm, cudaStream_t stream, int64_t* launches) {
  MeanNormArgs a;
  std::memset(&a, 0, sizeof a);
  a.W = W;
  for (int w = 0; w < W; ++w) a.grads[w] = grads[w];
  a.n = n_pad;
  a.mean = W <= kDirectRanks ? nullptr : clip_mean(workspace);
  a.wide = 1;
  for (int w = 0; w < W; ++w) a.wide = a.wide && host::aligned32(grads[w]);
  a.inv_w = static_cast<float>(1.0 / W);
  a.ws = norm_space(workspace);
  a.norm = norm;
  const MeanNormFn fn = grad_dtype == kF16 ? pick_mean_norm<__half>(W) : pick_mean_norm<__nv_bfloat16>(W);
  const int64_t resident = static_cast<int64_t>(sm_count()) * kMeanBlocksPerSm;
  const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>({n_pad / 16 / kThreads + 1, resident, kMaxBlocks}));
  ++*launches;
  return launch_chained(fn, dim3(static_cast<unsigned>(blocks)), kThreads, 0, stream, a);
}

cudaError_t launch_clipped_update(const FusedLaunch& f, const float* mean, const float* norm, float max_norm,
                                  cudaStream_t stream, int64_t* launches) {
  if (f.nseg <= 0) return cudaSuccess;
  ClippedArgs a;
  std::memset(&a, 0, sizeof a);
  const int direct = f.W <= kDirectRanks ? f.W : 0;
  a.mean = mean;
  for (int w = 0; w < direct; ++w) a.grads[w] = f.grads[w];
  a.master = f.master;
  a.m = f.m;
  a.v = f.v;
  int64_t longest = 0;
  for (int s = 0; s < f.nseg; ++s) {
    a.segs[s] = f.segs[s];
    longest = std::max(longest, f.segs[s].len);
  }
  a.coef = f.coef;
  a.norm = norm;
  a.max_norm = max_norm;
  const int64_t per_seg = ceil_div(static_cast<int64_t>(sm_count()) * 2, f.nseg);
  const int64_t bx = std::max<int64_t>(1, std::min<int64_t>(per_seg, longest / 8 / kThreads + 1));
  const dim3 grid(static_cast<unsigned>(bx), static_cast<unsigned>(f.nseg));
  ++*launches;
  return launch_chained(pick_clipped(f.grad_dtype, f.work_dtype, direct), grid, kThreads, 0, stream, a);
}

}  // namespace zero

using namespace zero;

extern "C" int64_t zero_grad_norm_workspace_bytes(void) { return kNormBytes; }

extern "C" int zero_grad_norm(int W, int64_t n_tensors, const int64_t* numels, int dtype, const void* const* grads,
                              float* norm, void* workspace, int64_t workspace_bytes, void* stream) {
  int rc = check_tensors(W, n_tensors, numels, dtype, grads, nullptr);
  if (rc || (rc = check_norm_args(norm, workspace, workspace_bytes))) return rc;
  const NormSpace ws = norm_space(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // every launch leaves its blocks' sums in slots of its own; the last one adds them up
  const int64_t launches = std::max<int64_t>(1, ceil_div(n_tensors, table_tensors(kLargeTable, W, false)));
  if (launches > kMaxBlocks) return fail(ZERO_E_ARG, "too many tensors (%lld)", (long long)n_tensors);
  unsigned first = 0;
  return for_tables(W, n_tensors, numels, grads, nullptr, [&](const auto& t, bool last) -> int {
    const unsigned blocks = pass_blocks(t.chunks, kMaxBlocks / launches);
    if (first + blocks > kMaxBlocks) return fail(ZERO_E_ARG, "too many elements");
    ZERO_CUDA(launch_tensors<false>(t, dtype, blocks, ws, first, last ? norm : nullptr, 0.f, s));
    first += blocks;
    return ZERO_OK;
  });
}

extern "C" int zero_grad_clip(int W, int64_t n_tensors, const int64_t* numels, int dtype, const void* const* grads,
                              const float* norm, double max_norm, void* const* out, void* stream) {
  if (n_tensors > 0 && out == nullptr) return fail(ZERO_E_ARG, "out is NULL");
  int rc = check_tensors(W, n_tensors, numels, dtype, grads, out);
  if (rc) return rc;
  if (norm == nullptr) return fail(ZERO_E_ARG, "norm is NULL");
  if (reinterpret_cast<uintptr_t>(norm) % 4) return fail(ZERO_E_ALIGN, "norm must be 4-byte aligned");
  const float limit = static_cast<float>(max_norm);
  if (!(limit > 0) || !std::isfinite(limit)) return fail(ZERO_E_ARG, "max_norm %g is not a positive finite fp32 value", max_norm);
  if (n_tensors == 0) return ZERO_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return for_tables(W, n_tensors, numels, grads, out, [&](const auto& t, bool) -> int {
    if (t.tensors == 0) return ZERO_OK;
    ZERO_CUDA(launch_tensors<true>(t, dtype, pass_blocks(t.chunks, INT32_MAX), NormSpace{nullptr, nullptr}, 0u,
                                   const_cast<float*>(norm), limit, s));
    return ZERO_OK;
  });
}
