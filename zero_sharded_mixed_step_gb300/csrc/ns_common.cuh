// What the kernels of the orthogonalised updates share: the description of a
// matrix, reading its values (or the step's direction, formed of the ranks'
// gradients and the momentum) and writing its results.  muon.cu says what is
// computed.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

#include "step_math.cuh"
#include "zero_internal.h"
#include "zero_step.h"

namespace zero {
namespace ns {

using dev::Fmt;

// How the workspace holds X, A and P: times powers of two.
constexpr float kScaleX = 4096.f, kScaleA = 4096.f, kScaleP = 512.f;

// One matrix of a call, in device memory.
struct Entry {
  int rows, cols;              // the caller's
  int transposed;              // X is its transpose
  int wide;                    // the caller's rows allow accesses of 8 values
  const void* in;              // zero_orthogonalize
  void* out;
  int64_t in_stride, out_stride;
  float* master;               // zero_muon_step
  float* momentum;
  void* p16;
  float* mean;                 // the ranks' mean gradient in workspace, or NULL
  float step, keep;            // lr s and 1 - lr wd
  unsigned tile0;              // first of its tiles in the elementwise passes
  int unused;
  uint16_t* x;                 // its first X: the high part, the low part x_part further
  int64_t x_part;
  int64_t ld;                  // of X
};

// What the passes leave for the products: 2^12 over the stored X's norm, and
// whether the input's norm is finite.
struct Norm {
  float unit;
  int finite;
};

constexpr int kMaxSteps = 32;

// ---- values in two parts, and results --------------------------------------------------

__device__ __forceinline__ void split8(const float (&v)[8], uint4& hi, uint4& lo) {
  hi = Fmt<__half>::pack8(v);
  float h[8], rest[8];
  Fmt<__half>::unpack8(hi, h);
#pragma unroll
  for (int k = 0; k < 8; ++k) rest[k] = v[k] - h[k];
  lo = Fmt<__half>::pack8(rest);
}

__device__ __forceinline__ void st_32B_words(void* p, const uint4& a, const uint4& b) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w),
               "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

__device__ __forceinline__ void ld_32B_words(const void* p, uint4& a, uint4& b) {
  asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
               : "l"(p));
}

__device__ __forceinline__ uint4 pack8(int dtype, const float (&v)[8]) {
  return dtype == ZERO_FP16 ? Fmt<__half>::pack8(v) : Fmt<__nv_bfloat16>::pack8(v);
}
__device__ __forceinline__ uint16_t pack1(int dtype, float v) {
  return dtype == ZERO_FP16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// Where N columns from col0 of a row of X lie with the caller, of `columns` that X has.
struct Where {
  bool wide;
  int64_t first, apart;
  int n;
};
template <int N>
__device__ __forceinline__ Where where(const Entry& e, int64_t stride, int columns, int row, int col0) {
  return {e.wide && !e.transposed, e.transposed ? col0 * stride + row : row * stride + col0,
          e.transposed ? stride : 1, min(N, columns - col0)};
}

// N values of the master.  They are read apart from where they are used, all
// before anything is written, so that they are waited for once or not at all.
template <int N>
__device__ __forceinline__ void read_master(const Entry& e, int columns, int row, int col0, uint4 (&w)[N / 4]) {
  const Where at = where<N>(e, e.cols, columns, row, col0);
  const float* p = e.master + at.first;
  if (at.wide) {
#pragma unroll
    for (int k = 0; k < N / 4; k += 2)
      if (4 * k < at.n) ld_32B_words(p + 4 * k, w[k], w[k + 1]);
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (k < at.n) (&w[k / 4].x)[k % 4] = __float_as_uint(p[k * at.apart]);
  }
}

// The new master's values from the old ones and the last product's.
template <int N>
__device__ __forceinline__ void step_master(const Entry& e, const uint4 (&w)[N / 4], float (&v)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = fmaf(-e.step, v[k], e.keep * __uint_as_float((&w[k / 4].x)[k % 4]));
}

// Columns [col0, col0 + N), as far as [0, columns) reaches, of this thread's row
// of X to the caller: the last product's, or the new master's and their 16-bit
// copy.
template <bool UPDATE, int N>
__device__ __forceinline__ void write_columns(int columns, const Entry& e, int dtype, int row, int col0,
                                              const float (&v)[N]) {
  const bool fp32 = !UPDATE && dtype == ZERO_FP32;
  const Where at = where<N>(e, UPDATE ? e.cols : e.out_stride, columns, row, col0);
  if (at.wide) {
    // multiples of 8 columns exist
#pragma unroll
    for (int k = 0; k < N; k += 16) {
      float a[8], b[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        a[q] = v[k + q];
        b[q] = v[k + 8 + q];
      }
      if (UPDATE || fp32) {
        float* to = (UPDATE ? e.master : static_cast<float*>(e.out)) + at.first + k;
        if (k < at.n) dev::st_32B(to, a);
        if (k + 8 < at.n) dev::st_32B(to + 8, b);
      }
      if (!fp32) {
        uint16_t* to = static_cast<uint16_t*>(UPDATE ? e.p16 : e.out) + at.first + k;
        const uint4 lo = pack8(dtype, a), hi = pack8(dtype, b);
        if (k + 8 < at.n && (reinterpret_cast<uintptr_t>(to) & 31) == 0) {
          st_32B_words(to, lo, hi);
        } else {
          if (k < at.n) dev::st_16B(to, lo);
          if (k + 8 < at.n) dev::st_16B(to + 8, hi);
        }
      }
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < N; ++k) {
    if (k >= at.n) break;
    const int64_t to = at.first + k * at.apart;
    if (UPDATE || fp32) (UPDATE ? e.master : static_cast<float*>(e.out))[to] = v[k];
    if (!fp32) static_cast<uint16_t*>(UPDATE ? e.p16 : e.out)[to] = pack1(dtype, v[k]);
  }
}

// ---- reading the matrices ----------------------------------------------------------------

constexpr int kPassThreads = 256, kPassRows = 32, kPassCols = 256;

struct PassArgs {
  const Entry* entries;
  const uint64_t* grads;       // zero_muon_step: W addresses for each entry
  int count;
  unsigned tiles;
  int W;
  float mu;
  int nesterov;
  int two;                     // the second pass writes low parts
  int turns;                   // some matrices are turned
  double* part;                // sums of squares at [block + entry]
  Norm* norms;
};

// A thread's sum of squares.  fp32 holds the squares of values between 2^-63 and 2^63 alone, and a momentum whose
// gradients stay 0 leaves that range in time: eight neighbours whose largest lies outside [2^-40, 2^55] are summed at
// a scale of their own (what vanishes beside that one is 2^-69 of it), so that every finite input has the norm it has.
struct Squares {
  float here = 0.f, low = 0.f, high = 0.f;      // of values as they are, times 2^100, times 2^-100

  // up to 8 values, n of which exist
  __device__ __forceinline__ void add(const float (&u)[8], int n) {
    float most = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) most = fmaxf(most, fabsf(u[k]));
    if (most >= 0x1p-40f && most <= 0x1p55f) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < n) here = fmaf(u[k], u[k], here);
      return;
    }
    const bool small = most < 0x1p-40f;          // or nothing but NaN
    const float scale = small ? 0x1p100f : 0x1p-100f;
    float s = small ? low : high;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) s = fmaf(u[k] * scale, u[k] * scale, s);
    (small ? low : high) = s;
  }
  __device__ __forceinline__ double total() const {
    double s = here;
    if (low != 0.f || high != 0.f) s += 0x1p-200 * low + 0x1p200 * high;
    return s;
  }
};

// Whether none of the squares in a plain sum has vanished or overflowed.  Inputs, whose first pass does little else,
// are summed plainly and, where this says no, read once more for Squares (1600 x 6400 in bf16 takes 16 us so, 19 with
// Squares alone, 14 without either).  For steps, which read much more, Squares cost 4 of 126 us, and a second reading
// beside them registers and 40 us.  fp16 inputs always fit.
__device__ __forceinline__ bool squares_held(float sum) { return sum >= 0x1p-80f && sum <= 0x1p120f; }

// How the first X is had from an input of the norm that a sum of squares gives: times a power of two, in two factors
// since fp32 may not hold it, that brings its norm to [2^12, 2^13).
struct First {
  float half, rest;            // the factors; 0 where the norm is not finite
  float unit;                  // 2^12 over the stored X's norm, 0 for a norm of 0
  bool finite;

  __device__ __forceinline__ explicit First(double squares) {
    const double norm64 = sqrt(squares);
    finite = isfinite(norm64);
    const bool some = finite && norm64 > 0.0;
    float norm = static_cast<float>(norm64);
    int apart = 0;             // the norm is 2^apart times this one, which fp32 holds with all its bits
    if (some && !(norm >= 0x1p-100f && norm <= 0x1p100f)) {
      apart = norm64 < 1.0 ? -100 : 100;
      norm = static_cast<float>(norm64 * (norm64 < 1.0 ? 0x1p100 : 0x1p-100));
    }
    const int up = some ? 12 - ilogbf(norm) : 0;
    unit = some ? kScaleX / (norm * exp2f(static_cast<float>(up))) : 0.f;
    half = finite ? exp2f(static_cast<float>((up - apart) / 2)) : 0.f;
    rest = exp2f(static_cast<float>(up - apart - (up - apart) / 2));
  }
  __device__ __forceinline__ float operator()(float u) const { return finite ? u * half * rest : 0.f; }
};

template <int THREADS = kPassThreads>
__device__ __forceinline__ double block_sum(double s) {
  __shared__ double of_warp[THREADS / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) of_warp[threadIdx.x >> 5] = s;
  __syncthreads();
  double all = 0.0;
  for (int k = 0; k < THREADS / 32; ++k) all += of_warp[k];
  return all;
}

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&f)[8]) {
  if constexpr (std::is_same<T, float>::value) dev::ld_32B(p, f);
  else Fmt<T>::unpack8(dev::ld_16B(p), f);
}
template <typename T>
__device__ __forceinline__ float load1(const T* p) {
  if constexpr (std::is_same<T, float>::value) return *p;
  else return Fmt<T>::load1(p, 0);
}

// 8 neighbours' (or, without `wide`, up to 8 neighbours' of which `n` exist)
// mean over the ranks, in rank order.
template <typename T>
__device__ __forceinline__ void rank_mean8(const uint64_t* grads, int W, int64_t at, bool wide, int n, float (&g)[8]) {
  const bool pow2 = (W & (W - 1)) == 0;
  const float inv_w = 1.f / W;
  if (wide) {
    for (int w0 = 0; w0 < W; w0 += 8) {
      uint4 raw[8];
#pragma unroll
      for (int w = 0; w < 8; ++w)
        if (w0 + w < W) raw[w] = dev::ld_16B(reinterpret_cast<const T*>(grads[w0 + w]) + at);
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        if (w0 + w >= W) break;
        float f[8];
        Fmt<T>::unpack8(raw[w], f);
#pragma unroll
        for (int k = 0; k < 8; ++k) g[k] = w0 + w == 0 ? f[k] : __fadd_rn(g[k], f[k]);
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      g[k] = 0.f;
      for (int w = 0; w < W && k < n; ++w) {
        const float f = Fmt<T>::load1(reinterpret_cast<const T*>(grads[w]), at + k);
        g[k] = w == 0 ? f : __fadd_rn(g[k], f);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) g[k] = dev::rank_mean(g[k], W, inv_w, pow2);
}

// The same of values that have been loaded.
template <typename T, int WC>
__device__ __forceinline__ void mean_of(const uint4 (&raw)[WC], float (&g)[8]) {
#pragma unroll
  for (int w = 0; w < WC; ++w) {
    float f[8];
    Fmt<T>::unpack8(raw[w], f);
#pragma unroll
    for (int k = 0; k < 8; ++k) g[k] = w == 0 ? f[k] : __fadd_rn(g[k], f[k]);
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) g[k] = dev::rank_mean(g[k], WC, 1.f / WC, (WC & (WC - 1)) == 0);
}

// 8 values of an fp32 vector; those that do not exist read as 0.
__device__ __forceinline__ void load_some(const float* p, bool wide, int n, float (&f)[8]) {
  if (wide) {
    dev::ld_32B(p, f);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = k < n ? p[k] : 0.f;
  }
}
__device__ __forceinline__ void store_some(float* p, bool wide, int n, const float (&f)[8]) {
  if (wide) {
    dev::st_32B(p, f);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) p[k] = f[k];
  }
}

// The matrix's values from (row, col) on, 8 of which n exist: the input, or
// the step's direction U and the new momentum.
template <typename T, bool MUON>
__device__ __forceinline__ void direction8(const PassArgs& p, const Entry& e, int which, int row, int col, int n,
                                           bool first, float (&u)[8], float (&m)[8]) {
  const bool wide = e.wide;
  if constexpr (!MUON) {
    const T* in = static_cast<const T*>(e.in) + row * e.in_stride + col;
    if (wide) {
      load8(in, u);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) u[k] = k < n ? load1(in + k) : 0.f;
    }
  } else {
    const int64_t at = static_cast<int64_t>(row) * e.cols + col;
    float g[8];
    if (first || e.mean == nullptr) rank_mean8<T>(p.grads + static_cast<int64_t>(which) * p.W, p.W, at, wide, n, g);
    else load_some(e.mean + at, wide, n, g);
    if (first && e.mean != nullptr) store_some(e.mean + at, wide, n, g);
    load_some(e.momentum + at, wide, n, m);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      m[k] = __fmaf_rn(p.mu, m[k], g[k]);
      u[k] = p.nesterov ? __fmaf_rn(p.mu, m[k], g[k]) : m[k];
    }
  }
}

// The list of matrices as a kernel's parameter, of two sizes: a launch's parameters hold no more than 32,764 bytes.
template <int BYTES>
struct TablePart {
  alignas(8) unsigned char data[BYTES];
};
constexpr int kSmallTable = 4 * 1024, kLargeTable = 28 * 1024;

// ---- the small matrices (muon_small.cu) -----------------------------------------------------

// One call's small matrices, and how they are treated.
struct SmallCall {
  const Entry* entries;
  const uint64_t* grads;       // W addresses for each entry, in the entries' order
  int count;
  bool muon;
  int in_dtype, out_dtype;
  int W;
  float mu;
  int nesterov;
  int steps, fine, first_parts;
  const double* coefficients;
  unsigned int* failures;
  cudaStream_t stream;
};

// Whether one cluster of CTAs can keep a matrix in its shared memory.
bool small_fits(int64_t rows, int64_t cols);
// All of them; `stall` as for the other launches.
int run_small(const SmallCall& c, bool& stall);
cudaError_t small_timeouts(unsigned int* out);

}  // namespace ns
}  // namespace zero
