// Embedding lookup with scaling, and the table's gradient by sorted tokens.
//
//   y_i = round(c T[x_i])                       (0 for an id outside [0, V))
//   dT_v = round(c sum_{i: x_i = v} dy_i (+ what was there))
//
// Both move bytes and do next to no arithmetic.  The lookup reads and writes
// one row per token.  The gradient sorts the (token, position) pairs, stably,
// so that the rows of one token stand together in the order of their
// positions; it then sums each run in fp32 in that order, which makes the
// result the same every time, and writes each table row once.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "step_math.cuh"
#include "zero_context.h"
#include "zero_internal.h"
#include "zero_step.h"

namespace zero {
namespace {

using dev::Fmt;
using host::ceil_div;
using host::fail;
using host::round_up;

// The id of token i, or V (one past the table) where it is outside [0, V).
__device__ __forceinline__ int load_id(const void* ids, int id_bytes, int64_t i, int vocab) {
  const int64_t t = id_bytes == 8 ? static_cast<const int64_t*>(ids)[i] : static_cast<const int32_t*>(ids)[i];
  return t >= 0 && t < vocab ? static_cast<int>(t) : vocab;
}

// ---- the lookup -----------------------------------------------------------------

constexpr int kLookupThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kLookupThreads) embed_lookup(const void* ids, int id_bytes, int tokens, int vocab,
                                                               int width8, const T* table, int64_t table_stride,
                                                               float scale, T* out, int64_t out_stride) {
  const int64_t total = static_cast<int64_t>(tokens) * width8;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * kLookupThreads + threadIdx.x; e < total;
       e += static_cast<int64_t>(gridDim.x) * kLookupThreads) {
    const int64_t row = e / width8, c = (e - row * width8) * 8;
    const int id = load_id(ids, id_bytes, row, vocab);
    uint4 x = make_uint4(0, 0, 0, 0);
    if (id < vocab) {
      float f[8];
      Fmt<T>::unpack8(dev::ld_16B(table + id * table_stride + c), f);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] *= scale;
      x = Fmt<T>::pack8(f);
    }
    dev::st_16B(out + row * out_stride + c, x);
  }
}

// ---- sorting the tokens -----------------------------------------------------------
//
// A stable radix sort of (id, position) pairs by id, in one cluster of CTAs:
// their barrier is hardware, so nothing spins, and each pass exchanges its
// digit counts through the cluster's shared memory.  Token i belongs to a
// fixed warp, in order, and a pass places the pairs of (digit, warp, order in
// the warp) one after another.  The launch's other clusters meanwhile set the
// gradient's rows to 0: the sort waits on latencies, the fill on bandwidth.

constexpr int kSortCtas = 8;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kRadix = 256;

struct SortArgs {
  const void* ids;
  int id_bytes, tokens, vocab;
  int passes, bits;            // digits of `bits` bits (at most 8)
  int* keys[2];                // after the last pass the sorted pairs are in [passes & 1]
  int* vals[2];
  char* fill;                  // rows to set to 0 (NULL: none)
  int64_t fill_stride;         // bytes
  int64_t fill_rows, row16;    // rows, and 16-byte words of a row
};

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ int peer_load(const int* p, uint32_t rank) {
  uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), r;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(r) : "memory");
  return v;
}

__global__ void __cluster_dims__(kSortCtas, 1, 1) __launch_bounds__(kSortThreads, 1) embed_sort(const SortArgs a) {
  const int tid = threadIdx.x;
  if (blockIdx.x >= kSortCtas) {
    const int64_t total = a.fill_rows * a.row16;
    for (int64_t e = static_cast<int64_t>(blockIdx.x - kSortCtas) * kSortThreads + tid; e < total;
         e += static_cast<int64_t>(gridDim.x - kSortCtas) * kSortThreads) {
      const int64_t row = e / a.row16;
      dev::st_16B(a.fill + row * a.fill_stride + (e - row * a.row16) * 16, make_uint4(0, 0, 0, 0));
    }
    return;
  }
  __shared__ int count[kSortWarps][kRadix];   // of each warp: how many of each digit, then where its next one goes
  __shared__ int cta_count[kRadix];           // read by the cluster's other CTAs
  __shared__ int digit_base[kRadix];
  __shared__ int warp_total[kRadix / 32];
  const int warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = blockIdx.x;
  // this warp's tokens: an even share of the groups of 32
  const int groups = (a.tokens + 31) / 32, warps = kSortCtas * kSortWarps;
  const int w = static_cast<int>(rank) * kSortWarps + warp;
  const int g0 = static_cast<int>(static_cast<int64_t>(groups) * w / warps);
  const int g1 = static_cast<int>(static_cast<int64_t>(groups) * (w + 1) / warps);
  const int mask = (1 << a.bits) - 1;
  for (int p = 0; p < a.passes; ++p) {
    const int shift = p * a.bits;
    const int* keys = a.keys[p & 1];
    const int* vals = a.vals[p & 1];
    int* keys_out = a.keys[(p & 1) ^ 1];
    int* vals_out = a.vals[(p & 1) ^ 1];
    auto key_at = [&](int i) { return p == 0 ? load_id(a.ids, a.id_bytes, i, a.vocab) : __ldcg(keys + i); };
    for (int d = lane; d < kRadix; d += 32) count[warp][d] = 0;
    __syncwarp();
    for (int g = g0; g < g1; ++g) {
      const int i = g * 32 + lane;
      if (i < a.tokens) atomicAdd(&count[warp][(key_at(i) >> shift) & mask], 1);
    }
    __syncthreads();
    if (tid < kRadix) {
      int sum = 0;
      for (int k = 0; k < kSortWarps; ++k) {
        const int c = count[k][tid];
        count[k][tid] = sum;
        sum += c;
      }
      cta_count[tid] = sum;
    }
    cluster_barrier();
    int before = 0, all = 0, inc = 0;
    if (tid < kRadix) {
#pragma unroll
      for (uint32_t c = 0; c < kSortCtas; ++c) {
        const int x = peer_load(&cta_count[tid], c);
        if (c < rank) before += x;
        all += x;
      }
      // prefix sum over the digits: inside each of the 8 warps, then over the warps
      inc = all;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
      }
      if (lane == 31) warp_total[warp] = inc;
    }
    __syncthreads();
    if (tid < kRadix) {
      int lower = 0;
      for (int k = 0; k < warp; ++k) lower += warp_total[k];
      digit_base[tid] = lower + inc - all + before;
    }
    __syncthreads();
    for (int d = lane; d < kRadix; d += 32) count[warp][d] += digit_base[d];
    __syncwarp();
    for (int g = g0; g < g1; ++g) {
      const int i = g * 32 + lane;
      const bool in = i < a.tokens;
      const int key = in ? key_at(i) : 0;
      // the lanes past the end form a group of their own
      const int d = in ? (key >> shift) & mask : kRadix;
      const unsigned same = __match_any_sync(0xffffffffu, d);
      const int ahead = __popc(same & ((1u << lane) - 1));
      int at = 0;
      if (in) at = count[warp][d] + ahead;
      __syncwarp();
      if (in && ahead == 0) count[warp][d] += __popc(same);
      __syncwarp();
      if (in) {
        __stcg(keys_out + at, key);
        __stcg(vals_out + at, p == 0 ? i : __ldcg(vals + i));
      }
    }
    // the pairs of this pass, and everyone's reads of cta_count, before the next pass
    cluster_barrier();
  }
}

// ---- summing the runs ---------------------------------------------------------------
//
// One CTA per chunk of kChunk sorted pairs, a thread per 8 columns.  Runs that
// lie inside the chunk are written at once; the part of a run that goes on
// from the chunk before (head) or into the chunk after (tail) is left in
// workspace in fp32, and embed_join adds those parts in order.

constexpr int kMaxChunk = 64;

struct RunArgs {
  const int* keys;
  const int* vals;
  int tokens, vocab, width8, chunk, chunks;
  const void* dout;
  int64_t dout_stride;
  void* dtable;
  int64_t dtable_stride;
  float* parts;                // [chunk][head, tail][width]
  float scale;
  int add;
};

template <typename T>
__device__ __forceinline__ void write_row(const RunArgs& a, int id, int64_t c, float (&sum)[8]) {
  if (id >= a.vocab) return;   // pairs without a row of the table
  T* out = static_cast<T*>(a.dtable) + id * a.dtable_stride + c;
  float old[8];
  if (a.add) Fmt<T>::unpack8(dev::ld_16B(out), old);
#pragma unroll
  for (int k = 0; k < 8; ++k) sum[k] = a.add ? fmaf(sum[k], a.scale, old[k]) : sum[k] * a.scale;
  dev::st_16B(out, Fmt<T>::pack8(sum));
}

template <typename T>
__global__ void __launch_bounds__(256) embed_runs(const RunArgs a) {
  __shared__ int key[kMaxChunk + 2];   // the chunk's, with one before and one after (-1: none)
  __shared__ int val[kMaxChunk];
  const int first = blockIdx.x * a.chunk, count = min(a.chunk, a.tokens - first);
  for (int k = threadIdx.x; k < count + 2; k += blockDim.x) {
    const int i = first + k - 1;
    key[k] = i >= 0 && i < a.tokens ? a.keys[i] : -1;
    if (k >= 1 && k <= count) val[k - 1] = a.vals[i];
  }
  __syncthreads();
  const T* dout = static_cast<const T*>(a.dout);
  const int64_t width = static_cast<int64_t>(a.width8) * 8;
  float* head = a.parts + static_cast<int64_t>(blockIdx.x) * 2 * width;
  for (int c8 = threadIdx.x; c8 < a.width8; c8 += blockDim.x) {
    const int64_t c = static_cast<int64_t>(c8) * 8;
    float sum[8];
    bool from_before = key[1] == key[0];   // the run that is being summed began in an earlier chunk
#pragma unroll
    for (int q = 0; q < 8; ++q) sum[q] = 0.f;
    for (int k0 = 0; k0 < count; k0 += 8) {
      uint4 x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k0 + k < count && key[k0 + k + 1] < a.vocab) x[k] = dev::ld_16B(dout + val[k0 + k] * a.dout_stride + c);
        else x[k] = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (k0 + k >= count) break;
        float f[8];
        Fmt<T>::unpack8(x[k], f);
#pragma unroll
        for (int q = 0; q < 8; ++q) sum[q] += f[q];
        const int id = key[k0 + k + 1];
        const bool last = k0 + k == count - 1;
        if (last || key[k0 + k + 2] != id) {
          if (from_before) dev::st_32B(head + c, sum);
          else if (last && key[k0 + k + 2] == id) dev::st_32B(head + width + c, sum);
          else write_row<T>(a, id, c, sum);
          from_before = false;
#pragma unroll
          for (int q = 0; q < 8; ++q) sum[q] = 0.f;
        }
      }
    }
  }
}

// The runs that begin in chunk blockIdx.x and go on past its end.
template <typename T>
__global__ void __launch_bounds__(256) embed_join(const RunArgs a) {
  const int b = blockIdx.x, end = (b + 1) * a.chunk;
  if (end >= a.tokens) return;
  const int id = a.keys[end - 1];
  if (id >= a.vocab || a.keys[end] != id) return;
  if (b > 0 && a.keys[b * a.chunk - 1] == id) return;   // began earlier
  const int64_t width = static_cast<int64_t>(a.width8) * 8;
  for (int c8 = threadIdx.x; c8 < a.width8; c8 += blockDim.x) {
    const int64_t c = static_cast<int64_t>(c8) * 8;
    float sum[8];
    dev::ld_32B(a.parts + (2 * static_cast<int64_t>(b) + 1) * width + c, sum);
    for (int j = b + 1; j < a.chunks && a.keys[j * a.chunk] == id; ++j) {
      float x[8];
      dev::ld_32B(a.parts + 2 * static_cast<int64_t>(j) * width + c, x);
#pragma unroll
      for (int q = 0; q < 8; ++q) sum[q] += x[q];
    }
    write_row<T>(a, id, c, sum);
  }
}

// ---- host -----------------------------------------------------------------------------

constexpr int64_t kMaxTokens = int64_t(1) << 24, kMaxVocab = int64_t(1) << 24, kMaxWidth = int64_t(1) << 16;
constexpr int kChunk = 16;

int check_ids(int64_t tokens, int64_t vocab, int64_t width, int dtype, const void* ids, int id_bytes) {
  if (tokens < 0 || tokens > kMaxTokens) return fail(ZERO_E_ARG, "tokens=%lld outside [0, 2^24]", (long long)tokens);
  if (vocab < 1 || vocab > kMaxVocab) return fail(ZERO_E_ARG, "vocab=%lld outside [1, 2^24]", (long long)vocab);
  if (width < 8 || width > kMaxWidth || width % 8)
    return fail(ZERO_E_ARG, "width=%lld must be a multiple of 8 in [8, 65536]", (long long)width);
  if (!host::valid_dtype(dtype)) return fail(ZERO_E_ARG, "the 16-bit format must be ZERO_FP16 or ZERO_BF16");
  if (id_bytes != 4 && id_bytes != 8) return fail(ZERO_E_ARG, "ids of %d bytes: 4 or 8 are supported", id_bytes);
  if (tokens > 0 && ids == nullptr) return fail(ZERO_E_ARG, "ids is NULL");
  if (reinterpret_cast<uintptr_t>(ids) % id_bytes) return fail(ZERO_E_ALIGN, "ids is not aligned to its type");
  return ZERO_OK;
}

int check_rows(const char* what, const void* p, int64_t stride, int64_t rows, int64_t width) {
  if (rows > 0 && p == nullptr) return fail(ZERO_E_ARG, "%s is NULL", what);
  if (stride < width || stride > (int64_t(1) << 32))
    return fail(ZERO_E_ARG, "%s: row stride %lld is below the width or too large", what, (long long)stride);
  if (!host::aligned16(p) || stride % 8) return fail(ZERO_E_ALIGN, "%s: rows must start on 16-byte boundaries", what);
  return ZERO_OK;
}

int check_scale(double scale) {
  if (!std::isfinite(static_cast<float>(scale))) return fail(ZERO_E_ARG, "scale %g is not a finite fp32 value", scale);
  return ZERO_OK;
}

int64_t pairs_bytes(int64_t tokens) { return round_up(tokens * 4, 256); }

int64_t space(int64_t tokens, int64_t width) {
  return std::max<int64_t>(256, 4 * pairs_bytes(tokens) + round_up(ceil_div(tokens, kChunk) * 2 * width * 4, 256));
}

template <typename T>
int lookup(int64_t tokens, int64_t vocab, int64_t width, const void* ids, int id_bytes, const void* table,
           int64_t table_stride, float scale, void* out, int64_t out_stride, cudaStream_t s) {
  const int64_t items = tokens * (width / 8);
  const int64_t blocks = std::min<int64_t>(ceil_div(items, kLookupThreads), static_cast<int64_t>(sm_count()) * 8);
  embed_lookup<T><<<static_cast<unsigned>(blocks), kLookupThreads, 0, s>>>(
      ids, id_bytes, static_cast<int>(tokens), static_cast<int>(vocab), static_cast<int>(width / 8),
      static_cast<const T*>(table), table_stride, scale, static_cast<T*>(out), out_stride);
  ZERO_CUDA(cudaGetLastError());
  return ZERO_OK;
}

template <typename T>
int sum_runs(const RunArgs& a, cudaStream_t s) {
  const int threads = static_cast<int>(std::min<int64_t>(256, round_up(a.width8, 32)));
  embed_runs<T><<<a.chunks, threads, 0, s>>>(a);
  ZERO_CUDA(cudaGetLastError());
  if (a.chunks > 1) {
    embed_join<T><<<a.chunks - 1, threads, 0, s>>>(a);
    ZERO_CUDA(cudaGetLastError());
  }
  return ZERO_OK;
}

}  // namespace
}  // namespace zero

using namespace zero;

extern "C" int zero_embedding(int64_t tokens, int64_t vocab, int64_t width, int dtype, const void* ids, int id_bytes,
                              const void* table, int64_t table_stride, double scale, void* out, int64_t out_stride,
                              void* stream) {
  int rc = check_ids(tokens, vocab, width, dtype, ids, id_bytes);
  if (rc || (rc = check_rows("table", table, table_stride, vocab, width)) ||
      (rc = check_rows("out", out, out_stride, tokens, width)) || (rc = check_scale(scale)))
    return rc;
  if (tokens == 0) return ZERO_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const float c = static_cast<float>(scale);
  return dtype == ZERO_FP16
             ? lookup<__half>(tokens, vocab, width, ids, id_bytes, table, table_stride, c, out, out_stride, s)
             : lookup<__nv_bfloat16>(tokens, vocab, width, ids, id_bytes, table, table_stride, c, out, out_stride, s);
}

extern "C" int64_t zero_embedding_workspace_bytes(int64_t tokens, int64_t width) {
  if (tokens < 0 || tokens > kMaxTokens) return fail(ZERO_E_ARG, "tokens=%lld outside [0, 2^24]", (long long)tokens);
  if (width < 8 || width > kMaxWidth || width % 8)
    return fail(ZERO_E_ARG, "width=%lld must be a multiple of 8 in [8, 65536]", (long long)width);
  return space(tokens, width);
}

extern "C" int zero_embedding_grad(int64_t tokens, int64_t vocab, int64_t width, int dtype, const void* ids,
                                   int id_bytes, const void* dout, int64_t dout_stride, double scale, void* dtable,
                                   int64_t dtable_stride, int accumulate, void* workspace, int64_t workspace_bytes,
                                   void* stream) {
  int rc = check_ids(tokens, vocab, width, dtype, ids, id_bytes);
  if (rc || (rc = check_rows("dout", dout, dout_stride, tokens, width)) ||
      (rc = check_rows("dtable", dtable, dtable_stride, vocab, width)) || (rc = check_scale(scale)))
    return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (tokens == 0) {
    if (!accumulate) ZERO_CUDA(cudaMemset2DAsync(dtable, dtable_stride * 2, 0, width * 2, vocab, s));
    return ZERO_OK;
  }
  if (workspace == nullptr) return fail(ZERO_E_ARG, "workspace is NULL");
  if (reinterpret_cast<uintptr_t>(workspace) % 256) return fail(ZERO_E_ALIGN, "workspace must be 256-byte aligned");
  if (workspace_bytes < space(tokens, width))
    return fail(ZERO_E_ARG, "workspace of %lld bytes: %lld are needed", (long long)workspace_bytes,
                (long long)space(tokens, width));
  char* ws = static_cast<char*>(workspace);
  const int64_t pb = pairs_bytes(tokens);
  SortArgs sa{};
  sa.ids = ids;
  sa.id_bytes = id_bytes;
  sa.tokens = static_cast<int>(tokens);
  sa.vocab = static_cast<int>(vocab);
  int key_bits = 1;   // of the ids 0..vocab (vocab: no row)
  while ((int64_t(1) << key_bits) <= vocab) ++key_bits;
  sa.passes = (key_bits + 7) / 8;
  sa.bits = (key_bits + sa.passes - 1) / sa.passes;
  for (int k = 0; k < 2; ++k) {
    sa.keys[k] = reinterpret_cast<int*>(ws + k * pb);
    sa.vals[k] = reinterpret_cast<int*>(ws + (2 + k) * pb);
  }
  unsigned grid = kSortCtas;
  if (!accumulate) {
    sa.fill = static_cast<char*>(dtable);
    sa.fill_stride = dtable_stride * 2;
    sa.fill_rows = vocab;
    sa.row16 = width / 8;
    const int64_t want = ceil_div(ceil_div(vocab * sa.row16, kSortThreads), kSortCtas);
    grid += kSortCtas * static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(sm_count() / kSortCtas - 1, want)));
  }
  embed_sort<<<grid, kSortThreads, 0, s>>>(sa);
  ZERO_CUDA(cudaGetLastError());
  RunArgs ra{};
  ra.keys = sa.keys[sa.passes & 1];
  ra.vals = sa.vals[sa.passes & 1];
  ra.tokens = sa.tokens;
  ra.vocab = sa.vocab;
  ra.width8 = static_cast<int>(width / 8);
  ra.chunk = kChunk;
  ra.chunks = static_cast<int>(ceil_div(tokens, kChunk));
  ra.dout = dout;
  ra.dout_stride = dout_stride;
  ra.dtable = dtable;
  ra.dtable_stride = dtable_stride;
  ra.parts = reinterpret_cast<float*>(ws + 4 * pb);
  ra.scale = static_cast<float>(scale);
  ra.add = accumulate != 0;
  return dtype == ZERO_FP16 ? sum_runs<__half>(ra, s) : sum_runs<__nv_bfloat16>(ra, s);
}
