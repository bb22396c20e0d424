// Embedding lookup with scaling, and the table's gradient by sorted tokens.
//
//   y_i = round(c T[x_i])                       (0 for an id outside [0, V))
//   dT_v = round(c sum_{i: x_i = v} dy_i (+ what was there))
//
// Both move bytes and do next to no arithmetic.  The lookup reads and writes
// one row per token.  The gradient sorts the (token, position) pairs, stably,
// so that the rows of one token stand together in the order of their
// positions; it then sums each run in fp32, in an order fixed by the ids (long
// runs in stretches), which makes the result the same every time, and writes
// each table row once.
//
// What bounds them.  This device writes at most about 4 TB/s, half of what it
// copies: the lookup of 32768 rows of 1600 writes 105 MB in 25.3 us (4.1
// TB/s), and a 50257 x 768 gradient alone takes 22.6 us to fill with zeros, by
// a memset too, of 28.6 us for 8192 tokens.  65535 tokens
// onto a 50257 x 1600 gradient take 94 us: 27 for the sort (latencies, 8 SMs),
// 58 for the runs (283 MB from and to DRAM, 4.7 TB/s) and 10 for the long ones.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "launch.cuh"
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
//
// A CTA takes some consecutive tokens whose ids it reads first, and then the
// 16-byte words of their rows: each thread issues kLookupBatch loads before
// the first store, so that the rows' latencies overlap.

constexpr int kLookupThreads = 256;
constexpr int kLookupBatch = 8;
constexpr int kLookupRows = 256;      // most tokens of a CTA

template <typename T>
__global__ void __launch_bounds__(kLookupThreads) embed_lookup(const void* ids, int id_bytes, int tokens, int vocab,
                                                               int width8, unsigned int inv_width8, int rows,
                                                               const T* table, int64_t table_stride, float scale, T* out,
                                                               int64_t out_stride) {
  __shared__ int id[kLookupRows];
  const int first = blockIdx.x * rows, count = min(rows, tokens - first);
  for (int r = threadIdx.x; r < count; r += kLookupThreads) id[r] = load_id(ids, id_bytes, first + r, vocab);
  __syncthreads();
  const int words = count * width8;
  for (int j0 = threadIdx.x; j0 < words; j0 += kLookupThreads * kLookupBatch) {
    uint4 x[kLookupBatch];
#pragma unroll
    for (int u = 0; u < kLookupBatch; ++u) {
      const int j = j0 + u * kLookupThreads;
      x[u] = make_uint4(0, 0, 0, 0);
      if (j < words) {
        // j / width8: exact, as j and width8 stay below 2^14 (see the host side)
        const int r = width8 == 1 ? j : static_cast<int>(__umulhi(j, inv_width8));
        if (id[r] < vocab) x[u] = dev::ld_16B(table + id[r] * table_stride + (j - r * width8) * 8);
      }
    }
#pragma unroll
    for (int u = 0; u < kLookupBatch; ++u) {
      const int j = j0 + u * kLookupThreads;
      if (j < words) {
        const int r = width8 == 1 ? j : static_cast<int>(__umulhi(j, inv_width8));
        float f[8];
        Fmt<T>::unpack8(x[u], f);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] *= scale;
        dev::st_16B(out + (first + r) * out_stride + (j - r * width8) * 8, Fmt<T>::pack8(f));
      }
    }
  }
}

// ---- sorting the tokens -----------------------------------------------------------
//
// A stable radix sort of (id, position) pairs by id, in one cluster of CTAs:
// their barrier is hardware, so nothing spins, and each pass exchanges its
// digit counts through the cluster's shared memory.  Token i belongs to a
// fixed warp, in order, and a pass places the pairs of (digit, warp, order in
// the warp) one after another.  The launch's other clusters meanwhile set
// rows of the gradient to 0: the sort waits on latencies, the fill on
// bandwidth.  Rows beyond what the sort's time covers are left to the next
// launch, which knows the ids and fills only those without any.

constexpr int kSortCtas = 8;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kRadix = 256;
constexpr int kSortBatch = 8;      // groups of 32 pairs whose loads a warp has in flight

struct SortArgs {
  const void* ids;
  int id_bytes, tokens, vocab;
  int passes, bits;            // digits of `bits` bits (at most 8)
  int2* pairs[2];              // (id, position); sorted in pairs[passes & 1] after the last pass
  int* runs;                   // a counter to set to 0 (RunArgs)
  char* fill;                  // rows to set to 0 (NULL: none)
  int64_t fill_stride;         // bytes
  int64_t fill_rows, row16;    // rows, and 16-byte words of a row
  int64_t fill_words;          // of all the rows (the last one may be short)
};

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The lanes whose 8-bit digit equals this lane's, by one vote for each bit
// (the match instruction takes time with every different value: a pass over
// 32 unequal digits took 2,500 cycles).  Lanes without a pair match nobody's.
__device__ __forceinline__ unsigned same_digit(int digit, bool real) {
  unsigned same = __ballot_sync(0xffffffffu, real);
#pragma unroll
  for (int b = 0; b < 8; ++b) {
    const unsigned one = __ballot_sync(0xffffffffu, (digit >> b) & 1);
    same &= (digit >> b) & 1 ? one : ~one;
  }
  return real ? same : 0u;
}

__device__ __forceinline__ int peer_load(const int* p, uint32_t rank) {
  uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), r;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(r) : "memory");
  return v;
}

__global__ void __cluster_dims__(kSortCtas, 1, 1) __launch_bounds__(kSortThreads, 1) embed_sort(const SortArgs a) {
  allow_next();
  await_previous();
  const int tid = threadIdx.x;
  if (blockIdx.x >= kSortCtas) {
    for (int64_t row = blockIdx.x - kSortCtas; row < a.fill_rows; row += gridDim.x - kSortCtas) {
      char* p = a.fill + row * a.fill_stride;
      const int64_t words = min(a.row16, a.fill_words - row * a.row16);
      for (int64_t c = tid; c < words; c += kSortThreads) dev::st_16B(p + c * 16, make_uint4(0, 0, 0, 0));
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
  if (blockIdx.x == 0 && tid == 0) *a.runs = 0;
  for (int p = 0; p < a.passes; ++p) {
    const int shift = p * a.bits;
    const int2* in = a.pairs[p & 1];
    int2* out = a.pairs[(p & 1) ^ 1];
    // the pair at i; (-1, i) past the end
    auto pair_at = [&](int i) {
      if (i >= a.tokens) return make_int2(-1, i);
      return p == 0 ? make_int2(load_id(a.ids, a.id_bytes, i, a.vocab), i) : __ldcg(in + i);
    };
    for (int d = lane; d < kRadix; d += 32) count[warp][d] = 0;
    __syncwarp();
    // a batch of groups: their pairs, and which lanes share each one's digit
    int2 x[kSortBatch];
    unsigned same[kSortBatch];
    auto load = [&](int g) {
#pragma unroll
      for (int u = 0; u < kSortBatch; ++u) x[u] = g + u < g1 ? pair_at((g + u) * 32 + lane) : make_int2(-1, 0);
#pragma unroll
      for (int u = 0; u < kSortBatch; ++u)
        same[u] = g + u < g1 ? same_digit((x[u].x >> shift) & mask, x[u].x >= 0) : 0u;
    };
    for (int g = g0; g < g1; g += kSortBatch) {
      load(g);
#pragma unroll
      for (int u = 0; u < kSortBatch; ++u) {
        if (same[u] && (same[u] & ((1u << lane) - 1)) == 0) count[warp][(x[u].x >> shift) & mask] += __popc(same[u]);
        __syncwarp();
      }
    }
    __syncthreads();
    if (tid < kRadix) {
      int sum = 0;
#pragma unroll
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
    for (int g = g0; g < g1; g += kSortBatch) {
      if (g1 - g0 > kSortBatch) load(g);   // else the one batch is still there
#pragma unroll
      for (int u = 0; u < kSortBatch; ++u) {
        const int d = (x[u].x >> shift) & mask;
        const int ahead = __popc(same[u] & ((1u << lane) - 1));
        int at = 0;
        if (same[u]) at = count[warp][d] + ahead;
        __syncwarp();
        if (same[u] && ahead == 0) count[warp][d] = at + __popc(same[u]);
        __syncwarp();
        if (same[u]) __stcg(out + at, x[u]);
      }
    }
    // the pairs of this pass, and everyone's reads of cta_count, before the next pass
    cluster_barrier();
  }
}

// ---- summing the runs ---------------------------------------------------------------
//
// One CTA per chunk of sorted pairs, a thread per 8 columns.  A run of at most
// a chunk's length belongs to the chunk it begins in, whole, even where it
// ends in the next one, and is written at once.  A longer run is cut at the
// chunks: its part of each is left in workspace in fp32 (head: it goes on from
// the chunk before; tail: it begins here and goes on), the run is noted, and
// embed_join adds its parts in order.

constexpr int kMinChunk = 8, kMaxChunk = 64;
constexpr int kAddBatch = 4;          // (with 8, two CTAs fewer fit an SM)

struct RunArgs {
  const int2* pairs;
  int tokens, vocab, width8, chunk, chunks;
  const void* dout;
  int64_t dout_stride;
  void* dtable;
  int64_t dtable_stride;
  float* parts;                // [chunk][head, tail][width]
  int* runs;                   // how many runs go past their chunk, and after it the chunks where they begin
  float scale;
  int fill_first, fills;       // rows from here on are still to be set to 0 where no id names them, by so many blocks
};

constexpr int kFillRows = 64;        // rows of a filling block
constexpr int kFillSteps = 8;        // block-wide looks at the pairs of those rows

// Set to 0 the rows [r0, r0 + kFillRows) that no sorted pair names.  Which ones
// are named the pairs themselves say, where they are few; where they are many
// (an id as frequent as padding is), each row looks for its id among them, so
// that the time does not grow with how often an id comes: 47,000 times the last
// of 50257 ids at width 768 took 222 us by the pairs alone.
template <typename T>
__device__ void fill_unnamed(const RunArgs& a, int r0) {
  __shared__ int named[kFillRows];
  __shared__ int start;
  const int r1 = min(r0 + kFillRows, a.vocab), lane = threadIdx.x & 31;
  for (int k = threadIdx.x; k < kFillRows; k += blockDim.x) named[k] = 0;
  if (threadIdx.x < 32) {
    // the first pair with an id of r0 or more: 32 probes at a time
    int lo = 0, hi = a.tokens;
    while (lo < hi) {
      const int step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step - 1;
      const int below = __popc(__ballot_sync(0xffffffffu, at < hi && a.pairs[at].x < r0));
      hi = min(hi, lo + (below + 1) * step - 1);
      lo = min(hi, lo + below * step);
    }
    if (lane == 0) start = lo;
  }
  __syncthreads();
  int base = start;      // at most 2^24 and some blocks' threads
  bool more = true;      // the pairs from base on may still be of these rows
  for (int step = 0; more && step < kFillSteps; ++step, base += blockDim.x) {
    const int i = base + static_cast<int>(threadIdx.x);
    const int id = i < a.tokens ? a.pairs[i].x : a.vocab;
    if (id < r1) named[id - r0] = 1;
    more = __syncthreads_or(threadIdx.x == blockDim.x - 1 && id < r1) != 0;
  }
  if (more) {
    for (int r = r0 + static_cast<int>(threadIdx.x); r < r1; r += blockDim.x) {
      int lo = base, hi = a.tokens;   // the first pair from base on with an id of r or more
      while (lo < hi) {
        const int mid = lo + (hi - lo) / 2;
        if (a.pairs[mid].x < r) lo = mid + 1;
        else hi = mid;
      }
      if (lo < a.tokens && a.pairs[lo].x == r) named[r - r0] = 1;
    }
    __syncthreads();
  }
  for (int r = r0; r < r1; ++r) {
    if (named[r - r0]) continue;
    T* out = static_cast<T*>(a.dtable) + r * a.dtable_stride;
    for (int c8 = threadIdx.x; c8 < a.width8; c8 += blockDim.x) dev::st_16B(out + c8 * 8, make_uint4(0, 0, 0, 0));
  }
}

// scale * sum (+ the old row) to a row of the table's gradient.
template <typename T, bool ADD>
__device__ __forceinline__ void write_row(const RunArgs& a, int id, int64_t c, float (&sum)[8], const uint4& old) {
  float f[8];
  if (ADD) Fmt<T>::unpack8(old, f);
#pragma unroll
  for (int k = 0; k < 8; ++k) sum[k] = ADD ? fmaf(sum[k], a.scale, f[k]) : sum[k] * a.scale;
  dev::st_16B(static_cast<T*>(a.dtable) + id * a.dtable_stride + c, Fmt<T>::pack8(sum));
}

template <typename T, bool ADD>
__global__ void __launch_bounds__(256) embed_runs(const RunArgs a) {
  allow_next();
  await_previous();
  const int block = static_cast<int>(blockIdx.x) - a.fills;
  if (!ADD && block < 0) {
    fill_unnamed<T>(a, a.fill_first + static_cast<int>(blockIdx.x) * kFillRows);
    return;
  }
  // pairs first - chunk - 1 .. first + 2 chunk (ids -1 and -2 outside the list)
  __shared__ int key[3 * kMaxChunk + 2];
  __shared__ int val[3 * kMaxChunk + 2];
  __shared__ int edge[4];
  const int c = a.chunk, first = block * c, last = min(first + c, a.tokens) - 1, low = first - c - 1;
  for (int k = threadIdx.x; k < 3 * c + 2; k += blockDim.x) {
    const int i = low + k;
    const int2 x = i < 0 ? make_int2(-1, 0) : i < a.tokens ? a.pairs[i] : make_int2(-2, 0);
    key[k] = x.x;
    val[k] = x.y;
  }
  // where the first pair's run begins and ends, and the last pair's; far
  // enough away where the window does not show it
  if (threadIdx.x < 4) edge[threadIdx.x] = threadIdx.x % 2 == 0 ? low : first + 2 * c + 1;
  __syncthreads();
  for (int k = threadIdx.x + 1; k < 3 * c + 2; k += blockDim.x) {
    if (key[k] == key[k - 1]) continue;
    const int i = low + k;   // a run begins at i, and one ends
    if (i <= first) atomicMax(&edge[0], i);
    else atomicMin(&edge[1], i);
    if (i <= last) atomicMax(&edge[2], i);
    else atomicMin(&edge[3], i);
  }
  __syncthreads();
  const bool long0 = edge[1] - edge[0] > c, long1 = edge[3] - edge[2] > c;
  const bool began_before = edge[0] < first, begins_here = edge[2] >= first;
  const int begin = began_before && !long0 ? min(edge[1], last + 1) : first;
  const int end = begins_here && !long1 ? edge[3] : last + 1;
  const bool continues = long1 && edge[3] > last + 1;     // the last pair's run, into the next chunk
  const bool head_first = began_before && long0;
  if (threadIdx.x == 0 && begins_here && continues && key[last - low] < a.vocab) a.runs[1 + atomicAdd(a.runs, 1)] = block;
  const T* dout = static_cast<const T*>(a.dout);
  const int64_t width = static_cast<int64_t>(a.width8) * 8;
  float* head = a.parts + static_cast<int64_t>(block) * 2 * width;
  constexpr int kRunBatch = ADD ? kAddBatch : 8;   // rows whose loads a thread has in flight
  for (int c8 = threadIdx.x; c8 < a.width8; c8 += blockDim.x) {
    const int64_t col = static_cast<int64_t>(c8) * 8;
    float sum[8];
    bool from_before = head_first;
#pragma unroll
    for (int q = 0; q < 8; ++q) sum[q] = 0.f;
    for (int k0 = begin - low; k0 < end - low; k0 += kRunBatch) {
      uint4 x[kRunBatch], old[ADD ? kRunBatch : 1];
#pragma unroll
      for (int k = 0; k < kRunBatch; ++k) {
        x[k] = make_uint4(0, 0, 0, 0);
        if (ADD) old[k] = x[k];
        if (k0 + k < end - low && key[k0 + k] < a.vocab) {
          x[k] = dev::ld_16B(dout + val[k0 + k] * a.dout_stride + col);
          if (ADD && key[k0 + k + 1] != key[k0 + k])
            old[k] = dev::ld_16B(static_cast<const T*>(a.dtable) + key[k0 + k] * a.dtable_stride + col);
        }
      }
#pragma unroll
      for (int k = 0; k < kRunBatch; ++k) {
        if (k0 + k >= end - low) break;
        float f[8];
        Fmt<T>::unpack8(x[k], f);
#pragma unroll
        for (int q = 0; q < 8; ++q) sum[q] += f[q];
        const int id = key[k0 + k];
        const bool at_end = k0 + k == end - low - 1;
        if (at_end || key[k0 + k + 1] != id) {
          if (from_before) dev::st_32B(head + col, sum);
          else if (at_end && continues) dev::st_32B(head + width + col, sum);
          else if (id < a.vocab) write_row<T, ADD>(a, id, col, sum, old[ADD ? k : 0]);
          from_before = false;
#pragma unroll
          for (int q = 0; q < 8; ++q) sum[q] = 0.f;
        }
      }
    }
  }
}

// The long runs.  An item is one run and 256 columns; kJoinSlices groups of 32
// threads each add a stretch of the run's parts, and the first adds the
// stretches, in order.
constexpr int kJoinSlices = 8;
constexpr int kJoinThreads = 32 * kJoinSlices;

template <typename T, bool ADD>
__global__ void __launch_bounds__(kJoinThreads) embed_join(const RunArgs a) {
  allow_next();
  await_previous();
  __shared__ float stretch[kJoinSlices][32][9];
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int blocks = (a.width8 + 31) / 32, items = a.runs[0] * blocks;
  const int64_t width = static_cast<int64_t>(a.width8) * 8;
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int b = a.runs[1 + item / blocks], c8 = item % blocks * 32 + lane;
    const int64_t c = static_cast<int64_t>(c8) * 8;
    const int id = a.pairs[(b + 1) * a.chunk - 1].x;
    // how many chunks after b the run reaches into: those that begin with its id
    int more = 0;
    for (;;) {
      const int64_t at = (static_cast<int64_t>(b) + 1 + more + threadIdx.x) * a.chunk;
      const int n = __syncthreads_count(at < a.tokens && a.pairs[at].x == id);
      more += n;
      if (n < kJoinThreads) break;
    }
    // parts 0..more: the tail of b, then the heads of the chunks after it
    const int p0 = (more + 1) * slice / kJoinSlices, p1 = (more + 1) * (slice + 1) / kJoinSlices;
    float sum[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) sum[q] = 0.f;
    if (c8 < a.width8) {
#pragma unroll 8
      for (int p = p0; p < p1; ++p) {
        float x[8];
        dev::ld_32B(a.parts + (2 * (static_cast<int64_t>(b) + p) + (p == 0 ? 1 : 0)) * width + c, x);
#pragma unroll
        for (int q = 0; q < 8; ++q) sum[q] += x[q];
      }
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) stretch[slice][lane][q] = sum[q];
    __syncthreads();
    if (slice == 0 && c8 < a.width8) {
      uint4 old = make_uint4(0, 0, 0, 0);
      if (ADD) old = dev::ld_16B(static_cast<const T*>(a.dtable) + id * a.dtable_stride + c);
      for (int k = 1; k < kJoinSlices; ++k)
#pragma unroll
        for (int q = 0; q < 8; ++q) sum[q] += stretch[k][lane][q];
      write_row<T, ADD>(a, id, c, sum, old);
    }
    __syncthreads();
  }
}

// ---- host -----------------------------------------------------------------------------

constexpr int64_t kMaxTokens = int64_t(1) << 24, kMaxVocab = int64_t(1) << 24, kMaxWidth = int64_t(1) << 16;

// Sorted pairs per chunk, a power of two: 608 to 1215 chunks where the tokens
// allow it (4 to 8 for each SM).  65535 tokens onto 50257 x 1600 took 94 us so
// and with 304, 100 with 1216 and 112 with 2432; 8192 tokens x 768 took 35 us
// with 304 and 33 with the others.
constexpr int kChunks = 608;
int chunk_of(int64_t tokens) {
  int c = kMinChunk;
  while (c < kMaxChunk && tokens / (2 * c) >= kChunks) c *= 2;
  return c;
}

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

int64_t pairs_bytes(int64_t tokens) { return round_up(tokens * 8, 256); }

// Most chunks that any count up to `tokens` is cut into.
int64_t most_chunks(int64_t tokens) {
  return std::min(ceil_div(tokens, kMinChunk), std::max<int64_t>(2 * kChunks + 1, ceil_div(tokens, kMaxChunk)));
}

int64_t runs_bytes(int64_t tokens) { return round_up((most_chunks(tokens) + 1) * 4, 256); }

int64_t space(int64_t tokens, int64_t width) {
  return std::max<int64_t>(256, 2 * pairs_bytes(tokens) + runs_bytes(tokens) + round_up(most_chunks(tokens) * 2 * width * 4, 256));
}

template <typename T>
int lookup(int64_t tokens, int64_t vocab, int64_t width, const void* ids, int id_bytes, const void* table,
           int64_t table_stride, float scale, void* out, int64_t out_stride, cudaStream_t s) {
  const int64_t width8 = width / 8;
  // one batch of every thread per CTA, and fewer rows while there are SMs without work
  const int64_t full = std::max<int64_t>(1, kLookupThreads * kLookupBatch / width8);
  const int64_t rows = std::max<int64_t>(1, std::min<int64_t>({full, kLookupRows, ceil_div(tokens, 2 * sm_count())}));
  const unsigned inv = width8 == 1 ? 0 : static_cast<unsigned>((uint64_t(1) << 32) / width8 + 1);
  embed_lookup<T><<<static_cast<unsigned>(ceil_div(tokens, rows)), kLookupThreads, 0, s>>>(
      ids, id_bytes, static_cast<int>(tokens), static_cast<int>(vocab), static_cast<int>(width8), inv,
      static_cast<int>(rows), static_cast<const T*>(table), table_stride, scale, static_cast<T*>(out), out_stride);
  ZERO_CUDA(cudaGetLastError());
  return ZERO_OK;
}

template <typename T, bool ADD>
int sum_runs(const RunArgs& a, cudaStream_t s) {
  const int threads = static_cast<int>(std::min<int64_t>(256, round_up(a.width8, 32)));
  ZERO_CUDA(launch_chained(embed_runs<T, ADD>, dim3(static_cast<unsigned>(a.chunks + a.fills)), threads, 0, s, a));
  if (a.chunks > 1) {
    const int64_t most = static_cast<int64_t>(a.chunks - 1) * ceil_div(a.width8, 32);
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(8 * sm_count(), most)));
    ZERO_CUDA(launch_chained(embed_join<T, ADD>, grid, kJoinThreads, 0, s, a));
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
  for (int k = 0; k < 2; ++k) sa.pairs[k] = reinterpret_cast<int2*>(ws + k * pb);
  sa.runs = reinterpret_cast<int*>(ws + 2 * pb);
  unsigned grid = kSortCtas;
  int64_t fill_now = 0;
  if (!accumulate) {
    // What is written while the ids are sorted: 30 MB and 1 KB for each id.  8192 tokens x 768 onto 50257 rows (77
    // MB) take 32.9 us with all rows filled there, 28.6 so, 29.4 with 20 MB, 29.6 with 40 and 31.0 with 50.
    fill_now = std::min(vocab, ceil_div(30'000'000 + tokens * 1000, width * 2));
    if (dtable_stride == width) {   // one stretch, in rows of 64 KB
      sa.fill_words = fill_now * (width / 8);
      sa.row16 = 4096;
      sa.fill_rows = ceil_div(sa.fill_words, sa.row16);
      sa.fill_stride = sa.row16 * 16;
    } else {
      sa.row16 = width / 8;
      sa.fill_rows = fill_now;
      sa.fill_words = fill_now * sa.row16;
      sa.fill_stride = dtable_stride * 2;
    }
    sa.fill = static_cast<char*>(dtable);
    const int64_t clusters = std::min<int64_t>(sm_count() / kSortCtas - 1, ceil_div(sa.fill_rows, kSortCtas));
    grid += kSortCtas * static_cast<unsigned>(std::max<int64_t>(1, clusters));
  }
  ZERO_CUDA(launch_chained(embed_sort, dim3(grid), kSortThreads, 0, s, sa));
  RunArgs ra{};
  ra.pairs = sa.pairs[sa.passes & 1];
  ra.tokens = sa.tokens;
  ra.vocab = sa.vocab;
  ra.width8 = static_cast<int>(width / 8);
  ra.chunk = chunk_of(tokens);
  ra.chunks = static_cast<int>(ceil_div(tokens, ra.chunk));
  ra.dout = dout;
  ra.dout_stride = dout_stride;
  ra.dtable = dtable;
  ra.dtable_stride = dtable_stride;
  ra.runs = sa.runs;
  ra.parts = reinterpret_cast<float*>(ws + 2 * pb + runs_bytes(tokens));
  ra.scale = static_cast<float>(scale);
  ra.fill_first = static_cast<int>(fill_now);
  ra.fills = accumulate ? 0 : static_cast<int>(ceil_div(vocab - fill_now, kFillRows));
  if (accumulate) return dtype == ZERO_FP16 ? sum_runs<__half, true>(ra, s) : sum_runs<__nv_bfloat16, true>(ra, s);
  return dtype == ZERO_FP16 ? sum_runs<__half, false>(ra, s) : sum_runs<__nv_bfloat16, false>(ra, s);
}
