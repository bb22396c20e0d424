// Log probabilities of given tokens under a language model's head, with the
// entropy of each distribution and its likeliest alternatives, and the
// gradients of a loss that is any function of the two.  The logits are never
// kept.
//
//   z = s h T^T            h: N tokens x d, T: V x d, both 16-bit, s > 0
//   lse_i = log sum_v exp(z_iv)
//   logp_i = z_{i,t_i} - lse_i
//   H_i = -sum_v p_iv log p_iv = lse_i - sum_v p_iv z_iv,   p_iv = exp(z_iv - lse_i)
//   the k largest z_iv with their v, the lower of two equal ones' v first
// and for a = dL/dlogp, b = dL/dH of each token
//   D_iv = a_i ([v = t_i] - p_iv) - b_i p_iv (log p_iv + H_i)
//   dh = s D T,   dT = s D^T h (+ what was there)
//
// The forward pass is one product of 2 N V d operations, whose epilogue keeps
// running sums and a list in each thread's registers while its pair of CTAs
// moves along a row of tiles (lm_gemm.cuh); the small kernels here join a
// row's few stretches.  For few tokens (few_tokens) the operands change
// places as in the loss; the logits then go to the workspace (4 V bytes a
// token, where alternatives are asked for), and the 32-row groups with the
// largest maxima are looked through again.
//
// The gradients' launches are the loss's (D, then both products, over pieces
// of the vocabulary) with another epilogue for D.  In fp16 D is scaled by a
// power of two such that its largest bound over the tokens, found on the
// device, comes below 2^14, and unscaled in the fp32 epilogues.

#include "lm_gemm.cuh"

namespace zero {
namespace {

constexpr int kMostTop = 16;

// Whether (a, at_a) comes before (b, at_b) in the list of alternatives; -1 as
// a place is that of none and comes last.
__device__ __forceinline__ bool before(float a, int at_a, float b, int at_b) {
  return a > b || (a == b && static_cast<unsigned>(at_a) < static_cast<unsigned>(at_b));
}

// The first of the 32 lanes' (v, at): two reductions of whole numbers in the
// floats' order (which -0 and 0 share).
__device__ __forceinline__ void first_of_warp(float& v, int& at) {
  const int bits = __float_as_int(v + 0.f);
  const unsigned key = static_cast<unsigned>(bits) ^ (bits < 0 ? 0xffffffffu : 0x80000000u);
  const unsigned most = __reduce_max_sync(0xffffffffu, key);
  at = static_cast<int>(__reduce_min_sync(0xffffffffu, key == most ? static_cast<unsigned>(at) : 0xffffffffu));
  v = __uint_as_float(most ^ (most & 0x80000000u ? 0x80000000u : 0xffffffffu));
}

// A list of the K first of what it is offered, in order; -infinity and NaN never are.
template <int K>
struct List {
  float v[K];
  int at[K];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      v[k] = -INFINITY;
      at[k] = -1;
    }
  }
  // in any order of places
  __device__ __forceinline__ void offer(float x, int x_at) {
    if (!before(x, x_at, v[K - 1], at[K - 1])) return;
#pragma unroll
    for (int k = K - 1; k >= 0; --k) {
      if (!before(x, x_at, v[k], at[k])) continue;
      const bool further = k > 0 && before(x, x_at, v[k > 0 ? k - 1 : 0], at[k > 0 ? k - 1 : 0]);
      v[k] = further ? v[k > 0 ? k - 1 : 0] : x;
      at[k] = further ? at[k > 0 ? k - 1 : 0] : x_at;
    }
  }
  // The first `count` of the lanes' lists, in order: lane r receives the r-th.  The lists are used up.
  __device__ __forceinline__ void first_of_lanes(int count, float& out_v, int& out_at) {
    const int lane = threadIdx.x & 31;
    out_v = -INFINITY;
    out_at = -1;
    for (int r = 0; r < count; ++r) {
      float w = v[0];
      int w_at = at[0];
      first_of_warp(w, w_at);
      if (w_at < 0) break;
      if (lane == r) {
        out_v = w;
        out_at = w_at;
      }
      if (at[0] == w_at) {
#pragma unroll
        for (int k = 0; k + 1 < K; ++k) {
          v[k] = v[k + 1];
          at[k] = at[k + 1];
        }
        v[K - 1] = -INFINITY;
        at[K - 1] = -1;
      }
    }
  }
};

// The sums of one token, joined with others of it.
struct Sums {
  float top, sum, tilt;

  __device__ __forceinline__ void join(float top2, float sum2, float tilt2, float scale2) {
    const float m = fmaxf(top, top2), ref = reference(m, scale2);
    rebase(sum, tilt, top * scale2, ref);
    rebase(sum2, tilt2, top2 * scale2, ref);
    top = m;
    sum += sum2;
    tilt += tilt2;
  }
  __device__ __forceinline__ void join_warp(float scale2) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float t = __shfl_xor_sync(0xffffffffu, top, o), s = __shfl_xor_sync(0xffffffffu, sum, o),
                  u = __shfl_xor_sync(0xffffffffu, tilt, o);
      join(t, s, u, scale2);
    }
    // the lanes' sums may differ in the last bit: each fuses another one of the two products
    top = __shfl_sync(0xffffffffu, top, 0);
    sum = __shfl_sync(0xffffffffu, sum, 0);
    tilt = __shfl_sync(0xffffffffu, tilt, 0);
  }
};

struct Combine {
  const float4* sums;
  const int2* best;
  const float* logits;
  int64_t logit_stride;
  const float* target_logit;
  const void* targets;
  int id_bytes, vocab, tokens;
  int pairs, tiles, n_tiles;   // of the stretches; kFew: n_tiles groups of 32 rows
  int top;
  float scale2;
  float *logp, *lse, *entropy, *top_logp;
  int* top_ids;
};

// Writes a token's results; one thread.
__device__ __forceinline__ void write_token(const Combine& g, int64_t row, const Sums& x) {
  const float ref = reference(x.top, g.scale2), log_sum = logf(x.sum);
  // both terms are at least 0, but for the rounding of the reference
  const float entropy = log_sum - kLn2 * __fdiv_rn(x.tilt, x.sum);
  g.lse[row] = fmaf(ref, kLn2, log_sum);
  g.entropy[row] = entropy < 0.f ? 0.f : entropy;
  const bool valid = load_target(g.targets, g.id_bytes, row, g.vocab) >= 0;
  g.logp[row] = valid ? kLn2 * fmaf(g.target_logit[row], g.scale2, -ref) - log_sum : 0.f;
}

// Writes a token's alternatives: lane r of the warp holds the r-th.
__device__ __forceinline__ void write_top(const Combine& g, int64_t row, const Sums& x, float v, int at) {
  const int lane = threadIdx.x & 31;
  if (lane >= g.top) return;
  const float ref = reference(x.top, g.scale2);
  g.top_ids[row * g.top + lane] = at;
  g.top_logp[row * g.top + lane] = kLn2 * fmaf(v, g.scale2, -ref) - logf(x.sum);
}

// Joins the stretches of each token's row: a warp a token.
template <int K>
__global__ void __launch_bounds__(kSmallThreads) join_stretches(const __grid_constant__ Combine g) {
  allow_next();
  await_previous();
  const int row = (blockIdx.x * kSmallThreads + threadIdx.x) / 32, lane = threadIdx.x & 31;
  if (row >= g.tokens) return;   // whole warps
  const int mt = row / kTileM;
  const int64_t t0 = static_cast<int64_t>(mt) * g.n_tiles, t1 = t0 + g.n_tiles;
  // the pairs whose stretches [tiles p / pairs, tiles (p + 1) / pairs) hold tiles of [t0, t1)
  auto start = [&](int64_t p) { return static_cast<int64_t>(g.tiles) * p / g.pairs; };
  int64_t first = t0 * g.pairs / g.tiles, last = (t1 - 1) * g.pairs / g.tiles;
  while (start(first + 1) <= t0) ++first;
  while (start(last + 1) < t1) ++last;
  const int parts = 2 * static_cast<int>(last - first + 1);
  auto place = [&](int q) { return ((first + (q >> 1) + mt) * kTileM + row % kTileM) * 2 + (q & 1); };
  Sums x = {-INFINITY, 0.f, 0.f};
  for (int q = lane; q < parts; q += 32) {
    const float4 y = g.sums[place(q)];
    x.join(y.x, y.y, y.z, g.scale2);
  }
  x.join_warp(g.scale2);
  if (lane == 0) write_token(g, row, x);
  if constexpr (K > 0) {
    // a stretch's list is in order: a lane takes one at a time
    float v = -INFINITY;
    int at = -1;
    for (int q0 = 0; q0 < parts; q0 += 32) {
      List<K> list;
      list.clear();
      if (q0 + lane < parts) {
        const int2* from = g.best + place(q0 + lane) * K;
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const int2 b = from[k];
          list.v[k] = __int_as_float(b.x);
          list.at[k] = b.y;
        }
      }
      float w;
      int w_at;
      list.first_of_lanes(g.top, w, w_at);
      if (q0 > 0) {
        // what there was before in the lower lanes, these in the upper ones
        List<1> one;
        const float there = __shfl_sync(0xffffffffu, w, lane & 15);
        const int there_at = __shfl_sync(0xffffffffu, w_at, lane & 15);
        one.v[0] = lane < 16 ? v : there;
        one.at[0] = lane < 16 ? at : there_at;
        one.first_of_lanes(g.top, w, w_at);
      }
      v = w;
      at = w_at;
    }
    write_top(g, row, x, v, at);
  }
}

// Threads of a token's block.  16 tokens x 50257 x 768 with 8 alternatives take 23 to 25 us so (in a graph, the same
// table call after call; 24 with another table each call); 4 us more with 256 threads, 3 with 1024.
constexpr int kGroupThreads = 512;

// The same of kFew's groups of 32 rows, which are many: a block a token.
// K: the length of its lists, 0 without alternatives; L: of a thread's, which
// sees at most L groups where L < K.
template <int K, int L>
__global__ void __launch_bounds__(kGroupThreads) join_groups(const __grid_constant__ Combine g) {
  constexpr int kWarps = kGroupThreads / 32, kList = K > 0 ? K : 2, kBatch = 4;
  __shared__ Sums of_warp[kWarps];
  __shared__ float group_max[kWarps][kList];
  __shared__ int group_at[kWarps][kList];
  __shared__ float found[32];
  __shared__ int found_at[32];
  allow_next();
  await_previous();
  const int row = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float4* p = g.sums + static_cast<int64_t>(row) * g.n_tiles;
  Sums x = {-INFINITY, 0.f, 0.f};
  // the groups with the largest maxima hold the largest logits: of this thread's groups first
  List<L> list;
  list.clear();
  for (int k0 = threadIdx.x; k0 < g.n_tiles; k0 += kBatch * kGroupThreads) {
    float4 y[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      y[k] = k0 + kGroupThreads * k < g.n_tiles ? p[k0 + kGroupThreads * k] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      x.join(y[k].x, y[k].y, y[k].z, g.scale2);
      if (K > 0 && y[k].x != -INFINITY) list.offer(y[k].x, k0 + kGroupThreads * k);
    }
  }
  x.join_warp(g.scale2);
  if (lane == 0) of_warp[warp] = x;
  if constexpr (K > 0) {
    float v;
    int at;
    list.first_of_lanes(g.top, v, at);
    if (lane < K) {
      group_max[warp][lane] = v;
      group_at[warp][lane] = at;
    }
  }
  __syncthreads();
  // one warp writes the token's results, another one its list
  if (warp > (K > 0 ? 1 : 0)) return;
  x = lane < kWarps ? of_warp[lane % kWarps] : Sums{-INFINITY, 0.f, 0.f};
  x.join_warp(g.scale2);
  if (warp == (K > 0 ? 1 : 0)) {
    if (lane == 0) write_token(g, row, x);
    return;
  }
  if constexpr (K > 0) {
    // half of a warp's list to a lane
    static_assert(kWarps == 16);
    List<kList / 2> half;
    float v;
    int at;
#pragma unroll
    for (int k = 0; k < K / 2; ++k) {
      half.v[k] = group_max[lane / 2][lane % 2 * (K / 2) + k];
      half.at[k] = group_at[lane / 2][lane % 2 * (K / 2) + k];
    }
    half.first_of_lanes(g.top, v, at);
    // then the logits of those groups, 32 each.  The maxima are so many logits already: none below the last of them is
    // listed, which leaves few.
    const float least = __shfl_sync(0xffffffffu, v, g.top - 1);
    float logit[K];
    int place[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int group = __shfl_sync(0xffffffffu, at, k);
      place[k] = group * 32 + lane;
      logit[k] = group >= 0 ? g.logits[row * g.logit_stride + place[k]] : -INFINITY;
    }
    int count = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const bool kept = logit[k] > -INFINITY && logit[k] >= least;
      const unsigned mask = __ballot_sync(0xffffffffu, kept);
      const int to = count + __popc(mask & ((1u << lane) - 1));
      if (kept && to < 32) {
        found[to] = logit[k];
        found_at[to] = place[k];
      }
      count += __popc(mask);
    }
    __syncwarp();
    if (count <= 32) {
      List<1> one;
      one.clear();
      if (lane < count) one.offer(found[lane], found_at[lane]);
      one.first_of_lanes(g.top, v, at);
    } else {
      List<K> all;
      all.clear();
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (logit[k] > -INFINITY) all.offer(logit[k], place[k]);
      all.first_of_lanes(g.top, v, at);
    }
    write_top(g, row, x, v, at);
  }
}

// ---- host -------------------------------------------------------------------------

// The length of the threads' lists for so many alternatives.
int list_length(int top) { return top == 0 ? 0 : top <= 8 ? 8 : 16; }

// Byte offsets of the workspace's parts for one slab of tokens.
struct Space {
  bool few;
  int m_tiles, n_tiles, tiles, bn;
  int64_t sums, best, logits, target_logit, total;
};

// Up to so many tokens the operands change places: as for the loss without
// alternatives, further with them, since with tokens as rows the lists of a few
// rows fill slowly, in few pairs' epilogues.  Exchanged and with tokens as rows,
// us, 8 and 16 alternatives (bf16, in a graph):
//            50257 x 768          50257 x 1600         32000 x 2048         8000 x 256
//   16       25  27    45   84    41  45    58   94    37  40    51   89    14  16    25  41
//   96       35  38    45  109    48  51    53  119    42  45    51  115    19  21    26  41
//   128      37  41    45  110    51  54    55  121    43  47    51  118    19  21    27  41
// Beyond, the logits that the exchanged form keeps, 4 V bytes a token, would take
// the workspace of a large batch past its few MB.
int64_t few_tokens(int top) { return top > 0 ? 128 : kFewTokens; }

Space space_of(int64_t tokens, int64_t vocab, int top, bool few) {
  Space s;
  s.few = few;
  s.bn = s.few ? static_cast<int>(round_up(std::max<int64_t>(tokens, 1), 32)) : kTileN;
  s.m_tiles = static_cast<int>(ceil_div(s.few ? vocab : tokens, kTileM));
  s.n_tiles = static_cast<int>(ceil_div(s.few ? tokens : vocab, s.bn));
  s.tiles = s.m_tiles * s.n_tiles;
  const int64_t entries = s.few ? tokens * s.m_tiles * 8 : (kPairs + s.m_tiles) * kTileM * 2;
  s.sums = kStatusBytes;
  s.best = s.sums + round_up(entries * 16, 256);
  s.logits = s.best + (s.few ? 0 : round_up(entries * list_length(top) * 8, 256));
  s.target_logit = s.logits + (s.few && top > 0 ? tokens * s.m_tiles * kTileM * 4 : 0);
  s.total = s.target_logit + round_up(tokens * 4, 256);
  return s;
}

Space space_of(int64_t tokens, int64_t vocab, int top) {
  return space_of(tokens, vocab, top, tokens <= few_tokens(top));
}

int check_top(int top, int64_t vocab) {
  if (top < 0 || top > kMostTop || top > vocab)
    return fail(ZERO_E_ARG, "top=%d outside [0, %d] or beyond the vocabulary", top, kMostTop);
  return ZERO_OK;
}

int check_scale(double scale) {
  const float f = static_cast<float>(scale);
  // the kernels work in powers of 2
  return std::isfinite(f * kLog2e) && f > 0.f ? ZERO_OK : fail(ZERO_E_ARG, "scale %g is not positive and below 2e38", scale);
}

int check_floats(const char* what, const void* p) {
  return reinterpret_cast<uintptr_t>(p) % 4 ? fail(ZERO_E_ALIGN, "%s must be 4-byte aligned", what) : ZERO_OK;
}

}  // namespace

cudaError_t logprobs_timeouts(unsigned int* out) { return cudaMemcpyFromSymbol(out, g_lm_timeouts, sizeof *out); }

}  // namespace zero

using namespace zero;

extern "C" int64_t zero_lm_logprobs_workspace_bytes(int64_t tokens, int64_t vocab, int64_t width, int top,
                                                    int with_grad) {
  int rc = check_sizes(tokens, vocab, width);
  if (rc || (rc = check_top(top, vocab))) return rc;
  // any smaller count of tokens and of alternatives has to fit too: the few tokens' form needs more for each token
  int64_t bytes = space_of(std::min(tokens, few_tokens(top)), vocab, top, true).total;
  if (tokens > kFewTokens) bytes = std::max(bytes, space_of(std::min(tokens, kSlab), vocab, top, false).total);
  if (with_grad) bytes = std::max(bytes, grad_bytes(tokens, vocab, width, 3));
  return bytes;
}

extern "C" int zero_lm_logprobs(int64_t tokens, int64_t vocab, int64_t width, int dtype, const void* hidden,
                                int64_t hidden_stride, const void* table, int64_t table_stride, const void* targets,
                                int id_bytes, double scale, int top, float* logp, float* entropy, float* lse,
                                float* top_logp, int32_t* top_ids, void* workspace, int64_t workspace_bytes,
                                void* stream) {
  bool stall = take_stall();
  int rc = check_common(tokens, vocab, width, dtype, hidden, hidden_stride, table, table_stride, targets, id_bytes,
                        workspace);
  if (rc || (rc = check_scale(scale)) || (rc = check_top(top, vocab))) return rc;
  if (tokens > 0 && (!logp || !entropy || !lse)) return fail(ZERO_E_ARG, "logp, entropy and lse are required");
  if (tokens > 0 && top > 0 && (!top_logp || !top_ids)) return fail(ZERO_E_ARG, "top=%d needs top_logp and top_ids", top);
  if ((rc = check_floats("logp", logp)) || (rc = check_floats("entropy", entropy)) || (rc = check_floats("lse", lse)) ||
      (rc = check_floats("top_logp", top_logp)) || (rc = check_floats("top_ids", top_ids)))
    return rc;
  if (tokens == 0) return ZERO_OK;
  const int64_t needed = space_of(std::min(tokens, kSlab), vocab, top).total;
  const int64_t rest = tokens > kSlab ? space_of(tokens % kSlab, vocab, top).total : 0;
  if (workspace_bytes < std::max(needed, rest))
    return fail(ZERO_E_ARG, "workspace of %lld bytes: %lld are needed", (long long)workspace_bytes,
                (long long)std::max(needed, rest));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  for (int64_t i0 = 0; i0 < tokens; i0 += kSlab) {
    const int64_t count = std::min(kSlab, tokens - i0);
    const Space sp = space_of(count, vocab, top);
    GemmArgs g;
    std::memset(&g, 0, sizeof g);
    Job& j = g.job[0];
    j.kind = sp.few ? kFew : kStats;
    j.M = static_cast<int>(sp.few ? vocab : count);
    j.N = static_cast<int>(sp.few ? count : vocab);
    j.bn = sp.bn;
    j.m_tiles = sp.m_tiles;
    j.n_tiles = sp.n_tiles;
    j.splits = 1;
    j.tiles = sp.tiles;
    j.kb_total = static_cast<int>(ceil_div(width, kTileK));
    j.stage_tx = 2 * (kOperandBytes + j.bn / 2 * kTileK * 2);
    g.jobs = 1;
    g.vocab = static_cast<int>(vocab);
    g.targets = static_cast<const char*>(targets) + i0 * id_bytes;
    g.id_bytes = id_bytes;
    g.failures = static_cast<unsigned int*>(workspace);
    g.scale2 = static_cast<float>(scale) * kLog2e;
    g.sums = reinterpret_cast<float4*>(ws + sp.sums);
    g.best = reinterpret_cast<int2*>(ws + sp.best);
    g.target_logit = reinterpret_cast<float*>(ws + sp.target_logit);
    if (sp.few && top > 0) {
      g.logits = reinterpret_cast<float*>(ws + sp.logits);
      g.logit_stride = int64_t{sp.m_tiles} * kTileM;
    }
    const uint16_t* rows = static_cast<const uint16_t*>(hidden) + i0 * hidden_stride;
    CUtensorMap *of_tokens = sp.few ? &g.b[0] : &g.a[0], *of_vocab = sp.few ? &g.a[0] : &g.b[0];
    if ((rc = make_map(of_tokens, dtype, rows, count, width, hidden_stride, sp.few ? j.bn / 2 : 128))) return rc;
    if ((rc = make_map(of_vocab, dtype, table, vocab, width, table_stride, sp.few ? 128 : j.bn / 2))) return rc;
    const int list = sp.few ? kFewK : list_length(top);
    rc = sp.few      ? launch_gemm<kLogprobs, kFewK>(g, dtype, s, stall)
         : list == 0 ? launch_gemm<kLogprobs, 0>(g, dtype, s, stall)
         : list == 8 ? launch_gemm<kLogprobs, 8>(g, dtype, s, stall)
                     : launch_gemm<kLogprobs, 16>(g, dtype, s, stall);
    if (rc) return rc;
    Combine c = {g.sums, g.best, g.logits, g.logit_stride, g.target_logit, g.targets, id_bytes, g.vocab,
                 static_cast<int>(count), pairs_for(sp.tiles), sp.tiles, sp.few ? sp.m_tiles * 8 : sp.n_tiles, top,
                 g.scale2, logp + i0, lse + i0, entropy + i0, top > 0 ? top_logp + i0 * top : nullptr,
                 top > 0 ? top_ids + i0 * top : nullptr};
    const int most = static_cast<int>(ceil_div(c.n_tiles, kGroupThreads));   // groups of a thread
    const auto fn = sp.few ? (list_length(top) == 0    ? join_groups<0, 1>
                              : list_length(top) == 8 ? (most <= 4 ? join_groups<8, 4> : join_groups<8, 8>)
                              : most <= 4             ? join_groups<16, 4>
                              : most <= 8             ? join_groups<16, 8>
                                                      : join_groups<16, 16>)
                           : (list == 0 ? join_stretches<0> : list == 8 ? join_stretches<8> : join_stretches<16>);
    const dim3 grid(static_cast<unsigned>(sp.few ? count : ceil_div(count * 32, kSmallThreads)));
    ZERO_CUDA(launch_chained(fn, grid, sp.few ? kGroupThreads : kSmallThreads, 0, s, c));
  }
  return ZERO_OK;
}

extern "C" int zero_lm_logprobs_grad(int64_t tokens, int64_t vocab, int64_t width, int dtype, const void* hidden,
                                     int64_t hidden_stride, const void* table, int64_t table_stride,
                                     const void* targets, int id_bytes, double scale, const float* lse,
                                     const float* dlogp, const float* entropy, const float* dentropy, void* dhidden,
                                     int64_t dhidden_stride, void* dtable, int64_t dtable_stride, int accumulate,
                                     void* workspace, int64_t workspace_bytes, void* stream) {
  bool stall = take_stall();
  int rc = check_common(tokens, vocab, width, dtype, hidden, hidden_stride, table, table_stride, targets, id_bytes,
                        workspace);
  if (rc || (rc = check_scale(scale))) return rc;
  if (tokens > 0 && (!lse || !dlogp)) return fail(ZERO_E_ARG, "lse and dlogp are required");
  if (tokens > 0 && dentropy && !entropy) return fail(ZERO_E_ARG, "dentropy needs the entropy");
  if ((rc = check_floats("lse", lse)) || (rc = check_floats("dlogp", dlogp)) ||
      (rc = check_floats("entropy", entropy)) || (rc = check_floats("dentropy", dentropy)))
    return rc;
  if ((rc = check_matrix("dhidden", dhidden, dhidden_stride, tokens, width))) return rc;
  if ((rc = check_matrix("dtable", dtable, dtable_stride, vocab, width))) return rc;
  const GradCall c = {tokens, vocab, width, dtype, hidden, hidden_stride, table, table_stride, targets, id_bytes, lse,
                      scale, dhidden, dhidden_stride, dtable, dtable_stride, accumulate, workspace, workspace_bytes,
                      static_cast<cudaStream_t>(stream), dlogp, dentropy, entropy, scale};
  return run_grad<kWeighted>(c, stall);
}
