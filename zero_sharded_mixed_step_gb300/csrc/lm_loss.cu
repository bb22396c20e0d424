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

#include <mutex>

#include "lm_gemm.cuh"

namespace zero {
namespace {

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

int64_t loss_space(int64_t tokens, int64_t vocab) {
  tokens = std::min(tokens, kSlab);
  const int64_t tiles = ceil_div(vocab, kTileN);
  const int64_t parts = std::max(tokens * tiles, std::min(tokens, kFewTokens) * tiles * 4);
  return kStatusBytes + round_up(parts * 16, 256) + round_up(tokens * 4, 256);
}

}  // namespace
}  // namespace zero

using namespace zero;

extern "C" int64_t zero_lm_workspace_bytes(int64_t tokens, int64_t vocab, int64_t width, int with_grad) {
  int rc = check_sizes(tokens, vocab, width);
  if (rc) return rc;
  int64_t bytes = std::max<int64_t>(256, loss_space(tokens, vocab));
  if (!with_grad) return bytes;
  return std::max(bytes, grad_bytes(tokens, vocab, width));
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
    if ((rc = launch_gemm<kLoss>(g, dtype, s, stall))) return rc;
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
  const GradCall c = {tokens, vocab, width, dtype, hidden, hidden_stride, table, table_stride, targets, id_bytes, lse,
                      scale, dhidden, dhidden_stride, dtable, dtable_stride, accumulate, workspace, workspace_bytes, s};
  return run_grad<kGrad>(c, stall);
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
  unsigned int n = 0, of_logprobs = 0, of_ns = 0;
  ZERO_CUDA(cudaMemcpyFromSymbol(&n, g_lm_timeouts, sizeof n));
  ZERO_CUDA(logprobs_timeouts(&of_logprobs));
  ZERO_CUDA(ns_timeouts(&of_ns));
  n += of_logprobs + of_ns;
  const unsigned int fresh = n - seen[device];
  seen[device] = n;
  if (fresh == 0) return ZERO_OK;
  return fail(ZERO_E_STATE, "%u bounded device waits gave up on the device; what they belonged to is incomplete", fresh);
}

extern "C" int zero_lm_inject_stall(void) {
  g_stall_next = true;
  return ZERO_OK;
}
