// Load-balance loss of the router over packed sequences, with per-expert counts
// and its gradient.  For sequence s with n_s valid tokens:
//   p_t = softmax(l_t), or sigmoid(l_t) / sum_j sigmoid(l_tj)   (the router's gating over all experts)
//   c_si = how often expert i was picked by its tokens
//   f_si = E c_si / (top_k n_s),  P_si = (1 / n_s) sum_t p_ti
//   loss = coef * mean over the sequences with tokens of sum_i f_si P_si
// and, the counts being constants, with a_si = d_loss * coef * f_si / (n_s live):
//   d_l = p (a - sum_j a_j p_j), times (1 - sigmoid(l)) for sigmoid gating.
//
// Bound by HBM at many tokens (the logits once per direction) and by latency
// at few.  A CTA takes a run of tokens, a warp a token at a time with its
// probabilities' sums in registers; what a CTA has of a sequence goes to slot
// (run + sequence) of the workspace -- no two pairs share one, since walking
// through the tokens advances either the run or the sequence -- and the slots
// are added in order: no float atomics, the same bits on every run.  Up to 128
// tokens of one sequence are one CTA and one launch.
#include <cmath>

#include "block_ops.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kWarps = 16;
constexpr int kSmallTokens = 128;

int run_length(int tokens) {   // tokens per CTA: at least two per warp, at most two CTAs' worth of runs per SM
  return std::max(2 * kWarps, (tokens + 2 * 148 - 1) / (2 * 148));
}
// Workspace: slots of 32-bit words (experts probability sums, experts counts,
// the valid tokens), then two words per sequence (its loss, whether it has tokens).
__host__ __device__ __forceinline__ int slot_stride(int experts) { return 2 * experts + 1; }
__host__ __device__ __forceinline__ int64_t totals_at(int tokens, int experts, int seqs, int run) {
  return ((int64_t)(tokens + run - 1) / run + seqs) * slot_stride(experts);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The probabilities of one token (expert lane + 32 i in p[i]); behind the last
// expert and for a token without a finite logit zeros.  kGrad: om = d p / d l
// over p's own share, 1 - sigmoid(l) or 1.
template <int kPL, bool kGrad>
__device__ __forceinline__ void probabilities(const float* __restrict__ l, int experts, int gating, float* p, float* om) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < kPL; ++i) p[i] = lane + 32 * i < experts ? __ldg(l + lane + 32 * i) : -INFINITY;
  float sum = 0.f, m = -INFINITY;
#pragma unroll
  for (int i = 0; i < kPL; ++i) m = fmaxf(m, p[i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  // far below zero sigmoid(l) is exp(l) to 1e-26, and its normalised form the softmax, which cannot underflow
  if (gating == 0 || m < -60.f) {
    if (m == -INFINITY) m = 0.f;
#pragma unroll
    for (int i = 0; i < kPL; ++i) {
      p[i] = expf(p[i] - m);
      sum += p[i];
      if (kGrad) om[i] = 1.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPL; ++i) {
      const float v = p[i], e = expf(-v);
      p[i] = 1.f / (1.f + e);
      sum += p[i];
      if (kGrad) om[i] = v > 0.f ? e * p[i] : 1.f - p[i];
    }
  }
  sum = warp_sum(sum);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int i = 0; i < kPL; ++i) p[i] *= inv;
}

// Sequence of token t, or -1: offsets[s] <= t < offsets[s + 1].
__device__ __forceinline__ int sequence_of(const int* __restrict__ offsets, int seqs, int t) {
  if (!offsets) return 0;
  if (t < __ldg(offsets) || t >= __ldg(offsets + seqs)) return -1;
  int lo = 0, hi = seqs;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(offsets + mid) <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// Slopes and loss of one sequence from its sums; called by a CTA.  Returns the
// loss (times the number of live sequences) in thread 0.
__device__ __forceinline__ float finish(const BalanceArgs& a, int s, float n, const float* s_p, const int* s_c, float* s_red) {
  float term = 0.f;
  for (int e = threadIdx.x; e < a.experts; e += blockDim.x) {
    const float f = n > 0.f ? (float)a.experts * (float)s_c[e] / ((float)a.top_k * n) : 0.f;
    const float slope = n > 0.f ? a.coef * f / n : 0.f;
    a.counts[(int64_t)s * a.experts + e] = s_c[e];
    a.slope[(int64_t)s * a.experts + e] = slope;
    term += f > 0.f ? slope * s_p[e] : 0.f;
  }
  term = warp_sum(term);
  if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = term;
  __syncthreads();
  float v = 0.f;
  if (threadIdx.x == 0)
    for (int i = 0; i < (int)(blockDim.x >> 5); ++i) v += s_red[i];
  return v;
}

template <int kPL>
__global__ void __launch_bounds__(kWarps * 32) balance_runs_kernel(const BalanceArgs a, int run, int whole) {
  extern __shared__ float s_mem[];              // [kWarps][experts] sums, [experts] counts
  int* s_c = reinterpret_cast<int*>(s_mem + kWarps * a.experts);
  __shared__ int s_n;
  __shared__ float s_red[kWarps];
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t0 = blockIdx.x * run, t1 = min(t0 + run, a.tokens);
  int t = t0;
  if (a.offsets) t = max(t, min(__ldg(a.offsets), t1));
  for (int s = whole ? 0 : t < t1 ? sequence_of(a.offsets, a.seqs, t) : -1; s >= 0 && s < a.seqs && (t < t1 || whole); ++s) {
    const int end = min(t1, a.offsets ? __ldg(a.offsets + s + 1) : a.tokens);
    if (end <= t && !whole) continue;            // an empty sequence
    for (int e = threadIdx.x; e < a.experts; e += blockDim.x) s_c[e] = 0;
    if (threadIdx.x == 0) s_n = 0;
    __syncthreads();
    float acc[kPL] = {};
    int valid = 0;
    for (int r = t + warp; r < end; r += kWarps) {
      if (a.mask && !__ldg(a.mask + r)) continue;
      ++valid;
      if (lane < a.top_k) {
        const int id = __ldg(a.ids + (int64_t)r * a.top_k + lane);
        if ((unsigned)id < (unsigned)a.experts) atomicAdd(s_c + id, 1);
      }
      float p[kPL];
      probabilities<kPL, false>(a.logits + r * a.ld, a.experts, a.gating, p, nullptr);
#pragma unroll
      for (int i = 0; i < kPL; ++i) acc[i] += p[i];
    }
#pragma unroll
    for (int i = 0; i < kPL; ++i)
      if (lane + 32 * i < a.experts) s_mem[warp * a.experts + lane + 32 * i] = acc[i];
    if (lane == 0 && valid) atomicAdd(&s_n, valid);
    __syncthreads();
    float* slot = a.partial + ((int64_t)blockIdx.x + s) * slot_stride(a.experts);
    for (int e = threadIdx.x; e < a.experts; e += blockDim.x) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += s_mem[w * a.experts + e];
      if (whole) {
        s_mem[e] = v;
      } else {
        slot[e] = v;
        reinterpret_cast<int*>(slot)[a.experts + e] = s_c[e];
      }
    }
    if (whole) {
      __syncthreads();
      const float v = finish(a, 0, (float)s_n, s_mem, s_c, s_red);
      if (threadIdx.x == 0) *a.loss = v;
      return;
    }
    if (threadIdx.x == 0) reinterpret_cast<int*>(slot)[2 * a.experts] = s_n;
    t = end;
    __syncthreads();
  }
}

// One CTA per sequence: its slots added in order.  seqs == 1: also the loss.
__global__ void __launch_bounds__(512) balance_sequences_kernel(const BalanceArgs a, int run) {
  extern __shared__ float s_p[];                 // [experts] sums, [experts] counts
  int* s_c = reinterpret_cast<int*>(s_p + a.experts);
  __shared__ float s_red[16];
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int s = blockIdx.x, stride = slot_stride(a.experts);
  int lo = a.offsets ? min(max(__ldg(a.offsets + s), 0), a.tokens) : 0;
  const int hi = a.offsets ? min(__ldg(a.offsets + s + 1), a.tokens) : a.tokens;
  int n = 0;
  const int c0 = lo / run, c1 = hi > lo ? (hi - 1) / run + 1 : c0;
  for (int c = c0; c < c1; ++c) n += __ldcg(reinterpret_cast<const int*>(a.partial) + ((int64_t)c + s) * stride + 2 * a.experts);
  for (int e = threadIdx.x; e < a.experts; e += blockDim.x) {
    float v = 0.f;
    int k = 0;
    for (int c = c0; c < c1; ++c) {
      const float* slot = a.partial + ((int64_t)c + s) * stride;
      v += __ldcg(slot + e);
      k += __ldcg(reinterpret_cast<const int*>(slot) + a.experts + e);
    }
    s_p[e] = v;
    s_c[e] = k;
  }
  __syncthreads();
  const float v = finish(a, s, (float)n, s_p, s_c, s_red);
  if (threadIdx.x == 0) {
    if (a.seqs == 1) {
      *a.loss = v;
    } else {
      float* totals = a.partial + totals_at(a.tokens, a.experts, a.seqs, run);
      totals[2 * s] = v;
      totals[2 * s + 1] = n > 0 ? 1.f : 0.f;
    }
  }
}

// Several sequences: the mean over those with tokens.
__global__ void __launch_bounds__(512) balance_mean_kernel(const BalanceArgs a, int run) {
  __shared__ float s_v[16], s_k[16];
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const float* totals = a.partial + totals_at(a.tokens, a.experts, a.seqs, run);
  float v = 0.f, k = 0.f;
  for (int s = threadIdx.x; s < a.seqs; s += blockDim.x) {
    v += __ldcg(totals + 2 * s);
    k += __ldcg(totals + 2 * s + 1);
  }
  v = warp_sum(v);
  k = warp_sum(k);
  if ((threadIdx.x & 31) == 0) {
    s_v[threadIdx.x >> 5] = v;
    s_k[threadIdx.x >> 5] = k;
  }
  __syncthreads();
  v = k = 0.f;
  for (int i = 0; i < (int)(blockDim.x >> 5); ++i) {
    v += s_v[i];
    k += s_k[i];
  }
  const float inv = k > 0.f ? 1.f / k : 0.f;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.loss = v * inv;
  const int64_t n = (int64_t)a.seqs * a.experts;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x)
    a.slope[i] *= inv;
}

// One warp per run of tokens.
template <int kPL>
__global__ void __launch_bounds__(256) balance_grad_kernel(const BalanceGradArgs a, int per_warp) {
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t first = ((int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) * per_warp;
  if (first >= a.tokens) return;
  const int t0 = (int)first, t1 = min(t0 + per_warp, a.tokens);
  const float up = a.d_loss ? __ldg(a.d_loss) : 1.f;
  int s = sequence_of(a.offsets, a.seqs, t0);
  for (int t = t0; t < t1; ++t) {
    if (a.offsets && (s < 0 || t >= __ldg(a.offsets + s + 1))) s = sequence_of(a.offsets, a.seqs, t);
    float* out = a.d_logits + t * a.ld_out;
    if (s < 0 || (a.mask && !__ldg(a.mask + t))) {
#pragma unroll
      for (int i = 0; i < kPL; ++i)
        if (lane + 32 * i < a.experts) out[lane + 32 * i] = 0.f;
      continue;
    }
    float p[kPL], om[kPL], k[kPL], dot = 0.f;
    const float* slope = a.slope + (int64_t)s * a.experts;
#pragma unroll
    for (int i = 0; i < kPL; ++i) k[i] = lane + 32 * i < a.experts ? up * __ldg(slope + lane + 32 * i) : 0.f;
    probabilities<kPL, true>(a.logits + t * a.ld, a.experts, a.gating, p, om);
#pragma unroll
    for (int i = 0; i < kPL; ++i) dot = fmaf(k[i], p[i], dot);
    dot = warp_sum(dot);
#pragma unroll
    for (int i = 0; i < kPL; ++i)
      if (lane + 32 * i < a.experts) out[lane + 32 * i] = p[i] * (k[i] - dot) * om[i];
  }
}

template <int kPL>
cudaError_t forward(const BalanceArgs& a, cudaStream_t st) {
  const bool whole = a.tokens <= kSmallTokens && a.seqs == 1 && !a.offsets;
  const int run = whole ? std::max(a.tokens, 1) : run_length(a.tokens), runs = std::max(1, (a.tokens + run - 1) / run);
  const size_t smem = (size_t)(kWarps + 1) * a.experts * 4;
  auto* kernel = balance_runs_kernel<kPL>;
  cudaError_t e = cudaSuccess;
  if (smem > 40 * 1024) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess)
    e = launch_dependent(kernel, dim3((unsigned)runs), dim3(kWarps * 32), smem, st, 1, a, run, whole ? 1 : 0);
  if (e != cudaSuccess || whole) return e;
  e = launch_dependent(balance_sequences_kernel, dim3((unsigned)a.seqs), dim3(512), (size_t)a.experts * 8, st, 1, a, run);
  if (e != cudaSuccess || a.seqs == 1) return e;
  const unsigned blocks = (unsigned)std::min<int64_t>(sm_count(), ((int64_t)a.seqs * a.experts + 511) / 512);
  return launch_dependent(balance_mean_kernel, dim3(blocks), dim3(512), 0, st, 1, a, run);
}

template <int kPL>
cudaError_t backward(const BalanceGradArgs& a, cudaStream_t st) {
  const int warps = sm_count() * 64;
  const int per_warp = std::max(1, (a.tokens + warps - 1) / warps);
  const int blocks = ((a.tokens + per_warp - 1) / per_warp + 7) / 8;
  return launch_dependent(balance_grad_kernel<kPL>, dim3((unsigned)blocks), dim3(256), 0, st, 1, a, per_warp);
}

}  // namespace

size_t balance_workspace(int tokens, int experts, int seqs) {
  return (size_t)(totals_at(tokens, experts, seqs, run_length(tokens)) + 2 * (int64_t)seqs) * 4;
}
int balance_launches(int tokens, int seqs, bool packed) {
  return tokens <= kSmallTokens && seqs == 1 && !packed ? 1 : seqs == 1 ? 2 : 3;
}
cudaError_t launch_balance(const BalanceArgs& a, cudaStream_t st) {
  return a.experts <= 128 ? forward<4>(a, st) : a.experts <= 256 ? forward<8>(a, st) : a.experts <= 512 ? forward<16>(a, st)
                                                                                            : forward<32>(a, st);
}
cudaError_t launch_balance_grad(const BalanceGradArgs& a, cudaStream_t st) {
  return a.experts <= 128 ? backward<4>(a, st) : a.experts <= 256 ? backward<8>(a, st) : a.experts <= 512 ? backward<16>(a, st)
                                                                                             : backward<32>(a, st);
}

}  // namespace moe
