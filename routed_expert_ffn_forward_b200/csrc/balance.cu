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
// Workspace, in 32-bit words: slots of the experts' probability sums, their
// counts and the valid tokens, each part padded to 4 words; then two words per
// sequence and column block (its share of the loss, whether it has tokens).
__host__ __device__ __forceinline__ int padded(int experts) { return (experts + 3) & ~3; }
__host__ __device__ __forceinline__ int slot_stride(int experts) { return 2 * padded(experts) + 4; }
__host__ __device__ __forceinline__ int64_t totals_at(int tokens, int experts, int seqs, int run) {
  return ((int64_t)(tokens + run - 1) / run + seqs) * slot_stride(experts);
}
constexpr int kBlockCols = 128;   // experts per CTA of the second step
__host__ __device__ __forceinline__ int column_blocks(int experts) { return (experts + kBlockCols - 1) / kBlockCols; }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Expert of this lane's value i of kPL: fours of them with kVec (16-byte
// accesses: experts and row stride multiples of 4, rows aligned), else every 32nd.
template <bool kVec>
__device__ __forceinline__ int expert_of(int i) {
  const int lane = threadIdx.x & 31;
  return kVec ? 128 * (i >> 2) + 4 * lane + (i & 3) : 32 * i + lane;
}
template <int kPL, bool kVec>
__device__ __forceinline__ void load_row(const float* __restrict__ l, int experts, float other, float* v) {
  if (kVec) {
#pragma unroll
    for (int i = 0; i < kPL; i += 4) {
      const int e = expert_of<true>(i);
      float4 q = make_float4(other, other, other, other);
      if (e < experts) q = __ldg(reinterpret_cast<const float4*>(l + e));
      v[i] = q.x;
      v[i + 1] = q.y;
      v[i + 2] = q.z;
      v[i + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPL; ++i) v[i] = expert_of<false>(i) < experts ? __ldg(l + expert_of<false>(i)) : other;
  }
}
template <int kPL, bool kVec>
__device__ __forceinline__ void store_row(float* l, int experts, const float* v) {
  if (kVec) {
#pragma unroll
    for (int i = 0; i < kPL; i += 4) {
      const int e = expert_of<true>(i);
      if (e < experts) *reinterpret_cast<float4*>(l + e) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPL; ++i)
      if (expert_of<false>(i) < experts) l[expert_of<false>(i)] = v[i];
  }
}

// A token's logits (-infinity behind the last expert) to its probabilities, in
// place; zeros for a token without a finite logit.  kGrad: om = 1 - sigmoid(l)
// or 1.  The exponential is the fast one (2 + 1.2 |l - max| steps of 2^-23):
// with the exact one and IEEE division, 40 instructions a logit, the pass over
// 65536 x 256 logits took 36 us, twice its HBM time.  In steps of 2^-24 a
// softmax is off by at most 4 + 3.4 d of its own exponential, d = max - l, as
// much of the others' (their mean d is at most log 1024), 37 of their sum and 2
// of the rest; a sigmoid's 9 + 2.4 |l| replace the exponentials'.
template <int kPL, bool kGrad>
__device__ __forceinline__ void probabilities(int gating, float* p, float* om) {
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
      p[i] = __expf(p[i] - m);
      sum += p[i];
      if (kGrad) om[i] = 1.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPL; ++i) {
      const float v = p[i], e = __expf(-v);
      p[i] = __fdividef(1.f, 1.f + e);   // 0 where e is out of range
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

// Slope and term of the loss of one expert of a sequence with n valid tokens.
__device__ __forceinline__ float finish(const BalanceArgs& a, int s, int e, float n, float sum, int count) {
  const float f = n > 0.f ? (float)a.experts * (float)count / ((float)a.top_k * n) : 0.f;
  const float slope = n > 0.f ? a.coef * f / n : 0.f;
  a.counts[(int64_t)s * a.experts + e] = count;
  a.slope[(int64_t)s * a.experts + e] = slope;
  return f > 0.f ? slope * sum : 0.f;
}
// Sum over the CTA, in thread 0.
__device__ __forceinline__ float block_sum(float v, float* s_red) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
  if (threadIdx.x == 0)
    for (int i = 0; i < (int)(blockDim.x >> 5); ++i) v += s_red[i];
  return v;
}

template <int kPL, bool kVec>
__global__ void __launch_bounds__(kWarps * 32) balance_runs_kernel(const BalanceArgs a, int run, int whole) {
  extern __shared__ __align__(16) float s_mem[];   // [kWarps][padded experts] sums (stored as float4), [experts] counts
  const int width = padded(a.experts);
  int* s_c = reinterpret_cast<int*>(s_mem + kWarps * width);
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
    // the next tokens' logits, picks and mask are on their way while these ones'
    // are summed (the picks' latency alone was 1.8 us a token): two tokens of up
    // to 256 experts per warp
    constexpr int kAhead = kPL <= 8 ? 2 : 1;
    float acc[kPL] = {}, next[kAhead][kPL];
    int pick[kAhead], counts[kAhead];
    int valid = 0;
    auto fetch = [&](int r, int j) {
      counts[j] = 0;
      if (r >= end) return;
      counts[j] = a.mask ? __ldg(a.mask + r) : 1;
      pick[j] = lane < a.top_k ? __ldg(a.ids + (int64_t)r * a.top_k + lane) : -1;
      load_row<kPL, kVec>(a.logits + r * a.ld, a.experts, -INFINITY, next[j]);
    };
#pragma unroll
    for (int j = 0; j < kAhead; ++j) fetch(t + warp + j * kWarps, j);
    for (int r0 = t + warp; r0 < end; r0 += kAhead * kWarps) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int now = counts[j], id = pick[j];
        float p[kPL];
#pragma unroll
        for (int i = 0; i < kPL; ++i) p[i] = next[j][i];
        fetch(r0 + (j + kAhead) * kWarps, j);
        if (!now) continue;
        ++valid;
        if ((unsigned)id < (unsigned)a.experts) atomicAdd(s_c + id, 1);
        probabilities<kPL, false>(a.gating, p, nullptr);
#pragma unroll
        for (int i = 0; i < kPL; ++i) acc[i] += p[i];
      }
    }
    store_row<kPL, kVec>(s_mem + warp * width, a.experts, acc);
    if (lane == 0 && valid) atomicAdd(&s_n, valid);
    __syncthreads();
    float* slot = a.partial + ((int64_t)blockIdx.x + s) * slot_stride(a.experts);
    float term = 0.f;
    for (int e = threadIdx.x; e < a.experts; e += blockDim.x) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += s_mem[w * width + e];
      if (whole) {
        term += finish(a, 0, e, (float)s_n, v, s_c[e]);
      } else {
        slot[e] = v;
        reinterpret_cast<int*>(slot)[width + e] = s_c[e];
      }
    }
    if (whole) {
      term = block_sum(term, s_red);
      if (threadIdx.x == 0) *a.loss = term;
      return;
    }
    if (threadIdx.x == 0) reinterpret_cast<int*>(slot)[2 * width] = s_n;
    t = end;
    __syncthreads();
  }
}

// One CTA per 128 experts of a sequence: its slots' shares added in order, lane
// l of a warp four experts, the warps' shares of the slots after one another.
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(kSumWarps * 32) balance_sequences_kernel(const BalanceArgs a, int run) {
  __shared__ float4 s_p[kSumWarps][33];
  __shared__ int4 s_c[kSumWarps][33];
  __shared__ int s_n;
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int s = blockIdx.y, stride = slot_stride(a.experts), width = padded(a.experts);
  const int lo = a.offsets ? min(max(__ldg(a.offsets + s), 0), a.tokens) : 0;
  const int hi = a.offsets ? min(__ldg(a.offsets + s + 1), a.tokens) : a.tokens;
  const int c0 = lo / run, c1 = hi > lo ? (hi - 1) / run + 1 : c0;
  if (threadIdx.x == 0) s_n = 0;
  __syncthreads();
  const int e = blockIdx.x * kBlockCols + 4 * lane;
  float4 p = make_float4(0.f, 0.f, 0.f, 0.f);
  int4 k = make_int4(0, 0, 0, 0);
  int n = 0;
#pragma unroll 4
  for (int c = c0 + warp; c < c1; c += kSumWarps) {
    const float* slot = a.partial + ((int64_t)c + s) * stride;
    if (e < width) {
      const float4 q = __ldcg(reinterpret_cast<const float4*>(slot + e));
      const int4 j = __ldcg(reinterpret_cast<const int4*>(slot + width + e));
      p.x += q.x; p.y += q.y; p.z += q.z; p.w += q.w;
      k.x += j.x; k.y += j.y; k.z += j.z; k.w += j.w;
    }
    if (lane == 0) n += __ldcg(reinterpret_cast<const int*>(slot) + 2 * width);
  }
  s_p[warp][lane] = p;
  s_c[warp][lane] = k;
  if (lane == 0 && n) atomicAdd(&s_n, n);
  __syncthreads();
  if (warp >= 4) return;
  // thread i of the first 128: expert i of the block
  const int i = threadIdx.x, mine = blockIdx.x * kBlockCols + i;
  float v = 0.f;
  int cnt = 0;
#pragma unroll 8
  for (int w = 0; w < kSumWarps; ++w) {
    v += reinterpret_cast<const float*>(&s_p[w][i >> 2])[i & 3];
    cnt += reinterpret_cast<const int*>(&s_c[w][i >> 2])[i & 3];
  }
  float term = mine < a.experts ? finish(a, s, mine, (float)s_n, v, cnt) : 0.f;
  term = warp_sum(term);
  __shared__ float s_red[4];
  if (lane == 0) s_red[warp] = term;
  ptx::named_barrier_sync(1, 128);
  if (i == 0) {
    float2* totals = reinterpret_cast<float2*>(a.partial + totals_at(a.tokens, a.experts, a.seqs, run));
    totals[(int64_t)s * gridDim.x + blockIdx.x] =
        make_float2(s_red[0] + s_red[1] + s_red[2] + s_red[3], s_n > 0 && blockIdx.x == 0 ? 1.f : 0.f);
  }
}

// The mean over the sequences with tokens; several of them: the slopes, too.
__global__ void __launch_bounds__(512) balance_mean_kernel(const BalanceArgs a, int run) {
  __shared__ float s_v[16], s_k[16];
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const float2* totals = reinterpret_cast<const float2*>(a.partial + totals_at(a.tokens, a.experts, a.seqs, run));
  float v = 0.f, k = 0.f;
  for (int s = threadIdx.x; s < a.seqs * column_blocks(a.experts); s += blockDim.x) {
    const float2 q = __ldcg(totals + s);
    v += q.x;
    k += q.y;
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
  if (a.seqs == 1) return;
  const int64_t n = (int64_t)a.seqs * a.experts;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x)
    a.slope[i] *= inv;
}

// One warp per run of tokens; the next token's logits are on their way.
template <int kPL, bool kVec>
__global__ void __launch_bounds__(256) balance_grad_kernel(const BalanceGradArgs a, int per_warp) {
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int64_t first = ((int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) * per_warp;
  if (first >= a.tokens) return;
  const int t0 = (int)first, t1 = min(t0 + per_warp, a.tokens);
  const float up = a.d_loss ? __ldg(a.d_loss) : 1.f;
  int s = -1, end = t0;   // the sequence whose slopes are in k, and where it ends
  float next[kPL], k[kPL];
  load_row<kPL, kVec>(a.logits + t0 * a.ld, a.experts, -INFINITY, next);
  for (int t = t0; t < t1; ++t) {
    float p[kPL], om[kPL];
#pragma unroll
    for (int i = 0; i < kPL; ++i) p[i] = next[i];
    if (t + 1 < t1) load_row<kPL, kVec>(a.logits + (t + 1) * a.ld, a.experts, -INFINITY, next);
    if (t >= end) {
      s = sequence_of(a.offsets, a.seqs, t);
      end = !a.offsets ? a.tokens : s >= 0 ? __ldg(a.offsets + s + 1) : t + 1;
      if (s >= 0) load_row<kPL, kVec>(a.slope + (int64_t)s * a.experts, a.experts, 0.f, k);
    }
    if (s < 0 || (a.mask && !__ldg(a.mask + t))) {
#pragma unroll
      for (int i = 0; i < kPL; ++i) p[i] = 0.f;
    } else {
      float dot = 0.f;
      probabilities<kPL, true>(a.gating, p, om);
#pragma unroll
      for (int i = 0; i < kPL; ++i) dot = fmaf(k[i], p[i], dot);
      dot = warp_sum(dot);
#pragma unroll
      for (int i = 0; i < kPL; ++i) p[i] *= up * (k[i] - dot) * om[i];
    }
    store_row<kPL, kVec>(a.d_logits + t * a.ld_out, a.experts, p);
  }
}

bool vectors_of_4(const void* p, int64_t ld, int experts) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 4 == 0 && experts % 4 == 0;
}

template <int kPL, bool kVec>
cudaError_t forward_as(const BalanceArgs& a, cudaStream_t st) {
  const bool whole = a.tokens <= kSmallTokens && a.seqs == 1 && !a.offsets;
  const int run = whole ? std::max(a.tokens, 1) : run_length(a.tokens), runs = std::max(1, (a.tokens + run - 1) / run);
  const size_t smem = ((size_t)kWarps * padded(a.experts) + a.experts) * 4;
  constexpr int kMost = (kWarps + 1) * 32 * kPL * 4;   // of this kernel's most experts
  auto* kernel = balance_runs_kernel<kPL, kVec>;
  cudaError_t e = cudaSuccess;
  // (what a kernel may take is a limit of its own, not of a launch: never a call's size, which may be less than that of
  // another thread's call)
  if (kMost > 40 * 1024) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
  if (e == cudaSuccess)
    e = launch_dependent(kernel, dim3((unsigned)runs), dim3(kWarps * 32), smem, st, 1, a, run, whole ? 1 : 0);
  if (e != cudaSuccess || whole) return e;
  e = launch_dependent(balance_sequences_kernel, dim3((unsigned)column_blocks(a.experts), (unsigned)a.seqs),
                       dim3(kSumWarps * 32), 0, st, 1, a, run);
  if (e != cudaSuccess) return e;
  const unsigned blocks =
      a.seqs == 1 ? 1 : (unsigned)std::min<int64_t>(sm_count(), ((int64_t)a.seqs * a.experts + 511) / 512);
  return launch_dependent(balance_mean_kernel, dim3(blocks), dim3(512), 0, st, 1, a, run);
}
template <int kPL>
cudaError_t forward(const BalanceArgs& a, cudaStream_t st) {
  return vectors_of_4(a.logits, a.ld, a.experts) ? forward_as<kPL, true>(a, st) : forward_as<kPL, false>(a, st);
}

template <int kPL>
cudaError_t backward(const BalanceGradArgs& a, cudaStream_t st) {
  const int warps = sm_count() * 64;
  const int per_warp = std::max(1, (a.tokens + warps - 1) / warps);
  const int blocks = ((a.tokens + per_warp - 1) / per_warp + 7) / 8;
  if (vectors_of_4(a.logits, a.ld, a.experts) && vectors_of_4(a.d_logits, a.ld_out, a.experts) &&
      vectors_of_4(a.slope, 0, a.experts))
    return launch_dependent(balance_grad_kernel<kPL, true>, dim3((unsigned)blocks), dim3(256), 0, st, 1, a, per_warp);
  return launch_dependent(balance_grad_kernel<kPL, false>, dim3((unsigned)blocks), dim3(256), 0, st, 1, a, per_warp);
}

}  // namespace

size_t balance_workspace(int tokens, int experts, int seqs) {
  return (size_t)(totals_at(tokens, experts, seqs, run_length(tokens)) +
                  2 * (int64_t)seqs * column_blocks(experts)) * 4;
}
int balance_launches(int tokens, int seqs, bool packed) {
  return tokens <= kSmallTokens && seqs == 1 && !packed ? 1 : 3;
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
