// The norms around a block, with its gate and residual, in one pass:
//   z    = y / rms(y) * w_post          rms(v) = sqrt(mean(v^2) + eps)
//   out  = h + scale * gate * z
//   next = out / rms(out) * w_pre       (from out before its rounding)
// and the gradients of all inputs.  With d = d(out) in full:
//   a = d_next * w_pre,  no = out / rms(out)
//   d = d_out + (a - no * mean(a * no)) / rms(out)
//   d_h = d,  d_z = scale * gate * d,  d_gate = scale * z * d (summed as gate is broadcast)
//   b = d_z * w_post,  ny = y / rms(y)
//   d_y = (b - ny * mean(b * ny)) / rms(y)
//   d_w_post = sum over rows of d_z * ny,  d_w_pre = sum over rows of d_next * no
// All sums and statistics are fp32; 1/rms of both norms is kept by the forward
// for the backward, which computes out again from h and y (the rounded out
// would put its rounding into every fp32 gradient).
//
// Bound by HBM: a CTA holds a row in registers (kV vectors of 8 values per
// thread), so every input is read once and every output written once.  The
// backward's CTAs walk over rows with the column sums of the weights'
// gradients in registers and leave one partial row each, which a second
// kernel adds in CTA order: no atomics, the same bits on every run.
#include "block_ops.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kVec = 8;

template <typename T>
__device__ __forceinline__ float up(T v);
template <>
__device__ __forceinline__ float up<float>(float v) { return v; }
template <>
__device__ __forceinline__ float up<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float up<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T down(float v);
template <>
__device__ __forceinline__ float down<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half down<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 down<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// eight values from column c of a row of `cols`; zeros behind its end.  Single
// 16-bit values are loaded plainly: __ldg of a half type is an asm statement
// that is not volatile, so the compiler may run it ahead of the test that
// guards it, with a pointer that is not valid.
template <typename T, bool kWide>
__device__ __forceinline__ void load8(const T* __restrict__ row, int c, int cols, float* v) {
  if (kWide) {   // cols is a multiple of 8
    if (c < cols) {
      constexpr int kWords = sizeof(T) / 2;
      uint4 raw[kWords];
#pragma unroll
      for (int i = 0; i < kWords; ++i) raw[i] = __ldg(reinterpret_cast<const uint4*>(row + c) + i);
      const T* e = reinterpret_cast<const T*>(raw);
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[i] = up<T>(e[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[i] = 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] = c + i < cols ? up<T>(row[c + i]) : 0.f;
  }
}
template <typename T, bool kWide>
__device__ __forceinline__ void store8(T* __restrict__ row, int c, int cols, const float* v) {
  if (kWide) {
    if (c >= cols) return;
    constexpr int kWords = sizeof(T) / 2;
    uint4 raw[kWords];
    T* e = reinterpret_cast<T*>(raw);
#pragma unroll
    for (int i = 0; i < kVec; ++i) e[i] = down<T>(v[i]);
#pragma unroll
    for (int i = 0; i < kWords; ++i) reinterpret_cast<uint4*>(row + c)[i] = raw[i];
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (c + i < cols) row[c + i] = down<T>(v[i]);
  }
}

// Sum of one (or two) values over the CTA, the same in every thread; the order
// depends on the CTA's size alone.  `s` holds 2 x 32 floats, used in turn.
struct BlockSum {
  float* s;
  int turn = 0;
  __device__ __forceinline__ float operator()(float v) {
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (warps == 1) return v;
    float* b = s + 32 * turn;
    turn ^= 1;   // the previous sum may still be read
    if (lane == 0) b[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < warps ? b[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
};

// the gate's eight values from column c
template <typename T, typename W, bool kWide>
__device__ __forceinline__ void load_gate(const NormArgs& a, int64_t row, int c, float* g) {
  if (a.gate_kind == kGateFull) {
    load8<T, kWide>(static_cast<const T*>(a.gate) + row * a.ld_gate, c, a.cols, g);
  } else if (a.gate_kind == kGateFeature) {
    load8<W, kWide>(static_cast<const W*>(a.gate), c, a.cols, g);
  } else {
    float v = 1.f;
    if (a.gate_kind == kGateToken) v = up<T>(static_cast<const T*>(a.gate)[row * a.ld_gate]);
#pragma unroll
    for (int i = 0; i < kVec; ++i) g[i] = v;
  }
}

template <typename T, typename W, int kV, bool kWide>
__global__ void __launch_bounds__(kV == 1 ? 1024 : 512) norm_kernel(const NormArgs a) {
  __shared__ float s_sum[64];
  BlockSum sum{s_sum};
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const float inv = 1.f / (float)a.cols;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    float o[kV][kVec];
#pragma unroll
    for (int k = 0; k < kV; ++k)
      load8<T, kWide>(static_cast<const T*>(a.h) + row * a.ld_h, (threadIdx.x + k * blockDim.x) * kVec, a.cols, o[k]);
    if (a.has_post) {
      float y[kV][kVec], q = 0.f;
#pragma unroll
      for (int k = 0; k < kV; ++k) {
        load8<T, kWide>(static_cast<const T*>(a.y) + row * a.ld_y, (threadIdx.x + k * blockDim.x) * kVec, a.cols, y[k]);
#pragma unroll
        for (int i = 0; i < kVec; ++i) q = fmaf(y[k][i], y[k][i], q);
      }
      const float r = rsqrtf(sum(q) * inv + a.eps);
      if (threadIdx.x == 0 && a.stats) a.stats[2 * row] = r;
#pragma unroll
      for (int k = 0; k < kV; ++k) {
        const int c = (threadIdx.x + k * blockDim.x) * kVec;
        float w[kVec], g[kVec];
        load8<W, kWide>(static_cast<const W*>(a.post), c, a.cols, w);
        load_gate<T, W, kWide>(a, row, c, g);
#pragma unroll
        for (int i = 0; i < kVec; ++i) o[k][i] = fmaf(a.scale * g[i], y[k][i] * r * w[i], o[k][i]);
        store8<T, kWide>(static_cast<T*>(a.out) + row * a.ld_out, c, a.cols, o[k]);
      }
    }
    if (a.pre) {
      float q = 0.f;
#pragma unroll
      for (int k = 0; k < kV; ++k)
#pragma unroll
        for (int i = 0; i < kVec; ++i) q = fmaf(o[k][i], o[k][i], q);
      const float r = rsqrtf(sum(q) * inv + a.eps);
      if (threadIdx.x == 0 && a.stats) a.stats[2 * row + 1] = r;
#pragma unroll
      for (int k = 0; k < kV; ++k) {
        const int c = (threadIdx.x + k * blockDim.x) * kVec;
        float w[kVec];
        load8<W, kWide>(static_cast<const W*>(a.pre), c, a.cols, w);
#pragma unroll
        for (int i = 0; i < kVec; ++i) w[i] *= o[k][i] * r;
        store8<T, kWide>(static_cast<T*>(a.next) + row * a.ld_next, c, a.cols, w);
      }
    }
  }
}

// Column sums: [CTA][which][cols], which = d_post, d_pre, d_gate (as wanted).
template <typename T, typename W, int kV, bool kWide>
__global__ void __launch_bounds__(512) norm_grad_kernel(const NormGradArgs a) {
  __shared__ float s_sum[64];
  BlockSum sum{s_sum};
  const NormArgs& f = a.f;
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const float inv = 1.f / (float)f.cols;
  float s_post[kV][kVec] = {}, s_pre[kV][kVec] = {}, s_gate[kV][kVec] = {};
  for (int64_t row = blockIdx.x; row < f.rows; row += gridDim.x) {
    const float ry = f.has_post ? f.stats[2 * row] : 0.f, ro = f.pre ? f.stats[2 * row + 1] : 0.f;
    float o[kV][kVec], y[kV][kVec], d[kV][kVec];   // o: out, later scale * gate
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      const int c = (threadIdx.x + k * blockDim.x) * kVec;
      load8<T, kWide>(static_cast<const T*>(f.h) + row * f.ld_h, c, f.cols, o[k]);
      if (f.has_post) {
        float w[kVec], g[kVec];
        load8<T, kWide>(static_cast<const T*>(f.y) + row * f.ld_y, c, f.cols, y[k]);
        load8<W, kWide>(static_cast<const W*>(f.post), c, f.cols, w);
        load_gate<T, W, kWide>(f, row, c, g);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          y[k][i] *= ry;
          o[k][i] = fmaf(f.scale * g[i], y[k][i] * w[i], o[k][i]);
        }
      }
      if (a.d_out) {
        load8<T, kWide>(static_cast<const T*>(a.d_out) + row * a.ld_d_out, c, f.cols, d[k]);
      } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) d[k][i] = 0.f;
      }
    }
    if (f.pre) {
      float e[kV][kVec], q = 0.f;
#pragma unroll
      for (int k = 0; k < kV; ++k) {
        const int c = (threadIdx.x + k * blockDim.x) * kVec;
        float w[kVec];
        load8<T, kWide>(static_cast<const T*>(a.d_next) + row * a.ld_d_next, c, f.cols, e[k]);
        load8<W, kWide>(static_cast<const W*>(f.pre), c, f.cols, w);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          o[k][i] *= ro;
          s_pre[k][i] = fmaf(e[k][i], o[k][i], s_pre[k][i]);
          e[k][i] *= w[i];
          q = fmaf(e[k][i], o[k][i], q);
        }
      }
      const float m = sum(q) * inv;
#pragma unroll
      for (int k = 0; k < kV; ++k)
#pragma unroll
        for (int i = 0; i < kVec; ++i) d[k][i] = fmaf(ro, fmaf(-o[k][i], m, e[k][i]), d[k][i]);
    }
#pragma unroll
    for (int k = 0; k < kV; ++k)
      store8<T, kWide>(static_cast<T*>(a.d_h) + row * a.ld_d_h, (threadIdx.x + k * blockDim.x) * kVec, f.cols, d[k]);
    if (f.has_post) {
      float q = 0.f, dg = 0.f;
#pragma unroll
      for (int k = 0; k < kV; ++k) {
        const int c = (threadIdx.x + k * blockDim.x) * kVec;
        float w[kVec], g[kVec];
        load8<W, kWide>(static_cast<const W*>(f.post), c, f.cols, w);
        load_gate<T, W, kWide>(f, row, c, g);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const float sd = f.scale * d[k][i], zn = y[k][i] * w[i];
          if (f.gate_kind == kGateToken) dg = fmaf(sd, zn, dg);
          if (f.gate_kind == kGateFeature) s_gate[k][i] = fmaf(sd, zn, s_gate[k][i]);
          const float dz = sd * g[i];
          g[i] = sd * zn;
          s_post[k][i] = fmaf(dz, y[k][i], s_post[k][i]);
          d[k][i] = dz * w[i];
          q = fmaf(d[k][i], y[k][i], q);
        }
        if (f.gate_kind == kGateFull) store8<T, kWide>(static_cast<T*>(a.d_gate) + row * a.ld_d_gate, c, f.cols, g);
      }
      if (f.gate_kind == kGateToken) {
        dg = sum(dg);
        if (threadIdx.x == 0) static_cast<T*>(a.d_gate)[row * a.ld_d_gate] = down<T>(dg);
      }
      const float m = sum(q) * inv;
#pragma unroll
      for (int k = 0; k < kV; ++k) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) d[k][i] = ry * fmaf(-y[k][i], m, d[k][i]);
        store8<T, kWide>(static_cast<T*>(a.d_y) + row * a.ld_d_y, (threadIdx.x + k * blockDim.x) * kVec, f.cols, d[k]);
      }
    }
  }
  const int64_t padded = (f.cols + 7) / 8 * 8;
  float* part = a.partial + (int64_t)blockIdx.x * a.n_sums * padded;
#pragma unroll
  for (int k = 0; k < kV; ++k) {
    const int c = (threadIdx.x + k * blockDim.x) * kVec;
    if (c >= f.cols) continue;
    float* p = part + c;
    if (f.has_post) {
      store8<float, true>(p, 0, kVec, s_post[k]);
      p += padded;
    }
    if (f.pre) {
      store8<float, true>(p, 0, kVec, s_pre[k]);
      p += padded;
    }
    if (f.has_post && f.gate_kind == kGateFeature) store8<float, true>(p, 0, kVec, s_gate[k]);
  }
}

// The CTAs' partial rows added in order, one warp row of 32 columns per warp
// and eight rows at a time.
template <typename W>
__global__ void __launch_bounds__(256) norm_sums_kernel(const float* __restrict__ partial, int n_parts, int n_sums,
                                                        int cols, W* o0, W* o1, W* o2) {
  __shared__ float s[8][33];
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int padded = (cols + 7) / 8 * 8;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane, which = blockIdx.y;
  float v = 0.f;
  if (c < cols)
    for (int p = warp; p < n_parts; p += 8) v += __ldcg(partial + ((int64_t)p * n_sums + which) * padded + c);
  s[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < cols) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += s[i][lane];
    W* o = which == 0 ? o0 : which == 1 ? o1 : o2;
    o[c] = down<W>(t);
  }
}

// Threads of a CTA for rows of `cols` with v vectors per thread.
int threads_for(int cols, int v) { return std::max(32, ((cols + kVec - 1) / kVec + v * 32 - 1) / (v * 32) * 32); }

template <typename T, typename W, bool kWide>
cudaError_t forward(const NormArgs& a, cudaStream_t st) {
  // one vector per thread up to 8192 columns while the rows do not fill the GPU (latency), else more per thread
  const int vecs = (a.cols + kVec - 1) / kVec;
  int v = vecs <= 1024 && a.rows <= sm_count() ? 1 : vecs <= 128 ? 1 : vecs <= 512 ? 2 : 4;
  const int threads = threads_for(a.cols, v);
  const unsigned grid = (unsigned)std::min<int64_t>(a.rows, 1 << 20);
  if (v == 1) return launch_dependent(norm_kernel<T, W, 1, kWide>, dim3(grid), dim3(threads), 0, st, 1, a);
  if (v == 2) return launch_dependent(norm_kernel<T, W, 2, kWide>, dim3(grid), dim3(threads), 0, st, 1, a);
  return launch_dependent(norm_kernel<T, W, 4, kWide>, dim3(grid), dim3(threads), 0, st, 1, a);
}

template <typename T, typename W, bool kWide>
cudaError_t backward(const NormGradArgs& a, cudaStream_t st) {
  const int vecs = (a.f.cols + kVec - 1) / kVec;
  const int v = vecs <= 512 ? 1 : vecs <= 1024 ? 2 : 4;
  const int threads = threads_for(a.f.cols, v);
  const unsigned grid = (unsigned)a.n_parts;
  cudaError_t e;
  if (v == 1) e = launch_dependent(norm_grad_kernel<T, W, 1, kWide>, dim3(grid), dim3(threads), 0, st, 1, a);
  else if (v == 2) e = launch_dependent(norm_grad_kernel<T, W, 2, kWide>, dim3(grid), dim3(threads), 0, st, 1, a);
  else e = launch_dependent(norm_grad_kernel<T, W, 4, kWide>, dim3(grid), dim3(threads), 0, st, 1, a);
  if (e != cudaSuccess) return e;
  W* o[3];
  int n = 0;
  if (a.f.has_post) o[n++] = static_cast<W*>(a.d_post);
  if (a.f.pre) o[n++] = static_cast<W*>(a.d_pre);
  if (a.f.has_post && a.f.gate_kind == kGateFeature) o[n++] = static_cast<W*>(a.d_gate);
  for (int i = n; i < 3; ++i) o[i] = nullptr;
  return launch_dependent(norm_sums_kernel<W>, dim3((a.f.cols + 31) / 32, n), dim3(256), 0, st, 1, a.partial,
                          a.n_parts, a.n_sums, a.f.cols, o[0], o[1], o[2]);
}

// f<T, W, wide>(...) for the argument types
#define NORM_DISPATCH(f, type, weight_type, wide, ...)                                                  \
  if (type == kF32) return wide ? f<float, float, true>(__VA_ARGS__) : f<float, float, false>(__VA_ARGS__); \
  if (type == kF16 && weight_type == kF16)                                                               \
    return wide ? f<__half, __half, true>(__VA_ARGS__) : f<__half, __half, false>(__VA_ARGS__);           \
  if (type == kF16)                                                                                      \
    return wide ? f<__half, float, true>(__VA_ARGS__) : f<__half, float, false>(__VA_ARGS__);             \
  if (weight_type == kBF16)                                                                              \
    return wide ? f<__nv_bfloat16, __nv_bfloat16, true>(__VA_ARGS__)                                     \
                : f<__nv_bfloat16, __nv_bfloat16, false>(__VA_ARGS__);                                   \
  return wide ? f<__nv_bfloat16, float, true>(__VA_ARGS__) : f<__nv_bfloat16, float, false>(__VA_ARGS__);

}  // namespace

int norm_grad_parts(int rows, int cols) {
  // CTAs of at most 512 threads, three to an SM
  return std::max(1, std::min(rows, 3 * sm_count()));
}

cudaError_t launch_norm(const NormArgs& a, cudaStream_t st) {
  NORM_DISPATCH(forward, a.type, a.weight_type, a.wide, a, st)
}
cudaError_t launch_norm_grad(const NormGradArgs& a, cudaStream_t st) {
  NORM_DISPATCH(backward, a.f.type, a.f.weight_type, a.f.wide, a, st)
}

}  // namespace moe
