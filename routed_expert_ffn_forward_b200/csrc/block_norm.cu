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
// Bound by HBM: every input is read once and every output written once, a row
// being held in registers between its two statistics.  Rows in number go
// through persistent CTAs (rows_kernel): one thread brings the rows ahead into
// a ring in shared memory with bulk copies, and the weights stay in shared
// memory, since reading 4-byte weights again for every 2-byte row costs more
// L2 traffic than the row.  Few rows, and rows too long for that, take one CTA
// per row (norm_kernel, norm_grad_kernel).  The backward keeps the column sums
// of the weights' gradients in registers and leaves one partial row per CTA,
// which a second kernel adds in a fixed order: no atomics, the same bits on
// every run.
#include "block_ops.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kVec = 8;

// Eight values as four pairs: products and sums run two to an instruction
// (the rows are bound by instruction issue otherwise: 450 a warp and row before,
// 72 us for 4096 x 7168).
struct V8 {
  float2 p[4];
  __device__ __forceinline__ float get(int i) const { return i & 1 ? p[i >> 1].y : p[i >> 1].x; }
  __device__ __forceinline__ void set(int i, float v) { (i & 1 ? p[i >> 1].y : p[i >> 1].x) = v; }
};
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ V8 all8(float v) { return {{both(v), both(v), both(v), both(v)}}; }
__device__ __forceinline__ V8 operator*(const V8& a, const V8& b) {
  V8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.p[i] = __fmul2_rn(a.p[i], b.p[i]);
  return r;
}
__device__ __forceinline__ V8 operator*(const V8& a, float s) {
  V8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.p[i] = __fmul2_rn(a.p[i], both(s));
  return r;
}
// a * b + c
__device__ __forceinline__ V8 fma8(const V8& a, const V8& b, const V8& c) {
  V8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.p[i] = __ffma2_rn(a.p[i], b.p[i], c.p[i]);
  return r;
}
__device__ __forceinline__ V8 fma8(const V8& a, float s, const V8& c) {
  V8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.p[i] = __ffma2_rn(a.p[i], both(s), c.p[i]);
  return r;
}
// q += a . b, over the pairs
__device__ __forceinline__ void dot8(const V8& a, const V8& b, float2& q) {
#pragma unroll
  for (int i = 0; i < 4; ++i) q = __ffma2_rn(a.p[i], b.p[i], q);
}

__device__ __forceinline__ float up(float v) { return v; }
__device__ __forceinline__ float up(__half v) { return __half2float(v); }
__device__ __forceinline__ float up(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T down(float v);
template <>
__device__ __forceinline__ float down<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half down<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 down<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// eight values of T in 16-byte words
template <typename T>
struct Packed;
template <>
struct Packed<float> {
  static constexpr int kWords = 2;
  static __device__ __forceinline__ V8 unpack(const uint4* w) {
    const float4* f = reinterpret_cast<const float4*>(w);
    return {{make_float2(f[0].x, f[0].y), make_float2(f[0].z, f[0].w), make_float2(f[1].x, f[1].y),
             make_float2(f[1].z, f[1].w)}};
  }
  using Pair = float2;
  static __device__ __forceinline__ float2 unpack2(float2 w) { return w; }
  static __device__ __forceinline__ float2 pack2(float2 v) { return v; }
  static __device__ __forceinline__ void pack(const V8& v, uint4* w) {
    float4* f = reinterpret_cast<float4*>(w);
    f[0] = make_float4(v.p[0].x, v.p[0].y, v.p[1].x, v.p[1].y);
    f[1] = make_float4(v.p[2].x, v.p[2].y, v.p[3].x, v.p[3].y);
  }
};
template <>
struct Packed<__half> {
  static constexpr int kWords = 1;
  static __device__ __forceinline__ V8 unpack(const uint4* w) {
    const __half2* h = reinterpret_cast<const __half2*>(w);
    return {{__half22float2(h[0]), __half22float2(h[1]), __half22float2(h[2]), __half22float2(h[3])}};
  }
  using Pair = __half2;
  static __device__ __forceinline__ float2 unpack2(__half2 w) { return __half22float2(w); }
  static __device__ __forceinline__ __half2 pack2(float2 v) { return __float22half2_rn(v); }
  static __device__ __forceinline__ void pack(const V8& v, uint4* w) {
    __half2* h = reinterpret_cast<__half2*>(w);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __float22half2_rn(v.p[i]);
  }
};
template <>
struct Packed<__nv_bfloat16> {
  static constexpr int kWords = 1;
  static __device__ __forceinline__ float2 two(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
  static __device__ __forceinline__ V8 unpack(const uint4* w) { return {{two(w->x), two(w->y), two(w->z), two(w->w)}}; }
  using Pair = __nv_bfloat162;
  static __device__ __forceinline__ float2 unpack2(__nv_bfloat162 w) { return two(*reinterpret_cast<const uint32_t*>(&w)); }
  static __device__ __forceinline__ __nv_bfloat162 pack2(float2 v) { return __float22bfloat162_rn(v); }
  static __device__ __forceinline__ void pack(const V8& v, uint4* w) {
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(w);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __float22bfloat162_rn(v.p[i]);
  }
};

// How rows are accessed.  kAligned: cols and row strides multiples of 8, bases
// aligned to 16 bytes.  kShifted: rows at any offset, read from a copy in
// shared memory at the same offset from a 16-byte boundary and stored in whole
// 16-byte words, both by shifting across word borders.  kPairs: cols and row
// strides even, bases aligned to two values, accesses of two.  kStrided: of one.
enum Access { kStrided, kPairs, kAligned, kShifted };

// The eight columns of vector k of this thread: consecutive ones, or with
// kPairs and kStrided every threads-th pair or value, so that a warp's accesses
// stay side by side.
template <Access kA>
__device__ __forceinline__ int column(int tid, int threads, int k, int i) {
  return kA == kStrided ? tid + (k * kVec + i) * threads
         : kA == kPairs ? 2 * (tid + (k * (kVec / 2) + i / 2) * threads) + i % 2
                        : (tid + k * threads) * kVec + i;
}
// A row's columns, the threads that share them and this one's number among them.
struct Span {
  int cols, threads, tid;
};
// Vector k of a row; zeros behind its end.  Single 16-bit values are loaded
// plainly: __ldg of a half type is an asm statement that is not volatile, so
// the compiler may run it ahead of the test that guards it, with a pointer
// that is not valid.
template <typename T, Access kA, bool kShared>
__device__ __forceinline__ V8 load8(const T* row, int k, const Span& sp) {
  V8 v = all8(0.f);
  constexpr int kWords = Packed<T>::kWords;
  if (kA == kStrided) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int c = column<kStrided>(sp.tid, sp.threads, k, i);
      if (c < sp.cols) v.set(i, up(row[c]));
    }
    return v;
  }
  if (kA == kPairs) {
#pragma unroll
    for (int i = 0; i < kVec / 2; ++i) {
      const int c = column<kPairs>(sp.tid, sp.threads, k, 2 * i);
      if (c < sp.cols) v.p[i] = Packed<T>::unpack2(*reinterpret_cast<const typename Packed<T>::Pair*>(row + c));
    }
    return v;
  }
  const int c = column<kAligned>(sp.tid, sp.threads, k, 0);
  if (c >= sp.cols) return v;
  if (kA == kAligned) {
    uint4 raw[kWords];
    const uint4* p = reinterpret_cast<const uint4*>(row + c);
#pragma unroll
    for (int i = 0; i < kWords; ++i) raw[i] = kShared ? p[i] : __ldg(p + i);
    return Packed<T>::unpack(raw);
  }
  // shared memory: the words that hold the vector and one more
  const uint32_t shift = (uint32_t)reinterpret_cast<uintptr_t>(row) & 15u;
  const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(row + c) - shift);
  uint4 raw[kWords + 1], out[kWords];
#pragma unroll
  for (int i = 0; i < kWords + 1; ++i) raw[i] = p[i];
  shifted_words<4 * kWords>(reinterpret_cast<const uint32_t*>(raw), shift, reinterpret_cast<uint32_t*>(out));
  v = Packed<T>::unpack(out);
  if (c + kVec > sp.cols) {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (c + i >= sp.cols) v.set(i, 0.f);
  }
  return v;
}
template <typename T, Access kA>
__device__ __forceinline__ void store8(T* row, int k, const Span& sp, const V8& v) {
  constexpr int kWords = Packed<T>::kWords;
  if (kA == kStrided) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int c = column<kStrided>(sp.tid, sp.threads, k, i);
      if (c < sp.cols) row[c] = down<T>(v.get(i));
    }
    return;
  }
  if (kA == kPairs) {
#pragma unroll
    for (int i = 0; i < kVec / 2; ++i) {
      const int c = column<kPairs>(sp.tid, sp.threads, k, 2 * i);
      if (c < sp.cols) *reinterpret_cast<typename Packed<T>::Pair*>(row + c) = Packed<T>::pack2(v.p[i]);
    }
    return;
  }
  const int c = column<kAligned>(sp.tid, sp.threads, k, 0);
  if (kA == kAligned) {
    if (c >= sp.cols) return;
    uint4 raw[kWords];
    Packed<T>::pack(v, raw);
#pragma unroll
    for (int i = 0; i < kWords; ++i) reinterpret_cast<uint4*>(row + c)[i] = raw[i];
    return;
  }
  // The whole warp: a lane stores the 16-byte words that end in its vector, with
  // the last bytes of the lane before; what no lane can store whole (a warp's
  // first and last bytes, a row's last vector) goes value by value.
  const int lane = threadIdx.x & 31;
  uint4 raw[kWords + 1], out[kWords];   // the previous lane's last word, then this vector
  Packed<T>::pack(v, raw + 1);
  const uint32_t* last = reinterpret_cast<const uint32_t*>(raw + kWords);
  uint32_t* before = reinterpret_cast<uint32_t*>(raw);
#pragma unroll
  for (int i = 0; i < 4; ++i) before[i] = __shfl_up_sync(0xffffffffu, last[i], 1);
  if (c >= sp.cols) return;
  const uint32_t shift = (uint32_t)reinterpret_cast<uintptr_t>(row) & 15u;
  const bool full = c + kVec <= sp.cols, next = lane < 31 && c + 2 * kVec <= sp.cols;
  uint4* q = reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(row + c) - shift);
  if (shift == 0) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) out[i] = raw[1 + i];
  } else {
    shifted_words<4 * kWords>(reinterpret_cast<const uint32_t*>(raw), 16 - shift, reinterpret_cast<uint32_t*>(out));
  }
  const bool merge = full && (lane > 0 || shift == 0);   // the first word is whole
#pragma unroll
  for (int i = 0; i < kWords; ++i)
    if (full && (i > 0 || merge)) q[i] = out[i];
  const int head = shift ? (16 - (int)shift) / (int)sizeof(T) : kVec, tail = kVec - (int)shift / (int)sizeof(T);
  if (!merge || !next) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const bool mine = full ? (!merge && i < head) || (!next && i >= tail) : c + i < sp.cols;
      if (mine) row[c + i] = down<T>(v.get(i));
    }
  }
}

// Sums over a team's threads, the same in every one; the order depends on the
// team's size alone.  `s` holds 2 x 32 pairs, used in turn.
struct BlockSum {
  float2* s;
  int threads, tid, barrier;   // a team of the CTA: its size, this thread's number in it, its barrier
  int turn = 0;
  __device__ __forceinline__ void sync() const { ptx::named_barrier_sync(barrier, threads); }
  __device__ __forceinline__ float2 operator()(float2 v) {
    const int warps = threads >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
      v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    if (warps == 1) return v;
    float2* b = s + 32 * turn;
    turn ^= 1;   // the previous sum may still be read
    if (lane == 0) b[tid >> 5] = v;
    sync();
    v = lane < warps ? b[lane] : make_float2(0.f, 0.f);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
      v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    return v;
  }
  __device__ __forceinline__ float operator()(float v) {
    const int warps = threads >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (warps == 1) return v;
    float* b = reinterpret_cast<float*>(s + 32 * turn);
    turn ^= 1;
    if (lane == 0) b[tid >> 5] = v;
    sync();
    v = lane < warps ? b[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
};

// Where one row's inputs are: global memory, or a stage of the ring.
template <typename T>
struct Row {
  const T *h, *y, *gate, *d_out, *d_next;
};
// The weights: global memory or the CTA's copy in shared memory.
template <typename W>
struct Weights {
  const W *post, *gate, *pre;
};

// v times scale and the gate
// Weights in shared memory are aligned where the rows are shifted.
template <typename W, Access kA, bool kShared>
__device__ __forceinline__ V8 weight8(const W* w, int k, const Span& sp) {
  return load8<W, kA == kShifted ? kAligned : kA, kShared>(w, k, sp);
}
template <typename T, typename W, Access kA, bool kShared>
__device__ __forceinline__ V8 gated(const NormArgs& a, const V8& v, float scale, const Row<T>& r, const Weights<W>& w, int k,
                                    const Span& sp) {
  if (a.gate_kind == kGateFull) return v * (load8<T, kA, kShared>(r.gate, k, sp) * scale);
  if (a.gate_kind == kGateFeature) return v * (weight8<W, kA, kShared>(w.gate, k, sp) * scale);
  return v * scale;
}
// scale, times a token's gate
template <typename T>
__device__ __forceinline__ float token_scale(const NormArgs& a, const Row<T>& r) {
  float s = a.scale;
  if (a.gate_kind == kGateToken) s *= up(*r.gate);
  return s;
}

// One row forward.  `read` is called by every thread once it has read the row.
template <typename T, typename W, int kV, Access kA, bool kShared, typename Read>
__device__ __forceinline__ void row_forward(const NormArgs& a, int64_t row, const Row<T>& in, const Weights<W>& wt,
                                            BlockSum& sum, Read read) {
  const float inv = 1.f / (float)a.cols;
  const Span sp = {a.cols, sum.threads, sum.tid};
  V8 o[kV];
  if (a.has_post) {
    V8 y[kV];
    float2 q = both(0.f);
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      y[k] = load8<T, kA, kShared>(in.y, k, sp);
      dot8(y[k], y[k], q);
    }
    const float sg = token_scale(a, in);
    const float r = rsqrtf(sum(q.x + q.y) * inv + a.eps);
    if (sp.tid == 0 && a.stats) a.stats[2 * row] = r;
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      const V8 z = y[k] * weight8<W, kA, kShared>(wt.post, k, sp);
      o[k] = fma8(gated<T, W, kA, kShared>(a, z, sg, in, wt, k, sp), r, load8<T, kA, kShared>(in.h, k, sp));
      store8<T, kA>(static_cast<T*>(a.out) + row * a.ld_out, k, sp, o[k]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < kV; ++k) o[k] = load8<T, kA, kShared>(in.h, k, sp);
  }
  read();
  if (a.pre) {
    float2 q = both(0.f);
#pragma unroll
    for (int k = 0; k < kV; ++k) dot8(o[k], o[k], q);
    const float r = rsqrtf(sum(q.x + q.y) * inv + a.eps);
    if (sp.tid == 0 && a.stats) a.stats[2 * row + 1] = r;
#pragma unroll
    for (int k = 0; k < kV; ++k)
      store8<T, kA>(static_cast<T*>(a.next) + row * a.ld_next, k, sp,
                       o[k] * r * weight8<W, kA, kShared>(wt.pre, k, sp));
  }
}

// Sums over the rows of a thread's columns: scale * d * ny, times the gate if it
// differs from row to row, which gives d_post and a feature gate's gradient
// (both are it times the other's weight), and d_pre.
template <int kV>
struct ColumnSums {
  V8 post[kV], pre[kV];
};

// One row backward; `read` as above.
template <typename T, typename W, int kV, Access kA, bool kShared, typename Read>
__device__ __forceinline__ void row_backward(const NormGradArgs& a, int64_t row, float2 stats, const Row<T>& in,
                                             const Weights<W>& wt, BlockSum& sum, ColumnSums<kV>& s, Read read) {
  const NormArgs& f = a.f;
  const float inv = 1.f / (float)f.cols, ry = stats.x, ro = stats.y;
  const Span sp = {f.cols, sum.threads, sum.tid};
  const float sg = f.has_post ? token_scale(f, in) : 0.f;
  V8 y[kV], d[kV];   // y: y / rms(y); d: the gradient of out
  if (f.pre) {
    V8 o[kV], e[kV];   // out / rms(out), d_next * pre
    float2 q = both(0.f);
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      o[k] = load8<T, kA, kShared>(in.h, k, sp);
      if (f.has_post) {
        y[k] = load8<T, kA, kShared>(in.y, k, sp) * ry;
        const V8 z = y[k] * weight8<W, kA, kShared>(wt.post, k, sp);
        o[k] = fma8(gated<T, W, kA, kShared>(f, z, sg, in, wt, k, sp), 1.f, o[k]);
      }
      o[k] = o[k] * ro;
      e[k] = load8<T, kA, kShared>(in.d_next, k, sp);
      s.pre[k] = fma8(e[k], o[k], s.pre[k]);
      e[k] = e[k] * weight8<W, kA, kShared>(wt.pre, k, sp);
      dot8(e[k], o[k], q);
    }
    const float m = sum(q.x + q.y) * inv;
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      d[k] = a.d_out ? load8<T, kA, kShared>(in.d_out, k, sp) : all8(0.f);
      d[k] = fma8(e[k], ro, fma8(o[k], -ro * m, d[k]));
    }
  } else {
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      y[k] = load8<T, kA, kShared>(in.y, k, sp) * ry;
      d[k] = a.d_out ? load8<T, kA, kShared>(in.d_out, k, sp) : all8(0.f);
    }
  }
#pragma unroll
  for (int k = 0; k < kV; ++k) store8<T, kA>(static_cast<T*>(a.d_h) + row * a.ld_d_h, k, sp, d[k]);
  if (f.has_post) {
    const bool token = f.gate_kind == kGateToken, full = f.gate_kind == kGateFull;
    float2 q = both(0.f), qg = both(0.f);   // b . ny, and a token's gate gradient
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      const V8 w = weight8<W, kA, kShared>(wt.post, k, sp);
      const V8 dz = gated<T, W, kA, kShared>(f, d[k], sg, in, wt, k, sp);
      if (token) dot8(d[k], y[k] * w, qg);
      if (full)
        store8<T, kA>(static_cast<T*>(a.d_gate) + row * a.ld_d_gate, k, sp, d[k] * (y[k] * w) * f.scale);
      s.post[k] = fma8(token || full ? dz : d[k] * f.scale, y[k], s.post[k]);
      d[k] = dz * w;
      dot8(d[k], y[k], q);
    }
    read();
    float m;
    if (token) {
      const float2 t = sum(make_float2(q.x + q.y, qg.x + qg.y));
      m = t.x;
      if (sp.tid == 0) static_cast<T*>(a.d_gate)[row * a.ld_d_gate] = down<T>(t.y * f.scale);
    } else {
      m = sum(q.x + q.y);
    }
    m *= inv;
#pragma unroll
    for (int k = 0; k < kV; ++k)
      store8<T, kA>(static_cast<T*>(a.d_y) + row * a.ld_d_y, k, sp, fma8(d[k], ry, y[k] * (-ry * m)));
  } else {
    read();
  }
}

// The CTA's partial row: [which][cols to 8], which = d_post, d_pre, d_gate (as wanted).
template <typename W, int kV, Access kA, bool kShared>
__device__ __forceinline__ void store_sums(const NormGradArgs& a, const Weights<W>& wt, const ColumnSums<kV>& s,
                                           int threads) {
  constexpr Access kSumAccess = kA == kShifted ? kAligned : kA;   // the partial rows are padded to whole vectors
  const Span sp = {a.f.cols, threads, (int)threadIdx.x};
  const int64_t padded = (sp.cols + 7) / 8 * 8;
  float* p = a.partial + (int64_t)blockIdx.x * a.n_sums * padded;
#pragma unroll
  for (int k = 0; k < kV; ++k) {
    float* q = p;
    if (a.f.has_post) {
      V8 post = s.post[k];
      if (a.f.gate_kind == kGateFeature) {
        store8<float, kSumAccess>(q + (a.f.pre ? 2 : 1) * padded, k, sp, post * weight8<W, kA, kShared>(wt.post, k, sp));
        post = post * weight8<W, kA, kShared>(wt.gate, k, sp);
      }
      store8<float, kSumAccess>(q, k, sp, post);
      q += padded;
    }
    if (a.f.pre) store8<float, kSumAccess>(q, k, sp, s.pre[k]);
  }
}

template <int kV>
__device__ __forceinline__ void clear(ColumnSums<kV>& s) {
#pragma unroll
  for (int k = 0; k < kV; ++k) s.post[k] = s.pre[k] = all8(0.f);
}
// 1/rms of y and out, as the forward left them
__device__ __forceinline__ float2 stats_of(const NormArgs& a, int64_t row) {
  return make_float2(a.has_post ? a.stats[2 * row] : 0.f, a.pre ? a.stats[2 * row + 1] : 0.f);
}

template <typename T, typename W>
__device__ __forceinline__ Weights<W> global_weights(const NormArgs& a) {
  return {static_cast<const W*>(a.post), static_cast<const W*>(a.gate), static_cast<const W*>(a.pre)};
}
template <typename T>
__device__ __forceinline__ Row<T> global_row(const NormArgs& a, int64_t row) {
  return {static_cast<const T*>(a.h) + row * a.ld_h, static_cast<const T*>(a.y) + row * a.ld_y,
          static_cast<const T*>(a.gate) + row * a.ld_gate, nullptr, nullptr};
}

// One CTA per row, everything from global memory.
template <typename T, typename W, int kV, Access kA>
__global__ void __launch_bounds__(kV == 1 ? 1024 : 512) norm_kernel(const NormArgs a) {
  __shared__ float2 s_sum[64];
  BlockSum sum{s_sum, (int)blockDim.x, (int)threadIdx.x, 1};
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x)
    row_forward<T, W, kV, kA, false>(a, row, global_row<T>(a, row), global_weights<T, W>(a), sum, [] {});
}
template <typename T, typename W, int kV, Access kA>
__global__ void __launch_bounds__(512) norm_grad_kernel(const NormGradArgs a) {
  __shared__ float2 s_sum[64];
  BlockSum sum{s_sum, (int)blockDim.x, (int)threadIdx.x, 1};
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  ColumnSums<kV> s;
  clear(s);
  for (int64_t row = blockIdx.x; row < a.f.rows; row += gridDim.x) {
    Row<T> in = global_row<T>(a.f, row);
    in.d_out = static_cast<const T*>(a.d_out) + row * a.ld_d_out;
    in.d_next = static_cast<const T*>(a.d_next) + row * a.ld_d_next;
    row_backward<T, W, kV, kA, false>(a, row, stats_of(a.f, row), in, global_weights<T, W>(a.f), sum, s, [] {});
  }
  store_sums<W, kV, kA, false>(a, global_weights<T, W>(a.f), s, blockDim.x);
}

// ---- persistent CTAs over a ring of rows -------------------------------------
// bit flags: a bounded wait that gave up
__device__ unsigned g_norm_err = 0;

// The most dynamic shared memory of a ring (ring_shape).  Every launch allows its
// kernel this much: the limit belongs to the kernel, not to the launch, and one
// that followed a call's own size could shrink below another thread's launch.
constexpr int kRingSmem = 220 * 1024 - 2048;

struct Ring {
  int teams;                  // of threads in a CTA, each with rows and stages of its own
  int stages, inputs, slot;   // stages (of all teams) of so many input rows of `slot` bytes
  int weights, weight;        // weight vectors and the bytes of one
  int ctas;                   // per SM
  size_t smem() const { return (size_t)weights * weight + (size_t)stages * inputs * slot; }
};

// kGrad: backward.  A stage holds the row's inputs h, y, full gate, d_out and
// d_next, each brought by one bulk copy of the 16-byte granules that hold it (a
// granule lies in one page, so that its bytes beside the row can be read, and
// they are not used).  The last warp issues the copies: in a computing thread
// they would hold up every barrier of the row (2.1 us a row against 1.3).
template <typename T, typename W, int kV, Access kA, bool kGrad, int kTeams>
__global__ void __launch_bounds__(kGrad ? 512 : 1024, 1) rows_kernel(const NormGradArgs a, const Ring ring) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float2 s_sum[2][64];
  __shared__ uint64_t s_full[8], s_empty[8];
  const NormArgs& f = a.f;
  const int threads = (blockDim.x - 32) / kTeams, stages = ring.stages / kTeams;
  W* s_w = reinterpret_cast<W*>(smem);
  uint8_t* s_rows = smem + ring.weights * ring.weight;
  const T* src[5] = {static_cast<const T*>(f.h), static_cast<const T*>(f.y),
                     f.gate_kind == kGateFull ? static_cast<const T*>(f.gate) : nullptr,
                     kGrad ? static_cast<const T*>(a.d_out) : nullptr, kGrad ? static_cast<const T*>(a.d_next) : nullptr};
  const int64_t ld[5] = {f.ld_h, f.ld_y, f.ld_gate, a.ld_d_out, a.ld_d_next};
  int place[5];   // the input's slot in a stage
  place[0] = 0;
#pragma unroll
  for (int i = 1; i < 5; ++i) place[i] = place[i - 1] + (src[i - 1] ? 1 : 0);
  if (threadIdx.x == 0) {
    for (int i = 0; i < ring.stages; ++i) {
      ptx::mbar_init(&s_full[i], 1);
      ptx::mbar_init(&s_empty[i], threads / 32);
    }
    ptx::fence_barrier_init();
  }
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  __syncthreads();
  // the last warp's lanes copy for one team each
  const bool copies = threadIdx.x >= threads * kTeams;
  const int lane = threadIdx.x & 31, team = kTeams == 1 ? 0 : copies ? lane & (kTeams - 1) : threadIdx.x / threads;
  const int64_t first = (int64_t)blockIdx.x * kTeams + team, step = (int64_t)gridDim.x * kTeams;
  uint64_t *full = s_full + team * stages, *empty = s_empty + team * stages;
  s_rows += (size_t)team * stages * ring.inputs * ring.slot;
  int s = 0;
  uint32_t ph = 0;
  if (copies) {
    // ------------------------------------------------------------ copies
    if (lane >= kTeams) return;   // lane l copies for team l
    const uint32_t bytes = f.cols * sizeof(T);
    ptx::IssueLog log;
    for (int64_t row = first; row < f.rows; row += step) {
      if (!ptx::mbar_wait(&empty[s], ph ^ 1u)) {
        atomicOr(&g_norm_err, 1u);
        log.drain(full, stages);   // never leave with a copy into shared memory in flight
        return;
      }
      uintptr_t p[5];
      uint32_t n[5], total = 0;
#pragma unroll
      for (int i = 0; i < 5; ++i) {
        p[i] = reinterpret_cast<uintptr_t>(src[i] + row * ld[i]);
        n[i] = src[i] ? ((uint32_t)(p[i] & 15) + bytes + 15) & ~15u : 0;
        total += n[i];
      }
      ptx::mbar_arrive_expect_tx(&full[s], total);
#pragma unroll
      for (int i = 0; i < 5; ++i)
        if (n[i])
          ptx::bulk_load(s_rows + ((size_t)s * ring.inputs + place[i]) * ring.slot,
                         reinterpret_cast<const void*>(p[i] & ~(uintptr_t)15), n[i], &full[s]);
      log.note(s, ph);
      if (++s == stages) {
        s = 0;
        ph ^= 1;
      }
    }
    return;
  }
  // -------------------------------------------------------------- rows
  const int tid = threadIdx.x - team * threads;
  BlockSum sum{s_sum[team], threads, tid, 1 + team};
  // this thread's columns of the weights, whole vectors of them (every team writes the same)
  const int padded = (f.cols + kVec - 1) / kVec * kVec;
  const int post_gate = f.has_post ? 1 + (f.gate_kind == kGateFeature ? 1 : 0) : 0;
  const Weights<W> wt = {s_w, s_w + ring.weight / sizeof(W), s_w + post_gate * (ring.weight / sizeof(W))};
  {
    const Weights<W> g = global_weights<T, W>(f);
#pragma unroll
    for (int k = 0; k < kV; ++k)
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const int c = column<kA>(tid, threads, k, i);
        if (c >= padded) continue;
        const bool in = c < f.cols;
        if (f.has_post) const_cast<W*>(wt.post)[c] = in ? g.post[c] : down<W>(0.f);
        if (f.has_post && f.gate_kind == kGateFeature) const_cast<W*>(wt.gate)[c] = in ? g.gate[c] : down<W>(0.f);
        if (f.pre) const_cast<W*>(wt.pre)[c] = in ? g.pre[c] : down<W>(0.f);
      }
  }
  ColumnSums<kV> sums;
  clear(sums);
  bool dead = false;
  float2 stats = both(0.f);
  if (kGrad && first < f.rows) stats = stats_of(f, first);
  for (int64_t row = first; row < f.rows; row += step) {
    const float2 now = stats;
    if (kGrad && row + step < f.rows) stats = stats_of(f, row + step);
    if (!dead && !ptx::mbar_wait(&full[s], ph)) {
      // the outputs are wrong from here; no thread may miss the sums' barriers, so the rows go on without waits
      atomicOr(&g_norm_err, 2u);
      dead = true;
    }
    auto at = [&](int i) {
      return reinterpret_cast<const T*>(s_rows + ((size_t)s * ring.inputs + place[i]) * ring.slot +
                                        (reinterpret_cast<uintptr_t>(src[i] + row * ld[i]) & 15));
    };
    Row<T> in = {at(0), at(1), at(2), at(3), at(4)};
    if (f.gate_kind == kGateToken) in.gate = static_cast<const T*>(f.gate) + row * f.ld_gate;
    auto read = [&] {   // this warp has read the stage
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&empty[s]);
    };
    if (kGrad)
      row_backward<T, W, kV, kA, true>(a, row, now, in, wt, sum, sums, read);
    else
      row_forward<T, W, kV, kA, true>(f, row, in, wt, sum, read);
    if (++s == stages) {
      s = 0;
      ph ^= 1;
    }
  }
  if (kGrad) store_sums<W, kV, kA, true>(a, wt, sums, threads);
}

// The partial rows added: lane l of a warp a column, the warps' shares of the
// parts in order.
template <typename W>
__global__ void __launch_bounds__(1024) norm_sums_kernel(const float* __restrict__ partial, int n_parts, int n_sums,
                                                         int cols, W* o0, W* o1, W* o2) {
  __shared__ float s[32][33];
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int padded = (cols + 7) / 8 * 8;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane, which = blockIdx.y;
  float v = 0.f;
  if (c < cols) {
    const float* p = partial + (int64_t)which * padded + c;
#pragma unroll 8
    for (int i = warp; i < n_parts; i += 32) v += __ldcg(p + (int64_t)i * n_sums * padded);
  }
  s[lane][warp] = v;
  __syncthreads();
  // warp w adds column w's 32 shares
  v = s[warp][lane];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int out = blockIdx.x * 32 + warp;
  if (lane == 0 && out < cols) {
    W* o = which == 0 ? o0 : which == 1 ? o1 : o2;
    o[out] = down<W>(v);
  }
}

// Threads of a CTA for rows of `cols` with v vectors per thread.
int threads_for(int cols, int v) { return std::max(32, ((cols + kVec - 1) / kVec + v * 32 - 1) / (v * 32) * 32); }
int vectors(int cols) { return (cols + kVec - 1) / kVec; }

// The persistent kernels' shape with v vectors per thread and so many teams; false where it does not fit.
bool ring_shape(const NormArgs& a, bool grad, bool d_out, int v, int teams, Ring* ring) {
  const int size = type_bytes(a.type), wsize = type_bytes(a.weight_type);
  const int threads = teams * threads_for(a.cols, v) + 32;
  ring->teams = teams;
  if (threads > (grad ? 512 : 1024)) return false;
  ring->slot = (a.cols * size + 64 + 127) / 128 * 128;   // up to 15 bytes before the row, and a word behind its last vector
  ring->weight = (a.cols * wsize + 127) / 128 * 128;
  ring->inputs = 1 + (a.has_post ? 1 : 0) + (a.gate_kind == kGateFull ? 1 : 0);
  if (grad) ring->inputs += (d_out ? 1 : 0) + (a.pre ? 1 : 0);
  ring->weights = (a.has_post ? 1 : 0) + (a.gate_kind == kGateFeature ? 1 : 0) + (a.pre ? 1 : 0);
  // CTAs per SM by registers (64 a thread forward, 128 or less backward) and by shared memory
  for (ring->ctas = std::max(1, std::min(8, (grad && v == 1 ? 640 : grad ? 512 : 1024) / threads)); ring->ctas >= 1; --ring->ctas) {
    const int64_t room = (kRingSmem + 2048) / ring->ctas - 2048 - (int64_t)ring->weights * ring->weight;
    ring->stages = (int)std::min<int64_t>(8, room / (ring->inputs * ring->slot)) / teams * teams;
    if (ring->stages >= 2 * teams) return true;
  }
  return false;
}

// Vectors per thread of the persistent kernels, 0 for one CTA per row.  From
// two rows per SM on there is something to bring ahead.  Two vectors per
// thread leave room for a second CTA on the SM, whose row runs while the first
// waits at its sums (forward, 4096 x 7168 bf16: 42 us against 54 with one CTA
// of one; 3584 columns 24 against 29); where the weights do not fit twice (fp32,
// 7168 columns), two teams of threads in one CTA share them.
int ring_for(const NormArgs& a, bool grad, bool d_out, Ring* ring) {
  const int vecs = vectors(a.cols);
  const bool single = !a.wide && a.type == kF32;
  if (a.rows < 2 * sm_count()) return 0;
  if (grad) {
    // (single accesses with two vectors per thread spill)
    if (vecs > 64 && !single && ring_shape(a, grad, d_out, 2, 1, ring)) return 2;
    return (vecs <= 64 || single) && ring_shape(a, grad, d_out, 1, 1, ring) ? 1 : 0;
  }
  if (vecs > 64 && !single && ring_shape(a, grad, d_out, 2, 1, ring) && ring->ctas >= 2) return 2;
  if (vecs > 512 && !single && ring_shape(a, grad, d_out, 2, 2, ring)) return 2;
  if (ring_shape(a, grad, d_out, 1, 1, ring)) return 1;
  return ring_shape(a, grad, d_out, 2, 1, ring) ? 2 : 0;
}

template <typename T, typename W, int kV, bool kWide, bool kGrad, int kTeams = 1>
cudaError_t launch_rows(const NormGradArgs& a, const Ring& ring, cudaStream_t st) {
  // Rows that are not aligned.  16-bit values: by pairs where all rows start at one, else by shifted words (neighbouring
  // widths, pairs against words: 16384 x 1002 bf16 forward 45 us, 1001 87, backward 141 against 199; 4096 x 7166 fp16
  // 76 against 113, 205 against 214; words against single accesses, 4096 x 4567 backward: 204 against 376).  32-bit
  // values: by single accesses (777 x 1003: 6 us forward against 11 by shifted words; 3000 x 2998 backward 80 us,
  // by pairs 124).
  constexpr Access kOther = sizeof(T) == 2 ? kShifted : kStrided, kEven = sizeof(T) == 2 ? kPairs : kOther;
  if constexpr (sizeof(T) == 4 && !kWide && (kTeams == 2 || (kGrad && kV == 2))) {
    return cudaErrorInvalidValue;   // ring_for chooses neither with single accesses
  } else {
    void (*kernel)(const NormGradArgs, const Ring);
    if constexpr (kWide) kernel = rows_kernel<T, W, kV, kAligned, kGrad, kTeams>;
    else kernel = a.f.even ? rows_kernel<T, W, kV, kEven, kGrad, kTeams> : rows_kernel<T, W, kV, kOther, kGrad, kTeams>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingSmem);
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, dim3((unsigned)std::min(a.f.rows, ring.ctas * sm_count())),
                            dim3(ring.teams * threads_for(a.f.cols, kV) + 32), ring.smem(), st, 1, a, ring);
  }
}

template <typename T, typename W, bool kWide>
cudaError_t forward(const NormArgs& a, cudaStream_t st) {
  constexpr Access kA = kWide ? kAligned : kStrided;
  Ring ring;
  const int vr = ring_for(a, false, false, &ring);
  if (vr) {
    NormGradArgs g = {};
    g.f = a;
    return ring.teams == 2 ? launch_rows<T, W, 2, kWide, false, 2>(g, ring, st)
           : vr == 1       ? launch_rows<T, W, 1, kWide, false>(g, ring, st)
                           : launch_rows<T, W, 2, kWide, false>(g, ring, st);
  }
  const int vecs = vectors(a.cols);
  const int v = vecs <= 1024 ? 1 : 4;
  const int threads = threads_for(a.cols, v);
  const unsigned grid = (unsigned)std::min<int64_t>(a.rows, 1 << 20);
  if (v == 1) return launch_dependent(norm_kernel<T, W, 1, kA>, dim3(grid), dim3(threads), 0, st, 1, a);
  return launch_dependent(norm_kernel<T, W, 4, kA>, dim3(grid), dim3(threads), 0, st, 1, a);
}

// CTAs of the backward, one partial row each
int grad_parts(const NormArgs& a, int v, const Ring& ring) {
  if (v) return std::min(a.rows, ring.ctas * sm_count());
  return std::max(1, std::min(a.rows, 2 * sm_count()));
}

template <typename T, typename W, bool kWide>
cudaError_t backward(NormGradArgs a, cudaStream_t st) {
  constexpr Access kA = kWide ? kAligned : kStrided;
  Ring ring;
  const int vr = ring_for(a.f, true, a.d_out != nullptr, &ring);
  a.n_parts = grad_parts(a.f, vr, ring);
  const int vecs = vectors(a.f.cols), v = vecs <= 512 ? 1 : vecs <= 1024 ? 2 : 4;
  const dim3 threads(threads_for(a.f.cols, v)), grid((unsigned)a.n_parts);
  cudaError_t e;
  if (vr == 1) e = launch_rows<T, W, 1, kWide, true>(a, ring, st);
  else if (vr == 2) e = launch_rows<T, W, 2, kWide, true>(a, ring, st);
  else if (v == 1) e = launch_dependent(norm_grad_kernel<T, W, 1, kA>, grid, threads, 0, st, 1, a);
  else if (v == 2) e = launch_dependent(norm_grad_kernel<T, W, 2, kA>, grid, threads, 0, st, 1, a);
  else e = launch_dependent(norm_grad_kernel<T, W, 4, kA>, grid, threads, 0, st, 1, a);
  if (e != cudaSuccess) return e;
  W* o[3];
  int n = 0;
  if (a.f.has_post) o[n++] = static_cast<W*>(a.d_post);
  if (a.f.pre) o[n++] = static_cast<W*>(a.d_pre);
  if (a.f.has_post && a.f.gate_kind == kGateFeature) o[n++] = static_cast<W*>(a.d_gate);
  for (int i = n; i < 3; ++i) o[i] = nullptr;
  return launch_dependent(norm_sums_kernel<W>, dim3((a.f.cols + 31) / 32, n), dim3(1024), 0, st, 1, a.partial,
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
  // the most CTAs that a backward over such rows may have (ring_shape, and two per SM without a ring)
  const int ctas = std::max(640 / (threads_for(cols, 1) + 32), 512 / (threads_for(cols, 2) + 32));
  return std::max(1, std::min(rows, std::max(2, std::min(8, ctas)) * sm_count()));
}

cudaError_t launch_norm(const NormArgs& a, cudaStream_t st) {
  NORM_DISPATCH(forward, a.type, a.weight_type, a.wide, a, st)
}
cudaError_t launch_norm_grad(const NormGradArgs& a, cudaStream_t st) {
  NORM_DISPATCH(backward, a.f.type, a.f.weight_type, a.f.wide, a, st)
}
cudaError_t norm_errors(unsigned* flags) {
  cudaError_t e = cudaMemcpyFromSymbol(flags, g_norm_err, sizeof(unsigned));
  const unsigned zero = 0;
  if (e == cudaSuccess && *flags) e = cudaMemcpyToSymbol(g_norm_err, &zero, sizeof(unsigned));
  return e;
}

}  // namespace moe
