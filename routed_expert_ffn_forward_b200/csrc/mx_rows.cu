// MXFP4 rows (OCP microscaling): x[r, 32 b .. 32 b + 31] ~ 2^(s - 127) * E2M1 codes.
//
// For a run of 32 values with largest magnitude a, the shared exponent is
// floor(log2 a) - 2 (2 = the exponent of E2M1's largest value, 6 = 1.5 * 2^2),
// and every value times 2^-exponent is rounded to the nearest E2M1 value, ties
// to even, magnitudes above 6 to 6.  The exponent is read off a's float bits,
// so it is exact, and the product with a power of two is exact too: the codes
// are the correctly rounded ones.  A run with an infinity or NaN gets the E8M0
// NaN (255).
//
// Codes keep the GGUF order within a run: byte j holds element j in its low
// and element 16 + j in its high nibble, so the rows are what GGUF blocks and
// the layer's MXFP4 weights hold, with the scales apart.
#include "block_ops.h"
#include "ptx.cuh"

namespace moe {
namespace {

template <typename T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_float<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

// Eight values times `mul` to eight codes (value i in nibble i): round to nearest even, saturating.
__device__ __forceinline__ uint32_t e2m1_codes(const float2* v, float mul) {
  const float2 m = make_float2(mul, mul);
  float2 t[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) t[i] = __fmul2_rn(v[i], m);
  uint32_t w;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(w)
      : "f"(t[0].x), "f"(t[0].y), "f"(t[1].x), "f"(t[1].y), "f"(t[2].x), "f"(t[2].y), "f"(t[3].x), "f"(t[3].y));
  return w;
}
// Two codes (a byte, the first in its low nibble) to their values in bf16, times
// 2^(s - 127), exactly: an E2M1 value is a bf16 number with a one-bit mantissa.
__device__ __forceinline__ uint32_t e2m1_bf16x2(uint32_t codes, float up) {
  auto value = [&](uint32_t c) {
    // codes 2..7 are floats 2^(c / 2 - 1) (1 + c % 2 / 2), 0 and 1 are 0 and 0.5
    const uint32_t m = c & 7u;
    const float a = m < 2 ? 0.5f * (float)m : __uint_as_float((126u + (m >> 1)) << 23 | (m & 1u) << 22);
    return __uint_as_float(__float_as_uint(a) | (c & 8u) << 28) * up;
  };
  const __nv_bfloat162 h = __floats2bfloat162_rn(value(codes), value(codes >> 4));
  return *reinterpret_cast<const uint32_t*>(&h);
}
// eight nibbles to the low nibbles of eight bytes
__device__ __forceinline__ uint2 spread_nibbles(uint32_t v) {
  uint32_t lo = v & 0xFFFFu, hi = v >> 16;
  lo = (lo | (lo << 8)) & 0x00FF00FFu;
  hi = (hi | (hi << 8)) & 0x00FF00FFu;
  return make_uint2((lo | (lo << 4)) & 0x0F0F0F0Fu, (hi | (hi << 4)) & 0x0F0F0F0Fu);
}

// Sixteen consecutive values of a row from column c as pairs, zeros behind its
// end; the raw words are kept until then, so that several loads are in flight.
// Rows that are not aligned are read in the 16-byte words that hold a byte of
// the values (such a word lies in one page with that byte), and shifted.
template <typename T, bool kVec>
struct Values16 {
  static constexpr int kWords = sizeof(T) * 16 / 16;
  uint4 raw[kWords + (kVec ? 0 : 1)];
  uint32_t shift;
  __device__ __forceinline__ void load(const T* __restrict__ row, int c, int cols) {
    const T* p = row + c;
    shift = 0;
    if (c + 16 <= cols) {
      if (!kVec) shift = (uint32_t)reinterpret_cast<uintptr_t>(p) & 15u;
      const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(p) - shift);
#pragma unroll
      for (int i = 0; i < kWords; ++i) raw[i] = __ldg(q + i);
      if (!kVec && shift) raw[kWords] = __ldg(q + kWords);
    } else {
      T* e = reinterpret_cast<T*>(raw);
#pragma unroll
      for (int i = 0; i < 16; ++i) e[i] = c + i < cols ? p[i] : T(0.f);
    }
  }
  __device__ __forceinline__ void pairs(float2* v) const {
    uint32_t w[4 * kWords];
    if (kVec) {
#pragma unroll
      for (int i = 0; i < 4 * kWords; ++i) w[i] = reinterpret_cast<const uint32_t*>(raw)[i];
    } else {
      shifted_words<4 * kWords>(reinterpret_cast<const uint32_t*>(raw), shift, w);
    }
    const T* e = reinterpret_cast<const T*>(w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = make_float2(to_float<T>(e[2 * i]), to_float<T>(e[2 * i + 1]));
  }
};

// A half warp takes kU chunks of 256 columns at a time, all their loads first;
// sixteen consecutive values per lane, so that a run is a pair of lanes, its
// maximum one shuffle and its bytes one trade of a word: lane 0 writes bytes
// 0..7 (elements 0..7 with 16..23), lane 1 bytes 8..15.  Bound by instruction
// issue for 16-bit values (with eight values per lane and a division per chunk
// 4096 x 7168 bf16 took 22.7 us), by HBM for 32-bit ones.
template <typename T, bool kVec, int kU>
__global__ void __launch_bounds__(256) quantize_kernel(const T* __restrict__ x, int64_t ld, uint32_t n, int cols, uint32_t kc,
                                                       uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                                                       __nv_bfloat16* __restrict__ values) {
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  __shared__ uint4 s_values[kVec ? 1 : 256 * 2];   // a lane's 16 values, where rows of values are not aligned
  const uint32_t lane = threadIdx.x & 15;
  const uint32_t halves = gridDim.x * (blockDim.x >> 4), step = halves * kU;
  uint32_t w0 = (blockIdx.x * (blockDim.x >> 4) + (threadIdx.x >> 4)) * kU;
  // (row, chunk) of w0, kept without a division per chunk
  uint32_t row0 = w0 / kc, chunk0 = w0 - row0 * kc;
  const uint32_t step_rows = step / kc, step_chunks = step - step_rows * kc;
  // a warp stays whole: its upper half may be behind the end
  for (uint32_t first = w0 - (threadIdx.x >> 4 & 1) * kU; first < n; first += step, w0 += step) {
    Values16<T, kVec> in[kU];
    uint32_t row = row0, chunk = chunk0;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      in[u].load(x + row * ld, w0 + u < n ? (int)(chunk * kMxChunk + lane * 16) : cols, cols);
      if (++chunk == kc) {
        chunk = 0;
        row = min(row + 1, (n - 1) / kc);
      }
    }
    row = row0;
    chunk = chunk0;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const uint32_t w = w0 + u;
      float2 v[8];
      in[u].pairs(v);
      uint32_t top = 0;   // magnitude bits order like the magnitudes, NaN above all
#pragma unroll
      for (int i = 0; i < 8; ++i)
        top = max(top, max(__float_as_uint(v[i].x) & 0x7FFFFFFFu, __float_as_uint(v[i].y) & 0x7FFFFFFFu));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      const int ef = (int)(top >> 23);
      const int s = ef == 255 ? 255 : max(ef - 2, 0);
      const float mul = __uint_as_float((uint32_t)(254 - min(s, 253)) << 23);   // 2^(127 - s)
      const uint32_t a = e2m1_codes(v, mul), b = e2m1_codes(v + 4, mul);   // this lane's first and last eight
      const bool upper = lane & 1;   // elements 16..31 of the run
      const uint32_t other = __shfl_xor_sync(0xffffffffu, upper ? a : b, 1);
      const uint2 lo = spread_nibbles(upper ? other : a), hi = spread_nibbles(upper ? b : other);
      if (w < n) {
        reinterpret_cast<uint2*>(codes)[(size_t)w * 16 + lane] = make_uint2(lo.x | hi.x << 4, lo.y | hi.y << 4);
        if (!upper) scales[(size_t)w * 8 + (lane >> 1)] = (uint8_t)s;
        if (values) {
          // 2^(s - 127); s = 0 is the subnormal 2^-127, s = 255 stands for NaN
          const float up = s == 255 ? __uint_as_float(0x7FC00000u) : s ? __uint_as_float((uint32_t)s << 23)
                                                                       : __uint_as_float(0x00400000u);
          const int c0 = (int)(chunk * kMxChunk + lane * 16);
          __nv_bfloat16* q = values + (size_t)row * cols + c0;
          uint32_t o[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            o[i] = e2m1_bf16x2(a >> (8 * i), up);
            o[4 + i] = e2m1_bf16x2(b >> (8 * i), up);
          }
          if (kVec) {
            if (c0 + 16 <= cols) {
              reinterpret_cast<uint4*>(q)[0] = make_uint4(o[0], o[1], o[2], o[3]);
              reinterpret_cast<uint4*>(q)[1] = make_uint4(o[4], o[5], o[6], o[7]);
            } else {
              const __nv_bfloat16* e = reinterpret_cast<const __nv_bfloat16*>(o);
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (c0 + i < cols) q[i] = e[i];
            }
          } else {
            uint4* mine = s_values + threadIdx.x * 2;
            mine[0] = make_uint4(o[0], o[1], o[2], o[3]);
            mine[1] = make_uint4(o[4], o[5], o[6], o[7]);
          }
        }
      }
      if (!kVec && values) {
        // neighbouring lanes store neighbouring values of the half warp's chunk
        __syncwarp();
        if (w < n) {
          const __nv_bfloat16* e = reinterpret_cast<const __nv_bfloat16*>(s_values + (threadIdx.x & ~15) * 2);
          const int c0 = (int)(chunk * kMxChunk + lane);
          __nv_bfloat16* q = values + (size_t)row * cols + c0;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (c0 + 16 * i < cols) q[16 * i] = e[lane + 16 * i];
        }
        __syncwarp();
      }
      if (++chunk == kc) {
        chunk = 0;
        ++row;
      }
    }
    row0 += step_rows;
    chunk0 += step_chunks;
    if (chunk0 >= kc) {
      chunk0 -= kc;
      ++row0;
    }
    row0 = min(row0, (n - 1) / kc);   // the upper half of the last warp loads nothing, from a row that is there
  }
}

// One CTA per block of the image (256 weight rows x one chunk).  Half h holds
// the rows 2 i + h of the tile (paired: row i of the first half of the matrix
// for h = 0, of the second for h = 1), so that one accumulator lane of the two
// halves holds two neighbouring features, or a gate and its up.
__global__ void __launch_bounds__(256) pack_kernel(const uint8_t* __restrict__ codes,
                                                   const uint8_t* __restrict__ scales, int rows, int kc, int row_tiles,
                                                   int paired, uint8_t* __restrict__ image) {
  const int64_t b = blockIdx.x;
  const int c = (int)(b % kc), rt = (int)((b / kc) % row_tiles);
  const int64_t mat = b / kc / row_tiles;
  uint8_t* dst = image + b * kMxBlockBytes;
  auto source_row = [&](int r) {   // row r of the block's 256: half r / 128, lane r % 128
    const int i = rt * 128 + (r & 127);
    if (paired) return i < rows / 2 ? i + (r >> 7) * (rows / 2) : -1;
    return 2 * i + (r >> 7) < rows ? 2 * i + (r >> 7) : -1;
  };
  for (int i = threadIdx.x; i < 256 * 8; i += blockDim.x) {
    const int r = i >> 3, k = i & 7, src = source_row(r);
    uint4 v = make_uint4(0, 0, 0, 0);
    if (src >= 0) v = __ldg(reinterpret_cast<const uint4*>(codes + ((mat * rows + src) * kc + c) * 128) + k);
    *reinterpret_cast<uint4*>(dst + (r >> 7) * kMxHalfCodes + (r & 127) * 128 + ((k ^ (r & 7)) << 4)) = v;
  }
  // scales: per 128 values of K a 512-byte tile, row r % 32 of 16 bytes with
  // four bytes for each of the rows r % 32 + {0, 32, 64, 96}
  for (int i = threadIdx.x; i < 256 * 2; i += blockDim.x) {
    const int r = i >> 1, k = i & 1, src = source_row(r);
    uint32_t v = 0x7F7F7F7Fu;
    if (src >= 0) v = __ldg(reinterpret_cast<const uint32_t*>(scales + ((mat * rows + src) * kc + c) * 8) + k);
    uint8_t* t = dst + 2 * kMxHalfCodes + (r >> 7) * kMxHalfScales + k * 512;
    *reinterpret_cast<uint32_t*>(t + (r & 31) * 16 + ((r & 127) >> 5) * 4) = v;
  }
}

template <typename T, bool kVec>
cudaError_t quantize_as(const T* x, int64_t ld, uint32_t n, int cols, uint8_t* codes, uint8_t* scales,
                        __nv_bfloat16* values, cudaStream_t st) {
  const uint32_t kc = mx_chunks(cols), sms = sm_count();
  // a chunk per half warp until the GPU is full of them, then two
  const bool many = n > sms * 128;
  const unsigned blocks = std::min(many ? (n + 31) / 32 : (n + 15) / 16, sms * 8);
  auto* kernel = many ? quantize_kernel<T, kVec, 2> : quantize_kernel<T, kVec, 1>;
  return launch_dependent(kernel, dim3(blocks), dim3(256), 0, st, 1, x, ld, n, cols, kc, codes, scales, values);
}
template <typename T>
cudaError_t quantize(const void* p, int64_t ld, int rows, int cols, uint8_t* codes, uint8_t* scales,
                     __nv_bfloat16* values, cudaStream_t st) {
  const T* x = static_cast<const T*>(p);
  const uint32_t n = (uint32_t)rows * mx_chunks(cols);
  const bool vec = (reinterpret_cast<uintptr_t>(x) % 16 == 0) && (ld * sizeof(T)) % 16 == 0 &&
                   (!values || (reinterpret_cast<uintptr_t>(values) % 16 == 0 && cols % 8 == 0));
  return vec ? quantize_as<T, true>(x, ld, n, cols, codes, scales, values, st)
             : quantize_as<T, false>(x, ld, n, cols, codes, scales, values, st);
}

}  // namespace

cudaError_t launch_mx_quantize(const void* x, int type, int64_t ld, int rows, int cols, uint8_t* codes,
                               uint8_t* scales, __nv_bfloat16* values, cudaStream_t st) {
  if (type == kF32) return quantize<float>(x, ld, rows, cols, codes, scales, values, st);
  if (type == kF16) return quantize<__half>(x, ld, rows, cols, codes, scales, values, st);
  return quantize<__nv_bfloat16>(x, ld, rows, cols, codes, scales, values, st);
}

cudaError_t launch_mx_pack(const uint8_t* codes, const uint8_t* scales, int n_mats, int rows, int cols, bool paired,
                           uint8_t* image, cudaStream_t st) {
  const int kc = mx_chunks(cols), rt = mx_row_tiles(rows);
  const int64_t blocks = (int64_t)n_mats * rt * kc;
  pack_kernel<<<(unsigned)blocks, 256, 0, st>>>(codes, scales, rows, kc, rt, paired ? 1 : 0, image);
  return cudaGetLastError();
}

}  // namespace moe
