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

// Eight values to eight codes (value i in nibble i): round to nearest even, saturating.
__device__ __forceinline__ uint32_t e2m1_codes(const float* v) {
  uint32_t w;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(w)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return w;
}
// E2M1 magnitude of a 3-bit code: codes 2..7 are floats with a one-bit
// mantissa, 0 and 1 are 0 and 0.5.
__device__ __forceinline__ float e2m1_value(uint32_t c) {
  const uint32_t m = c & 7u;
  const float a = m < 2 ? 0.5f * (float)m : __uint_as_float((126u + (m >> 1)) << 23 | (m & 1u) << 22);
  return c & 8u ? -a : a;
}
// four nibbles (low half word) to the low nibbles of four bytes
__device__ __forceinline__ uint32_t spread_nibbles(uint32_t v) {
  v = (v | (v << 8)) & 0x00FF00FFu;
  return (v | (v << 4)) & 0x0F0F0F0Fu;
}

// Eight consecutive values of a row from column c; zeros behind its end.
template <typename T, bool kVec>
__device__ __forceinline__ void load8(const T* __restrict__ p, int c, int cols, float* v) {
  if (kVec && c + 8 <= cols) {
    constexpr int kWords = sizeof(T) / 2;
    uint4 raw[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) raw[i] = __ldg(reinterpret_cast<const uint4*>(p + c) + i);
    const T* e = reinterpret_cast<const T*>(raw);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_float<T>(e[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < cols ? to_float<T>(p[c + i]) : 0.f;
  }
}

// A warp takes kU chunks of 256 columns at a time, all their loads first; eight
// consecutive values per lane, so that a run is a quad of lanes and its
// maximum two shuffles.  Bound by HBM (7168 x 2048 fp32: see kU in quantize).
template <typename T, bool kVec, int kU>
__global__ void __launch_bounds__(256) quantize_kernel(const T* __restrict__ x, int64_t ld, uint32_t n, int cols, uint32_t kc,
                                                       uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                                                       __nv_bfloat16* __restrict__ values) {
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const uint32_t step = gridDim.x * (blockDim.x >> 5) * kU;
  for (uint32_t w0 = (blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) * kU; w0 < n; w0 += step) {
    float v[kU][8];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const uint32_t w = min(w0 + u, n - 1), row = w / kc;
      load8<T, kVec>(x + row * ld, (w - row * kc) * kMxChunk + lane * 8, cols, v[u]);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const uint32_t w = w0 + u;
      if (w >= n) break;
      uint32_t top = 0;   // magnitude bits order like the magnitudes, NaN above all
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[u][i]) & 0x7FFFFFFFu);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int ef = (int)(top >> 23);
      const int s = ef == 255 ? 255 : max(ef - 2, 0);
      const float mul = __uint_as_float((uint32_t)(254 - min(s, 253)) << 23);   // 2^(127 - s)
      float t[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = v[u][i] * mul;
      const uint32_t w8 = e2m1_codes(t);
      // lanes q and q ^ 2 of a quad hold elements j.. and 16 + j..: each writes
      // one 32-bit word that pairs four of the lower with four of the upper
      const uint32_t other = __shfl_xor_sync(0xffffffffu, w8, 2);
      const bool upper = lane & 2;
      const uint32_t lo = upper ? other >> 16 : w8 & 0xFFFFu;
      const uint32_t hi = upper ? w8 >> 16 : other & 0xFFFFu;
      const int word = (lane & ~3) + 2 * (lane & 1) + (upper ? 1 : 0);
      reinterpret_cast<uint32_t*>(codes)[(size_t)w * 32 + word] = spread_nibbles(lo) | spread_nibbles(hi) << 4;
      if ((lane & 3) == 0) scales[(size_t)w * 8 + (lane >> 2)] = (uint8_t)s;
      if (values) {
        // 2^(s - 127); s = 0 is the subnormal 2^-127, s = 255 stands for NaN
        const float up = s == 255 ? __uint_as_float(0x7FC00000u) : s ? __uint_as_float((uint32_t)s << 23)
                                                                     : __uint_as_float(0x00400000u);
        __nv_bfloat162 o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)   // exact
          o[i] = __floats2bfloat162_rn(e2m1_value(w8 >> (8 * i)) * up, e2m1_value(w8 >> (8 * i + 4)) * up);
        const uint32_t row = w / kc;
        const int c0 = (w - row * kc) * kMxChunk + lane * 8;
        __nv_bfloat16* q = values + (size_t)row * cols + c0;
        if (kVec && c0 + 8 <= cols && cols % 8 == 0) {
          *reinterpret_cast<uint4*>(q) = *reinterpret_cast<const uint4*>(o);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (c0 + i < cols) q[i] = i & 1 ? o[i >> 1].y : o[i >> 1].x;
        }
      }
    }
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
  // a chunk per warp until the GPU is full of warps, then four
  const bool many = n > sms * 64;
  const unsigned blocks = std::min(many ? (n + 31) / 32 : (n + 7) / 8, sms * 8);
  auto* kernel = many ? quantize_kernel<T, kVec, 4> : quantize_kernel<T, kVec, 1>;
  return launch_dependent(kernel, dim3(blocks), dim3(256), 0, st, 1, x, ld, n, cols, kc, codes, scales, values);
}
template <typename T>
cudaError_t quantize(const void* p, int64_t ld, int rows, int cols, uint8_t* codes, uint8_t* scales,
                     __nv_bfloat16* values, cudaStream_t st) {
  const T* x = static_cast<const T*>(p);
  const uint32_t n = (uint32_t)rows * mx_chunks(cols);
  const bool vec = (reinterpret_cast<uintptr_t>(x) % 16 == 0) && (ld * sizeof(T)) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(values) % 16 == 0;
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
