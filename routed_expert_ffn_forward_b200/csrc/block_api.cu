// C entries of the operators around the layer (include/moe.h): argument checks
// and launches.  None of them allocates, keeps state between calls or waits
// for the GPU, so every call can be captured in a CUDA graph.
#include <atomic>
#include <cstdarg>
#include <cstdio>

#include "../../include/moe.h"
#include "block_ops.h"
#include "moe_internal.h"

namespace moe {

int sm_count() {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> counts[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 148;
  int n = counts[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 148;
    counts[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

}  // namespace moe

namespace {

using namespace moe;

moe_status fail(moe_status s, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return (moe_status)report_error(s, buf);
}

// The launch's status; the runtime's last-error record is cleared on failure.
moe_status launched(cudaError_t e, unsigned launches, const char* what) {
  if (e == cudaSuccess) {
    count_launches(launches);
    return MOE_OK;
  }
  (void)cudaGetLastError();
  return fail(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool known_type(int t) { return t == kF32 || t == kF16 || t == kBF16; }
bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

constexpr int kMaxMxCols = 1 << 16, kMaxMxRows = 1 << 20, kMaxMats = 1024, kMaxRows = 1 << 24;

bool mx_shape(int n_mats, int rows, int cols) {
  return n_mats >= 1 && n_mats <= kMaxMats && rows >= 1 && rows <= kMaxMxRows && cols >= 1 && cols <= kMaxMxCols;
}

}  // namespace

extern "C" {

moe_status moe_mx_quantize(const void* x, moe_type type, int64_t ld, int rows, int cols, uint8_t* codes,
                           uint8_t* scales, void* values, void* stream) {
  clear_error();
  if (rows < 0 || rows > kMaxRows || cols < 1 || cols > kMaxMxCols || ld < cols)
    return fail(MOE_ERR_INVALID_ARG, "rows=%d cols=%d ld=%lld", rows, cols, (long long)ld);
  if (!known_type(type)) return fail(MOE_ERR_UNSUPPORTED, "type %d (supported: F32=0, F16=1, BF16=30)", (int)type);
  if (rows == 0) return MOE_OK;
  if (!x || !codes || !scales) return fail(MOE_ERR_INVALID_ARG, "null pointer");
  if (!aligned(x, type_bytes(type)) || !aligned(codes, 16) || !aligned(scales, 8) || !aligned(values, 2))
    return fail(MOE_ERR_INVALID_ARG, "x and values must be aligned to their type, codes to 16 and scales to 8 bytes");
  return launched(launch_mx_quantize(x, type, ld, rows, cols, codes, scales, static_cast<__nv_bfloat16*>(values),
                                     static_cast<cudaStream_t>(stream)), 1, "MXFP4 quantisation");
}

size_t moe_mx_image_bytes(int n_mats, int rows, int cols) {
  if (!mx_shape(n_mats, rows, cols)) return 0;
  return (size_t)n_mats * mx_row_tiles(rows) * mx_chunks(cols) * kMxBlockBytes;
}

moe_status moe_mx_pack(const uint8_t* codes, const uint8_t* scales, int n_mats, int rows, int cols, int paired,
                       void* image, void* stream) {
  clear_error();
  if (!mx_shape(n_mats, rows, cols) || (paired && rows % 2))
    return fail(MOE_ERR_INVALID_ARG, "n_mats=%d rows=%d cols=%d paired=%d", n_mats, rows, cols, paired);
  if ((long long)n_mats * mx_row_tiles(rows) * mx_chunks(cols) > 0x7FFFFFFFll)
    return fail(MOE_ERR_UNSUPPORTED, "n_mats=%d rows=%d cols=%d: too many blocks", n_mats, rows, cols);
  if (!codes || !scales || !image) return fail(MOE_ERR_INVALID_ARG, "null pointer");
  if (!aligned(codes, 16) || !aligned(scales, 8) || !aligned(image, 16))
    return fail(MOE_ERR_INVALID_ARG, "codes and image must be aligned to 16 bytes, scales to 8");
  return launched(launch_mx_pack(codes, scales, n_mats, rows, cols, paired != 0, static_cast<uint8_t*>(image),
                                 static_cast<cudaStream_t>(stream)), 1, "MXFP4 packing");
}

moe_status moe_mx_product(const uint8_t* codes, const uint8_t* scales, int n_x, const void* image, int n_mats,
                          int rows, int cols, int paired, const int32_t* offsets, const int32_t* index, int n_rows,
                          void* out, moe_type out_type, int64_t ld, void* stream) {
  clear_error();
  if (!mx_shape(n_mats, rows, cols) || (paired && rows % 2))
    return fail(MOE_ERR_INVALID_ARG, "n_mats=%d rows=%d cols=%d paired=%d", n_mats, rows, cols, paired);
  const int features = paired ? rows / 2 : rows;
  if (n_x < 0 || n_x > kMaxRows || n_rows < 0 || n_rows > kMaxRows || ld < features)
    return fail(MOE_ERR_INVALID_ARG, "n_x=%d n_rows=%d ld=%lld (%d features)", n_x, n_rows, (long long)ld, features);
  if (out_type != MOE_BF16 && out_type != MOE_F32)
    return fail(MOE_ERR_UNSUPPORTED, "output type %d (supported: F32=0, BF16=30)", (int)out_type);
  if (!offsets && n_mats != 1) return fail(MOE_ERR_INVALID_ARG, "%d matrices need offsets", n_mats);
  if (!index && n_rows > n_x) return fail(MOE_ERR_INVALID_ARG, "%d rows of %d without an index", n_rows, n_x);
  if (((long long)n_mats + n_rows / 64 + 1) * mx_row_tiles(rows) > 0x7FFFFFFFll)
    return fail(MOE_ERR_UNSUPPORTED, "n_rows=%d rows=%d: too many tiles", n_rows, rows);
  if (n_rows == 0) return MOE_OK;
  if (!codes || !scales || !image || !out) return fail(MOE_ERR_INVALID_ARG, "null pointer");
  const size_t size = type_bytes(out_type);
  if (!aligned(codes, 16) || !aligned(scales, 8) || !aligned(image, 16) || !aligned(offsets, 4) ||
      !aligned(index, 4) || !aligned(out, size))
    return fail(MOE_ERR_INVALID_ARG, "codes and image must be aligned to 16 bytes, scales to 8, the rest to its type");
  MxProductArgs a = {};
  a.codes = codes;
  a.scales = scales;
  a.image = static_cast<const uint8_t*>(image);
  a.offsets = offsets;
  a.index = index;
  a.out = out;
  a.ld = ld;
  a.n_x = n_x;
  a.n_rows = n_rows;
  a.groups = n_mats;
  a.kc = mx_chunks(cols);
  a.row_tiles = mx_row_tiles(rows);
  a.features = features;
  a.out_type = out_type;
  a.paired = paired != 0;
  a.wide_store = ld % 2 == 0 && aligned(out, 2 * size);
  return launched(launch_mx_product(a, static_cast<cudaStream_t>(stream)), 1, "MXFP4 product");
}

moe_status moe_mx_check(void) {
  clear_error();
  unsigned flags = 0;
  const cudaError_t e = mx_product_errors(&flags);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return fail(MOE_ERR_CUDA, "%s", cudaGetErrorString(e));
  }
  if (flags) return fail(MOE_ERR_CUDA, "an MXFP4 product gave up waiting (flags 0x%x)", flags);
  return MOE_OK;
}

}  // extern "C"
