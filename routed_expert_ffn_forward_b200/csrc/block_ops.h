// Launchers of the operators around the layer (include/moe.h, "Operators
// around the layer"): MXFP4 rows and products, block norms, balance loss.
// They keep no state and allocate nothing; arguments are checked by the C
// entries in block_api.cu.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace moe {

// element types (GGML type ids)
constexpr int kF32 = 0, kF16 = 1, kBF16 = 30;
inline int type_bytes(int t) { return t == kF32 ? 4 : 2; }

int sm_count();                    // of the current device
void count_launches(unsigned n);   // into moe_stats.launches

// Launch `kernel` as a programmatic dependent of the stream's previous work:
// it may start early but waits (griddepcontrol.wait) before it touches memory.
template <typename... KArgs, typename... Args>
cudaError_t launch_dependent(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, int cluster,
                             Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// ---- MXFP4 ------------------------------------------------------------------
// A row of `cols` values is stored as ceil(cols / 256) chunks of 256: 128 bytes
// of E2M1 codes and 8 E8M0 scales per chunk, the padding zero codes.
constexpr int kMxChunk = 256;
inline int mx_chunks(int cols) { return (cols + kMxChunk - 1) / kMxChunk; }
// Packed weight image: blocks of 256 weight rows x one chunk -- two halves of
// 128 rows, their codes K-major with the 128-byte swizzle (16384 bytes each),
// then their scales in tensor-memory order (1024 bytes each).
constexpr int kMxHalfCodes = 128 * 128;
constexpr int kMxHalfScales = 2 * 512;
constexpr int kMxBlockBytes = 2 * (kMxHalfCodes + kMxHalfScales);
inline int mx_row_tiles(int rows) { return (rows + 255) / 256; }

cudaError_t launch_mx_quantize(const void* x, int type, int64_t ld, int rows, int cols, uint8_t* codes,
                               uint8_t* scales, __nv_bfloat16* values, cudaStream_t st);
cudaError_t launch_mx_pack(const uint8_t* codes, const uint8_t* scales, int n_mats, int rows, int cols, bool paired,
                           uint8_t* image, cudaStream_t st);

struct MxProductArgs {
  const uint8_t* codes;    // [n_x, 128 * kc]
  const uint8_t* scales;   // [n_x, 8 * kc]
  const uint8_t* image;    // [groups][row tiles][kc][kMxBlockBytes]
  const int* offsets;      // [groups + 1] or null (one group of all rows)
  const int* index;        // [n_rows] or null (row r is row r of x)
  void* out;               // [n_rows, ld]
  int64_t ld;
  int n_x, n_rows, groups, kc, row_tiles, features, out_type;
  bool paired, wide_store;
};
cudaError_t launch_mx_product(const MxProductArgs& a, cudaStream_t st);
// bit flags of products whose kernel gave up on a bounded wait since the last
// call (waits for the current device)
cudaError_t mx_product_errors(unsigned* flags);

}  // namespace moe
