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

#ifdef __CUDACC__
// kN words of a stream of kN + 4 words from byte `shift` (0..15) on
template <int kN>
__device__ __forceinline__ void shifted_words(const uint32_t* w, uint32_t shift, uint32_t* out) {
  const bool two = shift & 8, one = shift & 4;
  const uint32_t bits = (shift & 3) * 8;
  uint32_t t[kN + 2], u[kN + 1];
#pragma unroll
  for (int i = 0; i < kN + 2; ++i) t[i] = two ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < kN + 1; ++i) u[i] = one ? t[i + 1] : t[i];
#pragma unroll
  for (int i = 0; i < kN; ++i) out[i] = __funnelshift_r(u[i], u[i + 1], bits);
}
#endif

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
  const int* index;        // [n_rows], index[r] / index_div is a row of x; or null (row r is row r of x)
  void* out;               // [n_rows, ld]
  int64_t ld;
  int index_div, n_x, n_rows, groups, kc, row_tiles, features, out_type;
  bool paired;
  bool wide_store;         // stores of two features: the launcher's, from out, ld and out_type
};
cudaError_t launch_mx_product(MxProductArgs a, cudaStream_t st);
// bit flags of products whose kernel gave up on a bounded wait since the last
// call (the GPU is idle)
cudaError_t mx_product_errors(unsigned* flags);

// ---- block norms ---------------------------------------------------------------
enum { kGateNone = 0, kGateToken = 1, kGateFeature = 2, kGateFull = 3 };
struct NormArgs {
  const void *h, *y, *post, *gate, *pre;   // y null: no block output; pre null: no norm behind it
  void *out, *next;
  float* stats;                            // [rows][2] 1/rms of y and of out, or null
  int64_t ld_h, ld_y, ld_gate, ld_out, ld_next;
  int rows, cols, type, weight_type, gate_kind;
  float scale, eps;
  bool has_post;                           // a norm of y (y is null without rows)
  bool even;                               // accesses of two values: cols and every ld even, bases aligned to two
  bool wide;                               // 16-byte accesses: cols and every ld a multiple of 8, bases aligned
};
struct NormGradArgs {
  NormArgs f;                              // out and next unused
  const void *d_out, *d_next;              // d_out null: zeros
  void *d_h, *d_y, *d_post, *d_gate, *d_pre;
  int64_t ld_d_out, ld_d_next, ld_d_h, ld_d_y, ld_d_gate;
  float* partial;                          // [n_parts][n_sums][cols to 8]
  int n_parts, n_sums;
};
int norm_grad_parts(int rows, int cols);
// bit flags of kernels that gave up on a bounded wait since the last call (the GPU is idle)
cudaError_t norm_errors(unsigned* flags);
cudaError_t launch_norm(const NormArgs& a, cudaStream_t st);
cudaError_t launch_norm_grad(const NormGradArgs& a, cudaStream_t st);

// ---- balance loss --------------------------------------------------------------
struct BalanceArgs {
  const float* logits;       // [tokens, ld]
  const int* ids;            // [tokens, top_k]
  const int* offsets;        // [seqs + 1] or null (one sequence)
  const uint8_t* mask;       // [tokens] or null
  int64_t ld;
  int tokens, experts, top_k, seqs, gating;
  float coef;
  float* loss;               // [1]
  int* counts;               // [seqs, experts]
  float* slope;              // [seqs, experts] d loss / d probability
  float* partial;            // workspace
};
struct BalanceGradArgs {
  const float *logits, *slope, *d_loss;
  const int* offsets;
  const uint8_t* mask;
  int64_t ld, ld_out;
  int tokens, experts, seqs, gating;
  float* d_logits;
};
size_t balance_workspace(int tokens, int experts, int seqs);
int balance_launches(int tokens, int seqs, bool packed);
cudaError_t launch_balance(const BalanceArgs& a, cudaStream_t st);
cudaError_t launch_balance_grad(const BalanceGradArgs& a, cudaStream_t st);

}  // namespace moe
