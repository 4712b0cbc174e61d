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

// 1024 matrices of 2^20 x 65536 are 2^30 blocks, and a product's units at most
// (1024 + 2^24 / 64) x 4096 < 2^31: both fit an int
constexpr int kMaxMxCols = 1 << 16, kMaxMxRows = 1 << 20, kMaxMats = 1024, kMaxRows = 1 << 24;

bool mx_shape(int n_mats, int rows, int cols) {
  return n_mats >= 1 && n_mats <= kMaxMats && rows >= 1 && rows <= kMaxMxRows && cols >= 1 && cols <= kMaxMxCols;
}

// Checks of a block norm's shapes, types and pointers; fills the kernels' form.
moe_status norm_args(const moe_norm_args* p, bool grad, NormArgs* a) {
  if (!p) return fail(MOE_ERR_INVALID_ARG, "null arguments");
  if (p->rows < 0 || p->rows > kMaxRows || p->cols < 1 || p->cols > 16384)
    return fail(MOE_ERR_INVALID_ARG, "rows=%d cols=%d (0..2^24, 1..16384)", p->rows, p->cols);
  if (!known_type(p->type) || (p->weight_type != p->type && p->weight_type != MOE_F32))
    return fail(MOE_ERR_UNSUPPORTED, "type %d with weights of type %d (F32=0, F16=1 or BF16=30; weights the same or F32)",
                (int)p->type, (int)p->weight_type);
  if (p->gate_kind < MOE_GATE_NONE || p->gate_kind > MOE_GATE_FULL)
    return fail(MOE_ERR_INVALID_ARG, "gate_kind=%d", (int)p->gate_kind);
  // without rows there is nothing to point at: the weights tell which norms there are
  const bool post = p->post != nullptr, pre = p->pre != nullptr, rows = p->rows > 0;
  if (!post && !pre) return fail(MOE_ERR_INVALID_ARG, "neither post nor pre weights");
  if (!post && (p->y || p->gate_kind != MOE_GATE_NONE)) return fail(MOE_ERR_INVALID_ARG, "y or a gate without post weights");
  if (rows && (!p->h || (post && !p->y) || (!grad && post && !p->out) || (!grad && pre && !p->next) || (grad && !p->stats)))
    return fail(MOE_ERR_INVALID_ARG, "null pointer");
  if (p->gate_kind != MOE_GATE_NONE && !p->gate && (rows || p->gate_kind == MOE_GATE_FEATURE))
    return fail(MOE_ERR_INVALID_ARG, "null gate");
  if (p->ld_h < p->cols || (post && p->ld_y < p->cols) || (p->gate_kind == MOE_GATE_FULL && p->ld_gate < p->cols) ||
      (p->gate_kind == MOE_GATE_TOKEN && p->ld_gate < 1) || (!grad && post && p->ld_out < p->cols) ||
      (!grad && pre && p->ld_next < p->cols))
    return fail(MOE_ERR_INVALID_ARG, "a row stride is shorter than its row");
  const size_t t = type_bytes(p->type), w = type_bytes(p->weight_type);
  if (!aligned(p->h, t) || !aligned(p->y, t) || !aligned(p->out, t) || !aligned(p->next, t) || !aligned(p->post, w) ||
      !aligned(p->pre, w) || !aligned(p->gate, p->gate_kind == MOE_GATE_FEATURE ? w : t) || !aligned(p->stats, 4))
    return fail(MOE_ERR_INVALID_ARG, "a pointer is not aligned to its type");
  a->h = p->h;
  a->y = post ? p->y : nullptr;
  a->post = p->post;
  a->gate = p->gate;
  a->pre = p->pre;
  a->out = p->out;
  a->next = p->next;
  a->stats = p->stats;
  a->ld_h = p->ld_h;
  a->ld_y = p->ld_y;
  a->ld_gate = p->ld_gate;
  a->ld_out = p->ld_out;
  a->ld_next = p->ld_next;
  a->rows = p->rows;
  a->cols = p->cols;
  a->type = p->type;
  a->weight_type = p->weight_type;
  a->gate_kind = p->gate_kind;
  a->has_post = post;
  a->scale = p->scale;
  a->eps = p->eps;
  // accesses of n values: 8 in 16-byte words, or 2
  auto every = [&](int n, size_t row_align, size_t weight_align) {
    auto fits = [&](const void* q, int64_t ld) { return aligned(q, row_align) && ld % n == 0; };
    return p->cols % n == 0 && fits(p->h, p->ld_h) && aligned(p->post, weight_align) && aligned(p->pre, weight_align) &&
           (!post || fits(p->y, p->ld_y)) && (p->gate_kind != MOE_GATE_FULL || fits(p->gate, p->ld_gate)) &&
           (p->gate_kind != MOE_GATE_FEATURE || aligned(p->gate, weight_align)) &&
           (grad || ((!post || fits(p->out, p->ld_out)) && (!pre || fits(p->next, p->ld_next))));
  };
  a->wide = every(8, 16, 16);
  a->even = every(2, 2 * t, 2 * w);
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_mx_quantize(const void* x, moe_type type, int64_t ld, int rows, int cols, uint8_t* codes,
                           uint8_t* scales, void* values, void* stream) {
  clear_error();
  if (rows < 0 || rows > kMaxRows || cols < 1 || cols > kMaxMxCols || ld < cols)
    return fail(MOE_ERR_INVALID_ARG, "rows=%d cols=%d ld=%lld", rows, cols, (long long)ld);
  if (!known_type(type)) return fail(MOE_ERR_UNSUPPORTED, "type %d (supported: F32=0, F16=1, BF16=30)", (int)type);
  if ((long long)rows * mx_chunks(cols) > 0x7FFFFFFFll)
    return fail(MOE_ERR_UNSUPPORTED, "rows=%d cols=%d: more than 2^31 chunks of 256", rows, cols);
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
  a.index_div = 1;
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
  return launched(launch_mx_product(a, static_cast<cudaStream_t>(stream)), 1, "MXFP4 product");
}

moe_status moe_block_check(void) {
  clear_error();
  unsigned mx = 0, norm = 0;
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = mx_product_errors(&mx);
  if (e == cudaSuccess) e = norm_errors(&norm);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return fail(MOE_ERR_CUDA, "%s", cudaGetErrorString(e));
  }
  if (mx) return fail(MOE_ERR_CUDA, "an MXFP4 product gave up waiting (flags 0x%x)", mx);
  if (norm) return fail(MOE_ERR_CUDA, "a block norm gave up waiting (flags 0x%x)", norm);
  return MOE_OK;
}

moe_status moe_block_norm(const moe_norm_args* args, void* stream) {
  clear_error();
  NormArgs a;
  const moe_status s = norm_args(args, false, &a);
  if (s != MOE_OK || a.rows == 0) return s;
  return launched(launch_norm(a, static_cast<cudaStream_t>(stream)), 1, "block norm");
}

size_t moe_block_norm_workspace(int rows, int cols) {
  if (rows < 0 || rows > kMaxRows || cols < 1 || cols > 16384) return 0;
  return (size_t)norm_grad_parts(rows, cols) * 3 * ((cols + 7) / 8 * 8) * 4;
}

moe_status moe_block_norm_grad(const moe_norm_args* args, const moe_norm_grads* g, void* workspace,
                               size_t workspace_bytes, void* stream) {
  clear_error();
  NormGradArgs a;
  const moe_status s = norm_args(args, true, &a.f);
  if (s != MOE_OK) return s;
  if (!g) return fail(MOE_ERR_INVALID_ARG, "null gradients");
  const NormArgs& f = a.f;
  const bool post = f.has_post, pre = f.pre != nullptr, gate = f.gate_kind != MOE_GATE_NONE, rows = f.rows > 0;
  if ((rows && (!g->d_h || (post && !g->d_y) || (pre && !g->d_next))) || (post && !g->d_post) || (pre && !g->d_pre) ||
      (gate && !g->d_gate && (rows || f.gate_kind == MOE_GATE_FEATURE)) || !workspace)
    return fail(MOE_ERR_INVALID_ARG, "null pointer");
  // the kernels bring every input that is there into a stage that holds what pre and post ask for
  if (!pre && g->d_next) return fail(MOE_ERR_INVALID_ARG, "d_next without pre weights");
  if ((g->d_out && g->ld_d_out < f.cols) || g->ld_d_h < f.cols || (pre && g->ld_d_next < f.cols) ||
      (post && g->ld_d_y < f.cols) || (f.gate_kind == MOE_GATE_FULL && g->ld_d_gate < f.cols) ||
      (f.gate_kind == MOE_GATE_TOKEN && g->ld_d_gate < 1))
    return fail(MOE_ERR_INVALID_ARG, "a row stride is shorter than its row");
  const size_t t = type_bytes(f.type), w = type_bytes(f.weight_type);
  if (!aligned(g->d_out, t) || !aligned(g->d_next, t) || !aligned(g->d_h, t) || !aligned(g->d_y, t) ||
      !aligned(g->d_post, w) || !aligned(g->d_pre, w) ||
      !aligned(g->d_gate, f.gate_kind == MOE_GATE_FEATURE ? w : t) || !aligned(workspace, 16))
    return fail(MOE_ERR_INVALID_ARG, "a pointer is not aligned to its type, or the workspace not to 16 bytes");
  if (workspace_bytes < moe_block_norm_workspace(f.rows, f.cols))
    return fail(MOE_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace_bytes,
                moe_block_norm_workspace(f.rows, f.cols));
  a.d_out = g->d_out;
  a.d_next = g->d_next;
  a.d_h = g->d_h;
  a.d_y = g->d_y;
  a.d_post = g->d_post;
  a.d_gate = g->d_gate;
  a.d_pre = g->d_pre;
  a.ld_d_out = g->ld_d_out;
  a.ld_d_next = g->ld_d_next;
  a.ld_d_h = g->ld_d_h;
  a.ld_d_y = g->ld_d_y;
  a.ld_d_gate = g->ld_d_gate;
  a.partial = static_cast<float*>(workspace);
  a.n_parts = 0;   // the launcher's choice, at most what the workspace holds
  a.n_sums = (post ? 1 : 0) + (pre ? 1 : 0) + (f.gate_kind == MOE_GATE_FEATURE ? 1 : 0);
  auto every = [&](int n, size_t align) {
    auto fits = [&](const void* q, int64_t ld) { return aligned(q, align) && ld % n == 0; };
    return fits(g->d_h, g->ld_d_h) && (!g->d_out || fits(g->d_out, g->ld_d_out)) && (!pre || fits(g->d_next, g->ld_d_next)) &&
           (!post || fits(g->d_y, g->ld_d_y)) && (f.gate_kind != MOE_GATE_FULL || fits(g->d_gate, g->ld_d_gate));
  };
  a.f.wide = f.wide && every(8, 16);
  a.f.even = f.even && every(2, 2 * t);
  return launched(launch_norm_grad(a, static_cast<cudaStream_t>(stream)), 2, "block norm gradient");
}

size_t moe_balance_workspace(int tokens, int experts, int seqs) {
  if (tokens < 0 || tokens > kMaxRows || experts < 1 || experts > 1024 || seqs < 1 || seqs > 65535) return 0;
  return balance_workspace(tokens, experts, seqs);
}

moe_status moe_balance_loss(const float* logits, int64_t ld, const int32_t* ids, int tokens, int experts, int top_k,
                            moe_gating gating, const int32_t* offsets, int seqs, const uint8_t* mask, float coef,
                            float* loss, int32_t* counts, float* slope, void* workspace, size_t workspace_bytes,
                            void* stream) {
  clear_error();
  if (tokens < 0 || tokens > kMaxRows || experts < 1 || experts > 1024 || top_k < 1 || top_k > 32 || ld < experts)
    return fail(MOE_ERR_INVALID_ARG, "tokens=%d experts=%d top_k=%d ld=%lld", tokens, experts, top_k, (long long)ld);
  if (gating != MOE_GATE_SOFTMAX_TOPK && gating != MOE_GATE_SIGMOID_RENORM)
    return fail(MOE_ERR_INVALID_ARG, "gating=%d", (int)gating);
  if (seqs < 1 || seqs > 65535 || (!offsets && seqs != 1))
    return fail(MOE_ERR_INVALID_ARG, "seqs=%d%s", seqs, offsets ? "" : " without offsets");
  if ((tokens && (!logits || !ids)) || !loss || !counts || !slope || !workspace)
    return fail(MOE_ERR_INVALID_ARG, "null pointer");
  if (!aligned(logits, 4) || !aligned(ids, 4) || !aligned(offsets, 4) || !aligned(loss, 4) || !aligned(counts, 4) ||
      !aligned(slope, 4) || !aligned(workspace, 16))
    return fail(MOE_ERR_INVALID_ARG, "pointers must be aligned to 4 bytes, the workspace to 16");
  if (workspace_bytes < balance_workspace(tokens, experts, seqs))
    return fail(MOE_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace_bytes,
                balance_workspace(tokens, experts, seqs));
  BalanceArgs a = {};
  a.logits = logits;
  a.ids = ids;
  a.offsets = offsets;
  a.mask = mask;
  a.ld = ld;
  a.tokens = tokens;
  a.experts = experts;
  a.top_k = top_k;
  a.seqs = seqs;
  a.gating = gating;
  a.coef = coef;
  a.loss = loss;
  a.counts = counts;
  a.slope = slope;
  a.partial = static_cast<float*>(workspace);
  return launched(launch_balance(a, static_cast<cudaStream_t>(stream)), balance_launches(tokens, seqs, offsets != nullptr),
                  "balance loss");
}

moe_status moe_balance_loss_grad(const float* d_loss, const float* slope, const float* logits, int64_t ld, int tokens,
                                 int experts, moe_gating gating, const int32_t* offsets, int seqs, const uint8_t* mask,
                                 float* d_logits, int64_t ld_out, void* stream) {
  clear_error();
  if (tokens < 0 || tokens > kMaxRows || experts < 1 || experts > 1024 || ld < experts || ld_out < experts)
    return fail(MOE_ERR_INVALID_ARG, "tokens=%d experts=%d ld=%lld ld_out=%lld", tokens, experts, (long long)ld,
                (long long)ld_out);
  if (gating != MOE_GATE_SOFTMAX_TOPK && gating != MOE_GATE_SIGMOID_RENORM)
    return fail(MOE_ERR_INVALID_ARG, "gating=%d", (int)gating);
  if (seqs < 1 || seqs > 65535 || (!offsets && seqs != 1))
    return fail(MOE_ERR_INVALID_ARG, "seqs=%d%s", seqs, offsets ? "" : " without offsets");
  if (tokens == 0) return MOE_OK;
  if (!slope || !logits || !d_logits) return fail(MOE_ERR_INVALID_ARG, "null pointer");
  if (!aligned(d_loss, 4) || !aligned(slope, 4) || !aligned(logits, 4) || !aligned(offsets, 4) || !aligned(d_logits, 4))
    return fail(MOE_ERR_INVALID_ARG, "pointers must be aligned to 4 bytes");
  BalanceGradArgs a = {};
  a.logits = logits;
  a.slope = slope;
  a.d_loss = d_loss;
  a.offsets = offsets;
  a.mask = mask;
  a.ld = ld;
  a.ld_out = ld_out;
  a.tokens = tokens;
  a.experts = experts;
  a.seqs = seqs;
  a.gating = gating;
  a.d_logits = d_logits;
  return launched(launch_balance_grad(a, static_cast<cudaStream_t>(stream)), 1, "balance loss gradient");
}

}  // extern "C"
