// Grouped product of MXFP4 rows with MXFP4 weights on the 5th-generation
// tensor cores: out[r, f] = sum_k w_g(r)[f, k] * x[index[r], k], fp32 sums.
//
// The block-scaled MMA (kind::mxf4) takes the E2M1 codes of both operands from
// shared memory and the E8M0 scales, one per 32 values of K, from tensor
// memory: nothing is dequantised, a product of two values is exact, and a
// weight costs its 17/32 byte of HBM and L2 traffic alone.
//
// A work unit is (group, 256 weight rows, tile of up to kNT of the group's
// rows).  The weights are the A operand as two M = 128 halves, the rows the B
// operand, so that few rows cost a short N, not an empty M.  K advances by
// chunks of 256 through a ring of stages; a stage's weights are one contiguous
// 34816-byte bulk copy from the packed image (mx_rows.cu), its rows 128-byte
// pieces gathered by `index`.
//
//   warps 0-3   rows: cp.async of codes (into the 128-byte swizzle) and scales
//   warp 4      weights: one bulk copy per stage
//   warp 5      TMEM; one thread copies the scales to tensor memory
//               (tcgen05.cp) and issues tcgen05.mma and tcgen05.commit
//   warps 8-15  epilogue: tcgen05.ld, SwiGLU, stores (a lane holds two
//               neighbouring features, so a warp stores 64 of them in a row)
//
// With few units (small batches of few groups) a cluster of up to 8 CTAs
// shares a unit: each takes a part of K, and the partial sums are added from
// the CTAs' shared memory in rank order.
#include "block_ops.h"
#include "moe_internal.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kMaxGroups = 1024;
constexpr int kThreads = 512;
constexpr int kRowWarps = 4, kWeightWarp = 4, kMmaWarp = 5, kFirstEpi = 8, kEpiWarps = 8;

// bit flags: which role gave up on a bounded wait
__device__ unsigned g_mx_err = 0;

template <int kNT, int kNS, int kNAcc>
struct Config {
  static constexpr int kScaleTiles = (kNT + 127) / 128;             // 512-byte scale tiles per 128 of K
  static constexpr int kRowCodes = kNT * 128, kRowScales = 2 * kScaleTiles * 512;
  static constexpr int kStage = kMxBlockBytes + ((kRowCodes + 1023) & ~1023) + kRowScales;
  static constexpr int kBars = 3 * kNS + 2 * kNAcc + 1;
  static constexpr size_t kSmem = 1024 + (size_t)kNS * kStage + 8 * kBars + 16 + 128 + 2 * 4 * (kMaxGroups + 4);
  // tensor memory columns: accumulators, then the scales of one stage
  static constexpr int kSA = 2 * kNT * kNAcc, kSB = kSA + 16;
  static_assert(kSB + 8 * kScaleTiles <= 512, "tensor memory");
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kNT % 16 == 0 && kStage % 1024 == 0, "layout");
};

struct Unit {
  int group, row0, count, row_tile;
};

// Unit u of the group-major list; a group's tiles of the same weights are
// neighbours, so that they share them in L2.
template <int kNT>
__device__ __forceinline__ Unit find_unit(int u, const int* s_off, const int* s_start, int groups) {
  int lo = 0, hi = groups;              // s_start[lo] <= u < s_start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s_start[mid] <= u) lo = mid; else hi = mid;
  }
  const int count = s_off[lo + 1] - s_off[lo], tiles = (count + kNT - 1) / kNT;
  const int local = u - s_start[lo], t = local % tiles;
  const int per = ((count + tiles - 1) / tiles + 15) & ~15;
  return {lo, s_off[lo] + t * per, min(per, count - t * per), local / tiles};
}

// Where a thread's accumulators go: lane i of the unit's 128, two accumulators
// each (features 2 i and 2 i + 1, or the gate and up of feature i).
template <bool kPaired, typename Out>
struct Store {
  Out* base;     // feature of row 0
  int64_t ld;
  int n;         // features this lane stores: 0, 1 or 2
  bool wide;
  __device__ __forceinline__ Store(const MxProductArgs& a, int i) : ld(a.ld), wide(a.wide_store) {
    const int f = kPaired ? i : 2 * i;
    base = static_cast<Out*>(a.out) + f;
    n = min(max(a.features - f, 0), kPaired ? 1 : 2);
  }
  __device__ __forceinline__ void operator()(Out* p, float v0, float v1) const {
    if (kPaired) {
      const float h = __fdividef(v0, 1.f + __expf(-v0)) * v1;   // silu(gate) * up, ~1e-6 relative
      if (n) put(p, h);
    } else if (n == 2 && wide) {
      put2(p, v0, v1);
    } else {
      if (n) put(p, v0);
      if (n == 2) put(p + 1, v1);
    }
  }
  static __device__ __forceinline__ void put(float* p, float v) { *p = v; }
  static __device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
  static __device__ __forceinline__ void put2(float* p, float v0, float v1) {
    *reinterpret_cast<float2*>(p) = make_float2(v0, v1);
  }
  static __device__ __forceinline__ void put2(__nv_bfloat16* p, float v0, float v1) {
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v0, v1);
  }
};

template <int kNT, int kNS, int kNAcc, bool kSplit, bool kPaired, typename Out>
__global__ void __launch_bounds__(kThreads, 1) mx_product_kernel(const MxProductArgs a, int cluster) {
  using C = Config<kNT, kNS, kNAcc>;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* w_full = reinterpret_cast<uint64_t*>(sm + (size_t)kNS * C::kStage);
  uint64_t* r_full = w_full + kNS;
  uint64_t* empty = r_full + kNS;
  uint64_t* acc_full = empty + kNS;
  uint64_t* acc_empty = acc_full + kNAcc;
  uint64_t* drain = acc_empty + kNAcc;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(drain + 1);
  int* s_warp = reinterpret_cast<int*>(s_tmem + 4);
  int* s_off = s_warp + 32;                     // [groups + 1] row offsets, in range
  int* s_start = s_off + kMaxGroups + 4;        // [groups + 1] first unit of each group
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < kNS; ++i) {
      ptx::mbar_init(&w_full[i], 1);
      ptx::mbar_init(&r_full[i], kRowWarps * 32);
      ptx::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < kNAcc; ++i) {
      ptx::mbar_init(&acc_full[i], 1);
      ptx::mbar_init(&acc_empty[i], kEpiWarps);
    }
    ptx::mbar_init(drain, 1);
    ptx::fence_barrier_init();
  }
  if (warp == kMmaWarp) ptx::tmem_alloc(s_tmem, 512);
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  // the groups' rows, kept in 0..n_rows whatever the offsets say
  for (int g = tid; g <= a.groups; g += kThreads)
    s_off[g] = a.offsets ? min(max(__ldg(a.offsets + g), 0), a.n_rows) : g * a.n_rows;
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  int n_units = 0;
  for (int g0 = 0; g0 < a.groups; g0 += kThreads) {
    const int g = g0 + tid;
    int mine = 0, total;
    if (g < a.groups) {
      // a group that ends before it starts has no rows
      const int count = max(s_off[g + 1] - s_off[g], 0);
      mine = (count + kNT - 1) / kNT * a.row_tiles;
    }
    const int before = block_exclusive_scan_1024(mine, &total, s_warp);
    if (g < a.groups) s_start[g] = n_units + before;
    n_units += total;
  }
  if (tid == 0) s_start[a.groups] = n_units;
  __syncthreads();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *s_tmem, 0);
  const int rank = kSplit ? (int)ptx::cluster_rank() : 0;
  const int first = kSplit ? blockIdx.x / cluster : blockIdx.x, step = kSplit ? gridDim.x / cluster : gridDim.x;
  const int k0 = kSplit ? a.kc * rank / cluster : 0, k1 = kSplit ? a.kc * (rank + 1) / cluster : a.kc;

  if (warp < kRowWarps) {
    // ------------------------------------------------------------ rows of x
    const int64_t pitch = (int64_t)a.kc * 128, spitch = (int64_t)a.kc * 8;
    const int piece = tid & 7;
    int it = 0;
    bool ok = true;
    for (int u = first; u < n_units && ok; u += step) {
      const Unit un = find_unit<kNT>(u, s_off, s_start, a.groups);
      // this thread's rows: one 16-byte piece of the codes of rows tid / 8 + 16 j,
      // and the scales of rows tid + 128 j; -1: not a row of x, read as zeros
      auto row_of = [&](int r) {
        if (r >= un.count) return -2;
        int src = a.index ? __ldg(a.index + un.row0 + r) : un.row0 + r;
        if (a.index_div > 1) src /= a.index_div;
        return (unsigned)src < (unsigned)a.n_x ? src : -1;
      };
      int rows[kNT / 16], srows[C::kScaleTiles];
#pragma unroll
      for (int j = 0; j < kNT / 16; ++j) rows[j] = row_of((tid >> 3) + 16 * j);
#pragma unroll
      for (int j = 0; j < C::kScaleTiles; ++j) srows[j] = row_of(tid + 128 * j);
      for (int k = k0; k < k1; ++k, ++it) {
        const int s = it % kNS;
        if (!ptx::mbar_wait(&empty[s], ((it / kNS) & 1) ^ 1)) {
          atomicOr(&g_mx_err, 1u);
          ok = false;
          break;
        }
        const uint32_t dst = ptx::smem_u32(sm + (size_t)s * C::kStage + kMxBlockBytes);
#pragma unroll
        for (int j = 0; j < kNT / 16; ++j) {
          if (rows[j] == -2) continue;
          const int r = (tid >> 3) + 16 * j;
          ptx::cp_async_16(dst + r * 128 + ((piece ^ (r & 7)) << 4),
                           a.codes + max(rows[j], 0) * pitch + k * 128 + piece * 16, rows[j] >= 0);
        }
        const uint32_t sdst = dst + ((C::kRowCodes + 1023) & ~1023) + (tid & 31) * 16 + (tid >> 5) * 4;
#pragma unroll
        for (int j = 0; j < C::kScaleTiles; ++j) {
          if (srows[j] == -2) continue;
          const uint8_t* src = a.scales + max(srows[j], 0) * spitch + k * 8;
          ptx::cp_async_4(sdst + j * 512, src, srows[j] >= 0);
          ptx::cp_async_4(sdst + (C::kScaleTiles + j) * 512, src + 4, srows[j] >= 0);
        }
        ptx::cp_async_arrive(&r_full[s]);
      }
    }
    ptx::cp_async_commit();
    ptx::cp_async_wait<0>();   // never leave with a copy into shared memory in flight
  } else if (warp == kWeightWarp) {
    // ------------------------------------------------------------ weights
    if (lane == 0) {
      ptx::IssueLog log;
      int it = 0;
      bool ok = true;
      for (int u = first; u < n_units && ok; u += step) {
        const Unit un = find_unit<kNT>(u, s_off, s_start, a.groups);
        const uint8_t* src = a.image + ((int64_t)un.group * a.row_tiles + un.row_tile) * a.kc * kMxBlockBytes;
        for (int k = k0; k < k1; ++k, ++it) {
          const int s = it % kNS;
          const uint32_t ph = (it / kNS) & 1;
          if (!ptx::mbar_wait(&empty[s], ph ^ 1)) {
            atomicOr(&g_mx_err, 2u);
            ok = false;
            break;
          }
          ptx::mbar_arrive_expect_tx(&w_full[s], kMxBlockBytes);
          ptx::bulk_load(sm + (size_t)s * C::kStage, src + (int64_t)k * kMxBlockBytes, kMxBlockBytes, &w_full[s]);
          log.note(s, ph);
        }
      }
      if (!ok) log.drain(w_full, kNS);   // never leave with a copy into shared memory in flight
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA (the whole warp; one lane's instructions)
    const uint32_t on = ptx::elect_one();
    const uint32_t ring = ptx::smem_u32(sm);
    int s = 0, n = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int u = first; u < n_units && ok; u += step, ++n) {
      const Unit un = find_unit<kNT>(u, s_off, s_start, a.groups);
      const int acc = n % kNAcc, N = __shfl_sync(0xffffffffu, (un.count + 15) & ~15, 0);
      const uint32_t id0 = ptx::umma_idesc_mxf4(128, N, 0), id1 = ptx::umma_idesc_mxf4(128, N, 1);
      const uint32_t d0 = tmem + acc * 2 * kNT, d1 = d0 + kNT;
      if (!ptx::mbar_wait(&acc_empty[acc], ((n / kNAcc) & 1) ^ 1)) {
        if (on) atomicOr(&g_mx_err, 4u);
        break;
      }
      ptx::tc_fence_after();
      for (int k = k0; k < k1; ++k) {
        if (!ptx::mbar_wait(&w_full[s], ph) || !ptx::mbar_wait(&r_full[s], ph)) {
          if (on) atomicOr(&g_mx_err, 4u);
          ok = false;
          break;
        }
        ptx::fence_proxy_async();   // the rows came through the generic proxy
        ptx::tc_fence_after();
        const uint32_t st = ring + s * C::kStage, rows = st + kMxBlockBytes;
        const uint64_t wd = ptx::umma_desc_sw128(st), rd = ptx::umma_desc_sw128(rows);
        const uint64_t wsd = ptx::scales_desc(st + 2 * kMxHalfCodes);
        const uint64_t rsd = ptx::scales_desc(rows + ((C::kRowCodes + 1023) & ~1023));
        // scale columns: A half h, 128 of K c: kSA + 4 (2 h + c); B: kSB + 4 (c tiles + j)
#pragma unroll
        for (int i = 0; i < 4; ++i) ptx::tmem_copy_scales(on, tmem + C::kSA + 4 * i, wsd + 32 * i);
#pragma unroll
        for (int i = 0; i < 2 * C::kScaleTiles; ++i) ptx::tmem_copy_scales(on, tmem + C::kSB + 4 * i, rsd + 32 * i);
#pragma unroll
        for (int q = 0; q < 4; ++q) {   // 64 of K each, 32 bytes of a row
          const uint32_t id = q & 1 ? id1 : id0, c = q >> 1;
          const uint32_t sb = tmem + C::kSB + 4 * C::kScaleTiles * c;
          const bool add = k > k0 || q > 0;
          ptx::umma_mxf4(on, d0, wd + 2 * q, rd + 2 * q, id, tmem + C::kSA + 4 * c, sb, add);
          ptx::umma_mxf4(on, d1, wd + kMxHalfCodes / 16 + 2 * q, rd + 2 * q, id, tmem + C::kSA + 8 + 4 * c, sb, add);
        }
        ptx::umma_commit_on(on, &empty[s]);
        if (++s == kNS) {
          s = 0;
          ph ^= 1;
        }
      }
      if (ok) ptx::umma_commit_on(on, &acc_full[acc]);
    }
    // wait for every MMA this warp issued before TMEM is released
    ptx::umma_commit_on(on, drain);
    if (!ptx::mbar_wait(drain, 0) && on) atomicOr(&g_mx_err, 4u);
  } else if (warp >= kFirstEpi) {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3, sub = (warp - kFirstEpi) >> 2;   // TMEM lane quarter; which 32-column chunks
    const int lrow = quarter * 32 + lane;
    int n = 0;
    for (int u = first; u < n_units; u += step, ++n) {
      const Unit un = find_unit<kNT>(u, s_off, s_start, a.groups);
      const int acc = n % kNAcc;
      const bool ready = ptx::mbar_wait_sleep(&acc_full[acc], (n / kNAcc) & 1, 100);
      __syncwarp();
      if (!ready) {
        atomicOr(&g_mx_err, 8u);
        break;
      }
      ptx::tc_fence_after();
      const Store<kPaired, Out> store(a, un.row_tile * 128 + lrow);
      const uint32_t t0 = tmem + acc * 2 * kNT + ((uint32_t)(quarter * 32) << 16);
      for (int c0 = 32 * sub; c0 < un.count; c0 += 32 * (kEpiWarps / 4)) {
        uint32_t v0[32], v1[32];
        ptx::tmem_ld32x2(t0 + c0, t0 + kNT + c0, v0, v1);
        if (kSplit) {
          // the ring is free: every copy of this CTA's one unit has been consumed
          float* part = reinterpret_cast<float*>(sm);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (c0 + i < un.count) {
              part[(c0 + i) * 256 + lrow] = __uint_as_float(v0[i]);
              part[(c0 + i) * 256 + 128 + lrow] = __uint_as_float(v1[i]);
            }
        } else {
          Out* p = store.base + (un.row0 + c0) * store.ld;
#pragma unroll
          for (int i = 0; i < 32; ++i, p += store.ld)
            if (c0 + i < un.count) store(p, __uint_as_float(v0[i]), __uint_as_float(v1[i]));
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&acc_empty[acc]);
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (kSplit) {
    __syncwarp();
    ptx::cluster_sync();
    if (first < n_units) {
      // rows rank, rank + cluster, ... of the unit, the parts added in rank order
      const Unit un = find_unit<kNT>(first, s_off, s_start, a.groups);
      const int i = tid & 127;
      const Store<kPaired, Out> store(a, un.row_tile * 128 + i);
      for (int c = rank + cluster * (tid >> 7); c < un.count; c += cluster * (kThreads >> 7)) {
        const uint32_t at = ptx::smem_u32(sm) + (c * 256 + i) * 4;
        float v0 = 0.f, v1 = 0.f;
        for (int r = 0; r < cluster; ++r) {
          v0 += ptx::ld_cluster_f32(at, r);
          v1 += ptx::ld_cluster_f32(at + 512, r);
        }
        store(store.base + (un.row0 + c) * store.ld, v0, v1);
      }
    }
    ptx::cluster_sync();   // no CTA leaves while its part is read
  }
  if (warp == kMmaWarp) {
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

template <int kNT, int kNS, int kNAcc, bool kSplit, bool kPaired, typename Out>
cudaError_t launch_as(const MxProductArgs& a, int cluster, int clusters, cudaStream_t st) {
  using C = Config<kNT, kNS, kNAcc>;
  static_assert(!kSplit || kNT * 256 * 4 <= kNS * C::kStage, "partial sums fit the ring");
  auto* kernel = mx_product_kernel<kNT, kNS, kNAcc, kSplit, kPaired, Out>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
  if (e != cudaSuccess) return e;
  return launch_dependent(kernel, dim3((unsigned)(clusters * cluster)), dim3(kThreads), C::kSmem, st,
                          kSplit ? cluster : 1, a, cluster);
}

template <int kNT, int kNS, int kNAcc, bool kSplit>
cudaError_t launch(const MxProductArgs& a, int cluster, int clusters, cudaStream_t st) {
  const bool f32 = a.out_type == kF32;
  if (a.paired)
    return f32 ? launch_as<kNT, kNS, kNAcc, kSplit, true, float>(a, cluster, clusters, st)
               : launch_as<kNT, kNS, kNAcc, kSplit, true, __nv_bfloat16>(a, cluster, clusters, st);
  return f32 ? launch_as<kNT, kNS, kNAcc, kSplit, false, float>(a, cluster, clusters, st)
             : launch_as<kNT, kNS, kNAcc, kSplit, false, __nv_bfloat16>(a, cluster, clusters, st);
}

}  // namespace

cudaError_t launch_mx_product(const MxProductArgs& a, cudaStream_t st) {
  const int sms = sm_count();
  if (a.n_rows > 1024) return launch<112, 4, 2, false>(a, 1, sms, st);
  // at most this many units: every group of a batch this small is one tile
  const int64_t units = (int64_t)std::min(a.n_rows <= 64 ? a.groups : a.groups + a.n_rows / 64, a.n_rows) * a.row_tiles;
  int cluster = 1;
  while (a.n_rows <= 64 && cluster < 8 && units * cluster * 2 <= sms && a.kc >= cluster * 4) cluster *= 2;
  if (cluster > 1) return launch<64, 5, 2, true>(a, cluster, (int)units, st);
  return launch<64, 5, 2, false>(a, 1, (int)std::min<int64_t>(units, sms), st);
}

cudaError_t mx_product_errors(unsigned* flags) {
  cudaError_t e = cudaMemcpyFromSymbol(flags, g_mx_err, sizeof(unsigned));
  const unsigned zero = 0;
  if (e == cudaSuccess && *flags) e = cudaMemcpyToSymbol(g_mx_err, &zero, sizeof(unsigned));
  return e;
}

}  // namespace moe
