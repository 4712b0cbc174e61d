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
//   warp 5      TMEM; scales to tensor memory (tcgen05.cp), tcgen05.mma and
//               tcgen05.commit, issued by the whole warp with uniform operands
//   warps 8-15  epilogue: tcgen05.ld, SwiGLU, stores (a lane holds two
//               neighbouring features, a pair of lanes four)
//
// Many rows: a CTA pair (cta_group::2) multiplies 512 weight rows by up to 240
// rows of x, of which each CTA holds half: 52 KB of shared-memory traffic per
// 960 tensor-core cycles and SM, against 67 KB for a CTA alone, which is more
// than L2 delivers.  Few units (small batches of few groups): a cluster of up
// to 8 CTAs shares a unit, each takes a part of K, and the partial sums are
// added from the CTAs' shared memory in rank order.
//
// Measured: one token of 8 experts, 7168 x 4096: 19.0 us, 6.6 TB/s of weights;
// 64 tokens of 54 experts, 2048 x 7168, 64 us, 6.6 TB/s; a step of 240 rows
// runs at the MMAs' own rate (960 cycles), and what a unit of many rows loses
// is its epilogue: its accumulators fill tensor memory.
#include <atomic>

#include "block_ops.h"
#include "moe_internal.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kMaxGroups = 1024;
constexpr int kManyRows = 128;   // a group with more is bound by the tensor cores
constexpr int kThreads = 512;
constexpr int kRowWarps = 4, kWeightWarp = 4, kMmaWarp = 5, kFirstEpi = 8, kEpiWarps = 8;

// bit flags: which role gave up on a bounded wait
__device__ unsigned g_mx_err = 0;

// How CTAs share units: each its own, a cluster the K of one unit, or a pair
// (cta_group::2) the rows of x.
enum Mode { kSingle, kSplitK, kPair };

template <int kNT, int kNS, int kNAcc, Mode kMode>
struct Config {
  static constexpr int kRows = kMode == kPair ? kNT / 2 : kNT;      // rows of codes in this CTA
  static constexpr int kScaleTiles = (kNT + 127) / 128;             // 512-byte scale tiles per 128 of K
  static constexpr int kRowCodes = (kRows * 128 + 1023) & ~1023, kRowScales = 2 * kScaleTiles * 512;
  static constexpr int kStage = kMxBlockBytes + kRowCodes + kRowScales;
  static constexpr int kLists = kNT > kManyRows ? 2 : 1;             // of units: see Units
  static constexpr int kBars = 3 * kNS + 2 * kNAcc + 1;
  // tensor memory: slots of accumulators of both halves, then the scales of one
  // stage.  Units take the slots in turn, so that the next unit's MMAs run while
  // the last one's rows are stored; a pair's two slots are the two sides of one
  // accumulator, which a unit of more than kNT / 2 rows takes whole (two parts
  // with MMAs of their own, so that half of it was free earlier, cost more in
  // short MMAs than they gained: 67 against 62 us for 4096 x 7168 x 4096).
  static constexpr int kSlotRows = kMode == kPair ? kNT / 2 : kNT;
  static constexpr __device__ uint32_t column(int slot, int half) {
    return kMode == kPair ? half * kNT + slot * kSlotRows : (2 * slot + half) * kNT;
  }
  static constexpr size_t kSmem = 1024 + (size_t)kNS * kStage + 8 * kBars + 16 + 128 + (1 + kLists) * 4 * (kMaxGroups + 4);
  static constexpr int kSA = kMode == kPair ? 2 * kNT : 2 * kNT * kNAcc, kSB = kSA + 16;
  static_assert(kMode != kPair || kNAcc == 2, "a pair's slots");
  static_assert(kSB + 8 * kScaleTiles <= 512, "tensor memory");
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kNT % 16 == 0 && kStage % 1024 == 0, "layout");
};

struct Unit {
  int group, row0, count, row_tile;
  bool once;   // the group's only tile of rows: its weights are read once
};

// The units of the CTAs (clusters) of one launch.  Groups with many rows are
// bound by the tensor cores, their weights read from L2 by neighbouring tiles;
// groups with few by HBM.  The two lists are interleaved evenly, so that the
// bounds overlap instead of adding up (each list is group-major, with a
// group's tiles of the same weights as neighbours), and CTA c of n takes one
// unit of every n, another place each time, so that no CTA meets one list
// alone.
struct Units {
  const int* off;        // [groups + 1] row offsets, in range
  const int* start[2];   // [groups + 1] first unit of each group in the list of few (0) and many (1) rows
  int groups, n[2];
  __device__ __forceinline__ int total() const { return n[0] + n[1]; }
  // unit of CTA c of `ctas` in its i-th turn; total() behind the last
  __device__ __forceinline__ int of(int c, int ctas, int i) const {
    if (n[0] == 0 || n[1] == 0) return min(i * ctas + c, total());
    const int p = i * ctas + (c + 17 * i) % ctas;   // a permutation of every full round
    const int q = i * ctas + c;
    return (i + 1) * ctas <= total() ? p : min(q, total());
  }
};

template <int kNT>
__device__ __forceinline__ Unit find_unit(int p, const Units& us) {
  int list = us.n[0] == 0, u = p;
  if (us.n[0] && us.n[1]) {
    const int before = (int)((int64_t)p * us.n[1] / us.total()), upto = (int)((int64_t)(p + 1) * us.n[1] / us.total());
    list = upto > before;
    u = list ? before : p - before;
  }
  const int* s_start = us.start[list];
  int lo = 0, hi = us.groups;           // s_start[lo] <= u < s_start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s_start[mid] <= u) lo = mid; else hi = mid;
  }
  const int count = us.off[lo + 1] - us.off[lo], tiles = (count + kNT - 1) / kNT;
  const int local = u - s_start[lo], t = local % tiles;
  const int per = ((count + tiles - 1) / tiles + 15) & ~15;
  return {lo, us.off[lo] + t * per, min(per, count - t * per), local / tiles, tiles == 1};
}

// Which slot a unit's accumulators take, in turn: the same for the MMA warp and
// the epilogue, which both walk through the units.  A unit that takes a pair's
// both slots counts as a use of each.
template <class C, int kNAcc, bool kTwo>
struct Slots {
  int turn = 0, used[2] = {0, 0};
  struct Plan {
    int slot;
    bool whole;               // a pair's both slots
    uint32_t use0, use1;      // parities of the uses of `slot`, and of the other one if whole
  };
  __device__ __forceinline__ Plan next(int count) {
    Plan p;
    p.whole = kTwo && ((count + 15) & ~15) > C::kSlotRows;
    p.slot = p.whole ? 0 : turn;
    turn = kNAcc == 1 || p.whole ? 0 : turn ^ 1;
    p.use0 = (p.slot ? used[1] : used[0]) & 1;
    p.use1 = used[1] & 1;
    if (p.slot || p.whole) ++used[1];
    if (!p.slot) ++used[0];
    return p;
  }
};

// silu(gate) * up; 0 from about g = -87.3 down, where silu is under 1.1e-36 (the fast division's range ends).  For bf16
// outputs by the fast exponential: within (5 + 1.2 |g|) steps of 2^-23, less than 1/250 of the output's half step.  For
// fp32 outputs by the exact one: within 7 steps of 2^-24 (the exponential 2, the sum 1/2, the division 4, the product 1/2).
template <typename Out>
__device__ __forceinline__ float swiglu(float g, float u) {
  return __fdividef(g, 1.f + (sizeof(Out) == 2 ? __expf(-g) : expf(-g))) * u;
}

// What a lane's bounded wait found, as one answer of the warp: lanes that went on while others gave up would wait for
// them at the next shuffle or tensor-memory load without a bound.
__device__ __forceinline__ bool warp_agrees(bool ok) { return __all_sync(0xffffffffu, ok); }

// Where a thread's accumulators go: lane i of the unit's 128, two accumulators
// each (features 2 i and 2 i + 1, or the gate and up of feature i).
template <bool kPaired, typename Out>
struct Store {
  Out* base;     // this lane's first feature, row 0
  int64_t ld;
  int n;         // features this lane stores: 0, 1 or 2
  bool wide, fast;
  __device__ __forceinline__ Store(const MxProductArgs& a, int i) : ld(a.ld), wide(a.wide_store) {
    const int f = kPaired ? i : 2 * i;
    base = static_cast<Out*>(a.out) + f;
    n = min(max(a.features - f, 0), kPaired ? 1 : 2);
    // whole warps of neighbouring features: lanes pair up (columns16)
    fast = wide && sizeof(Out) == 2 && __all_sync(0xffffffffu, n == (kPaired ? 1 : 2)) && (!kPaired || ld % 2 == 0) &&
           (kPaired || (ld % 4 == 0 && reinterpret_cast<uintptr_t>(a.out) % 8 == 0));
  }
  __device__ __forceinline__ void one(Out* p, float v0, float v1) const {
    if (kPaired) {
      if (n) put(p, swiglu<Out>(v0, v1));
    } else if (n == 2 && wide) {
      put2(p, v0, v1);
    } else {
      if (n) put(p, v0);
      if (n == 2) put(p + 1, v1);
    }
  }
  // 16 columns (rows `row`..) of which `count` are stored; v: both accumulators.
  // Fast: the lanes of a pair trade one of every two rows, so that each stores
  // twice as many neighbouring features of the other (half the stores).
  __device__ __forceinline__ void columns16(int row, int count, const uint32_t* v) const {
    Out* p = base + row * ld;
    if (sizeof(Out) == 2 && fast && count >= 16) {
      const bool odd = threadIdx.x & 1;
      char* q = reinterpret_cast<char*>(p + (odd ? ld - (kPaired ? 1 : 2) : 0));
#pragma unroll
      for (int i = 0; i < 16; i += 2, q += 4 * ld) {
        if (kPaired) {
          const float a = swiglu<Out>(__uint_as_float(v[i]), __uint_as_float(v[16 + i]));
          const float b = swiglu<Out>(__uint_as_float(v[i + 1]), __uint_as_float(v[17 + i]));
          const float c = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
          *reinterpret_cast<uint32_t*>(q) = odd ? bf16x2(c, b) : bf16x2(a, c);
        } else {
          const uint32_t a = bf16x2(__uint_as_float(v[i]), __uint_as_float(v[16 + i]));
          const uint32_t b = bf16x2(__uint_as_float(v[i + 1]), __uint_as_float(v[17 + i]));
          const uint32_t c = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
          *reinterpret_cast<uint2*>(q) = odd ? make_uint2(c, b) : make_uint2(a, c);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i, p += ld)
        if (i < count) one(p, __uint_as_float(v[i]), __uint_as_float(v[16 + i]));
    }
  }
  static __device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
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

template <int kNT, int kNS, int kNAcc, Mode kMode, bool kPaired, typename Out>
__global__ void __launch_bounds__(kThreads, 1) mx_product_kernel(const MxProductArgs a, int cluster) {
  using C = Config<kNT, kNS, kNAcc, kMode>;
  constexpr bool kSplit = kMode == kSplitK, kTwo = kMode == kPair;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + (size_t)kNS * C::kStage);
  uint64_t* empty = full + kNS;
  uint64_t* peer_full = empty + kNS;            // pair, first CTA: the second one's stage
  uint64_t* acc_full = peer_full + kNS;
  uint64_t* acc_empty = acc_full + kNAcc;
  uint64_t* drain = acc_empty + kNAcc;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(drain + 1);
  int* s_warp = reinterpret_cast<int*>(s_tmem + 4);
  int* s_off = s_warp + 32;                     // [groups + 1] row offsets, in range
  int* s_start = s_off + kMaxGroups + 4;        // [2][groups + 1] first unit of each group in either list
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  const int rank = kMode == kSingle ? 0 : (int)ptx::cluster_rank();

  if (tid == 0) {
    // a stage is full with its weights and the copies of every row thread; that
    // the second CTA's is, the first learns on a barrier of its own (on this one
    // its arrivals took longer: 1.17 times the product's time for 4096 tokens of
    // 256 experts, both on one box, before the epilogue was what it is now)
    for (int i = 0; i < kNS; ++i) {
      ptx::mbar_init(&full[i], 1 + kRowWarps * 32);
      ptx::mbar_init(&empty[i], 1);
      ptx::mbar_init(&peer_full[i], 1);
    }
    for (int i = 0; i < kNAcc; ++i) {
      ptx::mbar_init(&acc_full[i], 1);
      ptx::mbar_init(&acc_empty[i], kTwo ? 2 * kEpiWarps : kEpiWarps);
    }
    ptx::mbar_init(drain, 1);
    ptx::fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    if (kTwo) ptx::tmem_alloc_pair(s_tmem, 512);
    else ptx::tmem_alloc(s_tmem, 512);
  }
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  // the groups' rows, kept in 0..n_rows whatever the offsets say
  for (int g = tid; g <= a.groups; g += kThreads)
    s_off[g] = a.offsets ? min(max(__ldg(a.offsets + g), 0), a.n_rows) : g * a.n_rows;
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const int tiles = kTwo ? (a.row_tiles + 1) / 2 : a.row_tiles;   // of weight rows: 512 for a pair
  Units us = {s_off, {s_start, s_start + (C::kLists - 1) * (kMaxGroups + 4)}, a.groups, {0, 0}};
  for (int g0 = 0; g0 < a.groups; g0 += kThreads) {
    const int g = g0 + tid;
    // a group that ends before it starts has no rows
    const int count = g < a.groups ? max(s_off[g + 1] - s_off[g], 0) : 0;
    const int mine = (count + kNT - 1) / kNT * tiles;
#pragma unroll
    for (int l = 0; l < C::kLists; ++l) {
      int total;
      const int before = block_exclusive_scan_1024(l == (C::kLists == 2 && count > kManyRows) ? mine : 0, &total, s_warp);
      if (g < a.groups) s_start[l * (kMaxGroups + 4) + g] = us.n[l] + before;
      us.n[l] += total;
    }
  }
  if (tid < C::kLists) s_start[tid * (kMaxGroups + 4) + a.groups] = us.n[tid];
  __syncthreads();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *s_tmem, 0);
  const int me = blockIdx.x / cluster, n_ctas = gridDim.x / cluster, n_units = us.total();
  // this CTA's (cluster's) i-th unit; with split K it has one
  auto unit_of = [&](int i) { return kSplit ? (i == 0 ? min(me, n_units) : n_units) : us.of(me, n_ctas, i); };
  // a pair: row tile 2 p + rank; one behind the last is computed like it and not stored
  auto row_tile_of = [&](const Unit& un) { return kTwo ? min(2 * un.row_tile + rank, a.row_tiles - 1) : un.row_tile; };
  if (kTwo) {
    __syncwarp();
    ptx::cluster_sync();   // the barriers of both CTAs are set up
  }
  const int k0 = kSplit ? a.kc * rank / cluster : 0, k1 = kSplit ? a.kc * (rank + 1) / cluster : a.kc;
  // Waits for the arrivals of the MMAs' commits on this CTA's barriers: of the last stages (`it` were consumed), which
  // no copy waits for any more, and of the drain behind them.  A pair's first CTA commits for both, and its arrivals
  // in the second are ordered by nothing else: one that came late would land in shared memory of the next CTA there.
  auto settle = [&](int it, uint64_t limit_ns) {
    bool ok = true;
    for (int i = max(it - kNS, 0); i < it; ++i) ok = ptx::mbar_wait(&empty[i % kNS], (i / kNS) & 1, limit_ns) && ok;
    return ptx::mbar_wait(drain, 0, limit_ns) && ok;
  };
  constexpr uint64_t kWait = 2000000000ull;

  if (warp < kRowWarps) {
    // ------------------------------------------------------------ rows of x
    const int64_t pitch = (int64_t)a.kc * 128, spitch = (int64_t)a.kc * 8;
    const int piece = tid & 7;
    int it = 0;
    bool ok = true;
    for (int i = 0, u; ok && (u = unit_of(i)) < n_units; ++i) {
      const Unit un = find_unit<kNT>(u, us);
      // this thread's rows: one 16-byte piece of the codes of rows tid / 8 + 16 j,
      // and the scales of rows tid + 128 j; -1: not a row of x, read as zeros
      // (a pair: this CTA's half of the rows' codes, and the scales of all rows)
      const int half = ((un.count + 15) & ~15) / 2;
      auto row_at = [&](int lr) { return !kTwo ? lr : lr < half ? rank * half + lr : un.count; };
      // (every lookup is made, so that none waits for another)
      auto lookup = [&](int r) { return a.index ? __ldg(a.index + min(un.row0 + r, a.n_rows - 1)) : un.row0 + r; };
      auto row_of = [&](int r, int src) {
        if (r >= un.count) return -2;
        if (a.index_div > 1) src /= a.index_div;
        return (unsigned)src < (unsigned)a.n_x ? src : -1;
      };
      constexpr int kJ = (C::kRows + 15) / 16;
      int rows[kJ], srows[C::kScaleTiles];
#pragma unroll
      for (int j = 0; j < kJ; ++j) rows[j] = lookup(row_at((tid >> 3) + 16 * j));
#pragma unroll
      for (int j = 0; j < C::kScaleTiles; ++j) srows[j] = lookup(tid + 128 * j);
#pragma unroll
      for (int j = 0; j < kJ; ++j) rows[j] = row_of(row_at((tid >> 3) + 16 * j), rows[j]);
#pragma unroll
      for (int j = 0; j < C::kScaleTiles; ++j) srows[j] = row_of(tid + 128 * j, srows[j]);
      for (int k = k0; k < k1; ++k, ++it) {
        const int s = it % kNS;
        if (!ptx::mbar_wait(&empty[s], ((it / kNS) & 1) ^ 1)) {
          atomicOr(&g_mx_err, 1u);
          ok = false;
          break;
        }
        const uint32_t dst = ptx::smem_u32(sm + (size_t)s * C::kStage + kMxBlockBytes);
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
          if (rows[j] == -2) continue;
          const int r = (tid >> 3) + 16 * j;
          ptx::cp_async_16(dst + r * 128 + ((piece ^ (r & 7)) << 4),
                           a.codes + max(rows[j], 0) * pitch + k * 128 + piece * 16, rows[j] >= 0);
        }
        const uint32_t sdst = dst + C::kRowCodes + (tid & 31) * 16 + (tid >> 5) * 4;
#pragma unroll
        for (int j = 0; j < C::kScaleTiles; ++j) {
          if (srows[j] == -2) continue;
          const uint8_t* src = a.scales + max(srows[j], 0) * spitch + k * 8;
          ptx::cp_async_4(sdst + j * 512, src, srows[j] >= 0);
          ptx::cp_async_4(sdst + (C::kScaleTiles + j) * 512, src + 4, srows[j] >= 0);
        }
        ptx::cp_async_arrive(&full[s]);
      }
    }
    ptx::cp_async_commit();
    ptx::cp_async_wait<0>();   // never leave with a copy into shared memory in flight
  } else if (warp == kWeightWarp) {
    // ------------------------------------------------------------ weights
    if (lane == 0) {
      const uint64_t once = ptx::policy_evict_first();
      const bool alone = n_units <= n_ctas;
      ptx::IssueLog log;
      int it = 0;
      bool ok = true;
      for (int i = 0, u; ok && (u = unit_of(i)) < n_units; ++i) {
        const Unit un = find_unit<kNT>(u, us);
        const uint8_t* src = a.image + ((int64_t)un.group * a.row_tiles + row_tile_of(un)) * a.kc * kMxBlockBytes;
        for (int k = k0; k < k1; ++k, ++it) {
          const int s = it % kNS;
          const uint32_t ph = (it / kNS) & 1;
          if (!ptx::mbar_wait(&empty[s], ph ^ 1)) {
            atomicOr(&g_mx_err, 2u);
            ok = false;
            break;
          }
          ptx::mbar_arrive_expect_tx(&full[s], kMxBlockBytes);
          if (un.once)
            ptx::bulk_load_hint(sm + (size_t)s * C::kStage, src + (int64_t)k * kMxBlockBytes, kMxBlockBytes, &full[s], once);
          else
            ptx::bulk_load(sm + (size_t)s * C::kStage, src + (int64_t)k * kMxBlockBytes, kMxBlockBytes, &full[s]);
          log.note(s, ph);
          // a CTA with one unit: the block behind the ring on its way to L2 (one token of 8 experts, 7168 x 4096:
          // 18.8 us against 22.2).  With more units it costs more L2 than it gains.
          if (alone && k + kNS + 1 < k1) ptx::bulk_prefetch(src + (int64_t)(k + kNS + 1) * kMxBlockBytes, kMxBlockBytes);
        }
      }
      // never leave with a copy into shared memory in flight (the stages may miss
      // their rows for good; the copies have landed long before these waits end)
      if (!ok) log.drain(full, kNS);
    }
  } else if (warp == kMmaWarp && kTwo && rank == 1) {
    // ------------------------------------------------------------ pair, second CTA: tell the first of each stage
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int i = 0, u; ok && (u = unit_of(i)) < n_units; ++i)
        for (int k = k0; k < k1; ++k, ++it) {
          const int s = it % kNS;
          const uint32_t ph = (it / kNS) & 1;
          if (!ptx::mbar_wait(&full[s], ph)) {
            atomicOr(&g_mx_err, 16u);
            ok = false;
            break;
          }
          ptx::fence_proxy_async();
          ptx::mbar_arrive_cluster(&peer_full[s], 0);
        }
      // (the first CTA may have to give up on waits of its own before its last commit)
      if (!settle(it, 4 * kWait)) atomicOr(&g_mx_err, 16u);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA (the whole warp; one lane's instructions)
    const uint32_t on = ptx::elect_one();
    const uint32_t ring = ptx::smem_u32(sm);
    using S = Slots<C, kNAcc, kTwo>;
    S slots;
    int s = 0, n = 0, it = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int u; ok && (u = unit_of(n)) < n_units; ++n) {
      const Unit un = find_unit<kNT>(u, us);
      const typename S::Plan pl = slots.next(un.count);
      const int N = __shfl_sync(0xffffffffu, (un.count + 15) & ~15, 0), slot = __shfl_sync(0xffffffffu, pl.slot, 0);
      constexpr int kM = kTwo ? 256 : 128;
      const uint32_t id0 = ptx::umma_idesc_mxf4(kM, N, 0), id1 = ptx::umma_idesc_mxf4(kM, N, 1);
      const uint32_t d0 = tmem + C::column(slot, 0), d1 = tmem + C::column(slot, 1);
      ok = warp_agrees(ptx::mbar_wait(&acc_empty[slot], pl.use0 ^ 1) &&
                       (!pl.whole || ptx::mbar_wait(&acc_empty[1], pl.use1 ^ 1)));
      ptx::tc_fence_after();
      for (int k = k0; k < k1 && ok; ++k) {
        ok = warp_agrees(ptx::mbar_wait(&full[s], ph) && (!kTwo || ptx::mbar_wait(&peer_full[s], ph)));
        if (!ok) break;
        ptx::fence_proxy_async();   // the rows came through the generic proxy
        ptx::tc_fence_after();
        const uint32_t st = ring + s * C::kStage, rows = st + kMxBlockBytes;
        const uint64_t wd = ptx::umma_desc_sw128(st), rd = ptx::umma_desc_sw128(rows);
        const uint64_t wsd = ptx::scales_desc(st + 2 * kMxHalfCodes);
        const uint64_t rsd = ptx::scales_desc(rows + C::kRowCodes);
        // scale columns: A half h, 128 of K c: kSA + 4 (2 h + c); B: kSB + 4 (c tiles + j)
#pragma unroll
        for (int i = 0; i < 4; ++i) ptx::tmem_copy_scales<kTwo>(on, tmem + C::kSA + 4 * i, wsd + 32 * i);
#pragma unroll
        for (int i = 0; i < 2 * C::kScaleTiles; ++i)
          if (C::kScaleTiles == 1 || i % 2 == 0 || N > 128) ptx::tmem_copy_scales<kTwo>(on, tmem + C::kSB + 4 * i, rsd + 32 * i);
#pragma unroll
        for (int q = 0; q < 4; ++q) {   // 64 of K each, 32 bytes of a row
          const uint32_t id = q & 1 ? id1 : id0, c = q >> 1;
          const uint32_t sb = tmem + C::kSB + 4 * C::kScaleTiles * c;
          const bool add = k > k0 || q > 0;
          ptx::umma_mxf4<kTwo>(on, d0, wd + 2 * q, rd + 2 * q, id, tmem + C::kSA + 4 * c, sb, add);
          ptx::umma_mxf4<kTwo>(on, d1, wd + kMxHalfCodes / 16 + 2 * q, rd + 2 * q, id, tmem + C::kSA + 8 + 4 * c, sb, add);
        }
        ptx::umma_commit_on<kTwo>(on, &empty[s]);
        ++it;
        if (++s == kNS) {
          s = 0;
          ph ^= 1;
        }
      }
      if (ok) {
        ptx::umma_commit_on<kTwo>(on, &acc_full[slot]);
        if (pl.whole) ptx::umma_commit_on<kTwo>(on, &acc_full[1]);
      } else if (on) {
        atomicOr(&g_mx_err, 4u);
      }
    }
    // wait for every MMA this warp issued before TMEM is released
    ptx::umma_commit_on<kTwo>(on, drain);
    if (!settle(it, kWait) && on) atomicOr(&g_mx_err, 4u);
  } else if (warp >= kFirstEpi) {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3, sub = (warp - kFirstEpi) >> 2;   // TMEM lane quarter; which 16-column chunks
    const int lrow = quarter * 32 + lane;
    Slots<C, kNAcc, kTwo> slots;
    using S = Slots<C, kNAcc, kTwo>;
    bool ok = true;
    for (int n = 0, u; ok && (u = unit_of(n)) < n_units; ++n) {
      const Unit un = find_unit<kNT>(u, us);
      const typename S::Plan pl = slots.next(un.count);
      const bool behind = kTwo && 2 * un.row_tile + rank >= a.row_tiles;
      const Store<kPaired, Out> store(a, row_tile_of(un) * 128 + lrow);
      // (both slots of a whole unit: the second one's parity is asked again by the unit after next, and a phase that had
      // not ended by then would look like the one before it)
      ok = warp_agrees(ptx::mbar_wait_sleep(&acc_full[pl.slot], pl.use0, 100) &&
                       (!pl.whole || ptx::mbar_wait_sleep(&acc_full[1], pl.use1, 100)));
      if (!ok) {
        atomicOr(&g_mx_err, 8u);
        break;
      }
      ptx::tc_fence_after();
      const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
      const uint32_t t0 = tmem + C::column(pl.slot, 0) + lanes, t1 = tmem + C::column(pl.slot, 1) + lanes;
      {
        // 16 columns at a time, the next ones on their way
        constexpr int kStride = 16 * (kEpiWarps / 4);
        uint32_t v[2][32];
        auto load = [&](int c, uint32_t* w) {
          ptx::tmem_ld16(t0 + c, w);
          ptx::tmem_ld16(t1 + c, w + 16);
        };
        auto take = [&](int c, const uint32_t* w) {
          if (kSplit) {
            // the ring is free: every copy of this CTA's one unit has been consumed
            float* part_sums = reinterpret_cast<float*>(sm);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (c + i < un.count) {
                part_sums[(c + i) * 256 + lrow] = __uint_as_float(w[i]);
                part_sums[(c + i) * 256 + 128 + lrow] = __uint_as_float(w[16 + i]);
              }
          } else if (!behind) {
            store.columns16(un.row0 + c, un.count - c, w);
          }
        };
        int c = 16 * sub;
        if (c < un.count) load(c, v[0]);
        while (c < un.count) {
          ptx::tmem_wait_ld(v[0]);
          if (c + kStride < un.count) load(c + kStride, v[1]);
          take(c, v[0]);
          c += kStride;
          if (c >= un.count) break;
          ptx::tmem_wait_ld(v[1]);
          if (c + kStride < un.count) load(c + kStride, v[0]);
          take(c, v[1]);
          c += kStride;
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (kTwo) ptx::mbar_arrive_cluster(&acc_empty[pl.slot], 0);
          else ptx::mbar_arrive(&acc_empty[pl.slot]);
          if (pl.whole) ptx::mbar_arrive_cluster(&acc_empty[1], 0);
        }
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (kTwo) {
    __syncwarp();
    ptx::cluster_sync();   // no CTA leaves while the other reads its memory or arrives on its barriers
  }
  if (kSplit) {
    __syncwarp();
    ptx::cluster_sync();
    if (me < n_units) {
      // rows rank, rank + cluster, ... of the unit, the parts added in rank order
      const Unit un = find_unit<kNT>(blockIdx.x / cluster, us);
      const int i = tid & 127;
      const Store<kPaired, Out> store(a, un.row_tile * 128 + i);
      for (int c = rank + cluster * (tid >> 7); c < un.count; c += cluster * (kThreads >> 7)) {
        const uint32_t at = ptx::smem_u32(sm) + (c * 256 + i) * 4;
        float v0 = 0.f, v1 = 0.f;
        for (int r = 0; r < cluster; ++r) {
          v0 += ptx::ld_cluster_f32(at, r);
          v1 += ptx::ld_cluster_f32(at + 512, r);
        }
        store.one(store.base + (un.row0 + c) * store.ld, v0, v1);
      }
    }
    __syncwarp();          // the rows' loop leaves a warp's lanes apart, and the barrier takes whole warps
    ptx::cluster_sync();   // no CTA leaves while its part is read
  }
  if (warp == kMmaWarp) {
    __syncwarp();
    ptx::tc_fence_after();
    if (kTwo) ptx::tmem_dealloc_pair(tmem, 512);
    else ptx::tmem_dealloc(tmem, 512);
  }
}

template <int kNT, int kNS, int kNAcc, Mode kMode, bool kPaired, typename Out>
cudaError_t launch_as(const MxProductArgs& a, int cluster, int clusters, cudaStream_t st) {
  using C = Config<kNT, kNS, kNAcc, kMode>;
  static_assert(kMode != kSplitK || kNT * 256 * 4 <= kNS * C::kStage, "partial sums fit the ring");
  auto* kernel = mx_product_kernel<kNT, kNS, kNAcc, kMode, kPaired, Out>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
  if (e != cudaSuccess) return e;
  return launch_dependent(kernel, dim3((unsigned)(clusters * cluster)), dim3(kThreads), C::kSmem, st, cluster, a, cluster);
}

template <int kNT, int kNS, int kNAcc, Mode kMode>
cudaError_t launch(const MxProductArgs& a, int cluster, int clusters, cudaStream_t st) {
  const bool f32 = a.out_type == kF32;
  if (a.paired)
    return f32 ? launch_as<kNT, kNS, kNAcc, kMode, true, float>(a, cluster, clusters, st)
               : launch_as<kNT, kNS, kNAcc, kMode, true, __nv_bfloat16>(a, cluster, clusters, st);
  return f32 ? launch_as<kNT, kNS, kNAcc, kMode, false, float>(a, cluster, clusters, st)
             : launch_as<kNT, kNS, kNAcc, kMode, false, __nv_bfloat16>(a, cluster, clusters, st);
}

// Clusters of so many CTAs of the split-K kernel that the GPU holds at a time
// (its processors come in groups that a cluster cannot span: fewer than SMs /
// cluster), looked up once per device.
int clusters_at_once(int cluster) {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> known[kMaxDevices][9];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  int n = known[dev][cluster].load(std::memory_order_relaxed);
  if (n == 0) {
    using C = Config<64, 5, 2, kSplitK>;
    auto* kernel = mx_product_kernel<64, 5, 2, kSplitK, false, float>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(sm_count() / cluster * cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
      (void)cudaGetLastError();
      return 0;
    }
    known[dev][cluster].store(n, std::memory_order_relaxed);
  }
  return n;
}

}  // namespace

cudaError_t launch_mx_product(MxProductArgs a, cudaStream_t st) {
  const int sms = sm_count();
  a.wide_store = a.ld % 2 == 0 && reinterpret_cast<uintptr_t>(a.out) % (2 * type_bytes(a.out_type)) == 0;
  // Many rows: pairs with tiles of up to 240 of them; fewer: tiles of 64, one CTA each, which are more units.  Pairs
  // against single CTAs, us: 4096 tokens of 8 of 256 groups, 7168 x 4096, 777 and 929; one group, 2048 x 7168: 4096 rows
  // 44..53 and 55..62, 2048 rows 25 and 33, 1100 rows 16 and 18, 512 rows 13 and 11.  The rule goes by the rows alone: few
  // features leave pairs without units (one group of 4096 rows, 2048 x 1024: 13.5 and 11.2, 2048 x 512: 13.1 and 7.4).
  if (a.n_rows > 1024 && a.row_tiles > 1) return launch<240, 4, 2, kPair>(a, 2, sms / 2, st);
  // at most this many units (up to 64 rows are one tile of any group)
  const int64_t units = (int64_t)std::min(a.n_rows <= 64 ? a.groups : a.groups + a.n_rows / 64, a.n_rows) * a.row_tiles;
  int cluster = 1;
  // in one wave (16 clusters of 8 are two: 7168 x 4096, one row, 12.6 us; 7.2 us in 16 of 4, 11.6 without clusters)
  if (a.n_rows <= 64 && units * 2 <= sms)
    for (int c = 8; c > 1 && cluster == 1; c /= 2)
      if (a.kc >= c * 2 && units <= clusters_at_once(c)) cluster = c;
  if (cluster > 1) return launch<64, 5, 2, kSplitK>(a, cluster, (int)units, st);
  return launch<64, 5, 2, kSingle>(a, 1, (int)std::min<int64_t>(units, sms), st);
}

cudaError_t mx_product_errors(unsigned* flags) {
  cudaError_t e = cudaMemcpyFromSymbol(flags, g_mx_err, sizeof(unsigned));
  const unsigned zero = 0;
  if (e == cudaSuccess && *flags) e = cudaMemcpyToSymbol(g_mx_err, &zero, sizeof(unsigned));
  return e;
}

}  // namespace moe
