// Matrix products on the 5th-generation tensor cores (mm.h), for operands whose
// rows are whole 16-byte vectors.
//
// One layout serves the three products: a tile of the result has 256 features f
// (the contiguous index of the output) in the lanes of tensor memory and up to
// 256 rows c in its columns, so
//   - the ragged side (an expert's rows) is the N extent of the MMA, which may
//     be any multiple of 32: a short range costs what it has, not a whole tile;
//   - a thread of the epilogue owns one feature, so bias and store addresses
//     are uniform along its registers and a warp stores 64 contiguous bytes.
// A pair of CTAs (a cluster of two SMs) computes one tile with cta_group::2:
// each holds 128 features of A and half of the rows of B, 64 deep per stage, so
// a stage moves 32 KB into each SM for 128 x 256 x 64 products.  Operands come
// by tensor copies into 128-byte-swizzled stages; accumulators are double
// buffered in tensor memory, so the epilogue of a tile runs under the products of
// the next one.
//
// An expert's rows lie in one range per source.  They are taken as one virtual
// row space in which every range is padded to a multiple of 8, the height of a
// swizzle atom; 8 aligned rows in a row of groups that are contiguous in memory
// are fetched by one 64-row copy, others by 8-row copies.  Padding rows hold a
// neighbour's data: in the forward product and the data gradient they are columns
// that are not stored; in the weight gradient, where rows are summed over, they
// are overwritten with zeros in shared memory before the MMA reads them.
//
// Warps of a CTA: 0 tensor copies, 1 MMA (of the pair's first CTA), 2 tensor
// memory and the zeroing, 4-11 epilogue.  Every wait is bounded: a wait that runs
// out sets bit 2 of the status, and all roles leave.
#include <atomic>
#include <cstdlib>
#include <cstring>

#include <cuda.h>

#include "mm.h"
#include "ptx_async.cuh"

namespace hoc {
namespace {

constexpr int kTcThreads = 384;
constexpr int kTcEpilogue = 8;                  // warps: two to each 32 lanes of tensor memory
constexpr int kTcColumns = 16;                  // accumulator columns of an epilogue step
constexpr int kTcStages = 6;
constexpr int kTcDepth = 64;                    // contraction elements of a stage: one 128-byte swizzled row
constexpr uint32_t kTcOperand = 128 * 128;      // bytes of one operand of a stage in one CTA
constexpr uint32_t kTcStage = 2 * kTcOperand;
constexpr int kTcFeatures = 256;                // of a pair's tile
constexpr int kTcRows = 256;                    // at most, of a tile
constexpr uint32_t kTcTmemColumns = 512;        // two accumulators of 256 columns
constexpr uint64_t kTcWaitNs = 2000000000ull;

struct TcParams {
  MmParams P;
  int tile_rows;     // forward, dgrad: rows of a tile, a multiple of 32
  uint32_t tx_pad;   // bytes that the copies' barriers expect beyond their loads (0; 16 under HOC_FAULT=mm_stall)
  uint64_t wait_ns;
  CUtensorMap w[kMaxRanks];                      // forward, dgrad
  CUtensorMap row64[kMaxRanks], row8[kMaxRanks]; // P.rows in boxes of 64 and 8 rows
  CUtensorMap dy64[kMaxRanks], dy8[kMaxRanks];   // wgrad
};

struct TcShared {
  uint64_t full[kTcStages];   // on the first CTA: both CTAs' loads of a stage
  uint64_t part[kTcStages];   // wgrad: this CTA's loads of a stage that holds padding rows
  uint64_t empty[kTcStages];
  uint64_t acc_full[2];
  uint64_t acc_empty[2];      // on the first CTA: the epilogue warps of both CTAs
  uint32_t tmem;
  volatile int dead;
  int vrows[kMmMaxGroups];
  unsigned tile0[kMmMaxGroups + 1];
};
constexpr size_t kTcSmem = 1024 + size_t(kTcStages) * kTcStage + sizeof(TcShared);

// ------------------------------------------------------------------ PTX
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address, in the cluster's shared memory, of the first CTA's copy of a local barrier.
__device__ __forceinline__ uint32_t on_first(const uint64_t* bar) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(ptx::smem_addr(bar)));
  return a;
}
__device__ __forceinline__ void arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// Announces `tx` bytes of copies.  Relaxed: nothing this thread wrote is handed
// over, and a release to the cluster made every stage wait for about 1000 cycles.
__device__ __forceinline__ void arrive_expect_cluster(uint32_t addr, uint32_t tx) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(addr), "r"(tx)
               : "memory");
}
// The same where only tensor memory, ordered by the tcgen05 fences, is handed over.
__device__ __forceinline__ void arrive_relaxed(uint32_t addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// Waits for the phase with `parity`; false when the limit passed here or in
// another role, after which the caller leaves its loop.
__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity, const TcParams& T, TcShared* S) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t deadline = ptx::global_ns() + T.wait_ns;
  while (!ptx::mbar_try_wait(bar, parity)) {
    if (S->dead) return false;
    if (ptx::global_ns() > deadline) {
      atomicOr(T.P.status, 4);
      S->dead = 1;
      return false;
    }
  }
  return true;
}
// The same by a whole warp, with one answer for all lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const TcParams& T, TcShared* S) {
  return __all_sync(0xFFFFFFFFu, wait_bounded(bar, parity, T, S));
}
// Tensor copies; the barrier may be the pair's other CTA's.
__device__ __forceinline__ void copy2(uint32_t dst, const CUtensorMap* m, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%3, "
      "%4}], [%2];" ::"r"(dst), "l"(m), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void copy3(uint32_t dst, const CUtensorMap* m, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%3, "
      "%4, %5}], [%2];" ::"r"(dst), "l"(m), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void copy5(uint32_t dst, const CUtensorMap* m, int x, int a, int b, int c, int d,
                                      uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%3, "
      "%4, %5, %6, %7}], [%2];" ::"r"(dst), "l"(m), "r"(bar), "r"(x), "r"(a), "r"(b), "r"(c), "r"(d)
      : "memory");
}
// Shared-memory operand descriptor, 128-byte swizzle; lbo and sbo in bytes.
// K-major: sbo is the distance of 8-row groups.  M/N-major: sbo is the distance
// of 8-deep groups along the contraction, lbo that of 64-element blocks.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return uint64_t((addr >> 4) & 0x3FFF) | (uint64_t((lbo >> 4) & 0x3FFF) << 16) | (uint64_t((sbo >> 4) & 0x3FFF) << 32) |
         (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(add)
      : "memory");
}
// Arrives on both CTAs' copy of `bar` when the MMAs issued so far are done.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          ptx::smem_addr(bar)),
      "h"(uint16_t(3))
      : "memory");
}
__device__ __forceinline__ void tmem_load(uint32_t (&r)[kTcColumns], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// ------------------------------------------------------------------ tiles
// A tile of the launch, as every role derives it for itself.
struct Tile {
  int p, g;     // rank buffer, expert
  int f0;       // first feature
  int c0, n;    // first row (virtual row; wgrad: out feature) and the MMA's N
  int steps;    // stages of the contraction
};

template <int MODE>
__device__ __forceinline__ Tile tile_at(const TcParams& T, const TcShared* S, unsigned t) {
  const MmParams& P = T.P;
  const int i = mm_find(S->tile0, P.parts * P.groups, t);
  Tile A;
  A.p = P.part0 + i / P.groups;
  A.g = P.group0 + i % P.groups;
  const unsigned lt = t - S->tile0[i];
  const int rows = S->vrows[i];
  const int per = MODE == kWgrad ? kTcRows : T.tile_rows, extent = MODE == kWgrad ? P.out : rows;
  const unsigned ctiles = (extent + per - 1) / per;
  const bool gated = MODE == kForward && P.act == HOC_ACT_SWIGLU;
  A.f0 = int(lt / ctiles) * (gated ? kTcFeatures / 2 : kTcFeatures);
  A.c0 = int(lt % ctiles) * per;
  A.n = (min(per, extent - A.c0) + 31) / 32 * 32;
  A.steps = ((MODE == kForward ? P.in : MODE == kDgrad ? P.out : rows) + kTcDepth - 1) / kTcDepth;
  return A;
}

// The ranges of one expert, one source per lane (reloaded 32 at a time where there are more).
struct Ranges {
  int64_t lo;
  int64_t n;
};
__device__ __forceinline__ Ranges load_ranges(const MmParams& P, int p, int g, int base) {
  const int s = base + int(threadIdx.x & 31);
  Ranges R{0, 0};
  if (s < (P.seg ? P.sources : 1)) mm_range(P, p, g, s, R.lo, R.n);
  return R;
}
// Each lane's group of 8 virtual rows at `v` (a multiple of 8): its first row in
// the buffer and how many rows its range has from there on (0: past the end).
// The whole warp calls it; R holds the first 32 sources' ranges.
__device__ __forceinline__ void group_at(const MmParams& P, int p, int g, Ranges R, int v, int& row, int& left) {
  const int ns = P.seg ? P.sources : 1;
  int64_t at = v;
  bool found = false;
  row = int(P.cap[p]);
  left = 0;
  for (int base = 0; base < ns; base += 32) {
    if (ns > 32) R = load_ranges(P, p, g, base);
    const int m = min(32, ns - base);
    for (int j = 0; j < m; ++j) {
      const int64_t lo = __shfl_sync(0xFFFFFFFFu, R.lo, j), n = __shfl_sync(0xFFFFFFFFu, R.n, j);
      const int64_t padded = (n + 7) & ~int64_t(7);
      if (!found && at < padded) {
        found = true;
        row = int(lo + at);
        left = int(n - at);
      }
      at -= padded;
    }
  }
}

// wgrad: the 64 virtual rows of stage s, a group of 8 per lane modulo 8.
// Returns (to all lanes) how many stages from s on are 64 rows each of the range
// that stage s begins in, without padding; 0 when stage s is not.
__device__ __forceinline__ int stage_rows(const MmParams& P, const Tile& A, const Ranges& R, int s, int& row,
                                          int& valid) {
  int left;
  group_at(P, A.p, A.g, R, s * kTcDepth + int(threadIdx.x & 7) * 8, row, left);
  valid = min(left, 8);
  return __shfl_sync(0xFFFFFFFFu, left, 0) / kTcDepth;
}

// ------------------------------------------------------------------ epilogue
template <int ACT>
struct ActTag {
  static constexpr int act = ACT;
};
// f(ActTag<act>) with the activation as a constant.
template <class F>
__device__ __forceinline__ void with_act(int act, F f) {
  switch (act) {
    case HOC_ACT_RELU: f(ActTag<HOC_ACT_RELU>{}); break;
    case HOC_ACT_GELU: f(ActTag<HOC_ACT_GELU>{}); break;
    case HOC_ACT_SILU: f(ActTag<HOC_ACT_SILU>{}); break;
    case HOC_ACT_SWIGLU: f(ActTag<HOC_ACT_SWIGLU>{}); break;
    default: f(ActTag<HOC_ACT_NONE>{}); break;
  }
}

// What the epilogue reads beside the accumulator for a step's columns: the residual,
// the pre-activation of the layer below, or the weights to add to.  Loaded one
// step ahead, so that its latency passes under other work.
struct Beside {
  uint32_t a[kTcColumns], b[kTcColumns];  // bf16 bits, or (wgrad, binary32 weights) floats
};

__device__ __forceinline__ uint32_t bits_of(const __nv_bfloat16* p) {
  return *reinterpret_cast<const uint16_t*>(p);
}
__device__ __forceinline__ float float_of(uint32_t bf16_bits) { return __uint_as_float(bf16_bits << 16); }

// Loads are unconditional, at places clamped to the tensors (values of rows or
// features that do not exist are never used): predicated ones made the compiler
// wait for each before it issued the next.
template <int MODE, int ACT>
__device__ __forceinline__ void load_beside(const MmParams& P, const Tile& A, int col, int f, int row, int valid,
                                            Beside& B) {
  if (col >= A.n) return;
  const bool upper = (threadIdx.x & 31) >= 16;
  const int fc = min(f, (MODE == kForward ? P.out : P.in) - 1);
  if constexpr (MODE == kWgrad) {
    if (!P.accumulate) return;
    const int64_t first = int64_t(A.g) * P.out * P.in + fc;
    if (P.out_f32) {
#pragma unroll
      for (int j = 0; j < kTcColumns; ++j)
        B.a[j] = __float_as_uint(
            static_cast<const float*>(P.y[A.p])[first + int64_t(min(A.c0 + col + j, P.out - 1)) * P.in]);
    } else {
#pragma unroll
      for (int j = 0; j < kTcColumns; ++j)
        B.a[j] = bits_of(static_cast<const __nv_bfloat16*>(P.y[A.p]) + first +
                         int64_t(min(A.c0 + col + j, P.out - 1)) * P.in);
    }
  } else if constexpr (MODE == kForward) {
    if (!P.res[A.p]) return;
#pragma unroll
    for (int q = 0; q < (ACT == HOC_ACT_SWIGLU ? 1 : 2); ++q) {
      const int gi = (col >> 3) + q + (ACT == HOC_ACT_SWIGLU && upper ? 1 : 0);
      const int r0 = __shfl_sync(0xFFFFFFFFu, row, gi & 31), nv = __shfl_sync(0xFFFFFFFFu, valid, gi & 31);
      const __nv_bfloat16* at = P.res[A.p] + int64_t(nv ? r0 : 0) * P.ld_res + fc;
#pragma unroll
      for (int j = 0; j < 8; ++j) B.a[q * 8 + j] = bits_of(at + (j < nv ? j * P.ld_res : 0));
    }
  } else if constexpr (ACT != HOC_ACT_NONE) {
    const int64_t ld = int64_t(P.in) * (ACT == HOC_ACT_SWIGLU ? 2 : 1);
#pragma unroll
    for (int q = 0; q < kTcColumns / 8; ++q) {
      const int gi = (col >> 3) + q;
      const int r0 = __shfl_sync(0xFFFFFFFFu, row, gi & 31), nv = __shfl_sync(0xFFFFFFFFu, valid, gi & 31);
      const __nv_bfloat16* at = P.pre[A.p] + int64_t(nv ? r0 : 0) * ld + fc;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t off = j < nv ? j * ld : 0;
        B.a[q * 8 + j] = bits_of(at + off);
        if (ACT == HOC_ACT_SWIGLU) B.b[q * 8 + j] = bits_of(at + off + P.in);
      }
    }
  }
}

// A step's columns of the accumulator: v[j] is feature `f` (of this lane) and column
// col + j; row and valid name the groups of 8 columns of the tile, one per lane.
template <int MODE, int ACT>
__device__ __forceinline__ void store_columns(const MmParams& P, const Tile& A, const uint32_t (&v)[kTcColumns], int col, int f,
                                              int row, int valid, float bias, const Beside& B) {
  constexpr bool gated = MODE == kForward && ACT == HOC_ACT_SWIGLU;
  if constexpr (MODE == kWgrad) {  // columns are out features
    if (f >= P.in) return;
    const int64_t first = (int64_t(A.g) * P.out + A.c0 + col) * P.in + f;
    const int m = min(kTcColumns, P.out - (A.c0 + col));
#pragma unroll
    for (int j = 0; j < kTcColumns; ++j)
      if (j < m) {
        float x = __uint_as_float(v[j]);
        if (P.out_f32) {
          if (P.accumulate) x += __uint_as_float(B.a[j]);
          static_cast<float*>(P.y[A.p])[first + int64_t(j) * P.in] = x;
        } else {
          if (P.accumulate) x += float_of(B.a[j]);
          static_cast<__nv_bfloat16*>(P.y[A.p])[first + int64_t(j) * P.in] = __float2bfloat16_rn(x);
        }
      }
  } else {
    const int width = MODE == kForward ? P.out : P.in;
    const bool mine = f < width;
    const int64_t wide = int64_t(P.out) * (gated ? 2 : 1);
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(P.y[A.p]);
    __nv_bfloat16* keep = static_cast<__nv_bfloat16*>(P.pre_out[A.p]);
    const bool res = MODE == kForward && P.res[A.p] != nullptr;
    if constexpr (gated) {
      // Lanes 0-15 hold the gates of 16 features, lanes 16-31 their values.  They
      // swap halves: each then has both for 8 of the 16 columns.
      const bool upper = (threadIdx.x & 31) >= 16;
      if (keep)
#pragma unroll
        for (int q = 0; q < kTcColumns / 8; ++q) {
          const int gi = (col >> 3) + q;
          const int r0 = __shfl_sync(0xFFFFFFFFu, row, gi & 31), nv = __shfl_sync(0xFFFFFFFFu, valid, gi & 31);
          __nv_bfloat16* at = keep + int64_t(r0) * wide + (upper ? P.out : 0) + f;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < nv && mine) at[j * wide] = __float2bfloat16_rn(__uint_as_float(v[q * 8 + j]) + bias);
        }
      const int gi = (col >> 3) + (upper ? 1 : 0);
      const int r0 = __shfl_sync(0xFFFFFFFFu, row, gi & 31), nv = __shfl_sync(0xFFFFFFFFu, valid, gi & 31);
      __nv_bfloat16* at = y + int64_t(r0) * P.ld_y + f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float other = __shfl_xor_sync(0xFFFFFFFFu, __uint_as_float(upper ? v[j] : v[8 + j]) + bias, 16);
        const float own = __uint_as_float(upper ? v[8 + j] : v[j]) + bias;
        float o = mm_act(HOC_ACT_SILU, upper ? other : own) * (upper ? own : other);
        if (res) o += float_of(B.a[j]);
        if (j < nv && mine) at[j * P.ld_y] = __float2bfloat16_rn(o);
      }
    } else {
#pragma unroll
      for (int q = 0; q < kTcColumns / 8; ++q) {
        const int gi = (col >> 3) + q;
        const int r0 = __shfl_sync(0xFFFFFFFFu, row, gi & 31), nv = __shfl_sync(0xFFFFFFFFu, valid, gi & 31);
        __nv_bfloat16* at = y + int64_t(r0) * P.ld_y + f;
        __nv_bfloat16* ak = keep + int64_t(r0) * wide + f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (j >= nv || !mine) continue;
          float x = __uint_as_float(v[q * 8 + j]);
          if (MODE == kForward) {
            x += bias;
            if (keep) ak[j * wide] = __float2bfloat16_rn(x);
            x = mm_act(ACT, x);
            if (res) x += float_of(B.a[q * 8 + j]);
            at[j * P.ld_y] = __float2bfloat16_rn(x);
          } else if (ACT == HOC_ACT_SWIGLU) {
            const float g = float_of(B.a[q * 8 + j]);
            at[j * P.ld_y] = __float2bfloat16_rn(x * float_of(B.b[q * 8 + j]) * mm_act_slope(HOC_ACT_SILU, g));
            at[j * P.ld_y + P.in] = __float2bfloat16_rn(x * mm_act(HOC_ACT_SILU, g));
          } else {
            at[j * P.ld_y] =
                __float2bfloat16_rn(ACT == HOC_ACT_NONE ? x : x * mm_act_slope(ACT, float_of(B.a[q * 8 + j])));
          }
        }
      }
    }
  }
}

// ------------------------------------------------------------------ kernel
template <int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kTcThreads, 1)
    mm_tc_kernel(const __grid_constant__ TcParams T) {
  extern __shared__ unsigned char raw[];
  const uint32_t base = (ptx::smem_addr(raw) + 1023u) & ~1023u;
  unsigned char* stages = raw + (base - ptx::smem_addr(raw));
  TcShared* S = reinterpret_cast<TcShared*>(stages + size_t(kTcStages) * kTcStage);
  const MmParams& P = T.P;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = int(cta_rank());
  const bool gated = MODE == kForward && P.act == HOC_ACT_SWIGLU;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kTcStages; ++s) {
      ptx::mbar_init(&S->full[s], 2);
      ptx::mbar_init(&S->part[s], 1);
      ptx::mbar_init(&S->empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(&S->acc_full[a], 1);
      ptx::mbar_init(&S->acc_empty[a], 2 * kTcEpilogue);
    }
    S->dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(ptx::smem_addr(&S->tmem)),
                 "r"(kTcTmemColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int fcount = MODE == kForward ? P.out : P.in;
  const int ftile = gated ? kTcFeatures / 2 : kTcFeatures;
  const unsigned ftiles = (fcount + ftile - 1) / ftile;
  mm_count(P, 8, S->vrows, S->tile0, [&](int rows) {
    const int per = MODE == kWgrad ? kTcRows : T.tile_rows, extent = MODE == kWgrad ? P.out : rows;
    return unsigned((extent + per - 1) / per) * ftiles;
  });
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  cluster_sync();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = S->tmem;
  const unsigned tiles = S->tile0[P.parts * P.groups];
  const unsigned first = blockIdx.x >> 1, stride = gridDim.x >> 1;

  if (warp == 0) {
    // ---- tensor copies.  The loop over a tile's stages runs on one lane
    // wherever the rows of a stage are contiguous (a warp whose lanes issue copies
    // in turn took 830 cycles a stage, more than the 512 of its MMAs).
    const uint32_t full0 = on_first(&S->full[0]);
    uint32_t k = 0;  // stages filled
    bool ok = true;
    for (unsigned t = first; ok && t < tiles; t += stride) {
      const Tile A = tile_at<MODE>(T, S, t);
      const Ranges R = load_ranges(P, A.p, A.g, 0);
      const int half = A.n / 2;  // rows of B in this CTA (wgrad: features)
      const int blocks = (half + 63) / 64;
      const int fa = A.f0 + rank * (gated ? 64 : 128);
      auto weights = [&](uint32_t a, int x, uint32_t bar) {
        if (MODE == kDgrad) {
          copy3(a, &T.w[A.p], fa, x, A.g, bar);
          copy3(a + 8192u, &T.w[A.p], fa + 64, x, A.g, bar);
        } else if (gated) {
          copy5(a, &T.w[A.p], x, 0, 0, fa / 16, A.g, bar);
        } else {
          copy3(a, &T.w[A.p], x, fa, A.g, bar);
        }
      };
      if (MODE != kWgrad) {
        int row, left;
        group_at(P, A.p, A.g, R, A.c0 + rank * half + lane * 8, row, left);
        const int start = __shfl_sync(0xFFFFFFFFu, row, lane & ~7);
        // 64-row blocks whose groups, as far as they hold rows, follow one another in the buffer
        const unsigned broken = __ballot_sync(0xFFFFFFFFu, lane * 8 < half && left > 0 && row != start + (lane & 7) * 8);
        const int row1 = __shfl_sync(0xFFFFFFFFu, row, 8);
        if (!broken) {
          if (lane == 0) {
            const uint32_t bytes = kTcOperand + uint32_t(blocks) * 8192u + T.tx_pad;
            for (int s = 0; s < A.steps; ++s, ++k) {
              const uint32_t st = k % kTcStages, round = k / kTcStages;
              if (round && !wait_bounded(&S->empty[st], (round - 1) & 1, T, S)) {
                ok = false;
                break;
              }
              const uint32_t a = base + st * kTcStage, bar = full0 + st * 8u;
              arrive_expect_cluster(bar, bytes);
              weights(a, s * kTcDepth, bar);
              copy2(a + kTcOperand, &T.row64[A.p], s * kTcDepth, row, bar);
              if (blocks > 1) copy2(a + kTcOperand + 8192u, &T.row64[A.p], s * kTcDepth, row1, bar);
            }
          }
        } else {
          for (int s = 0; s < A.steps; ++s, ++k) {
            const uint32_t st = k % kTcStages, round = k / kTcStages;
            if (round && !warp_wait(&S->empty[st], (round - 1) & 1, T, S)) {
              ok = false;
              break;
            }
            const uint32_t a = base + st * kTcStage, bar = full0 + st * 8u;
            if (lane == 0) {
              arrive_expect_cluster(bar, kTcOperand + uint32_t(half) * 128u + T.tx_pad);
              weights(a, s * kTcDepth, bar);
            }
            __syncwarp();
            if (lane * 8 < half)
              copy2(a + kTcOperand + uint32_t(lane) * 1024u, &T.row8[A.p], s * kTcDepth, row, bar);
            __syncwarp();
          }
        }
        k = __shfl_sync(0xFFFFFFFFu, k, 0);
        ok = __shfl_sync(0xFFFFFFFFu, int(ok), 0);
      } else {
        const uint32_t bytes = kTcOperand + uint32_t(blocks) * 8192u + T.tx_pad;
        for (int s = 0; ok && s < A.steps;) {
          int row, valid;
          const int run = stage_rows(P, A, R, s, row, valid);
          if (run > 0) {
            if (lane == 0)
              for (int i = 0; i < run; ++i, ++k) {
                const uint32_t st = k % kTcStages, round = k / kTcStages;
                if (round && !wait_bounded(&S->empty[st], (round - 1) & 1, T, S)) {
                  ok = false;
                  break;
                }
                const uint32_t a = base + st * kTcStage, bar = full0 + st * 8u;
                const int r = row + i * kTcDepth;
                arrive_expect_cluster(bar, bytes);
                copy2(a, &T.row64[A.p], A.f0 + rank * 128, r, bar);
                copy2(a + 8192u, &T.row64[A.p], A.f0 + rank * 128 + 64, r, bar);
                copy2(a + kTcOperand, &T.dy64[A.p], A.c0 + rank * half, r, bar);
                if (blocks > 1) copy2(a + kTcOperand + 8192u, &T.dy64[A.p], A.c0 + rank * half + 64, r, bar);
              }
            k = __shfl_sync(0xFFFFFFFFu, k, 0);
            ok = __shfl_sync(0xFFFFFFFFu, int(ok), 0);
            s += run;
            continue;
          }
          const uint32_t st = k % kTcStages, round = k / kTcStages;
          if (round && !warp_wait(&S->empty[st], (round - 1) & 1, T, S)) {
            ok = false;
            break;
          }
          const uint32_t a = base + st * kTcStage, bar = ptx::smem_addr(&S->part[st]);
          // rows that follow one another (padding at the end): one copy per 64 features
          const int start = __shfl_sync(0xFFFFFFFFu, row, 0);
          const bool in_line = __all_sync(0xFFFFFFFFu, valid == 0 || row == start + (lane & 7) * 8);
          if (lane == 0) arrive_expect_cluster(bar, bytes);
          __syncwarp();
          // lanes: block of 64 features (0, 1 of x, then those of dy) x group of 8 rows
          const int which = lane >> 3;
          const int x = which < 2 ? A.f0 + rank * 128 + which * 64 : A.c0 + rank * half + (which - 2) * 64;
          if (which < 2 + blocks) {
            const uint32_t to = a + uint32_t(which) * 8192u;
            if (!in_line)
              copy2(to + uint32_t(lane & 7) * 1024u, which < 2 ? &T.row8[A.p] : &T.dy8[A.p], x, row, bar);
            else if ((lane & 7) == 0)
              copy2(to, which < 2 ? &T.row64[A.p] : &T.dy64[A.p], x, row, bar);
          }
          __syncwarp();
          ++s;
          ++k;
        }
      }
    }
    // The MMAs' last releases of the stages have to land before this CTA may leave.
    for (uint32_t j = k > uint32_t(kTcStages) ? k - kTcStages : 0; ok && j < k; ++j)
      ok = warp_wait(&S->empty[j % kTcStages], (j / kTcStages) & 1, T, S);
  } else if (warp == 1 && rank == 0) {
    // ---- MMA
    if (lane == 0) {
      uint32_t k = 0, it = 0;
      bool ok = true;
      const uint32_t kind = (1u << 4) | (1u << 7) | (1u << 10) | (MODE != kForward ? 1u << 15 : 0u) |
                            (MODE == kWgrad ? 1u << 16 : 0u) | (uint32_t(kTcFeatures / 16) << 24);
      for (unsigned t = first; ok && t < tiles; t += stride) {
        const Tile A = tile_at<MODE>(T, S, t);
        if (A.steps == 0) continue;  // an expert without rows: the epilogue writes zeros
        const uint32_t idesc = kind | (uint32_t(A.n / 8) << 17);
        const uint32_t acc = it & 1, d = tmem + acc * 256u;
        if (it >= 2 && !wait_bounded(&S->acc_empty[acc], ((it >> 1) - 1) & 1, T, S)) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        for (int s = 0; s < A.steps; ++s, ++k) {
          const uint32_t st = k % kTcStages;
          if (!wait_bounded(&S->full[st], (k / kTcStages) & 1, T, S)) {
            ok = false;
            break;
          }
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint32_t a = base + st * kTcStage, b = a + kTcOperand;
          const uint64_t da = MODE == kForward ? smem_desc(a, 16, 1024) : smem_desc(a, 8192, 1024);
          const uint64_t db = MODE == kWgrad ? smem_desc(b, 8192, 1024) : smem_desc(b, 16, 1024);
#pragma unroll
          for (int q = 0; q < kTcDepth / 16; ++q)  // 16 deep: 32 bytes along a K-major row, 16 rows of an M/N-major block
            mma_pair(d, da + q * (MODE == kForward ? 2 : 128), db + q * (MODE == kWgrad ? 128 : 2), idesc, s | q);
          commit_pair(&S->empty[st]);
        }
        if (ok) commit_pair(&S->acc_full[acc]);
        ++it;
      }
    }
    __syncwarp();
  } else if (MODE == kWgrad && warp == 2) {
    // ---- zero the padding rows of the stages that hold any, then hand them to the MMA
    const uint32_t full0 = on_first(&S->full[0]);
    uint32_t k = 0, phases = 0;  // bit st: parity of part[st]
    bool ok = true;
    for (unsigned t = first; ok && t < tiles; t += stride) {
      const Tile A = tile_at<MODE>(T, S, t);
      const Ranges R = load_ranges(P, A.p, A.g, 0);
      for (int s = 0; s < A.steps;) {
        int row, valid;
        const int run = stage_rows(P, A, R, s, row, valid);
        s += run > 0 ? run : 1;
        k += run;
        if (run > 0) continue;
        const uint32_t st = k % kTcStages;
        ++k;
        if (!warp_wait(&S->part[st], (phases >> st) & 1, T, S)) {
          ok = false;
          break;
        }
        phases ^= 1u << st;
        // lanes: 4 blocks of 64 features (2 of x, 2 of dy) x 8 vectors of a 128-byte row
        unsigned char* at = stages + size_t(st) * kTcStage + (lane >> 3) * 8192 + (lane & 7) * 16;
        for (int gi = 0; gi < 8; ++gi)
          for (int r = __shfl_sync(0xFFFFFFFFu, valid, gi); r < 8; ++r)
            *reinterpret_cast<uint4*>(at + (gi * 8 + r) * 128) = make_uint4(0, 0, 0, 0);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) arrive_cluster(full0 + st * 8u);
      }
    }
  } else if (warp >= 4) {
    // ---- epilogue: warps q and q + 4 have the tensor-memory lanes 32 q .. and take turns along the columns
    const int q = warp & 3, col0 = (warp - 4) / 4 * kTcColumns;
    uint32_t it = 0;
    for (unsigned t = first; t < tiles; t += stride) {
      const Tile A = tile_at<MODE>(T, S, t);
      const int f = gated ? A.f0 + rank * 64 + q * 16 + (lane & 15) : A.f0 + rank * 128 + q * 32 + lane;
      int row = 0, valid = 0;
      float bias = 0.f;
      if (MODE != kWgrad) {
        group_at(P, A.p, A.g, load_ranges(P, A.p, A.g, 0), A.c0 + lane * 8, row, valid);
        valid = lane * 8 < T.tile_rows ? min(valid, 8) : 0;  // past them: the next tile's rows
        if (MODE == kForward && P.bias[A.p] && f < P.out)
          bias = bf16_of(P.bias[A.p] + int64_t(A.g) * (gated ? 2 : 1) * P.out + (gated && lane >= 16 ? P.out : 0) + f);
      }
      if (A.steps == 0) {  // wgrad of an expert without rows
        uint32_t v[kTcColumns];
#pragma unroll
        for (int j = 0; j < kTcColumns; ++j) v[j] = 0;
        Beside none;
        if (!P.accumulate)
          for (int col = col0; col < A.n; col += 2 * kTcColumns)
            store_columns<MODE, HOC_ACT_NONE>(P, A, v, col, f, row, valid, bias, none);
        continue;
      }
      const uint32_t acc = it & 1;
      const uint32_t at = tmem + acc * 256u + (uint32_t(q * 32) << 16);
      bool ok = true;
      auto columns = [&](auto tag) {
        constexpr int act = decltype(tag)::act;
        Beside B, next;
        load_beside<MODE, act>(P, A, col0, f, row, valid, B);
        ok = warp_wait(&S->acc_full[acc], (it >> 1) & 1, T, S);
        if (!ok) return;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        for (int col = col0; col < A.n; col += 2 * kTcColumns) {
          load_beside<MODE, act>(P, A, col + 2 * kTcColumns, f, row, valid, next);
          uint32_t v[kTcColumns];
          tmem_load(v, at + uint32_t(col));
          store_columns<MODE, act>(P, A, v, col, f, row, valid, bias, B);
          B = next;
        }
      };
      if (MODE == kWgrad) columns(ActTag<HOC_ACT_NONE>{});
      else with_act(P.act, columns);
      if (!ok) break;
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) arrive_relaxed(on_first(&S->acc_empty[acc]));
      ++it;
    }
  }
  __syncwarp();
  if (S->dead) {
    // A wait gave up.  Copies already issued have had the whole limit of that
    // wait to land, those of a role that was still moving land within this pause.
    for (int i = 0; i < 64; ++i) __nanosleep(1000);
  }
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  cluster_sync();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (warp == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTcTmemColumns));
}

using TcFn = void (*)(TcParams);
const TcFn kTc[3] = {mm_tc_kernel<kForward>, mm_tc_kernel<kDgrad>, mm_tc_kernel<kWgrad>};

// ------------------------------------------------------------------ host
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder() {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// A map of bf16 values with 128-byte swizzle; dims and box innermost first,
// strides in elements of the dimensions after the first.
bool encode(CUtensorMap* m, const void* at, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
  cuuint64_t bytes[5];
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
  for (int i = 0; i + 1 < rank; ++i) bytes[i] = strides[i] * 2;
  return encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, cuuint32_t(rank), const_cast<void*>(at), dims, bytes, box, ones,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_rows(CUtensorMap* m, const void* at, int64_t width, int64_t rows, int64_t ld, int height) {
  const cuuint64_t dims[2] = {cuuint64_t(width), cuuint64_t(rows)}, strides[1] = {cuuint64_t(ld)};
  const cuuint32_t box[2] = {kTcDepth, cuuint32_t(height)};
  return encode(m, at, 2, dims, strides, box);
}

bool encode_weight(CUtensorMap* m, const MmParams& P, int mode, const void* at) {
  const cuuint64_t in = P.in, out = P.out, ne = P.experts;
  if (mode == kForward && P.act == HOC_ACT_SWIGLU) {
    // [expert][gate, value][out / 16][16][in], fetched so that 16 gates and their 16 values alternate
    const cuuint64_t dims[5] = {in, 16, 2, out / 16, ne}, strides[4] = {in, out * in, 16 * in, 2 * out * in};
    const cuuint32_t box[5] = {kTcDepth, 16, 2, 4, 1};
    return encode(m, at, 5, dims, strides, box);
  }
  const cuuint64_t dims[3] = {in, out, ne}, strides[2] = {in, out * in};
  const cuuint32_t box[3] = {kTcDepth, mode == kForward ? 128u : 64u, 1};
  return encode(m, at, 3, dims, strides, box);
}

}  // namespace

bool mm_tc_takes(const MmParams& P, int mode) {
  const bool gated = mode == kForward && P.act == HOC_ACT_SWIGLU;
  if (P.in % 8 || P.out % (gated ? 16 : 8) || P.ld_rows % 8 || (mode == kWgrad && P.ld_dy % 8)) return false;
  uintptr_t at = 0;
  for (int p = 0; p < P.parts; ++p)
    at |= reinterpret_cast<uintptr_t>(P.rows[p]) | reinterpret_cast<uintptr_t>(P.dy[p]) | reinterpret_cast<uintptr_t>(P.w[p]);
  return (at & 15u) == 0 && encoder() != nullptr;
}

cudaError_t launch_mm_tc(const MmParams& P, int mode, cudaStream_t s) {
  TcParams T;
  T.P = P;
  T.tile_rows = kTcRows;
  const char* fault = getenv("HOC_FAULT");
  const bool stall = fault && !strcmp(fault, "mm_stall");
  T.tx_pad = stall ? 16u : 0u;
  T.wait_ns = stall ? 100000000ull : kTcWaitNs;
  int64_t tiles = 0;
  const int ftile = mode == kForward && P.act == HOC_ACT_SWIGLU ? kTcFeatures / 2 : kTcFeatures;
  const int64_t ftiles = ((mode == kForward ? P.out : P.in) + ftile - 1) / ftile;
  for (int p = P.part0; p < P.part0 + P.parts; ++p) {
    tiles += ftiles * (mode == kWgrad ? int64_t(P.groups) * ((P.out + kTcRows - 1) / kTcRows)
                                      : P.cap[p] / T.tile_rows + int64_t(P.groups) * (1 + P.sources * 8 / T.tile_rows));
    bool ok = mode == kWgrad || encode_weight(&T.w[p], P, mode, P.w[p]);
    if (P.cap[p] > 0) {  // a buffer without rows has no tile that reads it
      const int64_t width = mode == kDgrad ? P.out : P.in;
      ok = ok && encode_rows(&T.row64[p], P.rows[p], width, P.cap[p], P.ld_rows, 64) &&
           encode_rows(&T.row8[p], P.rows[p], width, P.cap[p], P.ld_rows, 8);
      if (mode == kWgrad)
        ok = ok && encode_rows(&T.dy64[p], P.dy[p], P.out, P.cap[p], P.ld_dy, 64) &&
             encode_rows(&T.dy8[p], P.dy[p], P.out, P.cap[p], P.ld_dy, 8);
    }
    if (!ok) return cudaErrorInvalidValue;
  }
  const void* fn = reinterpret_cast<const void*>(kTc[mode]);
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kTcSmem));
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kTcThreads);
  cfg.dynamicSmemBytes = kTcSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(2);
  // CTA pairs that fit the device at once: asked once for each kernel and device
  static std::atomic<int> known[3][64];
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int pairs = dev < 64 ? known[mode][dev].load() : 0;
  if (pairs == 0) {
    e = cudaOccupancyMaxActiveClusters(&pairs, fn, &cfg);
    if (e != cudaSuccess) return e;
    if (dev < 64) known[mode][dev].store(pairs);
  }
  cfg.numAttrs = 2;
  cfg.gridDim = dim3(2 * unsigned(tiles < 1 ? 1 : tiles < pairs ? tiles : pairs > 0 ? pairs : 1));
  return cudaLaunchKernelEx(&cfg, kTc[mode], T);
}

cudaError_t mm_tc_preload() {
  for (TcFn f : kTc) {
    cudaFuncAttributes a;
    const cudaError_t e = cudaFuncGetAttributes(&a, reinterpret_cast<const void*>(f));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace hoc
