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
// memory and the zeroing, 4-7 epilogue.  Every wait is bounded: a wait that runs
// out sets bit 2 of the status, and all roles leave.
#include <atomic>
#include <cstdlib>
#include <cstring>

#include <cuda.h>

#include "mm.h"
#include "ptx_async.cuh"

namespace hoc {
namespace {

constexpr int kTcThreads = 256;
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
  uint64_t full[kTcStages];   // forward, dgrad: the pair's loads, on the first CTA; wgrad: this CTA's loads
  uint64_t ready[kTcStages];  // wgrad: both CTAs' stages are loaded and their padding rows zero (first CTA)
  uint64_t empty[kTcStages];
  uint64_t acc_full[2];
  uint64_t acc_empty[2];      // on the first CTA: 4 epilogue warps of both CTAs
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
__device__ __forceinline__ bool try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(ptx::smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// Waits for the phase with `parity`; false when the limit passed here or in
// another role, after which the caller leaves its loop.
__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity, const TcParams& T, TcShared* S) {
  if (try_wait_cluster(bar, parity)) return true;
  const uint64_t deadline = ptx::global_ns() + T.wait_ns;
  while (!try_wait_cluster(bar, parity)) {
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
__device__ __forceinline__ void tmem_load32(uint32_t (&r)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,"
      "%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
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
// the buffer and how many of the 8 are the expert's (0: past the end).  The
// whole warp calls it; R holds the first 32 sources' ranges.
__device__ __forceinline__ void group_at(const MmParams& P, int p, int g, Ranges R, int v, int& row, int& valid) {
  const int ns = P.seg ? P.sources : 1;
  int64_t at = v;
  bool found = false;
  row = int(P.cap[p]);
  valid = 0;
  for (int base = 0; base < ns; base += 32) {
    if (base) R = load_ranges(P, p, g, base);
    const int m = min(32, ns - base);
    for (int j = 0; j < m; ++j) {
      const int64_t lo = __shfl_sync(0xFFFFFFFFu, R.lo, j), n = __shfl_sync(0xFFFFFFFFu, R.n, j);
      const int64_t padded = (n + 7) & ~int64_t(7);
      if (!found && at < padded) {
        found = true;
        row = int(lo + at);
        valid = int(n - at < 8 ? n - at : 8);
      }
      at -= padded;
    }
  }
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

// 32 columns of the accumulator: v[j] is feature `f` (of this lane) and column
// col + j; row and valid name the groups of 8 columns of the tile, one per lane.
template <int MODE, int ACT>
__device__ __forceinline__ void store_columns(const MmParams& P, const Tile& A, const uint32_t (&v)[32], int col, int f,
                                              int row, int valid, float bias) {
  const int lane = threadIdx.x & 31;
  constexpr bool gated = MODE == kForward && ACT == HOC_ACT_SWIGLU;
  const int width = MODE == kForward ? P.out : P.in;
  const bool mine = f < width;
  const int64_t wide = int64_t(P.out) * (gated ? 2 : 1);
  __nv_bfloat16* y = static_cast<__nv_bfloat16*>(P.y[A.p]);
  __nv_bfloat16* keep = static_cast<__nv_bfloat16*>(P.pre_out[A.p]);
  const __nv_bfloat16* res = P.res[A.p];
  const __nv_bfloat16* pre = P.pre[A.p];
  if constexpr (gated) {
    // Lanes 0-15 hold the gates of 16 features, lanes 16-31 their values.  They
    // swap halves: each then has both for 16 of the 32 columns.
    const bool upper = lane >= 16;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int gi = (col >> 3) + q;
      const int r0 = __shfl_sync(0xFFFFFFFFu, row, gi & 31), nv = __shfl_sync(0xFFFFFFFFu, valid, gi & 31);
      if (col + q * 8 < A.n && keep && mine)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < nv)
            keep[int64_t(r0 + j) * wide + (upper ? P.out : 0) + f] =
                __float2bfloat16_rn(__uint_as_float(v[q * 8 + j]) + bias);
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float other = __shfl_xor_sync(0xFFFFFFFFu, __uint_as_float(upper ? v[j] : v[16 + j]) + bias, 16);
      const float own = __uint_as_float(upper ? v[16 + j] : v[j]) + bias;
      const int gl = (col >> 3) + (j >> 3), gi = gl + (upper ? 2 : 0);
      const int r0 = __shfl_sync(0xFFFFFFFFu, row, gi & 31), nv = __shfl_sync(0xFFFFFFFFu, valid, gi & 31);
      if (gi * 8 < A.n && (j & 7) < nv && mine) {
        const float g = upper ? other : own, u = upper ? own : other;
        const int64_t r = r0 + (j & 7);
        float o = mm_act(HOC_ACT_SILU, g) * u;
        if (res) o += bf16_of(res + r * P.ld_res + f);
        y[r * P.ld_y + f] = __float2bfloat16_rn(o);
      }
    }
  } else {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int gi = (col >> 3) + q;
    const int r0 = __shfl_sync(0xFFFFFFFFu, row, gi & 31), nv = __shfl_sync(0xFFFFFFFFu, valid, gi & 31);
    if (col + q * 8 >= A.n || !mine) continue;
    float a[8], b[8];
    if (MODE == kDgrad && ACT != HOC_ACT_NONE) {
      const int64_t ldp = int64_t(P.in) * (ACT == HOC_ACT_SWIGLU ? 2 : 1);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        a[j] = j < nv ? bf16_of(pre + int64_t(r0 + j) * ldp + f) : 0.f;
        if (ACT == HOC_ACT_SWIGLU) b[j] = j < nv ? bf16_of(pre + int64_t(r0 + j) * ldp + P.in + f) : 0.f;
      }
    }
    if (MODE == kForward && res) {
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] = j < nv ? bf16_of(res + int64_t(r0 + j) * P.ld_res + f) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j >= nv) continue;
      const int64_t r = r0 + j;
      float x = __uint_as_float(v[q * 8 + j]);
      __nv_bfloat16* o = y + r * P.ld_y + f;
      if (MODE == kForward) {
        x += bias;
        if (keep) keep[r * wide + f] = __float2bfloat16_rn(x);
        x = mm_act(ACT, x);
        if (res) x += a[j];
        *o = __float2bfloat16_rn(x);
      } else if (ACT == HOC_ACT_SWIGLU) {
        o[0] = __float2bfloat16_rn(x * b[j] * mm_act_slope(HOC_ACT_SILU, a[j]));
        o[P.in] = __float2bfloat16_rn(x * mm_act(HOC_ACT_SILU, a[j]));
      } else {
        *o = __float2bfloat16_rn(ACT == HOC_ACT_NONE ? x : x * mm_act_slope(ACT, a[j]));
      }
    }
  }
  }
}

// wgrad: columns are out features, lanes in features.
__device__ __forceinline__ void store_weights(const MmParams& P, const Tile& A, const uint32_t (&v)[32], int col,
                                              int f) {
  if (f >= P.in) return;
  const int64_t first = (int64_t(A.g) * P.out + A.c0 + col) * P.in + f;
  const int m = min(32, P.out - (A.c0 + col));
  if (P.out_f32) {
    float* o = static_cast<float*>(P.y[A.p]) + first;
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < m) {
        const float x = __uint_as_float(v[j]);
        o[int64_t(j) * P.in] = P.accumulate ? o[int64_t(j) * P.in] + x : x;
      }
  } else {
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(P.y[A.p]) + first;
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < m) {
        const float x = __uint_as_float(v[j]);
        o[int64_t(j) * P.in] = __float2bfloat16_rn(P.accumulate ? bf16_of(o + int64_t(j) * P.in) + x : x);
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
      ptx::mbar_init(&S->full[s], 1);
      ptx::mbar_init(&S->ready[s], 2);
      ptx::mbar_init(&S->empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(&S->acc_full[a], 1);
      ptx::mbar_init(&S->acc_empty[a], 8);
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
    // ---- tensor copies
    uint32_t k = 0;  // stages filled
    bool ok = true;
    for (unsigned t = first; ok && t < tiles; t += stride) {
      const Tile A = tile_at<MODE>(T, S, t);
      const Ranges R = load_ranges(P, A.p, A.g, 0);
      const int half = A.n / 2;  // rows of B in this CTA
      int row = 0, valid = 0;
      bool whole = false;
      if (MODE != kWgrad) {
        group_at(P, A.p, A.g, R, A.c0 + rank * half + lane * 8, row, valid);
        const int start = __shfl_sync(0xFFFFFFFFu, row, lane & ~7);
        const unsigned same = __ballot_sync(0xFFFFFFFFu, valid > 0 && row == start + (lane & 7) * 8);
        whole = ((same >> (lane & ~7)) & 0xFFu) == 0xFFu && (lane | 7) * 8 < half;
      }
      const int blocks = (half + 63) / 64;  // wgrad: 64-feature blocks of dy
      const int fa = A.f0 + rank * (gated ? 64 : 128);
      for (int s = 0; s < A.steps; ++s, ++k) {
        const uint32_t st = k % kTcStages, round = k / kTcStages;
        if (round && !warp_wait(&S->empty[st], (round - 1) & 1, T, S)) {
          ok = false;
          break;
        }
        const uint32_t a = base + st * kTcStage, b = a + kTcOperand;
        uint32_t bar;
        if (MODE == kWgrad) {
          group_at(P, A.p, A.g, R, s * kTcDepth + (lane & 7) * 8, row, valid);
          const int start = __shfl_sync(0xFFFFFFFFu, row, 0);
          whole = __all_sync(0xFFFFFFFFu, valid > 0 && row == start + (lane & 7) * 8);
          if (whole) row = start;  // lane i then fetches block i, of all 64 rows
          bar = ptx::smem_addr(&S->full[st]);
          if (lane == 0) ptx::mbar_arrive_expect_tx(&S->full[st], kTcOperand + uint32_t(blocks) * 8192u + T.tx_pad);
        } else {
          bar = on_first(&S->full[st]);
          if (rank == 0 && lane == 0)
            ptx::mbar_arrive_expect_tx(&S->full[st], 2 * (kTcOperand + uint32_t(half) * 128u) + T.tx_pad);
        }
        __syncwarp();
        if (MODE == kWgrad) {
          // operand blocks of 64 features: 0, 1 x; 2, 3 dy
          const int which = whole ? lane : lane >> 3;
          const int x = which < 2 ? A.f0 + rank * 128 + which * 64 : A.c0 + rank * half + (which - 2) * 64;
          const uint32_t to = a + uint32_t(which) * 8192u;
          if (which < 2 + blocks) {
            if (whole)
              copy2(to, which < 2 ? &T.row64[A.p] : &T.dy64[A.p], x, row, bar);
            else
              copy2(to + uint32_t(lane & 7) * 1024u, which < 2 ? &T.row8[A.p] : &T.dy8[A.p], x, row, bar);
          }
        } else {
          const int x = s * kTcDepth;
          if (whole) {
            if ((lane & 7) == 0) copy2(b + uint32_t(lane) * 1024u, &T.row64[A.p], x, row, bar);
          } else if (lane * 8 < half) {
            copy2(b + uint32_t(lane) * 1024u, &T.row8[A.p], x, row, bar);
          }
          if (lane == 31) {
            if (MODE == kDgrad) {
              copy3(a, &T.w[A.p], fa, x, A.g, bar);
              copy3(a + 8192u, &T.w[A.p], fa + 64, x, A.g, bar);
            } else if (gated) {
              copy5(a, &T.w[A.p], x, 0, 0, fa / 16, A.g, bar);
            } else {
              copy3(a, &T.w[A.p], x, fa, A.g, bar);
            }
          }
        }
        __syncwarp();
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
          if (!wait_bounded(MODE == kWgrad ? &S->ready[st] : &S->full[st], (k / kTcStages) & 1, T, S)) {
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
    // ---- zero the padding rows of each stage, then hand it to the MMA
    uint32_t k = 0;
    bool ok = true;
    for (unsigned t = first; ok && t < tiles; t += stride) {
      const Tile A = tile_at<MODE>(T, S, t);
      const Ranges R = load_ranges(P, A.p, A.g, 0);
      for (int s = 0; s < A.steps; ++s, ++k) {
        const uint32_t st = k % kTcStages;
        int row, valid;
        group_at(P, A.p, A.g, R, s * kTcDepth + (lane & 7) * 8, row, valid);
        unsigned part = __ballot_sync(0xFFFFFFFFu, valid > 0 && valid < 8) & 0xFFu;
        if (!warp_wait(&S->full[st], (k / kTcStages) & 1, T, S)) {
          ok = false;
          break;
        }
        while (part) {
          const int gi = __ffs(part) - 1;
          part &= part - 1;
          // lanes: 4 blocks of 64 features (2 of x, 2 of dy) x 8 vectors of a 128-byte row
          unsigned char* at = stages + size_t(st) * kTcStage + (lane >> 3) * 8192 + gi * 1024 + (lane & 7) * 16;
          for (int r = __shfl_sync(0xFFFFFFFFu, valid, gi); r < 8; ++r)
            *reinterpret_cast<uint4*>(at + r * 128) = make_uint4(0, 0, 0, 0);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) arrive_cluster(on_first(&S->ready[st]));
      }
    }
  } else if (warp >= 4) {
    // ---- epilogue: warp q of 4 has the 32 tensor-memory lanes 32 q ..
    const int q = warp & 3;
    uint32_t it = 0;
    for (unsigned t = first; t < tiles; t += stride) {
      const Tile A = tile_at<MODE>(T, S, t);
      const int f = gated ? A.f0 + rank * 64 + q * 16 + (lane & 15) : A.f0 + rank * 128 + q * 32 + lane;
      int row = 0, valid = 0;
      float bias = 0.f;
      if (MODE != kWgrad) {
        group_at(P, A.p, A.g, load_ranges(P, A.p, A.g, 0), A.c0 + lane * 8, row, valid);
        if (lane * 8 >= T.tile_rows) valid = 0;  // the next tile's rows
        if (MODE == kForward && P.bias[A.p] && f < P.out)
          bias = bf16_of(P.bias[A.p] + int64_t(A.g) * (gated ? 2 : 1) * P.out + (gated && lane >= 16 ? P.out : 0) + f);
      }
      if (A.steps == 0) {  // wgrad of an expert without rows
        uint32_t v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = 0;
        if (!P.accumulate)
          for (int col = 0; col < A.n; col += 32) store_weights(P, A, v, col, f);
        continue;
      }
      const uint32_t acc = it & 1;
      if (!warp_wait(&S->acc_full[acc], (it >> 1) & 1, T, S)) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t at = tmem + acc * 256u + (uint32_t(q * 32) << 16);
      auto columns = [&](auto tag) {
        for (int col = 0; col < A.n; col += 32) {
          uint32_t v[32];
          tmem_load32(v, at + uint32_t(col));
          if constexpr (MODE == kWgrad) store_weights(P, A, v, col, f);
          else store_columns<MODE, decltype(tag)::act>(P, A, v, col, f, row, valid, bias);
        }
      };
      if (MODE == kWgrad) columns(ActTag<HOC_ACT_NONE>{});
      else with_act(P.act, columns);
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) arrive_cluster(on_first(&S->acc_empty[acc]));
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
