// Matrix products on the 5th-generation tensor cores (mm.h), for operands whose
// rows are whole 16-byte vectors.
//
// One layout serves the three products: a tile of the result has 256 features f
// (the contiguous index of the output) in the lanes of tensor memory and up to
// 256 rows c in its columns, so
//   - the ragged side (an expert's rows) is the N extent of the MMA, which may
//     be any multiple of 32: a short range costs what it has, not a whole tile;
//   - a thread of the epilogue owns one feature, whose bias is one register, and
//     what it stores lies beside what its neighbours store.
// A pair of CTAs (a cluster of two SMs) computes one tile with cta_group::2:
// each holds 128 features of A and half of the rows of B, 64 deep per stage, so
// a stage moves 32 KB into each SM for 128 x 256 x 64 products.  Operands come
// by tensor copies into 128-byte-swizzled stages; accumulators are double
// buffered in tensor memory, so the epilogue of a tile runs under the products of
// the next one.  Where one range of rows makes few tiles, two or four pairs of a
// cluster share the contraction of a tile.
//
// An expert's rows lie in one range per source.  They are taken as one virtual
// row space in which every range is padded to a multiple of 8, the height of a
// swizzle atom; 64 virtual rows that are contiguous in memory are fetched by one
// copy, others by copies of 32, 16 and 8.  Padding rows hold a neighbour's data: in
// the forward product and the data gradient they are columns that are not stored;
// in the weight gradient, where rows are summed over, they are overwritten with
// zeros in shared memory before the MMA reads them.  There, the whole multiples of
// 64 rows of the ranges come first, each stage one copy per 64 features, and what
// remains of the ranges is packed into the last stages.
//
// Warps of a CTA: 0 and 2 tensor copies of the rows, 64 each; 3 those of the
// weights; 1 MMA (of the pair's first CTA); 4-11 epilogue.  In the weight gradient
// warps 0 and 12 issue all copies of every second stage, and warps 2, 3 and 13-15
// zero padding rows (one range: warp 2, and the others sum the bias gradient).  Every
// wait is bounded: one that runs out sets bit 2 of the status, and all roles leave.
//
// Measured, single calls from a flushed cache; the peaks measured on this GPU are 1951
// TFLOP/s and 6.69 TB/s.  One range of rows: 4096 x 4096 x 4096 forward 81 us (1706
// TFLOP/s), gradients 79 us (1750); 8192 rows of 4096 -> 8192 forward and data
// gradient 287 and 289 us (1913, 1900), weight gradient 318 us (1728); bound by the tensor
// cores and, in the first, by the waves' ends.  8 ranks x 4096 tokens, top-6 of 64 experts,
// Zipf (196,608 rows in 512 ranges): 2048 -> 1280 gated with its pre-activation 1208 us (1710
// TFLOP/s), weight gradient of 2048 x 2560 1426 us (1450; the packed remainders of
// ranges and stores of 671 MB), and at half the tokens the data gradient 1280 <- 2048
// through the gate 411 us (1250 TFLOP/s and 4.2 TB/s: 313 of them without the rows that
// the epilogue reads and writes).  16 tokens instead of 4096: 129 us.  Calls in a row, in
// which the large ones run into the power limit: 1390, 1520, 465 and 108 us (the last 6.0
// TB/s: bound by reading the experts' weights).
#include <atomic>
#include <climits>
#include <cstdlib>
#include <cstring>

#include <cuda.h>

#include "mm.h"
#include "ptx_async.cuh"

namespace hoc {
namespace {

template <int MODE>
constexpr int kTcThreads = MODE == kWgrad ? 512 : 384;
constexpr int kTcEpilogue = 8;                  // warps: two to each 32 lanes of tensor memory
constexpr int kTcColumns = 16;                  // accumulator columns of an epilogue step
constexpr int kTcDepth = 64;                    // contraction elements of a stage: one 128-byte swizzled row
constexpr uint32_t kTcOperand = 128 * 128;      // bytes of one operand of a stage in one CTA
constexpr uint32_t kTcStage = 2 * kTcOperand;
constexpr int kTcFeatures = 256;                // of a pair's tile
constexpr int kTcRows = 256;                    // at most, of a tile
constexpr unsigned kTcPanel = 8;                // row tiles of a panel (see tile_at)
constexpr int kTcMostShares = 2;                // log2: clusters of 8 CTAs
constexpr uint32_t kTcTmemColumns = 512;        // two accumulators of 256 columns
constexpr uint64_t kTcWaitNs = 2000000000ull;

// Division of numbers below 2^31 by a number that the host knows: a multiplication
// and a shift.  (The compiler's division takes over 100 cycles; a warp that looks up
// its first tile did it seven times before its first copy.)
struct Divisor {
  uint32_t d, m, s;
  __device__ __forceinline__ unsigned of(unsigned n) const { return unsigned((uint64_t(n) * m) >> s); }
};
Divisor divisor(uint32_t d) {
  uint32_t log = 0;
  while ((uint64_t(1) << log) < d) ++log;
  return {d, uint32_t((uint64_t(1) << (31 + log)) / d + 1), 31 + log};
}

struct TcParams {  // but for the tensor maps
  Divisor ftiles;    // feature tiles
  Divisor ctiles, each;  // wgrad: tiles of out features, and all tiles of an expert
  Divisor groups;    // P.groups
  Divisor rows;      // tile_rows
  int tile_rows;     // most rows c of a tile, a multiple of 32
  uint32_t stage;    // bytes of a stage: 128 x 64 of A, half of tile_rows x 64 of B
  uint32_t stages;   // as many as the epilogue's planes leave room for: 5 or 6 of a tile of 256 rows
  uint32_t planes;   // of kTcPlane bytes for each of the two epilogue groups
  int sums;          // wgrad of one range: spare warps sum the columns of dy, to P.pre_out[0]
  int loose;         // what the epilogue moves is not whole 16-byte vectors
  int log_shares;    // CTA pairs that share the contraction of a tile: 1, 2 or 4, all of one cluster
  int per;           // stages of each of them (the last may have fewer); INT_MAX where there is one
  uint32_t tx_pad;   // bytes that the copies' barriers expect beyond their loads (0; 16 under HOC_FAULT=mm_stall)
  uint64_t wait_ns;  // 2 s; 0.1 s under HOC_FAULT=mm_stall, 1 ms under mm_hurry
  MmParams P;
};
// RAGGED: ranges of rows of experts, on any ranks; else all rows of one buffer.  That
// is a kernel of its own because what a cold start costs is code and parameters that
// come from memory.  Without the look-up of ranges and the 15 other ranks' maps (18 KB)
// a product of 64 x 64 x 256 takes 10.2 us from a flushed cache instead of 12.3, and 3.9
// instead of 4.6 among others; 4096 x 2048 x 2048 33 instead of 36.
template <bool RAGGED>
struct TcLaunch {
  static constexpr int kRanks = RAGGED ? kMaxRanks : 1;
  TcParams T;
  CUtensorMap w[kRanks];       // forward, dgrad
  CUtensorMap row[kRanks][4];  // P.rows in boxes of 8 << i rows
  CUtensorMap dy[kRanks][4];   // wgrad
};

constexpr int kTcMostStages = 8;

struct TcShared {
  uint64_t full[kTcMostStages];   // on the first CTA: both CTAs' loads of a stage
  uint64_t part[kTcMostStages];   // wgrad: this CTA's loads of a stage that holds padding rows
  uint64_t empty[kTcMostStages];
  uint64_t acc_full[2];
  uint64_t acc_empty[2];      // on the first CTA: the epilogue warps of both CTAs
  uint64_t go, came;          // shares: the others' stages may be written to; their sums for this one's columns are here
  float sum[2][4][16];         // wgrad of one range: column sums of dy by each spare warp
  uint32_t tmem;
  volatile int dead;
  volatile unsigned moved;             // wgrad: changes whenever the copies go on to another stage
  int vrows[kMmMaxGroups];
  unsigned tile0[kMmMaxGroups + 1];    // forward, dgrad: whole tiles of the pairs before
  unsigned short order[kMmMaxGroups];  // forward, dgrad: pairs with a lower tile at their end; wgrad: all; most rows first
  int key[256], rank[256];             // what the order goes by, while it is made
  int lower;                           // forward, dgrad: how many of those
};

// ------------------------------------------------------------------ PTX
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// The address, in the cluster's shared memory, of another CTA's copy of what is at a
// local address; of the pair's first CTA's copy of a barrier.
__device__ __forceinline__ uint32_t on_cta(uint32_t addr, uint32_t cta) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(cta));
  return a;
}
__device__ __forceinline__ uint32_t on_first(const uint64_t* bar) { return on_cta(ptx::smem_addr(bar), cta_rank() & ~1u); }
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
__device__ __forceinline__ bool try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(ptx::smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// Waits for the phase with `parity`; false when the limit passed here or in
// another role, after which the caller leaves its loop.  The limit is on standing
// still: in the weight gradient, whose epilogue may wait through any number of stages
// for the end of a contraction, it starts anew whenever the CTA's copies have moved
// on (they are finite, and a stage's copies wait for the products before them).  CLUSTER:
// what other CTAs' threads wrote before they arrived is to be read.
template <bool CLUSTER>
__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity, const TcParams& T, TcShared* S) {
  auto came = [&]() { return CLUSTER ? try_wait_cluster(bar, parity) : ptx::mbar_try_wait(bar, parity); };
  if (came()) return true;
  uint64_t deadline = ptx::global_ns() + T.wait_ns;
  unsigned moved = S->moved;
  while (!came()) {
    if (S->dead) return false;
    const uint64_t now = ptx::global_ns();
    if (const unsigned m = S->moved; m != moved) {
      moved = m;
      deadline = now + T.wait_ns;
    } else if (now > deadline) {
      atomicOr(T.P.status, 4);
      S->dead = 1;
      return false;
    }
  }
  return true;
}
// The same by a whole warp, with one answer for all lanes.
template <bool CLUSTER = false>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const TcParams& T, TcShared* S) {
  return __all_sync(0xFFFFFFFFu, wait_bounded<CLUSTER>(bar, parity, T, S));
}
// Programmatic dependent launch: waits for the kernel before this one on the
// stream, then lets the next one start.
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
// One lane of a warp, for the instructions that one thread issues.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// The stage that is next in turn, and the parity of its current round.
struct Turn {
  uint32_t stages, st = 0, round = 0;
  __device__ __forceinline__ explicit Turn(uint32_t n) : stages(n) {}
  __device__ __forceinline__ void next() {
    if (++st == stages) {
      st = 0;
      ++round;
    }
  }
};
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
      "h"(uint16_t(3u << (cta_rank() & ~1u)))
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
  int steps;    // stages of the contraction, this share's
};

// The order of the tiles: whole ones first, pair by pair, then the lower tile that
// ends a pair's rows, the one with the most rows first (wgrad: the tiles of the
// pair with the most rows first).  Tiles of falling cost, dealt to the CTA pairs in
// turn and every second time backwards, come out within 1 to 7 % of an even share
// at the expert layer's Zipf(1.1) loads (in the given order and always forwards 2
// to 25 %).
__device__ __forceinline__ unsigned dealt(unsigned i, unsigned who, unsigned of) {
  return i * of + (i & 1 ? of - 1 - who : who);
}

// Fills S->order and S->lower from S->vrows.  The whole CTA calls it.
template <int MODE>
__device__ __forceinline__ void order_pairs(const TcParams& T, TcShared* S) {
  const int n = T.P.parts * T.P.groups;
  auto key = [&](int i) {
    const int rows = S->vrows[i];
    return MODE == kWgrad ? rows : rows - int(T.rows.of(rows)) * T.tile_rows;
  };
  if (threadIdx.x == 0) S->lower = 0;
  if (n <= 256) {  // rank of each pair by counting; beyond that the sort would cost more than it gains
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      S->key[i] = key(i);
      S->rank[i] = 0;
    }
    __syncthreads();
    // a warp per 32 pairs and share of the others
    const int blocks = (n + 31) / 32, warps = int(blockDim.x) / 32, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int shares = warps / blocks > 0 ? warps / blocks : 1;
    for (int w = warp; w < blocks * shares; w += warps) {
      const int i = w % blocks * 32 + lane, share = w / blocks;
      const int mine = i < n ? S->key[i] : 0;
      int before = 0;
#pragma unroll 4
      for (int j = share; j < n; j += shares) before += S->key[j] > mine || (S->key[j] == mine && j < i);
      if (i < n) atomicAdd(&S->rank[i], before);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      S->order[S->rank[i]] = static_cast<unsigned short>(i);
      if (S->key[i] > 0) atomicAdd(&S->lower, 1);
    }
  } else {
    __syncthreads();
    if (threadIdx.x < 32) {
      int at = 0;
      for (int i0 = 0; i0 < n; i0 += 32) {
        const int i = i0 + int(threadIdx.x);
        const bool take = i < n && (MODE == kWgrad || key(i) > 0);
        const unsigned some = __ballot_sync(0xFFFFFFFFu, take);
        if (take) S->order[at + __popc(some & ((1u << threadIdx.x) - 1u))] = static_cast<unsigned short>(i);
        at += __popc(some);
      }
      if (threadIdx.x == 0) S->lower = at;
    }
  }
  __syncthreads();
}

// Tiles of the launch.
template <int MODE, bool RAGGED>
__device__ __forceinline__ unsigned tile_count(const TcParams& T, const TcShared* S) {
  const MmParams& P = T.P;
  if (MODE == kWgrad) return unsigned(P.parts * P.groups) * T.each.d;
  if (RAGGED) return S->tile0[P.parts * P.groups] + unsigned(S->lower) * T.ftiles.d;
  return T.rows.of(unsigned(P.cap[0]) + T.tile_rows - 1) * T.ftiles.d;
}
// (Not inlined: every role calls it, once for 32 tiles, and shares its instructions.)
template <int MODE, bool RAGGED>
__device__ __noinline__ Tile tile_at(const TcParams& T, const TcShared* S, unsigned t) {
  const MmParams& P = T.P;
  const int n = P.parts * P.groups;
  const int ftile = MODE == kForward && P.act == HOC_ACT_SWIGLU ? kTcFeatures / 2 : kTcFeatures;
  unsigned i = 0, ct, ft;
  if (MODE == kWgrad) {
    const unsigned at = RAGGED ? T.each.of(t) : 0, u = t - at * T.each.d;
    if (RAGGED) i = S->order[at];
    ft = T.ctiles.of(u);
    ct = u - ft * T.ctiles.d;
  } else {
    const unsigned all = RAGGED ? S->tile0[n] : T.rows.of(unsigned(P.cap[0])) * T.ftiles.d;  // whole tiles
    if (t < all) {
      if (RAGGED) i = mm_find(S->tile0, n, t);
      // panels of 8 row tiles, so that the tiles in flight share rows and features about evenly
      const unsigned t0 = RAGGED ? S->tile0[i] : 0, lt = t - t0;
      const unsigned whole = T.ftiles.of((RAGGED ? S->tile0[i + 1] : all) - t0);
      const unsigned panel = T.ftiles.of(lt) / kTcPanel, u = lt - panel * kTcPanel * T.ftiles.d;
      const unsigned high = min(kTcPanel, whole - panel * kTcPanel);
      ft = high == kTcPanel ? u / kTcPanel : u / high;
      ct = panel * kTcPanel + u - ft * high;
    } else {
      const unsigned u = t - all, at = RAGGED ? T.ftiles.of(u) : 0;
      if (RAGGED) i = S->order[at];
      ct = T.ftiles.of(RAGGED ? S->tile0[i + 1] - S->tile0[i] : all);
      ft = u - at * T.ftiles.d;
    }
  }
  const unsigned part = RAGGED ? T.groups.of(i) : 0;
  Tile A;
  A.p = RAGGED ? P.part0 + part : 0;
  A.g = RAGGED ? P.group0 + i - part * T.groups.d : 0;
  A.f0 = int(ft) * ftile;
  A.c0 = int(ct) * T.tile_rows;
  const int rows = RAGGED ? S->vrows[i] : int(P.cap[0]);
  A.n = (min(T.tile_rows, (MODE == kWgrad ? P.out : rows) - A.c0) + 31) / 32 * 32;
  A.steps = ((MODE == kForward ? P.in : MODE == kDgrad ? P.out : rows) + kTcDepth - 1) / kTcDepth;
  if (!RAGGED) A.steps = min(A.steps - int(cta_rank() >> 1) * T.per, T.per);
  return A;
}

// The ranges of one expert, one source per lane: first row, rows, and the
// virtual row they start at (of the 32 sources at hand; `all`: past the last).
// PAD 8: sources one after another, each padded to 8.  PAD 64: first the whole
// multiples of 64 rows of every range, then what remains of them (`rest`), each
// padded to 8, and the end padded to 64 (mm_count counts the same).
struct Ranges {
  int lo, n, start, rest, wholes, all;
};
// What a lane reads for it: issued a tile ahead, so that nothing waits for it.
struct Ends {
  int64_t from, to;
};
template <bool RAGGED>
__device__ __forceinline__ Ends load_ends(const MmParams& P, int p, int g, int base) {
  const int s = base + int(threadIdx.x & 31);
  Ends E{0, 0};
  if (RAGGED && s < P.sources) {
    const int64_t* at = P.seg + int64_t(p) * (int64_t(P.sources) * P.experts + 1) + int64_t(s) * P.experts + g;
    E = {at[0], at[1]};
  }
  return E;
}
template <int PAD, bool RAGGED>
__device__ __forceinline__ Ranges load_ranges(const MmParams& P, int p, Ends E) {
  Ranges R{};
  if (!RAGGED) {  // virtual rows are the buffer's rows
    R.n = int(P.cap[0]);
    R.wholes = R.n / PAD * PAD;
    return R;
  }
  const int lane = threadIdx.x & 31;
  int64_t lo, n;
  mm_cut(P.cap[p], E.from, E.to, lo, n);
  R.lo = int(lo);
  R.n = int(n);
  const int whole = PAD == 8 ? 0 : R.n / PAD * PAD, rest = (R.n - whole + 7) & ~7;
  int a = whole, b = rest;
  const int ns = P.sources;
  for (int off = 1; off < 32 && off < ns; off <<= 1) {
    const int x = __shfl_up_sync(0xFFFFFFFFu, a, off), y = __shfl_up_sync(0xFFFFFFFFu, b, off);
    if (lane >= off) {
      a += x;
      b += y;
    }
  }
  const int last = min(ns, 32) - 1;  // lanes past the sources add nothing
  const int wholes = __shfl_sync(0xFFFFFFFFu, a, last);
  R.wholes = wholes;
  R.rest = wholes + b - rest;
  R.start = PAD == 8 ? R.rest : a - whole;
  if (lane >= ns) R.start = R.rest = INT_MAX;  // no source: starts past everything
  R.all = (wholes + __shfl_sync(0xFFFFFFFFu, b, last) + PAD - 1) / PAD * PAD;
  return R;
}
// Each lane's group of 8 virtual rows at `v` (a multiple of 8): its first row in
// the buffer and how many rows its range has from there on (0: past the end).
// The whole warp calls it; R holds the first 32 sources' ranges.
template <int PAD, bool RAGGED>
__device__ __forceinline__ void group_at(const MmParams& P, int p, int g, Ranges R, int v, int& row, int& left) {
  if (!RAGGED) {
    row = min(v, R.n);
    left = R.n - row;
    return;
  }
  const int ns = P.sources;
  row = int(P.cap[p]);
  left = 0;
  for (int base = 0; base < ns; base += 32) {
    if (ns > 32) R = load_ranges<PAD, true>(P, p, load_ends<true>(P, p, g, base));
    // whole multiples of PAD, or what remains (for PAD 64 all lanes alike: their v share a multiple of 64)
    const bool whole = PAD > 8 && v < R.wholes;
    const int key = whole ? R.start : R.rest;
    int j = 0;  // the last source that starts at or before v
    for (int step = ns > 8 ? 16 : ns > 1 ? 4 : 0; step; step >>= 1) {
      const int at = __shfl_sync(0xFFFFFFFFu, key, j + step);
      if (at <= v) j += step;
    }
    const int lo = __shfl_sync(0xFFFFFFFFu, R.lo, j), n = __shfl_sync(0xFFFFFFFFu, R.n, j);
    const int off = v - __shfl_sync(0xFFFFFFFFu, key, j), cut = PAD > 8 ? n / PAD * PAD : 0;
    if (v >= 0 && off < (whole ? cut : n - cut)) {
      row = lo + (whole ? 0 : cut) + off;
      left = (whole ? cut : n - cut) - off;
    }
    v -= R.all;  // negative once it was found
  }
}

// The tiles of one CTA pair, as each warp walks them.  The lanes work out 32 tiles
// at a time, one each (a tile takes several divisions, which between two tiles
// would cost as much as a stage's products), and what a warp reads to find a tile's
// rows is read a tile ahead.
template <bool RAGGED>
struct Work {
  const TcParams& T;
  const TcShared* S;
  unsigned who, of, tiles, i = 0;
  bool more = false, ahead_more = false;
  Tile now, ahead, mine;
  Ends ends, ahead_ends;
  __device__ __forceinline__ Work(const TcParams& t, const TcShared* s, unsigned w, unsigned o, unsigned n)
      : T(t), S(s), who(w), of(o), tiles(n) {}
  template <int MODE>
  __device__ __forceinline__ void look_ahead(bool rows = true) {
    const unsigned at = i & 31;
    if (at == 0) {
      const unsigned t = dealt(i + (threadIdx.x & 31), who, of);
      mine.n = 0;
      if (t < tiles) mine = tile_at<MODE, RAGGED>(T, S, t);
      __syncwarp();
    }
    ++i;
    ahead.n = __shfl_sync(0xFFFFFFFFu, mine.n, at);
    ahead.p = __shfl_sync(0xFFFFFFFFu, mine.p, at);
    ahead.g = __shfl_sync(0xFFFFFFFFu, mine.g, at);
    ahead.f0 = __shfl_sync(0xFFFFFFFFu, mine.f0, at);
    ahead.c0 = __shfl_sync(0xFFFFFFFFu, mine.c0, at);
    ahead.steps = __shfl_sync(0xFFFFFFFFu, mine.steps, at);
    ahead_more = ahead.n > 0;  // only the last round may be short
    if (ahead_more && rows) ahead_ends = load_ends<RAGGED>(T.P, ahead.p, ahead.g, 0);
  }
  __device__ __forceinline__ void next() {
    more = ahead_more;
    now = ahead;
    ends = ahead_ends;
  }
};
// Before a warp uses what the cluster's CTAs set up, and reads or writes what the kernel
// before this one may: each does it once, when it has looked up its first tile.
template <bool RAGGED>
__device__ __forceinline__ void begin() {
  __syncwarp();
  cluster_wait();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (!RAGGED) after_previous();  // with ranges, it was needed before they were read
}
// f() for each tile, W.now being the tile and the next one looked up already; until
// it returns false.
template <int MODE, bool RAGGED, class F>
__device__ __forceinline__ void each_tile(Work<RAGGED>& W, bool rows, F f) {
  for (;;) {  // once without a tile, so that the look-up stands in one place
    W.template look_ahead<MODE>(rows);
    if (!W.more) begin<RAGGED>();
    if (W.more && !f()) return;
    if (!W.ahead_more) return;
    W.next();
  }
}

// How 64 virtual rows, a group of 8 per lane modulo 8, are fetched: a run of groups
// that follow one another in the buffer by copies of 64, 32, 16 and 8 rows, as the
// binary digits of its length say (groups without rows make runs too).  Returns
// log2 of the groups of the copy that starts at this lane's group, or -1.
__device__ __forceinline__ int box_at(int row, int left) {
  const int j = threadIdx.x & 7;
  const int r = __shfl_up_sync(0xFFFFFFFFu, row, 1), l = __shfl_up_sync(0xFFFFFFFFu, left, 1);
  const bool goes_on = j > 0 && (left > 0 ? l > 0 && row == r + 8 : l <= 0);
  const unsigned starts = (__ballot_sync(0xFFFFFFFFu, !goes_on) & 0xFFu) | 0x100u;
  const int from = 31 - __clz(starts & ((2u << j) - 1u));
  const int len = __ffs(starts >> (j + 1)) + j - from, at = j - from;
  if (len == 8) return at == 0 ? 3 : -1;
  if ((len & 4) && at == 0) return 2;
  if ((len & 2) && at == (len & 4)) return 1;
  return (len & 1) && at == (len & 6) ? 0 : -1;
}

// wgrad: the 64 virtual rows of stage s, a group of 8 per lane modulo 8 (row, and
// valid rows of the 8).  Returns (to all lanes) how many stages from s on are 64
// rows each of one range; 0 when stage s is not.
template <bool RAGGED>
__device__ __forceinline__ int stage_rows(const MmParams& P, const Tile& A, const Ranges& R, int s, int& row,
                                          int& valid) {
  int left;
  group_at<kTcDepth, RAGGED>(P, A.p, A.g, R, s * kTcDepth + int(threadIdx.x & 7) * 8, row, left);
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

// A lane of tensor memory holds one feature, a row in global memory is contiguous in
// features: the sums cross over through shared memory.  Four warps put
// kTcColumns columns of 128 features there as binary32 and take them out as 8
// features of one row per thread, so that what is stored, and a residual, moves as
// 16-byte vectors straight between registers and global memory.  (Stores of single
// values were what bounded the kernel at the expert layer's widths; staging the rounded
// values took 1263 us for the gated product of 2048 -> 1280 with its pre-activation,
// this takes 1205.)

// The rows of a tensor from a feature on.
struct Strip {
  char* at;        // that feature in row 0
  int64_t pitch;   // bytes of a row
  int left;        // features from there to the end of a row; none of them when it is not positive
  bool loose;      // rows are not whole 16-byte vectors: moved value by value
};
__device__ __forceinline__ uint4 get8(const Strip& G, int row) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (row < 0 || G.left <= 0) return v;
  const char* at = G.at + row * G.pitch;
  if (!G.loose) {
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(at));
    return v;
  }
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < G.left) w[e / 2] |= uint32_t(reinterpret_cast<const uint16_t*>(at)[e]) << (16 * (e & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void put8(const Strip& G, int row, const float (&z)[8]) {
  if (row < 0 || G.left <= 0) return;
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 pair = __floats2bfloat162_rn(z[2 * e], z[2 * e + 1]);
    w[e] = *reinterpret_cast<const uint32_t*>(&pair);
  }
  char* at = G.at + row * G.pitch;
  if (!G.loose) {
    *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < G.left) reinterpret_cast<uint16_t*>(at)[e] = uint16_t(w[e / 2] >> (16 * (e & 1)));
}
__device__ __forceinline__ void unpack8(const uint4& v, float (&z)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    z[2 * e] = __uint_as_float(w[e] << 16);
    z[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
  }
}
// The first `left` of 8 values, one by one.
__device__ __forceinline__ void put_loose(char* to, const unsigned char* from, int left) {
  for (int e = 0; e < 8; ++e)
    if (e < left) *reinterpret_cast<uint16_t*>(to + e * 2) = *reinterpret_cast<const uint16_t*>(from + e * 2);
}

constexpr uint32_t kTcRowBytes = 256;
constexpr uint32_t kTcPlane = kTcColumns * kTcRowBytes;  // one staged array

__device__ __forceinline__ void group_barrier(int eg) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + eg), "n"(128) : "memory");
}
// Whether `ok` holds in all four warps.
__device__ __forceinline__ bool group_all(int eg, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbar.red.and.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(int(ok)), "r"(1 + eg), "n"(128)
      : "memory");
  return r != 0;
}
// The row that column `c` of the step at `col` stands for, -1 if none.  Whole warps call it.
__device__ __forceinline__ int row_of(int col, int c, int row, int valid) {
  const int gi = ((col + c) >> 3) & 31;
  const int r0 = __shfl_sync(0xFFFFFFFFu, row, gi), nv = __shfl_sync(0xFFFFFFFFu, valid, gi);
  return (c & 7) < nv ? r0 + (c & 7) : -1;
}
// The rows that this thread moves in a step at `col`: vector (i + 128 h) % CHUNKS
// of column (i + 128 h) / CHUNKS, i its number in the group.  at(c): the row of
// column c of the step, or -1.
template <int CHUNKS>
struct Rows {
  int r[kTcColumns * CHUNKS / 128];
  template <class At>
  __device__ __forceinline__ explicit Rows(At at) {
#pragma unroll
    for (int h = 0; h < kTcColumns * CHUNKS / 128; ++h) r[h] = at((int(threadIdx.x & 127) + 128 * h) / CHUNKS);
  }
};
// kTcColumns rows of CHUNKS vectors from a strip into shared memory (rows of
// 16 * CHUNKS bytes) and back, by 128 threads.
template <int CHUNKS>
__device__ __forceinline__ void fetch_rows(uint32_t smem, const Strip& G, const Rows<CHUNKS>& R) {
  const int i = int(threadIdx.x) & 127, v = i % CHUNKS;
  if (G.loose) {
#pragma unroll
    for (int h = 0; h < kTcColumns * CHUNKS / 128; ++h)
      for (int e = 0; e < 8; ++e)
        if (R.r[h] >= 0 && v * 8 + e < G.left) {
          const uint16_t x = *reinterpret_cast<const uint16_t*>(G.at + R.r[h] * G.pitch + (v * 8 + e) * 2);
          asm volatile("st.shared.u16 [%0], %1;" ::"r"(smem + uint32_t(i + 128 * h) * 16u + e * 2), "h"(x) : "memory");
        }
    return;
  }
#pragma unroll
  for (int h = 0; h < kTcColumns * CHUNKS / 128; ++h)
    if (R.r[h] >= 0 && v * 8 < G.left)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem + uint32_t(i + 128 * h) * 16u),
                   "l"(G.at + R.r[h] * G.pitch + v * 16)
                   : "memory");
}
template <int CHUNKS>
__device__ __forceinline__ void put_rows(const unsigned char* smem, const Strip& G, const Rows<CHUNKS>& R) {
  const int i = int(threadIdx.x) & 127, v = i % CHUNKS;
  if (G.loose) {
#pragma unroll
    for (int h = 0; h < kTcColumns * CHUNKS / 128; ++h)
      put_loose(G.at + R.r[h] * G.pitch + v * 16, smem + (i + 128 * h) * 16, R.r[h] >= 0 ? G.left - v * 8 : 0);
    return;
  }
#pragma unroll
  for (int h = 0; h < kTcColumns * CHUNKS / 128; ++h)
    if (R.r[h] >= 0 && v * 8 < G.left)
      *reinterpret_cast<uint4*>(G.at + R.r[h] * G.pitch + v * 16) =
          *reinterpret_cast<const uint4*>(smem + (i + 128 * h) * 16);
}

__device__ __forceinline__ float bf16_at(const unsigned char* p) {
  return __uint_as_float(uint32_t(*reinterpret_cast<const uint16_t*>(p)) << 16);
}
__device__ __forceinline__ void put_bf16(unsigned char* p, float v) {
  *reinterpret_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(v);
}

// Shares of a contraction.  Where a product has few tiles, the CTA pairs of a cluster
// compute one together, each from a part of the contraction: one pair would stream
// its operands through two SMs while the others idle.  Each then has sums of the
// whole tile; the columns are dealt out in blocks of two epilogue steps, and a CTA
// sends the sums of the others' columns into their stages, which are free once all
// products of those CTAs are done.  The sums are added in the order of the shares,
// whoever adds them.  64 rows of 7168 -> 512 columns take 20 us with four shares, 26
// with two and 36 with one; 64 x 4096 x 4096 22 us with two and 26 with one; the weight
// gradient of 8192 rows of 512 x 512 22, 26 and 38 us.
constexpr uint32_t kTcSums = kTcColumns * 128 * 4;  // bytes of a step: [4 columns][lane][4]

// Where the sums of share `from` for the step at `col` lie in the stages of the step's owner `to`.
__device__ __forceinline__ uint32_t sums_at(const TcParams& T, int col, int from, int to) {
  const int j = col / kTcColumns, others = (1 << T.log_shares) - 1;
  return uint32_t(((j >> (1 + T.log_shares)) * 2 + (j & 1)) * others + (from < to ? from : from - 1)) * kTcSums +
         (threadIdx.x & 127) * 16u;
}
// Sends the sums of the other shares' columns (of the steps whose number is eg modulo
// 2) and waits for those of this one's.  Whole warps call it, after their accumulator came.
__device__ __forceinline__ bool exchange_sums(const TcParams& T, TcShared* S, int n, uint32_t stages, uint32_t acc_at,
                                              int eg) {
  const int cta = int(cta_rank()), mine = cta >> 1, rank = cta & 1, shares = 1 << T.log_shares, lane = threadIdx.x & 31;
  if ((threadIdx.x & ~31u) == 128 && lane < shares && lane != mine)  // this CTA's products are done
    arrive_cluster(on_cta(ptx::smem_addr(&S->go), 2 * lane + rank));
  __syncwarp();
  if (!warp_wait<true>(&S->go, 0, T, S)) return false;
  for (int col = eg * kTcColumns; col < n; col += 2 * kTcColumns) {
    const int to = (col / (2 * kTcColumns)) & (shares - 1);
    if (to == mine) continue;
    uint32_t v[kTcColumns];
    tmem_load(v, acc_at + uint32_t(col));
    const uint32_t at = on_cta(stages + sums_at(T, col, mine, to), 2 * to + rank);
#pragma unroll
    for (int j = 0; j < kTcColumns; j += 4)
      asm volatile("st.shared::cluster.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at + j * 512u), "r"(v[j]), "r"(v[j + 1]),
                   "r"(v[j + 2]), "r"(v[j + 3])
                   : "memory");
  }
  __syncwarp();
  if (lane < shares && lane != mine) arrive_cluster(on_cta(ptx::smem_addr(&S->came), 2 * lane + rank));
  __syncwarp();
  return warp_wait<true>(&S->came, 0, T, S);
}
// Adds the other shares' sums to this one's, v, of the step at `col`.
__device__ __forceinline__ void add_sums(const TcParams& T, uint32_t (&v)[kTcColumns], uint32_t stages, int col) {
  const int mine = int(cta_rank()) >> 1, shares = 1 << T.log_shares;
  float sum[kTcColumns];
#pragma unroll
  for (int j = 0; j < kTcColumns; ++j) sum[j] = 0.f;
  for (int s = 0; s < shares; ++s) {
    const uint32_t at = stages + sums_at(T, col, s, mine);
#pragma unroll
    for (int j = 0; j < kTcColumns; j += 4) {
      uint32_t x[4] = {v[j], v[j + 1], v[j + 2], v[j + 3]};
      if (s != mine)
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                     : "r"(at + j * 512u));
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[j + i] += __uint_as_float(x[i]);
    }
  }
#pragma unroll
  for (int j = 0; j < kTcColumns; ++j) v[j] = __float_as_uint(sum[j]);
}

// The epilogue of one tile by group `eg` of four warps (warp q of it has tensor
// memory lanes 32 q ..): the steps of kTcColumns columns whose number is eg modulo
// 2 (of this share's).  (MODE kDgrad: with no activation.)  plane: the group's staging,
// [column][128 features] binary32, in which the 16-byte quads of a warp's 32 features are
// exchanged by q, so that both sides reach all banks.  False when the accumulator did not come.
template <int MODE, int ACT, bool RAGGED>
__device__ __forceinline__ bool run_epilogue(const TcParams& T, TcShared* S, const Tile& A, uint32_t stages, uint32_t plane,
                                             uint32_t acc_at, uint64_t* acc_full, uint32_t parity, int eg, int q, int rank,
                                             int row, int valid, float bias) {
  constexpr bool gated = MODE == kForward && ACT == HOC_ACT_SWIGLU;
  constexpr int kVectors = gated ? 8 : 16;                         // of 8 features, in a row
  constexpr int kPer = kTcColumns * kVectors / 128;                // of a thread, in a step
  const MmParams& P = T.P;
  const int lane = threadIdx.x & 31, i = threadIdx.x & 127;
  const int u = i % kVectors, c0 = i / kVectors;  // this thread's vector, and its first column
  const int width = MODE == kForward ? P.out : P.in;
  const int64_t wide = int64_t(width) * (ACT == HOC_ACT_SWIGLU ? 2 : 1);  // of pre
  const bool res = MODE == kForward && P.res[A.p] != nullptr;
  const bool keep = MODE == kForward && P.pre_out[A.p] != nullptr;
  // clamped so that no pointer is formed past the tensors
  const int f0 = A.f0 + rank * (gated ? 64 : 128) + u * 8, left = width - f0, fs = left > 0 ? f0 : 0;
  auto strip = [&](const void* at, int64_t ld) {
    return Strip{static_cast<char*>(const_cast<void*>(at)) + 2 * int64_t(fs), 2 * ld, left, T.loose != 0};
  };
  auto second = [&](Strip s) {
    s.at += 2 * int64_t(width);
    return s;
  };
  const Strip y = strip(P.y[A.p], P.ld_y), kept = strip(P.pre_out[A.p], wide);
  const Strip beside = strip(P.res[A.p], P.ld_res);
  int r[kPer];      // this thread's rows of a step
  uint4 add[kPer];  // and the residual there, loaded a step ahead
  auto load = [&](int col) {
#pragma unroll
    for (int h = 0; h < kPer; ++h) {
      r[h] = row_of(col, c0 + h * (kTcColumns / kPer), row, valid);
      if (res && col < A.n) add[h] = get8(beside, r[h]);
    }
  };
  const int share = RAGGED ? 0 : int(cta_rank()) >> 1, stride = RAGGED ? 2 * kTcColumns : (2 * kTcColumns) << T.log_shares;
  const int first = (eg + 2 * share) * kTcColumns;
  if (res) {
    // The tile's residual into L2, a row of 128 features per lane and warp: a step is shorter than the latency of
    // HBM (8192 rows of 512 -> 4096 with a residual 64 us, 78 without this).
    const int from = A.f0 + rank * (gated ? 64 : 128), w = eg * 4 + q;
    if (w < valid)
      for (int f = from; f < from + (gated ? 64 : 128) && f < width; f += 64)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(P.res[A.p] + (row + w) * P.ld_res + f));
  }
  load(first);
  bool ok = warp_wait(acc_full, parity, T, S);
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (!RAGGED && ok && T.log_shares) ok = exchange_sums(T, S, A.n, stages, acc_at, eg);
  if (!group_all(eg, ok)) return false;
  const uint32_t put_at = plane + uint32_t(((q * 8 + (lane >> 2)) ^ q) * 16 + (lane & 3) * 4);
  for (int col = first; col < A.n; col += stride) {
    uint32_t v[kTcColumns];
    tmem_load(v, acc_at + uint32_t(col));
    if (!RAGGED && T.log_shares) add_sums(T, v, stages, col);
#pragma unroll
    for (int j = 0; j < kTcColumns; ++j)
      asm volatile("st.shared.f32 [%0], %1;" ::"r"(put_at + j * 512u), "f"(__uint_as_float(v[j]) + bias) : "memory");
    group_barrier(eg);
    float z[kPer][gated ? 16 : 8];
#pragma unroll
    for (int h = 0; h < kPer; ++h)
#pragma unroll
      for (int k = 0; k < (gated ? 4 : 2); ++k) {
        const int quad = gated ? (4 * u + k) ^ (u >> 1) : (2 * u + k) ^ (u >> 2);
        asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                     : "=f"(z[h][4 * k]), "=f"(z[h][4 * k + 1]), "=f"(z[h][4 * k + 2]), "=f"(z[h][4 * k + 3])
                     : "r"(plane + (c0 + h * (kTcColumns / kPer)) * 512u + uint32_t(quad) * 16u)
                     : "memory");
      }
    group_barrier(eg);  // the plane is free again
#pragma unroll
    for (int h = 0; h < kPer; ++h) {
      float o[8], x[8];
      if (res) unpack8(add[h], x);
      if constexpr (gated) {
        float g[8], l[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          g[e] = z[h][e];
          l[e] = z[h][8 + e];
          o[e] = mm_act(HOC_ACT_SILU, g[e]) * l[e];
          if (res) o[e] += x[e];
        }
        if (keep) {
          put8(kept, r[h], g);
          put8(second(kept), r[h], l);
        }
      } else if constexpr (MODE == kForward) {
        if (keep) put8(kept, r[h], z[h]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          o[e] = mm_act(ACT, z[h][e]);
          if (res) o[e] += x[e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = z[h][e];
      }
      put8(y, r[h], o);
    }
    load(col + stride);
  }
  return true;
}

// The data gradient through an activation reads a row, or with gates two, for each
// that it writes.  Loads into registers cannot be kept in flight long enough there (444
// us through the gate for the data gradient of 1280 <- 2048, where this takes 411, and 179
// against 126 through SiLU for 36,432 rows of 1984 <- 392): rows come into shared memory by asynchronous copies two
// steps ahead, and results, staged as bf16, take the place of what was read.  plane: the
// group's three buffers, with gates of two planes each.
template <int ACT, bool RAGGED>
__device__ __forceinline__ bool run_slope_epilogue(const TcParams& T, TcShared* S, const Tile& A, uint32_t stages,
                                                   unsigned char* planes, uint32_t& buffer, uint32_t acc_at, uint64_t* acc_full,
                                                   uint32_t parity, int eg, int q, int rank, int row, int valid) {
  constexpr bool twice = ACT == HOC_ACT_SWIGLU;  // two inputs, two outputs
  const MmParams& P = T.P;
  const int lane = threadIdx.x & 31, width = P.in, f0 = A.f0 + rank * 128;
  const int64_t wide = int64_t(width) * (twice ? 2 : 1);  // of pre
  const uint32_t planes_addr = ptx::smem_addr(planes);
  // clamped so that no pointer is formed past the tensors
  const int left = width - f0, fs = left > 0 ? f0 : 0;
  const Strip y{static_cast<char*>(P.y[A.p]) + 2 * int64_t(fs), 2 * P.ld_y, left, T.loose != 0};
  const Strip beside{reinterpret_cast<char*>(const_cast<__nv_bfloat16*>(P.pre[A.p])) + 2 * int64_t(fs), 2 * wide, left,
                     T.loose != 0};
  auto second = [&](Strip s) {
    s.at += 2 * int64_t(width);
    return s;
  };
  constexpr uint32_t kBuffer = 2 * kTcPlane;
  auto fetch = [&](int col, uint32_t buffer) {
    if (col < A.n) {
      const Rows<16> r([&](int c) { return row_of(col, c, row, valid); });
      fetch_rows(planes_addr + buffer * kBuffer, beside, r);
      if constexpr (twice) fetch_rows(planes_addr + buffer * kBuffer + kTcPlane, second(beside), r);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  const int share = RAGGED ? 0 : int(cta_rank()) >> 1, stride = RAGGED ? 2 * kTcColumns : (2 * kTcColumns) << T.log_shares;
  const int first = (eg + 2 * share) * kTcColumns;
  // the buffer of the last tile's last step may still be read: the two others
  fetch(first, buffer);
  fetch(first + stride, buffer == 2 ? 0 : buffer + 1);
  bool ok = warp_wait(acc_full, parity, T, S);
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (!RAGGED && ok && T.log_shares) ok = exchange_sums(T, S, A.n, stages, acc_at, eg);
  if (!group_all(eg, ok)) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    return false;
  }
  for (int col = first; col < A.n; col += stride) {
    uint32_t v[kTcColumns];
    tmem_load(v, acc_at + uint32_t(col));
    if (!RAGGED && T.log_shares) add_sums(T, v, stages, col);
    unsigned char* x = planes + buffer * kBuffer;
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    group_barrier(eg);  // this step's input is there, and the buffer of the step before is free
    fetch(col + 2 * stride, buffer == 0 ? 2 : buffer - 1);
    buffer = buffer == 2 ? 0 : buffer + 1;
    const Rows<16> r([&](int c) { return row_of(col, c, row, valid); });
#pragma unroll
    for (int j = 0; j < kTcColumns; ++j) {
      unsigned char* z = x + j * kTcRowBytes + (q * 32 + lane) * 2;
      float d = __uint_as_float(v[j]);
      const float g = bf16_at(z);
      if constexpr (twice) {
        const float u = bf16_at(z + kTcPlane);
        put_bf16(z + kTcPlane, d * mm_act(HOC_ACT_SILU, g));
        d *= u * mm_act_slope(HOC_ACT_SILU, g);
      } else {
        d = mm_act_back(ACT, g, d);
      }
      put_bf16(z, d);
    }
    group_barrier(eg);
    put_rows(x, y, r);
    if constexpr (twice) put_rows(x + kTcPlane, second(y), r);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  return true;
}

// The same for the weight gradient: columns are out features, rows of the weight;
// nothing is read but the weights that are added to.
constexpr int kWgColumns = 16;
template <bool RAGGED>
__device__ __forceinline__ bool run_wgrad_epilogue(const TcParams& T, TcShared* S, const Tile& A, uint32_t stages,
                                                   unsigned char* out, uint32_t& turn, uint32_t acc_at, uint64_t* acc_full,
                                                   uint32_t parity, int eg, int q, int rank) {
  const MmParams& P = T.P;
  const int lane = threadIdx.x & 31, i = int(threadIdx.x) & 127;
  const int f0 = A.f0 + rank * 128, f = f0 + q * 32 + lane, left = P.in - f0;
  bool ok = true;
  if (A.steps > 0) {
    ok = warp_wait(acc_full, parity, T, S);
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if (!RAGGED && ok && T.log_shares) ok = exchange_sums(T, S, A.n, stages, acc_at, eg);
  }
  if (!group_all(eg, ok)) return false;
  const int share = RAGGED ? 0 : int(cta_rank()) >> 1, stride = RAGGED ? 2 * kWgColumns : (2 * kWgColumns) << T.log_shares;
  for (int col = (eg + 2 * share) * kWgColumns; col < A.n; col += stride) {
    uint32_t v[kWgColumns];
    if (A.steps > 0) {
      tmem_load(v, acc_at + uint32_t(col));
      if (!RAGGED && T.log_shares) add_sums(T, v, stages, col);
    } else {
#pragma unroll
      for (int j = 0; j < kWgColumns; ++j) v[j] = 0;
    }
    const int c0 = A.c0 + col;
    const int64_t at = (int64_t(A.g) * P.out + c0) * P.in;  // weight [c0][0]
    if (P.out_f32) {
      float* o = static_cast<float*>(P.y[A.p]) + at + f;
      if (P.accumulate) {
        float add[kWgColumns];
#pragma unroll
        for (int j = 0; j < kWgColumns; ++j) add[j] = f < P.in && c0 + j < P.out ? o[int64_t(j) * P.in] : 0.f;
#pragma unroll
        for (int j = 0; j < kWgColumns; ++j) v[j] = __float_as_uint(add[j] + __uint_as_float(v[j]));
      }
#pragma unroll
      for (int j = 0; j < kWgColumns; ++j)
        if (f < P.in && c0 + j < P.out) o[int64_t(j) * P.in] = __uint_as_float(v[j]);
      continue;
    }
    if (P.accumulate) {
      const __nv_bfloat16* w = static_cast<const __nv_bfloat16*>(P.y[A.p]) + at + f;
      float add[kWgColumns];
#pragma unroll
      for (int j = 0; j < kWgColumns; ++j) add[j] = f < P.in && c0 + j < P.out ? bf16_of(w + int64_t(j) * P.in) : 0.f;
#pragma unroll
      for (int j = 0; j < kWgColumns; ++j) v[j] = __float_as_uint(add[j] + __uint_as_float(v[j]));
    }
    unsigned char* o = out + (turn++ & 1) * (kWgColumns * kTcRowBytes);
#pragma unroll
    for (int j = 0; j < kWgColumns; ++j) put_bf16(o + j * kTcRowBytes + (q * 32 + lane) * 2, __uint_as_float(v[j]));
    group_barrier(eg);
    // 128 threads: 8 rows of 16 vectors at a time
    const int c = i / 16, u = i % 16;
    char* to = reinterpret_cast<char*>(static_cast<__nv_bfloat16*>(P.y[A.p]) + at) +
               (int64_t(c) * P.in + (left > 0 ? f0 : 0)) * 2 + u * 16;
#pragma unroll
    for (int h = 0; h < kWgColumns / 8; ++h) {
      const unsigned char* from = o + (i + 128 * h) * 16;
      char* row = to + int64_t(h) * 16 * P.in;
      const bool there = c0 + c + 8 * h < P.out && u * 8 < left;
      if (T.loose) put_loose(row, from, there ? left - u * 8 : 0);
      else if (there) *reinterpret_cast<uint4*>(row) = *reinterpret_cast<const uint4*>(from);
    }
  }
  return true;
}

// Bias gradient of one range of rows: the sums of dy's columns, 16 of them (a 32-byte
// sector) per CTA in turn, by four warps that have nothing else to do; their loads run
// beside the product's.  (A kernel of its own finds no room beside the product's CTAs
// and runs after them.)  Binary32; lanes, then warps, are added in a fixed order.  The
// weight gradient of 4096 rows of 4096 x 4096 takes 78 us, 80 with these sums, 86 with
// the kernel; 2047 rows of 2048 x 1408 19.5, 20.9 and 23.1.
__device__ __forceinline__ void sum_columns(const MmParams& P, TcShared* S, int w) {
  constexpr int kLoads = 8;  // in flight, of 64 rows each
  const int lane = threadIdx.x & 31, half = lane & 1, rows = int(P.cap[0]);
  int buffer = 0;
  for (int c0 = int(blockIdx.x) * 16; c0 < P.out; c0 += int(gridDim.x) * 16, buffer ^= 1) {
    const __nv_bfloat16* q = P.dy[0] + c0 + half * 8;
    const int end = c0 + half * 8 < P.out ? rows : 0;
    float acc[8] = {};
    for (int64_t r = w * 16 + (lane >> 1); r < end; r += kLoads * 64) {
      uint4 v[kLoads];
#pragma unroll
      for (int j = 0; j < kLoads; ++j)
        v[j] = r + 64 * j < end ? __ldg(reinterpret_cast<const uint4*>(q + (r + 64 * j) * P.ld_dy)) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const uint32_t x[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[2 * e] += __uint_as_float(x[e] << 16);
          acc[2 * e + 1] += __uint_as_float(x[e] & 0xFFFF0000u);
        }
      }
    }
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      for (int off = 16; off > 1; off >>= 1) acc[e] += __shfl_xor_sync(0xFFFFFFFFu, acc[e], off);
      if (lane < 2) S->sum[buffer][w][half * 8 + e] = acc[e];
    }
    asm volatile("bar.sync 3, 128;" ::: "memory");
    const int c = c0 + lane;
    if (w == 0 && lane < 16 && c < P.out) {
      float v = 0.f;
      for (int i = 0; i < 4; ++i) v += S->sum[buffer][i][lane];
      if (P.out_f32) {
        float* o = static_cast<float*>(P.pre_out[0]) + c;
        *o = P.accumulate ? *o + v : v;
      } else {
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(P.pre_out[0]) + c;
        *o = __float2bfloat16_rn(P.accumulate ? bf16_of(o) + v : v);
      }
    }
  }
}

// ------------------------------------------------------------------ kernel
// Shared memory: the stages, the planes of the two epilogue groups (two, or the six of
// three input buffers), the barriers and tile counts.
constexpr uint32_t kTcSmem = 232448;  // 227 KB
constexpr uint32_t planes_of(int mode, int act) { return mode == kDgrad && act != HOC_ACT_NONE ? 6 : 2; }
constexpr uint32_t stages_in(uint32_t planes, uint32_t stage) {
  const uint32_t n = (kTcSmem - 1024 - uint32_t(sizeof(TcShared)) - 2 * planes * kTcPlane) / stage;
  return n < uint32_t(kTcMostStages) ? n : uint32_t(kTcMostStages);
}
static_assert(kWgColumns == kTcColumns, "the planes are of one size");
static_assert(stages_in(2, kTcStage) == 6 && stages_in(6, kTcStage) == 5, "stages of a tile of 256 rows");

template <int MODE, bool RAGGED>
__global__ void __launch_bounds__(kTcThreads<MODE>, 1)
    mm_tc_kernel(const __grid_constant__ TcLaunch<RAGGED> L) {
  const TcParams& T = L.T;
  extern __shared__ unsigned char raw[];
  const uint32_t base = (ptx::smem_addr(raw) + 1023u) & ~1023u;
  unsigned char* stages = raw + (base - ptx::smem_addr(raw));
  unsigned char* planes = stages + T.stages * T.stage;
  TcShared* S = reinterpret_cast<TcShared*>(planes + 2 * T.planes * kTcPlane);
  const MmParams& P = T.P;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = int(cta_rank()) & 1;  // in the pair
  const int from = RAGGED ? 0 : int(cta_rank() >> 1) * T.per;  // this share's first stage
  const bool gated = MODE == kForward && P.act == HOC_ACT_SWIGLU;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kTcMostStages; ++s) {
      ptx::mbar_init(&S->full[s], MODE == kWgrad ? 2 : 6);  // both CTAs' producer warps
      ptx::mbar_init(&S->part[s], 1);
      ptx::mbar_init(&S->empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(&S->acc_full[a], 1);
      ptx::mbar_init(&S->acc_empty[a], 2 * kTcEpilogue);
    }
    ptx::mbar_init(&S->go, (1 << T.log_shares) - 1 + (T.log_shares == 0));
    ptx::mbar_init(&S->came, ((1 << T.log_shares) - 1) * kTcEpilogue + (T.log_shares == 0));
    S->dead = 0;
    S->moved = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(ptx::smem_addr(&S->tmem)),
                 "r"(kTcTmemColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  if (warp == 3 && lane < P.parts) {
    auto prefetch = [](const CUtensorMap* m) { asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory"); };
    if (MODE != kWgrad) prefetch(&L.w[P.part0 + lane]);
    if (P.cap[P.part0 + lane] > 0) prefetch(&L.row[P.part0 + lane][3]);
    if (MODE == kWgrad && P.cap[P.part0 + lane] > 0) prefetch(&L.dy[P.part0 + lane][3]);
  }
  // The other CTA's barriers are first used after the wait below.
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncwarp();
  cluster_arrive();
  if (RAGGED) {
    after_previous();
    mm_count(P, MODE == kWgrad ? kTcDepth : 8, S->vrows, S->tile0,
             [&](int rows) { return MODE == kWgrad ? 0u : T.rows.of(rows) * T.ftiles.d; });
    order_pairs<MODE>(T, S);
  }
  const unsigned tiles = tile_count<MODE, RAGGED>(T, S);
  const int log = RAGGED ? 1 : 1 + T.log_shares;  // of the cluster's CTAs
  const unsigned who = blockIdx.x >> log, of = gridDim.x >> log;

  if (warp == 0 || warp == (MODE == kWgrad ? 12 : 2)) {
    // ---- tensor copies of the rows.  The whole warp walks the stages, so that
    // addresses stay in uniform registers, and one lane issues what it can.
    const bool one = elect_one();
    const uint32_t full0 = on_first(&S->full[0]);
    const int block = warp != 0;  // forward, dgrad: the 64 rows of this CTA's half that the warp fetches
    auto own = [&](uint32_t st) { return MODE != kWgrad || int(st & 1) == block; };  // wgrad: its stages
    Turn k(T.stages);
    bool ok = true;
    // Waits until the MMAs have released the stage's last filling.
    auto free = [&]() { return k.round == 0 || warp_wait(&S->empty[k.st], (k.round - 1) & 1, T, S); };
    Work<RAGGED> W(T, S, who, of, tiles);
    each_tile<MODE, RAGGED>(W, true, [&]() {
      const Tile& A = W.now;
      const Ranges R = load_ranges<MODE == kWgrad ? kTcDepth : 8, RAGGED>(P, A.p, W.ends);
      const int half = A.n / 2;  // rows of B in this CTA (wgrad: features)
      if (MODE != kWgrad) {
        // This warp's 64 rows of B, a group of 8 per lane modulo 8
        const int mine = min(half - block * 64, 64);
        int row, left;
        group_at<8, RAGGED>(P, A.p, A.g, R, A.c0 + rank * half + block * 64 + (lane & 7) * 8, row, left);
        if ((lane & 7) * 8 >= mine) left = 0;
        // Columns of groups without rows are not stored: they are not fetched.
        const int any = box_at(row, left), box = left > 0 ? any : -1;
        const uint32_t bytes = uint32_t(__popc(__ballot_sync(0xFFFFFFFFu, left > 0) & 0xFFu)) * 1024u + T.tx_pad;
        const CUtensorMap* map = &L.row[A.p][box < 0 ? 0 : box];
        for (int s = 0; s < A.steps; ++s, k.next()) {
          if (!free()) {
            ok = false;
            break;
          }
          const uint32_t b = base + k.st * T.stage + kTcOperand + block * 8192u, bar = full0 + k.st * 8u;
          if (one) arrive_expect_cluster(bar, bytes);
          __syncwarp();
          if (lane < 8 && box >= 0) copy2(b + uint32_t(lane) * 1024u, map, (from + s) * kTcDepth, row, bar);
          __syncwarp();
        }
      } else {
        const int blocks = (half + 63) / 64;
        const uint32_t bytes = kTcOperand + uint32_t(blocks) * 8192u + T.tx_pad;
        const int fx = A.f0 + rank * 128, fd = A.c0 + rank * half;
        for (int s = 0; ok && s < A.steps;) {
          if (P.sources <= 32 && from + s >= R.wholes / kTcDepth && !own(k.st)) {  // remainders, the other warp's
            ++s;
            k.next();
            continue;
          }
          int row, valid;
          const int run = min(stage_rows<RAGGED>(P, A, R, from + s, row, valid), A.steps - s);
          int r = __shfl_sync(0xFFFFFFFFu, row, 0);
          for (int i = 0; i < run; ++i, r += kTcDepth, k.next()) {
            if (!own(k.st)) continue;
            if (!free()) {
              ok = false;
              break;
            }
            const uint32_t a = base + k.st * T.stage, bar = full0 + k.st * 8u;
            if (one) {
              S->moved = k.round * kTcMostStages + k.st + 1;
              arrive_expect_cluster(bar, bytes);
              copy2(a, &L.row[A.p][3], fx, r, bar);
              copy2(a + 8192u, &L.row[A.p][3], fx + 64, r, bar);
              copy2(a + kTcOperand, &L.dy[A.p][3], fd, r, bar);
              if (blocks > 1) copy2(a + kTcOperand + 8192u, &L.dy[A.p][3], fd + 64, r, bar);
            }
            __syncwarp();
          }
          s += run;
          if (run > 0) continue;
          if (!own(k.st)) {
            ++s;
            k.next();
            continue;
          }
          if (!free()) {
            ok = false;
            break;
          }
          // runs of several ranges: lanes are blocks of 64 features (0, 1 of x, then those of dy) x groups
          const uint32_t a = base + k.st * T.stage, bar = ptx::smem_addr(&S->part[k.st]);
          const int box = box_at(row, valid), which = lane >> 3;
          if (one) {
            S->moved = k.round * kTcMostStages + k.st + 1;
            arrive_expect_cluster(bar, bytes);
          }
          __syncwarp();
          if (which < 2 + blocks && box >= 0)
            copy2(a + uint32_t(which) * 8192u + uint32_t(lane & 7) * 1024u,
                  which < 2 ? &L.row[A.p][box] : &L.dy[A.p][box],
                  which < 2 ? fx + which * 64 : fd + (which - 2) * 64, row, bar);
          __syncwarp();
          ++s;
          k.next();
        }
      }
      return ok;
    });
    // The MMAs' last releases of the stages have to land before this CTA may leave.
    for (uint32_t j = 0; ok && j < T.stages; ++j, k.next()) ok = !own(k.st) || free();
  } else if (MODE != kWgrad && warp == 3) {
    // ---- tensor copies of the weights
    const bool one = elect_one();
    const uint32_t full0 = on_first(&S->full[0]);
    Turn k(T.stages);
    bool ok = true;
    Work<RAGGED> W(T, S, who, of, tiles);
    each_tile<MODE, RAGGED>(W, false, [&]() {
      const Tile& A = W.now;
      const int fa = A.f0 + rank * (gated ? 64 : 128);
      for (int s = 0; s < A.steps; ++s, k.next()) {
        if (k.round && !warp_wait(&S->empty[k.st], (k.round - 1) & 1, T, S)) {
          ok = false;
          break;
        }
        const uint32_t a = base + k.st * T.stage, bar = full0 + k.st * 8u;
        const int x = (from + s) * kTcDepth;
        if (one) {
          arrive_expect_cluster(bar, kTcOperand);
          if (MODE == kDgrad) {
            copy3(a, &L.w[A.p], fa, x, A.g, bar);
            copy3(a + 8192u, &L.w[A.p], fa + 64, x, A.g, bar);
          } else if (gated) {
            copy5(a, &L.w[A.p], x, 0, 0, fa / 8, A.g, bar);
          } else {
            copy3(a, &L.w[A.p], x, fa, A.g, bar);
          }
        }
        __syncwarp();
      }
      return ok;
    });
  } else if (warp == 1 && rank == 0) {
    // ---- MMA
    const bool one = elect_one();
    Turn k(T.stages);
    uint32_t it = 0;
    bool ok = true;
    const uint32_t kind = (1u << 4) | (1u << 7) | (1u << 10) | (MODE != kForward ? 1u << 15 : 0u) |
                          (MODE == kWgrad ? 1u << 16 : 0u) | (uint32_t(kTcFeatures / 16) << 24);
    const uint64_t a0 = MODE == kForward ? smem_desc(base, 16, 1024) : smem_desc(base, 8192, 1024);
    const uint64_t b0 = MODE == kWgrad ? smem_desc(base + kTcOperand, 8192, 1024) : smem_desc(base + kTcOperand, 16, 1024);
    Work<RAGGED> W(T, S, who, of, tiles);
    for (;;) {  // once without a tile: the next one is looked up under a tile's first products
      const Tile& A = W.now;
      const bool run = W.more && A.steps > 0;  // an expert without rows: the epilogue writes zeros
      const uint32_t idesc = kind | (uint32_t(A.n / 8) << 17);
      const uint32_t acc = it & 1, d = S->tmem + acc * 256u;
      if (run && it >= 2 && !warp_wait(&S->acc_empty[acc], ((it >> 1) - 1) & 1, T, S)) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const int steps = run ? A.steps : 1;
      for (int s = 0; s < steps; ++s) {
        if (run) {
          if (!warp_wait<MODE == kWgrad>(&S->full[k.st], k.round & 1, T, S)) {  // wgrad: the other CTA's zeros too
            ok = false;
            break;
          }
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint64_t da = a0 + k.st * (T.stage >> 4), db = b0 + k.st * (T.stage >> 4);
          if (one) {
#pragma unroll
            for (int q = 0; q < kTcDepth / 16; ++q)  // 16 deep: 32 bytes along a K-major row, 16 rows of an M/N-major block
              mma_pair(d, da + q * (MODE == kForward ? 2 : 128), db + q * (MODE == kWgrad ? 128 : 2), idesc, s | q);
            commit_pair(&S->empty[k.st]);
          }
          __syncwarp();
          k.next();
        }
        if (s == 0) W.template look_ahead<MODE>(false);
      }
      if (!W.more) begin<RAGGED>();
      if (!ok) break;
      if (run) {
        if (one) commit_pair(&S->acc_full[acc]);
        __syncwarp();
        ++it;
      }
      if (!W.ahead_more) break;
      W.next();
    }
  } else if (MODE == kWgrad && !RAGGED && (warp == 3 || warp > 12)) {
    begin<RAGGED>();
    if (T.sums) sum_columns(P, S, warp == 3 ? 0 : warp - 12);
  } else if (MODE == kWgrad && (warp == 2 || warp == 3 || warp > 12)) {
    // ---- zero the padding rows of the stages that hold any, then hand them to the
    // MMA.  A release to the cluster takes about 1400 cycles, the MMAs of a stage 512:
    // five warps, each with stages of its own, so that a warp waits on every phase of
    // the barriers that it waits on.  (One range has one such stage at most: one warp.)
    const uint32_t own = warp < 4 ? warp - 2 : warp - 11;
    const uint32_t full0 = on_first(&S->full[0]);
    Turn k(T.stages);
    uint32_t phases = 0;  // bit st: parity of part[st]
    bool ok = true;
    Work<RAGGED> W(T, S, who, of, tiles);
    each_tile<MODE, RAGGED>(W, true, [&]() {
      const Tile& A = W.now;
      const Ranges R = load_ranges<kTcDepth, RAGGED>(P, A.p, W.ends);
      for (int s = 0; s < A.steps;) {
        int row, valid;
        const int run = min(stage_rows<RAGGED>(P, A, R, from + s, row, valid), A.steps - s);
        for (int i = 0; i < run; ++i) k.next();
        s += run;
        if (run > 0) continue;
        const uint32_t st = k.st;
        k.next();
        ++s;
        if (RAGGED && st % 5 != own) continue;
        if (!warp_wait(&S->part[st], (phases >> st) & 1, T, S)) {
          ok = false;
          break;
        }
        phases ^= 1u << st;
        // lanes: 4 blocks of 64 features (2 of x, 2 of dy) x 8 vectors of a 128-byte row
        // (a group without rows came from past the buffer's end: zeros already)
        unsigned char* at = stages + size_t(st) * T.stage + (lane >> 3) * 8192 + (lane & 7) * 16;
        unsigned partial = __ballot_sync(0xFFFFFFFFu, valid > 0 && valid < 8) & 0xFFu;
        while (partial) {
          const int gi = __ffs(partial) - 1;
          partial &= partial - 1;
          const int nv = __shfl_sync(0xFFFFFFFFu, valid, gi);
#pragma unroll
          for (int r = 1; r < 8; ++r)
            if (r >= nv) *reinterpret_cast<uint4*>(at + (gi * 8 + r) * 128) = make_uint4(0, 0, 0, 0);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) arrive_cluster(full0 + st * 8u);
      }
      return ok;
    });
  } else if (warp >= 4 && warp < 4 + kTcEpilogue) {
    // ---- epilogue: two groups of four warps take turns along the columns
    const int q = warp & 3, eg = (warp - 4) / 4;
    unsigned char* mine = planes + eg * T.planes * kTcPlane;
    uint32_t it = 0, turn = 0, buffer = 0;
    Work<RAGGED> W(T, S, who, of, tiles);
    each_tile<MODE, RAGGED>(W, MODE != kWgrad, [&]() {
      const Tile& A = W.now;
      int row = 0, valid = 0;
      float bias = 0.f;
      if (MODE != kWgrad) {
        group_at<8, RAGGED>(P, A.p, A.g, load_ranges<8, RAGGED>(P, A.p, W.ends), A.c0 + lane * 8, row, valid);
        valid = lane * 8 < T.tile_rows ? min(valid, 8) : 0;  // past them: the next tile's rows
        const int f = gated ? A.f0 + rank * 64 + q * 16 + lane / 16 * 8 + (lane & 7) : A.f0 + rank * 128 + q * 32 + lane;
        if (MODE == kForward && P.bias[A.p] && f < P.out)
          bias = bf16_of(P.bias[A.p] + int64_t(A.g) * (gated ? 2 : 1) * P.out + (gated && (lane & 8) ? P.out : 0) + f);
      }
      if (MODE == kWgrad && A.steps == 0 && P.accumulate) return true;  // an expert without rows adds nothing
      const uint32_t acc = it & 1;
      const uint32_t at = S->tmem + acc * 256u + (uint32_t(q * 32) << 16);
      bool ok = true;
      if constexpr (MODE == kWgrad) {
        ok = run_wgrad_epilogue<RAGGED>(T, S, A, base, mine, turn, at, &S->acc_full[acc], (it >> 1) & 1, eg, q, rank);
      } else {
        with_act(P.act, [&](auto tag) {
          constexpr int act = decltype(tag)::act;
          if constexpr (MODE == kDgrad && act != HOC_ACT_NONE)
            ok = run_slope_epilogue<act, RAGGED>(T, S, A, base, mine, buffer, at, &S->acc_full[acc], (it >> 1) & 1, eg, q,
                                                 rank, row, valid);
          else
            ok = run_epilogue<MODE, act, RAGGED>(T, S, A, base, ptx::smem_addr(mine), at, &S->acc_full[acc], (it >> 1) & 1,
                                                 eg, q, rank, row, valid, bias);
        });
      }
      if (!ok) return false;
      if (A.steps == 0) return true;  // no accumulator was used
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) arrive_relaxed(on_first(&S->acc_empty[acc]));
      ++it;
      return true;
    });
  } else {
    begin<RAGGED>();
  }
  __syncwarp();
  if (S->dead) {
    // A wait gave up.  Copies already issued have had the whole limit of that
    // wait to land, those of a role that was still moving land within this pause.
    for (int i = 0; i < 64; ++i) __nanosleep(1000);
  }
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  cluster_arrive();
  cluster_wait();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (warp == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(S->tmem), "r"(kTcTmemColumns));
}

template <bool RAGGED>
using TcFn = void (*)(TcLaunch<RAGGED>);
template <bool RAGGED>
constexpr TcFn<RAGGED> kTc[3] = {mm_tc_kernel<kForward, RAGGED>, mm_tc_kernel<kDgrad, RAGGED>, mm_tc_kernel<kWgrad, RAGGED>};

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
  const cuuint64_t in = P.in, out = P.out, ld = P.ld_w, rows = P.out_w, ne = P.experts;
  if (mode == kForward && P.act == HOC_ACT_SWIGLU) {
    // [expert][gate, value][out / 8][8][in], fetched so that 8 gates and their 8 values alternate
    // (16 and 16 would need copies of the weights where out is no multiple of 16)
    const cuuint64_t dims[5] = {in, 8, 2, rows / 8, ne}, strides[4] = {ld, rows * ld, 8 * ld, 2 * rows * ld};
    const cuuint32_t box[5] = {kTcDepth, 8, 2, 8, 1};
    return encode(m, at, 5, dims, strides, box);
  }
  const cuuint64_t dims[3] = {in, out, ne}, strides[2] = {ld, rows * ld};
  const cuuint32_t box[3] = {kTcDepth, mode == kForward ? 128u : 64u, 1};
  return encode(m, at, 3, dims, strides, box);
}

// Ragged rows: 256, since a tile's MMAs are only as wide as the rows that it has,
// unless the buffers' room says that an expert has few rows on average; lower tiles
// then leave shared memory for more stages, and the weights that a decoding step
// streams need many bytes in flight.
int choose_rows_ragged(const MmParams& P) {
  int64_t rows = 0;
  for (int p = P.part0; p < P.part0 + P.parts; ++p) rows += P.cap[p];
  const int64_t each = rows / P.parts / P.experts;
  return each <= 32 ? 64 : each <= 64 ? 128 : kTcRows;
}

// The launch but for its grid and stream, and the clusters that fit the device at
// once (asked once for each kernel, cluster size and device).
cudaError_t configure(const void* fn, int mode, bool ragged, int log_shares, cudaLaunchAttribute (&attr)[2],
                      cudaLaunchConfig_t& cfg, int& clusters) {
  static std::atomic<int> known[3][kTcMostShares + 2][64];  // ragged ones last
  const int kind = ragged ? kTcMostShares + 1 : log_shares;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2u << log_shares;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(mode == kWgrad ? kTcThreads<kWgrad> : kTcThreads<kForward>);
  cfg.dynamicSmemBytes = kTcSmem;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  clusters = dev < 64 ? known[mode][kind][dev].load() : 0;
  if (clusters > 0) return cudaSuccess;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kTcSmem));
  if (e != cudaSuccess) return e;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(2u << log_shares);
  e = cudaOccupancyMaxActiveClusters(&clusters, fn, &cfg);
  cfg.numAttrs = 2;
  if (e == cudaSuccess && clusters < 1) e = cudaErrorInvalidConfiguration;
  if (e == cudaSuccess && dev < 64) known[mode][kind][dev].store(clusters);
  return e;
}

// Rows of a tile, and shares of its contraction, where the number of rows is known (one
// range, or the features of the weight gradient): those that take the fewest cycles.
// With several waves of tiles a stage of r rows costs about 256 + r (its features'
// operand comes with every tile), e.g. 4096 rows x 16 feature tiles on 76 pairs: 4 waves
// of 224 rows instead of 4 of 256 (101 -> 95 us at 4096 deep); a single wave waits for
// memory, about 640 a stage whatever its height.  Sharing costs two hand-overs across
// the cluster and the sums' way.
struct Cut {
  int rows, log_shares;
};
Cut choose_cut(int64_t rows, int64_t others, int64_t steps, const int* clusters, int most_shares) {
  Cut best{kTcRows, 0};
  int64_t least = INT64_MAX;
  for (int r = kTcRows; r >= 64; r -= 32)
    for (int log = 0; log <= most_shares; ++log) {
      const int64_t tiles = (rows + r - 1) / r * others, waves = (tiles + clusters[log] - 1) / clusters[log];
      const int64_t per = (steps + (1 << log) - 1) >> log;
      if (log && (waves > 1 || per * ((1 << log) - 1) >= steps)) continue;
      const int64_t stage = waves == 1 ? 640 : waves * (r < 144 ? 400 : 256 + r);
      const int64_t cost = stage * per + (16 * r >> log) + (log == 0 ? 0 : log == 1 ? 3000 + 32 * r : 4000 + 48 * r);
      if (cost < least) {
        least = cost;
        best = {r, log};
      }
    }
  return best;
}

}  // namespace

bool mm_tc_takes(const MmParams& P, int mode) {
  const bool gated = mode == kForward && P.act == HOC_ACT_SWIGLU;
  if (P.ld_rows % 8 || (mode == kWgrad ? P.ld_dy % 8 : P.ld_w % 8) || (gated && P.out_w % 8)) return false;
  uintptr_t at = 0;
  for (int p = 0; p < P.parts; ++p)
    at |= reinterpret_cast<uintptr_t>(P.rows[p]) | reinterpret_cast<uintptr_t>(P.dy[p]) | reinterpret_cast<uintptr_t>(P.w[p]);
  return (at & 15u) == 0 && encoder() != nullptr;
}

bool mm_tc_loose(const MmParams& P, int mode) {
  const int width = mode == kForward ? P.out : P.in;
  if (width % 8 || P.ld_y % 8) return true;
  uintptr_t at = 0;
  for (int p = P.part0; p < P.part0 + P.parts; ++p) {
    at |= reinterpret_cast<uintptr_t>(P.y[p]) | reinterpret_cast<uintptr_t>(P.pre[p]) | reinterpret_cast<uintptr_t>(P.res[p]);
    if (mode == kForward) at |= reinterpret_cast<uintptr_t>(P.pre_out[p]);
    if (P.res[p] && P.ld_res % 8) return true;
  }
  return (at & 15u) != 0;
}

template <bool RAGGED>
static cudaError_t launch(const MmParams& P, int mode, cudaStream_t s, bool* summed) {
  TcLaunch<RAGGED> L;
  TcParams& T = L.T;
  T.P = P;
  T.loose = mm_tc_loose(P, mode);
  const char* fault = getenv("HOC_FAULT");
  const bool stall = fault && !strcmp(fault, "mm_stall");
  T.tx_pad = stall ? 16u : 0u;
  T.wait_ns = stall ? 100000000ull : fault && !strcmp(fault, "mm_hurry") ? 1000000ull : kTcWaitNs;
  const void* fn = reinterpret_cast<const void*>(kTc<RAGGED>[mode]);
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = {};
  cudaError_t e = cudaSuccess;
  int64_t tiles = 0;
  const int ftile = mode == kForward && P.act == HOC_ACT_SWIGLU ? kTcFeatures / 2 : kTcFeatures;
  const int64_t ftiles = ((mode == kForward ? P.out : P.in) + ftile - 1) / ftile;
  const int64_t depth = mode == kForward ? P.in : mode == kDgrad ? P.out : P.cap[P.part0];
  const int64_t steps = (depth + kTcDepth - 1) / kTcDepth;
  Cut cut{0, 0};
  int clusters[kTcMostShares + 1] = {};
  const int most = RAGGED ? 0 : kTcMostShares;
  for (int log = most; log >= 0 && e == cudaSuccess; --log) e = configure(fn, mode, RAGGED, log, attr, cfg, clusters[log]);
  if (e != cudaSuccess) return e;
  if (mode == kWgrad) cut = choose_cut(P.out, ftiles * P.groups * P.parts, steps, clusters, most);
  else if (!RAGGED) cut = choose_cut(P.cap[0], ftiles, steps, clusters, most);
  else cut.rows = choose_rows_ragged(P);
  T.tile_rows = cut.rows;
  T.log_shares = cut.log_shares;
  T.per = T.log_shares ? int((steps + (1 << T.log_shares) - 1) >> T.log_shares) : INT_MAX;
  if (T.log_shares) e = configure(fn, mode, RAGGED, T.log_shares, attr, cfg, clusters[T.log_shares]);
  if (e != cudaSuccess) return e;
  cfg.stream = s;
  T.stage = mode == kWgrad ? kTcStage : kTcOperand + uint32_t(T.tile_rows) * (kTcDepth * 2 / 2);
  T.planes = planes_of(mode, P.act);
  T.ftiles = divisor(uint32_t(ftiles));
  T.ctiles = divisor(uint32_t((P.out + T.tile_rows - 1) / T.tile_rows));
  T.each = divisor(T.ctiles.d * T.ftiles.d);
  T.groups = divisor(uint32_t(P.groups));
  T.rows = divisor(uint32_t(T.tile_rows));
  T.stages = stages_in(T.planes, T.stage);
  for (int p = P.part0; p < P.part0 + P.parts; ++p) {
    tiles += ftiles * (mode == kWgrad ? int64_t(P.groups) * ((P.out + T.tile_rows - 1) / T.tile_rows)
                                      : P.cap[p] / T.tile_rows + int64_t(P.groups) * (1 + P.sources * 8 / T.tile_rows));
    bool ok = mode == kWgrad || encode_weight(&L.w[p], P, mode, P.w[p]);
    if (P.cap[p] > 0) {  // a buffer without rows has no tile that reads it
      const int64_t width = mode == kDgrad ? P.out : P.in;
      for (int i = 0; i < 4; ++i) {
        ok = ok && encode_rows(&L.row[p][i], P.rows[p], width, P.cap[p], P.ld_rows, 8 << i);
        if (mode == kWgrad) ok = ok && encode_rows(&L.dy[p][i], P.dy[p], P.out, P.cap[p], P.ld_dy, 8 << i);
      }
    }
    if (!ok) return cudaErrorInvalidValue;
  }
  const int at_once = clusters[T.log_shares];
  cfg.gridDim = dim3(unsigned(tiles < 1 ? 1 : tiles < at_once ? tiles : at_once) << (1 + T.log_shares));
  T.sums = 0;
  if (!RAGGED && mode == kWgrad && P.pre_out[0] && P.out % 8 == 0) {
    // Where it takes no longer than the product: a round of 16 columns takes about half as long as a wave of tiles.
    const int64_t rounds = ((P.out + 15) / 16 + cfg.gridDim.x - 1) / cfg.gridDim.x, waves = (tiles + at_once - 1) / at_once;
    T.sums = (rounds << T.log_shares) <= 2 * waves;
    *summed = T.sums;
  }
  return cudaLaunchKernelEx(&cfg, kTc<RAGGED>[mode], L);
}

cudaError_t launch_mm_tc(const MmParams& P, int mode, cudaStream_t s, bool* summed) {
  return P.seg == nullptr ? launch<false>(P, mode, s, summed) : launch<true>(P, mode, s, summed);
}

cudaError_t mm_tc_preload() {
  cudaError_t e = cudaSuccess;
  auto load = [&](auto fn) {
    cudaFuncAttributes a;
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, reinterpret_cast<const void*>(fn));
  };
  for (auto fn : kTc<false>) load(fn);
  for (auto fn : kTc<true>) load(fn);
  return e;
}

}  // namespace hoc
