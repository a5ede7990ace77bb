// Routing of tokens to experts, and its gradient (hoc_block.h).
//
// L neighbouring lanes take a token, so that a warp works on 32 / L of them at a time: what
// is done once a token and round is bound by instructions, not by bytes.  Lane q of a
// token holds the logits of the experts q * epl .. (q + 1) * epl - 1, so that the lowest of
// several lanes with the same key has the lowest expert, and a group of neighbouring
// experts is a run of lanes.  A lane sorts its keys once, as unsigned numbers whose last bits
// are the expert's place in the lane; the topk largest are then found one after the other:
// a maximum over the lanes' first keys, and the lane that had it moves its others up.
//
// Which of two near keys is larger is decided as 64-bit arithmetic decides it.  Keys are
// binary32 without their last bits, with a bound on their error.  Where two neighbours in the
// order lie within it, the keys that may be chosen are worked out again in binary64, a lane each, and ranked; where a
// group's place is in doubt, or more keys than lanes, the whole token is done again.  For normal logits of standard
// deviation 1 and 256 experts these are 0.2 % and 0.03 % of the tokens.  It depends on the scores: the softmax's
// bound is that of its largest score, so that peaked ones leave many keys in doubt that a bias alone tells apart.  32,768
// tokens, binary32 logits, a bias in steps of 0.001: top-6 of 64 by softmax 12.9, 32.6 and 105 us at standard deviations 1, 4
// and 8, by sigmoid 8.0, 8.0 and 9.8; top-8 of 256 in 4 of 8 groups 43, 187 and 385 us, and 26.6, 28.3 and 32.1.
// Keys with the same logit and the same bias are equal in any arithmetic, so that logits
// of few bits do not send their tokens there.  bf16 logits that are keys themselves have the bits
// to spare and are exact.
#include <cfloat>
#include <type_traits>
#include <utility>

#include "block.h"

namespace hoc {
namespace {

using namespace block;

constexpr int kRouteWarps = 8;
constexpr int kMaxExperts = HOC_ROUTE_MAX_EXPERTS;
constexpr int kMaxGroups = 32;

struct RouteArgs {
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* gate;
  int64_t ld;
  int tokens, experts, topk, groups, top_groups, softmax, renorm;
  int epl, vec;            // experts of a lane where L lanes take a token, and elements of an access to the logits
  int epl_warp, vec_warp;  // the same where a warp does
  int vec_bias;            // and of one to the bias
  float scale;
};

__device__ __forceinline__ float warp_max(float v) {  // (a NaN takes no part)
  asm volatile("redux.sync.max.f32 %0, %0, 0xffffffff;" : "+f"(v));
  return v;
}

// Keys as unsigned numbers in the same order; 0: not to be chosen (-inf and NaN).
// Both zeros are one.
__device__ __forceinline__ uint32_t ordered(float k) {
  const uint32_t b = __float_as_uint(k + 0.f);
  return k > -INFINITY ? b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u) : 0u;
}
__device__ __forceinline__ uint64_t ordered(double k) {
  const uint64_t b = uint64_t(__double_as_longlong(k + 0.0));
  return k > -INFINITY ? (b >> 63 ? ~b : b | (uint64_t(1) << 63)) : uint64_t(0);
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return o ? __uint_as_float(o >> 31 ? o & 0x7FFFFFFFu : ~o) : -INFINITY;
}
__device__ __forceinline__ double value_of(uint64_t o) {
  return o ? __longlong_as_double(int64_t(o >> 63 ? o & ~(uint64_t(1) << 63) : ~o)) : -double(INFINITY);
}

__device__ __forceinline__ uint32_t warp_most(uint32_t v) { return __reduce_max_sync(kAll, v); }
__device__ __forceinline__ uint64_t warp_most(uint64_t v) {
  const uint32_t hi = __reduce_max_sync(kAll, uint32_t(v >> 32));
  return uint64_t(hi) << 32 | __reduce_max_sync(kAll, uint32_t(v >> 32) == hi ? uint32_t(v) : 0u);
}

// The L lanes of a token.
template <int L>
__device__ __forceinline__ uint32_t most_of(uint32_t v) {
  if constexpr (L == 32) {
    return warp_most(v);
  } else if constexpr (L == 16) {  // two reductions of a warp are fewer instructions than four exchanges
    const bool low = (threadIdx.x & 16) == 0;
    const uint32_t a = warp_most(low ? v : 0u), b = warp_most(low ? 0u : v);
    return low ? a : b;
  } else {
#pragma unroll
    for (int off = L / 2; off; off >>= 1) v = max(v, __shfl_xor_sync(kAll, v, off));
    return v;
  }
}
template <int L>
__device__ __forceinline__ uint64_t most_of(uint64_t v) {
#pragma unroll
  for (int off = L / 2; off; off >>= 1) {
    const uint64_t w = __shfl_xor_sync(kAll, v, off);
    v = w > v ? w : v;
  }
  return v;
}
template <int L>
__device__ __forceinline__ float max_of(float v) {  // (a NaN takes no part)
  if constexpr (L == 32) {
    return warp_max(v);
  } else {
#pragma unroll
    for (int off = L / 2; off; off >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, off));
    return v;
  }
}
template <int L, class K>
__device__ __forceinline__ K sum_of(K v) {
#pragma unroll
  for (int off = L / 2; off; off >>= 1) v += __shfl_xor_sync(kAll, v, off);
  return v;
}
// The lanes of the token for which `yes` holds, a bit each.
template <int L>
__device__ __forceinline__ uint32_t lanes_of(bool yes) {
  const uint32_t all = __ballot_sync(kAll, yes);
  return L == 32 ? all : all >> (threadIdx.x & 31 & ~(L - 1)) & ((1u << (L & 31)) - 1);
}

// Calls by(elements of an access), known when compiling; vec divides a lane's share.
template <class T, int EPL, class By>
__device__ __forceinline__ void with_access(int vec, By by) {
  if (EPL >= 8 && sizeof(T) == 2 && vec == 8) by(std::integral_constant<int, EPL >= 8 && sizeof(T) == 2 ? 8 : 1>{});
  else if (EPL >= 4 && vec == 4) by(std::integral_constant<int, EPL >= 4 ? 4 : 1>{});
  else if (EPL >= 2 && vec == 2) by(std::integral_constant<int, EPL >= 2 ? 2 : 1>{});
  else by(std::integral_constant<int, 1>{});
}

// The logits of a token's lane q; -inf for experts there are none of, and for NaN.
template <class T, int EPL>
__device__ __forceinline__ void load_logits(const T* row, int experts, int epl, int vec, int q, float (&z)[EPL]) {
  const int e0 = q * epl;
  auto by = [&](auto step) {
    constexpr int S = decltype(step)::value;
#pragma unroll
    for (int i = 0; i < EPL; i += S) {
      Vec<T, S> v;
      const bool in = i < epl && e0 + i < experts;
      if (in) v = *reinterpret_cast<const Vec<T, S>*>(row + e0 + i);
#pragma unroll
      for (int e = 0; e < S; ++e) {
        z[i + e] = in ? fmaxf(widen(v.v[e]), -INFINITY) : -INFINITY;  // (of a number and NaN the number)
      }
    }
  };
  with_access<T, EPL>(vec, by);
}

// exp(z - most) of a softmax: 1 for the largest also where it is infinite, 0 for a masked one.
__device__ __forceinline__ float share(float z, float most) {
  return z == -INFINITY ? 0.f : z == most ? 1.f : expf(z - most);
}
__device__ __forceinline__ double share(double z, double most) {
  return z == -double(INFINITY) ? 0.0 : z == most ? 1.0 : exp(z - most);
}

// For keys: 1 / (1 + 2^(-z log2 e)) by the approximate instructions.
__device__ __forceinline__ float sigmoid(float z) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.44269504088896341f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(1.f + e));
  return e;
}
__device__ __forceinline__ double sigmoid(double z) { return 1.0 / (1.0 + exp(-z)); }

// Bounds on the error of a binary32 score, relative to the largest score there can be.
// Sigmoid: its exponent is rounded, which changes s by |z| s (1 - s) 2^-24 < 0.23 * 2^-24, the
// exponential by 2 units of 2^-23 of itself, s by a quarter of that; 1 + e and the reciprocal by
// 2^-24 and 2^-23: below 2^-21.
constexpr float kSigmoidError = 0x1p-21f;
// Softmax, in units of 2^-24: z - most is rounded, which changes exp by |z - most| of itself, 0.4 at
// most beside the largest (x exp(-x)); expf 4; the reciprocal of the sum and the product with it
// 1 each; in the sum EPL + 5 additions, and of its terms 4 for expf and their mean |z - most|, which
// is below log(1024) = 7: EPL + 23 in all.
template <int EPL>
constexpr float kSoftmaxError = float(EPL + 32) * 0x1p-24f;

// The largest and second largest key of a set (0: none).
template <class U>
struct Two {
  U a, b;
  __device__ __forceinline__ void add(U v) {
    b = max(b, min(a, v));
    a = max(a, v);
  }
  __device__ __forceinline__ void join(U a2, U b2) {
    b = max(min(a, a2), max(b, b2));
    a = max(a, a2);
  }
};

// Which groups are kept, a bit each: the top_groups largest scores, lane g having group g's.
// *last and *next: the least that is kept and the largest that is not (0: there is none).
template <int L, class U>
__device__ __forceinline__ uint32_t keep_groups(int top_groups, U mine, int q, U* last, U* next) {
  uint32_t kept = 0;
  *last = 0;
  for (int r = 0; r < top_groups; ++r) {
    const U most = most_of<L>(mine);
    const int winner = __ffs(lanes_of<L>(mine == most)) - 1;
    if (most) {
      *last = most;
      kept |= 1u << winner;
    }
    if (q == winner) mine = 0;
  }
  *next = most_of<L>(mine);
  return kept;
}

// The two largest keys of every group, at lane g for group g.
template <int EPL, int L = 32, class U>
__device__ __forceinline__ Two<U> two_of_groups(int experts, int groups, int epl, int q, const U (&u)[EPL]) {
  const int per = experts / groups;
  Two<U> mine{0, 0};
  for (int g = 0; g < groups; ++g) {
    Two<U> t{0, 0};
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = q * epl + i;
      if (i < epl && e >= g * per && e < (g + 1) * per) t.add(u[i]);
    }
    for (int off = 1; off < L; off <<= 1) {
      const U a = __shfl_xor_sync(kAll, t.a, off), b = __shfl_xor_sync(kAll, t.b, off);
      t.join(a, b);
    }
    if (q == g) mine = t;
  }
  return mine;
}

// Takes the largest key of the warp out of u.  Returns its expert; -1 where there is none left.
template <class U, int EPL>
__device__ __forceinline__ int pop(U (&u)[EPL], U& best, int epl, int lane) {
  const U m = warp_most(best);
  if (m == 0) return -1;
  const int winner = __ffs(__ballot_sync(kAll, best == m)) - 1;
  int at = 0;
  if (lane == winner) {
    best = 0;
    bool found = false;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const bool it = !found && u[i] == m;
      if (it) {
        at = i;
        u[i] = 0;
        found = true;
      }
      best = u[i] > best ? u[i] : best;
    }
  }
  return winner * epl + __shfl_sync(kAll, at, winner);
}

// The token once more in binary64, by the whole warp: lane j's slot j.
template <class T, int EPL>
__device__ __noinline__ int route_exactly(const RouteArgs& A, const T* row, int lane) {
  const bool grouped = A.top_groups < A.groups, scored = A.bias || grouped;
  const int epl = A.epl_warp;
  float z[EPL];
  load_logits<T, EPL>(row, A.experts, epl, A.vec_warp, lane, z);
  double most = -INFINITY, sum = 0;
  if (scored && A.softmax) {
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i) top = fmaxf(top, z[i]);
    most = warp_max(top);
#pragma unroll
    for (int i = 0; i < EPL; ++i) sum += share(double(z[i]), most);
    sum = sum_of<32>(sum);
  }
  uint64_t u[EPL], best = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane * epl + i;
    u[i] = 0;
    if (i < epl && e < A.experts && z[i] > -INFINITY) {
      const double k = !scored ? double(z[i]) : A.softmax ? share(double(z[i]), most) / sum : sigmoid(double(z[i]));
      u[i] = ordered(k + (A.bias ? double(A.bias[e]) : 0.0));
    }
  }
  if (grouped) {
    const int per = A.experts / A.groups, run = per / epl;
    Two<uint64_t> t{0, 0};
    if (per % epl == 0 && (run & (run - 1)) == 0) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) t.add(u[i]);
      for (int off = 1; off < run; off <<= 1) {
        const uint64_t a = __shfl_xor_sync(kAll, t.a, off), b = __shfl_xor_sync(kAll, t.b, off);
        t.join(a, b);
      }
      t.a = __shfl_sync(kAll, t.a, lane * run & 31);
      t.b = __shfl_sync(kAll, t.b, lane * run & 31);
    } else {
      t = two_of_groups<EPL>(A.experts, A.groups, epl, lane, u);
    }
    const double score = t.b ? value_of(t.a) + value_of(t.b) : value_of(t.a);
    uint64_t last, next;
    const uint32_t kept = keep_groups<32>(A.top_groups, lane < A.groups ? ordered(score) : uint64_t(0), lane, &last, &next);
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (u[i] && !(kept >> ((lane * epl + i) / per) & 1)) u[i] = 0;
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) best = u[i] > best ? u[i] : best;
  int mine = -1;
  for (int r = 0; r < A.topk; ++r) {
    const int id = pop(u, best, epl, lane);
    if (id < 0) break;
    if (lane == r) mine = id;
  }
  return mine;
}

// The exchanges of Batcher's odd-even merge sort of N keys, worked out by the compiler (loops
// that it does not unroll leave the keys in local memory: top-1 of 256 for 32,768 tokens 31.7 us,
// so 14.2).
template <int N>
struct Exchanges {
  int n = 0;
  unsigned char a[N * 8] = {}, b[N * 8] = {};
  constexpr Exchanges() {
    for (int p = 1; p < N; p <<= 1)
      for (int k = p; k >= 1; k >>= 1)
        for (int j = k % p; j + k < N; j += 2 * k)
          for (int i = 0; i < k && i + j + k < N; ++i)
            if ((i + j) / (2 * p) == (i + j + k) / (2 * p)) {
              a[n] = static_cast<unsigned char>(i + j);
              b[n++] = static_cast<unsigned char>(i + j + k);
            }
  }
};

template <int A, int B, int N>
__device__ __forceinline__ void exchange(uint32_t (&u)[N]) {
  const uint32_t a = u[A], b = u[B];
  u[A] = max(a, b);
  u[B] = min(a, b);
}

template <int N, size_t... I>
__device__ __forceinline__ void sort_keys(uint32_t (&u)[N], std::index_sequence<I...>) {
  constexpr Exchanges<N> net{};
  (exchange<net.a[I], net.b[I]>(u), ...);
}

// Largest first.
template <int N>
__device__ __forceinline__ void sort_keys(uint32_t (&u)[N]) {
  constexpr size_t n = Exchanges<N>{}.n;
  sort_keys<N>(u, std::make_index_sequence<n>{});
}

// The next of the token's sorted keys: its lane, and the key in *key (0: none is left).  The
// lanes' first keys are compared without their places, but with the lane in their stead: of
// equal ones the first lane's is the largest.
template <int EPL, int L>
__device__ __forceinline__ int pop_sorted(uint32_t (&u)[EPL], int q, uint32_t* key) {
  constexpr uint32_t kLow = (EPL > L ? EPL : L) - 1;
  const uint32_t m = most_of<L>((u[0] & ~kLow) | uint32_t(L - 1 - q));
  const int winner = L - 1 - int(m & (L - 1));
  *key = __shfl_sync(kAll, u[0], winner, L);
  if (q == winner) {
#pragma unroll
    for (int i = 0; i + 1 < EPL; ++i) u[i] = u[i + 1];
    u[EPL - 1] = 0;
  }
  return winner;
}

// Bound by its instructions (comparisons and logic run at half the rate of additions): 32,768 tokens,
// top-8 of 256 sigmoids with a bias in 4 of 8 groups 27 us, of which 13 are loading, packing and
// sorting, 0.4 each round of the choice, 5 the groups; the bytes alone would take 5.
template <class T, int EPL, int L, bool SOFTMAX>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(const __grid_constant__ RouteArgs A) {
  after_the_last();
  constexpr uint32_t kPlaces = EPL - 1, kLow = (EPL > L ? EPL : L) - 1;  // (kLow: as in pop_sorted)
  // what comparing keys without their last bits may change, relative to a key
  constexpr float kCut = float(EPL > L ? EPL : L) * 0x1p-23f;
  constexpr int kTokens = 32 / L;                // of a warp
  const int lane = threadIdx.x & 31, q = lane & (L - 1);
  const bool grouped = A.top_groups < A.groups;
  const bool scored = A.bias || grouped;                // keys are scores, not logits
  const bool whole = SOFTMAX && (scored || !A.renorm);  // the softmax's sum is needed
  const bool check = scored || sizeof(T) == 4;          // keys are not exact
  const int64_t t0 = (int64_t(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5)) * kTokens;
  if (t0 >= A.tokens) return;
  const int64_t t = t0 + lane / L;
  const bool there = t < A.tokens;
  const T* row = static_cast<const T*>(A.logits) + (there ? t : t0) * A.ld;
  uint32_t u[EPL];
  float most = -INFINITY, sum = 1.f, tol = 0.f;
  {
    float z[EPL];
    load_logits<T, EPL>(row, A.experts, A.epl, A.vec, q, z);
    if (whole) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) most = fmaxf(most, z[i]);
      most = max_of<L>(most);
      sum = 0.f;
#pragma unroll
      for (int i = 0; i < EPL; ++i) sum += share(z[i], most);
      sum = sum_of<L>(sum);  // 0 for a token without experts
    }
    if (scored) {
      const float inv = SOFTMAX ? 1.f / sum : 1.f;
      tol = SOFTMAX ? kSoftmaxError<EPL> * inv : kSigmoidError;  // (inv: the largest score)
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        z[i] = z[i] > -INFINITY ? (SOFTMAX ? share(z[i], most) * inv : sigmoid(z[i])) : -INFINITY;
      if (A.bias) {
        float b[EPL];
        load_logits<float, EPL>(A.bias, A.experts, A.epl, A.vec_bias, q, b);
#pragma unroll
        for (int i = 0; i < EPL; ++i) z[i] += b[i];  // (-inf for a NaN)
      }
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const uint32_t b = __float_as_uint(z[i] + 0.f);  // as ordered(), with the place
      u[i] = z[i] > -INFINITY ? ((b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u)) & ~kPlaces) | (kPlaces - i) : 0u;
    }
  }
  auto is_near = [&](float a, float b) {
    return !(a - b > 2.f * tol + fmaxf(fabsf(a), fabsf(b)) * (kCut + 0x1p-22f) + 0x1p-140f);
  };
  // The softmax's sum in 64 bits for the tokens that ask for it, each by the whole warp; and expert e's key,
  // which needs it.
  double sum64 = 1;
  auto sum_in_64 = [&](bool asked) {
    if (!SOFTMAX || !scored) return;
    for (uint32_t left = __ballot_sync(kAll, asked && there && q == 0); left; left &= left - 1) {
      const int first = __ffs(left) - 1;
      const T* it = static_cast<const T*>(A.logits) + (t0 + first / L) * A.ld;
      const double top = __shfl_sync(kAll, most, first);
      double part = 0;
      for (int e = lane; e < A.experts; e += 32) part += share(double(fmaxf(widen(it[e]), -INFINITY)), top);
      part = sum_of<32>(part);
      if (lane / L == first / L) sum64 = part;
    }
  };
  auto key_in_64 = [&](int e) {
    const double z = widen(row[e]), s = !scored ? z : SOFTMAX ? share(z, double(most)) / sum64 : sigmoid(z);
    return ordered(s + (A.bias ? double(A.bias[e]) : 0.0));
  };
  bool exactly = false;  // the token is done again
  if (grouped) {
    const int per = A.experts / A.groups, run = per / A.epl;
    const bool runs = per % A.epl == 0 && (run & (run - 1)) == 0;  // a group is `run` lanes, a power of two
    Two<uint32_t> g;
    if (runs) {
      sort_keys(u);
      g = {u[0], EPL > 1 ? u[EPL > 1 ? 1 : 0] : 0u};
      for (int off = 1; off < run; off <<= 1) {
        const uint32_t a = __shfl_xor_sync(kAll, g.a, off), b = __shfl_xor_sync(kAll, g.b, off);
        g.join(a, b);
      }
      g.a = __shfl_sync(kAll, g.a, q * run & (L - 1), L);  // to lane g
      g.b = __shfl_sync(kAll, g.b, q * run & (L - 1), L);
    } else {
      g = two_of_groups<EPL, L>(A.experts, A.groups, A.epl, q, u);
    }
    // A group's score is within err of this sum, whose keys are cut to their places, rounded, and off by tol each.  The
    // sum of two of the lowest keys is -inf: the score is below all binary32 numbers then, and its group there all the same.
    const float ga = value_of(g.a & ~kPlaces), gb = g.b ? value_of(g.b & ~kPlaces) : 0.f, score = ga + gb;
    const float err = 2.f * tol + (fabsf(ga) + fabsf(gb)) * (float(EPL) * 0x1p-23f + 0x1p-22f);
    const bool some = q < A.groups && g.a;
    // scores with their lanes as last bits: of equal ones the first group is the largest
    constexpr uint32_t kLane = L - 1;
    uint32_t mark = some ? (ordered(fmaxf(score, -FLT_MAX)) & ~kLane) | (kLane - q) : 0u, kept = 0;
    for (int r = 0; r < A.top_groups; ++r) {
      const uint32_t m = most_of<L>(mark);
      kept |= m ? 1u << (kLane - (m & kLane)) : 0u;
      mark = mark == m ? 0u : mark;
    }
    // in doubt unless the least that a kept score may be is above the most that another may be (ordered() of -inf and of
    // inf - inf is 0: as low as can be)
    const bool in = kept >> q & 1;
    const uint32_t low = ~most_of<L>(some && in ? ~ordered(score - err) : 0u);
    const uint32_t high = most_of<L>(some && !in ? ordered(fmaxf(score + err, -FLT_MAX)) : 0u);
    const bool near = high && low <= high;
    if (!runs) {
      exactly = near;
    } else if (__any_sync(kAll, near)) {
      // The group's scores by 64-bit keys: of a lane's three largest, unless a fourth may be among them.
      sum_in_64(near);
      Two<uint64_t> t{0, 0};
#pragma unroll
      for (int i = 0; i < (EPL < 3 ? EPL : 3); ++i)
        if (u[i]) t.add(key_in_64(q * A.epl + int(kPlaces - (u[i] & kPlaces))));
      constexpr int kFourth = EPL > 3 ? 3 : 0;
      const bool more = EPL > 3 && u[kFourth] && is_near(value_of(u[EPL > 1 ? 1 : 0] & ~kPlaces), value_of(u[kFourth] & ~kPlaces));
      for (int off = 1; off < run; off <<= 1) {
        const uint64_t a = __shfl_xor_sync(kAll, t.a, off), b = __shfl_xor_sync(kAll, t.b, off);
        t.join(a, b);
      }
      t.a = __shfl_sync(kAll, t.a, q * run & (L - 1), L);
      t.b = __shfl_sync(kAll, t.b, q * run & (L - 1), L);
      const double sum = t.b ? value_of(t.a) + value_of(t.b) : value_of(t.a);
      uint64_t last64, next64;
      const uint32_t kept64 = keep_groups<L>(A.top_groups, q < A.groups ? ordered(sum) : uint64_t(0), q, &last64, &next64);
      const uint32_t doubt = lanes_of<L>(more);
      exactly = near && doubt;
      if (near) kept = kept64;
    }
    if (runs) {
      const bool out = !(kept >> (q / run) & 1);
#pragma unroll
      for (int i = 0; i < EPL; ++i) u[i] = out ? 0u : u[i];
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (u[i] && !(kept >> ((q * A.epl + i) / per) & 1)) u[i] = 0;
      sort_keys(u);
    }
  } else {
    sort_keys(u);
  }
  uint32_t key = 0;  // lane j: slot j's; slot topk is the first that is left out
  int owner = 0;
  const int slots = A.topk + check;
  for (int r = 0; r < slots; ++r) {
    uint32_t k;
    const int from = pop_sorted<EPL, L>(u, q, &k);
    if (q == r) {
      key = k;
      owner = from;
    }
  }
  int mine = key ? owner * A.epl + int(kPlaces - (key & kPlaces)) : -1;
  if (check) {
    // Keys that are near the one before them; where that holds for the first that is left out,
    // what follows it is taken too (lanes topk + 1, ..), as far as it is near the last chosen.  They are compared by what
    // orders them, without the bits that a lane may stand for (kLow): a key is at most that much above it, also those
    // that are still in their lanes, which may be larger than the one that was found before them.
    const float k = value_of(key & ~kLow), before = __shfl_up_sync(kAll, k, 1, L);
    bool by = q > 0 && key && is_near(before, k);
    if (__any_sync(kAll, by)) {
      const uint32_t close = lanes_of<L>(by);  // (by all lanes: the rest is a token's own)
      bool more = !exactly && (close >> A.topk & 1);
      const float least = __shfl_sync(kAll, k, A.topk - 1, L);
      for (int r = A.topk + 1; __any_sync(kAll, more); ++r) {
        uint32_t next;
        const int from = pop_sorted<EPL, L>(u, q, &next);
        more = more && next && is_near(least, value_of(next & ~kLow));
        if (more && q == r) {
          key = next;
          mine = from * A.epl + int(kPlaces - (next & kPlaces));
          by = true;
        }
        exactly = exactly || (more && r >= L);  // more of them than lanes
        more = more && r < L;
      }
      // near ones that are not equals: their order by 64-bit keys
      const int prev = __shfl_up_sync(kAll, mine, 1, L);
      const uint32_t doubt = lanes_of<L>(by && (row[prev] != row[mine] || (A.bias && A.bias[prev] != A.bias[mine])));
      if (__any_sync(kAll, doubt)) {
        sum_in_64(doubt);
        const uint64_t key64 = mine >= 0 ? key_in_64(mine) : 0;
        int place = 0;
        for (int r = 0; r < L; ++r) {
          const uint64_t other = __shfl_sync(kAll, key64, r, L);
          const int id = __shfl_sync(kAll, mine, r, L);
          place += other > key64 || (other == key64 && id < mine && id >= 0);
        }
        if (mine < 0) place = L;
        int sorted = -1;
        for (int r = 0; r < L; ++r) {
          const int id = __shfl_sync(kAll, mine, r, L);
          if (__shfl_sync(kAll, place, r, L) == q) sorted = id;
        }
        if (doubt) mine = sorted;
      }
    }
    for (uint32_t left = __ballot_sync(kAll, exactly && there && q == 0); left; left &= left - 1) {
      const int first = __ffs(left) - 1;
      const T* it = static_cast<const T*>(A.logits) + (t0 + first / L) * A.ld;
      const int id = __shfl_sync(kAll, route_exactly<T, (EPL * L + 31) / 32>(A, it, lane), q);
      if (lane / L == first / L) mine = id;
    }
  }
  if (q >= A.topk) mine = -1;
  const float zc = mine >= 0 ? widen(row[mine]) : -INFINITY;
  float s = 0.f;
  if (A.renorm) {
    const float top = max_of<L>(zc);
    if (mine >= 0) {
      if (SOFTMAX) {
        s = share(zc, top);
      } else {  // sigmoids, all divided by exp of the largest logit where that is below 0
        const float m = fminf(top, 0.f);
        s = __fdividef(1.f, expf(m) + expf(m - zc));
      }
    }
    const float total = sum_of<L>(s);
    s = mine >= 0 ? __fdividef(s, total) : 0.f;
  } else if (mine >= 0) {
    s = SOFTMAX ? __fdividef(share(zc, most), sum) : __fdividef(1.f, 1.f + expf(-zc));
  }
  if (there && q < A.topk) {
    A.ids[t * A.topk + q] = mine;
    A.gate[t * A.topk + q] = s * A.scale;
  }
}

// ------------------------------------------------------------------ gradient
struct RouteGradArgs {
  const void* logits;
  const int32_t* ids;
  const float* dgate;
  void* out;
  int64_t ld, ldd;
  int tokens, experts, topk, renorm;
  float scale;
};

// A slot of a token: its expert, -1 for one that adds nothing; the gradient for its score times
// scale, and its logit (-inf with -1).
struct Slot {
  int id;
  float dg, z;
};

template <class T>
__device__ __forceinline__ Slot slot_of(const RouteGradArgs& A, const T* row, int64_t t, int q, bool there) {
  Slot s;
  s.id = there && q < A.topk ? A.ids[t * A.topk + q] : -1;
  if (s.id >= A.experts || s.id < 0) s.id = -1;
  s.z = s.id >= 0 ? fmaxf(widen(row[s.id]), -INFINITY) : -INFINITY;
  s.dg = s.z > -INFINITY ? A.dgate[t * A.topk + q] * A.scale : 0.f;
  return s;
}

// An expert that several slots name gets their sum, at the first of them: *same has the
// lanes of a lane's expert.
template <int L>
__device__ __forceinline__ float sum_same(int id, int topk, float v, uint32_t* same) {
  const int lane = threadIdx.x & 31;
  *same = __match_any_sync(kAll, id < 0 ? -1 : id + (lane / L) * kMaxExperts);
  if (__any_sync(kAll, id >= 0 && (*same & (*same - 1)))) {
    float sum = 0.f;
    for (int j = 0; j < topk; ++j) {
      const float w = __shfl_sync(kAll, v, j, L);
      if (*same >> (lane / L * L + j) & 1) sum += w;
    }
    v = sum;
  }
  return v;
}

// Every gate but those of a softmax that is not renormalised depends on the chosen logits alone:
// they are all that is read, and the row is zeros but for them.  L lanes take a token.
// Bound by its stores: 32,768 x 256 binary32 11.8 us.  S: elements of a store.
template <class T, int S, int L, bool SOFTMAX>
__global__ void __launch_bounds__(kRouteWarps * 32) route_grad_kernel(const __grid_constant__ RouteGradArgs A) {
  after_the_last();
  const int lane = threadIdx.x & 31, q = lane & (L - 1);
  const int64_t t = (int64_t(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5)) * (32 / L) + lane / L;
  const bool there = t < A.tokens;
  const T* row = static_cast<const T*>(A.logits) + (there ? t : 0) * A.ld;
  T* out = static_cast<T*>(A.out) + (there ? t : 0) * A.ldd;
  const Slot c = slot_of(A, row, t, q, there);
  const bool on = c.z > -INFINITY;
  float v = 0.f;
  if (A.renorm) {
    const float top = max_of<L>(c.z), m = fminf(top, 0.f);
    float s = 0.f, slope = 1.f;
    if (on) {
      s = SOFTMAX ? share(c.z, top) : 1.f / (expf(m) + expf(m - c.z));
      if (!SOFTMAX) slope = 1.f / (1.f + expf(c.z));  // 1 - sigmoid
    }
    const float total = sum_of<L>(s), p = on ? s / total : 0.f;
    // p_j (dg_j - sum p_i dg_i) by differences, which vanish where the dg are equal
    const uint32_t any = lanes_of<L>(on);
    const float first = __shfl_sync(kAll, c.dg, any ? __ffs(any) - 1 : 0, L);
    const float mean = sum_of<L>(on ? p * (c.dg - first) : 0.f);
    v = on ? p * slope * ((c.dg - first) - mean) : 0.f;
  } else {  // sigmoid
    const float e = expf(-fabsf(c.z));
    v = on ? c.dg * e / ((1.f + e) * (1.f + e)) : 0.f;
  }
  uint32_t same;
  v = sum_same<L>(c.id, A.topk, v, &same);
  __syncwarp();  // the logits have been read: dlogits may be they
  if (there) {
    Vec<T, S> zero;
#pragma unroll
    for (int e = 0; e < S; ++e) zero.v[e] = narrow<T>(0.f);
#pragma unroll 4
    for (int e = q * S; e < A.experts; e += L * S) *reinterpret_cast<Vec<T, S>*>(out + e) = zero;
  }
  __syncwarp();  // (orders the stores of the lanes)
  if (c.id >= 0 && __ffs(same) - 1 == lane) out[c.id] = narrow<T>(v);
}

// Gates that are a whole softmax's: every logit has a part.  L lanes take a token; lane q has the
// vectors q, q + L, .. of 16 bytes, EPL elements in all, also where they are accessed one by
// one: the sums' order does not depend on the alignment.  32,768 x 256 binary32 17 us, bound by its
// instructions (exponentials, sums over lanes).
template <class T, bool VEC, int EPL, int L>
__global__ void __launch_bounds__(kRouteWarps * 32) route_softmax_grad_kernel(const __grid_constant__ RouteGradArgs A) {
  after_the_last();
  const int lane = threadIdx.x & 31, q = lane & (L - 1);
  constexpr int S = 16 / sizeof(T);
  const int64_t t = (int64_t(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5)) * (32 / L) + lane / L;
  const bool there = t < A.tokens;
  const T* row = static_cast<const T*>(A.logits) + (there ? t : 0) * A.ld;
  T* out = static_cast<T*>(A.out) + (there ? t : 0) * A.ldd;
  const Slot c = slot_of(A, row, t, q, there);
  float z[EPL], most = -INFINITY, sum = 0.f;
#pragma unroll
  for (int i = 0; i < EPL; i += S) {
    const int e0 = i * L + q * S;
    Vec<T, S> v;
    if (VEC && e0 < A.experts) v = *reinterpret_cast<const Vec<T, S>*>(row + e0);
#pragma unroll
    for (int e = 0; e < S; ++e) {
      if (!VEC && e0 + e < A.experts) v.v[e] = row[e0 + e];
      z[i + e] = e0 + e < A.experts ? fmaxf(widen(v.v[e]), -INFINITY) : -INFINITY;
      most = fmaxf(most, z[i + e]);
    }
  }
  most = max_of<L>(most);
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    z[i] = share(z[i], most);
    sum += z[i];
  }
  const float inv = 1.f / sum_of<L>(sum);
  const bool on = c.z > -INFINITY;
  const float s = on ? share(c.z, most) * inv : 0.f;
  const float dot = sum_of<L>(on ? s * c.dg : 0.f);
  uint32_t same;
  const float v = sum_same<L>(c.id, A.topk, on ? s * c.dg : 0.f, &same);
  __syncwarp();  // the logits have been read: dlogits may be they
#pragma unroll
  for (int i = 0; i < EPL; i += S) {
    const int e0 = i * L + q * S;
    if (!there || e0 >= A.experts) continue;
    Vec<T, S> o;
#pragma unroll
    for (int e = 0; e < S; ++e) o.v[e] = narrow<T>(z[i + e] > 0.f ? -(z[i + e] * inv) * dot : 0.f);
    if (VEC) *reinterpret_cast<Vec<T, S>*>(out + e0) = o;
#pragma unroll
    for (int e = 0; e < S; ++e)
      if (!VEC && e0 + e < A.experts) out[e0 + e] = o.v[e];
  }
  __syncwarp();  // (orders the stores of the lanes)
  if (c.id >= 0 && __ffs(same) - 1 == lane) out[c.id] = narrow<T>(on ? v - s * dot : 0.f);
}

// ------------------------------------------------------------------ host side
// Elements of an access to a row: a power of two that divides a lane's share and the row.
int access_of(const void* p, size_t ld, int experts, int epl, size_t elem) {
  int v = int(16 / elem);
  while (v > 1 && (epl % v || experts % v || !aligned(p, v * elem) || ld % v)) v >>= 1;
  return v;
}

// The lanes that take a token: as few as hold its experts in registers, have one lane for each
// slot and the first that is left out (for scores of bf16 logits, among which many are equal,
// three more), and one for each group.  32,768 tokens, top-8 of 256 in 4 of 8 groups: 27.0 us with 16
// lanes, 30.8 with 32; top-6 of 64 in bf16: 5.9 us with 8, 10.1 with 32.  Where there are not enough
// tokens to keep the SMs busy a warp each has less to do one after the other: 1024 tokens 6.8 us
// with 32 lanes, 8.5 with 16; 2.5 and 2.9.  The sides meet near 3000 tokens at 64 experts and
// between 8192 and 32,768 at 256.
template <class T, bool SOFTMAX>
void (*route_pick(int tokens, int experts, int topk, int groups, bool scored, int* lanes))(RouteArgs) {
  const int slots = topk + (scored && sizeof(T) == 2 ? 4 : 1);
  const int need = tokens <= kSms * (experts <= 128 ? 16 : 64) ? 32 : slots > groups ? slots : groups;
  if (experts <= 32 && need <= 8) {
    *lanes = 8;
    return route_kernel<T, 4, 8, SOFTMAX>;
  }
  if (experts <= 64 && need <= 8) {
    *lanes = 8;
    return route_kernel<T, 8, 8, SOFTMAX>;
  }
  if (experts <= 64 && need <= 16) {
    *lanes = 16;
    return route_kernel<T, 4, 16, SOFTMAX>;
  }
  if (experts <= 128 && need <= 16) {
    *lanes = 16;
    return route_kernel<T, 8, 16, SOFTMAX>;
  }
  if (experts <= 256 && need <= 16) {
    *lanes = 16;
    return route_kernel<T, 16, 16, SOFTMAX>;
  }
  *lanes = 32;
  return experts <= 32    ? route_kernel<T, 1, 32, SOFTMAX>
         : experts <= 64  ? route_kernel<T, 2, 32, SOFTMAX>
         : experts <= 128 ? route_kernel<T, 4, 32, SOFTMAX>
         : experts <= 256 ? route_kernel<T, 8, 32, SOFTMAX>
         : experts <= 512 ? route_kernel<T, 16, 32, SOFTMAX>
                          : route_kernel<T, 32, 32, SOFTMAX>;
}

template <class T, int S, bool SOFTMAX>
void (*route_grad_lanes(int topk, int* lanes))(RouteGradArgs) {
  if (topk <= 8) {
    *lanes = 8;
    return route_grad_kernel<T, S, 8, SOFTMAX>;
  }
  if (topk <= 16) {
    *lanes = 16;
    return route_grad_kernel<T, S, 16, SOFTMAX>;
  }
  {
    *lanes = 32;
    return route_grad_kernel<T, S, 32, SOFTMAX>;
  }
}

template <class T, int S>
void (*route_grad_pick(const RouteGradArgs& A, bool softmax, int* lanes))(RouteGradArgs) {
  if (!softmax) return route_grad_lanes<T, S, false>(A.topk, lanes);
  if (A.renorm) return route_grad_lanes<T, S, true>(A.topk, lanes);
  const int e = A.experts;
  constexpr bool vec = S > 1;
  // as few lanes as hold the experts in 8 elements each, and a slot: 32,768 tokens, 64 experts, bf16 5.3 us with
  // 8 lanes, 13.8 with 32; 256 experts, bf16 13.7 us with 16, 15.4 with 32, binary32 19.1 and 17.3
  if (e <= 64 && A.topk <= 8) {
    *lanes = 8;
    return route_softmax_grad_kernel<T, vec, 8, 8>;
  }
  if (e <= 128 && A.topk <= 16) {
    *lanes = 16;
    return route_softmax_grad_kernel<T, vec, 8, 16>;
  }
  if (sizeof(T) == 2 && e <= 256 && A.topk <= 16) {
    *lanes = 16;
    return route_softmax_grad_kernel<T, vec, 16, 16>;
  }
  *lanes = 32;
  return e <= 256   ? route_softmax_grad_kernel<T, vec, 8, 32>
         : e <= 512 ? route_softmax_grad_kernel<T, vec, 16, 32>
                    : route_softmax_grad_kernel<T, vec, 32, 32>;
}

template <class T>
void (*route_grad_pick(const RouteGradArgs& A, bool softmax, bool vec, int* lanes))(RouteGradArgs) {
  return vec ? route_grad_pick<T, 16 / sizeof(T)>(A, softmax, lanes) : route_grad_pick<T, 1>(A, softmax, lanes);
}

// CTAs for `tokens` tokens of `lanes` lanes each.
dim3 route_grid(int tokens, int lanes) { return dim3(unsigned((int64_t(tokens) * lanes + kRouteWarps * 32 - 1) / (kRouteWarps * 32))); }

const char* bad_route(int tokens, int experts, int topk, const void* logits, int dtype, size_t ld, int score, const float* scale) {
  if (tokens < 0 || experts < 1 || experts > kMaxExperts) return "tokens or experts out of range";
  if (topk < 1 || topk > experts || topk > HOC_ROUTE_MAX_TOPK) return "topk out of range";
  if (!row_dtype(dtype)) return "dtype must be HOC_FLOAT32 or HOC_BFLOAT16";
  if (score != HOC_SCORE_SOFTMAX && score != HOC_SCORE_SIGMOID) return "score must be one of hocScore_t";
  if (!scale || !(*scale - *scale == 0.f)) return "scale must be given, and finite";
  return bad_rows(logits, ld, tokens, experts, bytes_of(dtype), tokens == 0);
}

}  // namespace

cudaError_t route_preload() {
  cudaError_t err = cudaSuccess;
  auto load = [&](const void* f) {
    cudaFuncAttributes a;
    if (err == cudaSuccess) err = cudaFuncGetAttributes(&a, f);
  };
  int lanes;
  for (int experts = 32; experts <= kMaxExperts; experts *= 2)
    for (int topk : {1, 12, 31}) {
      for (int groups : {1, 16})
        for (int tokens : {1, 1 << 30}) {
          load(reinterpret_cast<const void*>(route_pick<float, false>(tokens, experts, topk, groups, false, &lanes)));
          load(reinterpret_cast<const void*>(route_pick<float, true>(tokens, experts, topk, groups, false, &lanes)));
          load(reinterpret_cast<const void*>(route_pick<__nv_bfloat16, false>(tokens, experts, topk, groups, false, &lanes)));
          load(reinterpret_cast<const void*>(route_pick<__nv_bfloat16, true>(tokens, experts, topk, groups, false, &lanes)));
        }
      RouteGradArgs A{};
      A.experts = experts;
      A.topk = topk;
      for (int renorm = 0; renorm < 2; ++renorm)
        for (int softmax = 0; softmax < 2; ++softmax)
          for (int vec = 0; vec < 2; ++vec) {
            A.renorm = renorm;
            load(reinterpret_cast<const void*>(route_grad_pick<float>(A, softmax, vec, &lanes)));
            load(reinterpret_cast<const void*>(route_grad_pick<__nv_bfloat16>(A, softmax, vec, &lanes)));
          }
    }
  return err;
}

}  // namespace hoc

using namespace hoc;
using namespace hoc::block;

extern "C" hocResult_t hoc_ep_route(int tokens, int experts, int topk, const void* logits, hocDataType_t dtype, size_t ldl,
                                    int score, const float* bias, int groups, int top_groups, int renormalise, const float* scale,
                                    int32_t* ids, float* gate, void* stream) {
  const char* who = "hoc_ep_route";
  const char* bad = bad_route(tokens, experts, topk, logits, dtype, ldl, score, scale);
  if (!bad && (groups < 1 || groups > kMaxGroups || experts % groups)) bad = "groups must divide the experts, and be at most 32";
  if (!bad && (top_groups < 1 || top_groups > groups || topk > experts / groups * top_groups))
    bad = "top_groups out of range, or fewer experts in so many groups than topk";
  if (!bad && !aligned(bias, 4)) bad = "bias must be aligned to its elements";
  if (!bad && tokens && (!ids || !gate || !aligned(ids, 4) || !aligned(gate, 4)))
    bad = "ids and gate must be given, aligned to their elements";
  if (bad) return refuse(who, bad);
  if (tokens == 0) return HOC_SUCCESS;
  const bool softmax = score == HOC_SCORE_SOFTMAX, scored = bias || top_groups < groups;
  const size_t b = bytes_of(dtype);
  int lanes;
  const auto kernel = dtype == HOC_FLOAT32
                          ? softmax ? route_pick<float, true>(tokens, experts, topk, groups, scored, &lanes) : route_pick<float, false>(tokens, experts, topk, groups, scored, &lanes)
                          : softmax ? route_pick<__nv_bfloat16, true>(tokens, experts, topk, groups, scored, &lanes)
                                    : route_pick<__nv_bfloat16, false>(tokens, experts, topk, groups, scored, &lanes);
  const int epl = (experts + lanes - 1) / lanes, epl_warp = (experts + 31) / 32;
  const RouteArgs A{logits, bias, ids, gate, int64_t(ldl), tokens, experts, topk, groups, top_groups, softmax, renormalise != 0,
                    epl, access_of(logits, ldl, experts, epl, b), epl_warp, access_of(logits, ldl, experts, epl_warp, b),
                    access_of(bias, 0, experts, epl, 4), *scale};
  return launched(who, launch(kernel, route_grid(tokens, lanes), dim3(kRouteWarps * 32), 0, static_cast<cudaStream_t>(stream), A));
}

extern "C" hocResult_t hoc_ep_route_grad(int tokens, int experts, int topk, const void* logits, hocDataType_t dtype,
                                         size_t ldl, int score, int renormalise, const float* scale, const int32_t* ids,
                                         const float* dgate, void* dlogits, size_t ldd, void* stream) {
  const char* who = "hoc_ep_route_grad";
  const char* bad = bad_route(tokens, experts, topk, logits, dtype, ldl, score, scale);
  if (!bad) bad = bad_rows(dlogits, ldd, tokens, experts, bytes_of(dtype), tokens == 0);
  if (!bad && tokens && (!ids || !dgate || !aligned(ids, 4) || !aligned(dgate, 4)))
    bad = "ids and dgate must be given, aligned to their elements";
  if (bad) return refuse(who, bad);
  if (tokens == 0) return HOC_SUCCESS;
  const size_t b = bytes_of(dtype);
  const bool softmax = score == HOC_SCORE_SOFTMAX;
  const bool vec = experts * b % 16 == 0 && vector_rows(dlogits, ldd, b) && vector_rows(logits, ldl, b);
  const RouteGradArgs A{logits, ids, dgate, dlogits, int64_t(ldl), int64_t(ldd), tokens, experts, topk, renormalise != 0, *scale};
  int lanes;
  const auto kernel = dtype == HOC_FLOAT32 ? route_grad_pick<float>(A, softmax, vec, &lanes)
                                           : route_grad_pick<__nv_bfloat16>(A, softmax, vec, &lanes);
  return launched(who, launch(kernel, route_grid(tokens, lanes), dim3(kRouteWarps * 32), 0, static_cast<cudaStream_t>(stream), A));
}
