// Routing of tokens to experts, and its gradient (hoc_block.h).
//
// A warp takes a token.  Lane l holds the logits of the experts l * epl .. (l + 1) *
// epl - 1, so that the lowest of several lanes with the same key has the lowest expert,
// and a group of neighbouring experts is a run of lanes.  The topk largest keys are found
// one after the other: a maximum over each lane's registers, one over the warp
// (redux.sync), and the lane that had it looks for its next.
//
// Which of two near keys is larger is decided as 64-bit arithmetic decides it.  Without a
// bias and groups the keys are the logits themselves, and there is nothing to round.  Else
// keys are binary32 with a bound on their error, and a token for which two keys that are
// compared lie within it (0.1 to 0.5 % of them, for normal logits) is done again in
// binary64.  Keys with the same logit and the same bias are equal in any arithmetic, so
// that logits of few bits do not send their tokens there.
#include <type_traits>

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
  int tokens, experts, topk, epl, groups, top_groups, softmax, renorm;
  int vec;  // elements of an access to the logits
  float scale;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(kAll, v, off);
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(kAll, v, off);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int off = 16; off; off >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, off));
  return v;
}

// Keys as unsigned numbers in the same order; 0: not to be chosen (-inf and NaN).
// Both zeros are one.
__device__ __forceinline__ uint32_t ordered(float k) {
  const uint32_t b = __float_as_uint(k + 0.f);
  return k > -INFINITY ? (b >> 31 ? ~b : b | 0x80000000u) : 0u;
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

template <class K>
struct Bits;
template <>
struct Bits<float> {
  using type = uint32_t;
};
template <>
struct Bits<double> {
  using type = uint64_t;
};

// Calls by(elements of an access), known when compiling; vec divides a lane's share.
template <class T, int EPL, class By>
__device__ __forceinline__ void with_access(int vec, By by) {
  if (EPL >= 8 && sizeof(T) == 2 && vec == 8) by(std::integral_constant<int, EPL >= 8 && sizeof(T) == 2 ? 8 : 1>{});
  else if (EPL >= 4 && vec == 4) by(std::integral_constant<int, EPL >= 4 ? 4 : 1>{});
  else if (EPL >= 2 && vec == 2) by(std::integral_constant<int, EPL >= 2 ? 2 : 1>{});
  else by(std::integral_constant<int, 1>{});
}

// A lane's logits; -inf for experts there are none of, and for NaN.
template <class T, int EPL>
__device__ __forceinline__ void load_logits(const T* row, int experts, int epl, int vec, int lane, float (&z)[EPL]) {
  const int e0 = lane * epl;
  auto by = [&](auto step) {
    constexpr int S = decltype(step)::value;
#pragma unroll
    for (int i = 0; i < EPL; i += S) {
      Vec<T, S> v;
      const bool in = i < epl && e0 + i < experts;
      if (in) v = *reinterpret_cast<const Vec<T, S>*>(row + e0 + i);
#pragma unroll
      for (int e = 0; e < S; ++e) {
        const float f = in ? widen(v.v[e]) : -INFINITY;
        z[i + e] = f == f ? f : -INFINITY;
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

__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.f, 1.f + expf(-z)); }
__device__ __forceinline__ double sigmoid(double z) { return 1.0 / (1.0 + exp(-z)); }

// Bounds on the error of a binary32 score relative to the largest score of the token.
// Sigmoid: expf is off by 2 units in the last place at most, 1 + e and the quotient by one
// each; in all below 4 * 2^-23.  Softmax: z - most is rounded, which changes exp by |z - most| 2^-24
// of itself, and x exp(-x) < 0.4; expf 2 units; up to 36 additions of the sum, the quotient:
// below 64 * 2^-23.
constexpr float kSigmoidError = 0x1p-21f, kSoftmaxError = 0x1p-17f;

// The largest and second largest key of a set (-inf: none).
template <class K>
struct Two {
  K a, b;
  __device__ __forceinline__ void add(K v) {
    b = v > a ? a : v > b ? v : b;
    a = v > a ? v : a;
  }
  __device__ __forceinline__ void join(K a2, K b2) {
    b = a2 > a ? (a > b2 ? a : b2) : (a2 > b ? a2 : b);
    a = a2 > a ? a2 : a;
  }
};

// Which groups are kept (a bit each).  near: whether the least kept and the best left out
// lie within `tol` and what the sums' own rounding adds.
template <class K, int EPL>
__device__ __forceinline__ uint32_t keep_groups(const RouteArgs& A, const typename Bits<K>::type (&u)[EPL], int lane,
                                                K tol, bool* near) {
  const int per = A.experts / A.groups, run = per / A.epl;
  K score = -K(INFINITY), size = 0;
  if (per % A.epl == 0 && (run & (run - 1)) == 0) {  // a group is `run` lanes, a power of two
    Two<K> t{-K(INFINITY), -K(INFINITY)};
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (i < A.epl) t.add(value_of(u[i]));
    for (int off = 1; off < run; off <<= 1) {
      const K a = __shfl_xor_sync(kAll, t.a, off), b = __shfl_xor_sync(kAll, t.b, off);
      t.join(a, b);
    }
    const int from = lane * run & 31;
    t.a = __shfl_sync(kAll, t.a, from);
    t.b = __shfl_sync(kAll, t.b, from);
    if (lane < A.groups) {
      score = t.b == -K(INFINITY) ? t.a : t.a + t.b;
      size = t.b == -K(INFINITY) ? K(0) : fabs(t.a) + fabs(t.b);
    }
  } else {
    for (int g = 0; g < A.groups; ++g) {
      Two<K> t{-K(INFINITY), -K(INFINITY)};
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = lane * A.epl + i;
        if (i < A.epl && e >= g * per && e < (g + 1) * per) t.add(value_of(u[i]));
      }
      for (int off = 1; off < 32; off <<= 1) {
        const K a = __shfl_xor_sync(kAll, t.a, off), b = __shfl_xor_sync(kAll, t.b, off);
        t.join(a, b);
      }
      if (lane == g) {
        score = t.b == -K(INFINITY) ? t.a : t.a + t.b;
        size = t.b == -K(INFINITY) ? K(0) : fabs(t.a) + fabs(t.b);
      }
    }
  }
  typename Bits<K>::type mine = ordered(score), last = 0;
  uint32_t kept = 0;
  for (int r = 0; r < A.top_groups; ++r) {
    const auto most = warp_most(mine);
    if (most == 0) return kept;
    last = most;
    const int winner = __ffs(__ballot_sync(kAll, mine == most)) - 1;
    kept |= 1u << winner;
    if (lane == winner) mine = 0;
  }
  const auto next = warp_most(mine);
  if (near && next) {
    const float most = warp_max(float(size));  // (finite: a sum of infinite keys has no near neighbour)
    *near = !(value_of(last) - value_of(next) > K(4) * tol + K(most) * K(0x1p-21f));
  }
  return kept;
}

// Takes the largest key of the warp out of u.  Returns its expert, and the key in *most; -1
// where there is none left.
template <class U, int EPL>
__device__ __forceinline__ int pop(U (&u)[EPL], U& best, int epl, int lane, U* most) {
  const U m = warp_most(best);
  *most = m;
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

// The token once more in binary64: lane j's slot j.
template <class T, int EPL>
__device__ __noinline__ int route_exactly(const RouteArgs& A, const T* row, int lane) {
  float z[EPL];
  load_logits<T, EPL>(row, A.experts, A.epl, A.vec, lane, z);
  double most = -INFINITY, sum = 0;
  if (A.softmax) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) most = z[i] > most ? double(z[i]) : most;
    most = warp_max(float(most));
#pragma unroll
    for (int i = 0; i < EPL; ++i) sum += share(double(z[i]), most);
    sum = warp_sum(sum);
  }
  uint64_t u[EPL], best = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane * A.epl + i;
    const bool in = i < A.epl && e < A.experts;
    const double s = A.softmax ? share(double(z[i]), most) / sum : sigmoid(double(z[i]));
    u[i] = in && z[i] > -INFINITY ? ordered(s + (A.bias ? double(A.bias[e]) : 0.0)) : 0;
  }
  if (A.top_groups < A.groups) {
    const uint32_t kept = keep_groups<double, EPL>(A, u, lane, 0.0, nullptr);
    const int per = A.experts / A.groups;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (i < A.epl && !(kept >> (lane * A.epl + i < A.experts ? (lane * A.epl + i) / per : 0) & 1)) u[i] = 0;
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) best = u[i] > best ? u[i] : best;
  int mine = -1;
  for (int r = 0; r < A.topk; ++r) {
    uint64_t key;
    const int id = pop(u, best, A.epl, lane, &key);
    if (id < 0) break;
    if (lane == r) mine = id;
  }
  return mine;
}

template <class T, int EPL>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(const __grid_constant__ RouteArgs A) {
  after_the_last();
  const int lane = threadIdx.x & 31;
  const bool scored = A.bias || A.top_groups < A.groups;  // keys are scores, not logits
  const bool whole = A.softmax && (scored || !A.renorm);  // the softmax's sum is needed
  float bias[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane * A.epl + i;
    bias[i] = A.bias && i < A.epl && e < A.experts ? A.bias[e] : 0.f;
  }
  for (int64_t t = int64_t(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5); t < A.tokens; t += int64_t(gridDim.x) * kRouteWarps) {
    const T* row = static_cast<const T*>(A.logits) + t * A.ld;
    float z[EPL];
    load_logits<T, EPL>(row, A.experts, A.epl, A.vec, lane, z);
    float most = -INFINITY, sum = 1.f;
    if (whole) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) most = fmaxf(most, z[i]);
      most = warp_max(most);
      sum = 0.f;
#pragma unroll
      for (int i = 0; i < EPL; ++i) sum += share(z[i], most);
      sum = warp_sum(sum);  // 0 for a token without experts
    }
    uint32_t u[EPL], best = 0;
    float tol = 0.f;
    bool near = false;
    if (!scored) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) u[i] = ordered(z[i]);
    } else {
      const float inv = A.softmax ? 1.f / sum : 1.f;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const float s = A.softmax ? share(z[i], most) * inv : sigmoid(z[i]);
        u[i] = z[i] > -INFINITY ? ordered(s + bias[i]) : 0u;
      }
      tol = A.softmax ? kSoftmaxError * inv : kSigmoidError;  // (inv: the largest score)
      if (A.top_groups < A.groups) {
        const uint32_t kept = keep_groups<float, EPL>(A, u, lane, tol, &near);
        const int per = A.experts / A.groups;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (i < A.epl && !(kept >> (lane * A.epl + i < A.experts ? (lane * A.epl + i) / per : 0) & 1)) u[i] = 0;
      }
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) best = u[i] > best ? u[i] : best;
    int mine = -1, last = -1;
    float key = -INFINITY;
    for (int r = 0; !near && r < A.topk; ++r) {
      uint32_t m;
      const int id = pop(u, best, A.epl, lane, &m);
      if (id < 0) break;
      const float k = value_of(m);
      if (lane == r) mine = id;
      if (scored && r > 0 && !(key - k > 2.f * tol + fmaxf(fabsf(key), fabsf(k)) * 0x1p-22f))
        near = row[last] != row[id] || (A.bias && A.bias[last] != A.bias[id]);
      last = id;
      key = k;
    }
    // and the first that is left out, of those that are not the last one's equals
    while (scored && !near && __shfl_sync(kAll, mine, A.topk - 1) >= 0) {
      uint32_t m;
      const int id = pop(u, best, A.epl, lane, &m);
      if (id < 0) break;
      const float k = value_of(m);
      if (key - k > 2.f * tol + fmaxf(fabsf(key), fabsf(k)) * 0x1p-22f) break;
      near = row[last] != row[id] || (A.bias && A.bias[last] != A.bias[id]);
    }
    if (near) mine = route_exactly<T, EPL>(A, row, lane);
    const float zc = mine >= 0 ? widen(row[mine]) : -INFINITY;
    float s = 0.f;
    if (A.renorm) {
      const float top = warp_max(zc);
      if (mine >= 0) {
        if (A.softmax) {
          s = share(zc, top);
        } else {  // sigmoids, all divided by exp of the largest logit where that is below 0
          const float m = fminf(top, 0.f);
          s = 1.f / (expf(m) + expf(m - zc));
        }
      }
      const float total = warp_sum(s);
      s = mine >= 0 ? s / total : 0.f;
    } else if (mine >= 0) {
      s = A.softmax ? share(zc, most) / sum : 1.f / (1.f + expf(-zc));
    }
    if (lane < A.topk) {
      A.ids[t * A.topk + lane] = mine;
      A.gate[t * A.topk + lane] = s * A.scale;
    }
  }
}

// ------------------------------------------------------------------ gradient
struct RouteGradArgs {
  const void* logits;
  const int32_t* ids;
  const float* dgate;
  void* out;
  int64_t ld, ldd;
  int tokens, experts, topk, epl, softmax, renorm;
  int vec, vec_out;
  float scale;
};

// A warp a token.  Only a softmax whose gates are not renormalised moves every logit: else
// the chosen ones are all that is read, and the row is zeros but for them.
template <class T, int EPL>
__global__ void __launch_bounds__(kRouteWarps * 32) route_grad_kernel(const __grid_constant__ RouteGradArgs A) {
  after_the_last();
  const int lane = threadIdx.x & 31;
  const bool all = A.softmax && !A.renorm;
  for (int64_t t = int64_t(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5); t < A.tokens; t += int64_t(gridDim.x) * kRouteWarps) {
    const T* row = static_cast<const T*>(A.logits) + t * A.ld;
    T* out = static_cast<T*>(A.out) + t * A.ldd;
    int id = lane < A.topk ? A.ids[t * A.topk + lane] : -1;
    if (id >= A.experts) id = -1;
    float dg = id >= 0 ? A.dgate[t * A.topk + lane] * A.scale : 0.f;
    float zc = id >= 0 ? widen(row[id]) : -INFINITY;
    if (zc != zc) zc = -INFINITY;
    if (zc == -INFINITY) dg = 0.f;
    float z[EPL], most = -INFINITY, inv = 0.f, dot = 0.f, v = 0.f;
    if (all) {
      load_logits<T, EPL>(row, A.experts, A.epl, A.vec, lane, z);
#pragma unroll
      for (int i = 0; i < EPL; ++i) most = fmaxf(most, z[i]);
      most = warp_max(most);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < EPL; ++i) sum += share(z[i], most);
      inv = 1.f / warp_sum(sum);
      const float s = share(zc, most) * inv;
      dot = warp_sum(zc > -INFINITY ? s * dg : 0.f);
      v = zc > -INFINITY ? s * dg : 0.f;  // and - s dot, once an expert
    } else if (A.renorm) {
      const float top = warp_max(zc), m = fminf(top, 0.f);
      float s = 0.f, slope = 1.f;
      if (zc > -INFINITY) {
        s = A.softmax ? share(zc, top) : 1.f / (expf(m) + expf(m - zc));
        if (!A.softmax) slope = 1.f / (1.f + expf(zc));  // 1 - sigmoid
      }
      const float total = warp_sum(s), p = zc > -INFINITY ? s / total : 0.f;
      // p_j (dg_j - sum p_i dg_i) as differences, which cancel exactly where the dg are equal
      float mean = 0.f;
      const float first = __shfl_sync(kAll, dg, __ffs(__ballot_sync(kAll, zc > -INFINITY) | 0x80000000u) - 1);
      mean = warp_sum(zc > -INFINITY ? p * (dg - first) : 0.f);
      v = zc > -INFINITY ? p * slope * ((dg - first) - mean) : 0.f;
    } else {
      const float e = expf(-fabsf(zc));
      v = zc > -INFINITY ? dg * e / ((1.f + e) * (1.f + e)) : 0.f;
    }
    // an expert that several slots name gets their sum
    const uint32_t same = __match_any_sync(kAll, id);
    if (__any_sync(kAll, id >= 0 && (same & (same - 1)))) {
      float sum = 0.f;
      for (int j = 0; j < A.topk; ++j) {
        const float w = __shfl_sync(kAll, v, j);
        if (same >> j & 1) sum += w;
      }
      v = sum;
    }
    if (all && zc > -INFINITY) v -= share(zc, most) * inv * dot;
    __syncwarp();  // the logits have been read: dlogits may be they
    auto store = [&](auto step) {
      constexpr int S = decltype(step)::value;
#pragma unroll
      for (int i = 0; i < EPL; i += S) {
        if (i >= A.epl || lane * A.epl + i >= A.experts) continue;
        Vec<T, S> o;
#pragma unroll
        for (int e = 0; e < S; ++e)
          o.v[e] = narrow<T>(all && z[i + e] > -INFINITY ? -share(z[i + e], most) * inv * dot : 0.f);
        *reinterpret_cast<Vec<T, S>*>(out + lane * A.epl + i) = o;
      }
    };
    with_access<T, EPL>(A.vec_out, store);
    __syncwarp();  // (orders the stores of the lanes)
    if (id >= 0 && __ffs(same) - 1 == lane) out[id] = narrow<T>(v);
  }
}

// ------------------------------------------------------------------ host side
// Elements of an access to a row: a power of two that divides a lane's share and the row.
int access_of(const void* p, size_t ld, int experts, int epl, size_t elem) {
  int v = int(16 / elem);
  while (v > 1 && (epl % v || experts % v || !aligned(p, v * elem) || ld % v)) v >>= 1;
  return v;
}

constexpr int kRouteCtas = kSms * 8;
int route_grid(int tokens) {
  const int want = (tokens + kRouteWarps - 1) / kRouteWarps;
  return want < kRouteCtas ? want : kRouteCtas;
}

#define HOC_ROUTE_PICK(KERNEL, T, E)                                                                         \
  ((E) <= 32 ? KERNEL<T, 1> : (E) <= 64 ? KERNEL<T, 2> : (E) <= 128 ? KERNEL<T, 4> : (E) <= 256 ? KERNEL<T, 8> \
                                                       : (E) <= 512 ? KERNEL<T, 16> : KERNEL<T, 32>)

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
  const void* fns[] = {
#define HOC_ROUTE_OF(T, N) \
  reinterpret_cast<const void*>(&route_kernel<T, N>), reinterpret_cast<const void*>(&route_grad_kernel<T, N>)
#define HOC_ROUTE_ALL(T) \
  HOC_ROUTE_OF(T, 1), HOC_ROUTE_OF(T, 2), HOC_ROUTE_OF(T, 4), HOC_ROUTE_OF(T, 8), HOC_ROUTE_OF(T, 16), HOC_ROUTE_OF(T, 32)
      HOC_ROUTE_ALL(float), HOC_ROUTE_ALL(__nv_bfloat16)};
#undef HOC_ROUTE_ALL
#undef HOC_ROUTE_OF
  for (const void* f : fns) {
    cudaFuncAttributes a;
    const cudaError_t e = cudaFuncGetAttributes(&a, f);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
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
  const int epl = (experts + 31) / 32;
  const RouteArgs A{logits, bias, ids, gate, int64_t(ldl), tokens, experts, topk, epl, groups, top_groups,
                    score == HOC_SCORE_SOFTMAX, renormalise != 0, access_of(logits, ldl, experts, epl, bytes_of(dtype)), *scale};
  const dim3 grid(route_grid(tokens)), cta(kRouteWarps * 32);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launched(who, dtype == HOC_FLOAT32 ? launch(HOC_ROUTE_PICK(route_kernel, float, experts), grid, cta, 0, s, A)
                                            : launch(HOC_ROUTE_PICK(route_kernel, __nv_bfloat16, experts), grid, cta, 0, s, A));
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
  const int epl = (experts + 31) / 32;
  const size_t b = bytes_of(dtype);
  const RouteGradArgs A{logits, ids, dgate, dlogits, int64_t(ldl), int64_t(ldd), tokens, experts, topk, epl,
                        score == HOC_SCORE_SOFTMAX, renormalise != 0, access_of(logits, ldl, experts, epl, b),
                        access_of(dlogits, ldd, experts, epl, b), *scale};
  const dim3 grid(route_grid(tokens)), cta(kRouteWarps * 32);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launched(who, dtype == HOC_FLOAT32 ? launch(HOC_ROUTE_PICK(route_grad_kernel, float, experts), grid, cta, 0, s, A)
                                            : launch(HOC_ROUTE_PICK(route_grad_kernel, __nv_bfloat16, experts), grid, cta, 0, s, A));
}
