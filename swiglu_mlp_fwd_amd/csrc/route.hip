// Router: the k best experts of each token's logits and their weights, and
// the gradient of the weights.
//
// Forward: ids_j = the j-th greatest logit (equal ones in order of index,
// -infinity never chosen), weights_j = scale * s_j, or scale * s_j / sum s
// over the chosen, with s = softmax(logits) or sigmoid(logits).  Choosing by
// logit and not by score keeps the choice exact: softmax and sigmoid are
// monotone, but rounded scores can tie where logits differ.
//
// Softmax scores are formed from e^(l - top), top = the greatest chosen
// logit, so the first is 1 and none overflows.  Renormalised sigmoid scores
// are formed as sigma(l) e^-t with t = min(top, 0), which is
//   1 / (1 + e^-l) for l > 0 (then t = 0),   e^(l - t) / (1 + e^l) otherwise:
// the factor cancels in the division, and the greatest is at least 1/2, so
// the sum does not vanish where every sigma(l) underflows.
//
// Backward, with q the weights before `scale` and d = scale * dweights:
//   softmax           p_e (d_e - m) over all e, p = softmax, d_e = 0 if not chosen
//   softmax, renorm   q_j (d_j - m) at the chosen, 0 elsewhere
//   sigmoid           d_j s_j (1 - s_j)
//   sigmoid, renorm   q_j (d_j - m) (1 - s_j),          m = sum_j q_j d_j
// recomputed from the logits, so nothing but ids is kept between the two.
//
// The work is HBM's for many tokens (the logits, and in the backward their
// gradients) and latency for few.  kL lanes (1 to 64, so that a lane holds 8
// or 16 logits) share a token, and a wave takes 64 / kL tokens.  A logit and
// its index make one key, so that a comparison settles ties too (Key below);
// each lane sorts its keys once, and a choice is the maximum of the lanes'
// first keys (on DPP moves for up to 16 lanes), after which its lane moves up
// by one.  32768 x 128, k = 8, bf16 6.9 us, fp32 10.5 (10.5 and 18.9 MB at
// 1.5 and 1.8 TB/s: the sort and the choices bound it, in fp32 their fp64
// keys).  Earlier forms: maxima over all of a lane's logits per choice 10.8 and
// 11.5; one wave per token and shuffles through LDS 38 (fp32).
// Times in this file are a launch's in a graph of 12 inputs in turn, in all
// more than the caches hold; where they hold them it is up to a fifth less.
//
// Chunks of 16 bytes load at any element's address; the one that would pass
// the row's end loads from E - kN instead and skips what its neighbour has.
#include <type_traits>

#include "block.hpp"
#include "common.hpp"
#include "swiglu.h"

namespace swg {

namespace {

constexpr int kThreads = 256;
constexpr float kInf = __builtin_inff();
typedef u32x4 u32x4_any __attribute__((aligned(2)));

// e^-a for a >= 0 to about two ulps; 0 from where it underflows, +inf included.
__device__ __forceinline__ float exp_neg(float a) {
  float p;
  int n;
  exp_neg_split(fminf(a, 1024.0f), p, n);
  return ldexpf(p, n);
}

template <typename T> struct Row;                // elements of a 16-byte chunk
template <> struct Row<float> {
  static constexpr int kN = 4;
  __device__ static float get(const u32x4& w, int i) { return bits_f32(w[i]); }
  __device__ static float one(const float* p) { return *p; }
  __device__ static u32x4 pack(const float* v) {
    return u32x4{f32_bits(v[0]), f32_bits(v[1]), f32_bits(v[2]), f32_bits(v[3])};
  }
};
template <> struct Row<bf16> {
  static constexpr int kN = 8;
  __device__ static float get(const u32x4& w, int i) {
    const uint32_t u = w[i >> 1];
    return bits_f32((i & 1) ? (u & 0xFFFF0000u) : (u << 16));
  }
  __device__ static float one(const bf16* p) { return from_bf16(*p); }
  __device__ static u32x4 pack(const float* v) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = (uint32_t)__builtin_bit_cast(uint16_t, to_bf16(v[2 * i])) |
             ((uint32_t)__builtin_bit_cast(uint16_t, to_bf16(v[2 * i + 1])) << 16);
    return w;
  }
};

// A lane's logits of a row: kC chunks, chunk c * kL + sub of the row.  first[c]
// is the expert of the chunk's first element and skip[c] how many of its
// elements another lane has (all of them past the row's end); those read as
// -infinity.  kTiny: rows shorter than a chunk, all on lane 0.
template <typename T, int kL, int kC, bool kTiny>
struct Logits {
  static constexpr int kN = Row<T>::kN, kV = kC * kN;
  int first[kC], skip[kC];
  float v[kV];
  __device__ __forceinline__ void load(const T* row, int E, int sub) {
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const int c0 = (c * kL + sub) * kN;
      if constexpr (kTiny) {
        first[c] = c0;
        skip[c] = c0 == 0 ? 0 : kN;
#pragma unroll
        for (int i = 0; i < kN; ++i) v[c * kN + i] = c0 + i < E ? Row<T>::one(row + c0 + i) : -kInf;
      } else {
        first[c] = c0 + kN <= E ? c0 : E - kN;
        skip[c] = c0 - first[c] < kN ? c0 - first[c] : kN;
        const u32x4 w = *reinterpret_cast<const u32x4_any*>(row + first[c]);
#pragma unroll
        for (int i = 0; i < kN; ++i) v[c * kN + i] = Row<T>::get(w, i);
      }
    }
    if constexpr (!kTiny) {
#pragma unroll
      for (int c = 0; c < kC; ++c)
        if (skip[c] != 0) {
#pragma unroll
          for (int i = 0; i < kN; ++i)
            if (i < skip[c]) v[c * kN + i] = -kInf;
        }
    }
  }
  __device__ __forceinline__ int expert(int i) const { return first[i / kN] + i % kN; }
  __device__ __forceinline__ void store(T* row, int E, const float (&o)[kV]) const {
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      if (!kTiny && skip[c] == 0) {
        *reinterpret_cast<u32x4_any*>(row + first[c]) = Row<T>::pack(o + c * kN);
      } else if (skip[c] < kN) {
#pragma unroll
        for (int i = 0; i < kN; ++i)
          if (i >= skip[c] && first[c] + i < E) row[first[c] + i] = (T)o[c * kN + i];
      }
    }
  }
};

// Keys order logits, and equal logits by index (the lower one is greater);
// kNone is below all.  NaN counts as -infinity.
//
// bf16: the 16 bits of the logit as an unsigned integer in its order, above
// the complement of the index.
template <typename T> struct Key;
template <> struct Key<bf16> {
  using Type = uint32_t;
  static constexpr Type kNone = 0x007F0000u;     // -infinity of an index past all
  __device__ __forceinline__ static Type make(float l, int expert) {
    uint32_t u = f32_bits(l + 0.0f);             // -0 and 0 are equal
    u = l == l ? u : 0xFF800000u;
    u ^= (u >> 31) ? 0xFFFF0000u : 0x80000000u;
    return u | (uint32_t)(0xFFFF - expert);
  }
  __device__ __forceinline__ static int expert(Type k) { return 0xFFFF - (int)(k & 0xFFFFu); }
  __device__ __forceinline__ static float logit(Type k) {
    const uint32_t u = k & 0xFFFF0000u;
    return bits_f32(u ^ ((u >> 31) ? 0x80000000u : 0xFFFF0000u));
  }
  __device__ __forceinline__ static Type greater(Type a, Type b) { return a > b ? a : b; }
  __device__ __forceinline__ static Type lesser(Type a, Type b) { return a < b ? a : b; }
};
// fp32: the logit in fp64, whose last 29 bits are then free: the index there
// makes a negative value smaller and a positive one, complemented, greater
// the lower it is.  Infinities become +-2^1023 (which round back to them).
// (As 64-bit integers, compared and selected, the sort is slower: 12.4 us.)
template <> struct Key<float> {
  using Type = double;
  static constexpr Type kNone = -0x1.8p1023;
  __device__ __forceinline__ static Type make(float l, int expert) {
    l = l == l ? l + 0.0f : -kInf;
    const double d = l == kInf ? 0x1p1023 : l == -kInf ? -0x1p1023 : (double)l;
    uint64_t u = __builtin_bit_cast(uint64_t, d);
    u |= (uint64_t)((u >> 63) ? expert : 0xFFFF - expert);
    return __builtin_bit_cast(double, u);
  }
  __device__ __forceinline__ static int expert(Type k) {
    const uint64_t u = __builtin_bit_cast(uint64_t, k);
    const int e = (int)(u & 0xFFFFu);
    return (u >> 63) ? e : 0xFFFF - e;
  }
  __device__ __forceinline__ static float logit(Type k) {
    return (float)__builtin_bit_cast(double, __builtin_bit_cast(uint64_t, k) & ~(uint64_t)0xFFFF);
  }
  __device__ __forceinline__ static Type greater(Type a, Type b) { return fmax(a, b); }
  __device__ __forceinline__ static Type lesser(Type a, Type b) { return fmin(a, b); }
};

// Where `up`: v without its first, one place up, kNone at the end.  In bits:
// written as selections, the compiler turns them into indexing.
template <class K, int kV>
__device__ __forceinline__ void move_up(typename K::Type (&v)[kV], bool up) {
  constexpr int kWords = sizeof(v[0]) / 4;
  struct Words { uint32_t w[kWords]; };
  const uint32_t m = up ? ~0u : 0u;
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const auto next = i + 1 < kV ? v[i + 1 < kV ? i + 1 : i] : K::kNone;
    const Words a = __builtin_bit_cast(Words, v[i]), b = __builtin_bit_cast(Words, next);
    Words o;
#pragma unroll
    for (int w = 0; w < kWords; ++w) o.w[w] = (b.w[w] & m) | (a.w[w] & ~m);
    v[i] = __builtin_bit_cast(typename K::Type, o);
  }
}

// Sorts v in descending order (a bitonic network).
template <class K, int kV>
__device__ __forceinline__ void sort_down(typename K::Type (&v)[kV]) {
#pragma unroll
  for (int k = 2; k <= kV; k *= 2)
#pragma unroll
    for (int j = k / 2; j >= 1; j /= 2)
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        const int o = i ^ j;
        if (o <= i) continue;
        const auto hi = K::greater(v[i], v[o]), lo = K::lesser(v[i], v[o]);
        v[i] = (i & k) == 0 ? hi : lo;
        v[o] = (i & k) == 0 ? lo : hi;
      }
}

// Over the kL lanes of a token, the result in each of them.
template <int kL, typename V, typename F>
__device__ __forceinline__ V over_lanes(V v, F f) {
  auto dpp = [](V x, auto ctrl) {
    constexpr int kC = decltype(ctrl)::value;
    if constexpr (sizeof(V) == 8) {
      const u32x2 w = __builtin_bit_cast(u32x2, x);
      return __builtin_bit_cast(V, u32x2{(uint32_t)__builtin_amdgcn_update_dpp(0, (int)w[0], kC, 0xF, 0xF, true),
                                         (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w[1], kC, 0xF, 0xF, true)});
    } else {
      return __builtin_bit_cast(V, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), kC, 0xF, 0xF, true));
    }
  };
  if constexpr (kL >= 2) v = f(v, dpp(v, std::integral_constant<int, 0xB1>{}));    // quad_perm: lane ^ 1
  if constexpr (kL >= 4) v = f(v, dpp(v, std::integral_constant<int, 0x4E>{}));    // quad_perm: lane ^ 2
  if constexpr (kL >= 8) v = f(v, dpp(v, std::integral_constant<int, 0x141>{}));   // row_half_mirror: the other quad of 8
  if constexpr (kL >= 16) v = f(v, dpp(v, std::integral_constant<int, 0x140>{}));   // row_mirror: the other 8 of 16
  if constexpr (kL >= 32) v = f(v, __shfl_xor(v, 16));
  if constexpr (kL >= 64) v = f(v, __shfl_xor(v, 32));
  return v;
}
template <int kL> __device__ __forceinline__ float lanes_sum(float v) {
  return over_lanes<kL>(v, [](float a, float b) { return a + b; });
}
template <int kL> __device__ __forceinline__ float lanes_max(float v) {
  return over_lanes<kL>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int kL> __device__ __forceinline__ int lanes_min(int v) {
  return over_lanes<kL>(v, [](int a, int b) { return a < b ? a : b; });
}

// The chosen logits' scores before division and scale (see above).
template <Score S>
__device__ __forceinline__ float chosen_score(float l, float top, bool renorm) {
  if constexpr (S == Score::kSoftmax) {
    return exp_neg(top - l);
  } else {
    float s, c;
    sigmoid_pair_f32(l, s, c);
    if (!renorm || l > 0.0f) return s;
    return exp_neg(fminf(top, 0.0f) - l) * c;
  }
}

// Entry j of a token's choice is held by lane j % kL, slot j / kL.
// (A choice has no more entries than the lanes have experts, 8 each at least.)
template <int kL> constexpr int kSlots = kL == 1 ? 8 : (SWIGLU_MAX_TOPK + kL - 1) / kL;

template <typename T, Score S, int kL, int kC, bool kTiny>
__global__ __launch_bounds__(kThreads) void route_fwd_kernel(RouteArgs a) {
  constexpr int kV = Logits<T, kL, kC, kTiny>::kV, kS = kSlots<kL>;
  const int sub = threadIdx.x % kL;
  const int64_t token = (int64_t)blockIdx.x * (kThreads / kL) + threadIdx.x / kL;
  const bool live = token < a.T;
  const int64_t t = live ? token : a.T - 1;        // lanes past the end repeat the last token and store nothing
  Logits<T, kL, kC, kTiny> l;
  l.load(static_cast<const T*>(a.logits) + t * a.E, a.E, sub);
  using K = Key<T>;
  typename K::Type key[kV];
  int bad = 0;
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    if (l.v[i] != l.v[i] || (S == Score::kSoftmax && l.v[i] == kInf)) bad = -1;
    key[i] = K::make(l.v[i], l.expert(i));
  }
  bad = lanes_min<kL>(bad);
  sort_down<K, kV>(key);
  typename K::Type chosen[kS], greatest = K::kNone;
#pragma unroll
  for (int s = 0; s < kS; ++s) chosen[s] = K::kNone;
  for (int j = 0; j < a.k; ++j) {
    const auto best = over_lanes<kL>(key[0], [](auto x, auto y) { return K::greater(x, y); });
    if (j == 0) greatest = best;
#pragma unroll
    for (int s = 0; s < kS; ++s)
      if (j == s * kL + sub) chosen[s] = best;
    move_up<K>(key, key[0] == best);               // keys are distinct, but for elements that a lane skips
  }
  const float top = K::logit(greatest);
  float mine[kS];
  int my_id[kS];
#pragma unroll
  for (int s = 0; s < kS; ++s) {
    mine[s] = K::logit(chosen[s]);
    my_id[s] = mine[s] == -kInf ? -1 : K::expert(chosen[s]);
  }
  float w[kS], z = 0.0f;
#pragma unroll
  for (int s = 0; s < kS; ++s) {
    w[s] = my_id[s] >= 0 ? chosen_score<S>(mine[s], top, a.renorm) : 0.0f;
    z += w[s];
  }
  if (a.renorm) {
    z = lanes_sum<kL>(z);
  } else if constexpr (S == Score::kSoftmax) {
    z = 0.0f;
#pragma unroll
    for (int i = 0; i < kV; ++i) z += l.v[i] == -kInf ? 0.0f : exp_neg(top - l.v[i]);
    z = lanes_sum<kL>(z);
  } else {
    z = 1.0f;
  }
#pragma unroll
  for (int s = 0; s < kS; ++s) {
    const int j = s * kL + sub;
    if (!live || j >= a.k) continue;
    float o = my_id[s] >= 0 ? a.scale * (w[s] / z) : 0.0f;
    if (bad != 0) o = __builtin_nanf("");
    a.weights[t * a.k + j] = o;
    a.ids[t * a.k + j] = my_id[s];
  }
}

// The gradient: the chosen logits and their weights again from the logits, a
// sum over the choice, and for a plain softmax one over the row, which every
// form reads: a NaN in it is one in all of its gradients.  32768 x 128, k = 8:
// bf16 10.6 us (18.9 MB, 1.8 TB/s), fp32 14.5 (35.7 MB, 2.5 TB/s), of which 4
// are a latency that 2048 tokens take too.
template <typename T, Score S, int kL, int kC, bool kTiny>
__global__ __launch_bounds__(kThreads) void route_bwd_kernel(RouteArgs a) {
  constexpr int kV = Logits<T, kL, kC, kTiny>::kV, kS = kSlots<kL>;
  const int sub = threadIdx.x % kL;
  const int64_t token = (int64_t)blockIdx.x * (kThreads / kL) + threadIdx.x / kL;
  const bool live = token < a.T;
  const int64_t t = live ? token : a.T - 1;
  const T* row = static_cast<const T*>(a.logits) + t * a.E;
  // Entries of the choice; skipped ones have id -1.
  int id[kS];
  float d[kS], lk[kS];
#pragma unroll
  for (int s = 0; s < kS; ++s) {
    const int j = s * kL + sub;
    id[s] = -1;
    d[s] = 0.0f;
    lk[s] = -kInf;
    if (j < a.k) {
      id[s] = a.ids_in[t * a.k + j];
      if (id[s] < 0 || id[s] >= a.E) id[s] = -1;
      if (id[s] >= 0) lk[s] = Row<T>::one(row + id[s]);
      if (lk[s] == -kInf) id[s] = -1;              // masked: no gradient
      if (id[s] >= 0) d[s] = a.scale * a.dweights[t * a.k + j];
    }
  }
  Logits<T, kL, kC, kTiny> l;
  l.load(row, a.E, sub);
  int bad = 0;
#pragma unroll
  for (int i = 0; i < kV; ++i)
    if (l.v[i] != l.v[i] || (S == Score::kSoftmax && l.v[i] == kInf)) bad = -1;
  bad = lanes_min<kL>(bad);
  const bool dense = S == Score::kSoftmax && !a.renorm;
  float top = -kInf;
  if (dense) {
#pragma unroll
    for (int i = 0; i < kV; ++i) top = fmaxf(top, l.v[i]);
  } else {
#pragma unroll
    for (int s = 0; s < kS; ++s) top = fmaxf(top, id[s] >= 0 ? lk[s] : -kInf);
  }
  top = lanes_max<kL>(top);
  float q[kS], p[kV], z = 0.0f;
#pragma unroll
  for (int s = 0; s < kS; ++s) {
    q[s] = id[s] >= 0 ? chosen_score<S>(lk[s], top, a.renorm) : 0.0f;
    if (!dense) z += q[s];
  }
  if (dense) {
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      p[i] = l.v[i] == -kInf ? 0.0f : exp_neg(top - l.v[i]);
      z += p[i];
    }
  }
  z = dense || a.renorm ? lanes_sum<kL>(z) : 1.0f;
  float m = 0.0f;
#pragma unroll
  for (int s = 0; s < kS; ++s) {
    if (id[s] >= 0) q[s] = q[s] / z;
    m += q[s] * d[s];
  }
  m = dense || a.renorm ? lanes_sum<kL>(m) : 0.0f;
  // The entry's term, to be added at its expert: the whole gradient, or for
  // the dense form d_e of p_e (d_e - m).
  float g[kS];
#pragma unroll
  for (int s = 0; s < kS; ++s) {
    g[s] = dense ? d[s] : q[s] * (d[s] - m);
    if constexpr (S == Score::kSigmoid) {
      float sg, c;
      sigmoid_pair_f32(lk[s], sg, c);
      g[s] *= c;
    }
    if (id[s] < 0) g[s] = 0.0f;
  }
  float acc[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i) acc[i] = 0.0f;
#pragma unroll
  for (int s = 0; s < kS; ++s)
    for (int j = s * kL; j < a.k && j < (s + 1) * kL; ++j) {
      const int ij = __shfl(id[s], j - s * kL, kL);
      const float gj = __shfl(g[s], j - s * kL, kL);
#pragma unroll
      for (int i = 0; i < kV; ++i)
        if (ij == l.expert(i)) acc[i] += gj;
    }
  const float rz = 1.0f / z;
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    if (dense) acc[i] = p[i] == 0.0f ? 0.0f : (p[i] * rz) * (acc[i] - m);
    if (bad != 0) acc[i] = __builtin_nanf("");
  }
  if (live) l.store(static_cast<T*>(a.dlogits) + t * a.E, a.E, acc);
}

template <typename T, Score S, int kL, int kC, bool kTiny = false>
hipError_t launch_lanes(bool fwd, const RouteArgs& a, hipStream_t s) {
  constexpr int per = kThreads / kL;
  const dim3 grid((unsigned)(((int64_t)a.T + per - 1) / per));
  if (fwd) hipLaunchKernelGGL((route_fwd_kernel<T, S, kL, kC, kTiny>), grid, dim3(kThreads), 0, s, a);
  else hipLaunchKernelGGL((route_bwd_kernel<T, S, kL, kC, kTiny>), grid, dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

// 8 logits to a lane: 8 to 64 lanes for up to 512 experts, 16 beyond.
// 32768 x 128, k = 8, forward: 6.9 us bf16 and 10.5 fp32, with 16 logits to
// a lane 8.8 and 13.2 (a longer sort), with 4 (32 lanes, half without logits)
// 11.6 and 17.7; backward with 8 or 16 nearly alike (10.6 and 10.7; 14.5 and
// 14.9), with 4 15.8 and 17.2.
// Fewer than 8 lanes for up to 32 experts, only where tokens fill the chip
// all the same: 524288 x 8 bf16 on one lane each forward 7.1 us and backward
// 9.4, on 8 27 and 26; 131072 x 32 on 4 lanes 9.0 and 10.3, on 8 12.6 and
// 13.5; 32768 x 8 3.2 and 4.6 against 4.1 and 4.6; but 8 x 8 2.7 and 3.7
// against 1.8 and 2.2 (a lane's longer chain; these by a kernel trace).
constexpr int kManyTokens = 32768;
template <typename T, Score S>
hipError_t launch_v(bool fwd, const RouteArgs& a, hipStream_t s) {
  constexpr int kN = Row<T>::kN, kC = 8 / kN;
  if (a.T >= kManyTokens) {
    if (a.E < kN) return launch_lanes<T, S, 1, 1, true>(fwd, a, s);
    if (a.E <= 8) return launch_lanes<T, S, 1, kC>(fwd, a, s);
    if (a.E <= 16) return launch_lanes<T, S, 2, kC>(fwd, a, s);
    if (a.E <= 32) return launch_lanes<T, S, 4, kC>(fwd, a, s);
  }
  if (a.E < kN) return launch_lanes<T, S, 8, 1, true>(fwd, a, s);
  if (a.E <= 64) return launch_lanes<T, S, 8, kC>(fwd, a, s);
  if (a.E <= 128) return launch_lanes<T, S, 16, kC>(fwd, a, s);
  if (a.E <= 256) return launch_lanes<T, S, 32, kC>(fwd, a, s);
  if (a.E <= 512) return launch_lanes<T, S, 64, kC>(fwd, a, s);
  return launch_lanes<T, S, 64, 2 * kC>(fwd, a, s);
}

hipError_t launch(bool fwd, Dt dt, Score score, const RouteArgs& a, hipStream_t s) {
  if (score == Score::kSoftmax)
    return dt == Dt::kBF16 ? launch_v<bf16, Score::kSoftmax>(fwd, a, s) : launch_v<float, Score::kSoftmax>(fwd, a, s);
  return dt == Dt::kBF16 ? launch_v<bf16, Score::kSigmoid>(fwd, a, s) : launch_v<float, Score::kSigmoid>(fwd, a, s);
}

}  // namespace

hipError_t launch_route_fwd(Dt dt, Score score, const RouteArgs& a, hipStream_t s) {
  return launch(true, dt, score, a, s);
}

hipError_t launch_route_bwd(Dt dt, Score score, const RouteArgs& a, hipStream_t s) {
  return launch(false, dt, score, a, s);
}

}  // namespace swg
