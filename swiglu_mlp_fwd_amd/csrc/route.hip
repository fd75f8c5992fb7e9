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
// One wave per token: lane l holds logits l, l + 64, ...
#include "block.hpp"
#include "common.hpp"

namespace swg {

namespace {

constexpr int kWavesPerBlock = 4;
constexpr float kInf = __builtin_inff();

// e^-a for a >= 0 to about two ulps; 0 from where it underflows, +inf included.
__device__ __forceinline__ float exp_neg(float a) {
  float p;
  int n;
  exp_neg_split(fminf(a, 1024.0f), p, n);
  return ldexpf(p, n);
}

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const bf16* p) { return from_bf16(*p); }
__device__ __forceinline__ void store_grad(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_grad(bf16* p, float v) { *p = to_bf16(v); }

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor(v, off));
  return v;
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

template <typename T, Score S, int V>
__global__ __launch_bounds__(kWavesPerBlock * 64) void route_fwd_kernel(RouteArgs a) {
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * kWavesPerBlock + (threadIdx.x >> 6);
  if (t >= a.T) return;
  const T* row = static_cast<const T*>(a.logits) + (int64_t)t * a.E;
  float l[V], left[V];
  bool bad = false;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * 64 + lane;
    l[v] = e < a.E ? load_logit(row + e) : -kInf;
    if (l[v] != l[v] || (S == Score::kSoftmax && l[v] == kInf)) bad = true;
    left[v] = l[v] != l[v] ? -kInf : l[v];
  }
  bad = __any(bad);
  float mine = -kInf;                              // lane j: the j-th choice
  int my_id = -1;
  for (int j = 0; j < a.k; ++j) {
    float best = -kInf;
    int at = 1 << 30;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (left[v] > best) { best = left[v]; at = v * 64 + lane; }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
      const float ob = __shfl_xor(best, off);
      const int oa = __shfl_xor(at, off);
      if (ob > best || (ob == best && oa < at)) { best = ob; at = oa; }
    }
    if (best == -kInf) break;                      // none left
    if (lane == j) { mine = best; my_id = at; }
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (at == v * 64 + lane) left[v] = -kInf;
  }
  const float top = __shfl(mine, 0);
  const bool have = my_id >= 0;
  float w = have ? chosen_score<S>(mine, top, a.renorm) : 0.0f;
  float z = 1.0f;
  if (a.renorm) {
    z = wave_sum(w);
  } else if constexpr (S == Score::kSoftmax) {
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) sum += l[v] == -kInf ? 0.0f : exp_neg(top - l[v]);
    z = wave_sum(sum);
  }
  if (lane < a.k) {
    w = have ? a.scale * (w / z) : 0.0f;
    if (bad) w = __builtin_nanf("");
    a.weights[(int64_t)t * a.k + lane] = w;
    a.ids[(int64_t)t * a.k + lane] = my_id;
  }
}

template <typename T, Score S, int V>
__global__ __launch_bounds__(kWavesPerBlock * 64) void route_bwd_kernel(RouteArgs a) {
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * kWavesPerBlock + (threadIdx.x >> 6);
  if (t >= a.T) return;
  const T* row = static_cast<const T*>(a.logits) + (int64_t)t * a.E;
  T* out = static_cast<T*>(a.dlogits) + (int64_t)t * a.E;
  float l[V];
  bool bad = false;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * 64 + lane;
    l[v] = e < a.E ? load_logit(row + e) : -kInf;
    if (l[v] != l[v] || (S == Score::kSoftmax && l[v] == kInf)) bad = true;
  }
  bad = __any(bad);
  // Lane j < k: entry j of the token's choice.
  int id = -1;
  float d = 0.0f, lk = -kInf;
  if (lane < a.k) {
    id = a.ids_in[(int64_t)t * a.k + lane];
    if (id < 0 || id >= a.E) id = -1;
    if (id >= 0) lk = load_logit(row + id);
    if (lk == -kInf) id = -1;                      // masked: no gradient
    if (id >= 0) d = a.scale * a.dweights[(int64_t)t * a.k + lane];
  }
  const bool dense = S == Score::kSoftmax && !a.renorm;
  float top;
  if (dense) {
    top = l[0];
#pragma unroll
    for (int v = 1; v < V; ++v) top = fmaxf(top, l[v]);
    top = wave_max(top);
  } else {
    top = wave_max(id >= 0 ? lk : -kInf);
  }
  float q = id >= 0 ? chosen_score<S>(lk, top, a.renorm) : 0.0f;
  float z = 1.0f;
  float p[V];
  if (dense) {
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      p[v] = l[v] == -kInf ? 0.0f : exp_neg(top - l[v]);
      sum += p[v];
    }
    z = wave_sum(sum);
  } else if (a.renorm) {
    z = wave_sum(q);
  }
  if (id >= 0) q = q / z;
  const float m = (dense || a.renorm) ? wave_sum(q * d) : 0.0f;
  // This lane's entry, to be added at its expert: the whole gradient, or for
  // the dense form d_e of p_e (d_e - m).
  float g = 0.0f;
  if (id >= 0) {
    if (dense) {
      g = d;
    } else {
      g = q * (d - m);
      if constexpr (S == Score::kSigmoid) {
        float s, c;
        sigmoid_pair_f32(lk, s, c);
        g *= c;
      }
    }
  }
  float acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.0f;
  for (int j = 0; j < a.k; ++j) {
    const int ij = __shfl(id, j);
    const float gj = __shfl(g, j);
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (ij == v * 64 + lane) acc[v] += gj;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * 64 + lane;
    if (e >= a.E) continue;
    float r = acc[v];
    if (dense) r = p[v] == 0.0f ? 0.0f : (p[v] / z) * (r - m);
    store_grad(out + e, bad ? __builtin_nanf("") : r);
  }
}

template <typename T, Score S>
hipError_t launch_v(bool fwd, const RouteArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)(((int64_t)a.T + kWavesPerBlock - 1) / kWavesPerBlock)), block(kWavesPerBlock * 64);
#define SWG_ROUTE(V)                                                               \
  if (a.E <= 64 * V) {                                                             \
    if (fwd) hipLaunchKernelGGL((route_fwd_kernel<T, S, V>), grid, block, 0, s, a); \
    else hipLaunchKernelGGL((route_bwd_kernel<T, S, V>), grid, block, 0, s, a);    \
    return hipGetLastError();                                                      \
  }
  SWG_ROUTE(1)
  SWG_ROUTE(2)
  SWG_ROUTE(4)
  SWG_ROUTE(8)
  SWG_ROUTE(16)
#undef SWG_ROUTE
  return hipErrorInvalidValue;
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
