// The norms around a block, forward and backward, each in one pass over its
// tensors (the backward's sums over rows take a second, small launch).
//
// Forward, per row, with RMS(v) = v / sqrt(mean(v^2) + eps):
//   n = RMS(y) (o + w_out),   r' = skip res + scale gate n,   z = RMS(r') (o + w_in)
// Backward, with RMS^T(v, d) = r (d - RMS(v) mean(d RMS(v))), r = 1 / sqrt(mean(v^2) + eps):
//   t  = dres_out + RMS^T(r', dz (o + w_in))
//   dy = RMS^T(y, scale t gate (o + w_out)),   dres = skip t
// and the sums over rows
//   a = sum t RMS(y) (per group; t y where there is no w_out),   b = sum dz RMS(r')
// from which dgate = scale a (o + w_out), dw_out = scale sum_groups gate a and
// dw_in = b: one sum serves both dgate and dw_out.
//
// The work is bound by HBM: 2 to 4 tensors forward, 4 to 6 backward.  A row
// is held in registers by `nt` threads as kCH 16-byte chunks each, so each
// tensor is read once: 16, 32 or 64 lanes of a wave for short rows (several
// rows per workgroup), otherwise a whole workgroup of as many waves as the
// row has chunks for.
//
// Rows need not be aligned nor a whole number of chunks: chunks load at any
// element's address, and the chunk that would pass the row's end is loaded
// from cols - kN instead, with the elements it shares with its neighbour
// (`skip` of them) set to zero on use, in the weights and gates as well as in
// the rows, and left to that neighbour, so every load is full and none is
// behind a branch.  Threads past the last chunk skip all
// of theirs.
#include <type_traits>

#include "block.hpp"
#include "common.hpp"
#include "validate.hpp"

namespace swg {

namespace {

// A 16-byte chunk of a row that may start at any element.
typedef u32x4 u32x4_any __attribute__((aligned(2)));

template <typename T> struct Ch;
template <> struct Ch<float> {
  static constexpr int kN = 4;
  __device__ static float get(const u32x4& w, int i) { return bits_f32(w[i]); }
  __device__ static u32x4 pack(const float (&v)[kN]) {
    return u32x4{f32_bits(v[0]), f32_bits(v[1]), f32_bits(v[2]), f32_bits(v[3])};
  }
};
template <> struct Ch<bf16> {
  static constexpr int kN = 8;
  __device__ static float get(const u32x4& w, int i) {
    const uint32_t u = w[i >> 1];
    return bits_f32((i & 1) ? (u & 0xFFFF0000u) : (u << 16));
  }
  __device__ static u32x4 pack(const float (&v)[kN]) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = (uint32_t)__builtin_bit_cast(uint16_t, to_bf16(v[2 * i])) |
             ((uint32_t)__builtin_bit_cast(uint16_t, to_bf16(v[2 * i + 1])) << 16);
    return w;
  }
};

// The chunk a thread holds: kN elements from `start`, of which the first
// `skip` are another's.  kTiny: rows shorter than a chunk (start 0; elements
// from cols on read as zero and are not stored).
template <typename T, bool kTiny>
struct Span {
  static constexpr int kN = Ch<T>::kN;
  int start, skip;
  __device__ __forceinline__ Span(int c, int cols) {
    const int c0 = c * kN;
    if constexpr (kTiny) {
      start = 0;
      skip = c == 0 ? 0 : kN;
    } else {
      start = c0 + kN <= cols ? c0 : cols - kN;
      const int d = c0 - start;
      skip = d < kN ? d : kN;
    }
  }
  // As it lies in memory: shared elements and all (kTiny: zeros past the end).
  __device__ __forceinline__ u32x4 load(const T* row, int cols) const {
    if constexpr (kTiny) {
      T tmp[kN] = {};
#pragma unroll
      for (int i = 0; i < kN - 1; ++i)
        if (skip == 0 && i < cols) tmp[i] = row[i];
      return __builtin_bit_cast(u32x4, tmp);
    } else {
      return *reinterpret_cast<const u32x4_any*>(row + start);
    }
  }
  // Without the elements to skip.  Apart from load, so that a row's loads are
  // all requested before the first is waited for.
  __device__ __forceinline__ u32x4 own(u32x4 w) const {
    constexpr int kPer = kN / 4;                 // elements per word
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (kPer == 2 && skip == 2 * i + 1) w[i] &= 0xFFFF0000u;
      if (skip >= kPer * (i + 1)) w[i] = 0;
    }
    return w;
  }
  __device__ __forceinline__ void store(T* row, int cols, const u32x4& w) const {
    if (!kTiny && skip == 0) {
      *reinterpret_cast<u32x4_any*>(row + start) = w;
    } else if (skip < kN) {
      T tmp[kN];
      __builtin_memcpy(tmp, &w, 16);
#pragma unroll
      for (int i = 0; i < kN; ++i)
        if (i >= skip && start + i < cols) row[start + i] = tmp[i];
    }
  }
};

// Lanes of a row: 16, 32 or 64 of a wave, or (kWide) every thread of the workgroup.
constexpr int kWide = 0;
constexpr int kMaxThreads = 1024;

// The sum over the 16 lanes of a DPP row, in each of them.
__device__ __forceinline__ float sum16(float v) {
  auto add = [&](auto ctrl) {
    v += bits_f32((uint32_t)__builtin_amdgcn_update_dpp(0, (int)f32_bits(v), decltype(ctrl)::value, 0xF, 0xF, true));
  };
  add(std::integral_constant<int, 0xB1>{});      // quad_perm: lane ^ 1
  add(std::integral_constant<int, 0x4E>{});      // quad_perm: lane ^ 2
  add(std::integral_constant<int, 0x141>{});     // row_half_mirror: the other quad of 8
  add(std::integral_constant<int, 0x140>{});     // row_mirror: the other 8 of 16
  return v;
}
__device__ __forceinline__ float sum32(float v) {
  v = sum16(v);
  return v + __shfl_xor(v, 16);
}
__device__ __forceinline__ float sum64(float v) {
  v = sum16(v);
  auto at = [&](int lane) { return bits_f32((uint32_t)__builtin_amdgcn_readlane((int)f32_bits(v), lane)); };
  return (at(0) + at(16)) + (at(32) + at(48));
}

// Sums of kS values over a row's threads, in a fixed order.  The caller
// alternates `slot` between 0 and 1, so one barrier per sum suffices: a
// buffer is rewritten only after every thread passed the other one's.  The
// sums are the critical path of a row where there are few rows, so lanes are
// added by DPP and the (at most 16) waves by the lanes of one DPP row.
template <int kL, int kS>
__device__ __forceinline__ void row_sum(float (&v)[kS], float (*buf)[kS][kMaxThreads / 64], int slot) {
#pragma unroll
  for (int s = 0; s < kS; ++s) v[s] = kL == 16 ? sum16(v[s]) : kL == 32 ? sum32(v[s]) : sum64(v[s]);
  if constexpr (kL == kWide) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, other = lane & 15;
    if (lane == 0)
#pragma unroll
      for (int s = 0; s < kS; ++s) buf[slot][s][wave] = v[s];
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kS; ++s) {
      const float part = buf[slot][s][other];
      v[s] = sum16(other < (int)(blockDim.x >> 6) ? part : 0.0f);
    }
  }
}

__device__ __forceinline__ float rstd_of(float sumsq, int cols, float eps) {
  return 1.0f / sqrtf(sumsq / (float)cols + eps);
}

// What a row's block adds: nothing, y itself, or y's norm.
enum class Join { kNone, kPlain, kNorm };

// Bound by HBM: 8192 x 4096 bf16 with both norms (two tensors read, two
// written, 268 MB) 45 to 48 us, 5.6 to 6.0 TB/s, where a copy reaches 5.1.  A
// few rows are bound by the chain load, sum, sum, store: 8 x 4096 3.5 us.
template <typename T, int kL, int kCH, Join J, bool kZ, bool kTiny>
__global__ __launch_bounds__(kMaxThreads) void norm_fwd_kernel(NormArgs a) {
  constexpr int kN = Ch<T>::kN;
  __shared__ float buf[2][1][kMaxThreads / 64];
  const int nt = kL == kWide ? blockDim.x : kL;
  const int tid = kL == kWide ? threadIdx.x : threadIdx.x % nt;
  const uint32_t row = kL == kWide ? blockIdx.x : blockIdx.x * (blockDim.x / nt) + threadIdx.x / nt;
  if (row >= a.rows) return;                     // whole rows, and no barrier follows where a workgroup has several
  const int64_t at = (int64_t)row * a.cols;
  const bool gated = a.groups > 0;
  const T* gate = static_cast<const T*>(a.gate);
  if (gated) gate += (int64_t)(row / (uint32_t)(a.rows / a.groups)) * a.cols;
  u32x4 res[kCH], y[kCH], wo[kCH], g[kCH], wi[kCH];
#pragma unroll
  for (int i = 0; i < kCH; ++i) {
    const Span<T, kTiny> sp(i * nt + tid, a.cols);
    res[i] = sp.load(static_cast<const T*>(a.res) + at, a.cols);
    if constexpr (J != Join::kNone) y[i] = sp.load(static_cast<const T*>(a.y) + at, a.cols);
  }
#pragma unroll
  for (int i = 0; i < kCH; ++i) {
    const Span<T, kTiny> sp(i * nt + tid, a.cols);
    if constexpr (J == Join::kNorm) wo[i] = sp.load(static_cast<const T*>(a.w_out), a.cols);
    if (J != Join::kNone && gated) g[i] = sp.load(gate, a.cols);
    if constexpr (kZ) wi[i] = sp.load(static_cast<const T*>(a.w_in), a.cols);
  }
#pragma unroll
  for (int i = 0; i < kCH; ++i) {
    const Span<T, kTiny> sp(i * nt + tid, a.cols);
    if (sp.skip != 0) {                          // weights too: 0 * inf is not 0
      res[i] = sp.own(res[i]);
      if constexpr (J != Join::kNone) y[i] = sp.own(y[i]);
      if constexpr (J == Join::kNorm) wo[i] = sp.own(wo[i]);
      if (J != Join::kNone && gated) g[i] = sp.own(g[i]);
    }
  }
  float r[kCH][kN];
  if constexpr (J == Join::kNone) {
#pragma unroll
    for (int i = 0; i < kCH; ++i)
#pragma unroll
      for (int e = 0; e < kN; ++e) r[i][e] = Ch<T>::get(res[i], e);
  } else {
    float k = a.scale;
    if constexpr (J == Join::kNorm) {
      float ss[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < kCH; ++i)
#pragma unroll
        for (int e = 0; e < kN; ++e) {
          const float v = Ch<T>::get(y[i], e);
          ss[0] = __builtin_fmaf(v, v, ss[0]);
        }
      row_sum<kL, 1>(ss, buf, 0);
      k = a.scale * rstd_of(ss[0], a.cols, a.eps);
    }
#pragma unroll
    for (int i = 0; i < kCH; ++i) {
      const Span<T, kTiny> sp(i * nt + tid, a.cols);
#pragma unroll
      for (int e = 0; e < kN; ++e) {
        float n = k * Ch<T>::get(y[i], e);
        if constexpr (J == Join::kNorm) n *= a.w_offset + Ch<T>::get(wo[i], e);
        if (gated) n *= Ch<T>::get(g[i], e);
        r[i][e] = __builtin_fmaf(a.skip, Ch<T>::get(res[i], e), n);
      }
      sp.store(static_cast<T*>(a.res_out) + at, a.cols, Ch<T>::pack(r[i]));
    }
  }
  if constexpr (kZ) {
    float ss[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < kCH; ++i)
#pragma unroll
      for (int e = 0; e < kN; ++e) ss[0] = __builtin_fmaf(r[i][e], r[i][e], ss[0]);
    row_sum<kL, 1>(ss, buf, 1);
    const float k = rstd_of(ss[0], a.cols, a.eps);
#pragma unroll
    for (int i = 0; i < kCH; ++i) {
      const Span<T, kTiny> sp(i * nt + tid, a.cols);
      float o[kN];
#pragma unroll
      for (int e = 0; e < kN; ++e) o[e] = r[i][e] * k * (a.w_offset + Ch<T>::get(wi[i], e));
      sp.store(static_cast<T*>(a.z) + at, a.cols, Ch<T>::pack(o));
    }
  }
}

// Backward: whether the threads' sums over rows lie in LDS.  With 16 elements
// of a row to a thread its registers do not hold them too: 2048 x 12288 bf16
// 138 us in LDS, 204 in registers (spilled).
template <typename T, int kL, int kCH> constexpr bool kSumsInLds = kL == kWide && kCH * Ch<T>::kN > 8;

// Backward.  A workgroup walks one part of the rows: of group p / per_group,
// those whose turn is p % per_group when the group's rows are dealt out R at
// a time (R rows of the workgroup in parallel).  Its sums a and b (over its R
// rows at a time, joined in LDS at the end) go to part[0][p] and part[1][p].
// The weights stay in registers for the whole walk, and with kAhead the next
// row's tensors are requested before the present row's sums, so the loads
// are in flight over the barriers.  Bound by HBM for many rows: 8192 x 4096
// bf16 with both norms (four tensors read, two written, 403 MB) 79 to 85 us,
// 4.8 to 5.1 TB/s (and 6 us for the parts); by a row's chain of loads and two
// sums where a workgroup has few: 1203 x 2051 fp32 in three groups, three
// rows each, 19 us.
template <typename T, int kL, int kCH, Join J, bool kZ, bool kTiny, bool kAhead>
__global__ __launch_bounds__(kMaxThreads) void norm_bwd_kernel(NormArgs a) {
  constexpr int kN = Ch<T>::kN;
  __shared__ float buf[2][2][kMaxThreads / 64];
  extern __shared__ float joined[];              // several rows per workgroup: [R][cols]; or the threads' sums
  const int nt = kL == kWide ? blockDim.x : kL;
  const int tid = kL == kWide ? threadIdx.x : threadIdx.x % nt;
  const int R = kL == kWide ? 1 : blockDim.x / nt, mine = kL == kWide ? 0 : threadIdx.x / nt;
  const uint32_t groups = a.groups > 0 ? (uint32_t)a.groups : 1u;
  const uint32_t p = blockIdx.x, grp = p / (uint32_t)a.per_group, turn = p % (uint32_t)a.per_group;
  const int64_t rpg = (uint32_t)a.rows / groups;
  const bool gated = a.groups > 0;
  const bool sum_a = J == Join::kNorm || gated;
  const bool need_y = J == Join::kNorm || (J == Join::kPlain && gated);
  u32x4 wo[kCH], g[kCH], wi[kCH];
#pragma unroll
  for (int i = 0; i < kCH; ++i) {
    const Span<T, kTiny> sp(i * nt + tid, a.cols);
    if constexpr (J == Join::kNorm) wo[i] = sp.own(sp.load(static_cast<const T*>(a.w_out), a.cols));
    if (J != Join::kNone && gated) g[i] = sp.own(sp.load(static_cast<const T*>(a.gate) + (int64_t)grp * a.cols, a.cols));
    if constexpr (kZ) wi[i] = sp.own(sp.load(static_cast<const T*>(a.w_in), a.cols));
  }
  // This thread's sums, 0: a and 1: b, in registers or LDS.
  float sums[2][kCH][kN];
  auto sum = [&](int s, int i, int e) -> float& {
    if constexpr (kSumsInLds<T, kL, kCH>) return joined[((s * kCH + i) * kN + e) * nt + tid];
    else return sums[s][i][e];
  };
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int i = 0; i < kCH; ++i)
#pragma unroll
      for (int e = 0; e < kN; ++e) sum(s, i, e) = 0.0f;

  struct Row { u32x4 t[kCH], dz[kCH], r[kCH], y[kCH]; };
  auto load = [&](int64_t q, Row& x) {
    const int64_t at = (grp * rpg + q) * a.cols;
#pragma unroll
    for (int i = 0; i < kCH; ++i) {
      const Span<T, kTiny> sp(i * nt + tid, a.cols);
      x.t[i] = u32x4{0u, 0u, 0u, 0u};
      if (a.dres_out != nullptr) x.t[i] = sp.load(static_cast<const T*>(a.dres_out) + at, a.cols);
      if constexpr (kZ) {
        x.dz[i] = sp.load(static_cast<const T*>(a.dz) + at, a.cols);
        x.r[i] = sp.load(static_cast<const T*>(a.res) + at, a.cols);
      }
      if (need_y) x.y[i] = sp.load(static_cast<const T*>(a.y) + at, a.cols);
    }
  };
  int slot = 0;                                  // alternates over the row sums (row_sum)
  auto walk = [&](int64_t q, Row& x) {
    const int64_t at = (grp * rpg + q) * a.cols;
#pragma unroll
    for (int i = 0; i < kCH; ++i) {
      const Span<T, kTiny> sp(i * nt + tid, a.cols);
      if (sp.skip != 0) {
        x.t[i] = sp.own(x.t[i]);
        if constexpr (kZ) {
          x.dz[i] = sp.own(x.dz[i]);
          x.r[i] = sp.own(x.r[i]);
        }
        if (need_y) x.y[i] = sp.own(x.y[i]);
      }
    }
    float t[kCH][kN];
#pragma unroll
    for (int i = 0; i < kCH; ++i)
#pragma unroll
      for (int e = 0; e < kN; ++e) t[i][e] = Ch<T>::get(x.t[i], e);
    if constexpr (kZ) {
      float s[2] = {0.0f, 0.0f};                 // sum r'^2, sum dz (o + w_in) r'
#pragma unroll
      for (int i = 0; i < kCH; ++i)
#pragma unroll
        for (int e = 0; e < kN; ++e) {
          const float v = Ch<T>::get(x.r[i], e);
          s[0] = __builtin_fmaf(v, v, s[0]);
          s[1] = __builtin_fmaf(Ch<T>::get(x.dz[i], e) * (a.w_offset + Ch<T>::get(wi[i], e)), v, s[1]);
        }
      row_sum<kL, 2>(s, buf, slot);
      slot ^= 1;
      const float k = rstd_of(s[0], a.cols, a.eps);
      const float m = k * (s[1] / (float)a.cols);   // mean of d RMS(r')
#pragma unroll
      for (int i = 0; i < kCH; ++i)
#pragma unroll
        for (int e = 0; e < kN; ++e) {
          const float h = Ch<T>::get(x.r[i], e) * k, d = Ch<T>::get(x.dz[i], e);
          sum(1, i, e) = __builtin_fmaf(d, h, sum(1, i, e));
          t[i][e] = __builtin_fmaf(k, d * (a.w_offset + Ch<T>::get(wi[i], e)) - h * m, t[i][e]);
        }
    }
    const float skip = J == Join::kNone ? 1.0f : a.skip;
#pragma unroll
    for (int i = 0; i < kCH; ++i) {
      const Span<T, kTiny> sp(i * nt + tid, a.cols);
      float o[kN];
#pragma unroll
      for (int e = 0; e < kN; ++e) o[e] = skip * t[i][e];
      sp.store(static_cast<T*>(a.dres) + at, a.cols, Ch<T>::pack(o));
    }
    // The gradient of n, scale t gate: t from here on where there is a gate
    // (a takes t before it).
    if constexpr (J == Join::kNorm) {
      float s[2] = {0.0f, 0.0f};                 // sum y^2, sum d y with d = scale t gate (o + w_out)
#pragma unroll
      for (int i = 0; i < kCH; ++i)
#pragma unroll
        for (int e = 0; e < kN; ++e) {
          const float v = Ch<T>::get(x.y[i], e);
          float d = a.scale * (a.w_offset + Ch<T>::get(wo[i], e));
          if (gated) d *= Ch<T>::get(g[i], e);
          s[0] = __builtin_fmaf(v, v, s[0]);
          s[1] = __builtin_fmaf(t[i][e] * d, v, s[1]);
        }
      row_sum<kL, 2>(s, buf, slot);
      slot ^= 1;
      const float k = rstd_of(s[0], a.cols, a.eps);
      const float m = k * (s[1] / (float)a.cols);   // mean of d RMS(y)
#pragma unroll
      for (int i = 0; i < kCH; ++i) {
        const Span<T, kTiny> sp(i * nt + tid, a.cols);
        float o[kN];
#pragma unroll
        for (int e = 0; e < kN; ++e) {
          const float h = Ch<T>::get(x.y[i], e) * k;
          float d = a.scale * (a.w_offset + Ch<T>::get(wo[i], e));
          if (gated) d *= Ch<T>::get(g[i], e);
          sum(0, i, e) = __builtin_fmaf(t[i][e], h, sum(0, i, e));
          o[e] = k * (t[i][e] * d - h * m);
        }
        sp.store(static_cast<T*>(a.dy) + at, a.cols, Ch<T>::pack(o));
      }
    } else if constexpr (J == Join::kPlain) {
#pragma unroll
      for (int i = 0; i < kCH; ++i) {
        const Span<T, kTiny> sp(i * nt + tid, a.cols);
        float o[kN];
#pragma unroll
        for (int e = 0; e < kN; ++e) {
          o[e] = a.scale * t[i][e];
          if (gated) {
            sum(0, i, e) = __builtin_fmaf(t[i][e], Ch<T>::get(x.y[i], e), sum(0, i, e));
            o[e] *= Ch<T>::get(g[i], e);
          }
        }
        sp.store(static_cast<T*>(a.dy) + at, a.cols, Ch<T>::pack(o));
      }
    }
  };
  const int64_t step = (int64_t)a.per_group * R;
  int64_t q = (int64_t)turn * R + mine;
  Row x;
  if constexpr (kAhead) {
    if (q < rpg) load(q, x);
    while (q < rpg) {
      Row next;
      if (q + step < rpg) load(q + step, next);
      walk(q, x);
      x = next;
      q += step;
    }
  } else {
    for (; q < rpg; q += step) {
      load(q, x);
      walk(q, x);
    }
  }
  // The part's sums.
  const int64_t parts = (int64_t)groups * a.per_group;
  auto put = [&](float* out, int s) {
    if constexpr (kL == kWide) {
#pragma unroll
      for (int i = 0; i < kCH; ++i) {
        const Span<T, kTiny> sp(i * nt + tid, a.cols);
        if (!kTiny && sp.skip == 0) {
#pragma unroll
          for (int e = 0; e < kN; e += 4)
            *reinterpret_cast<u32x4_any*>(out + sp.start + e) =
                u32x4{f32_bits(sum(s, i, e)), f32_bits(sum(s, i, e + 1)), f32_bits(sum(s, i, e + 2)),
                      f32_bits(sum(s, i, e + 3))};
        } else {
#pragma unroll
          for (int e = 0; e < kN; ++e)
            if (e >= sp.skip && (!kTiny || e < a.cols)) out[sp.start + e] = sum(s, i, e);
        }
      }
    } else {
      __syncthreads();                           // the last sums have been read
#pragma unroll
      for (int i = 0; i < kCH; ++i) {
        const Span<T, kTiny> sp(i * nt + tid, a.cols);
#pragma unroll
        for (int e = 0; e < kN; ++e)
          if (e >= sp.skip && (!kTiny || e < a.cols)) joined[mine * a.cols + sp.start + e] = sum(s, i, e);
      }
      __syncthreads();
      for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
        float total = joined[c];
        for (int r = 1; r < R; ++r) total += joined[r * a.cols + c];
        out[c] = total;
      }
    }
  };
  if (sum_a) put(a.part + (int64_t)p * a.cols, 0);
  if constexpr (kZ) put(a.part + (parts + p) * a.cols, 1);
}

// Adds the parts.  A workgroup takes 64 columns of the sums a (blockIdx.y =
// 0: dgate and dw_out) or b (1: dw_in).  With few groups its 16 waves share
// each group's parts and are joined in wave order; from 16 groups on a wave
// takes whole groups.  8 loads are in flight per lane.  At 512 parts of 4096
// columns (16.8 MB): 6 us; one load at a time by 4 waves 63 us; 16 columns
// per workgroup 9.5 us (two of them, on two L2s, share each 128-byte line).
constexpr int kSumWaves = 16, kSumThreads = kSumWaves * 64;

__device__ __forceinline__ float sum_parts(const float* __restrict__ p, int64_t n, int64_t first, int64_t step,
                                           int64_t cols) {
  float s = 0.0f;
  int64_t i = first;
  auto turn = [&](auto loads) {
    constexpr int kU = decltype(loads)::value;
    float v[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) v[u] = p[(i + u * step) * cols];
#pragma unroll
    for (int u = 0; u < kU; ++u) s += v[u];
    i += kU * step;
  };
  while (i + 7 * step < n) turn(std::integral_constant<int, 8>{});
  if (i + 3 * step < n) turn(std::integral_constant<int, 4>{});
  if (i + step < n) turn(std::integral_constant<int, 2>{});
  if (i < n) turn(std::integral_constant<int, 1>{});
  return s;
}

template <typename T>
__global__ __launch_bounds__(kSumThreads) void norm_parts_kernel(NormArgs a) {
  constexpr int kGroups = 4;                     // groups joined at a time
  __shared__ float buf[2][kGroups][kSumWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  const bool in = c < a.cols;
  const int64_t groups = a.groups > 0 ? a.groups : 1;
  const int64_t per = a.rows > 0 ? a.per_group : 0, parts = groups * a.per_group;
  // kS sums of the waves, to every wave, in wave order.
  int slot = 0;
  auto join = [&](auto& v) {
    constexpr int kS = sizeof(v) / sizeof(float);
#pragma unroll
    for (int i = 0; i < kS; ++i) buf[slot][i][wave][lane] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kS; ++i) {
      v[i] = buf[slot][i][0][lane];
#pragma unroll
      for (int w = 1; w < kSumWaves; ++w) v[i] += buf[slot][i][w][lane];
    }
    slot ^= 1;
  };
  if (blockIdx.y == 1) {
    if (a.dw_in == nullptr) return;
    float s[1] = {in ? sum_parts(a.part + parts * a.cols + c, per * groups, wave, kSumWaves, a.cols) : 0.0f};
    join(s);
    if (wave == 0 && in) static_cast<T*>(a.dw_in)[c] = (T)s[0];
    return;
  }
  const bool with_gate = a.dgate != nullptr, with_out = a.dw_out != nullptr;
  if (!with_gate && !with_out) return;
  const float w = with_out && in ? a.w_offset + (float)static_cast<const T*>(a.w_out)[c] : 1.0f;
  float dw = 0.0f;
  auto group = [&](int64_t g, float s, bool store) {
    s *= a.scale;
    if (with_gate && store) static_cast<T*>(a.dgate)[g * a.cols + c] = (T)(s * w);
    const float gv = with_gate ? (float)static_cast<const T*>(a.gate)[g * a.cols + c] : 1.0f;
    dw = __builtin_fmaf(gv, s, dw);
  };
  if (groups < kSumWaves) {
    for (int64_t g0 = 0; g0 < groups; g0 += kGroups) {
      float s[kGroups];
#pragma unroll
      for (int i = 0; i < kGroups; ++i)
        s[i] = in && g0 + i < groups ? sum_parts(a.part + (g0 + i) * per * a.cols + c, per, wave, kSumWaves, a.cols) : 0.0f;
      join(s);
#pragma unroll
      for (int i = 0; i < kGroups; ++i)
        if (in && g0 + i < groups) group(g0 + i, s[i], wave == 0);
    }
  } else {
    if (in)
      for (int64_t g = wave; g < groups; g += kSumWaves)
        group(g, sum_parts(a.part + g * per * a.cols + c, per, 0, 1, a.cols), true);
    float s[1] = {dw};
    join(s);
    dw = s[0];
  }
  if (with_out && wave == 0 && in) static_cast<T*>(a.dw_out)[c] = (T)dw;
}

template <typename T>
hipError_t launch_parts(const NormArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(norm_parts_kernel<T>, dim3((unsigned)((a.cols + 63) / 64), 2), dim3(kSumThreads), 0, s, a);
  return hipGetLastError();
}

// One launch: rows of kL lanes (kWide: of as many waves as hold the row).
// Forward workgroups of several rows have 256 threads, backward ones 512.
template <typename T, int kL, int kCH, Join J, bool kZ, bool kTiny = false>
hipError_t launch_cfg(bool fwd, NormArgs a, hipStream_t s) {
  constexpr int kN = Ch<T>::kN;
  const int nch = (a.cols + kN - 1) / kN;
  int threads = norm_wide_threads(nch, kCH);
  if (fwd) {
    const int R = kL == kWide ? 1 : 256 / (kL == kWide ? 1 : kL);
    if (kL != kWide) threads = 256;
    hipLaunchKernelGGL((norm_fwd_kernel<T, kL, kCH, J, kZ, kTiny>), dim3((unsigned)((a.rows + R - 1) / R)),
                       dim3(threads), 0, s, a);
    return hipGetLastError();
  }
  const int64_t groups = a.groups > 0 ? a.groups : 1;
  const int R = kL == kWide ? 1 : kNormThreads / (kL == kWide ? 1 : kL);
  if (kL != kWide) threads = kNormThreads;
  a.per_group = (int)norm_bwd_parts((int)sizeof(T), a.rows, a.cols, a.groups);
  const size_t lds = kSumsInLds<T, kL, kCH> ? (size_t)2 * kCH * kN * threads * 4 : kL == kWide ? 0 : (size_t)R * a.cols * 4;
  // Next-row loads where the 128 registers of a thread hold two rows: with
  // two fp32 chunks each they do not, 2048 x 8192 107 us with them, 87 without.
  constexpr bool kAhead = kCH == 1;
  constexpr auto kernel = &norm_bwd_kernel<T, kL, kCH, J, kZ, kTiny, kAhead>;
  hipError_t e = hipSuccess;
  if constexpr (kSumsInLds<T, kL, kCH>) e = allow_lds<kernel>((size_t)2 * kCH * kN * kMaxThreads * 4);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(groups * a.per_group)), dim3(threads), lds, s, a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (a.dw_out == nullptr && a.dgate == nullptr && a.dw_in == nullptr) return hipSuccess;
  return launch_parts<T>(a, s);
}

// As few lanes as hold a row one chunk each: 65536 rows of 256 bf16 columns
// forward 23 us on 32 lanes against 35 on 64, backward 36 against 56; of 128
// columns forward 12.8 on 16 lanes against 35.  Long forward rows take two
// chunks to a thread where there are rows enough: 8192 x 4096 bf16 47.8 us
// against 50.2, 2048 x 8192 26.6 against 30.6, 8192 x 4096 fp32 98 against 104,
// with 1024 rows the same, and with fewer the shorter chain of one chunk counts.
template <typename T, Join J, bool kZ>
hipError_t launch_cols(bool fwd, const NormArgs& a, hipStream_t s) {
  constexpr int kN = Ch<T>::kN;
  const int nch = (a.cols + kN - 1) / kN;
  if (a.cols < kN) return launch_cfg<T, 16, 1, J, kZ, true>(fwd, a, s);
  const int lanes = norm_lanes(nch), chunks = norm_chunks(nch);
  if (lanes == 16) return launch_cfg<T, 16, 1, J, kZ>(fwd, a, s);
  if (lanes == 32) return launch_cfg<T, 32, 1, J, kZ>(fwd, a, s);
  if (lanes == 64) return launch_cfg<T, 64, 1, J, kZ>(fwd, a, s);
  if (fwd && a.rows > 512 && nch > 256 && chunks == 1) return launch_cfg<T, kWide, 2, J, kZ>(fwd, a, s);
  if (chunks == 1) return launch_cfg<T, kWide, 1, J, kZ>(fwd, a, s);
  if (chunks == 2) return launch_cfg<T, kWide, 2, J, kZ>(fwd, a, s);
  if constexpr (sizeof(T) == 4) return launch_cfg<T, kWide, 4, J, kZ>(fwd, a, s);
  return hipErrorInvalidValue;                   // past the checked number of columns
}

template <typename T>
hipError_t launch_t(bool fwd, const NormArgs& a, hipStream_t s) {
  const bool z = a.w_in != nullptr;
  if (a.y == nullptr) return launch_cols<T, Join::kNone, true>(fwd, a, s);
  if (a.w_out == nullptr)
    return z ? launch_cols<T, Join::kPlain, true>(fwd, a, s) : launch_cols<T, Join::kPlain, false>(fwd, a, s);
  return z ? launch_cols<T, Join::kNorm, true>(fwd, a, s) : launch_cols<T, Join::kNorm, false>(fwd, a, s);
}

}  // namespace

hipError_t launch_norm_fwd(Dt dt, const NormArgs& a, hipStream_t s) {
  return dt == Dt::kBF16 ? launch_t<bf16>(true, a, s) : launch_t<float>(true, a, s);
}

hipError_t launch_norm_bwd(Dt dt, const NormArgs& a, hipStream_t s) {
  if (a.rows > 0) return dt == Dt::kBF16 ? launch_t<bf16>(false, a, s) : launch_t<float>(false, a, s);
  if (a.dw_out == nullptr && a.dgate == nullptr && a.dw_in == nullptr) return hipSuccess;
  return dt == Dt::kBF16 ? launch_parts<bf16>(a, s) : launch_parts<float>(a, s);   // sums over no rows
}

}  // namespace swg
