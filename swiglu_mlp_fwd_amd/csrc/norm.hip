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
// is held in registers by kNT threads (one wave, or a whole workgroup) as
// kCH 16-byte chunks each, so each tensor is read once; rows need not be
// aligned (chunks load at any element's address, and the last chunk of a row
// that is not whole goes element by element).
#include "block.hpp"
#include "common.hpp"

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

// Chunk c of the row at p; elements past cols read as zero.
template <typename T>
__device__ __forceinline__ u32x4 load_chunk(const T* p, int c, int cols) {
  constexpr int kN = Ch<T>::kN;
  const int c0 = c * kN;
  if (c0 + kN <= cols) return *reinterpret_cast<const u32x4_any*>(p + c0);
  u32x4 w = {0u, 0u, 0u, 0u};
  if (c0 < cols) {
    T tmp[kN] = {};
#pragma unroll
    for (int i = 0; i < kN - 1; ++i)
      if (c0 + i < cols) tmp[i] = p[c0 + i];
    w = __builtin_bit_cast(u32x4, tmp);
  }
  return w;
}

template <typename T>
__device__ __forceinline__ void store_chunk(T* p, int c, int cols, const u32x4& w) {
  constexpr int kN = Ch<T>::kN;
  const int c0 = c * kN;
  if (c0 + kN <= cols) {
    *reinterpret_cast<u32x4_any*>(p + c0) = w;
  } else if (c0 < cols) {
    T tmp[kN];
    __builtin_memcpy(tmp, &w, 16);
#pragma unroll
    for (int i = 0; i < kN - 1; ++i)
      if (c0 + i < cols) p[c0 + i] = tmp[i];
  }
}

// Threads per workgroup for rows of kNT threads: 4 rows of one wave each, or
// one row of the whole workgroup.
template <int kNT> constexpr int kBlock = kNT == 64 ? 256 : kNT;

// Sums of kS values over the kNT threads of a row, in a fixed order.  The
// caller alternates `slot` between 0 and 1, so one barrier per sum suffices:
// a buffer is rewritten only after every thread passed the other one's.
template <int kNT, int kS>
__device__ __forceinline__ void row_sum(float (&v)[kS], float (*buf)[kS][kNT / 64], int slot) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1)
#pragma unroll
    for (int s = 0; s < kS; ++s) v[s] += __shfl_xor(v[s], off);
  if constexpr (kNT > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int s = 0; s < kS; ++s) buf[slot][s][wave] = v[s];
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kS; ++s) {
      float sum = buf[slot][s][0];
#pragma unroll
      for (int w = 1; w < kNT / 64; ++w) sum += buf[slot][s][w];
      v[s] = sum;
    }
  }
}

__device__ __forceinline__ float rstd_of(float sumsq, int cols, float eps) {
  return 1.0f / sqrtf(sumsq / (float)cols + eps);
}

// What a row's block adds: nothing, y itself, or y's norm.
enum class Join { kNone, kPlain, kNorm };

template <typename T, int kNT, int kCH, Join J, bool kZ>
__global__ __launch_bounds__(kBlock<kNT>) void norm_fwd_kernel(NormArgs a) {
  constexpr int kN = Ch<T>::kN;
  __shared__ float buf[2][1][kNT / 64];
  const int tid = threadIdx.x % kNT;
  const uint32_t row = kNT == 64 ? blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  if (row >= a.rows) return;                     // a whole wave of a one-wave row
  const int64_t at = (int64_t)row * a.cols;
  const T* w_out = static_cast<const T*>(a.w_out);
  const T* w_in = static_cast<const T*>(a.w_in);
  u32x4 res[kCH], y[kCH];
#pragma unroll
  for (int i = 0; i < kCH; ++i) {
    res[i] = load_chunk(static_cast<const T*>(a.res) + at, i * kNT + tid, a.cols);
    if constexpr (J != Join::kNone) y[i] = load_chunk(static_cast<const T*>(a.y) + at, i * kNT + tid, a.cols);
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
      row_sum<kNT, 1>(ss, buf, 0);
      k = a.scale * rstd_of(ss[0], a.cols, a.eps);
    }
    const T* gate = nullptr;
    if (a.groups > 0) gate = static_cast<const T*>(a.gate) + (int64_t)(row / (uint32_t)(a.rows / a.groups)) * a.cols;
#pragma unroll
    for (int i = 0; i < kCH; ++i) {
      const int c = i * kNT + tid;
      u32x4 w = {0u, 0u, 0u, 0u}, g = w;
      if constexpr (J == Join::kNorm) w = load_chunk(w_out, c, a.cols);
      if (gate != nullptr) g = load_chunk(gate, c, a.cols);
      float o[kN];
#pragma unroll
      for (int e = 0; e < kN; ++e) {
        float n = k * Ch<T>::get(y[i], e);
        if constexpr (J == Join::kNorm) n *= a.w_offset + Ch<T>::get(w, e);
        if (gate != nullptr) n *= Ch<T>::get(g, e);
        r[i][e] = o[e] = __builtin_fmaf(a.skip, Ch<T>::get(res[i], e), n);
      }
      store_chunk(static_cast<T*>(a.res_out) + at, c, a.cols, Ch<T>::pack(o));
    }
  }
  if constexpr (kZ) {
    float ss[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < kCH; ++i)
#pragma unroll
      for (int e = 0; e < kN; ++e) ss[0] = __builtin_fmaf(r[i][e], r[i][e], ss[0]);   // 0 past the row's end
    row_sum<kNT, 1>(ss, buf, 1);
    const float k = rstd_of(ss[0], a.cols, a.eps);
#pragma unroll
    for (int i = 0; i < kCH; ++i) {
      const int c = i * kNT + tid;
      const u32x4 w = load_chunk(w_in, c, a.cols);
      float o[kN];
#pragma unroll
      for (int e = 0; e < kN; ++e) o[e] = r[i][e] * k * (a.w_offset + Ch<T>::get(w, e));
      store_chunk(static_cast<T*>(a.z) + at, c, a.cols, Ch<T>::pack(o));
    }
  }
}

// Part p of the rows: those of group p / per_group whose index in the group
// is p % per_group modulo per_group.  A part is walked by the kNT threads of
// one row; its sums a and b go to part[0][p] and part[1][p].
template <typename T, int kNT, int kCH, Join J, bool kZ>
__global__ __launch_bounds__(kBlock<kNT>) void norm_bwd_kernel(NormArgs a) {
  constexpr int kN = Ch<T>::kN;
  __shared__ float buf[2][2][kNT / 64];
  const int tid = threadIdx.x % kNT;
  const int64_t groups = a.groups > 0 ? a.groups : 1;
  const int64_t parts = groups * a.per_group;
  const int64_t p = kNT == 64 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : (int64_t)blockIdx.x;
  if (p >= parts) return;
  const int64_t rpg = a.rows / groups, g = p / a.per_group;
  const T* gate = a.groups > 0 ? static_cast<const T*>(a.gate) + g * a.cols : nullptr;
  const bool sum_a = J == Join::kNorm || gate != nullptr;
  float sa[kCH][kN], sb[kCH][kN];
#pragma unroll
  for (int i = 0; i < kCH; ++i)
#pragma unroll
    for (int e = 0; e < kN; ++e) sa[i][e] = sb[i][e] = 0.0f;

  int slot = 0;                                  // alternates over the row sums (row_sum)
  for (int64_t q = p % a.per_group; q < rpg; q += a.per_group) {
    const int64_t at = (g * rpg + q) * a.cols;
    u32x4 t4[kCH], dz[kCH], rr[kCH], y[kCH];
#pragma unroll
    for (int i = 0; i < kCH; ++i) {
      const int c = i * kNT + tid;
      t4[i] = u32x4{0u, 0u, 0u, 0u};
      if (a.dres_out != nullptr) t4[i] = load_chunk(static_cast<const T*>(a.dres_out) + at, c, a.cols);
      if constexpr (kZ) {
        dz[i] = load_chunk(static_cast<const T*>(a.dz) + at, c, a.cols);
        rr[i] = load_chunk(static_cast<const T*>(a.res) + at, c, a.cols);
      }
      if (J == Join::kNorm || (J == Join::kPlain && gate != nullptr))
        y[i] = load_chunk(static_cast<const T*>(a.y) + at, c, a.cols);
    }
    float t[kCH][kN];
#pragma unroll
    for (int i = 0; i < kCH; ++i)
#pragma unroll
      for (int e = 0; e < kN; ++e) t[i][e] = Ch<T>::get(t4[i], e);
    if constexpr (kZ) {
      float s[2] = {0.0f, 0.0f};                 // sum r'^2, sum dz (o + w_in) r'
#pragma unroll
      for (int i = 0; i < kCH; ++i) {
        const u32x4 w = load_chunk(static_cast<const T*>(a.w_in), i * kNT + tid, a.cols);
#pragma unroll
        for (int e = 0; e < kN; ++e) {
          const float v = Ch<T>::get(rr[i], e);
          s[0] = __builtin_fmaf(v, v, s[0]);
          s[1] = __builtin_fmaf(Ch<T>::get(dz[i], e) * (a.w_offset + Ch<T>::get(w, e)), v, s[1]);
        }
      }
      row_sum<kNT, 2>(s, buf, slot);
      slot ^= 1;
      const float k = rstd_of(s[0], a.cols, a.eps);
      const float m = k * (s[1] / (float)a.cols);   // mean of d RMS(r')
#pragma unroll
      for (int i = 0; i < kCH; ++i) {
        const u32x4 w = load_chunk(static_cast<const T*>(a.w_in), i * kNT + tid, a.cols);
#pragma unroll
        for (int e = 0; e < kN; ++e) {
          const float v = Ch<T>::get(rr[i], e), d = Ch<T>::get(dz[i], e);
          sb[i][e] = __builtin_fmaf(d, v * k, sb[i][e]);
          t[i][e] += k * (d * (a.w_offset + Ch<T>::get(w, e)) - v * k * m);
        }
      }
    }
    const float skip = J == Join::kNone ? 1.0f : a.skip;
#pragma unroll
    for (int i = 0; i < kCH; ++i) {
      float o[kN];
#pragma unroll
      for (int e = 0; e < kN; ++e) o[e] = skip * t[i][e];
      store_chunk(static_cast<T*>(a.dres) + at, i * kNT + tid, a.cols, Ch<T>::pack(o));
    }
    if constexpr (J == Join::kNorm) {
      float s[2] = {0.0f, 0.0f};                 // sum y^2, sum d y with d = scale t gate (o + w_out)
#pragma unroll
      for (int i = 0; i < kCH; ++i) {
        const int c = i * kNT + tid;
        const u32x4 w = load_chunk(static_cast<const T*>(a.w_out), c, a.cols);
        u32x4 g4 = {0u, 0u, 0u, 0u};
        if (gate != nullptr) g4 = load_chunk(gate, c, a.cols);
#pragma unroll
        for (int e = 0; e < kN; ++e) {
          const float v = Ch<T>::get(y[i], e);
          float d = a.scale * (a.w_offset + Ch<T>::get(w, e));
          if (gate != nullptr) d *= Ch<T>::get(g4, e);
          s[0] = __builtin_fmaf(v, v, s[0]);
          s[1] = __builtin_fmaf(t[i][e] * d, v, s[1]);
        }
      }
      row_sum<kNT, 2>(s, buf, slot);
      slot ^= 1;
      const float k = rstd_of(s[0], a.cols, a.eps);
      const float m = k * (s[1] / (float)a.cols);   // mean of d RMS(y)
#pragma unroll
      for (int i = 0; i < kCH; ++i) {
        const int c = i * kNT + tid;
        const u32x4 w = load_chunk(static_cast<const T*>(a.w_out), c, a.cols);
        u32x4 g4 = {0u, 0u, 0u, 0u};
        if (gate != nullptr) g4 = load_chunk(gate, c, a.cols);
        float o[kN];
#pragma unroll
        for (int e = 0; e < kN; ++e) {
          const float v = Ch<T>::get(y[i], e);
          float d = a.scale * (a.w_offset + Ch<T>::get(w, e));
          if (gate != nullptr) d *= Ch<T>::get(g4, e);
          sa[i][e] = __builtin_fmaf(t[i][e], v * k, sa[i][e]);
          o[e] = k * (t[i][e] * d - v * k * m);
        }
        store_chunk(static_cast<T*>(a.dy) + at, c, a.cols, Ch<T>::pack(o));
      }
    } else if constexpr (J == Join::kPlain) {
#pragma unroll
      for (int i = 0; i < kCH; ++i) {
        const int c = i * kNT + tid;
        float o[kN];
        if (gate != nullptr) {
          const u32x4 g4 = load_chunk(gate, c, a.cols);
#pragma unroll
          for (int e = 0; e < kN; ++e) {
            sa[i][e] = __builtin_fmaf(t[i][e], Ch<T>::get(y[i], e), sa[i][e]);
            o[e] = a.scale * t[i][e] * Ch<T>::get(g4, e);
          }
        } else {
#pragma unroll
          for (int e = 0; e < kN; ++e) o[e] = a.scale * t[i][e];
        }
        store_chunk(static_cast<T*>(a.dy) + at, c, a.cols, Ch<T>::pack(o));
      }
    }
  }
  // The part's sums.
#pragma unroll
  for (int i = 0; i < kCH; ++i)
#pragma unroll
    for (int e = 0; e < kN; ++e) {
      const int c = (i * kNT + tid) * kN + e;
      if (c >= a.cols) continue;
      if (sum_a) a.part[p * a.cols + c] = sa[i][e];
      if (kZ) a.part[(parts + p) * a.cols + c] = sb[i][e];
    }
}

// Adds the parts: a workgroup takes 64 columns, its 4 waves every fourth
// part, joined in wave order.
template <typename T>
__global__ __launch_bounds__(256) void norm_parts_kernel(NormArgs a) {
  __shared__ float buf[2][4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  const bool in = c < a.cols;
  const int64_t groups = a.groups > 0 ? a.groups : 1;
  const int64_t per = a.rows > 0 ? a.per_group : 0, parts = groups * a.per_group;
  const bool with_gate = a.dgate != nullptr, with_out = a.dw_out != nullptr;
  const float w = with_out && in ? a.w_offset + (float)static_cast<const T*>(a.w_out)[c] : 1.0f;
  int slot = 0;
  auto total = [&](const float* base) {          // sum over `per` parts, to every wave
    float s = 0.0f;
    if (in)
      for (int64_t i = wave; i < per; i += 4) s += base[i * a.cols + c];
    buf[slot][wave][lane] = s;
    __syncthreads();
    s = buf[slot][0][lane] + buf[slot][1][lane] + buf[slot][2][lane] + buf[slot][3][lane];
    slot ^= 1;
    return s;
  };
  if (with_gate || with_out) {
    float dw = 0.0f;
    for (int64_t g = 0; g < groups; ++g) {
      const float s = a.scale * total(a.part + g * per * a.cols);
      if (with_gate && wave == 0 && in) static_cast<T*>(a.dgate)[g * a.cols + c] = (T)(s * w);
      const float gv = with_gate && in ? (float)static_cast<const T*>(a.gate)[g * a.cols + c] : 1.0f;
      dw = __builtin_fmaf(gv, s, dw);
    }
    if (with_out && wave == 0 && in) static_cast<T*>(a.dw_out)[c] = (T)dw;
  }
  if (a.dw_in != nullptr) {
    float s = 0.0f;
    for (int64_t g = 0; g < groups; ++g) s += total(a.part + (parts + g * per) * a.cols);
    if (wave == 0 && in) static_cast<T*>(a.dw_in)[c] = (T)s;
  }
}

template <typename T, int kNT, int kCH, Join J, bool kZ>
hipError_t launch_cfg(bool fwd, const NormArgs& a, hipStream_t s) {
  const int64_t units = fwd ? a.rows : (a.groups > 0 ? a.groups : 1) * a.per_group;
  const int64_t blocks = kNT == 64 ? (units + 3) / 4 : units;
  if (fwd)
    hipLaunchKernelGGL((norm_fwd_kernel<T, kNT, kCH, J, kZ>), dim3((unsigned)blocks), dim3(kBlock<kNT>), 0, s, a);
  else
    hipLaunchKernelGGL((norm_bwd_kernel<T, kNT, kCH, J, kZ>), dim3((unsigned)blocks), dim3(kBlock<kNT>), 0, s, a);
  return hipGetLastError();
}

template <typename T, Join J, bool kZ>
hipError_t launch_cols(bool fwd, const NormArgs& a, hipStream_t s) {
  const int nch = (a.cols + Ch<T>::kN - 1) / Ch<T>::kN;
  if (nch <= 64) return launch_cfg<T, 64, 1, J, kZ>(fwd, a, s);
  if (nch <= 128) return launch_cfg<T, 64, 2, J, kZ>(fwd, a, s);
  if (nch <= 256) return launch_cfg<T, 256, 1, J, kZ>(fwd, a, s);
  if (nch <= 512) return launch_cfg<T, 256, 2, J, kZ>(fwd, a, s);
  if (nch <= 1024) return launch_cfg<T, 512, 2, J, kZ>(fwd, a, s);
  if (nch <= 2048) return launch_cfg<T, 1024, 2, J, kZ>(fwd, a, s);
  if constexpr (sizeof(T) == 4) {
    if (nch <= 4096) return launch_cfg<T, 1024, 4, J, kZ>(fwd, a, s);
  }
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
  if (a.rows > 0) {
    const hipError_t e = dt == Dt::kBF16 ? launch_t<bf16>(false, a, s) : launch_t<float>(false, a, s);
    if (e != hipSuccess) return e;
  }
  if (a.dw_out == nullptr && a.dgate == nullptr && a.dw_in == nullptr) return hipSuccess;
  const dim3 grid((unsigned)((a.cols + 63) / 64));
  if (dt == Dt::kBF16) hipLaunchKernelGGL(norm_parts_kernel<bf16>, grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(norm_parts_kernel<float>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace swg
