// The order of rows by expert, and tokens to rows and back.
//
//   plan          pairs (token, choice) sorted by expert, equal ones in order
//                 of the pair: offsets, src (row -> pair) and pos (pair -> row)
//   gather        rows from tokens
//   combine       y[t] = sum_j w[t, j] rows[pos[t, j]], and its gradients
//
// Everything is in a fixed order, without atomics on memory.  The plan is a
// counting sort: every wave counts its run of pairs by expert in LDS, the
// counts of earlier waves (and blocks) give each wave its first row per
// expert, and it then places its pairs 64 at a time, a pair's rank among the
// 64 from ballots over the bits of the expert.  Up to kPlanOne pairs take one
// workgroup and one launch; more take a launch that counts and one that
// places, in which every block adds up the counts of the blocks before it.
// 512 pairs take 3.3 us (10.6 with the call), 262144 pairs of 128 experts
// 3.3 + 12.2 us.  The second launch is bound by the sum over all blocks'
// counts, 128 x (E + 1) of them in every block, each a load, a remainder and
// up to two LDS atomics: 5.4 us with 8 experts, 6.8 with 32, 12.2 with 128,
// 31 with 512.
// Gather and combine move each row once in 16-byte chunks, a wave taking one
// token (or a part of its columns), whose pairs' rows and weights are scalars.
// HBM bounds them: combine of 4096 tokens of 8 rows of 2048 bf16 24-26 us (151 MB,
// 5.9 TB/s), its gradient for 8192 tokens of 2 rows of 4096 62-65 us (336 MB,
// 5.2 TB/s).  Gather of 32768 rows of 2048 bf16 takes 41 us (151 MB, 3.7 TB/s):
// a lane has one chunk in flight, behind the load of its row's index.
#include "common.hpp"
#include "grouped.hpp"
#include "mfma.hpp"
#include "validate.hpp"

namespace swg {

namespace {

// ------------------------------------------------------------------- plan

constexpr int kPlanWaves = kPlanThreads / 64;

// Key of pair i: its expert, E where it has none; -1 behind the last pair.
__device__ __forceinline__ int plan_key(const PlanArgs& p, int i) {
  if (i >= p.n) return -1;
  const int e = p.ids[i];
  return e >= 0 && e < p.E ? e : p.E;
}

// Lanes of the wave with the same key (bits: those of keys up to E).
__device__ __forceinline__ uint64_t same_key(int key, int bits) {
  uint64_t m = __ballot(key >= 0);
  for (int b = 0; b < bits; ++b) {
    const bool one = (key >> b) & 1;
    const uint64_t with = __ballot(one);
    m &= one ? with : ~with;
  }
  return m;
}

// kCount: counts of the block's pairs to hist.  Otherwise offsets, src and
// pos; with more than one block, hist holds all blocks' counts.
template <bool kCount>
__global__ __launch_bounds__(kPlanThreads) void plan_kernel(PlanArgs p, int per_block) {
  extern __shared__ int32_t cnt[];                        // [kPlanWaves][E + 1], then twice [E + 1]
  const int keys = p.E + 1;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int i = tid; i < kPlanWaves * keys; i += kPlanThreads) cnt[i] = 0;
  __syncthreads();
  // A wave's run: a whole number of 64 pairs.
  const int per_wave = per_block / kPlanWaves;
  const int64_t first = (int64_t)blockIdx.x * per_block + (int64_t)wave * per_wave;
  int32_t* mine = cnt + wave * keys;
  for (int s = 0; s < per_wave; s += 64) {
    const int64_t i = first + s + lane;
    const int key = i < p.n ? plan_key(p, (int)i) : -1;
    if (key >= 0) atomicAdd(mine + key, 1);               // LDS; only the sums are used
  }
  __syncthreads();
  int32_t* start = cnt + kPlanWaves * keys;               // the block's, then all counts of each key
  int32_t* before = start + keys;                         // the earlier blocks' (more than one)
  // Per key: counts of earlier waves into each wave's place.
  for (int e = tid; e < keys; e += kPlanThreads) {
    int sum = 0;
    for (int w = 0; w < kPlanWaves; ++w) {
      const int c = cnt[w * keys + e];
      cnt[w * keys + e] = sum;
      sum += c;
    }
    if constexpr (kCount) p.hist[(int64_t)blockIdx.x * keys + e] = sum;
    start[e] = gridDim.x > 1 ? 0 : sum;
    before[e] = 0;
  }
  if (!kCount && gridDim.x > 1) {
    // Every block's counts, all threads over the whole array at once (one key
    // to a thread took 30 us for 128 blocks, a chain of loads).
    __syncthreads();
    const int n = (int)gridDim.x * keys, mine_from = (int)blockIdx.x * keys;
    for (int i = tid; i < n; i += kPlanThreads) {
      const int c = p.hist[i];
      if (c != 0) {
        atomicAdd(start + i % keys, c);
        if (i < mine_from) atomicAdd(before + i % keys, c);
      }
    }
  }
  if constexpr (kCount) return;
  __syncthreads();
  // Exclusive sum over keys, by the first wave.
  if (wave == 0) {
    int base = 0;
    for (int c = 0; c < keys; c += 64) {
      const int e = c + lane;
      const int v = e < keys ? start[e] : 0;
      int scan = v;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(scan, d);
        if (lane >= d) scan += o;
      }
      if (e < keys) {
        start[e] = base + scan - v;
        if (blockIdx.x == 0) p.offsets[e] = base + scan - v;
      }
      base += __builtin_amdgcn_readlane(scan, 63);
    }
  }
  __syncthreads();
  const int bits = 32 - __builtin_clz(p.E);
  for (int s = 0; s < per_wave; s += 64) {
    const int64_t i = first + s + lane;
    const int key = i < p.n ? plan_key(p, (int)i) : -1;
    const uint64_t same = same_key(key, bits);
    if (key >= 0) {
      const int rank = __popcll(same & ((uint64_t(1) << lane) - 1));
      const int at = mine[key];
      const int row = start[key] + before[key] + at + rank;
      p.src[row] = key < p.E ? (int)i : ~(int)i;
      p.pos[i] = key < p.E ? row : ~row;
      // The first of each key's lanes moves it on; the wave's LDS accesses
      // are in order, so every lane has read it.
      asm volatile("" ::: "memory");
      if (rank == 0) mine[key] = at + __popcll(same);
    }
    asm volatile("" ::: "memory");
  }
}

// --------------------------------------------------------- rows and tokens

template <typename T> struct Chunk;                       // 16 bytes of a row
template <> struct Chunk<bf16> {
  static constexpr int kN = 8;
  __device__ static void get(const u32x4& v, float (&f)[8]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      f[2 * q] = bits_f32(v[q] << 16);
      f[2 * q + 1] = bits_f32(v[q] & 0xFFFF0000u);
    }
  }
  __device__ static u32x4 put(const float (&f)[8]) {
    u32x4 v;
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = __builtin_bit_cast(uint32_t, bf16x2{to_bf16(f[2 * q]), to_bf16(f[2 * q + 1])});
    return v;
  }
};
template <> struct Chunk<float> {
  static constexpr int kN = 4;
  __device__ static void get(const u32x4& v, float (&f)[4]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) f[q] = bits_f32(v[q]);
  }
  __device__ static u32x4 put(const float (&f)[4]) {
    return u32x4{f32_bits(f[0]), f32_bits(f[1]), f32_bits(f[2]), f32_bits(f[3])};
  }
};

constexpr int kRowThreads = 256;

template <typename T>
__global__ __launch_bounds__(kRowThreads) void gather_kernel(int T_, int k, int nch, int per_row, const u32x4* x,
                                                             const int32_t* src, u32x4* out) {
  const int64_t task = (int64_t)blockIdx.x * (kRowThreads / 64) + (threadIdx.x >> 6);
  const int64_t r = task / per_row;
  if (r >= (int64_t)T_ * k) return;
  const int c = (int)(task % per_row) * 64 + (threadIdx.x & 63);
  if (c >= nch) return;
  const int pair = src[r];
  const int t = pair / k;
  u32x4 v = {0, 0, 0, 0};
  if (pair >= 0 && t < T_) v = x[(int64_t)t * nch + c];
  out[r * nch + c] = v;
}

// A wave: one token, 64 chunks of its columns.  The rows of kJ pairs are
// requested together.
template <typename T, int kJ>
__global__ __launch_bounds__(kRowThreads) void combine_kernel(CombineArgs p, int nch, int per_row) {
  constexpr int kN = Chunk<T>::kN;
  const int lane = threadIdx.x & 63;
  const int64_t task = (int64_t)blockIdx.x * (kRowThreads / 64) + (threadIdx.x >> 6);
  const int64_t t = task / per_row;
  if (t >= p.T) return;
  const int c = (int)(task % per_row) * 64 + lane;
  const int R = p.T * p.k;
  int mypos = -1;
  float myw = 0.0f;
  if (lane < p.k) {
    mypos = p.pos[t * p.k + lane];
    myw = p.weights != nullptr ? p.weights[t * p.k + lane] : 1.0f;
  }
  const u32x4* y = static_cast<const u32x4*>(p.y);
  float sum[kN];
#pragma unroll
  for (int q = 0; q < kN; ++q) sum[q] = 0.0f;
  for (int j0 = 0; j0 < p.k; j0 += kJ) {
    u32x4 v[kJ];
    bool on[kJ];
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      const int row = __builtin_amdgcn_readlane(mypos, (j0 + j) & 63);   // lanes past k hold -1
      on[j] = row >= 0 && row < R;
      v[j] = u32x4{0, 0, 0, 0};
      if (on[j] && c < nch) v[j] = y[(int64_t)row * nch + c];
    }
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      const float w = bits_f32(__builtin_amdgcn_readlane(f32_bits(myw), (j0 + j) & 63));
      if (on[j]) {
        float f[kN];
        Chunk<T>::get(v[j], f);
#pragma unroll
        for (int q = 0; q < kN; ++q) sum[q] = __builtin_fmaf(w, f[q], sum[q]);
      }
    }
  }
  if (c < nch) static_cast<u32x4*>(p.out)[t * nch + c] = Chunk<T>::put(sum);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// One token to kWaves waves (1, or 4: a workgroup, whose sums meet in LDS).
// A dropped pair (pos = ~row) has zeros: its row's gradient and its weight's.
template <typename T, int kWaves, int kJ>
__global__ __launch_bounds__(kRowThreads) void combine_bwd_kernel(CombineArgs p, int nch) {
  constexpr int kN = Chunk<T>::kN;
  __shared__ float part[kWaves > 1 ? kWaves : 1][kJ];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * (kRowThreads / 64 / kWaves) + (kWaves > 1 ? 0 : wave);
  if (t >= p.T) return;
  const int R = p.T * p.k;
  const u32x4* y = static_cast<const u32x4*>(p.y);
  const u32x4* dy = static_cast<const u32x4*>(p.dy) + t * nch;
  u32x4* dyr = static_cast<u32x4*>(p.dyr);
  int mypos = 0;
  float myw = 0.0f;
  if (lane < p.k) {
    mypos = p.pos[t * p.k + lane];
    myw = p.weights != nullptr ? p.weights[t * p.k + lane] : 1.0f;
  }
  for (int j0 = 0; j0 < p.k; j0 += kJ) {
    float dot[kJ], weight[kJ];
    int row[kJ];
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      dot[j] = 0.0f;
      row[j] = __builtin_amdgcn_readlane(mypos, (j0 + j) & 63);
      weight[j] = bits_f32(__builtin_amdgcn_readlane(f32_bits(myw), (j0 + j) & 63));
    }
    for (int c = (kWaves > 1 ? wave * 64 : 0) + lane; c < nch; c += 64 * kWaves) {
      u32x4 v[kJ];
      const u32x4 d4 = dy[c];
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        v[j] = u32x4{0, 0, 0, 0};
        if (j0 + j < p.k && row[j] >= 0 && row[j] < R) v[j] = y[(int64_t)row[j] * nch + c];
      }
      float d[kN];
      Chunk<T>::get(d4, d);
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        if (j0 + j >= p.k) continue;
        const bool live = row[j] >= 0;
        const int to = live ? row[j] : ~row[j];
        if (to >= R) continue;
        float f[kN], o[kN];
        Chunk<T>::get(v[j], f);
#pragma unroll
        for (int q = 0; q < kN; ++q) {
          dot[j] = __builtin_fmaf(d[q], f[q], dot[j]);
          o[q] = live ? weight[j] * d[q] : 0.0f;
        }
        if (!live) dot[j] = 0.0f;
        dyr[(int64_t)to * nch + c] = Chunk<T>::put(o);
      }
    }
#pragma unroll
    for (int j = 0; j < kJ; ++j) dot[j] = wave_sum(dot[j]);
    if constexpr (kWaves > 1) {
      if (lane == 0)
#pragma unroll
        for (int j = 0; j < kJ; ++j) part[wave][j] = dot[j];
      __syncthreads();
      if (wave == 0 && lane < kJ && j0 + lane < p.k && p.dweights != nullptr) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) s += part[w][lane];
        p.dweights[t * p.k + j0 + lane] = s;
      }
      __syncthreads();
    } else if (p.dweights != nullptr) {
#pragma unroll
      for (int j = 0; j < kJ; ++j)
        if (lane == j && j0 + j < p.k) p.dweights[t * p.k + j0 + j] = dot[j];
    }
  }
}

template <typename T>
hipError_t gather_t(int T_, int k, int K, const void* x, const int32_t* src, void* out, hipStream_t s) {
  const int nch = K / Chunk<T>::kN, per_row = (nch + 63) / 64;
  const int64_t blocks = ((int64_t)T_ * k * per_row + kRowThreads / 64 - 1) / (kRowThreads / 64);
  if (blocks == 0) return hipSuccess;
  hipLaunchKernelGGL((gather_kernel<T>), dim3((unsigned)blocks), dim3(kRowThreads), 0, s, T_, k, nch, per_row,
                     static_cast<const u32x4*>(x), src, static_cast<u32x4*>(out));
  return hipGetLastError();
}

template <typename T, int kJ>
hipError_t combine_t(const CombineArgs& a, hipStream_t s) {
  const int nch = a.K / Chunk<T>::kN, per_row = (nch + 63) / 64;
  const int64_t blocks = ((int64_t)a.T * per_row + kRowThreads / 64 - 1) / (kRowThreads / 64);
  hipLaunchKernelGGL((combine_kernel<T, kJ>), dim3((unsigned)blocks), dim3(kRowThreads), 0, s, a, nch, per_row);
  return hipGetLastError();
}

template <typename T, int kJ>
hipError_t combine_bwd_t(const CombineArgs& a, hipStream_t s) {
  const int nch = a.K / Chunk<T>::kN;
  if (nch <= 64)
    hipLaunchKernelGGL((combine_bwd_kernel<T, 1, kJ>), dim3((unsigned)((a.T + 3) / 4)), dim3(kRowThreads), 0, s, a, nch);
  else
    hipLaunchKernelGGL((combine_bwd_kernel<T, 4, kJ>), dim3((unsigned)a.T), dim3(kRowThreads), 0, s, a, nch);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_plan(const PlanArgs& a, hipStream_t s) {
  const int blocks = plan_blocks(a.n);
  const int per_block = plan_per_block(a.n);
  const size_t lds = (size_t)(kPlanWaves + 2) * (a.E + 1) * 4;
  hipError_t e = allow_lds<&plan_kernel<false>>((size_t)(kPlanWaves + 2) * (SWIGLU_MAX_EXPERTS + 1) * 4);
  if (e != hipSuccess) return e;
  if (blocks > 1) {
    e = allow_lds<&plan_kernel<true>>((size_t)(kPlanWaves + 2) * (SWIGLU_MAX_EXPERTS + 1) * 4);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((plan_kernel<true>), dim3(blocks), dim3(kPlanThreads), lds, s, a, per_block);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  hipLaunchKernelGGL((plan_kernel<false>), dim3(blocks), dim3(kPlanThreads), lds, s, a, per_block);
  return hipGetLastError();
}

hipError_t launch_gather(Dt dt, int T, int k, int K, const void* x, const int32_t* src, void* out, hipStream_t s) {
  return dt == Dt::kBF16 ? gather_t<bf16>(T, k, K, x, src, out, s) : gather_t<float>(T, k, K, x, src, out, s);
}

// Rows requested together: all of a token's up to 8.
hipError_t launch_combine(Dt dt, const CombineArgs& a, hipStream_t s) {
  if (dt == Dt::kBF16)
    return a.k <= 1 ? combine_t<bf16, 1>(a, s) : a.k <= 2 ? combine_t<bf16, 2>(a, s)
         : a.k <= 4 ? combine_t<bf16, 4>(a, s) : combine_t<bf16, 8>(a, s);
  return a.k <= 1 ? combine_t<float, 1>(a, s) : a.k <= 2 ? combine_t<float, 2>(a, s)
       : a.k <= 4 ? combine_t<float, 4>(a, s) : combine_t<float, 8>(a, s);
}

hipError_t launch_combine_bwd(Dt dt, const CombineArgs& a, hipStream_t s) {
  if (dt == Dt::kBF16)
    return a.k <= 1 ? combine_bwd_t<bf16, 1>(a, s) : a.k <= 2 ? combine_bwd_t<bf16, 2>(a, s)
         : a.k <= 4 ? combine_bwd_t<bf16, 4>(a, s) : combine_bwd_t<bf16, 8>(a, s);
  return a.k <= 1 ? combine_bwd_t<float, 1>(a, s) : a.k <= 2 ? combine_bwd_t<float, 2>(a, s)
       : a.k <= 4 ? combine_bwd_t<float, 4>(a, s) : combine_bwd_t<float, 8>(a, s);
}

}  // namespace swg
