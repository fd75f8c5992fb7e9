// The norm of many gradients together, and their clipping.
//
//   norm = sqrt(sum over all elements of g^2)
//   g   <- g * min(1, max_norm / (norm + eps))
//
// The tensors' addresses and sizes are kernel arguments (a table of up to
// kClipNormTensors or kClipScaleTensors of them to a launch), so nothing is
// copied to the device and a captured call replays by itself.  A workgroup
// takes chunks of 32 KiB in turn, a chunk of one tensor, found by a binary
// search over the tensors' first chunks.  Squares are formed and added in
// fp64 (exact products of the inputs, no overflow or underflow for any fp32
// value); every workgroup writes its sum to a place of its own and one
// workgroup adds them, all in a fixed order.  The scaling pass reads the
// factor that this leaves in memory and ends at once where it is 1 and the
// gradients stay where they are: a step under the limit reads them once.
//
// HBM bounds the kernels of large lists: 345 MB of bf16 into other tensors take
// 58 us (5.9 TB/s; the fp64 squares cost nothing beside it, sums in fp32 take as
// long) and 109 us (6.3 TB/s); in place 166 us together, under the limit 61.  Lists of many small tensors are bound by the host,
// which reads each tensor's address, size, type and layout: 420 tensors 130 us,
// of which the kernels run 25.
#include "common.hpp"
#include "grouped.hpp"
#include "validate.hpp"

namespace swg {

namespace {

constexpr int kThreads = 256;

// Addresses have 48 bits: a tensor's address and where it ends in its last
// chunk, less one, in one word.
template <int kTensors, bool kOut>
struct Table {
  uint64_t at[kTensors];
  uint64_t to[kOut ? kTensors : 1];
  uint32_t first[kTensors + 1];       // first chunk of each tensor; behind the last: all chunks
  int count;
};
static_assert(sizeof(Table<kClipNormTensors, false>) <= 4096 - 64, "kernel arguments");
static_assert(sizeof(Table<kClipScaleTensors, true>) <= 4096 - 64, "kernel arguments");

template <typename T> constexpr int64_t kChunk = kClipChunkBytes / (int64_t)sizeof(T);

template <typename T> struct Elems;
template <> struct Elems<bf16> {
  static constexpr int kN = 8;
  __device__ static float get(const u32x4& v, int i) {
    return bits_f32((i & 1) ? v[i >> 1] & 0xFFFF0000u : v[i >> 1] << 16);
  }
};
template <> struct Elems<float> {
  static constexpr int kN = 4;
  __device__ static float get(const u32x4& v, int i) { return bits_f32(v[i]); }
};

// Addresses out of the table's words, known to be global memory's; 16 bytes
// at any element boundary.
typedef __attribute__((address_space(1))) char global_char;
typedef u32x4 piece_t __attribute__((aligned(2)));
typedef __attribute__((address_space(1))) piece_t global_piece;
__device__ __forceinline__ u32x4 load16(const global_char* p) { return *(const global_piece*)p; }
__device__ __forceinline__ void store16(global_char* p, const u32x4& v) { *(global_piece*)p = v; }
__device__ __forceinline__ u32x4 stream16(const global_char* p) {
  return __builtin_nontemporal_load((const global_piece*)p);
}
__device__ __forceinline__ void stream16(global_char* p, const u32x4& v) {
  __builtin_nontemporal_store((piece_t)v, (global_piece*)p);
}
__device__ __forceinline__ float load1(bf16, const global_char* p) {
  return bits_f32((uint32_t) * (const __attribute__((address_space(1))) uint16_t*)p << 16);
}
__device__ __forceinline__ float load1(float, const global_char* p) {
  return *(const __attribute__((address_space(1))) float*)p;
}
__device__ __forceinline__ void store1(bf16, global_char* p, float v) {
  *(__attribute__((address_space(1))) uint16_t*)p = __builtin_bit_cast(uint16_t, to_bf16(v));
}
__device__ __forceinline__ void store1(float, global_char* p, float v) {
  *(__attribute__((address_space(1))) float*)p = v;
}

template <class Tab>
__device__ __forceinline__ int tensor_of(const Tab& t, uint32_t chunk) {
  int lo = 0, hi = t.count - 1;                           // the last tensor whose first chunk is not past it
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// A chunk: 32 KiB of memory from a 16-byte boundary on, of which the elements
// lo .. hi - 1 are its tensor's (all of them but in a tensor's first and last
// chunk).  Chunks start on 16 bytes wherever their tensor does: loads of
// views that start at odd elements took 15 % longer.
struct Chunk {
  uint64_t at;       // address of element 0
  int64_t element;   // its number in the tensor (negative in front of it)
  int tensor, lo, hi;
};
template <typename T, class Tab>
__device__ __forceinline__ Chunk chunk_of(const Tab& t, uint32_t c) {
  Chunk k;
  k.tensor = tensor_of(t, c);
  const uint64_t word = t.at[k.tensor], at = word >> 16;
  const uint32_t i = c - t.first[k.tensor];
  const int skip = (int)(at & 15) / (int)sizeof(T);
  k.at = (at & ~(uint64_t)15) + (uint64_t)i * kClipChunkBytes;
  k.element = (int64_t)i * kChunk<T> - skip;
  k.lo = i == 0 ? skip : 0;
  k.hi = c + 1 == t.first[k.tensor + 1] ? (int)(word & 0xFFFF) + 1 : (int)kChunk<T>;
  return k;
}

constexpr int kU = 8;                                     // 16-byte pieces of a whole chunk per thread
static_assert(kClipChunkBytes == (int64_t)kU * kThreads * 16, "a chunk is kU pieces per thread");

// The pieces of a chunk that is not whole: f(piece) for its whole 16-byte
// pieces, g(element) for the few elements in front of them and behind.
template <int kN, class P, class E>
__device__ __forceinline__ void ragged(const Chunk& k, P&& piece, E&& element) {
  const int tid = threadIdx.x, p0 = (k.lo + kN - 1) / kN, p1 = k.hi / kN;
  for (int u = p0 + tid; u < p1; u += kThreads) piece(u);
  const int head = p0 * kN < k.hi ? p0 * kN : k.hi;       // elements lo .. head - 1
  const int tail = p1 * kN > head ? p1 * kN : head;       // elements tail .. hi - 1
  if (k.lo + tid < head) element(k.lo + tid);
  if (tail + tid < k.hi) element(tail + tid);
}

template <typename T>
__global__ __launch_bounds__(kThreads) void norm_kernel(Table<kClipNormTensors, false> t, double* part) {
  constexpr int kN = Elems<T>::kN;
  const int tid = threadIdx.x;
  const uint32_t chunks = t.first[t.count];
  double acc[4] = {0.0, 0.0, 0.0, 0.0};
  auto add = [&](const u32x4& v) {
#pragma unroll
    for (int q = 0; q < kN; ++q) {
      const double d = (double)Elems<T>::get(v, q);
      acc[q & 3] = __builtin_fma(d, d, acc[q & 3]);
    }
  };
  Chunk next = chunk_of<T>(t, blockIdx.x);
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const Chunk k = next;
    const global_char* g = (const global_char*)k.at;
    const uint32_t after = c + gridDim.x < chunks ? c + gridDim.x : c;
    if (k.lo == 0 && k.hi == (int)kChunk<T>) {
      u32x4 v[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) v[u] = load16(g + (u * kThreads + tid) * 16);
      next = chunk_of<T>(t, after);                       // while the loads are on their way
#pragma unroll
      for (int u = 0; u < kU; ++u) add(v[u]);
    } else {
      next = chunk_of<T>(t, after);
      ragged<kN>(k, [&](int u) { add(load16(g + u * 16)); },
                 [&](int e) {
                   const double d = (double)load1(T{}, g + e * (int)sizeof(T));
                   acc[0] = __builtin_fma(d, d, acc[0]);
                 });
    }
  }
  double s = (acc[0] + acc[1]) + (acc[2] + acc[3]);
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d);
  __shared__ double wave[kThreads / 64];
  if ((tid & 63) == 0) wave[tid >> 6] = s;
  __syncthreads();
  if (tid == 0) part[blockIdx.x] = (wave[0] + wave[1]) + (wave[2] + wave[3]);
}

// One workgroup: the norm and, where factor is asked for, the factor.
constexpr int kTotalThreads = 1024;
__global__ __launch_bounds__(kTotalThreads) void total_kernel(const double* part, int n, double max_norm, double eps,
                                                              float* norm, float* factor) {
  const int tid = threadIdx.x;
  double s = 0.0;
  for (int i = tid; i < n; i += kTotalThreads) s += part[i];
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d);
  __shared__ double wave[kTotalThreads / 64];
  if ((tid & 63) == 0) wave[tid >> 6] = s;
  __syncthreads();
  if (tid == 0) {
    double all = 0.0;
    for (int w = 0; w < kTotalThreads / 64; ++w) all += wave[w];
    const double r = sqrt(all);
    *norm = (float)r;
    if (factor != nullptr) {
      // No quotient where the limit is infinite (nothing is clipped, also at an
      // infinite norm) or r + eps is 0 (only zeros there); a NaN stays one.
      const bool none = (__builtin_isinf(max_norm) || r + eps == 0.0) && r == r;
      const double f = none ? 1.0 : max_norm / (r + eps);
      *factor = f > 1.0 ? 1.0f : (float)f;
    }
  }
}

template <typename T> __device__ __forceinline__ u32x4 scaled(const u32x4& v, float f) {
  u32x4 o;
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      o[q] = __builtin_bit_cast(uint32_t, bf16x2{to_bf16(f * bits_f32(v[q] << 16)), to_bf16(f * bits_f32(v[q] & 0xFFFF0000u))});
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = f32_bits(f * bits_f32(v[q]));
  }
  return o;
}

// kStream: past the caches (results beside the gradients, both together more
// than the caches hold).
template <typename T, class Tab, bool kOut, bool kStream>
__global__ __launch_bounds__(kThreads) void scale_kernel(Tab t, const float* factor) {
  constexpr int kN = Elems<T>::kN;
  const float f = *factor;
  if (!kOut && f == 1.0f) return;
  const int tid = threadIdx.x;
  const uint32_t chunks = t.first[t.count];
  // From the last chunk back: what the norm's pass read last is still in the
  // memory-side cache (256 MB).
  Chunk next = chunk_of<T>(t, chunks - 1 - blockIdx.x);
  for (uint32_t b = blockIdx.x; b < chunks; b += gridDim.x) {
    const Chunk k = next;
    const global_char* g = (const global_char*)k.at;
    global_char* o = kOut ? (global_char*)(t.to[k.tensor] + (uint64_t)(k.element * (int64_t)sizeof(T))) : (global_char*)k.at;
    const uint32_t after = chunks - 1 - (b + gridDim.x < chunks ? b + gridDim.x : b);
    if (k.lo == 0 && k.hi == (int)kChunk<T>) {
      u32x4 v[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        if constexpr (kStream) v[u] = stream16(g + (u * kThreads + tid) * 16);
        else v[u] = load16(g + (u * kThreads + tid) * 16);
      }
      next = chunk_of<T>(t, after);
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        if constexpr (kStream) stream16(o + (u * kThreads + tid) * 16, scaled<T>(v[u], f));
        else store16(o + (u * kThreads + tid) * 16, scaled<T>(v[u], f));
      }
    } else {
      next = chunk_of<T>(t, after);
      ragged<kN>(k, [&](int u) { store16(o + u * 16, scaled<T>(load16(g + u * 16), f)); },
                 [&](int e) {
                   const int at = e * (int)sizeof(T);
                   store1(T{}, o + at, f * load1(T{}, g + at));
                 });
    }
  }
}

template <typename T, class Tab>
uint32_t fill(Tab& t, const GradSpan* spans, int count, bool out) {
  uint32_t chunks = 0;
  for (int i = 0; i < count; ++i) {
    const int64_t end = spans[i].n + (int64_t)((reinterpret_cast<uint64_t>(spans[i].g) & 15) / sizeof(T));
    const int64_t n = (end + kChunk<T> - 1) / kChunk<T>;
    const int64_t tail = end - (n - 1) * kChunk<T>;
    t.at[i] = (reinterpret_cast<uint64_t>(spans[i].g) << 16) | (uint64_t)(tail - 1);
    if (out) t.to[i] = reinterpret_cast<uint64_t>(spans[i].out);
    t.first[i] = chunks;
    chunks += (uint32_t)n;
  }
  t.first[count] = chunks;
  t.count = count;
  return chunks;
}

template <typename T>
hipError_t norm_t(const GradSpan* spans, int count, int* blocks, double* part, hipStream_t s) {
  Table<kClipNormTensors, false> t;
  const uint32_t chunks = fill<T>(t, spans, count, false);
  *blocks = chunks < (uint32_t)kClipBlocks ? (int)chunks : kClipBlocks;
  hipLaunchKernelGGL((norm_kernel<T>), dim3(*blocks), dim3(kThreads), 0, s, t, part);
  return hipGetLastError();
}

// Results of more than 160 MB go past the memory-side cache: left there, half
// of them would still have to be written while the next kernel reads.  Norm and
// scaling together, results past the caches and not: 120 MB 62.7 and 61.2 us,
// 160 81.2 and 81.9, 345 169 and 202, 1024 538 and 578; with a reader of the
// results behind them 88 and 84, 113 and 114, 231 and 274, 714 and 762.
constexpr uint32_t kStreamChunks = 160u * 1024 * 1024 / kClipChunkBytes;

template <typename T, bool kOut, int kTensors>
hipError_t scale_t(const GradSpan* spans, int count, const float* factor, hipStream_t s) {
  using Tab = Table<kTensors, kOut>;
  Tab t;
  const uint32_t chunks = fill<T>(t, spans, count, kOut);
  const unsigned blocks = chunks < 2u * kClipBlocks ? chunks : 2u * kClipBlocks;
  if constexpr (kOut)
    if (chunks > kStreamChunks) {
      hipLaunchKernelGGL((scale_kernel<T, Tab, kOut, true>), dim3(blocks), dim3(kThreads), 0, s, t, factor);
      return hipGetLastError();
    }
  hipLaunchKernelGGL((scale_kernel<T, Tab, kOut, false>), dim3(blocks), dim3(kThreads), 0, s, t, factor);
  return hipGetLastError();
}

// The spans of one type in runs of at most `most`, in the order given.
template <class F>
hipError_t for_runs(Dt dt, int64_t count, const int* dtypes, const void* const* grads, const int64_t* sizes,
                    void* const* outs, int most, F&& f) {
  GradSpan run[kClipNormTensors];
  int n = 0;
  hipError_t e = hipSuccess;
  for (int64_t i = 0; i < count && e == hipSuccess; ++i) {
    if (sizes[i] == 0 || dtypes[i] != (dt == Dt::kBF16 ? SWIGLU_BF16 : SWIGLU_F32)) continue;
    run[n++] = GradSpan{grads[i], outs != nullptr ? outs[i] : const_cast<void*>(grads[i]), sizes[i]};
    if (n == most) {
      e = f(run, n);
      n = 0;
    }
  }
  if (n > 0 && e == hipSuccess) e = f(run, n);
  return e;
}

}  // namespace

hipError_t launch_clip(const ClipArgs& a, hipStream_t s) {
  int parts = 0;
  hipError_t e = hipSuccess;
  for (Dt dt : {Dt::kBF16, Dt::kF32}) {
    e = for_runs(dt, a.count, a.dtypes, a.grads, a.sizes, nullptr, kClipNormTensors, [&](const GradSpan* r, int n) {
      int blocks = 0;
      const hipError_t err = dt == Dt::kBF16 ? norm_t<bf16>(r, n, &blocks, a.part + parts, s)
                                             : norm_t<float>(r, n, &blocks, a.part + parts, s);
      parts += blocks;
      return err;
    });
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(total_kernel, dim3(1), dim3(kTotalThreads), 0, s, a.part, parts, a.max_norm, a.eps, a.norm,
                     a.clip ? a.factor : nullptr);
  if ((e = hipGetLastError()) != hipSuccess || !a.clip) return e;
  for (Dt dt : {Dt::kBF16, Dt::kF32}) {
    const bool b16 = dt == Dt::kBF16;
    if (a.outs != nullptr)
      e = for_runs(dt, a.count, a.dtypes, a.grads, a.sizes, a.outs, kClipScaleTensors, [&](const GradSpan* r, int n) {
        return b16 ? scale_t<bf16, true, kClipScaleTensors>(r, n, a.factor, s)
                   : scale_t<float, true, kClipScaleTensors>(r, n, a.factor, s);
      });
    else
      e = for_runs(dt, a.count, a.dtypes, a.grads, a.sizes, nullptr, kClipNormTensors, [&](const GradSpan* r, int n) {
        return b16 ? scale_t<bf16, false, kClipNormTensors>(r, n, a.factor, s)
                   : scale_t<float, false, kClipNormTensors>(r, n, a.factor, s);
      });
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace swg
