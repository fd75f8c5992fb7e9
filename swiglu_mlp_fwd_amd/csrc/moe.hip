// The routed SwiGLU MLP for a few tokens (bf16, at most 64):
//   y[t] = sum_j w[t, j] * Wd_e (act(Wg_e x[t]) * (Wu_e x[t])),  e = ids[t, j].
//
// The work is bound by reading the touched experts' weights from HBM once,
// as the dense decode kernel's (gemv.hip), so both products stream weights
// the same way: a workgroup owns 16 weight rows of one expert, its 8 waves
// split the reduction into slabs of 128 and load the weights coalesced
// (256 contiguous bytes of a row per quarter-wave), pass them through a
// wave-private LDS tile into the operand layout of v_mfma_f32_16x16x32_bf16,
// and multiply them with up to 16 kG of the expert's tokens at once; the
// waves' partial sums meet in LDS and are added in wave order.
//
// moe_up:    h of each (token, expert) pair, kept as two bf16 (h = hi + lo,
//            16 significant bits), the second product's operands.
// moe_down:  Wd_e (hi + lo), two products into one accumulator, to
//            part[pair] in fp32.
// moe_sum:   y = sum_j w_j part, in order of j, rounded once.
//
// A grid slice (blockIdx.y) is the slot of an expert in use: every workgroup
// finds its expert and the pairs that name it from ids (at most 1024).
#include "block.hpp"
#include "common.hpp"

namespace swg {

namespace {

constexpr int kWaves = 8;
constexpr int kThreads = kWaves * 64;
constexpr int kSlabK = 128;                      // reduction elements per slab
constexpr int kCPR = kSlabK / 8;                 // 16-byte chunks per row per slab
constexpr int kRowsPerInst = 64 / kCPR;          // rows one load instruction covers
constexpr int kInst = 16 / kRowsPerInst;         // load instructions per slab of 16 rows
constexpr int kSteps = kSlabK / 32;              // MFMA steps per slab
constexpr int kTile = 16 * kCPR;                 // 16-byte chunks of a slab of 16 rows
constexpr int kMaxPairs = 64 * 16;
static_assert(kMaxPairs <= 2 * kThreads, "two ids per thread cover every pair");

// The pairs (t k + j, in increasing order) that name the slot-th expert in
// use, in order of expert.
struct Found {
  uint32_t mask[32];
  int wave_count[2][kWaves];
  uint16_t list[kMaxPairs];
};

// Returns the expert (-1: fewer than slot + 1 are in use) and sets n.
__device__ __forceinline__ int find_pairs(Found& f, const int32_t* __restrict__ ids, int pairs, int E, int slot,
                                          int tid, int& n) {
  const int lane = tid & 63, wave = tid >> 6;
  if (tid < 32) f.mask[tid] = 0;
  __syncthreads();
  int id[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int p = tid + i * kThreads;
    id[i] = p < pairs ? ids[p] : -1;
    if (id[i] >= 0 && id[i] < E) atomicOr(&f.mask[id[i] >> 5], 1u << (id[i] & 31));
  }
  __syncthreads();
  // Every wave: lane w < 32 holds mask word w; the word of the slot-th set bit.
  uint32_t m = lane < 32 ? f.mask[lane] : 0u;
  const int c = __popc(m);
  int before = c;                                // inclusive prefix sum
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up(before, off);
    if (lane >= off) before += o;
  }
  before -= c;
  const uint64_t has = __ballot(lane < 32 && slot >= before && slot < before + c);
  if (has == 0) return -1;
  const int word = __ffsll((unsigned long long)has) - 1;
  m = __shfl(m, word);
  for (int i = slot - __shfl(before, word); i > 0; --i) m &= m - 1;
  const int expert = word * 32 + __ffs(m) - 1;
  uint64_t hit[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    hit[i] = __ballot(id[i] == expert);
    if (lane == 0) f.wave_count[i][wave] = __popcll(hit[i]);
  }
  __syncthreads();
  n = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    for (int w = 0; w < kWaves; ++w) {
      if (w == wave && id[i] == expert)
        f.list[n + __popcll(hit[i] & ((1ull << lane) - 1))] = (uint16_t)(tid + i * kThreads);
      n += f.wave_count[i][w];
    }
  __syncthreads();
  return expert;
}

// One pass of 16 rows (n0 ..) of kW weights over the tokens of one group of
// 16 kG pairs: acc[w][g] in the MFMA's layout, summed over the workgroup's
// waves, in the registers of wave g (of the waves g < kG).
//   w4[i]    weight i, row r at w4[i] + r * nch chunks; rows past `rows` read as zero
//   b4[i]    kB token operands (their products add up), token row r16 of group g
//            at b4[i] + brow[g] * nch, absent (zero) where brow[g] < 0
template <int kW, int kB, int kG>
__device__ __forceinline__ void stream_rows(u32x4* lds, const u32x4* const (&w4)[kW], const u32x4* const (&b4)[kB],
                                            const int (&brow)[kG], int n0, int rows, int nch, int tid,
                                            f32x4 (&acc)[kW][kG]) {
  const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nslab = (nch + kCPR - 1) / kCPR;
  const int s0 = (int)((int64_t)wave * nslab / kWaves), s1 = (int)((int64_t)(wave + 1) * nslab / kWaves);
  u32x4* tile = lds + wave * kW * kTile;
  const int lc = lane % kCPR, lr = lane / kCPR;
  const int r16 = lane & 15, q4 = lane >> 4;
  const u32x4 zero = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int w = 0; w < kW; ++w)
#pragma unroll
    for (int g = 0; g < kG; ++g) acc[w][g] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int s = s0; s < s1; ++s) {
    const int c = s * kCPR + lc;
    u32x4 v[kW][kInst];
#pragma unroll
    for (int i = 0; i < kInst; ++i) {
      const int n = n0 + i * kRowsPerInst + lr;
      const bool in = n < rows && c < nch;
      const int64_t off = in ? (int64_t)n * nch + c : 0;
#pragma unroll
      for (int w = 0; w < kW; ++w) v[w][i] = in ? __builtin_nontemporal_load(w4[w] + off) : zero;
    }
    // Row r, chunk c of a tile sits at chunk c ^ (r & 15): see gemv.hip.
#pragma unroll
    for (int i = 0; i < kInst; ++i) {
      const int r = i * kRowsPerInst + lr;
#pragma unroll
      for (int w = 0; w < kW; ++w) tile[w * kTile + r * kCPR + (lc ^ r)] = v[w][i];
    }
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      const int pc = (4 * j + q4) ^ r16;
      const int cb = s * kCPR + 4 * j + q4;
#pragma unroll
      for (int g = 0; g < kG; ++g) {
#pragma unroll
        for (int b = 0; b < kB; ++b) {
          const bool in = brow[g] >= 0 && cb < nch;
          const u32x4 xv = in ? b4[b][(int64_t)brow[g] * nch + cb] : zero;
#pragma unroll
          for (int w = 0; w < kW; ++w)
            acc[w][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                __builtin_bit_cast(bf16x8, tile[w * kTile + r16 * kCPR + pc]), __builtin_bit_cast(bf16x8, xv),
                acc[w][g], 0, 0, 0);
        }
      }
    }
  }
  __syncthreads();                               // every wave is done with its tiles
  f32x4* red = reinterpret_cast<f32x4*>(lds);    // [kW][kG][wave][lane]
#pragma unroll
  for (int w = 0; w < kW; ++w)
#pragma unroll
    for (int g = 0; g < kG; ++g) red[((w * kG + g) * kWaves + wave) * 64 + lane] = acc[w][g];
  __syncthreads();
  if (wave < kG) {
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      f32x4 sum = red[((w * kG + wave) * kWaves) * 64 + lane];
      for (int o = 1; o < kWaves; ++o) sum += red[((w * kG + wave) * kWaves + o) * 64 + lane];
      acc[w][0] = sum;
    }
  }
}

constexpr size_t lds_bytes(int kW, int kG) {
  const size_t tiles = (size_t)kWaves * kW * kTile * 16, red = (size_t)kW * kG * kWaves * 64 * 16;
  return tiles > red ? tiles : red;
}

// This lane's token rows: token row r16 of group g is entry p0 + 16 g + r16
// of the list; -1 past its end.
template <int kG>
__device__ __forceinline__ void pair_rows(const Found& f, int p0, int n, int r16, int (&pair)[kG]) {
#pragma unroll
  for (int g = 0; g < kG; ++g) {
    const int i = p0 + 16 * g + r16;
    pair[g] = i < n ? (int)f.list[i] : -1;
  }
}

template <Act A, int kG>
__global__ __launch_bounds__(kThreads) void moe_up_kernel(MoeArgs a) {
  extern __shared__ u32x4 lds[];
  __shared__ Found found;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int n;
  const int e = find_pairs(found, a.ids, a.T * a.k, a.E, blockIdx.y, tid, n);
  if (e < 0) return;
  const int n0 = blockIdx.x * 16, nch = a.K >> 3;
  const u32x4* const w4[2] = {
      reinterpret_cast<const u32x4*>(static_cast<const bf16*>(a.wg) + e * a.wg_stride),
      reinterpret_cast<const u32x4*>(static_cast<const bf16*>(a.wu) + e * a.wu_stride)};
  const u32x4* const b4[1] = {static_cast<const u32x4*>(a.x)};
  for (int p0 = 0; p0 < n; p0 += 16 * kG) {
    int pair[kG], row[kG];
    pair_rows(found, p0, n, lane & 15, pair);
#pragma unroll
    for (int g = 0; g < kG; ++g) row[g] = pair[g] < 0 ? -1 : pair[g] / a.k;
    f32x4 acc[2][kG];
    stream_rows<2, 1, kG>(lds, w4, b4, row, n0, a.N, nch, tid, acc);
    // Lane l element i: weight row n0 + 4 (l / 16) + i of token row l % 16.
    const int i = p0 + 16 * wave + (lane & 15), nb = n0 + 4 * (lane >> 4);
    if (wave < kG && i < n && nb < a.N) {        // N % 8 == 0: four columns lie inside or outside together
      uint16_t hi[4], lo[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float g = acc[0][0][q];
        const float h = (A == Act::kGeluTanh ? gelu_tanh_f32(g) : silu_f32(g)) * acc[1][0][q];
        const bf16 b = to_bf16(h);
        const float f = from_bf16(b);
        hi[q] = __builtin_bit_cast(uint16_t, b);
        lo[q] = __builtin_bit_cast(uint16_t, to_bf16(fabsf(f) < __builtin_inff() ? h - f : 0.0f));
      }
      const int64_t at = (int64_t)found.list[i] * a.N + nb;
      *reinterpret_cast<u32x2*>(static_cast<bf16*>(a.h_hi) + at) = __builtin_bit_cast(u32x2, hi);
      *reinterpret_cast<u32x2*>(static_cast<bf16*>(a.h_lo) + at) = __builtin_bit_cast(u32x2, lo);
    }
    __syncthreads();                             // the sums are read before the next tiles are written
  }
}

template <int kG>
__global__ __launch_bounds__(kThreads) void moe_down_kernel(MoeArgs a) {
  extern __shared__ u32x4 lds[];
  __shared__ Found found;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int n;
  const int e = find_pairs(found, a.ids, a.T * a.k, a.E, blockIdx.y, tid, n);
  if (e < 0) return;
  const int n0 = blockIdx.x * 16, nch = a.N >> 3;
  const u32x4* const w4[1] = {reinterpret_cast<const u32x4*>(static_cast<const bf16*>(a.wd) + e * a.wd_stride)};
  const u32x4* const b4[2] = {static_cast<const u32x4*>(a.h_hi), static_cast<const u32x4*>(a.h_lo)};
  for (int p0 = 0; p0 < n; p0 += 16 * kG) {
    int pair[kG];
    pair_rows(found, p0, n, lane & 15, pair);
    f32x4 acc[1][kG];
    stream_rows<1, 2, kG>(lds, w4, b4, pair, n0, a.K, nch, tid, acc);
    const int i = p0 + 16 * wave + (lane & 15), nb = n0 + 4 * (lane >> 4);
    if (wave < kG && i < n && nb < a.K)
      *reinterpret_cast<f32x4*>(a.part + (int64_t)found.list[i] * a.K + nb) = acc[0][0];
    __syncthreads();
  }
}

// Thread: four columns of a token.
__global__ __launch_bounds__(256) void moe_sum_kernel(MoeArgs a) {
  const int c = (blockIdx.x * 256 + threadIdx.x) * 4, t = blockIdx.y;
  if (c >= a.K) return;
  f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int j = 0; j < a.k; ++j) {
    const int p = t * a.k + j, id = a.ids[p];
    if (id < 0 || id >= a.E) continue;
    const float w = a.weights[p];
    const f32x4 v = *reinterpret_cast<const f32x4*>(a.part + (int64_t)p * a.K + c);
#pragma unroll
    for (int q = 0; q < 4; ++q) y[q] = __builtin_fmaf(w, v[q], y[q]);
  }
  uint16_t o[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) o[q] = __builtin_bit_cast(uint16_t, to_bf16(y[q]));
  *reinterpret_cast<u32x2*>(static_cast<bf16*>(a.y) + (int64_t)t * a.K + c) = __builtin_bit_cast(u32x2, o);
}

template <Act A, int kG>
hipError_t launch_g(const MoeArgs& a, hipStream_t s) {
  const unsigned slots = (unsigned)(a.E < a.T * a.k ? a.E : a.T * a.k);
  constexpr size_t up_lds = lds_bytes(2, kG), down_lds = lds_bytes(1, kG);
  hipError_t e;
  if ((e = allow_lds<&moe_up_kernel<A, kG>>(up_lds)) != hipSuccess) return e;
  if ((e = allow_lds<&moe_down_kernel<kG>>(down_lds)) != hipSuccess) return e;
  hipLaunchKernelGGL((moe_up_kernel<A, kG>), dim3((a.N + 15) / 16, slots), dim3(kThreads), up_lds, s, a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  hipLaunchKernelGGL((moe_down_kernel<kG>), dim3((a.K + 15) / 16, slots), dim3(kThreads), down_lds, s, a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  hipLaunchKernelGGL(moe_sum_kernel, dim3((a.K + 1023) / 1024, a.T), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <Act A>
hipError_t launch_a(const MoeArgs& a, hipStream_t s) {
  if (a.T <= 16) return launch_g<A, 1>(a, s);
  if (a.T <= 32) return launch_g<A, 2>(a, s);
  return launch_g<A, 4>(a, s);
}

}  // namespace

hipError_t launch_moe(Act act, const MoeArgs& a, hipStream_t s) {
  return act == Act::kGeluTanh ? launch_a<Act::kGeluTanh>(a, s) : launch_a<Act::kSilu>(a, s);
}

}  // namespace swg
