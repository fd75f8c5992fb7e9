// Pieces shared by the matrix-core kernels: tile shapes, MFMA forms and their
// accumulator layouts, LDS-DMA helpers.
#pragma once

#include "common.hpp"

namespace swg {

// Block tile kBM x kBN (rows of A x rows of each B), waves in a kWGM x kWGN
// grid, each wave owning (kBM / kWGM) x (kBN / kWGN) of every B operand.
template <int BM_, int BN_, int WGM_, int WGN_, int OCC_ = 0>
struct Tile {
  static constexpr int kBM = BM_, kBN = BN_, kWGM = WGM_, kWGN = WGN_;
  static constexpr int kThreads = 64 * WGM_ * WGN_;
  // Waves per SIMD the register budget is sized for (default: one workgroup per CU).
  static constexpr int kOcc = OCC_ > 0 ? OCC_ : kThreads / 256;
  static constexpr int kWM = BM_ / WGM_, kWN = BN_ / WGN_;   // wave tile
};

template <typename T> struct Mma;

template <> struct Mma<bf16> {
  static constexpr int kPerChunk = 8;
  __device__ __forceinline__ static void run(f32x16& acc, const u32x4& a, const u32x4& b) {
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                  __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
  }
};

template <> struct Mma<float> {
  static constexpr int kPerChunk = 4;
  __device__ __forceinline__ static void run(f32x16& acc, const u32x4& a, const u32x4& b) {
#pragma unroll
    for (int t = 0; t < 4; ++t)
      acc = __builtin_amdgcn_mfma_f32_32x32x2f32(bits_f32(a[t]), bits_f32(b[t]), acc, 0, 0, 0);
  }
};

// MFMA accumulator layouts.  kMN = 32 (v_mfma_f32_32x32x*): 16 floats per
// lane, lane l element e at row 8 (e >> 2) + 4 (l >> 5) + (e & 3), column
// l & 31.  kMN = 16 (v_mfma_f32_16x16x32_bf16): 4 floats per lane, lane l
// element e at row 4 (l >> 4) + e, column l & 15.  In both, elements 4q ..
// 4q + 3 are 4 consecutive rows of one column, and the 16 lanes of a group
// hold one 16-column run of those rows.
template <int kMN> struct AccL;
template <> struct AccL<32> {
  using V = f32x16;
  static constexpr int kE = 16;
  __device__ __forceinline__ static int row(int lane, int e) { return 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3); }
  __device__ __forceinline__ static int col(int lane) { return lane & 31; }
};
template <> struct AccL<16> {
  using V = f32x4;
  static constexpr int kE = 4;
  __device__ __forceinline__ static int row(int lane, int e) { return 4 * (lane >> 4) + e; }
  __device__ __forceinline__ static int col(int lane) { return lane & 15; }
};

template <typename T> __device__ __forceinline__ T cvt_out(float v);
template <> __device__ __forceinline__ bf16 cvt_out<bf16>(float v) { return to_bf16(v); }
template <> __device__ __forceinline__ float cvt_out<float>(float v) { return v; }

template <typename T> __device__ __forceinline__ float load_in(const T* p);
template <> __device__ __forceinline__ float load_in<bf16>(const bf16* p) { return from_bf16(*p); }
template <> __device__ __forceinline__ float load_in<float>(const float* p) { return *p; }

typedef __attribute__((ext_vector_type(4))) short short4_t;
typedef __attribute__((address_space(3))) short4_t lds_short4_t;
typedef __attribute__((address_space(3))) char lds_char_t;

// s_waitcnt that only bounds the vector-memory counter (gfx9 encoding:
// vmcnt in bits [3:0] and [15:14]; expcnt [6:4] and lgkmcnt [11:8] left at
// their maxima).  The LDS DMA loads below count as vector-memory operations.
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

typedef __attribute__((address_space(3))) void lds_void_t;

// Raw buffer descriptor over [base, base + bytes): reads past the end return
// zero.  Every field goes through readfirstlane so the descriptor is known to
// be wave-uniform and lives in scalar registers (a descriptor the compiler
// thinks divergent turns each buffer access into a waterfall loop).
template <typename T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t uniform_rsrc(const T* base, int64_t bytes) {
  const uint64_t bp = reinterpret_cast<uint64_t>(base);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)bp);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(bp >> 32));
  const int n = __builtin_amdgcn_readfirstlane((int)bytes);
  void* ub = reinterpret_cast<void*>(((uint64_t)hi << 32) | lo);
  return __builtin_amdgcn_make_buffer_rsrc(ub, (short)0, n, 0x00020000);
}

// Workgroup barrier without the memory fence of __syncthreads (which waits
// for every outstanding vector-memory operation, i.e. would drain the DMA
// ring).  Each wave has already waited for its own DMA of the step with
// wait_vmcnt; the empty asm statements keep the compiler from moving LDS
// accesses across the barrier.
__device__ __forceinline__ void barrier_no_fence() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

}  // namespace swg
