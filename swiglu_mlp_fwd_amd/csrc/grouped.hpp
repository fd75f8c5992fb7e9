// Internal launch interface of the operators over rows in order of expert:
// their order, grouped products, combine and gradient clipping (not part of
// the ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm.hpp"

namespace swg {

// Rows lie in order of expert: those of expert e are offsets[e] up to
// offsets[e + 1] of R.  Rows of no expert are zero rows of every output that
// has a row for each of them.
struct GroupedArgs {
  const int32_t* offsets;   // [E + 1], device
  int E, R;
  const void* a;            // see the forms in grouped.hip
  int64_t lda;              // elements
  const int32_t* src;       // NT: row r of A is row src[r] / k of a [T, lda] array (NULL: row r)
  int T, k;
  const void *b0, *b1;
  int64_t ldb;
  int64_t b0_stride, b1_stride;   // elements between experts
  int m, n, r;              // TN: m rows of a half; columns; reduction length of a half (NT, NN)
  bool stagger;             // NT: column tiles start at different places of the reduction
  int halves;               // NN: halves of the reduction, TN: of the rows (1 or 2)
  void *out0, *out1;        // TN: the two halves' outputs
  int64_t ldo;
  const void* dh;           // recompute: [R, n]
  int parts;                // NN, TN: the reduction in parts (split_parts, split_row_parts of validate.hpp), their
  float* part;              // sums fp32 in workspace, as many times the outputs; parts <= 1: unused
};

hipError_t launch_grouped_gated(Dt dt, Act act, const GroupedArgs& a, hipStream_t s);
hipError_t launch_grouped_dgated(Dt dt, Act act, const GroupedArgs& a, hipStream_t s);
hipError_t launch_grouped_nt(Dt dt, const GroupedArgs& a, hipStream_t s);
hipError_t launch_grouped_nn(Dt dt, const GroupedArgs& a, hipStream_t s);
hipError_t launch_grouped_tn(Dt dt, const GroupedArgs& a, hipStream_t s);

// The order of pairs by expert (dispatch.hip).
struct PlanArgs {
  const int32_t* ids;       // [n]
  int n, E;
  int32_t *offsets, *src, *pos;
  int32_t* hist;            // workspace: [blocks, E + 1] (one block: unused)
};
hipError_t launch_plan(const PlanArgs& a, hipStream_t s);

struct CombineArgs {
  int T, k, K;
  const int32_t* pos;       // [T, k]
  const float* weights;     // [T, k] or NULL (ones)
  const void* y;            // [T k, K]
  void* out;                // forward: [T, K]
  const void* dy;           // backward: [T, K]
  void* dyr;                // backward: [T k, K]
  float* dweights;          // backward: [T, k]
};
hipError_t launch_combine(Dt dt, const CombineArgs& a, hipStream_t s);
hipError_t launch_combine_bwd(Dt dt, const CombineArgs& a, hipStream_t s);

// out[r] = x[src[r] / k], 0 where src[r] names no pair of the T tokens.
hipError_t launch_gather(Dt dt, int T, int k, int K, const void* x, const int32_t* src, void* out, hipStream_t s);

// The norm of many gradients together and their clipping (clip.hip).
struct GradSpan { const void* g; void* out; int64_t n; };
struct ClipArgs {
  int64_t count;            // host arrays of `count`
  const int* dtypes;
  const void* const* grads;
  const int64_t* sizes;
  void* const* outs;        // NULL: in place
  bool clip;                // false: the norm alone
  double max_norm, eps;
  float* norm;
  float* factor;            // workspace: one float
  double* part;             // workspace: sums of the workgroups
};
hipError_t launch_clip(const ClipArgs& a, hipStream_t s);

}  // namespace swg
