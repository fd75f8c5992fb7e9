// Internal launch interface of the routed block's kernels: router, few-token
// experts and block norms (not part of the ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm.hpp"

namespace swg {

enum class Score { kSoftmax = 0, kSigmoid = 1 };

struct RouteArgs {
  const void* logits;       // [T, E]
  int T, E, k;
  bool renorm;
  float scale;
  float* weights;           // forward: [T, k]
  int32_t* ids;             // forward: [T, k] output
  const int32_t* ids_in;    // backward: [T, k]
  const float* dweights;    // backward: [T, k]
  void* dlogits;            // backward: [T, E]
};
hipError_t launch_route_fwd(Dt dt, Score score, const RouteArgs& a, hipStream_t s);
hipError_t launch_route_bwd(Dt dt, Score score, const RouteArgs& a, hipStream_t s);

struct MoeArgs {
  const void* x;            // [T, K] bf16
  const int32_t* ids;       // [T, k]
  const float* weights;     // [T, k]
  const void *wg, *wu, *wd; // expert e at + e * stride
  int64_t wg_stride, wu_stride, wd_stride;
  void* y;                  // [T, K] bf16
  void* h;                  // workspace: hidden activations, 2 T k N bf16 (see moe.hip)
  float* part;              // workspace: parts of y, [parts, T, K]
  int T, E, k, N, K;
};
hipError_t launch_moe(Act act, const MoeArgs& a, hipStream_t s);

struct NormArgs {
  int64_t rows;
  int cols;
  int64_t groups;           // gate rows (0: no gate)
  const void *res, *y, *w_out, *gate, *w_in;   // res: the backward's res_out
  float skip, scale, w_offset, eps;
  void *res_out, *z;        // forward
  const void *dres_out, *dz;                   // backward
  void *dres, *dy, *dw_out, *dgate, *dw_in;
  float* part;              // backward: sums over the rows of each part (see norm.hip)
  int per_group;            // backward: parts per group
};
hipError_t launch_norm_fwd(Dt dt, const NormArgs& a, hipStream_t s);
hipError_t launch_norm_bwd(Dt dt, const NormArgs& a, hipStream_t s);

}  // namespace swg
