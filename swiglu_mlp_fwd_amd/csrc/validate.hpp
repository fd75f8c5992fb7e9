// Host-side argument validation and workspace layout for the C ABI.
// Pure C++ (no HIP), so it can be compiled and tested without a GPU.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <algorithm>
#include <initializer_list>
#include <new>
#include <vector>

#include "swiglu.h"

namespace swg {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

inline int elem_size(int dtype) { return dtype == SWIGLU_BF16 ? 2 : 4; }
// Elements per 16-byte row chunk: rows must be whole chunks for 128-bit loads.
inline int chunk_elems(int dtype) { return dtype == SWIGLU_BF16 ? 8 : 4; }

inline int check_dtype(int dtype) {
  return (dtype == SWIGLU_F32 || dtype == SWIGLU_BF16) ? SWIGLU_OK : SWIGLU_ERR_DTYPE;
}

inline int check_dims(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 0) return SWIGLU_ERR_SHAPE;
  if (M > kMaxDim || N > kMaxDim || K > kMaxDim) return SWIGLU_ERR_SHAPE;
  return SWIGLU_OK;
}

// GEMM tiles are 128 x 128; the launch grid must stay below 2^31 workgroups.
inline bool tiles_fit(int64_t m, int64_t n) {
  return ((m + 127) / 128) * ((n + 127) / 128) < (int64_t(1) << 31);
}

inline int check_ptr(const void* p) {
  if (p == nullptr) return SWIGLU_ERR_NULL;
  if (!aligned(p, 16)) return SWIGLU_ERR_ALIGN;
  return SWIGLU_OK;
}

// Backward workspace, regions starting on 256-byte boundaries.
//   D   [M, 2 Np]     dg in columns [0, Np), du in [Np, 2 Np), zero padded
//   DT  [2 Np, Mp]    transpose of D, zero padded along M
//   XT  [K, Mp]       transpose of x, zero padded along M
//   WT  [K, 2 Np]     [Wg; Wu] transposed, zero padded along N
// with Mp = round_up(M, 8); Np = round_up(N, 64) for bf16 (its tiles and
// 64-element reduction steps then never straddle the dg / du halves) and
// round_up(N, 8) for fp32.
struct BwdLayout {
  int64_t Mp, Np;
  size_t off_d, off_dt, off_xt, off_wt, total;
};

inline BwdLayout bwd_layout(int dtype, int64_t M, int64_t N, int64_t K) {
  BwdLayout L;
  const size_t es = (size_t)elem_size(dtype);
  const bool bf16 = dtype == SWIGLU_BF16;
  L.Mp = round_up(M, 8);
  L.Np = round_up(N, bf16 ? 64 : 8);
  auto a256 = [](size_t v) { return (v + 255) / 256 * 256; };
  size_t off = 0;
  L.off_d = off;  off += a256((size_t)M * 2 * L.Np * es);
  L.off_dt = off; off += a256((size_t)2 * L.Np * L.Mp * es);
  L.off_xt = off; off += a256((size_t)K * L.Mp * es);
  L.off_wt = off; off += a256((size_t)K * 2 * L.Np * es);
  L.total = off;
  return L;
}

// The GEMM kernels address an operand tile through a buffer descriptor whose
// size and byte offsets are 32-bit: a tile spans at most 512 bytes per unit
// of row stride (256 bf16 rows or 128 fp32 rows), and the out-of-range
// offset 2^31 must lie past it, so every row stride a GEMM reads with (K for
// the forward products, 2 Np and Mp for the backward ones) is capped for
// both element types.  The cap is also the largest padded row count the
// transposes' grids cover (65,535 tiles of 64 rows).
constexpr int64_t kMaxLd = (int64_t(1) << 22) - 64;

inline int validate_fwd(int dtype, int64_t M, int64_t N, int64_t K, const void* x, const void* wg,
                        const void* wu, const void* h) {
  int st = check_dtype(dtype);
  if (st) return st;
  if ((st = check_dims(M, N, K))) return st;
  if (K % chunk_elems(dtype) != 0) return SWIGLU_ERR_SHAPE;
  if (!tiles_fit(M, N)) return SWIGLU_ERR_UNSUPPORTED;
  if (K > kMaxLd) return SWIGLU_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return SWIGLU_OK;
  if ((st = check_ptr(h))) return st;
  if (K > 0) {
    if ((st = check_ptr(x))) return st;
    if ((st = check_ptr(wg))) return st;
    if ((st = check_ptr(wu))) return st;
  }
  return SWIGLU_OK;
}

// The sizes the backward accepts, pointers aside: valid dims, grids that fit,
// and every row stride its GEMMs read with (K, 2 Np, Mp) within kMaxLd.  Within
// these limits every region of bwd_layout is below 2^46 bytes, so its sizes
// cannot wrap.
inline int bwd_shape_status(int dtype, int64_t M, int64_t N, int64_t K) {
  int st = check_dtype(dtype);
  if (st) return st;
  if ((st = check_dims(M, N, K))) return st;
  if (K % chunk_elems(dtype) != 0) return SWIGLU_ERR_SHAPE;
  const int64_t Mp = round_up(M, 8), Np = round_up(N, dtype == SWIGLU_BF16 ? 64 : 8);
  if (K > kMaxLd || 2 * Np > kMaxLd || Mp > kMaxLd) return SWIGLU_ERR_UNSUPPORTED;
  if (!tiles_fit(M, Np) || !tiles_fit(M, K) || !tiles_fit(2 * Np, K)) return SWIGLU_ERR_UNSUPPORTED;
  return SWIGLU_OK;
}

// Workspace bytes of a backward the library accepts; 0 for any other sizes.
inline size_t bwd_workspace_total(int dtype, int64_t M, int64_t N, int64_t K) {
  return bwd_shape_status(dtype, M, N, K) == SWIGLU_OK ? bwd_layout(dtype, M, N, K).total : 0;
}

inline int validate_bwd(int dtype, int64_t M, int64_t N, int64_t K, const void* x, const void* wg,
                        const void* wu, const void* dh, const void* dx, const void* dwg,
                        const void* dwu, const void* ws, size_t ws_bytes) {
  int st = bwd_shape_status(dtype, M, N, K);
  if (st) return st;
  const BwdLayout L = bwd_layout(dtype, M, N, K);
  if (K == 0) return SWIGLU_OK;                       // every output is empty
  if (M > 0 && (st = check_ptr(dx))) return st;
  if (N > 0 && (st = check_ptr(dwg))) return st;
  if (N > 0 && (st = check_ptr(dwu))) return st;
  if (M == 0 || N == 0) return SWIGLU_OK;             // outputs are zero-filled
  if ((st = check_ptr(x))) return st;
  if ((st = check_ptr(wg))) return st;
  if ((st = check_ptr(wu))) return st;
  if ((st = check_ptr(dh))) return st;
  if (ws == nullptr) return SWIGLU_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return SWIGLU_ERR_ALIGN;
  if (ws_bytes < L.total) return SWIGLU_ERR_WORKSPACE;
  return SWIGLU_OK;
}

inline int validate_gemv(int64_t M, int64_t N, int64_t K, const void* x, const void* wg,
                         const void* wu, const void* h) {
  if (M < 0 || M > 8) return SWIGLU_ERR_SHAPE;
  int st = check_dims(M, N, K);
  if (st) return st;
  if (K % 8 != 0) return SWIGLU_ERR_SHAPE;
  if (M == 0 || N == 0) return SWIGLU_OK;
  if ((st = check_ptr(h))) return st;
  if (K > 0) {
    if ((st = check_ptr(x))) return st;
    if ((st = check_ptr(wg))) return st;
    if ((st = check_ptr(wu))) return st;
  }
  return SWIGLU_OK;
}

inline int validate_fwd_fp8(int64_t M, int64_t N, int64_t K, const void* x, const void* wg,
                            const void* wu, const void* q, const void* scale, const void* h_out) {
  int st;
  if ((st = check_dims(M, N, K))) return st;
  if (K % chunk_elems(SWIGLU_BF16) != 0 || N % 32 != 0) return SWIGLU_ERR_SHAPE;
  if (!tiles_fit(M, N)) return SWIGLU_ERR_UNSUPPORTED;
  if (K > kMaxLd) return SWIGLU_ERR_UNSUPPORTED;
  if (h_out != nullptr && !aligned(h_out, 16)) return SWIGLU_ERR_ALIGN;
  if (M == 0 || N == 0) return SWIGLU_OK;
  if ((st = check_ptr(q))) return st;
  if (scale == nullptr) return SWIGLU_ERR_NULL;
  if (K > 0) {
    if ((st = check_ptr(x))) return st;
    if ((st = check_ptr(wg))) return st;
    if ((st = check_ptr(wu))) return st;
  }
  return SWIGLU_OK;
}

inline int validate_act_fwd(int out_dtype, int64_t rows, int64_t cols, const float* gate, const float* up,
                            float L, const void* h, const void* count) {
  int st = check_dtype(out_dtype);
  if (st) return st;
  if (rows < 0 || cols < 0) return SWIGLU_ERR_SHAPE;
  if (cols % 8 != 0) return SWIGLU_ERR_SHAPE;         // the interface's row granularity (the kernel needs 4)
  if (rows > 0 && cols > (int64_t(1) << 40) / rows) return SWIGLU_ERR_SHAPE;
  if (!(L > 0.0f)) return SWIGLU_ERR_ARG;             // rejects NaN, zero and negatives
  if (count != nullptr && !aligned(count, 8)) return SWIGLU_ERR_ALIGN;
  if (rows == 0 || cols == 0) return SWIGLU_OK;
  if ((st = check_ptr(gate))) return st;
  if ((st = check_ptr(up))) return st;
  if ((st = check_ptr(h))) return st;
  return SWIGLU_OK;
}

inline int validate_act_quant(int64_t rows, int64_t cols, const float* gate, const float* up,
                              float L, const void* q, const void* scale, const void* count,
                              const void* hout) {
  if (rows < 0 || cols < 0) return SWIGLU_ERR_SHAPE;
  if (cols % 32 != 0) return SWIGLU_ERR_SHAPE;
  if (rows > 0 && cols > (int64_t(1) << 40) / rows) return SWIGLU_ERR_SHAPE;
  if (!(L > 0.0f)) return SWIGLU_ERR_ARG;             // rejects NaN, zero and negatives
  if (count != nullptr && !aligned(count, 8)) return SWIGLU_ERR_ALIGN;
  if (rows == 0 || cols == 0) return SWIGLU_OK;
  int st;
  if ((st = check_ptr(gate))) return st;
  if ((st = check_ptr(up))) return st;
  if ((st = check_ptr(q))) return st;
  if ((st = check_ptr(scale))) return st;
  if (hout != nullptr && !aligned(hout, 16)) return SWIGLU_ERR_ALIGN;
  return SWIGLU_OK;
}

inline int validate_act_bwd(int dtype, int64_t rows, int64_t cols, const void* gate, const void* up,
                            const void* dy, const float* weights, float L, const void* dgate,
                            const void* dup, const float* wgrad) {
  int st0 = check_dtype(dtype);
  if (st0) return st0;
  if (rows < 0 || cols < 0) return SWIGLU_ERR_SHAPE;
  if (cols % chunk_elems(dtype) != 0) return SWIGLU_ERR_SHAPE;   // 16-byte rows
  if (rows > 0 && cols > (int64_t(1) << 40) / rows) return SWIGLU_ERR_SHAPE;
  if (!(L > 0.0f)) return SWIGLU_ERR_ARG;             // rejects NaN, zero and negatives
  if (weights != nullptr && !aligned(weights, 4)) return SWIGLU_ERR_ALIGN;
  if (wgrad != nullptr && !aligned(wgrad, 4)) return SWIGLU_ERR_ALIGN;
  if (rows == 0) return SWIGLU_OK;
  if (cols > 0) {
    int st;
    if ((st = check_ptr(gate))) return st;
    if ((st = check_ptr(up))) return st;
    if ((st = check_ptr(dy))) return st;
    if ((st = check_ptr(dgate))) return st;
    if ((st = check_ptr(dup))) return st;
  }
  return SWIGLU_OK;
}

inline int validate_act_bwd_fp8(int dtype, int64_t rows, int64_t cols, const void* gate, const void* up,
                                const void* dy, const float* weights, float L, const void* qg, const void* sg,
                                const void* qu, const void* su, const float* wgrad) {
  int st = check_dtype(dtype);
  if (st) return st;
  if (rows < 0 || cols < 0) return SWIGLU_ERR_SHAPE;
  if (cols % 32 != 0) return SWIGLU_ERR_SHAPE;        // whole 1x32 blocks per row
  if (rows > 0 && cols > (int64_t(1) << 40) / rows) return SWIGLU_ERR_SHAPE;
  if (!(L > 0.0f)) return SWIGLU_ERR_ARG;             // rejects NaN, zero and negatives
  if (weights != nullptr && !aligned(weights, 4)) return SWIGLU_ERR_ALIGN;
  if (wgrad != nullptr && !aligned(wgrad, 4)) return SWIGLU_ERR_ALIGN;
  if (rows == 0 || cols == 0) return SWIGLU_OK;
  if ((st = check_ptr(gate))) return st;
  if ((st = check_ptr(up))) return st;
  if ((st = check_ptr(dy))) return st;
  if ((st = check_ptr(qg))) return st;
  if ((st = check_ptr(qu))) return st;
  if (sg == nullptr || su == nullptr) return SWIGLU_ERR_NULL;
  return SWIGLU_OK;
}

// ---- routed block

inline int check_route(int64_t T, int64_t E, int64_t k) {
  if (T < 0 || T > kMaxDim || E < 1 || E > SWIGLU_MAX_EXPERTS) return SWIGLU_ERR_SHAPE;
  if (k < 1 || k > E || k > SWIGLU_MAX_TOPK) return SWIGLU_ERR_SHAPE;
  return SWIGLU_OK;
}

// Elements of a tensor that one launch walks: a launch has at most 2^32 - 1
// threads, and the kernels take one for 4 to 16 elements (and at least 8 for
// a token, 16 for a row).
constexpr int64_t kBlockMaxElems = int64_t(1) << 33;

inline bool finite_f(float v) { return v - v == 0.0f; }

// weights / dweights: `f`; ids: `i`; dlogits: `d` (nullptr in the forward's
// check, which has no such argument: has_d says whether it must be there).
inline int validate_route(int score, int dtype, int64_t T, int64_t E, int64_t k, const void* logits, float scale,
                          const void* f, const void* i, const void* d, bool has_d) {
  if (score != SWIGLU_SCORE_SOFTMAX && score != SWIGLU_SCORE_SIGMOID) return SWIGLU_ERR_ARG;
  int st = check_dtype(dtype);
  if (st) return st;
  if ((st = check_route(T, E, k))) return st;
  if (!finite_f(scale)) return SWIGLU_ERR_ARG;
  if (T * (E > 64 ? E : 64) > kBlockMaxElems) return SWIGLU_ERR_UNSUPPORTED;
  if (T == 0) return SWIGLU_OK;
  if ((st = check_ptr(logits))) return st;
  if (f == nullptr || i == nullptr) return SWIGLU_ERR_NULL;
  if (!aligned(f, 4) || !aligned(i, 4)) return SWIGLU_ERR_ALIGN;
  if (has_d && (st = check_ptr(d))) return st;
  return SWIGLU_OK;
}

constexpr int64_t kMoeMaxDim = int64_t(1) << 20;

inline int moe_shape_status(int64_t T, int64_t N, int64_t K, int64_t k) {
  if (T < 0 || T > SWIGLU_MOE_MAX_TOKENS || N < 0 || K < 0) return SWIGLU_ERR_SHAPE;
  if (k < 1 || k > SWIGLU_MAX_TOPK) return SWIGLU_ERR_SHAPE;
  if (K % 8 != 0 || N % 8 != 0) return SWIGLU_ERR_SHAPE;
  if (N > kMoeMaxDim || K > kMoeMaxDim) return SWIGLU_ERR_UNSUPPORTED;
  return SWIGLU_OK;
}

// Parts that the second product's reduction is split into, at most, where its
// tiles of `cols` columns (16 or 32) leave many of the 256 CUs without a
// workgroup.
constexpr int64_t kMoeFullBlocks = 160;
inline int64_t moe_parts(int64_t K, int64_t cols) {
  const int64_t blocks = (K + cols - 1) / cols;
  return blocks == 0 || blocks > kMoeFullBlocks ? 1 : (256 + blocks - 1) / blocks;
}

// Workgroups of `waves` waves and `lds` bytes of LDS (static and dynamic) that
// a CU holds at a time, where `cu_waves` of their waves fit its registers; 1
// at least.
inline int moe_resident(int waves, int cu_waves, size_t lds) {
  const int by_waves = cu_waves / waves, by_lds = lds == 0 ? by_waves : (int)(size_t(160 * 1024) / lds);
  const int n = by_waves < by_lds ? by_waves : by_lds;
  return n < 1 ? 1 : n;
}

// Workspace of the few-token experts, regions on 256-byte boundaries: the
// hidden activations of T k (token, expert) entries, two bf16 each, and the
// parts of y in fp32.
struct MoeLayout {
  size_t off_part, total;
};
inline MoeLayout moe_layout(int64_t T, int64_t N, int64_t K, int64_t k) {
  auto a256 = [](size_t v) { return (v + 255) / 256 * 256; };
  const int64_t parts = moe_parts(K, 32);          // never fewer than of 16 columns
  MoeLayout L;
  L.off_part = a256((size_t)T * k * N * 4);
  L.total = L.off_part + (parts > 1 ? a256((size_t)parts * T * K * 4) : 0);
  return L;
}
inline size_t moe_workspace_total(int64_t T, int64_t N, int64_t K, int64_t k) {
  return moe_shape_status(T, N, K, k) == SWIGLU_OK ? moe_layout(T, N, K, k).total : 0;
}

inline int validate_moe(int64_t T, int64_t E, int64_t k, int64_t N, int64_t K, const void* x, const void* ids,
                        const void* weights, const void* wg, int64_t wg_stride, const void* wu,
                        int64_t wu_stride, const void* wd, int64_t wd_stride, const void* y, const void* ws, size_t ws_bytes) {
  int st = moe_shape_status(T, N, K, k);
  if (st) return st;
  if ((st = check_route(T, E, k))) return st;
  for (int64_t stride : {wg_stride, wu_stride, wd_stride}) {
    if (stride < 0 || stride % 8 != 0 || stride > (int64_t(1) << 48)) return SWIGLU_ERR_SHAPE;
    if (stride < N * K && E > 1) return SWIGLU_ERR_SHAPE;
  }
  if (T == 0 || K == 0) return SWIGLU_OK;
  if ((st = check_ptr(y))) return st;
  if (N == 0) return SWIGLU_OK;                       // y is zero-filled
  if ((st = check_ptr(x))) return st;
  if (ids == nullptr || weights == nullptr) return SWIGLU_ERR_NULL;
  if (!aligned(ids, 4) || !aligned(weights, 4)) return SWIGLU_ERR_ALIGN;
  if ((st = check_ptr(wg))) return st;
  if ((st = check_ptr(wu))) return st;
  if ((st = check_ptr(wd))) return st;
  if (ws == nullptr) return SWIGLU_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return SWIGLU_ERR_ALIGN;
  if (ws_bytes < moe_workspace_total(T, N, K, k)) return SWIGLU_ERR_WORKSPACE;
  return SWIGLU_OK;
}

constexpr int64_t kNormMaxCols = 16384;
constexpr int64_t kNormMaxGroups = int64_t(1) << 20;   // a workgroup of the backward each

// A row of `nch` 16-byte chunks is held by 16, 32 or 64 lanes of a wave, one
// chunk each, or (lanes 0) by a whole workgroup, 1, 2 or 4 chunks to a thread.
inline int norm_lanes(int64_t nch) { return nch <= 16 ? 16 : nch <= 32 ? 32 : nch <= 64 ? 64 : 0; }
inline int norm_chunks(int64_t nch) { return nch <= 1024 ? 1 : nch <= 2048 ? 2 : 4; }
constexpr int kNormThreads = 512;                      // backward workgroups of several rows
inline int norm_wide_threads(int64_t nch, int chunks) { return (int)(((nch + chunks - 1) / chunks + 63) / 64 * 64); }

// Parts that the backward's sums over rows are split into.  A part is the walk
// of one workgroup, which takes R rows at a time.  Narrow rows have small
// workgroups and more parts, to fill the chip.
constexpr int64_t kNormMinParts = 512, kNormMaxParts = 2048;
inline int64_t norm_parts(int64_t cols) {
  const int64_t n = (int64_t(1) << 21) / cols;
  return n < kNormMinParts ? kNormMinParts : (n > kNormMaxParts ? kNormMaxParts : n);
}
// Parts per group that the workspace has room for: norm_parts shared out among
// the groups, at least one and no more than its rows to each.
inline int64_t norm_most_parts(int64_t rows, int64_t cols, int64_t groups) {
  const int64_t g = groups > 0 ? groups : 1, rpg = rows / g, per = norm_parts(cols) / g;
  return per > rpg ? rpg : per < 1 && rows > 0 ? 1 : per;
}
// Parts per group of a launch.  Two workgroups of 512 threads per CU, more of
// smaller ones (512 against 1024 parts: 8192 x 4096 bf16 98 against 102 us with
// the sums of the parts, 32768 x 1024 154 against 97); then as few as give
// every part as many turns as the longest has.  Beyond 512 rows at a time a
// part has three turns at least: a turn more costs less than the sum of as
// many more parts (1692 x 395 fp32 in 4 groups 15.5 us in all against 19.2,
// 996 x 1864 bf16 16.7 against 18.7).  Never more than the workspace has room
// for, whatever a workgroup's threads.
inline int64_t norm_bwd_parts(int elem, int64_t rows, int64_t cols, int64_t groups) {
  if (rows == 0) return 0;
  const int64_t nch = (cols * elem + 15) / 16, g = groups > 0 ? groups : 1, rpg = rows / g;
  const int lanes = norm_lanes(nch);
  const int64_t threads = lanes ? kNormThreads : norm_wide_threads(nch, norm_chunks(nch));
  const int64_t R = lanes ? kNormThreads / lanes : 1, most = norm_most_parts(rows, cols, groups);
  int64_t per = norm_parts(threads * 8) / g;
  if (per < 1) per = 1;
  if (per > most) per = most;
  int64_t turns = (rpg + R * per - 1) / (R * per);
  if (turns < 3 && rows > 512 * R) turns = 3;
  return (rpg + R * turns - 1) / (R * turns);
}

inline int norm_shape_status(int64_t rows, int64_t cols, int64_t groups) {
  if (rows < 0 || rows > kMaxDim || cols < 1 || groups < 0 || groups > kMaxDim) return SWIGLU_ERR_SHAPE;
  if (groups > 0 && rows % groups != 0) return SWIGLU_ERR_SHAPE;
  if (cols > kNormMaxCols || groups > kNormMaxGroups) return SWIGLU_ERR_UNSUPPORTED;
  if (rows * (cols > 128 ? cols : 128) > kBlockMaxElems) return SWIGLU_ERR_UNSUPPORTED;
  return SWIGLU_OK;
}

// Two fp32 sums of [cols] per part.
inline size_t norm_bwd_workspace_total(int64_t rows, int64_t cols, int64_t groups) {
  if (norm_shape_status(rows, cols, groups) != SWIGLU_OK) return 0;
  const size_t n = (size_t)2 * (groups > 0 ? groups : 1) * norm_most_parts(rows, cols, groups) * cols * 4;
  return (n + 255) / 256 * 256;
}

inline int validate_norm(int dtype, int64_t rows, int64_t cols, int64_t groups, const void* y, const void* w_out,
                         const void* gate, const void* w_in, float skip, float scale, float w_offset, float eps) {
  int st = check_dtype(dtype);
  if (st) return st;
  if ((st = norm_shape_status(rows, cols, groups))) return st;
  if (!finite_f(skip) || !finite_f(scale) || !finite_f(w_offset) || !finite_f(eps) || !(eps > 0.0f))
    return SWIGLU_ERR_ARG;
  // Without rows y is empty, and an empty tensor may be NULL.
  if (rows > 0 && y == nullptr && (w_out != nullptr || gate != nullptr || w_in == nullptr)) return SWIGLU_ERR_ARG;
  if ((gate == nullptr) != (groups == 0)) return SWIGLU_ERR_ARG;
  return SWIGLU_OK;
}

// Each pointer aligned to an element; `need`ed ones not NULL, the others NULL.
struct PtrRule { const void* p; bool need; };
inline int check_elems(int dtype, const PtrRule* r, int n) {
  for (int i = 0; i < n; ++i) {
    if (r[i].need && r[i].p == nullptr) return SWIGLU_ERR_NULL;
    if (!r[i].need && r[i].p != nullptr) return SWIGLU_ERR_ARG;
    if (r[i].p != nullptr && !aligned(r[i].p, (uintptr_t)elem_size(dtype))) return SWIGLU_ERR_ALIGN;
  }
  return SWIGLU_OK;
}

inline int validate_norm_fwd(int dtype, int64_t rows, int64_t cols, int64_t groups, const void* res, const void* y,
                             const void* w_out, const void* gate, const void* w_in, float skip, float scale,
                             float w_offset, float eps, const void* res_out, const void* z) {
  int st = validate_norm(dtype, rows, cols, groups, y, w_out, gate, w_in, skip, scale, w_offset, eps);
  if (st || rows == 0) return st;
  const PtrRule r[] = {{res, true}, {y, y != nullptr}, {w_out, w_out != nullptr}, {gate, gate != nullptr},
                       {w_in, w_in != nullptr}, {res_out, y != nullptr}, {z, w_in != nullptr}};
  return check_elems(dtype, r, 7);
}

inline int validate_norm_bwd(int dtype, int64_t rows, int64_t cols, int64_t groups, const void* res_out,
                             const void* y, const void* w_out, const void* gate, const void* w_in,
                             const void* dres_out, const void* dz, float skip, float scale, float w_offset, float eps,
                             const void* dres, const void* dy, const void* dw_out, const void* dgate,
                             const void* dw_in, const void* ws, size_t ws_bytes) {
  int st = validate_norm(dtype, rows, cols, groups, y, w_out, gate, w_in, skip, scale, w_offset, eps);
  if (st) return st;
  const PtrRule grads[] = {{dw_out, w_out != nullptr}, {dgate, gate != nullptr}, {dw_in, w_in != nullptr}};
  if ((st = check_elems(dtype, grads, 3))) return st;
  if (rows == 0) return SWIGLU_OK;                    // the weights' gradients are zero-filled
  const PtrRule r[] = {{y, y != nullptr}, {w_out, w_out != nullptr}, {gate, gate != nullptr},
                       {w_in, w_in != nullptr}, {dz, w_in != nullptr}, {dres, true}, {dy, y != nullptr},
                       {res_out, w_in != nullptr || res_out != nullptr},
                       {dres_out, dres_out != nullptr}};
  if ((st = check_elems(dtype, r, 9))) return st;
  if (w_out == nullptr && gate == nullptr && w_in == nullptr) return SWIGLU_OK;   // nothing is summed over rows
  if (ws == nullptr) return SWIGLU_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return SWIGLU_ERR_ALIGN;
  if (ws_bytes < norm_bwd_workspace_total(rows, cols, groups)) return SWIGLU_ERR_WORKSPACE;
  return SWIGLU_OK;
}

// ---- rows in order of expert

// The plan's counting sort: one workgroup of kPlanThreads for up to kPlanOne
// pairs, otherwise at most kPlanBlocks, each a whole number of 64 pairs to a
// wave.
constexpr int kPlanThreads = 1024;
constexpr int64_t kPlanOne = 8192, kPlanBlocks = 128;
inline int plan_per_block(int64_t n) {
  return (int)round_up(n <= kPlanOne ? (n < 1 ? 1 : n) : (n + kPlanBlocks - 1) / kPlanBlocks, kPlanThreads);
}
inline int plan_blocks(int64_t n) {
  const int64_t per = plan_per_block(n);
  return n < 1 ? 1 : (int)((n + per - 1) / per);
}

inline int check_pairs(int64_t T, int64_t k) {
  if (T < 0 || k < 1 || k > SWIGLU_MAX_TOPK) return SWIGLU_ERR_SHAPE;
  if (T > kMaxDim / k) return SWIGLU_ERR_SHAPE;
  return SWIGLU_OK;
}

inline int plan_status(int64_t T, int64_t k, int64_t E) {
  if (E < 1 || E > SWIGLU_MAX_EXPERTS) return SWIGLU_ERR_SHAPE;
  return check_pairs(T, k);
}
inline size_t plan_workspace_total(int64_t T, int64_t k, int64_t E) {
  if (plan_status(T, k, E) != SWIGLU_OK) return 0;
  const int blocks = plan_blocks(T * k);
  return blocks > 1 ? (size_t)round_up((int64_t)blocks * (E + 1) * 4, 256) : 0;
}

inline int check_int(const void* p) {
  if (p == nullptr) return SWIGLU_ERR_NULL;
  return aligned(p, 4) ? SWIGLU_OK : SWIGLU_ERR_ALIGN;
}

inline int validate_plan(int64_t T, int64_t k, int64_t E, const void* ids, const void* offsets, const void* src,
                         const void* pos, const void* ws, size_t ws_bytes) {
  int st = plan_status(T, k, E);
  if (st) return st;
  if ((st = check_int(offsets))) return st;
  if (T > 0) {
    for (const void* p : {ids, src, pos})
      if ((st = check_int(p))) return st;
  }
  const size_t need = plan_workspace_total(T, k, E);
  if (need > 0) {
    if (ws == nullptr || ws_bytes < need) return SWIGLU_ERR_WORKSPACE;
    if (!aligned(ws, 256)) return SWIGLU_ERR_ALIGN;
  }
  return SWIGLU_OK;
}

// Sizes of gather and combine: whole 16-byte chunks per row; a wave for 64
// chunks of a row, 4 waves to a workgroup and at most 2^32 - 1 threads to a
// launch.
inline int rows_status(int dtype, int64_t T, int64_t k, int64_t K) {
  int st = check_dtype(dtype);
  if (st) return st;
  if ((st = check_pairs(T, k))) return st;
  if (K < 0 || K > kMaxDim || K % chunk_elems(dtype) != 0) return SWIGLU_ERR_SHAPE;
  if (T > 0 && (K / chunk_elems(dtype) + 63) / 64 > (int64_t(1) << 25) / (T * k)) return SWIGLU_ERR_UNSUPPORTED;
  if (T > (int64_t(1) << 23)) return SWIGLU_ERR_UNSUPPORTED;   // (a workgroup to a token of the backward)
  return SWIGLU_OK;
}

// rows: tensors of whole rows; ints: 4-byte elements; opt: those that may be NULL.
inline int validate_rows(int dtype, int64_t T, int64_t k, int64_t K, std::initializer_list<const void*> rows,
                         std::initializer_list<const void*> ints, std::initializer_list<const void*> opt) {
  int st = rows_status(dtype, T, k, K);
  if (st || T == 0) return st;
  for (const void* p : ints)
    if ((st = check_int(p))) return st;
  for (const void* p : opt)
    if (!aligned(p, 4)) return SWIGLU_ERR_ALIGN;
  if (K == 0) return SWIGLU_OK;
  for (const void* p : rows)
    if ((st = check_ptr(p))) return st;
  return SWIGLU_OK;
}

// Grouped products.  Their grids hold the row tiles of R rows in E + 2 groups
// (NT, NN), or all tiles of the experts' weights (TN); tiles are 128 rows by
// 64 columns at least where there are many, and a launch has at most 2^32 - 1
// threads, 512 to a workgroup.
constexpr int64_t kGroupedMaxTiles = (int64_t(1) << 23) - 1;
inline int grouped_shape_status(int dtype, int64_t R, int64_t E, int64_t N, int64_t K) {
  int st = check_dtype(dtype);
  if (st) return st;
  if ((st = check_dims(R, N, K))) return st;
  if (E < 1 || E > SWIGLU_MAX_EXPERTS) return SWIGLU_ERR_SHAPE;
  if (N % chunk_elems(dtype) != 0 || K % chunk_elems(dtype) != 0) return SWIGLU_ERR_SHAPE;
  if (2 * N > kMaxLd || K > kMaxLd) return SWIGLU_ERR_UNSUPPORTED;
  const int64_t cols = ((N > K ? N : K) + 63) / 64, wt = 2 * ((N + 127) / 128) * ((K + 127) / 128);
  if (cols > 0 && R / 128 + E + 2 > kGroupedMaxTiles / cols) return SWIGLU_ERR_UNSUPPORTED;
  if (wt > 0 && E > kGroupedMaxTiles / wt) return SWIGLU_ERR_UNSUPPORTED;
  return SWIGLU_OK;
}

inline int check_expert_stride(int dtype, int64_t E, int64_t N, int64_t K, int64_t stride) {
  if (stride < 0 || stride % chunk_elems(dtype) != 0 || stride > (int64_t(1) << 48)) return SWIGLU_ERR_SHAPE;
  return E > 1 && stride < N * K ? SWIGLU_ERR_SHAPE : SWIGLU_OK;
}

// src given: x is [T, K], R = T k.
inline int check_src(int dtype, int64_t R, int64_t K, int64_t T, int64_t k, const void* src) {
  if (src == nullptr) return SWIGLU_OK;
  int st = check_pairs(T, k);
  if (st) return st;
  if (R != T * k) return SWIGLU_ERR_SHAPE;
  if (!aligned(src, 4)) return SWIGLU_ERR_ALIGN;
  // Byte offsets of a token's row are 32-bit.
  return T * K * elem_size(dtype) < (int64_t(1) << 31) ? SWIGLU_OK : SWIGLU_ERR_UNSUPPORTED;
}

inline int validate_grouped_fwd(int dtype, int64_t R, int64_t E, int64_t N, int64_t K, const void* x, int64_t T,
                                int64_t k, const void* src, const void* offsets, const void* wg, int64_t sg,
                                const void* wu, int64_t su, const void* h) {
  int st = grouped_shape_status(dtype, R, E, N, K);
  if (st) return st;
  if ((st = check_expert_stride(dtype, E, N, K, sg)) || (st = check_expert_stride(dtype, E, N, K, su))) return st;
  if ((st = check_src(dtype, R, K, T, k, src))) return st;
  if (R == 0 || N == 0) return SWIGLU_OK;
  if ((st = check_int(offsets)) || (st = check_ptr(h))) return st;
  if (K == 0) return SWIGLU_OK;
  for (const void* p : {x, wg, wu})
    if ((st = check_ptr(p))) return st;
  return SWIGLU_OK;
}

// Which tile of rows and columns a product of rows takes.  bf16: the small one
// where the large ones would leave many of the 256 CUs without a workgroup, and
// up to so many rows per expert (rows drawn with a spread of a half,
// logarithmic):
// gate/up 64, of 64 x (1024, 2048) with 32 rows each 115 us with large tiles,
// 104 with small, with 64 152 and 112, with 128 160 and 161; of 8 x (14336, 4096)
// with 32 365 and 328, with 64 410 and 376, with 96 406 and 471;
// the down product 32, of 64 x (2048, 1024) with 16 rows each 57 and 52, with 32
// 59 and 59; of 8 x (6912, 1536) 40 and 36, 43 and 36, with 64 43 and 47; of
// 8 x (4096, 2048) with 64 (160 large tiles) 51 and 33, with 128 (192) 53 and 45
// -- the limit of 176 tiles lies between these and gives the latter the large
// tile, 15 % slower there; nothing between was measured;
// dx 16, of 64 x (1024, 2048) with 16 rows each 63 and 51, with 32 66 and 70.
// (One workgroup to a CU, twice the columns and a ring of four took as long
// for the same number of tiles but more where a last round is nearly empty:
// 114 for the first of these.)  The recompute has the large one only: the small
// tile's ring has no room for the dh tile.
// fp32, whose tiles are bound by the matrix cores: tiles of 32 rows up to 128
// rows per expert, and where the large ones are fewer than the CUs.  64
// experts of (1024, 2048), gate/up: 16 rows each 484 us with large tiles, 208
// with small, 128 862 and 701, 512 2222 and 2316; 5 of (200, 264): 23 and 14.
enum class RowForm { kGated, kRecompute, kNT, kNN };
struct RowTile {
  int bm, bn, threads;
  constexpr bool operator==(const RowTile& o) const { return bm == o.bm && bn == o.bn && threads == o.threads; }
};
struct TileRule {
  RowTile large, few;
  int rows, tiles;   // the small one up to so many rows per expert, or so many large tiles
};
constexpr TileRule tile_rule(int dtype, RowForm form) {
  if (dtype == SWIGLU_F32)
    return form == RowForm::kGated || form == RowForm::kRecompute
               ? TileRule{{128, 64, 256}, {32, 64, 128}, 128, 256}
               : TileRule{{128, 128, 256}, {32, 64, 128}, 128, 256};
  return form == RowForm::kGated     ? TileRule{{256, 128, 512}, {64, 64, 512}, 64, 176}
         : form == RowForm::kRecompute ? TileRule{{256, 128, 512}, {256, 128, 512}, 0, 0}
         : form == RowForm::kNT      ? TileRule{{256, 256, 512}, {64, 128, 512}, 32, 176}
                                     : TileRule{{256, 256, 512}, {64, 256, 256}, 16, 176};
}
// Tiles of R rows in at most min(E + 2, R) groups that have any, by n columns.
inline int64_t row_column_tiles(const RowTile& t, int64_t R, int64_t E, int64_t n) {
  return (R / t.bm + (E + 2 < R ? E + 2 : R)) * ((n + t.bn - 1) / t.bn);
}
inline RowTile row_tile(int dtype, RowForm form, int64_t R, int64_t E, int64_t n) {
  const TileRule r = tile_rule(dtype, form);
  const int64_t large = (R / r.large.bm + (E < R ? E : R)) * ((n + r.large.bn - 1) / r.large.bn);
  if (R > r.rows * E && large > r.tiles) return r.large;
  // A launch has fewer than 2^32 threads; grouped_shape_status bounds the tiles
  // of 128 x 64 and larger.
  return row_column_tiles(r.few, R, E, n) * r.few.threads < (int64_t(1) << 32) ? r.few : r.large;
}

// Column tiles start apart up to 256 rows per expert, where the weights' stream
// bounds the product.  64 x (1024, 2048) with 32 rows each, gate/up 123 us from
// the same place, 95 apart, with 128 146 and 136; 8 x (14336, 4096) with 128 470
// and 446; fp32, 16 x (4096, 1024) with 16 160 and 128, from 32 on the same.
// With 512 it costs as much (bf16, 8 x (4096, 2048): 167 and 168) or more, since
// column tiles share rows of x.
inline bool weights_bound(int64_t R, int64_t E) { return R <= 256 * E; }

// The gradient of x where rows are few: its reduction, over r columns of each of
// `halves` matrices, in so many parts that the small tiles of R rows in E experts
// and n columns give every CU its workgroups, a part being 8 k-steps at least.
// 1: not split.  8 experts of (6912, 1536), bf16, 16 rows each: 148 us in one
// part, 41 split, with 128 153 and 77; fp32, 16 rows each 185 and 104.
struct SplitTile { int bm, bn, step, target; };
constexpr SplitTile kSplitBf16 = {64, 256, 64, 512}, kSplitF32 = {32, 64, 32, 1024};
inline int split_parts(int dtype, int64_t R, int64_t E, int64_t n, int64_t r, int halves) {
  const SplitTile t = dtype == SWIGLU_BF16 ? kSplitBf16 : kSplitF32;
  const int64_t tiles = (R / t.bm + (E + 2 < R ? E + 2 : R)) * ((n + t.bn - 1) / t.bn);
  if (tiles <= 0) return 1;
  const int64_t steps = halves * ((r + t.step - 1) / t.step), parts = t.target / tiles;
  const int64_t p = parts < steps / 8 ? parts : steps / 8;
  return p < 2 ? 1 : (int)p;
}
// Bytes of the parts' sums for any number of experts (one makes the fewest
// tiles).
inline size_t split_bytes(int dtype, int64_t R, int64_t n, int64_t r, int halves) {
  const int parts = split_parts(dtype, R, 1, n, r, halves);
  return parts > 1 ? (size_t)round_up((int64_t)parts * R * n * 4, 256) : 0;
}

// The weights' gradients where weights are small: each expert's rows (their number
// is known to the device only; R / E of them here) in so many parts that the
// tiles of E experts' halves of m x n give every CU its workgroups.  The gate/up
// gradients of 290000 rows, 2 experts of (152, 320), bf16: 4.64 ms in one part
// (16 tiles), 0.84 split.
constexpr SplitTile kSplitRowsBf16 = {256, 256, 64, 256}, kSplitRowsF32 = {128, 128, 32, 512};
inline int64_t weight_tiles(const SplitTile& t, int64_t m, int64_t n, int halves) {
  return halves * ((m + t.bm - 1) / t.bm) * ((n + t.bn - 1) / t.bn);
}
inline int split_row_parts(int dtype, int64_t R, int64_t E, int64_t m, int64_t n, int halves) {
  const SplitTile t = dtype == SWIGLU_BF16 ? kSplitRowsBf16 : kSplitRowsF32;
  const int64_t tiles = E * weight_tiles(t, m, n, halves);
  if (tiles <= 0) return 1;
  const int64_t parts = t.target / tiles, steps = R / (E * t.step);
  const int64_t p = parts < steps / 8 ? parts : steps / 8;
  return p < 2 ? 1 : (int)p;
}
// Bytes of the parts' sums for any number of experts: E parts(E) is parts(1) at
// most.
inline size_t split_row_bytes(int dtype, int64_t R, int64_t m, int64_t n, int halves) {
  const SplitTile t = dtype == SWIGLU_BF16 ? kSplitRowsBf16 : kSplitRowsF32;
  const int64_t tiles = weight_tiles(t, m, n, halves);
  if (tiles <= 0) return 0;
  const int64_t parts = t.target / tiles, steps = R / t.step / 8;
  const int64_t p = parts < steps ? parts : steps;
  return p < 2 ? 0 : (size_t)round_up(p * halves * m * n * 4, 256);
}
// Both gradients' sums use the same workspace, one after the other: what a call
// with E experts needs, or (E = 0) with any number of them.  64 experts of (1024,
// 2048), 32768 rows: none, for any number 67 MB.
inline size_t split_grads_bytes(int dtype, int64_t R, int64_t E, int64_t N, int64_t K, int halves) {
  size_t x, w;
  if (E == 0) {
    x = split_bytes(dtype, R, K, N, halves);
    w = split_row_bytes(dtype, R, N, K, halves);
  } else {
    const int64_t px = split_parts(dtype, R, E, K, N, halves), pw = split_row_parts(dtype, R, E, N, K, halves);
    x = px > 1 ? (size_t)round_up(px * R * K * 4, 256) : 0;
    w = pw > 1 ? (size_t)round_up(pw * E * halves * N * K * 4, 256) : 0;
  }
  return x > w ? x : w;
}

// Workspace of the grouped backward, regions on 256-byte boundaries: D =
// [dg | du], [R, 2 N], the gathered rows of x, [R, K], and the parts' sums of
// split gradients (of E experts; E = 0: of any number).
struct GroupedBwdLayout { size_t off_x, off_part, total; };
inline GroupedBwdLayout grouped_bwd_layout(int dtype, int64_t R, int64_t E, int64_t N, int64_t K, bool gathered) {
  GroupedBwdLayout L;
  const size_t es = (size_t)elem_size(dtype);
  L.off_x = (size_t)round_up((int64_t)(R * 2 * N * es), 256);
  L.off_part = L.off_x + (gathered ? (size_t)round_up((int64_t)(R * K * es), 256) : 0);
  L.total = L.off_part + split_grads_bytes(dtype, R, E, N, K, 2);
  return L;
}
inline size_t grouped_bwd_workspace_total(int dtype, int64_t R, int64_t N, int64_t K, bool gathered) {
  return grouped_shape_status(dtype, R, 1, N, K) == SWIGLU_OK ? grouped_bwd_layout(dtype, R, 0, N, K, gathered).total : 0;
}
inline size_t grouped_bwd_workspace_of(int dtype, int64_t R, int64_t E, int64_t N, int64_t K, bool gathered) {
  return grouped_shape_status(dtype, R, E, N, K) == SWIGLU_OK ? grouped_bwd_layout(dtype, R, E, N, K, gathered).total : 0;
}

inline int validate_grouped_bwd(int dtype, int64_t R, int64_t E, int64_t N, int64_t K, const void* x, int64_t T,
                                int64_t k, const void* src, const void* offsets, const void* wg, int64_t sg,
                                const void* wu, int64_t su, const void* dh, const void* dx, const void* dwg,
                                const void* dwu, const void* ws, size_t ws_bytes) {
  int st = grouped_shape_status(dtype, R, E, N, K);
  if (st) return st;
  if ((st = check_expert_stride(dtype, E, N, K, sg)) || (st = check_expert_stride(dtype, E, N, K, su))) return st;
  if ((st = check_src(dtype, R, K, T, k, src))) return st;
  if (src != nullptr && (st = rows_status(dtype, T, k, K))) return st;
  if ((dwg == nullptr) != (dwu == nullptr)) return SWIGLU_ERR_ARG;
  for (const void* p : {dx, dwg, dwu})
    if (!aligned(p, 16)) return SWIGLU_ERR_ALIGN;
  if (K == 0 || (dx == nullptr && dwg == nullptr)) {
    // Nothing to compute; an output that has elements must be asked for.
    return K > 0 && ((R > 0) || (N > 0)) ? SWIGLU_ERR_NULL : SWIGLU_OK;
  }
  if (R > 0 || N > 0) {
    if ((st = check_int(offsets))) return st;
  }
  if (R == 0 || N == 0) return SWIGLU_OK;             // outputs are zero-filled
  for (const void* p : {x, wg, wu, dh})
    if ((st = check_ptr(p))) return st;
  if (ws == nullptr) return SWIGLU_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return SWIGLU_ERR_ALIGN;
  if (ws_bytes < grouped_bwd_layout(dtype, R, E, N, K, src != nullptr).total) return SWIGLU_ERR_WORKSPACE;
  return SWIGLU_OK;
}

inline int validate_grouped_mm(int dtype, int64_t R, int64_t E, int64_t N, int64_t K, const void* x,
                               const void* offsets, const void* w, int64_t sw, const void* y) {
  int st = grouped_shape_status(dtype, R, E, N, K);
  if (st) return st;
  if ((st = check_expert_stride(dtype, E, N, K, sw))) return st;
  if (R == 0 || N == 0) return SWIGLU_OK;
  if ((st = check_int(offsets)) || (st = check_ptr(y))) return st;
  if (K == 0) return SWIGLU_OK;
  if ((st = check_ptr(x))) return st;
  return check_ptr(w);
}

inline int validate_grouped_mm_bwd(int dtype, int64_t R, int64_t E, int64_t N, int64_t K, const void* x,
                                   const void* offsets, const void* w, int64_t sw, const void* dy, const void* dx,
                                   const void* dw) {
  int st = grouped_shape_status(dtype, R, E, N, K);
  if (st) return st;
  if ((st = check_expert_stride(dtype, E, N, K, sw))) return st;
  if (!aligned(dx, 16) || !aligned(dw, 16)) return SWIGLU_ERR_ALIGN;
  if (K == 0 || (R == 0 && N == 0)) return SWIGLU_OK;
  if (dx == nullptr && dw == nullptr) return SWIGLU_ERR_NULL;
  if ((st = check_int(offsets))) return st;
  if (R == 0 || N == 0) return SWIGLU_OK;             // outputs are zero-filled
  if ((st = check_ptr(dy))) return st;
  if (dw != nullptr && (st = check_ptr(x))) return st;
  if (dx != nullptr && (st = check_ptr(w))) return st;
  return SWIGLU_OK;
}

inline size_t grouped_mm_bwd_workspace_total(int dtype, int64_t R, int64_t N, int64_t K) {
  return grouped_shape_status(dtype, R, 1, N, K) == SWIGLU_OK ? split_grads_bytes(dtype, R, 0, N, K, 1) : 0;
}
inline size_t grouped_mm_bwd_workspace_of(int dtype, int64_t R, int64_t E, int64_t N, int64_t K) {
  return grouped_shape_status(dtype, R, E, N, K) == SWIGLU_OK ? split_grads_bytes(dtype, R, E, N, K, 1) : 0;
}
inline int validate_grouped_mm_bwd_workspace(int dtype, int64_t R, int64_t E, int64_t N, int64_t K, const void* ws,
                                             size_t ws_bytes) {
  const size_t need = grouped_mm_bwd_workspace_of(dtype, R, E, N, K);
  if (need == 0) return SWIGLU_OK;
  if (ws == nullptr || ws_bytes < need) return SWIGLU_ERR_WORKSPACE;
  return aligned(ws, 256) ? SWIGLU_OK : SWIGLU_ERR_ALIGN;
}

// ---- gradient norm and clipping

// A chunk of a gradient is the work of one workgroup at a time; a launch takes
// the tensors that its arguments hold, 4 KiB at most.
constexpr int64_t kClipChunkBytes = 32768;
constexpr int kClipNormTensors = 320, kClipScaleTensors = 192;
constexpr int kClipBlocks = 2048;
constexpr int64_t kClipMaxElems = int64_t(1) << 35;

inline int64_t clip_norm_launches(int64_t count) {    // of each type at least one more
  return (count + kClipNormTensors - 1) / kClipNormTensors + 1;
}
inline size_t grad_norm_workspace_total(int64_t count) {
  if (count < 0 || count > (int64_t(1) << 20)) return 0;
  return 256 + (size_t)clip_norm_launches(count) * kClipBlocks * 8;
}

struct ByteRange { uintptr_t first, end; };

// Whether two of the ranges written to overlap (also: others that are written),
// or one that is written overlaps one that is read for another tensor (or its
// own, but for the same).
inline int check_disjoint(int64_t count, const int* dtypes, const void* const* grads, const int64_t* sizes,
                          void* const* outs, std::initializer_list<ByteRange> also = {}) {
  try {
    std::vector<ByteRange> w(also);
    w.reserve((size_t)count + also.size());
    auto range = [&](const void* p, int64_t i) {
      const uintptr_t a = reinterpret_cast<uintptr_t>(p);
      return ByteRange{a, a + (uintptr_t)(sizes[i] * elem_size(dtypes[i]))};
    };
    for (int64_t i = 0; i < count; ++i)
      if (sizes[i] > 0) w.push_back(range(outs != nullptr ? outs[i] : grads[i], i));
    std::sort(w.begin(), w.end(), [](const ByteRange& a, const ByteRange& b) { return a.first < b.first; });
    for (size_t i = 1; i < w.size(); ++i)
      if (w[i].first < w[i - 1].end) return SWIGLU_ERR_ARG;
    if (outs == nullptr) return SWIGLU_OK;
    for (int64_t i = 0; i < count; ++i) {
      if (sizes[i] == 0 || grads[i] == outs[i]) continue;
      const ByteRange g = range(grads[i], i);
      // The first written range that ends behind g's start.
      auto it = std::upper_bound(w.begin(), w.end(), g.first, [](uintptr_t v, const ByteRange& r) { return v < r.end; });
      if (it != w.end() && it->first < g.end) return SWIGLU_ERR_ARG;
    }
    return SWIGLU_OK;
  } catch (const std::bad_alloc&) {
    return SWIGLU_ERR_UNSUPPORTED;
  }
}

// clip: gradients are written (in place, or to outs).
inline int validate_grads(int64_t count, const int* dtypes, const void* const* grads, const int64_t* sizes,
                          void* const* outs, bool clip, double max_norm, double eps, const void* norm, const void* ws,
                          size_t ws_bytes) {
  if (count < 0 || count > (int64_t(1) << 20)) return SWIGLU_ERR_SHAPE;
  if (count > 0 && (dtypes == nullptr || grads == nullptr || sizes == nullptr)) return SWIGLU_ERR_NULL;
  int st;
  for (int64_t i = 0; i < count; ++i) {
    if ((st = check_dtype(dtypes[i]))) return st;
    if (sizes[i] < 0) return SWIGLU_ERR_SHAPE;
    if (sizes[i] > kClipMaxElems) return SWIGLU_ERR_UNSUPPORTED;
    if (sizes[i] == 0) continue;
    if (grads[i] == nullptr || (outs != nullptr && outs[i] == nullptr)) return SWIGLU_ERR_NULL;
    const uintptr_t es = (uintptr_t)elem_size(dtypes[i]);
    if (!aligned(grads[i], es) || (outs != nullptr && !aligned(outs[i], es))) return SWIGLU_ERR_ALIGN;
  }
  // max_norm and eps at least 0 and not NaN; an infinite max_norm clips nothing
  // (the factor is 1 whatever the norm, but for NaN).
  if (clip && (!(max_norm >= 0.0) || !(eps >= 0.0) || eps - eps != 0.0)) return SWIGLU_ERR_ARG;
  if ((st = check_int(norm))) return st;
  if (ws == nullptr || ws_bytes < grad_norm_workspace_total(count)) return SWIGLU_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return SWIGLU_ERR_ALIGN;
  if (!clip) return SWIGLU_OK;
  auto bytes = [](const void* p, size_t n) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return ByteRange{a, a + n};
  };
  return check_disjoint(count, dtypes, grads, sizes, outs,
                        {bytes(norm, sizeof(float)), bytes(ws, grad_norm_workspace_total(count))});
}

}  // namespace swg
