// Host-side argument validation and workspace layout for the C ABI.
// Pure C++ (no HIP), so it can be compiled and tested without a GPU.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

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

}  // namespace swg
