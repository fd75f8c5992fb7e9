// The routed SwiGLU MLP for a few tokens (bf16, at most 64):
//   y[t] = sum_j w[t, j] * Wd_e (act(Wg_e x[t]) * (Wu_e x[t])),  e = ids[t, j].
//
// The work is bound by reading the weights of the experts in use from HBM
// once, so both kernels stream weights as the dense decode kernel does
// (gemv.hip): a wave loads a slab of 16 weight rows x 128 coalesced (256
// contiguous bytes of a row per quarter-wave), passes it through a
// wave-private LDS tile into the operand layout of v_mfma_f32_16x16x32_bf16
// and multiplies it with the expert's tokens, up to 16 at a time.  A wave
// requests its next slab's weights before it multiplies the present one, and
// that slab's token operands (from L2) after it, into the registers it has
// just used: loads complete in order, so they arrive with the weights.
//
// moe_up_kernel: h = act(Wg_e x) * (Wu_e x) of each (token, expert), kept as
//   two bf16 rows (h = hi + lo, 16 significant bits: rounding h to one bf16
//   would cost as much as the rounding of y; against an fp32 h 0.25 to 0.5 %
//   of y round the other way, and the error against fp64, 1.66e-3 normwise, is
//   the same to five digits).  A workgroup takes an equal
//   share of the (expert in use, 16-row tile) sequence; its waves split the
//   reduction and meet in LDS at the end of each tile, with the next tile's
//   slab already requested.
// moe_down_kernel: y.  A workgroup takes 8, 16 or 32 columns of y over all
//   experts in use (or, where that leaves CUs without work, over one of S
//   equal parts), its waves equal shares of the (expert, slab) sequence;
//   hi and lo are two of the 16 token columns of one product, 8 tokens at a
//   time, so they cost no second product; at the end of an expert the two
//   are added, weighted and added to the wave's own fp32 y in LDS.  The
//   waves' y are added in wave order.  Only with S > 1 do partial sums leave
//   the workgroup, for moe_sum_kernel to add in order.  The order of every sum
//   is fixed, and y is rounded once.
//
// Measured, of the weights' bytes: 8 tokens, two of 8 x (11008, 4096) each,
// 1.30 GB in 198 us (6.5 TB/s) and 649 MB in 105 (6.2); 64 tokens, 8 of
// 64 x (1024, 2048), 537 MB in 90 us (6.0) and 268 MB in 51 (5.2), 5 for the
// sum; one token, two of 8 x (6912, 1536), 85 MB in 18 us and 42 MB in 14, of
// which 6 and 4 are launch, routing and the first loads' latency.  Without
// token operands the streams of the 64 tokens take 82 and 49 us.  Far from the
// read rate: rows that are not whole lines, 56 x (5256, 616) with 4 tokens each
// 725 MB in 185 us (3.9) and 363 in 82 (4.4); many tokens, 13 x (3456, 2304)
// with 15 each 414 MB in 104 (4.0) and 207 in 55 (3.8).
//
// Which experts are in use, and by which tokens, every workgroup finds from
// ids itself: from up to 64 ids without LDS or barriers (kFew), from up to
// 1024 through a token mask per expert in LDS (set with atomic or, whose order
// makes no difference).
#include "block.hpp"
#include "common.hpp"
#include "validate.hpp"

namespace swg {

namespace {

constexpr int kSlabK = 128;                      // reduction elements per slab of 16 rows
constexpr int kCPR = kSlabK / 8;                 // 16-byte chunks per row per slab
constexpr int kInst = 4;                         // load instructions per slab and weight (1 KiB each)
constexpr int kSteps = kSlabK / 32;              // MFMA steps per slab of 16 rows
constexpr int kTile = 256;                       // 16-byte chunks of a slab
constexpr int kMaxTokens = 64, kMaxPairs = 64 * 16, kMaxExperts = 1024;

// Waits for this wave's LDS operations and joins the workgroup, without
// waiting for global loads in flight (__syncthreads waits for those too).
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);            // lgkmcnt(0), other counters free
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

__device__ __forceinline__ int nth_set_bit(uint64_t m, int n) {
  int at = 0;
#pragma unroll
  for (int half = 32; half >= 1; half >>= 1) {
    const int c = __popcll(m & ((1ull << half) - 1));
    if (n >= c) {
      n -= c;
      m >>= half;
      at += half;
    }
  }
  return at;
}

// The sequence of (expert in use, pass) and who uses the expert.  A pass
// takes at most kCap of an expert's tokens; an expert with more has several,
// each of which reads its weights again.  All values are the same in every
// lane unless said otherwise.  kPairs: with the pairs' ids and weights (id_of,
// weight_of), which the first product does not need.
template <bool kFew, int kCap, bool kPairs> struct Route;

// Passes of n tokens.
template <int kCap> __device__ __forceinline__ int passes_of(int n) { return (n + kCap - 1) / kCap; }

// Per lane: the sum of v over this lane and those before it.
__device__ __forceinline__ int running_sum(int v, int lane) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(v, off);
    if (lane >= off) v += o;
  }
  return v;
}

// Of the lanes' counts, the lane where the running sum passes n, and n less
// the sum before that lane (-1: the counts sum to n or less).  `sum` is their
// total.
__device__ __forceinline__ int lane_of(int count, int lane, int& n, int& sum) {
  const int incl = running_sum(count, lane);
  sum = __builtin_amdgcn_readlane(incl, 63);
  const uint64_t past = __ballot(incl > n);
  if (past == 0) return -1;
  const int at = __ffsll((unsigned long long)past) - 1;
  n -= __builtin_amdgcn_readlane(incl - count, at);
  return at;
}

// Up to 64 (token, choice) pairs: lane p holds the id of pair p, and, where p
// is the first pair that names its expert, the expert's passes.
template <int kCap, bool kPairs> struct Route<true, kCap, kPairs> {
  struct Shared {};
  int id, k, T, lane;
  int passes, before;                            // per lane: of its expert; tokens of the experts before it
  float weight;                                  // per lane: of pair `lane`
  uint64_t first;                                // lanes with passes
  __device__ __forceinline__ void init(Shared&, const MoeArgs& a, int tid) {
    const int pairs = a.T * a.k;
    lane = tid & 63;
    k = a.k;
    T = a.T;
    id = lane < pairs ? a.ids[lane] : -1;
    weight = kPairs && lane < pairs ? a.weights[lane] : 0.0f;
    if (id < 0 || id >= a.E) id = -1;
    uint64_t same = ~0ull;                       // lanes with this lane's id
#pragma unroll
    for (int b = 0; b < 10; ++b) {
      const uint64_t m = __ballot((id >> b) & 1);
      same &= (id >> b) & 1 ? m : ~m;
    }
    same &= __ballot(id >= 0);
    const uint64_t earlier = (1ull << lane) - 1;
    const bool is_first = id >= 0 && (same & earlier) == 0;
    first = __ballot(is_first);
    // Tokens of the expert: a token that names it again counts once, so that no pass is without tokens.
    const uint64_t of_token = ((1ull << k) - 1) << (lane / k * k);   // the pairs of this lane's token
    const uint64_t once = __ballot(id >= 0 && (same & of_token & earlier) == 0);
    const int n = is_first ? __popcll(same & once) : 0;
    passes = passes_of<kCap>(n);
    before = running_sum(n, lane) - n;
  }
  __device__ __forceinline__ int count() const {
    if (kCap >= kMaxTokens) return __popcll(first);
    int n = 64 * kMaxTokens, sum;
    lane_of(passes, lane, n, sum);
    return sum;
  }
  struct At { int pair, pass; };
  __device__ __forceinline__ At at(int slot) const {   // slot < count()
    if (kCap >= kMaxTokens) return At{nth_set_bit(first, slot), 0};
    int sum;
    const int p = lane_of(passes, lane, slot, sum);
    return At{p, slot};
  }
  __device__ __forceinline__ int expert(const At& p) const { return __builtin_amdgcn_readlane(id, p.pair); }
  __device__ __forceinline__ int base(const At& p) const { return __builtin_amdgcn_readlane(before, p.pair); }
  __device__ __forceinline__ void next(At& p) const {
    if (kCap < kMaxTokens && ++p.pass < __builtin_amdgcn_readlane(passes, p.pair)) return;
    const uint64_t rest = p.pair < 63 ? first >> (p.pair + 1) : 0;
    p.pair = rest == 0 ? 0 : p.pair + __ffsll((unsigned long long)rest);
    p.pass = 0;
  }
  // Tokens that name e.
  __device__ __forceinline__ uint64_t tokens(int e) const {
    const uint64_t pairs = __ballot(id == e);
    bool in = false;
    if (lane < T) in = (pairs >> (lane * k) & ((k < 64 ? 1ull << k : 0ull) - 1)) != 0;
    return __ballot(in);
  }
  __device__ __forceinline__ int id_of(int pair) const { return __shfl(id, pair); }
  __device__ __forceinline__ float weight_of(int pair) const { return __shfl(weight, pair); }
};

template <bool kPairs> struct PairsOf {
  int ids[kMaxPairs];
  float weights[kMaxPairs];
};
template <> struct PairsOf<false> {};

template <int kCap, bool kPairs> struct Route<false, kCap, kPairs> {
  struct Shared : PairsOf<kPairs> {
    uint32_t mask[kMaxExperts][2];               // tokens of each expert
  };
  const Shared* s;
  int E, lane;
  __device__ __forceinline__ void init(Shared& sh, const MoeArgs& a, int tid) {
    s = &sh;
    E = a.E;
    lane = tid & 63;
    for (int e = tid; e < a.E; e += blockDim.x) sh.mask[e][0] = sh.mask[e][1] = 0;
    __syncthreads();
    for (int p = tid; p < a.T * a.k; p += blockDim.x) {
      const int id = a.ids[p], t = p / a.k;
      if constexpr (kPairs) {
        sh.ids[p] = id;
        sh.weights[p] = a.weights[p];
      }
      if (id >= 0 && id < a.E) atomicOr(&sh.mask[id][t >> 5], 1u << (t & 31));
    }
    __syncthreads();
  }
  // Passes of expert base + lane (per lane).
  __device__ __forceinline__ int passes(int base) const {
    const int e = base + lane;
    return e < E ? passes_of<kCap>(__popc(s->mask[e][0]) + __popc(s->mask[e][1])) : 0;
  }
  __device__ __forceinline__ int count() const {
    int n = 0;
    for (int b = 0; b < E; b += 64) {
      int huge = 64 * kMaxTokens, sum;
      lane_of(passes(b), lane, huge, sum);
      n += sum;
    }
    return n;
  }
  struct At { int e, pass, before; };
  __device__ __forceinline__ At at(int slot) const {   // slot < count()
    int before = 0;                              // tokens of the experts before, expert by expert
    for (int b = 0;; b += 64) {
      const int e = b + lane, n = e < E ? __popc(s->mask[e][0]) + __popc(s->mask[e][1]) : 0;
      const int incl = running_sum(n, lane);
      int sum;
      const int l = lane_of(passes(b), lane, slot, sum);
      if (l >= 0) return At{b + l, slot, before + __builtin_amdgcn_readlane(incl - n, l)};
      slot -= sum;
      before += __builtin_amdgcn_readlane(incl, 63);
    }
  }
  __device__ __forceinline__ int expert(const At& p) const { return p.e; }
  __device__ __forceinline__ int base(const At& p) const { return p.before; }
  __device__ __forceinline__ void next(At& p) const {
    const int n = __popcll(tokens(p.e));
    if (kCap < kMaxTokens && ++p.pass < passes_of<kCap>(n)) return;
    p.pass = 0;
    p.before += n;
    // The next expert with tokens: in the rest of its 64, then 64 at a time.
    for (int from = p.e + 1; from < E; from = (from & ~63) + 64) {
      const int base = from & ~63;
      const uint64_t used = __ballot(passes(base) != 0) >> (from - base);
      if (used != 0) {
        p.e = from + __ffsll((unsigned long long)used) - 1;
        return;
      }
    }
  }
  __device__ __forceinline__ uint64_t tokens(int e) const {
    return (uint64_t)s->mask[e][1] << 32 | s->mask[e][0];
  }
  __device__ __forceinline__ int id_of(int pair) const { return s->ids[pair]; }
  __device__ __forceinline__ float weight_of(int pair) const { return s->weights[pair]; }
};

// The token of row r of the expert's list (-1 past its end).
__device__ __forceinline__ int token_of(uint64_t tokens, int r) {
  return r < __popcll(tokens) ? nth_set_bit(tokens, r) : -1;
}

// h of row r of an expert's list lies in entry base + r (base: the entries of
// the experts before it), chunk by chunk with the entries of a chunk side by
// side, hi then lo: [N / 8][entries][2] chunks of 8.  The 16 token columns of
// one chunk are then 256 contiguous bytes.  (Entry by entry, [entries][2][N],
// the 16 columns of N = 1024 lie 2 KiB apart, on two of an L2's 16 channels:
// 64 tokens of 64 x (1024, 2048) took 37 us longer.)
__device__ __forceinline__ int64_t h_chunk(int c, int entries, int entry, int half) {
  return ((int64_t)c * entries + entry) * 2 + half;
}

// kRows weight rows (8 or 16); a slab is 128 * kQ of the reduction,
// kQ = 16 / kRows.  Load instruction i covers rows 4 i + lane / 16 of the
// slab's piece i / (kRows / 4).
template <int kRows> constexpr int kPieces = 16 / kRows;

// The token operands of slab s: chunk c of this lane's column g lies at
// b4[brow[g] * row_step + c * step]; zero where brow[g] < 0.
struct Tokens {
  const u32x4* b4;
  int row_step, step;
};
template <int kQ, int kG>
__device__ __forceinline__ void load_tokens(u32x4 (&v)[kG][kSteps * kQ], const Tokens& x, const int (&brow)[kG],
                                            int groups, int s, int nch, int lane) {
#pragma unroll
  for (int g = 0; g < kG; ++g) {
    if (g > 0 && g >= groups) break;
#pragma unroll
    for (int j = 0; j < kSteps * kQ; ++j) {
      const int c = s * kQ * kCPR + 4 * j + (lane >> 4);
      v[g][j] = brow[g] >= 0 && c < nch ? x.b4[(int64_t)brow[g] * x.row_step + (int64_t)c * x.step]
                                        : u32x4{0u, 0u, 0u, 0u};
    }
  }
}

// A wave's slab in flight: 4 KiB of each of kW weights.  Rows of whole
// 128-byte lines are read once and bypass the caches; in others neighbouring
// slabs share a line, which the bypass would read from HBM twice (1.4 times
// the bytes at K = 1160).
// The tiles are of kW weights, or of one weight, kRows rows after each other (kDown).
template <int kRows, int kW, bool kDown>
__device__ __forceinline__ void load_slab(u32x4 (&v)[kW][kInst], const u32x4* const (&w4)[kW], int n0, int rows, int s,
                                          int nch, int lane) {
  constexpr int kQ = kPieces<kRows>;
  const u32x4 zero = {0u, 0u, 0u, 0u};
  const int lc = lane % kCPR, lr = lane / kCPR;
  auto load = [&](auto get) {
#pragma unroll
    for (int i = 0; i < kInst; ++i) {
      const int n = n0 + (i % (kRows / 4)) * 4 + lr, c = (s * kQ + i / (kRows / 4)) * kCPR + lc;
      if constexpr (kDown) {
#pragma unroll
        for (int w = 0; w < kW; ++w) {
          const bool in = n + w * kRows < rows && c < nch;
          v[w][i] = in ? get(w4[w] + (in ? (int64_t)n * nch + c : 0)) : zero;
        }
      } else {
        const bool in = n < rows && c < nch;
        const int64_t off = in ? (int64_t)n * nch + c : 0;
#pragma unroll
        for (int w = 0; w < kW; ++w) v[w][i] = in ? get(w4[w] + off) : zero;
      }
    }
  };
  if (nch % 8 == 0) load([](const u32x4* p) { return __builtin_nontemporal_load(p); });
  else load([](const u32x4* p) { return *p; });
}

// Row r, chunk c of a 16-chunk piece sits at chunk c ^ (r & 15): the 16 lanes
// that write one row and the 16 that read one chunk of 16 rows each hit 16
// distinct 16-byte bank groups.
template <int kRows, int kW>
__device__ __forceinline__ void to_tile(const u32x4 (&v)[kW][kInst], u32x4* tile, int lane) {
  const int lc = lane % kCPR, lr = lane / kCPR;
#pragma unroll
  for (int i = 0; i < kInst; ++i) {
    const int r = (i % (kRows / 4)) * 4 + lr, piece = i / (kRows / 4);
#pragma unroll
    for (int w = 0; w < kW; ++w) tile[w * kTile + (piece * kRows + r) * kCPR + (lc ^ r)] = v[w][i];
  }
}

// The slab in the tile times the token columns.
template <int kRows, int kW, int kG>
__device__ __forceinline__ void multiply(const u32x4* tile, const u32x4 (&b)[kG][kSteps * kPieces<kRows>], int groups,
                                         int lane, f32x4 (&acc)[kW][kG]) {
  const int r = (lane & 15) % kRows, q4 = lane >> 4;
#pragma unroll
  for (int j = 0; j < kSteps * kPieces<kRows>; ++j) {
    const int pc = (4 * (j % kSteps) + q4) ^ r;
    u32x4 w[kW];
#pragma unroll
    for (int i = 0; i < kW; ++i) w[i] = tile[i * kTile + ((j / kSteps) * kRows + r) * kCPR + pc];
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      if (g > 0 && g >= groups) break;
#pragma unroll
      for (int i = 0; i < kW; ++i)
        acc[i][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w[i]),
                                                            __builtin_bit_cast(bf16x8, b[g][j]), acc[i][g], 0, 0, 0);
    }
  }
}

// ---------------------------------------------------------------- first product

constexpr int kUpWaves = 8;
// Waves per SIMD: the operands of more token groups take more registers.
template <int kG> constexpr int kUpOcc = kG == 1 ? 4 : kG == 2 ? 3 : 2;
template <bool kFew, int kG> using UpRoute = Route<kFew, 16 * kG, false>;

template <Act A, bool kFew, int kG>
__global__ __launch_bounds__(kUpWaves * 64, kUpOcc<kG>) void moe_up_kernel(MoeArgs a) {
  extern __shared__ u32x4 lds[];
  using R = UpRoute<kFew, kG>;
  __shared__ typename R::Shared shared;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nw = blockDim.x >> 6, r16 = lane & 15, q4 = lane >> 4;
  R route;
  route.init(shared, a, tid);
  // This workgroup's share of the (pass, tile) sequence.
  const int ntiles = (a.N + 15) / 16;
  const int64_t total = (int64_t)route.count() * ntiles;
  int64_t u = (int64_t)blockIdx.x * total / gridDim.x;
  const int64_t u1 = (int64_t)(blockIdx.x + 1) * total / gridDim.x;
  if (u >= u1) return;
  auto at = route.at((int)(u / ntiles));
  int t = (int)(u % ntiles);

  const int nch = a.K >> 3, nslab = (nch + kCPR - 1) / kCPR;
  // The expert being multiplied: its tokens, and this lane's rows of x.
  int e = __builtin_amdgcn_readfirstlane(route.expert(at)), first, base, groups, row[kG];
  uint64_t tokens;
  auto enter = [&] {
    tokens = route.tokens(e);
    first = at.pass * 16 * kG;
    base = route.base(at);
    groups = min(kG, (__popcll(tokens) - first + 15) / 16);
#pragma unroll
    for (int g = 0; g < kG; ++g) row[g] = token_of(tokens, first + 16 * g + r16);
  };
  const u32x4* w4[2];                            // of the expert whose slab is in flight
  auto weights_of = [&](int expert) {
    w4[0] = reinterpret_cast<const u32x4*>(static_cast<const bf16*>(a.wg) + expert * a.wg_stride);
    w4[1] = reinterpret_cast<const u32x4*>(static_cast<const bf16*>(a.wu) + expert * a.wu_stride);
  };
  const Tokens x{static_cast<const u32x4*>(a.x), nch, 1};
  u32x4* tile = lds + wave * 2 * kTile;
  // This wave's slabs of each tile: a run of them, or where rows are not whole
  // lines every nw-th, so that the waves read neighbouring slabs at the same
  // time and the lines that two of them share are fetched once: K = 1720, 8
  // tokens of 32 experts, 72 us against 81 (1.05 and 1.34 times the bytes).
  // With whole lines runs are as fast or faster (K = 2048: 6 us of 137).
  const bool lines = nch % 8 == 0;
  const int s0 = lines ? wave * nslab / nw : wave, s1 = lines ? (wave + 1) * nslab / nw : nslab, ds = lines ? 1 : nw;
  f32x4 acc[2][kG];
  auto clear = [&] {
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int g = 0; g < kG; ++g) acc[w][g] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  };
  clear();
  weights_of(e);
  u32x4 v[2][kInst], b[kG][kSteps];
  if (s0 < s1) load_slab<16, 2, false>(v, w4, t * 16, a.N, s0, nch, lane);
  enter();
  if (s0 < s1) load_tokens<1>(b, x, row, groups, s0, nch, lane);
  for (; u < u1; ++u) {
    const bool more = u + 1 < u1, other = t + 1 == ntiles;   // another tile; of another pass
    const int t2 = other ? 0 : t + 1;
    int e2 = e;
    if (more && other) {
      route.next(at);
      e2 = __builtin_amdgcn_readfirstlane(route.expert(at));
    }
    for (int s = s0; s < s1; s += ds) {
      const bool within = s + ds < s1;           // the next slab is of this tile
      to_tile<16, 2>(v, tile, lane);
      if (within) {
        load_slab<16, 2, false>(v, w4, t * 16, a.N, s + ds, nch, lane);
      } else if (more) {
        if (other) weights_of(e2);
        load_slab<16, 2, false>(v, w4, t2 * 16, a.N, s0, nch, lane);
      }
      multiply<16, 2, kG>(tile, b, groups, lane, acc);
      if (within || (more && !other)) load_tokens<1>(b, x, row, groups, within ? s + ds : s0, nch, lane);
    }
    // The waves' sums in wave order: group g and weight w by wave 2 g + w % nw.
    lds_barrier();                               // every wave is done with its tile
    f32x4* red = reinterpret_cast<f32x4*>(lds);  // [kG][2][wave][lane]
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      if (g >= groups) break;
#pragma unroll
      for (int w = 0; w < 2; ++w) red[((g * 2 + w) * nw + wave) * 64 + lane] = acc[w][g];
    }
    clear();
    lds_barrier();
    for (int g = wave; g < groups; g += nw) {
      f32x4 sum[2];
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        sum[w] = red[((g * 2 + w) * nw) * 64 + lane];
        for (int o = 1; o < nw; ++o) sum[w] += red[((g * 2 + w) * nw + o) * 64 + lane];
      }
      // Lane l element i: weight row 16 t + 4 (l / 16) + i of token row l % 16.
      const int at_row = first + 16 * g + r16, nb = t * 16 + 4 * q4;
      if (at_row < __popcll(tokens) && nb < a.N) {               // N % 8 == 0: four columns lie inside or outside together
        uint16_t hi[4], lo[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float z = sum[0][q];
          const float h = (A == Act::kGeluTanh ? gelu_tanh_f32(z) : silu_f32(z)) * sum[1][q];
          const bf16 b = to_bf16(h);
          const float f = from_bf16(b);
          hi[q] = __builtin_bit_cast(uint16_t, b);
          lo[q] = __builtin_bit_cast(uint16_t, to_bf16(fabsf(f) < __builtin_inff() ? h - f : 0.0f));
        }
        bf16* h = static_cast<bf16*>(a.h) + h_chunk(nb >> 3, a.T * a.k, base + at_row, 0) * 8 + (nb & 7);
        *reinterpret_cast<u32x2*>(h) = __builtin_bit_cast(u32x2, hi);
        *reinterpret_cast<u32x2*>(h + 8) = __builtin_bit_cast(u32x2, lo);
      }
    }
    lds_barrier();                               // the sums are read before the next tile is written
    t = t2;
    if (more && other) {
      e = e2;
      enter();
      if (s0 < s1) load_tokens<1>(b, x, row, groups, s0, nch, lane);
    }
  }
}

// --------------------------------------------------------------- second product

// kCols columns of y: tiles of 8 or 16 weight rows, two of 16 for 32.
template <int kCols> constexpr int kTileRows = kCols < 16 ? kCols : 16;
// Waves: the operands of more token groups take more registers, and the
// waves' y of 32 columns more LDS.
template <int kG> constexpr int kDownWaves = kG == 1 ? 16 : 8;
// Waves that fit a CU by their registers.
template <int kG> constexpr int kDownCuWaves = kG <= 2 ? 16 : 8;
template <bool kFew, int kG> using DownRoute = Route<kFew, 8 * kG, true>;

template <bool kFew, int kG, int kCols>
__global__ __launch_bounds__((kDownWaves<kG> * 64)) void moe_down_kernel(MoeArgs a) {
  constexpr int kRows = kTileRows<kCols>, kT = kCols / kRows, kQ = kPieces<kRows>;
  extern __shared__ u32x4 lds[];
  using R = DownRoute<kFew, kG>;
  __shared__ typename R::Shared shared;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nw = blockDim.x >> 6, r16 = lane & 15, q4 = lane >> 4;
  u32x4* tile = lds + wave * kT * kTile;
  float* ys = reinterpret_cast<float*>(lds + nw * kT * kTile);   // [wave][T][kCols]
  for (int i = tid; i < nw * a.T * kCols; i += blockDim.x) ys[i] = 0.0f;
  R route;
  route.init(shared, a, tid);
  __syncthreads();
  float* mine = ys + wave * a.T * kCols;

  const int n0 = blockIdx.x * kCols, nch = a.N >> 3, nslab = (nch + kQ * kCPR - 1) / (kQ * kCPR);
  // Neighbouring workgroups go through an expert's slabs from different ones
  // on: from slab 0 all of them would read the same 256 of every N * 2 bytes
  // at a time, which for a power of two is a few of the memory channels.
  const int turn = nch % 8 == 0 ? blockIdx.x % nslab : 0;
  auto slab = [&](int s) { return s + turn < nslab ? s + turn : s + turn - nslab; };
  const Tokens x{static_cast<const u32x4*>(a.h), 1, 2 * a.T * a.k};
  const int r8 = lane & 7, half = r16 >> 3;      // token column r16: token r8 of a group of 8, its hi or lo row
  // This wave's share of this workgroup's part of the (pass, slab) sequence.
  const int total = route.count() * nslab;
  const int p0 = (int)((int64_t)blockIdx.y * total / gridDim.y);
  const int p1 = (int)((int64_t)(blockIdx.y + 1) * total / gridDim.y);
  int u = p0 + (int)((int64_t)wave * (p1 - p0) / nw);
  const int u1 = p0 + (int)((int64_t)(wave + 1) * (p1 - p0) / nw);
  if (u < u1) {
    auto at = route.at(u / nslab);
    int s = u % nslab;
    // The expert being multiplied: its tokens, and this lane's entries of h.
    int e, first, groups, row[kG];
    uint64_t tokens;
    const u32x4* w4[kT];
    auto enter = [&] {
      tokens = route.tokens(e);
      first = at.pass * 8 * kG;
      groups = min(kG, (__popcll(tokens) - first + 7) / 8);
#pragma unroll
      for (int g = 0; g < kG; ++g) {
        const int r = first + 8 * g + r8;
        row[g] = r < __popcll(tokens) ? (route.base(at) + r) * 2 + half : -1;
      }
    };
    auto weights_of = [&](int expert) {
      w4[0] = reinterpret_cast<const u32x4*>(static_cast<const bf16*>(a.wd) + expert * a.wd_stride);
#pragma unroll
      for (int i = 1; i < kT; ++i) w4[i] = w4[0] + (int64_t)kRows * i * nch;
    };
    e = __builtin_amdgcn_readfirstlane(route.expert(at));
    weights_of(e);
    u32x4 v[kT][kInst], b[kG][kSteps * kQ];
    load_slab<kRows, kT, true>(v, w4, n0, a.K, slab(s), nch, lane);
    enter();
    load_tokens<kQ>(b, x, row, groups, slab(s), nch, lane);
    f32x4 acc[kT][kG];
#pragma unroll
    for (int i = 0; i < kT; ++i)
#pragma unroll
      for (int g = 0; g < kG; ++g) acc[i][g] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (; u < u1; ++u) {
      to_tile<kRows, kT>(v, tile, lane);
      const bool last = s + 1 == nslab, more = u + 1 < u1;   // of this pass; of this wave
      int e2 = e;
      if (more) {
        if (last) {
          route.next(at);
          e2 = __builtin_amdgcn_readfirstlane(route.expert(at));
          weights_of(e2);
        }
        load_slab<kRows, kT, true>(v, w4, n0, a.K, slab(last ? 0 : s + 1), nch, lane);
      }
      multiply<kRows, kT, kG>(tile, b, groups, lane, acc);
      ++s;
      if (last || !more) {                       // weighted, into this wave's y
#pragma unroll
        for (int g = 0; g < kG; ++g) {
          if (g >= groups) break;
          const int t = token_of(tokens, first + 8 * g + r8);
          float w = 0.0f;
          for (int j = 0; j < a.k; ++j) {
            const int p = t < 0 ? 0 : t * a.k + j;
            const float wj = route.weight_of(p);
            w += route.id_of(p) == e ? wj : 0.0f;
          }
#pragma unroll
          for (int i = 0; i < kT; ++i) {
            f32x4 o = acc[i][g];
#pragma unroll
            for (int q = 0; q < 4; ++q) o[q] += __shfl_xor(o[q], 8);   // hi + lo
            // Rows 4 q4 .. + 3 of the tile; with 8 rows the upper half repeats the lower.
            if (t >= 0 && half == 0 && 4 * q4 < kRows) {
              f32x4* y = reinterpret_cast<f32x4*>(mine + t * kCols + 16 * i + 4 * q4);
              f32x4 sum = *y;
#pragma unroll
              for (int q = 0; q < 4; ++q) sum[q] = __builtin_fmaf(w, o[q], sum[q]);
              *y = sum;
            }
            acc[i][g] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
          }
        }
        if (more) {
          e = e2;
          s = 0;
          enter();
        }
      }
      if (more) load_tokens<kQ>(b, x, row, groups, slab(s), nch, lane);
    }
  }
  __syncthreads();
  for (int i = tid; i < a.T * kCols; i += blockDim.x) {
    float y = ys[i];
    for (int w = 1; w < nw; ++w) y += ys[w * a.T * kCols + i];
    const int t = i / kCols, c = n0 + i % kCols;
    if (c >= a.K) continue;
    if (gridDim.y == 1) static_cast<bf16*>(a.y)[(int64_t)t * a.K + c] = to_bf16(y);
    else a.part[((int64_t)blockIdx.y * a.T + t) * a.K + c] = y;
  }
}

// y from the S parts, four columns to a thread (K % 8 == 0).
__global__ __launch_bounds__(256) void moe_sum_kernel(MoeArgs a, int parts) {
  const int i = (blockIdx.x * 256 + threadIdx.x) * 4, n = a.T * a.K;
  if (i >= n) return;
  f32x4 y = *reinterpret_cast<const f32x4*>(a.part + i);
  for (int p = 1; p < parts; ++p) y += *reinterpret_cast<const f32x4*>(a.part + (int64_t)p * n + i);
  uint16_t o[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) o[q] = __builtin_bit_cast(uint16_t, to_bf16(y[q]));
  *reinterpret_cast<u32x2*>(static_cast<bf16*>(a.y) + i) = __builtin_bit_cast(u32x2, o);
}

// ---------------------------------------------------------------------- launch

template <Act A, bool kFew, int kG>
hipError_t launch_up(const MoeArgs& a, hipStream_t s) {
  const int slots = a.E < a.T * a.k ? a.E : a.T * a.k;
  const int nslab = (a.K / 8 + kCPR - 1) / kCPR, ntiles = (a.N + 15) / 16;
  // Tiles (8 KiB a wave) or sums (2 kG KiB a wave).
  auto lds_of = [](int n) { return (size_t)n * 64 * 16 * (2 * kG > 8 ? 2 * kG : 8); };
  // As many workgroups as are resident at once by their registers and LDS
  // (256 CUs), or as there can be tiles (a second pass of an expert lengthens
  // the shares, it adds no workgroups).  4 to 8 waves (a slab each at most):
  // those with the shortest chain of slabs, tiles per workgroup times slabs
  // per wave.  At 2 x 432 tiles of 12 slabs 4 waves (1 x 3) take 19.6 us, 6
  // (2 x 2) 20.6.  LDS is what binds from 65 pairs on, and a workgroup more
  // than it holds is a second round: 64 tokens of 64 x (256, 1536), four of 40
  // KiB to a CU, 22.5 us; with the pairs' ids and weights in it too (48 KiB,
  // three to a CU) 27.6.
  const int64_t tiles = (int64_t)ntiles * slots;
  int nw = 0;
  int64_t resident = 0, best = 0;
  for (int n = nslab < kUpWaves ? nslab : kUpWaves; n >= 4 || nw == 0; --n) {
    const int64_t res = 256 * moe_resident(n, 4 * kUpOcc<kG>, lds_of(n) + sizeof(typename UpRoute<kFew, kG>::Shared));
    const int64_t chain = (tiles + res - 1) / res * ((nslab + n - 1) / n);
    if (nw == 0 || chain < best) {
      nw = n;
      resident = res;
      best = chain;
    }
  }
  const hipError_t e = allow_lds<&moe_up_kernel<A, kFew, kG>>(lds_of(kUpWaves));
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((moe_up_kernel<A, kFew, kG>), dim3((unsigned)(tiles < resident ? tiles : resident)),
                     dim3(nw * 64), lds_of(nw), s, a);
  return hipGetLastError();
}

template <bool kFew, int kG, int kCols>
hipError_t launch_down(const MoeArgs& a, hipStream_t s) {
  constexpr int kMost = kDownWaves<kG>, kT = kCols / kTileRows<kCols>;
  const int blocks = (a.K + kCols - 1) / kCols;
  // As many waves as the registers allow, or two workgroups of 8 per CU where
  // there are enough of them.
  const int nw = blocks > 256 ? 8 : kMost;
  constexpr size_t most = (size_t)kMost * (kT * kTile * 16 + kMaxTokens * kCols * 4);
  const size_t lds = (size_t)nw * (kT * kTile * 16 + a.T * kCols * 4);
  // Parts: as many as shorten the waves' chain of slabs, over all rounds of
  // the workgroups that fit the CUs, by more than the sum of the parts takes,
  // about three slabs' time (4.5 us).
  int parts = 1;
  if (kCols >= 16) {
    const int per_cu = moe_resident(nw, kDownCuWaves<kG>, lds + sizeof(typename DownRoute<kFew, kG>::Shared));
    const int slots = a.E < a.T * a.k ? a.E : a.T * a.k;
    const int64_t units = (int64_t)slots * ((a.N / 8 + kCPR - 1) / kCPR);
    auto chain = [&](int64_t p) {
      return ((blocks * p + 256 * per_cu - 1) / (256 * per_cu)) * ((units + p * nw - 1) / (p * nw)) + (p > 1 ? 3 : 0);
    };
    for (int p = 2; p <= moe_parts(a.K, kCols); ++p)
      if (chain(p) < chain(parts)) parts = p;
  }
  hipError_t e = allow_lds<&moe_down_kernel<kFew, kG, kCols>>(most);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((moe_down_kernel<kFew, kG, kCols>), dim3(blocks, parts), dim3(nw * 64), lds, s, a);
  if ((e = hipGetLastError()) != hipSuccess || parts == 1) return e;
  hipLaunchKernelGGL(moe_sum_kernel, dim3((a.T * a.K / 4 + 255) / 256), dim3(256), 0, s, a, parts);
  return hipGetLastError();
}

template <bool kFew, int kG>
hipError_t launch_up_act(Act act, const MoeArgs& a, hipStream_t s) {
  return act == Act::kGeluTanh ? launch_up<Act::kGeluTanh, kFew, kG>(a, s) : launch_up<Act::kSilu, kFew, kG>(a, s);
}

// Columns of y to a workgroup, by the token groups of a pass.
// kG 2 and 4 (more than 8 tokens, 4 or more per expert): 32.  A slab's token
//   operands are as many bytes per 8 tokens as its weights for 16 columns.  The
//   whole call, 32 against 16: 48 tokens of 13 x (3456, 2304), 4 each, 174 us
//   against 191; 64 of 64 x (1024, 4096), 8 each, 258 against 279; 64 of 64 x
//   (1024, 2048), 8 each, the same.
// kG 1: 16, or with fewer than 4 tokens per expert 8, where 16 would need a
//   split and 8 do not: at K = 2048 with 2 tokens per expert the kernel takes
//   46 us against 49 (with the parts' sum).
// kG 8 (over 32 tokens, 17 or more per expert): 16; with 32 the kernel takes,
//   parts' sum included, 47 us against 53 at 64 tokens of 8 x (2048, 4096),
//   4 each, 50 against 61 at 8 x (8192, 1024).
template <bool kFew, int kG>
hipError_t launch_down_cols(const MoeArgs& a, hipStream_t s) {
  if constexpr (kG == 1)
    if (moe_parts(a.K, 16) > 1 && a.K > 8 * kMoeFullBlocks && a.T * a.k < 4 * a.E) return launch_down<kFew, 1, 8>(a, s);
  return launch_down<kFew, kG, kG == 2 || kG == 4 ? 32 : 16>(a, s);
}

// Tokens of one expert that a pass takes: all that there can be where T is
// small, otherwise at least about twice as many as an expert has on average
// (T k / E), so that few experts need a second pass.
template <bool kFew>
hipError_t launch_few(Act act, const MoeArgs& a, hipStream_t s) {
  const int avg = a.T * a.k / a.E;
  const hipError_t e = a.T <= 16 || avg <= 8   ? launch_up_act<kFew, 1>(act, a, s)
                       : a.T <= 32 || avg <= 16 ? launch_up_act<kFew, 2>(act, a, s)
                                                : launch_up_act<kFew, 4>(act, a, s);
  if (e != hipSuccess) return e;
  if (a.T <= 8 || avg <= 3) return launch_down_cols<kFew, 1>(a, s);
  if (a.T <= 16 || avg <= 8) return launch_down_cols<kFew, 2>(a, s);
  if (a.T <= 32 || avg <= 16) return launch_down_cols<kFew, 4>(a, s);
  return launch_down_cols<kFew, 8>(a, s);
}

}  // namespace

hipError_t launch_moe(Act act, const MoeArgs& a, hipStream_t s) {
  return a.T * a.k <= 64 ? launch_few<true>(act, a, s) : launch_few<false>(act, a, s);
}

}  // namespace swg
