// Matrix products grouped by expert, with ragged groups, on gfx950 matrix
// cores.
//
// R rows lie in order of expert, those of expert e from offsets[e] up to
// offsets[e + 1], which only the device knows.  Three forms of product, each
// C[m, n] = sum_r A(m, r) B(n, r) within one expert:
//   NT  m a row, n an output column, r an input column: A and B have the
//       reduction contiguous (y = x W^T; with two B operands the gate/up
//       stage and its recompute in the backward);
//   NN  m a row, n an input column, r an output column: B = W [r, n] has the
//       reduction along its rows (dx = dy W; with two halves dg Wg + du Wu);
//   TN  m an output column, n an input column, r the expert's rows: A and B
//       both have the reduction along their rows (dW = dy^T x).
// An operand whose reduction is contiguous is staged in LDS as rows of 128
// bytes of reduction; one whose reduction runs along its rows as k rows of
// its columns, and its MFMA fragments are formed by the transposing LDS
// reads of gfx950 (ds_read_b64_tr_b16: 16 lanes address a 4 x 16 block and
// receive a column each), so no operand is ever transposed in memory.
//
// Tiles: NT and NN cut every expert's rows into tiles of BM; a workgroup
// finds its tile by a scan over the experts' tile counts, one expert to a
// lane, so the host needs no sizes and nothing has to be planned.  Rows in
// front of the first and behind the last expert form two groups of zero rows.
// The grid covers the most tiles that R rows in E groups can make; the
// workgroups beyond the tiles there are end at once.  In an expert's last
// tile, waves whose rows all lie behind its end load their share of the
// operands and skip the products, so the others have the matrix cores.
//
// The main loops: operands come by 16-byte LDS DMA, a wave moving a share of
// each.  bf16 NT runs in turns (a ring of k-steps, the halves of the workgroup
// half a k-step apart); the forms with transposing reads and fp32 have a double
// buffer of k-steps and of fragments.  (The compiler lets every transposing
// read wait for all LDS DMA, so a longer ring gains them nothing.)  Products are
// formed transposed, so that a lane holds neighbouring columns of one row and
// results go from registers to memory without LDS.
//
// What bounds them.  Many rows: the matrix cores and what feeds them.  The
// gate/up stage of 16384 rows, 8 experts of (14336, 4096), takes 3.3-3.45 ms,
// 1.12-1.17 PFLOP/s (its gradients 11.9 ms, 0.97): matrix cores busy 60-65 % of the cycles, at 1.65 GHz (the
// clock falls with the power drawn); a large dense library product reaches 1.2-1.5.
// Of 8 experts of (4096, 11008), 16384 rows: dx 1.40 ms, dW 1.38 ms (1.05-1.07
// PFLOP/s; dW with loads that fetch nothing 1.0 ms: L2 delivers 64 KB per CU and
// 64-deep k-step).  64 experts with 512 rows each: 183-186 us for (2048, 1024),
// 0.75 PFLOP/s (111 us as one dense library product); the last tile of an expert
// is half empty there, and a large tile's ring has the CU's LDS to itself, so
// that its search, first loads and stores have no other workgroup beside them
// over only 16 to 32 k-steps.  Few rows: the weights, at 5-5.9 TB/s; small tiles
// then (row_tile of validate.hpp).  fp32: 2048 rows each 118-127 TFLOP/s forward,
// 103-108 dx and dW, of a library's 151.  Gradients whose tiles
// are too few for the CUs have their reduction in parts (blockIdx.y), whose fp32
// sums a second kernel adds in order.
#include "common.hpp"
#include "grouped.hpp"
#include "mfma.hpp"
#include "validate.hpp"

namespace swg {

namespace {

enum class Form { kNT, kNN, kTN };
enum class Out { kGated, kDGated, kStore, kPart };

// act(z) and, for the gradient, act'(z): SiLU a = z s, a' = s (1 + z (1 - s)),
// s = sigma(z); GELU (tanh form) a = z s, a' = s + z s (1 - s) t'(z),
// s = sigma(t), t = z (c1 + c3 z^2).  kShort: for results rounded to bf16.
template <Act A, bool kShort>
__device__ __forceinline__ float act_of(float z) {
  if constexpr (A == Act::kGeluTanh) return kShort ? gelu_tanh_bf16out(z) : gelu_tanh_f32(z);
  else if constexpr (kShort) {
    float s, a;
    sigmoid_silu_bf16out(z, s, a);
    return a;
  } else {
    return silu_f32(z);
  }
}

template <Act A, bool kShort>
__device__ __forceinline__ void act_and_slope(float z, float& a, float& da) {
  if constexpr (A == Act::kGeluTanh) {
    const float z2 = z * z;
    const float t = z * __builtin_fmaf(kGeluC3, z2, kGeluC1);
    float s, c;
    if constexpr (kShort) {
      constexpr float kL2e = 1.44269504088896340736f;
      s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-t * kL2e));
      c = 1.0f - s;
    } else {
      sigmoid_pair_f32(t, s, c);
    }
    a = z * s;
    da = s + a * c * __builtin_fmaf(3.0f * kGeluC3, z2, kGeluC1);
  } else {
    float s;
    if constexpr (kShort) sigmoid_silu_bf16out(z, s, a);
    else sigmoid_silu_f32(z, s, a);
    da = s * (1.0f + z * (1.0f - s));
  }
}

// ------------------------------------------------------------ tile of rows

struct Spot {
  int e;        // expert; -1: rows of no expert
  int row0;     // first row of the tile
  int rows;     // its rows
  int tn;
};

__device__ __forceinline__ int wave_scan(int v) {   // inclusive, over 64 lanes
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(v, d);
    if ((int)(threadIdx.x & 63) >= d) v += o;
  }
  return v;
}

// The rows of group g: 0 in front of the first expert, 1 .. E the experts',
// E + 1 behind the last.  Offsets are taken into [0, R], so that none of any
// value leads outside the arrays.
__device__ __forceinline__ void group_rows(const GroupedArgs& p, int g, int& first, int& count) {
  auto at = [&](int i) {
    const int v = p.offsets[i];
    return v < 0 ? 0 : (v > p.R ? p.R : v);
  };
  first = g == 0 ? 0 : at(g - 1);
  const int end = g > p.E ? p.R : at(g);
  count = end > first ? end - first : 0;
}

// The tile of workgroup `bid`: experts in order, within one kGroupM row tiles
// at a time down the columns.  kZero: rows of no expert have tiles too.
template <int BM, int kGroupM, bool kZero>
__device__ __forceinline__ bool find_tile(const GroupedArgs& p, int ntn, int bid, Spot& spot) {
  const int lane = threadIdx.x & 63;
  const int ng = p.E + 2;
  auto tiles_of = [&](int g, int& first, int& count) -> int {
    first = count = 0;
    if (g >= ng) return 0;
    group_rows(p, g, first, count);
    if (!kZero && (g == 0 || g == ng - 1)) return 0;
    return (int)(((int64_t)count + BM - 1) / BM);
  };
  int first, count;
  int mine = tiles_of(lane, first, count);
  int scan = wave_scan(mine);
  int64_t total = __builtin_amdgcn_readlane(scan, 63);
  for (int c = 64; c < ng; c += 64) {
    int f, n;
    total += __builtin_amdgcn_readlane(wave_scan(tiles_of(c + lane, f, n)), 63);
  }
  // Offsets that decrease may make more tiles than the grid has: no tile then.
  if (bid >= total * ntn || total * ntn > (int64_t)gridDim.x) return false;
  const int tile = xcd_remap(bid, (int)total * ntn);
  const int want = tile / ntn;
  int before = 0;                                       // tiles of the groups before this chunk
  for (int c = 0; c < ng; c += 64) {
    if (c > 0) {
      mine = tiles_of(c + lane, first, count);
      scan = wave_scan(mine);
    }
    const uint64_t past = __ballot(before + scan > want);
    if (past != 0) {
      const int l = __builtin_ctzll(past);
      const int mt = __builtin_amdgcn_readlane(mine, l);
      const int s0 = before + __builtin_amdgcn_readlane(scan, l) - mt;
      const int f = __builtin_amdgcn_readlane(first, l), n = __builtin_amdgcn_readlane(count, l);
      const int g = c + l;
      const int local = tile - s0 * ntn;                // within the group: mt x ntn
      const int band = kGroupM * ntn;
      const int m0 = (local / band) * kGroupM;
      const int gm = mt - m0 < kGroupM ? mt - m0 : kGroupM;
      const int tm = m0 + (local % band) % gm;
      spot.tn = (local % band) / gm;
      spot.e = (g == 0 || g == ng - 1) ? -1 : g - 1;
      spot.row0 = f + tm * BM;
      spot.rows = n - tm * BM < BM ? n - tm * BM : BM;
      return true;
    }
    before += __builtin_amdgcn_readlane(scan, 63);
  }
  return false;
}

// --------------------------------------------------------------- the kernel

// The ring of k-steps in LDS: 16-byte chunks of reduction to a k-step, and
// k-steps.  bf16 NT: five short ones (tiles of 64 rows, two workgroups to a CU:
// three of full length), taken in turns by the halves of the workgroup.
// Otherwise a double buffer.
template <typename T, Form F, class TL> struct Ring {
  static constexpr bool kTurns = sizeof(T) == 2 && F == Form::kNT && TL::kThreads == 512;
  static constexpr bool kShort = kTurns && TL::kBM > 64;
  static constexpr int kChunks = kShort ? 4 : 8, kDepth = !kTurns ? 2 : kShort ? 5 : 3;
};

// dh tile in LDS: row r at r * 2 BN bytes, its 16-byte chunk c at physical
// chunk c ^ (r & 15).
template <class TL>
struct DhTile {
  static constexpr int kCPR = TL::kBN / 8;
  static constexpr int kPitch = TL::kBN * 2;
  __device__ static int offset(int row, int col) {
    return row * kPitch + (((col >> 3) ^ (row & 15)) << 4) + (col & 7) * 2;
  }
};

template <typename T, Form F, Out O, Act ACT, int NB, class TL, int kGroupM>
__global__ __launch_bounds__(TL::kThreads) __attribute__((amdgpu_waves_per_eu(TL::kOcc, TL::kOcc)))
void grouped_kernel(GroupedArgs p) {
  constexpr bool kB16 = sizeof(T) == 2;
  constexpr int kMN = kB16 ? 16 : 32;                     // MFMA tile
  constexpr int kBM = TL::kBM, kBN = TL::kBN, kThreads = TL::kThreads, kWaves = kThreads / 64;
  constexpr int kWM = TL::kWM, kWN = TL::kWN, kTM = kWM / kMN, kTN = kWN / kMN;
  using R = Ring<T, F, TL>;
  constexpr int KC = R::kChunks, S = R::kDepth, kRowBytes = KC * 16;
  constexpr int kPer = 16 / (int)sizeof(T);               // elements per chunk
  constexpr int kStep = KC * kPer;                        // reduction per k-step
  constexpr int kABytes = kBM * kRowBytes, kBBytes = kBN * kRowBytes;
  constexpr int kStageBytes = kABytes + NB * kBBytes;
  constexpr int kDmaA = kABytes / 1024 / kWaves, kDmaB = kBBytes / 1024 / kWaves;   // per wave and k-step
  constexpr int kDma = kDmaA + NB * kDmaB;
  constexpr bool kAT = F == Form::kTN, kBT = F != Form::kNT;   // reduction along the operand's rows
  static_assert(kABytes % (1024 * kWaves) == 0 && kBBytes % (1024 * kWaves) == 0, "DMA split");
  extern __shared__ u32x4 lds[];
  char* const lds_bytes = reinterpret_cast<char*>(lds);

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / TL::kWGN, wn = wave % TL::kWGN;
  const int ntn = (p.n + kBN - 1) / kBN;

  // This workgroup's tile: rows, expert, columns.
  int e, tn, row0, rows, half = 0, m0 = 0, mrows;         // row0, rows: of the expert (TN: the reduction)
  if constexpr (F == Form::kTN) {
    // Every XCD takes an eighth of each expert's tiles, so that experts with
    // many rows do not fall to one.
    const int ntm = (p.m + kBM - 1) / kBM, per = p.halves * ntm * ntn, share = (per + 7) / 8;
    const int xcd = blockIdx.x % 8, turn = blockIdx.x / 8;
    e = turn / share;
    const int local = xcd * share + turn % share;
    if (local >= per) return;
    const int band = kGroupM * ntn, nm = p.halves * ntm;
    const int g0 = (local / band) * kGroupM, gm = nm - g0 < kGroupM ? nm - g0 : kGroupM;
    const int tm = g0 + (local % band) % gm;
    tn = (local % band) / gm;
    half = tm / ntm;
    m0 = (tm - half * ntm) * kBM;
    mrows = p.m - m0 < kBM ? p.m - m0 : kBM;
    group_rows(p, e + 1, row0, rows);
    row0 = __builtin_amdgcn_readfirstlane(row0);
    rows = __builtin_amdgcn_readfirstlane(rows);
  } else {
    Spot spot;
    if (!find_tile<kBM, kGroupM, O != Out::kDGated>(p, ntn, blockIdx.x, spot)) return;
    e = spot.e; tn = spot.tn; row0 = spot.row0; rows = mrows = spot.rows;
  }
  const int n0 = tn * kBN;
  const bool live = e >= 0;
  const int es = (int)sizeof(T);

  // Reduction: k-steps per half (NN has one or two halves, TN one over rows).
  const int red = F == Form::kTN ? rows : p.r;
  const int nkh = live ? (red + kStep - 1) / kStep : 0;
  const int nks = (F == Form::kNN ? p.halves : 1) * nkh;
  // kPart: the part's k-steps, ks0 up to ks0 + nk.
  const int per_part = O == Out::kPart ? (nks + p.parts - 1) / p.parts : nks;
  const int ks0 = O == Out::kPart ? (int)blockIdx.y * per_part : 0;
  const int nk = O != Out::kPart || nks - ks0 > per_part ? per_part : (nks > ks0 ? nks - ks0 : 0);

  // ---- operand A
  // Contiguous: instruction d of the wave fills kRowsDma LDS rows from
  // kRowsDma (d kWaves + wave) on, a lane physical chunk lane % KC of one, from
  // logical chunk (lane % KC) ^ ((row >> kSwz) % KC).
  // Along rows: it fills 1 KiB of k rows, kCPR chunks each; k row kr's pair
  // of chunks q lies at pair q ^ f(kr) (bf16: f = (kr & 3) | ((kr >> 3) & 1)
  // << 2, so that the transposing reads of two 16-lane groups meet 8 different
  // pairs; fp32: chunk bit 3 ^= (kr >> 2) & 1, the halves of a wave).
  // Lanes' offsets are the same for every d but for whole rows and, where a
  // pass has 8 k rows, f's third bit: odd passes then have chunk bit 3 turned.
  constexpr int kRowsDma = 64 / KC, kRowsPass = kRowsDma * kWaves;   // contiguous rows per instruction, per d
  auto swz = [](int row) { return KC == 8 ? (row >> 1) & 7 : -(row >> 2) & 3; };
  auto lane_contig = [&](int& row, int& chunk) {
    row = kRowsDma * wave + lane / KC;
    chunk = (lane % KC) ^ swz(row);
  };
  static_assert(kRowsPass % 16 == 0, "a pass over d leaves the swizzle of a lane's rows alone");
  auto lane_along = [&](auto cpr_c, int& kr, int& chunk) {
    constexpr int cpr = decltype(cpr_c)::value;           // chunks per k row
    constexpr int rpi = 64 / cpr;                         // k rows per instruction
    static_assert((rpi * kWaves) % 8 == 0, "f is the same for every second d");
    kr = rpi * wave + lane / cpr;
    const int c = lane % cpr;
    if constexpr (kB16) chunk = c ^ (((kr & 3) | (((kr >> 3) & 1) << 2)) << 1);
    else chunk = c ^ (((kr >> 2) & 1) << 3);
  };
  constexpr uint32_t kOob = 0x80000000u;                  // past every descriptor: reads zero

  const T* abase = static_cast<const T*>(p.a);
  int64_t abytes = 0;                                     // contiguous: descriptor; along rows: all that is left
  uint32_t avoff[kAT ? 2 : kDmaA];
  int achunk = 0;
  constexpr int kACpr = kBM / kPer, kBCpr = kBN / kPer;
  constexpr bool kATurn = kB16 && 64 / kACpr * kWaves == 8, kBTurn = kB16 && 64 / kBCpr * kWaves == 8;
  if constexpr (kAT) {
    int kr;
    lane_along(std::integral_constant<int, kACpr>{}, kr, achunk);
    abase += (int64_t)row0 * p.lda + (int64_t)half * p.m + m0;
    abytes = rows > 0 ? ((int64_t)rows * p.lda - half * p.m - m0) * es : 0;
    avoff[0] = (uint32_t)(kr * (int)p.lda * es + achunk * 16);
    avoff[1] = kATurn ? avoff[0] - achunk * 16 + (achunk ^ 8) * 16 : avoff[0];
  } else {
    int r;
    lane_contig(r, achunk);
    if (F == Form::kNT && p.src != nullptr) {
      abytes = (int64_t)p.T * p.lda * es;
#pragma unroll
      for (int d = 0; d < kDmaA; ++d) {
        const int rr = r + d * kRowsPass;
        avoff[d] = kOob;
        if (live && rr < rows) {
          const int pair = p.src[row0 + rr];
          const int t = pair / p.k;
          if (pair >= 0 && t < p.T) avoff[d] = (uint32_t)t * (uint32_t)(p.lda * es) + (uint32_t)(achunk * 16);
        }
      }
    } else {
      abase += (int64_t)row0 * p.lda;
      abytes = live ? (int64_t)rows * p.lda * es : 0;
#pragma unroll
      for (int d = 0; d < kDmaA; ++d)
        avoff[d] = (uint32_t)((r + d * kRowsPass) * (int)p.lda * es + achunk * 16);
    }
  }
  // ---- operand B
  const T* bbase[2];
  int64_t bbytes;
  uint32_t bvoff[2];
  int bchunk;
  const int64_t ebase = live ? e : 0;
  if constexpr (F == Form::kTN) {
    bbase[0] = bbase[1] = static_cast<const T*>(p.b0) + (int64_t)row0 * p.ldb + n0;
    bbytes = rows > 0 ? ((int64_t)rows * p.ldb - n0) * es : 0;
  } else {
    bbase[0] = static_cast<const T*>(p.b0) + ebase * p.b0_stride;
    bbase[1] = static_cast<const T*>(p.b1 != nullptr ? p.b1 : p.b0) + (p.b1 != nullptr ? ebase * p.b1_stride : ebase * p.b0_stride);
    if constexpr (F == Form::kNN) {
      bbase[0] += n0;
      bbase[1] += n0;
      bbytes = ((int64_t)p.r * p.ldb - n0) * es;
    } else {
      bbase[0] += (int64_t)n0 * p.ldb;
      bbase[1] += (int64_t)n0 * p.ldb;
      const int left = p.n - n0;
      bbytes = (int64_t)(left < kBN ? left : kBN) * p.ldb * es;
    }
  }
  if constexpr (kBT) {
    int kr;
    lane_along(std::integral_constant<int, kBCpr>{}, kr, bchunk);
    bvoff[0] = (uint32_t)(kr * (int)p.ldb * es + bchunk * 16);
    bvoff[1] = kBTurn ? bvoff[0] - bchunk * 16 + (bchunk ^ 8) * 16 : bvoff[0];
  } else {
    int r;
    lane_contig(r, bchunk);
    bvoff[0] = bvoff[1] = (uint32_t)(r * (int)p.ldb * es + bchunk * 16);
  }
  constexpr int kBRowsPass = kBT ? 64 / kBCpr * kWaves : kRowsPass;
  constexpr int kARowsPass = 64 / kACpr * kWaves;         // (along rows)
  const uint32_t bpass = (uint32_t)(kBRowsPass * (int)p.ldb * es);
  const uint32_t apass = (uint32_t)(kARowsPass * (int)p.lda * es);

  // Bytes of an operand along rows that k-step s of a half may read: its kStep
  // rows, no more than are left.
  auto step_bytes = [&](int64_t all, int64_t ld, int s) -> int64_t {
    const int64_t step = (int64_t)kStep * ld * es;
    const int64_t left = all - s * step;
    return left < 0 ? 0 : (left < step ? left : step);
  };
  // Where rows are few, all workgroups stream weights at once.  Those of a
  // column tile start where its number says, and go round: from the same place
  // in all rows, at a power-of-two distance from each other, they would keep
  // asking a few of the memory's channels.  (The order depends on the expert and
  // the column tile, and R and E say whether there is one, as they say which
  // tile is taken and how many parts: a row's bits depend on how many rows and
  // experts there are, not on what the other rows hold or whose they are.)
  const int first = F == Form::kNT && p.stagger && nk > 0 ? (e * ntn + tn) % nk : 0;
  // Instruction q of this wave's kDma for k-step ks, into a slot: A's first.
  auto issue_one = [&](int ks, int slot, int q) {
    const int h = F == Form::kNN && ks0 + ks >= nkh ? 1 : 0;
    int s = ks0 + ks - h * nkh;
    if constexpr (F == Form::kNT) s = s + first < nk ? s + first : s + first - nk;
    const int rem = (red + kPer - 1) / kPer - s * KC;     // chunks of reduction left (contiguous)
    const bool past = ks >= nk;
    char* dst = lds_bytes + slot * kStageBytes + wave * 1024;
    if (q < kDmaA) {
      dst += q * kWaves * 1024;
      if constexpr (kAT) {
        const __amdgpu_buffer_rsrc_t rs =
            uniform_rsrc(abase + (int64_t)s * kStep * p.lda, past ? 0 : step_bytes(abytes, p.lda, s));
        const uint32_t off = avoff[q & 1] + q * apass;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void_t*)dst, 16, off, 0, 0, 0);
      } else {
        const __amdgpu_buffer_rsrc_t rs = uniform_rsrc(abase, past ? 0 : abytes);
        const uint32_t off = achunk < rem ? avoff[q % (kAT ? 2 : kDmaA)] + (uint32_t)((h * p.r + s * kStep) * es) : kOob;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void_t*)dst, 16, off, 0, 0, 0);
      }
    } else {
      const int w = (q - kDmaA) / kDmaB, d = (q - kDmaA) % kDmaB;
      dst += kABytes + w * kBBytes + d * kWaves * 1024;
      if constexpr (kBT) {
        const __amdgpu_buffer_rsrc_t rs =
            uniform_rsrc(bbase[F == Form::kNN ? h : 0] + (int64_t)s * kStep * p.ldb, past ? 0 : step_bytes(bbytes, p.ldb, s));
        const uint32_t off = bvoff[d & 1] + d * bpass;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void_t*)dst, 16, off, 0, 0, 0);
      } else {
        const __amdgpu_buffer_rsrc_t rs = uniform_rsrc(bbase[w], past ? 0 : bbytes);
        const uint32_t off = bchunk < rem ? bvoff[0] + (uint32_t)(s * kStep * es) + d * bpass : kOob;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void_t*)dst, 16, off, 0, 0, 0);
      }
    }
  };
  auto issue = [&](int ks, int slot) {
#pragma unroll
    for (int q = 0; q < kDma; ++q) issue_one(ks, slot, q);
  };

  // The dh tile (recompute, bf16) by DMA, its two halves of rows in place of
  // the two k-steps behind the last: an instruction fills 1 KiB of rows, a
  // lane's chunk c of row r from logical chunk c ^ (r & 15); chunks past the
  // last column and rows past the tile's read zero (n is a multiple of 8).
  constexpr bool kDh = O == Out::kDGated && kB16;
  auto issue_dh = [&](int part, int slot, int d) {
    constexpr int kCPR = DhTile<TL>::kCPR, kRpi = 64 / kCPR, kHalf = kBM / 2;
    static_assert(!kDh || (kCPR == 16 && kHalf * DhTile<TL>::kPitch == kStageBytes && kHalf / (kRpi * kWaves) == kDma),
                  "a half of the dh tile fills a slot by as many instructions");
    const T* d0 = static_cast<const T*>(p.dh) + (int64_t)row0 * p.n + n0;
    const __amdgpu_buffer_rsrc_t rd = uniform_rsrc(d0, ((int64_t)rows * p.n - n0) * es);
    char* dst = lds_bytes + slot * kStageBytes + (d * kWaves + wave) * 1024;
    const int r = part * kHalf + (d * kWaves + wave) * kRpi + lane / kCPR;
    const int c = (lane % kCPR) ^ (r & 15);
    const uint32_t off = n0 + c * 8 < p.n && r < rows ? (uint32_t)(r * p.n * es + c * 16) : kOob;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rd, (lds_void_t*)dst, 16, off, 0, 0, 0);
  };

  typename AccL<kMN>::V acc[NB][kTM][kTN];
#pragma unroll
  for (int w = 0; w < NB; ++w)
#pragma unroll
    for (int i = 0; i < kTM; ++i)
#pragma unroll
      for (int j = 0; j < kTN; ++j)
#pragma unroll
        for (int q = 0; q < AccL<kMN>::kE; ++q) acc[w][i][j][q] = 0.0f;

  // fp32: the sums of every kFold k-steps (256 products) are added to a second
  // set.  Over a reduction of 13448 one chain of additions was off by 2.0e-6 of
  // the result's norm, this by 3.1e-7.
  constexpr int kFold = 8;
  [[maybe_unused]] typename AccL<kMN>::V sum[kB16 ? 1 : NB][kB16 ? 1 : kTM][kB16 ? 1 : kTN] = {};
  auto fold = [&]() {
    if constexpr (!kB16) {
#pragma unroll
      for (int w = 0; w < NB; ++w)
#pragma unroll
        for (int i = 0; i < kTM; ++i)
#pragma unroll
          for (int j = 0; j < kTN; ++j)
#pragma unroll
            for (int q = 0; q < AccL<kMN>::kE; ++q) {
              sum[w][i][j][q] += acc[w][i][j][q];
              acc[w][i][j][q] = 0.0f;
            }
    }
  };

  // ---- fragments.  Sub-step kk: lane l supplies row l % kMN of its operand
  // tile and reduction chunk kCPS kk + l / kMN.
  constexpr int kCPS = 64 / kMN;
  constexpr int kKK = KC / kCPS;
  const int rl = lane % kMN, ql = lane / kMN;
  auto frag_contig = [&](const char* L, int row, int kk) -> u32x4 {
    const int pc = (kCPS * kk + ql) ^ swz(row);
    return *reinterpret_cast<const u32x4*>(L + row * kRowBytes + pc * 16);
  };
  // Along rows, columns c0 .. c0 + kMN - 1 of tiles of `cols` columns.
  auto frag_along = [&](const char* L, auto cols_c, int c0, int kk) -> u32x4 {
    constexpr int kPitch = decltype(cols_c)::value * (int)sizeof(T);
    if constexpr (kB16) {
      const int s = lane & 15, g = lane >> 4;
      const int f = (s >> 2) | ((g & 1) << 2);
      const char* at = L + (32 * kk + 8 * g + (s >> 2)) * kPitch + (((c0 >> 4) ^ f) << 5) + (s & 3) * 8;
      const short4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4_t*)(lds_char_t*)(at));
      const short4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4_t*)(lds_char_t*)(at + 4 * kPitch));
      const u32x2 a = __builtin_bit_cast(u32x2, lo), b = __builtin_bit_cast(u32x2, hi);
      return u32x4{a[0], a[1], b[0], b[1]};
    } else {
      const int h = lane >> 5;
      const char* at = L + (8 * kk + 4 * h) * kPitch + (((c0 + rl) * 4) ^ (h << 7));
      u32x4 v;
#pragma unroll
      for (int t = 0; t < 4; ++t) v[t] = *reinterpret_cast<const uint32_t*>(at + t * kPitch);
      return v;
    }
  };
  u32x4 av[2][kTM], bv[2][NB][kTN];
  auto read_frags = [&](int buf, const char* L, int kk) {
#pragma unroll
    for (int i = 0; i < kTM; ++i) {
      if constexpr (kAT) av[buf][i] = frag_along(L, std::integral_constant<int, kBM>{}, wm * kWM + i * kMN, kk);
      else av[buf][i] = frag_contig(L, wm * kWM + i * kMN + rl, kk);
    }
#pragma unroll
    for (int w = 0; w < NB; ++w)
#pragma unroll
      for (int j = 0; j < kTN; ++j) {
        const char* LB = L + kABytes + w * kBBytes;
        if constexpr (kBT) bv[buf][w][j] = frag_along(LB, std::integral_constant<int, kBN>{}, wn * kWN + j * kMN, kk);
        else bv[buf][w][j] = frag_contig(LB, wn * kWN + j * kMN + rl, kk);
      }
  };
  constexpr int kMf = NB * kTM * kTN;                     // MFMAs of a sub-step
  auto mfmas = [&](int buf, int from, int to) {
#pragma unroll
    for (int w = 0; w < NB; ++w)
#pragma unroll
      for (int i = 0; i < kTM; ++i)
#pragma unroll
        for (int j = 0; j < kTN; ++j) {
          const int at = (w * kTM + i) * kTN + j;
          if (at < from || at >= to) continue;
          if constexpr (kB16)
            acc[w][i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, bv[buf][w][j]),
                                                                   __builtin_bit_cast(bf16x8, av[buf][i]),
                                                                   acc[w][i][j], 0, 0, 0);
          else
            Mma<T>::run(acc[w][i][j], bv[buf][w][j], av[buf][i]);
        }
  };
  auto landed = [&]() {                                   // this wave's DMA has landed, its LDS reads are done
    wait_vmcnt<0>();
    __builtin_amdgcn_s_waitcnt(0xC07F);
  };
  // Some row of the wave's is the tile's.
  const bool active = wm * kWM < mrows;

  if constexpr (R::kTurns) {
    // Two halves of the workgroup, one wave of each on a SIMD, half a k-step
    // apart: in turn `it` the first half reads its fragments of k-step `it` and
    // multiplies them, the second multiplies those of the k-step before and
    // then reads, so that one half's reads fall into the other's products.
    // One barrier to a turn: behind it k-step `it` is in LDS and k-step it - 1
    // has been read by all, so its slot is filled with k-step it + S - 1, an
    // instruction at a time between the products.  Every k-step of the ring is
    // requested, also those behind the last, which read nothing (or the dh
    // tile), so that the count of loads in flight says which have landed.
    static_assert(kWaves == 8 && kKK <= 2, "two waves to a SIMD, fragments of a whole k-step in registers");
    auto read = [&](const char* L) {
#pragma unroll
      for (int kk = 0; kk < kKK; ++kk) read_frags(kk, L, kk);
    };
    auto multiply = [&](int from, int to) {
#pragma unroll
      for (int kk = 0; kk < kKK; ++kk) mfmas(kk, from - kk * kMf, to - kk * kMf);
    };
    auto request = [&](int ks, int slot, int q) {
      if (kDh && (ks == nk || ks == nk + 1)) issue_dh(ks - nk, slot, q);
      else issue_one(ks, slot, q);
    };
#pragma unroll
    for (int t = 0; t < S - 1; ++t)
#pragma unroll
      for (int q = 0; q < kDma; ++q) request(t, t, q);
    int slot = 0, next = S - 1;                           // of k-step it and of it + S - 1
    auto products = [&](int it) {
#pragma unroll
      for (int q = 0; q < kDma; ++q) {
        __builtin_amdgcn_sched_barrier(0);
        request(it + S - 1, next, q);
        __builtin_amdgcn_sched_barrier(0);
        multiply(q * kKK * kMf / kDma, (q + 1) * kKK * kMf / kDma);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    auto turn = [&]() {                                   // k-step `it` has landed, it - 1 is read
      wait_vmcnt<(S - 2) * kDma>();
      __builtin_amdgcn_s_waitcnt(0xC07F);
      barrier_no_fence();
    };
    auto advance = [&]() {
      next = slot;
      slot = slot + 1 == S ? 0 : slot + 1;
    };
    if (!active) {
      for (int it = 0; it < nk; ++it) {
        turn();
#pragma unroll
        for (int q = 0; q < kDma; ++q) request(it + S - 1, next, q);
        advance();
      }
      barrier_no_fence();
    } else if (wave < 4) {
      for (int it = 0; it < nk; ++it) {
        turn();
        read(lds_bytes + slot * kStageBytes);
        products(it);
        advance();
      }
      barrier_no_fence();
    } else {
      turn();
      if (nk > 0) {
        read(lds_bytes);
#pragma unroll
        for (int q = 0; q < kDma; ++q) request(S - 1, next, q);
        advance();
        for (int it = 1; it < nk; ++it) {
          turn();
          products(it);
          read(lds_bytes + slot * kStageBytes);
          advance();
        }
        turn();
        multiply(0, kKK * kMf);
      }
    }
  } else {
    // A double buffer of LDS and of fragments: the fragments of a sub-step are
    // read between the products of the one before, the step boundary lies in
    // the last sub-step.
    static_assert(S == 2 && (KC / kCPS) % 2 == 0, "the next step's first fragments go to buffer 0");
    constexpr int kKK = KC / kCPS;
    constexpr int kRd = kTM * (kAT ? 2 : 1) + NB * kTN * (kBT ? 2 : 1);   // LDS reads of a sub-step (bf16)
    issue(0, 0);
    issue(1, 1);
    wait_vmcnt<kDma>();
    barrier_no_fence();
    if (active) {
      if (nk > 0) read_frags(0, lds_bytes, 0);
      auto kstep = [&](int ks, bool more) {
        const char* L = lds_bytes + (ks % S) * kStageBytes;
#pragma unroll
        for (int kk = 0; kk < kKK; ++kk) {
          __builtin_amdgcn_sched_barrier(0);
          if (kk + 1 < kKK) {
            read_frags((kk + 1) & 1, L, kk + 1);
            if constexpr (kB16) {
              mfmas(kk & 1, 0, kMf);
#pragma unroll
              for (int t = 0; t < kRd; ++t) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
              }
              __builtin_amdgcn_sched_group_barrier(0x008, kMf, 0);
              continue;
            }
          } else if (more) {
            landed();                                     // step ks + 1
            barrier_no_fence();                           // and every wave has read step ks
            __builtin_amdgcn_sched_barrier(0);
            read_frags(0, lds_bytes + ((ks + 1) % S) * kStageBytes, 0);
            issue(ks + S, ks % S);
            if constexpr (kB16) {
              mfmas(kk & 1, 0, kMf);
              constexpr int kLead = kMf / kDma > 0 ? kMf / kDma : 1;
              __builtin_amdgcn_sched_group_barrier(0x008, kLead, 0);
              __builtin_amdgcn_sched_group_barrier(0x100, kRd, 0);
              __builtin_amdgcn_sched_group_barrier(0x020, kDma, 0);
              __builtin_amdgcn_sched_group_barrier(0x008, kMf - kLead, 0);
              continue;
            }
          }
          __builtin_amdgcn_sched_barrier(0);
          mfmas(kk & 1, 0, kMf);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (!kB16 && ks % kFold == kFold - 1) fold();
      };
      for (int ks = 0; ks + 1 < nk; ++ks) kstep(ks, true);
      if (nk > 0) kstep(nk - 1, false);
      fold();
    } else {
      // Only rows behind the expert's last: this wave's share of the operands.
      for (int ks = 0; ks + 1 < nk; ++ks) {
        landed();
        barrier_no_fence();
        issue(ks + S, ks % S);
      }
    }
  }
  if constexpr (kDh) {                                    // the dh tile is there
    landed();
    barrier_no_fence();
  } else {
    wait_vmcnt<0>();                                      // no load still lands in LDS when the waves end
  }
  if (!active) return;

  // ---- results, from the registers.  The products are formed transposed
  // (B's fragment first), so a lane's 4 consecutive accumulators are columns
  // of one row.
  T* const out0 = static_cast<T*>(half == 0 ? p.out0 : p.out1);
  const int64_t orow0 = F == Form::kTN ? (int64_t)e * p.m + m0 : row0;
  // One value of output `o` (dg, du of the recompute) from the accumulators.
  // dg and du are rounded to T: they are operands of the gradients' products,
  // and the bf16 matrix instructions take no wider ones (as hi + lo pairs they
  // would double these products).  It adds half a step of each to dx and dW:
  // 2.3e-3 of the norm, 1.7e-3 for fp32 dg and du.
  auto value = [&](int o, float g, float u, float dh) -> float {
    if constexpr (O == Out::kGated) {
      return act_of<ACT, kB16>(g) * u;
    } else if constexpr (O == Out::kDGated) {
      float a, da;
      act_and_slope<ACT, kB16>(g, a, da);
      return o == 0 ? dh * u * da : dh * a;
    } else {
      return g;
    }
  };
  constexpr int kOuts = O == Out::kDGated ? 2 : 1;
  if constexpr (O == Out::kPart) {
    const int64_t before = F == Form::kTN ? ((int64_t)blockIdx.y * p.halves + half) * p.E * p.m : (int64_t)blockIdx.y * p.R;
    float* const o0 = p.part + (before + orow0) * p.n;
#pragma unroll
    for (int i = 0; i < kTM; ++i) {
      const int row = wm * kWM + i * kMN + lane % kMN;
      if (row >= mrows) continue;
#pragma unroll
      for (int j = 0; j < kTN; ++j)
#pragma unroll
        for (int q = 0; q < AccL<kMN>::kE; q += 4) {
          const int col = n0 + wn * kWN + j * kMN + (kB16 ? 4 * (lane >> 4) : AccL<32>::row(lane, q));
          if (col >= p.n) continue;
          f32x4 v;
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            if constexpr (kB16) v[z] = acc[0][i][j][q + z];
            else v[z] = sum[0][i][j][q + z];
          }
          *reinterpret_cast<f32x4*>(o0 + (int64_t)row * p.n + col) = v;
        }
    }
  } else if constexpr (kB16) {
    // Two tiles of 16 columns together: a swap of 16-lane rows gives every
    // lane 8 neighbouring columns, and the four lanes of a row 64 bytes.
    const int g = lane >> 4;
    const int mycol = n0 + wn * kWN + (g & 1) * 16 + (g >> 1) * 8;
#pragma unroll
    for (int i = 0; i < kTM; ++i) {
      const int row = wm * kWM + i * 16 + (lane & 15);
      const bool in = row < mrows;
      T* o = out0 + (orow0 + row) * p.ldo + mycol;
#pragma unroll
      for (int j = 0; j < kTN; j += 2) {
        u32x2 dh[2];
        if constexpr (O == Out::kDGated) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const char* D = lds_bytes + ((nk + (row < kBM / 2 ? 0 : 1)) % S) * kStageBytes;
            dh[t] = *reinterpret_cast<const u32x2*>(
                D + DhTile<TL>::offset(row % (kBM / 2), wn * kWN + (j + t) * 16 + 4 * g));
          }
        }
#pragma unroll
        for (int out = 0; out < kOuts; ++out) {
          u32x2 v[2];
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int q = 0; q < 4; q += 2) {
              float f[2];
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                float d = 0.0f;
                if constexpr (O == Out::kDGated) d = bits_f32(z ? dh[t][q >> 1] & 0xFFFF0000u : dh[t][q >> 1] << 16);
                f[z] = value(out, acc[0][i][j + t][q + z], acc[NB - 1][i][j + t][q + z], d);
              }
              v[t][q >> 1] = __builtin_bit_cast(uint32_t, bf16x2{to_bf16(f[0]), to_bf16(f[1])});
            }
          const auto lo = __builtin_amdgcn_permlane16_swap(v[0][0], v[1][0], false, false);
          const auto hi = __builtin_amdgcn_permlane16_swap(v[0][1], v[1][1], false, false);
          if (in && mycol + j * 16 < p.n)
            *reinterpret_cast<u32x4*>(o + out * (int64_t)p.n + j * 16) = u32x4{lo[0], hi[0], lo[1], hi[1]};
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kTM; ++i) {
      const int row = wm * kWM + i * 32 + (lane & 31);
      if (row >= mrows) continue;
#pragma unroll
      for (int j = 0; j < kTN; ++j)
#pragma unroll
        for (int q = 0; q < 16; q += 4) {
          const int col = n0 + wn * kWN + j * 32 + AccL<32>::row(lane, q);
          if (col >= p.n) continue;
          T* o = out0 + (orow0 + row) * p.ldo + col;
          f32x4 dh = {0.0f, 0.0f, 0.0f, 0.0f};
          if constexpr (O == Out::kDGated)
            dh = *reinterpret_cast<const f32x4*>(static_cast<const float*>(p.dh) + (int64_t)(row0 + row) * p.n + col);
#pragma unroll
          for (int out = 0; out < kOuts; ++out) {
            f32x4 v;
#pragma unroll
            for (int z = 0; z < 4; ++z) v[z] = value(out, sum[0][i][j][q + z], sum[NB - 1][i][j][q + z], dh[z]);
            *reinterpret_cast<f32x4*>(o + out * (int64_t)p.n) = v;
          }
        }
    }
  }
}

template <class TL> constexpr RowTile kTileOf = {TL::kBM, TL::kBN, TL::kThreads};

template <typename T, Form F, Out O, Act ACT, int NB, class TL, int kGroupM = 8>
hipError_t launch(const GroupedArgs& a, hipStream_t s) {
  const int64_t ntn = ((int64_t)a.n + TL::kBN - 1) / TL::kBN;
  int64_t tiles;
  if (F == Form::kTN) {
    tiles = 8 * (int64_t)a.E * ((a.halves * (((int64_t)a.m + TL::kBM - 1) / TL::kBM) * ntn + 7) / 8);
  } else {
    tiles = row_column_tiles(kTileOf<TL>, a.R, a.E, a.n);
  }
  if (tiles == 0) return hipSuccess;
  const size_t lds = (size_t)Ring<T, F, TL>::kDepth * (TL::kBM + NB * TL::kBN) * Ring<T, F, TL>::kChunks * 16;
  const hipError_t attr = allow_lds<&grouped_kernel<T, F, O, ACT, NB, TL, kGroupM>>(lds);
  if (attr != hipSuccess) return attr;
  hipLaunchKernelGGL((grouped_kernel<T, F, O, ACT, NB, TL, kGroupM>),
                     dim3((unsigned)tiles, O == Out::kPart ? (unsigned)a.parts : 1u), dim3(TL::kThreads), lds, s, a);
  return hipGetLastError();
}

// out = the parts' sums in order, four elements to a thread.
constexpr int kSumThreads = 256;
template <typename T>
__global__ __launch_bounds__(kSumThreads) void sum_parts_kernel(const f32x4* part, int parts, int64_t stride4,
                                                                int64_t n4, T* out) {
  const int64_t i = (int64_t)blockIdx.x * kSumThreads + threadIdx.x;
  if (i >= n4) return;
  f32x4 v = part[i];
  for (int p = 1; p < parts; ++p) v += part[p * stride4 + i];
  if constexpr (sizeof(T) == 2) {
    u32x2 o;
#pragma unroll
    for (int q = 0; q < 2; ++q) o[q] = __builtin_bit_cast(uint32_t, bf16x2{to_bf16(v[2 * q]), to_bf16(v[2 * q + 1])});
    reinterpret_cast<u32x2*>(out)[i] = o;
  } else {
    reinterpret_cast<f32x4*>(out)[i] = v;
  }
}

template <typename T, Form F, class TL, int kGroupM>
hipError_t launch_parts(const GroupedArgs& a, hipStream_t s) {
  hipError_t e = launch<T, F, Out::kPart, Act::kSilu, 1, TL, kGroupM>(a, s);
  const int halves = F == Form::kTN ? a.halves : 1;        // outputs
  const int64_t n4 = (F == Form::kTN ? (int64_t)a.E * a.m : (int64_t)a.R) * a.n / 4;
  for (int h = 0; h < halves && e == hipSuccess; ++h) {
    hipLaunchKernelGGL((sum_parts_kernel<T>), dim3((unsigned)((n4 + kSumThreads - 1) / kSumThreads)), dim3(kSumThreads),
                       0, s, reinterpret_cast<const f32x4*>(a.part) + h * n4, a.parts, halves * n4, n4,
                       static_cast<T*>(h == 0 ? a.out0 : a.out1));
    e = hipGetLastError();
  }
  return e;
}

using Dual = Tile<256, 128, 4, 2>;
using Single = Tile<256, 256, 4, 2>;
using DualFew = Tile<64, 64, 4, 2, 4>;
using SingleFewNT = Tile<64, 128, 4, 2, 4>;
using SingleFew = Tile<64, 256, 2, 2, 2>;
using DualF32 = Tile<128, 64, 2, 2, 2>;
using SingleF32 = Tile<128, 128, 2, 2, 2>;
using DualF32Few = Tile<32, 64, 1, 2, 2>;
using SingleF32Few = DualF32Few;

// Which of a form's two tiles a call takes, and where its column tiles start, is
// told in validate.hpp (row_tile, weights_bound); these are the tiles it names.
template <class Large, class Few> constexpr bool kRuleNames(const TileRule& r) {
  return r.large == kTileOf<Large> && r.few == kTileOf<Few>;
}
static_assert(kRuleNames<Dual, DualFew>(tile_rule(SWIGLU_BF16, RowForm::kGated)) &&
              kRuleNames<Dual, Dual>(tile_rule(SWIGLU_BF16, RowForm::kRecompute)) &&
              kRuleNames<Single, SingleFewNT>(tile_rule(SWIGLU_BF16, RowForm::kNT)) &&
              kRuleNames<Single, SingleFew>(tile_rule(SWIGLU_BF16, RowForm::kNN)) &&
              kRuleNames<DualF32, DualF32Few>(tile_rule(SWIGLU_F32, RowForm::kGated)) &&
              kRuleNames<DualF32, DualF32Few>(tile_rule(SWIGLU_F32, RowForm::kRecompute)) &&
              kRuleNames<SingleF32, SingleF32Few>(tile_rule(SWIGLU_F32, RowForm::kNT)) &&
              kRuleNames<SingleF32, SingleF32Few>(tile_rule(SWIGLU_F32, RowForm::kNN)), "the tiles of the rules");
bool takes_few(Dt dt, RowForm form, const GroupedArgs& a) {
  const int code = dt == Dt::kBF16 ? SWIGLU_BF16 : SWIGLU_F32;
  return row_tile(code, form, a.R, a.E, a.n) == tile_rule(code, form).few;
}

template <Out O, Act A>
hipError_t dual(Dt dt, GroupedArgs a, hipStream_t s) {
  constexpr RowForm kForm = O == Out::kGated ? RowForm::kGated : RowForm::kRecompute;
  a.stagger = weights_bound(a.R, a.E);
  if (dt == Dt::kF32)
    return takes_few(dt, kForm, a) ? launch<float, Form::kNT, O, A, 2, DualF32Few>(a, s)
                                   : launch<float, Form::kNT, O, A, 2, DualF32>(a, s);
  if constexpr (O == Out::kGated)
    if (takes_few(dt, kForm, a)) return launch<bf16, Form::kNT, O, A, 2, DualFew>(a, s);
  return launch<bf16, Form::kNT, O, A, 2, Dual>(a, s);
}

template <Form F>
hipError_t single(Dt dt, GroupedArgs a, hipStream_t s) {
  constexpr RowForm kForm = F == Form::kNT ? RowForm::kNT : RowForm::kNN;
  a.stagger = F == Form::kNT && weights_bound(a.R, a.E);
  using Few = std::conditional_t<F == Form::kNT, SingleFewNT, SingleFew>;
  if constexpr (F == Form::kNN) {
    static_assert(SingleFew::kBM == kSplitBf16.bm && SingleFew::kBN == kSplitBf16.bn && SingleF32Few::kBM == kSplitF32.bm &&
                  SingleF32Few::kBN == kSplitF32.bn, "split_parts counts these tiles");
    if (a.parts > 1)
      return dt == Dt::kF32 ? launch_parts<float, F, SingleF32Few, 8>(a, s) : launch_parts<bf16, F, SingleFew, 4>(a, s);
  }
  if (dt == Dt::kF32)
    return takes_few(dt, kForm, a) ? launch<float, F, Out::kStore, Act::kSilu, 1, SingleF32Few>(a, s)
                                   : launch<float, F, Out::kStore, Act::kSilu, 1, SingleF32>(a, s);
  return takes_few(dt, kForm, a) ? launch<bf16, F, Out::kStore, Act::kSilu, 1, Few, 4>(a, s)
                                 : launch<bf16, F, Out::kStore, Act::kSilu, 1, Single, 4>(a, s);
}

}  // namespace

hipError_t launch_grouped_gated(Dt dt, Act act, const GroupedArgs& a, hipStream_t s) {
  return act == Act::kGeluTanh ? dual<Out::kGated, Act::kGeluTanh>(dt, a, s) : dual<Out::kGated, Act::kSilu>(dt, a, s);
}

hipError_t launch_grouped_dgated(Dt dt, Act act, const GroupedArgs& a, hipStream_t s) {
  return act == Act::kGeluTanh ? dual<Out::kDGated, Act::kGeluTanh>(dt, a, s) : dual<Out::kDGated, Act::kSilu>(dt, a, s);
}

hipError_t launch_grouped_nt(Dt dt, const GroupedArgs& a, hipStream_t s) { return single<Form::kNT>(dt, a, s); }

hipError_t launch_grouped_nn(Dt dt, const GroupedArgs& a, hipStream_t s) { return single<Form::kNN>(dt, a, s); }

hipError_t launch_grouped_tn(Dt dt, const GroupedArgs& a, hipStream_t s) {
  static_assert(Single::kBM == kSplitRowsBf16.bm && Single::kBN == kSplitRowsBf16.bn && SingleF32::kBM == kSplitRowsF32.bm &&
                SingleF32::kBN == kSplitRowsF32.bn, "split_row_parts counts these tiles");
  if (a.parts > 1)
    return dt == Dt::kBF16 ? launch_parts<bf16, Form::kTN, Single, 4>(a, s)
                           : launch_parts<float, Form::kTN, SingleF32, 8>(a, s);
  return dt == Dt::kBF16 ? launch<bf16, Form::kTN, Out::kStore, Act::kSilu, 1, Single, 4>(a, s)
                         : launch<float, Form::kTN, Out::kStore, Act::kSilu, 1, SingleF32, 8>(a, s);
}

}  // namespace swg
