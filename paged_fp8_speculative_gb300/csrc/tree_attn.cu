// Attention of draft trees over the paged cache, on the sm_100-family tensor cores (tcgen05,
// TMA, TMEM).
//
// Work.  The query rows of a (sequence, KV head) are its nodes times the GQA ratio, row r being
// node r / ratio, head r % ratio of the group; they are cut into tiles of 128 rows.  A unit is
// one row tile of one (sequence, KV head); it takes ceil(seq_len / 128) key tiles, and about
// kUnitTiles' time more for its Q and its output.  All units stand in a line, a place for each of
// these, which is cut into equal pieces, one per CTA (worked out from seq_lens and cu_seqlens_q on
// the device, so a captured call follows its buffers).  A unit whose key tiles lie in one piece is
// written out at once; a unit cut by piece borders leaves one partial output and log-sum-exp per
// piece in the workspace, and tree_reduce_kernel joins them: the CTA that has a unit's first
// key tile leaves a note on it.  A CTA has at most two partial units, the first and the last of its piece:
// two slots per CTA.  Units are not cut, and the CTAs get as many each, where so many of the longest
// take no more tiles longer than equal pieces than joining costs: kCutTiles, and one for kCutPieces
// full tiles of 128 rows written and read as partials, divided by the units a CTA gets.  Measured,
// whole units against pieces: 2 tiles of 64 rows 10.5 and 11.0 us, 3 tiles 11.6 and 11.2; 40 units of
// 8 tiles of 64 rows 21.2 and 17.6; 76 units of 20 full tiles 40.5 and 36.0, 100 units 42.4 and 43.3,
// 140 units 46.2 and 54.3; 128 units of 65 full tiles 97.8 and 101.5; 160 units of 4 full tiles 35.4
// and 34.0; 256 units of 3 tiles of 32 rows 26.5 and 30.7, 1024 of them 92.2 and 98.0.  A unit weighs
// kUnitTiles tiles more than it has (its rows' preparation and its output): with 2 the ragged batch
// takes 46.3 instead of 44.9 us, with 4 or 5 the same.
//
// Roles (512 threads; warp 3 only reports sequences whose rows are not known):
//   warp 0      the CTA's walk over its piece, published segment by segment, and the K pages by
//               TMA (two 128-byte-wide boxes a page, 128B-swizzled), whole key tiles;
//   warp 1      MMA: one elected lane issues tcgen05.mma and commits; owns the TMEM allocation;
//   warp 2      the V pages by TMA, 64 keys (half a tile) a stage;
//   warps 4-7   widen each half tile of V to f16, PV's operand;
//   warps 8-15  softmax: thread = query row = TMEM lane, two warps a row quarter that take 64 of a
//               tile's 128 keys each and exchange their maxima; also the Q operand, and half of
//               the output's dims each.
// The block takes all of the shared memory, which leaves 5 KB of L1: a spilled register costs an L2
// access, and the roles' loops have to share the instruction cache, so one warp alone walks over the
// sequences and every role's loop is written once.
//
// Precision.  K enters as its e4m3 codes, Q as the sum of two e4m3 terms of x = q 2^a (a per row,
// max |x| in [128, 256)): hi = e4m3(x), lo = e4m3(x - hi), both products into one accumulator.  A
// bf16 value has 8 significant bits and hi and lo keep 4 each, so x = hi + lo for every element
// within 2^-10 of the row's largest; below that the error stays under 2^-17 of the largest.
// P is rounded once, to f16, and V widened to f16 exactly: a second pair of e4m3 terms would be
// as fast on the tensor cores, but its smallest step, 2^-14 of the reference weight, loses the
// many small weights behind one large one; f16 keeps weights down to 2^-32 of it.
//
// Online softmax in the log2 domain with a lazy reference m: raised, and O rescaled in TMEM, only
// when a tile's row maximum exceeds it by more than kTau, so p_s = 2^(s - m + kShift) <= 2^14.
//
// Masks.  A tile that reaches into the tree takes each row's word, shifted to the tile's keys, as
// 128 bits.  Places that no row sees in full are kept out of PV by value too, since 0 * NaN is
// NaN: V rows behind the sequence are stored as zeros, and NaN codes of tree nodes are stored as
// 0 and put back (per row that sees them) in the epilogue.
//
// TMEM: S double buffer at columns 0 and 128 (a tile's P, f16 pairs, overwrites columns 0..63 of
// its buffer), O at 256..511.  The MMA warp issues QK(u), PV(u-1), QK(u+1), ...: MMAs of one
// thread execute in issue order, so QK(u+2) overwrites P(u) only after PV(u) has read it.
#include "common.cuh"
#include "host_checks.cuh"
#include "sm100.cuh"

#include "../../include/mtp_tree.h"

#include <cuda_fp8.h>
#include <math.h>

#include <algorithm>
#include <atomic>

namespace mtpattn {
namespace {

using namespace sm100;

constexpr int kTreeThreads = 512;
constexpr int kRows = 128;                         // query rows per tile
constexpr int kKeys = 128;                         // keys per tile
constexpr int kTilePages = kKeys / kPage;          // 8
constexpr int kHalfKeys = 64;                      // V is staged half a tile at a time
constexpr int kWarpWiden = 4, kWidenWarps = 4, kWarpSoft = 8, kSoftWarps = 8;
constexpr int kQHalf = kRows * 128;                // 128 of the 256 dims of one Q term
constexpr int kQTerm = 2 * kQHalf;                 // 32 KB: hi, then lo
constexpr int kKHalf = kKeys * 128;
constexpr int kKTile = 2 * kKHalf;                 // 32 KB per stage
constexpr int kKStages = 2;                        // as many as S buffers
constexpr int kV8Half = kHalfKeys * 128;           // 128 dims of 64 keys, e4m3
constexpr int kV8Stage = 2 * kV8Half;              // 16 KB per stage
constexpr int kVAtom = kHalfKeys * 128;            // 64 dims of 64 keys, f16
constexpr int kVStage = 4 * kVAtom;                // 32 KB per stage
constexpr int kVStages = 2;                        // of the codes, and of the operand
constexpr int kOffQ = 0;
constexpr int kOffK = kOffQ + 2 * kQTerm;
constexpr int kOffV8 = kOffK + kKStages * kKTile;
constexpr int kOffV = kOffV8 + kVStages * kV8Stage;
constexpr int kOffXch = kOffV + kVStages * kVStage;
constexpr int kOffBar = kOffXch + 2 * 2 * kRows * 4;   // exchange: [parity][half][row] floats
constexpr int kBarBytes = 1024;
constexpr int kSmemTree = kOffBar + kBarBytes;
static_assert(kSmemTree == 232448, "all that a block may have");
constexpr int kSCols = 128, kOCol = 256, kTmemCols = 512;
constexpr float kTau = 6.f, kShift = 8.f;
constexpr int kCutTiles = 4, kCutPieces = 40, kUnitTiles = 3;
constexpr uint32_t kBadLse = 0x7fd0bad1u;          // a partial of a sequence with a bad page (a NaN
                                                   // that no arithmetic makes)

// What the reduce goes by: a unit's note, written by the CTA that has its first key tile.
struct JoinNote {
  int pieces;                // it lies in; 1: written out whole
  int first, first_slot;     // the first of them, and the unit's slot there (in the others, 0)
  int q0, h, m, rows;        // its first node, KV head, row tile; valid rows of the tile
  int pad;
};

struct TreeAttnParams {
  CUtensorMap tmap_k, tmap_v;
  const __nv_bfloat16* q;
  int64_t q_stride_tok, q_stride_head;
  const uint8_t* v_cache;
  int64_t num_pages;
  const int32_t* block_tables;
  int32_t max_pages;
  const int32_t* seq_lens;
  const int32_t* cu_q;
  const uint64_t* mask;
  int32_t num_seqs, total_q, hq, hkv, ratio;
  const float* k_descale;
  const float* v_descale;
  float scale_log2;
  __nv_bfloat16* out;
  int64_t out_stride_tok, out_stride_head;
  int32_t* status;
  int32_t ctas;              // pieces of the line, at most
  float* o_part;             // [ctas][2][64][128][4]: blocks of 4 dims, rows, dims
  float* lse_part;           // [ctas][2][128]
  int32_t* units;            // for the reduce: the number of units (0: none was cut),
  JoinNote* notes;           // [units], at most unit_bound of them
  int32_t unit_bound;
};

struct Segment {             // part of one unit, key tiles t0 .. t1 - 1 of nt
  int b, h, q0, n, L;
  int m, t0, t1, nt, T;
  int16_t first;             // it starts the CTA's piece
  int16_t end;               // no segment: the piece is done
  int16_t bad;               // set on the way: it met a page outside the pool
  int16_t nan;               // ... the V of one of its tree nodes holds a NaN code
};
constexpr int kSegRing = 8;
constexpr int kNoScale = -128;

struct TreeBars {
  uint64_t k_full[kKStages], v_full[kVStages], v_empty[kVStages];
  uint64_t v8_full[kVStages], v8_empty[kVStages];
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t q_ready, o_free, final_mma;
  uint64_t xch[4][2];        // a row quarter's two warps meet, in turn on two barriers
  uint64_t seg_full[kSegRing], seg_free[kSegRing];
  Segment seg[kSegRing];     // written by the K producer, given back by the softmax warps
  uint32_t tmem_base;
  int32_t abort;
  int8_t q_scale[2][kRows];  // by segment parity: a of each row's x = q 2^a; kNoScale: not finite
  int32_t v8_note[kVStages][4];   // of a stage: keys of the sequence, first key of the tree, segment
};
static_assert(sizeof(TreeBars) <= kBarBytes, "barrier block");

// ---- the line of key tiles ---------------------------------------------------------------------

// One sequence on the line: T row tiles of nt key tiles for each KV head.  Rows whose place is not
// known (cu_seqlens_q out of order) take no part; other errors cost one key tile a unit.
struct Seq {
  int q0, n, L, T, nt, w, err;
};

__device__ __forceinline__ Seq seq_of(const TreeAttnParams& p, int q0, int q1, int L) {
  Seq s;
  s.q0 = q0;
  s.n = q1 - q0;
  s.L = L;
  s.err = 0;
  if (q0 < 0 || q1 <= q0 || q1 > p.total_q) {
    s.err = MTPATTN_ERR_QLEN;
    s.n = s.T = s.nt = s.w = 0;
    return s;
  }
  if (s.n > MTP_TREE_MAX_NODES) s.err = MTPATTN_ERR_QLEN;
  else if (s.n > L) s.err = MTPATTN_ERR_QLEN_GT_SEQ;
  else if (L > p.max_pages * kPage) s.err = MTPATTN_ERR_SEQ_TOO_LONG;
  s.T = (s.n * p.ratio + kRows - 1) / kRows;
  s.nt = s.err ? 1 : (L + kKeys - 1) / kKeys;
  s.w = s.T * (s.nt + kUnitTiles) * p.hkv;
  return s;
}

// Lane l's sequence b0 + l; past the last one of no weight.
__device__ __forceinline__ Seq seq_at(const TreeAttnParams& p, int b) {
  if (b < p.num_seqs) return seq_of(p, p.cu_q[b], p.cu_q[b + 1], p.seq_lens[b]);
  Seq s;
  s.q0 = s.n = s.L = s.T = s.nt = s.w = s.err = 0;
  return s;
}

__device__ __forceinline__ int warp_scan(int x, int lane) {    // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// How the line is cut: pieces of C places, piece g from g C on.  With V > 0 every unit takes V
// places on the line, and C is a multiple of V: no unit is cut.
struct Cut {
  int C, V, length, units;
};
__device__ __forceinline__ int weight_of(const Seq& s, int hkv, int V) { return V ? s.T * hkv * V : s.w; }

// Sum over the warp of numbers from 0 to 2^31 - 1.
__device__ __forceinline__ int64_t warp_total(int v) {
  return (static_cast<int64_t>(__reduce_add_sync(0xffffffffu, v >> 16)) << 16) + __reduce_add_sync(0xffffffffu, v & 0xffff);
}
__device__ __forceinline__ int add_up_to_max(int a, int b) {
  return static_cast<int>(min(static_cast<uint32_t>(a) + static_cast<uint32_t>(b), static_cast<uint32_t>(INT32_MAX)));
}

// By the whole warp; `mine` is lane l's sequence l (of the first 32).
__device__ __forceinline__ Cut cut_line(const TreeAttnParams& p, int lane, const Seq& mine) {
  int W = mine.w, N = mine.n, U = mine.T * p.hkv, longest = mine.nt;
#pragma unroll 1
  for (int b0 = 32; b0 < p.num_seqs; b0 += 32) {
    const Seq x = seq_at(p, b0 + lane);
    W = add_up_to_max(W, x.w);
    N = add_up_to_max(N, x.n);
    U += x.T * p.hkv;
    longest = max(longest, x.nt);
  }
  // Sequences that claim the same rows again and again (cu_seqlens_q far out of order) could make the line
  // longer than any call's is: then nothing is computed.
  const int64_t all = warp_total(W);
  if (all > INT32_MAX || warp_total(N) > 2ll * p.total_q) {
    if (blockIdx.x == 0 && lane == 0) set_status(p.status, MTPATTN_ERR_QLEN);
    return {1, 1, 0, 0};
  }
  W = static_cast<int>(all);
  U = __reduce_add_sync(0xffffffffu, U);
  longest = __reduce_max_sync(0xffffffffu, longest);
  Cut c;
  c.C = max(1, (W + p.ctas - 1) / p.ctas);
  c.V = 0;
  c.length = W;
  c.units = U;
  // What cutting costs, in tiles: the join, and its bytes (pieces, less for tiles that are not full).
  const float rows = static_cast<float>(p.total_q) * static_cast<float>(p.ratio * p.hkv);
  const float full = fminf(1.f, rows / static_cast<float>(kRows * max(U, 1)));
  const int join = kCutTiles + static_cast<int>(static_cast<float>(U + p.ctas) * full * (1.f / kCutPieces));
  const int each = max(1, (U + p.ctas - 1) / p.ctas);
  if (static_cast<int64_t>(each) * (longest + kUnitTiles) <= c.C + join / each &&
      static_cast<int64_t>(U) * longest <= INT32_MAX) {
    c.V = longest;
    c.C = each * longest;
    c.length = U * longest;
  }
  return c;
}

// The K producer's walk over the units of its CTA's piece; 32 sequences are held, one a lane.
struct Walker {
  int pos, hi, lo;
  int b0, before;            // the held sequences, and the line before the first of them
  int units_before;          // ... and the units
  Seq mine;
  int upto, units_upto;      // running sums of the held sequences' weights and units
  int unit, unit0, unit_places;  // the last segment's unit: its number, and place on the line
  Cut cut;

  __device__ __forceinline__ void start(const TreeAttnParams& p, int lane) {
    b0 = before = units_before = unit = unit0 = unit_places = 0;
    mine = seq_at(p, lane);
    cut = cut_line(p, lane, mine);
    upto = warp_scan(weight_of(mine, p.hkv, cut.V), lane);
    units_upto = warp_scan(mine.T * p.hkv, lane);
    lo = pos = min(static_cast<int64_t>(cut.length), static_cast<int64_t>(blockIdx.x) * cut.C);
    hi = min(static_cast<int64_t>(cut.length), static_cast<int64_t>(lo) + cut.C);
  }
  // The next segment; s.end if there is none.  Returns the sequence's error bits.
  __device__ __forceinline__ int next(const TreeAttnParams& p, int lane, Segment& s) {
    s.end = 1;
#pragma unroll 1
    while (pos < hi) {
      const int all = __shfl_sync(0xffffffffu, upto, 31);
      if (pos >= before + all) {
        before += all;
        units_before += __shfl_sync(0xffffffffu, units_upto, 31);
        b0 += 32;
        if (b0 >= p.num_seqs) return 0;             // lengths changed under the call
        mine = seq_at(p, b0 + lane);
        upto = warp_scan(weight_of(mine, p.hkv, cut.V), lane);
        units_upto = warp_scan(mine.T * p.hkv, lane);
        continue;
      }
      const int at = pos - before;
      const int f = __ffs(__ballot_sync(0xffffffffu, upto > at)) - 1;
      const int nt = __shfl_sync(0xffffffffu, mine.nt, f), T = __shfl_sync(0xffffffffu, mine.T, f);
      const int extra = cut.V ? 0 : kUnitTiles;     // places ahead of the unit's key tiles
      const int places = cut.V ? cut.V : nt + extra;
      const int in = at - (f ? __shfl_sync(0xffffffffu, upto, f - 1) : 0);
      const int nth = in / places, in_unit = in - nth * places;
      unit = units_before + nth + (f ? __shfl_sync(0xffffffffu, units_upto, f - 1) : 0);
      unit0 = pos - in_unit;
      unit_places = places;
      const int to = min(places, in_unit + hi - pos);                // of the unit, in this piece
      s.t0 = max(0, in_unit - extra);
      s.t1 = min(nt, to - extra);
      pos += to - in_unit;
      if (s.t0 >= s.t1) continue;                   // none of its key tiles
      s.b = b0 + f;
      s.q0 = __shfl_sync(0xffffffffu, mine.q0, f);
      s.n = __shfl_sync(0xffffffffu, mine.n, f);
      s.L = __shfl_sync(0xffffffffu, mine.L, f);
      s.h = nth / T;
      s.m = nth - s.h * T;
      s.nt = nt;
      s.T = T;
      s.first = unit0 <= lo;
      s.end = s.bad = s.nan = 0;
      return __shfl_sync(0xffffffffu, mine.err, f);
    }
    return 0;
  }
  // What the reduce has to know of the last segment's unit.
  __device__ __forceinline__ JoinNote note(const TreeAttnParams& p, const Segment& s) const {
    JoinNote n;
    n.first = blockIdx.x;
    n.pieces = cut.V ? 1 : (unit0 + unit_places - 1) / cut.C - n.first + 1;
    n.first_slot = s.first ? 0 : 1;
    n.q0 = s.q0;
    n.h = s.h;
    n.m = s.m;
    n.rows = min(kRows, s.n * p.ratio - s.m * kRows);
    n.pad = 0;
    return n;
  }
};

__device__ __forceinline__ int tile_pages(int L, int t) {   // pages of key tile t
  return min(kTilePages, (L + kPage - 1) / kPage - t * kTilePages);
}

// ---- arithmetic --------------------------------------------------------------------------------

__device__ __forceinline__ float exp2_hw(float x) {   // 2^x, hardware approximation
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// (a0, a1) = (a0, a1) * b + c, one instruction for the pair
__device__ __forceinline__ void fma_pair(float& a0, float& a1, float b, float c) {
  asm("{\n .reg .b64 ra, rb, rc;\n mov.b64 ra, {%0, %1};\n mov.b64 rb, {%2, %2};\n"
      " mov.b64 rc, {%3, %3};\n fma.rn.f32x2 ra, ra, rb, rc;\n mov.b64 {%0, %1}, ra;\n}\n"
      : "+f"(a0), "+f"(a1)
      : "f"(b), "f"(c));
}
__device__ __forceinline__ void add_pair(float& a0, float& a1, float b0, float b1) {
  asm("{\n .reg .b64 ra, rb;\n mov.b64 ra, {%0, %1};\n mov.b64 rb, {%2, %3};\n"
      " add.rn.f32x2 ra, ra, rb;\n mov.b64 {%0, %1}, ra;\n}\n"
      : "+f"(a0), "+f"(a1)
      : "f"(b0), "f"(b1));
}
// two f32 -> f16x2 (a in the low half: the lower K index of a TMEM A-operand cell)
__device__ __forceinline__ uint32_t half2_of(float a, float b) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(d) : "f"(b), "f"(a));
  return d;
}
// four e4m3 codes (lowest byte first) -> two f16x2 words, exactly
__device__ __forceinline__ void widen(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n"
      " cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
// Four bf16 values (two words) scaled by f (bf16x2, powers of two: exact) as e4m3 codes hi + lo,
// lowest byte first.  In f16 a scaled value is exact down to 2^-17, and so is the remainder.
__device__ __forceinline__ void two_terms(uint32_t w0, uint32_t w1, uint32_t f, uint32_t& hi, uint32_t& lo) {
  asm("{\n"
      " .reg .b16 a0, a1, b0, b1, h0, h1, l0, l1, z;\n"
      " .reg .b32 x0, x1, e0, e1, e2, e3, g0, g1;\n"
      " mul.rn.bf16x2 x0, %2, %4;\n"
      " mul.rn.bf16x2 x1, %3, %4;\n"
      " mov.b16 z, 0;\n"
      " mov.b32 {a0, a1}, x0;\n"
      " mov.b32 {b0, b1}, x1;\n"
      " mov.b32 e0, {z, a0};\n"
      " mov.b32 e1, {z, a1};\n"
      " mov.b32 e2, {z, b0};\n"
      " mov.b32 e3, {z, b1};\n"
      " cvt.rn.f16x2.f32 x0, e1, e0;\n"
      " cvt.rn.f16x2.f32 x1, e3, e2;\n"
      " cvt.rn.satfinite.e4m3x2.f16x2 h0, x0;\n"
      " cvt.rn.satfinite.e4m3x2.f16x2 h1, x1;\n"
      " cvt.rn.f16x2.e4m3x2 g0, h0;\n"
      " cvt.rn.f16x2.e4m3x2 g1, h1;\n"
      " sub.rn.f16x2 x0, x0, g0;\n"
      " sub.rn.f16x2 x1, x1, g1;\n"
      " cvt.rn.satfinite.e4m3x2.f16x2 l0, x0;\n"
      " cvt.rn.satfinite.e4m3x2.f16x2 l1, x1;\n"
      " mov.b32 %0, {h0, h1};\n"
      " mov.b32 %1, {l0, l1};\n"
      "}\n"
      : "=r"(hi), "=r"(lo)
      : "r"(w0), "r"(w1), "r"(f));
}
// The larger |value| of two bf16 pairs, half by half; NaN is above all.
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
  return __vmaxu2(a & 0x7fff7fffu, b & 0x7fff7fffu);
}
// mbar_wait of sm100.cuh in fewer instructions (there are many waits, and the loops of all the
// roles share one instruction cache): a 32-bit clock, in which kWaitCycles fits.
static_assert(kWaitCycles < (1ll << 32), "32-bit clock");
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int* abort) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint32_t t0 = static_cast<uint32_t>(clock());
#pragma unroll 1
  while (!mbar_try_wait(bar, parity)) {
    if (static_cast<uint32_t>(clock()) - t0 > static_cast<uint32_t>(kWaitCycles)) *abort = 1;
    if (*abort) return false;
  }
  return true;
}

// A load that stays before the arrival behind it (volatile, as that is)
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// tcgen05.mma kind::f16 (f16 x f16 -> f32), A from tensor memory, B from shared memory.
__device__ __forceinline__ void mma_pv(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__global__ void __launch_bounds__(kTreeThreads, 1)
tree_attn_kernel(const __grid_constant__ TreeAttnParams p) {
  extern __shared__ __align__(1024) unsigned char base[];
  if (smem_u32(base) & 1023) {                     // the operands' swizzle needs it; no kernel sets
    if (threadIdx.x == 0) set_status(p.status, MTPATTN_ERR_TIMEOUT);   // other shared memory aside
    return;
  }
  TreeBars& bars = *reinterpret_cast<TreeBars*>(base + kOffBar);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = &bars.abort;

  // ---- set-up ------------------------------------------------------------------------------
  if (warp == 1) {
    tmem_alloc(smem_u32(&bars.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < kKStages; ++i) mbar_init(smem_u32(&bars.k_full[i]), 1);
    for (int i = 0; i < kVStages; ++i) {
      mbar_init(smem_u32(&bars.v_full[i]), kWidenWarps);
      mbar_init(smem_u32(&bars.v_empty[i]), 1);
      mbar_init(smem_u32(&bars.v8_full[i]), 1);
      mbar_init(smem_u32(&bars.v8_empty[i]), kWidenWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars.s_full[i]), 1);
      mbar_init(smem_u32(&bars.p_full[i]), kSoftWarps);
      mbar_init(smem_u32(&bars.pv_done[i]), 1);
    }
    mbar_init(smem_u32(&bars.q_ready), kSoftWarps);
    mbar_init(smem_u32(&bars.o_free), kSoftWarps);
    for (int i = 0; i < 8; ++i) mbar_init(smem_u32(&bars.xch[i >> 1][i & 1]), 2);
    for (int i = 0; i < kSegRing; ++i) {
      mbar_init(smem_u32(&bars.seg_full[i]), 1);
      mbar_init(smem_u32(&bars.seg_free[i]), kSoftWarps);
    }
    mbar_init(smem_u32(&bars.final_mma), 1);
    bars.abort = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem_base;
  // A programmatic dependent of the previous work on the stream: nothing global was touched so
  // far; and the reduce may be scheduled (it waits for this grid before it reads partials).
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");

  // Segment e as the K producer published it; false after an abort.
  auto seg_wait = [&](int e) -> bool {
    return __all_sync(0xffffffffu, wait_for(smem_u32(&bars.seg_full[e % kSegRing]),
                                             (e / kSegRing) & 1, abort_flag));
  };

  if (warp == 0) {
    // ============================== K producer, and the CTA's walk ================================
    if (lane == 0) prefetch_tmap(&p.tmap_k);
    Walker walk;
    walk.start(p, lane);
    if (blockIdx.x == 0 && lane == 0) *p.units = walk.cut.V ? 0 : min(walk.cut.units, p.unit_bound);
    // keys that other row tiles will read again stay in L2
    const uint64_t once = l2_policy_evict_first();
    uint64_t again;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;\n" : "=l"(again));
    uint32_t u = 0;
    int e = 0;
    bool ok = true;
    while (ok) {
      Segment s;
      const int err = walk.next(p, lane, s);
      auto leave_note = [&]() {
        if (lane == 0 && s.t0 == 0 && !walk.cut.V && walk.unit < p.unit_bound) p.notes[walk.unit] = walk.note(p, s);
      };
      if (err && !s.end) {
        leave_note();
        // zeros for the rows of a sequence that cannot be computed, here: it has no key tiles
        if (lane == 0) set_status(p.status, err);
        const int rows = min(kRows, s.n * p.ratio - s.m * kRows);
#pragma unroll 1
        for (int i = 0; i < rows; ++i) {
          const int rr = s.m * kRows + i, t = rr / p.ratio;
          reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(s.q0 + t) * p.out_stride_tok +
                                   static_cast<int64_t>(s.h * p.ratio + rr - t * p.ratio) * p.out_stride_head)[lane] =
              make_uint4(0u, 0u, 0u, 0u);
        }
        continue;
      }
      ok = __all_sync(0xffffffffu, wait_for(smem_u32(&bars.seg_free[e % kSegRing]),
                                             ((e / kSegRing) & 1) ^ 1, abort_flag));
      if (!ok) break;
      if (lane == 0) {
        bars.seg[e % kSegRing] = s;
        mbar_arrive(smem_u32(&bars.seg_full[e % kSegRing]));
      }
      if (s.end) break;
      ++e;
      leave_note();
      const int32_t* bt = p.block_tables + static_cast<int64_t>(s.b) * p.max_pages;
      const uint64_t pol = s.T == 1 ? once : again;
      // Table entries, a lane one of four tiles' 32, with the next 32 on the way: a load of its own
      // per tile would put its latency, some 2000 cycles, into every turn.
      const int pages = (s.L + kPage - 1) / kPage;
      auto entries = [&](int t) -> int {
        const int pg = t * kTilePages + lane;
        return pg < pages ? bt[pg] : 0;
      };
      int now = entries(s.t0), ahead = entries(s.t0 + 4);
#pragma unroll 1
      for (int t = s.t0; t < s.t1; ++t, ++u) {
        const int np = tile_pages(s.L, t), st = u % kKStages;
        const int four = (t - s.t0) & 3;
        if (four == 0 && t > s.t0) {
          now = ahead;
          ahead = entries(t + 4);
        }
        const int phys = __shfl_sync(0xffffffffu, now, (four * kTilePages + lane) & 31);
        const uint32_t fb = smem_u32(&bars.k_full[st]);
        if (lane == 0) {
          // tile u - 2, of the same stage, has been multiplied when its S is there
          ok = u < kKStages || wait_for(smem_u32(&bars.s_full[st]), ((u / kKStages) & 1) ^ 1, abort_flag);
          if (ok) mbar_arrive_expect_tx(fb, np * 2 * 2048);
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        if (lane < np) {                            // a page outside the pool reads as zeros
          const uint32_t dst = smem_u32(base + kOffK + st * kKTile) + lane * 2048;
          tma_load_4d(dst, &p.tmap_k, fb, 0, s.h, 0, phys, pol);
          tma_load_4d(dst + kKHalf, &p.tmap_k, fb, 128, s.h, 0, phys, pol);
        }
      }
    }
    // never leave with copies in flight
    if (lane == 0) {
      volatile int no_abort = 0;
      for (uint32_t k = 1; k <= kKStages && k <= u; ++k)
        wait_for(smem_u32(&bars.k_full[(u - k) % kKStages]), ((u - k) / kKStages) & 1, &no_abort);
    }
  } else if (warp == 1) {
    // ======================================== MMA issuer ==========================================
    constexpr uint32_t kIdescQK = idesc_e4m3_f32(kRows, kKeys, false);
    constexpr uint32_t kIdescPV = idesc_e4m3_f32(kRows, kHeadDim, true);   // f16: format code 0
    const uint64_t q_desc = sdesc_sw128(smem_u32(base + kOffQ), 16, 1024);
    const uint64_t k_desc = sdesc_sw128(smem_u32(base + kOffK), 16, 1024);
    const uint64_t v_desc = sdesc_sw128(smem_u32(base + kOffV), kVAtom, 1024);
    // One thread runs the whole loop: whatever it does between products leaves the tensor cores
    // idle once their short queue is empty, so it takes no votes and as few commits as it can (a
    // K stage is free when its S buffer is full: both are tile u's, u mod 2).
    if (elect_one()) {
      auto wait = [&](uint64_t& bar, uint32_t parity) -> bool {
        return wait_for(smem_u32(&bar), parity, abort_flag);
      };
      // A turn is QK of a tile and the products of the tile before it; a segment's last products
      // go out in a turn of their own, before the next segment is waited for.
      uint32_t u = 0, v = 0;                        // key tiles, half tiles of V
      int seg = 0, t = 0, t0 = 0, t1 = 0, pages = 0;
      int pv_pages = 0;                             // of tile u - 1, 0: nothing outstanding
      uint32_t pv_acc = 0;                          // ... 0: it starts its segment's sums
      while (true) {
        const bool more = t < t1 || pv_pages == 0;
        if (t >= t1 && more) {
          if (!wait(bars.seg_full[seg % kSegRing], (seg / kSegRing) & 1)) break;
          const Segment& s = bars.seg[seg % kSegRing];
          if (s.end) break;
          t = t0 = s.t0;
          t1 = s.t1;
          pages = (s.L + kPage - 1) / kPage;
          if (!wait(bars.q_ready, seg & 1)) break;
          ++seg;
        }
        if (more) {
          const int st = u % kKStages;
          if (!wait(bars.k_full[st], (u / kKStages) & 1)) break;
          tc_fence_after();
          const uint64_t kd = k_desc + (st * kKTile >> 4);
#pragma unroll
          for (int k = 0; k < 16; ++k) {            // hi: dims 32 k .. + 31, then lo
            const uint32_t a_off = (k >> 3) * kQTerm + ((k >> 2) & 1) * kQHalf + (k & 3) * 32;
            const uint32_t b_off = ((k >> 2) & 1) * kKHalf + (k & 3) * 32;
            mma_f8_ss(tmem + (u & 1) * kSCols, q_desc + (a_off >> 4), kd + (b_off >> 4), kIdescQK,
                      k > 0 ? 1u : 0u);
          }
          mma_commit(smem_u32(&bars.s_full[u & 1]));
        }
        if (pv_pages > 0) {
          const uint32_t ut = u - 1;
          // a segment's first products overwrite O: the epilogue before it has read it
          if (pv_acc == 0 && seg > 1 && !wait(bars.o_free, (seg - 2) & 1)) break;
          if (!wait(bars.p_full[ut & 1], (ut >> 1) & 1)) break;
          bool ok = true;
#pragma unroll 1
          for (int k0 = 0; k0 < pv_pages; k0 += 4, ++v) {   // a half tile: four pages, 16 keys each
            const int st = v % kVStages;
            ok = wait(bars.v_full[st], (v / kVStages) & 1);
            if (!ok) break;
            tc_fence_after();
            const uint32_t p_tmem = tmem + (ut & 1) * kSCols + 8 * k0;
            const uint64_t vd = v_desc + (st * kVStage >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (k0 + k < pv_pages) mma_pv(tmem + kOCol, p_tmem + 8 * k, vd + (k * 2048 >> 4), kIdescPV, pv_acc);
              pv_acc = 1;
            }
            mma_commit(smem_u32(&bars.v_empty[st]));
          }
          if (!ok) break;
          mma_commit(smem_u32(&bars.pv_done[ut & 1]));
        }
        pv_pages = 0;
        if (more) {
          pv_pages = min(kTilePages, pages - t * kTilePages);
          pv_acc = t != t0;
          ++t;
          ++u;
        }
      }
      mma_commit(smem_u32(&bars.final_mma));
      volatile int no_abort = 0;
      wait_for(smem_u32(&bars.final_mma), 0, &no_abort);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ======================================== V producer ==========================================
    if (lane == 0) prefetch_tmap(&p.tmap_v);
    const uint64_t once = l2_policy_evict_first();
    uint64_t again;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;\n" : "=l"(again));
    uint32_t v = 0;                                 // half tiles
    bool ok = true;
#pragma unroll 1
    for (int e = 0; ok; ++e) {
      if (!seg_wait(e)) break;
      Segment& s = bars.seg[e % kSegRing];
      if (s.end) break;
      const int32_t* bt = p.block_tables + static_cast<int64_t>(s.b) * p.max_pages;
      const uint64_t pol = s.T == 1 ? once : again;
      const int pages = (s.L + kPage - 1) / kPage, h = s.h, L = s.L, tree0 = s.L - s.n;
      const int h0 = 2 * s.t0, h1 = min(2 * s.t1, (pages + 3) / 4);
      auto entries = [&](int hf) -> int {           // of eight half tiles, the next eight ahead
        const int pg = 4 * hf + lane;
        return pg < pages ? bt[pg] : 0;
      };
      int now = entries(h0), ahead = entries(h0 + 8);
#pragma unroll 1
      for (int hf = h0; hf < h1; ++hf, ++v) {
        const int np = min(4, pages - 4 * hf), st = v % kVStages;
        const int eight = (hf - h0) & 7;
        if (eight == 0 && hf > h0) {
          now = ahead;
          ahead = entries(hf + 8);
        }
#ifdef MTPATTN_TEST_STALL
        if (blockIdx.x == 0 && v == 0) continue;    // test builds: the wait for these codes runs out
#endif
        const int phys = __shfl_sync(0xffffffffu, now, (4 * eight + lane) & 31);
        const bool bad = __any_sync(0xffffffffu, lane < np && (phys < 0 || phys >= p.num_pages));
        const uint32_t fb = smem_u32(&bars.v8_full[st]);
        if (lane == 0) {
          ok = wait_for(smem_u32(&bars.v8_empty[st]), ((v / kVStages) & 1) ^ 1, abort_flag);
          if (ok) {
            if (bad) s.bad = 1;
            bars.v8_note[st][0] = L - hf * kHalfKeys;
            bars.v8_note[st][1] = tree0 - hf * kHalfKeys;
            bars.v8_note[st][2] = e % kSegRing;
            mbar_arrive_expect_tx(fb, np * 2 * 2048);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        if (lane < np) {
          const uint32_t dst = smem_u32(base + kOffV8 + st * kV8Stage) + lane * 2048;
          tma_load_4d(dst, &p.tmap_v, fb, 0, h, 0, phys, pol);
          tma_load_4d(dst + kV8Half, &p.tmap_v, fb, 128, h, 0, phys, pol);
        }
      }
    }
    // the last stages' copies, and the end for the widening warps (which have seen those by then)
    if (lane == 0) {
      volatile int no_abort = 0;
      for (uint32_t k = 1; k <= kVStages && k <= v; ++k)
        wait_for(smem_u32(&bars.v8_full[(v - k) % kVStages]), ((v - k) / kVStages) & 1, &no_abort);
      const int st = v % kVStages;
      if (ok && wait_for(smem_u32(&bars.v8_empty[st]), ((v / kVStages) & 1) ^ 1, abort_flag)) {
        bars.v8_note[st][2] = -1;
        mbar_arrive(smem_u32(&bars.v8_full[st]));
      }
    }
  } else if (warp == 3) {
    // ============================ sequences whose rows are not known ==============================
    if (blockIdx.x == 0)
#pragma unroll 1
      for (int b0 = 0; b0 < p.num_seqs; b0 += 32) {
        const Seq x = seq_at(p, b0 + lane);
        if (x.err && x.T == 0) set_status(p.status, x.err);
      }
  } else if (warp >= kWarpWiden && warp < kWarpSoft) {
    // ======================================== V widening ==========================================
    // A thread takes one 16-byte chunk (16 dims) of the keys key0 + 16 i in both 128-dim halves: all
    // have the same key % 8, hence the same swizzled positions.  The eight threads of a load or
    // store phase take chunks 0-3 of a key and 4-7 of its neighbour (or the other way round): these
    // lie in all eight 16-byte positions of the codes' rows, and, as the operand's two f16 chunks
    // each, of its 64-dim atoms too.
    const int c = threadIdx.x - kWarpWiden * 32;
    const int key0 = 2 * (c >> 4) + ((c >> 2) & 1), x7 = key0 & 7;
    const int chunk = (c & 7) ^ (((c >> 3) & 1) << 2);
    const uint32_t from = key0 * 128 + ((chunk ^ x7) << 4);
    const uint32_t to = (chunk >> 2) * kVAtom + key0 * 128;
    const uint32_t to0 = to + (((2 * (chunk & 3)) ^ x7) << 4), to1 = to + (((2 * (chunk & 3) + 1) ^ x7) << 4);
#pragma unroll 1
    for (uint32_t v = 0;; ++v) {
      const int st = v % kVStages;
      const uint32_t parity = (v / kVStages) & 1;
      if (!__all_sync(0xffffffffu, wait_for(smem_u32(&bars.v8_full[st]), parity, abort_flag))) break;
      const int keys = bars.v8_note[st][0], tree = bars.v8_note[st][1], seg = bars.v8_note[st][2];
      if (seg < 0) break;
      const unsigned char* src = base + kOffV8 + st * kV8Stage + from;
      unsigned char* dst = base + kOffV + st * kVStage;
      uint4 a[8];                                   // keys key0 + 16 (i % 4), half i / 4
#pragma unroll
      for (int i = 0; i < 8; ++i)
        a[i] = lds128(smem_u32(src) + (i >> 2) * kV8Half + (i & 3) * 2048);
      // the codes are in registers: the stage can be loaded again while they are widened
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars.v8_empty[st]));
      if (keys < kHalfKeys) {                       // places behind the sequence: zeros
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (key0 + 16 * (i & 3) >= keys) a[i] = make_uint4(0u, 0u, 0u, 0u);
      }
      bool nan = false;
      if (tree < kHalfKeys) {                       // NaN codes of tree nodes: noted, and 0 instead
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t any = ((a[i].x & 0x7f7f7f7fu) + 0x01010101u) | ((a[i].y & 0x7f7f7f7fu) + 0x01010101u) |
                               ((a[i].z & 0x7f7f7f7fu) + 0x01010101u) | ((a[i].w & 0x7f7f7f7fu) + 0x01010101u);
          nan |= key0 + 16 * (i & 3) >= tree && (any & 0x80808080u);
        }
      }
      if (!__all_sync(0xffffffffu, wait_for(smem_u32(&bars.v_empty[st]), parity ^ 1, abort_flag))) break;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint4 c0, c1;
        widen(a[i].x, c0.x, c0.y);
        widen(a[i].y, c0.z, c0.w);
        widen(a[i].z, c1.x, c1.y);
        widen(a[i].w, c1.z, c1.w);
        unsigned char* d = dst + (i >> 2) * 2 * kVAtom + (i & 3) * 2048;
        *reinterpret_cast<uint4*>(d + to0) = c0;
        *reinterpret_cast<uint4*>(d + to1) = c1;
      }
      if (nan) {                                    // this thread's chunks once more, as they were stored
        bars.seg[seg].nan = 1;
#pragma unroll 1
        for (int i = 0; i < 16; ++i) {
          uint32_t* x = reinterpret_cast<uint32_t*>(dst + (i >> 3) * 2 * kVAtom + (i & 3) * 2048 + ((i & 4) ? to1 : to0));
          if (key0 + 16 * (i & 3) >= tree)
#pragma unroll 1
            for (int d = 0; d < 4; ++d) {
              const uint32_t h = x[d];
              x[d] = ((h & 0x7fffu) > 0x7c00u ? 0u : h & 0xffffu) |
                     ((h & 0x7fff0000u) > 0x7c000000u ? 0u : h & 0xffff0000u);
            }
        }
      }
      fence_proxy_async_smem();                     // visible to the tensor cores behind v_full
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars.v_full[st]));
    }
  } else if (warp >= kWarpSoft) {
    // ======================================= softmax (rows) =======================================
    const int quad = warp & 3;                      // TMEM lane quarter
    const int half = (warp - kWarpSoft) >> 2;       // keys 64 half .. + 63, output dims 128 half ..
    const int r = 32 * quad + lane;                 // query row of the tile, TMEM lane
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(32 * quad) << 16);
    float* xch = reinterpret_cast<float*>(base + kOffXch);
    // A negative factor goes into Q, so that the factors are positive; one of 0 is taken as the
    // smallest float, under which all logits are alike.
    const float sl_in = p.scale_log2 * __ldg(p.k_descale);
    const float sl = fmaxf(fabsf(sl_in), 1.17549435e-38f);
    const uint32_t flip = sl_in < 0.f ? 0x80008000u : 0u;
    const float vd = __ldg(p.v_descale);
    uint32_t u = 0;                                 // key tiles so far
    // The two warps of a row quarter meet: what each wrote to shared memory before, the other
    // sees after.  Bounded like every wait.
    uint32_t meets = 0;
    auto meet = [&]() -> bool {
      const uint32_t bar = smem_u32(&bars.xch[quad][meets & 1]);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
      const bool ok = __all_sync(0xffffffffu, wait_for(bar, (meets >> 1) & 1, abort_flag));
      ++meets;
      return ok;
    };

    // The rows as two e4m3 terms into the Q operand: warp w of the 8 takes rows w, w + 8, ..., so that
    // few rows are soon done (by quarters the warps of a full tile take as long, those of 64 rows
    // twice as long).  A row fills four 128-byte lines there (terms x 128-dim halves), as many bytes
    // as in bf16: the rows are first copied to where their own terms will be, all in flight, and then
    // taken four at a time by the whole warp (8 dims a lane).  Loops stay rolled: fetching
    // straight-line code for 8 rows at a time cost 9000 cycles at the start of every CTA.  What a
    // row was scaled by goes to q_scale, from where `factor`, this thread's row's factor from raw products
    // to log2 units (NaN for a row that is not finite), is made when all warps are done.
    auto prepare_q = [&](const Segment& y, int e, float& factor) -> bool {
      const int w = warp - kWarpSoft;
      const int rows = y.n * p.ratio - y.m * kRows;                  // valid rows of the tile, or more
      // a row quarter without any valid row is not computed; one with some is finite throughout
      const int upto = 4 * min(4, (rows + 31) >> 5);
      const int mine = y.m * kRows + 8 * (lane & 15) + w;
      const int t = mine / p.ratio, g = mine - t * p.ratio;
      const int64_t at = static_cast<int64_t>(y.q0 + t) * p.q_stride_tok +
                         static_cast<int64_t>(y.h * p.ratio + g) * p.q_stride_head;
      // 16 bytes a lane: block lane / 8 of the four, 16 (lane % 8) bytes into the row's 128 there
      const uint32_t own = smem_u32(base + kOffQ) + (lane >> 4) * kQTerm + ((lane >> 3) & 1) * kQHalf +
                           w * 128 + (lane & 7) * 16;
#pragma unroll 4
      for (int i = 0; i < upto; ++i) {
        const int64_t src = __shfl_sync(0xffffffffu, at, i);
        const bool in = 8 * i + w < rows;                            // if not, zeros are written
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(own + i * 1024),
                     "l"(p.q + (in ? src : 0) + 8 * lane), "r"(in ? 16u : 0u) : "memory");
      }
      asm volatile("cp.async.wait_all;\n" ::: "memory");
      unsigned char* q_hi = base + kOffQ + (lane >> 4) * kQHalf + w * 128 + 8 * (lane & 1) +
                            ((((lane & 15) >> 1) ^ w) << 4);
#pragma unroll 1
      for (int i0 = 0; i0 < upto; i0 += 4) {         // four rows' chains of steps side by side
        uint4 x[4];
        uint32_t top[4];                             // the largest |q| by its bits (NaN above all)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = lds128(own + (i0 + i) * 1024);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t m = max_abs2(max_abs2(x[i].x, x[i].y), max_abs2(x[i].z, x[i].w));
          top[i] = max(m << 16, m & 0xffff0000u);    // as an f32's bits
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) top[i] = __reduce_max_sync(0xffffffffu, top[i]);
        __syncwarp();                                // every lane has read its part of the rows
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e8 = static_cast<int>(top[i] >> 23);             // exponent field
          // 2^a takes the largest into [128, 256), as far as a = 126 does
          const int a = top[i] == 0u ? 0 : min(126, 134 - e8);
          const uint32_t f = (static_cast<uint32_t>(a + 127) << 7) * 0x10001u | flip;
          uint32_t hi[2], lo[2];
          two_terms(x[i].x, x[i].y, f, hi[0], lo[0]);
          two_terms(x[i].z, x[i].w, f, hi[1], lo[1]);
          unsigned char* dst = q_hi + (i0 + i) * 1024;
          *reinterpret_cast<uint2*>(dst) = make_uint2(hi[0], hi[1]);
          *reinterpret_cast<uint2*>(dst + kQTerm) = make_uint2(lo[0], lo[1]);
          if (lane == i) bars.q_scale[e & 1][8 * (i0 + i) + w] = static_cast<int8_t>(e8 == 255 ? kNoScale : a);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      const uint32_t bar = smem_u32(&bars.q_ready);
      if (lane == 0) mbar_arrive(bar);
      if (!__all_sync(0xffffffffu, wait_for(bar, e & 1, abort_flag))) return false;
      const int a = *reinterpret_cast<const volatile int8_t*>(&bars.q_scale[e & 1][r]);
      factor = a == kNoScale || sl_in != sl_in ? __int_as_float(0x7fc00000)
                                               : fmaxf(sl * __int_as_float((127 - a) << 23), 1.17549435e-38f);
      return true;
    };

    float m = -INFINITY, l = 0.f;                   // of this thread's row in the segment at hand
    uint64_t word = 0;                              // the tree nodes it sees
    bool valid = false, active = false, nan_row = false, alive = true;
    // A turn: the next segment's Q while the last products of the one before run, that one's
    // epilogue, then the segment's tiles.  The first turn has no epilogue, the last nothing else.
#pragma unroll 1
    for (int e = 0; alive; ++e) {
      if (!seg_wait(e)) break;
      const Segment& y = bars.seg[e % kSegRing];
      const bool end = y.end != 0;
      float sl2_next = 0.f;
      if (!end && !prepare_q(y, e, sl2_next)) break;
      if (e > 0) {
        const Segment& s = bars.seg[(e - 1) % kSegRing];
        // the row's sum over both halves
        if (active) {
          float* both = xch + (meets & 1) * 2 * kRows;
          both[half * kRows + r] = l;
          if (!meet()) break;
          l += both[(half ^ 1) * kRows + r];
          if (nan_row && l != 0.f) l = __int_as_float(0x7fc00000);
        }
        const uint32_t last = u - 1;
        // ---- epilogue: o = v_descale O / l, lse = m + log2 l ---------------------------------------
        if (!__all_sync(0xffffffffu,
                        (s.t1 == s.t0 + 1 ||
                         wait_for(smem_u32(&bars.pv_done[(last - 1) & 1]), ((last - 1) >> 1) & 1, abort_flag)) &&
                            wait_for(smem_u32(&bars.pv_done[last & 1]), (last >> 1) & 1, abort_flag)))
          break;
        tc_fence_after();
        const bool bad = *reinterpret_cast<const volatile int16_t*>(&s.bad) != 0;
        const bool nan_v = *reinterpret_cast<const volatile int16_t*>(&s.nan) != 0;
        if (bad && lane == 0 && half == 0) set_status(p.status, MTPATTN_ERR_PAGE);
        const bool whole = s.t0 == 0 && s.t1 == s.nt;
        if (active) {
          const float sc = l != 0.f && !bad ? vd / l : 0.f;   // NaN stays NaN
          const int slot = 2 * blockIdx.x + (s.first ? 0 : 1);
          const int rr = s.m * kRows + r, node = rr / p.ratio;
          // where this thread's row goes: an output row, or dims 0 .. 3 of a partial one, whose blocks
          // of 4 dims are 128 rows apart, so that a warp's store is 512 bytes in a piece
          __nv_bfloat16* row_out = p.out + static_cast<int64_t>(s.q0 + node) * p.out_stride_tok +
                                   static_cast<int64_t>(s.h * p.ratio + rr - node * p.ratio) * p.out_stride_head;
          float* row_part = p.o_part + (static_cast<int64_t>(slot) * (kHeadDim / 4) * kRows + r) * 4;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            const int d0 = 128 * half + 32 * c;
            uint32_t o[32];
            tmem_ld32(lane_addr + kOCol + d0, o);
            tmem_ld_wait(o);
#pragma unroll
            for (int i = 0; i < 32; ++i)             // a factor of 0 (no key seen, or a bad page) gives
              o[i] = sc == 0.f ? 0u : __float_as_uint(__uint_as_float(o[i]) * sc);   // zeros in any case
            if (valid) {
              if (whole) {
#pragma unroll
                for (int i = 0; i < 32; i += 8) {
                  uint32_t w[4];
#pragma unroll
                  for (int k = 0; k < 4; ++k) {
                    const __nv_bfloat162 x = __floats2bfloat162_rn(__uint_as_float(o[i + 2 * k]), __uint_as_float(o[i + 2 * k + 1]));
                    w[k] = *reinterpret_cast<const uint32_t*>(&x);
                  }
                  *reinterpret_cast<uint4*>(row_out + d0 + i) = make_uint4(w[0], w[1], w[2], w[3]);
                }
              } else {
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                  *reinterpret_cast<uint4*>(row_part + (d0 + i) * kRows) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
              }
            }
          }
          if (nan_v && !bad && valid) {
            // NaN values of the nodes that this row sees
#pragma unroll 1
            for (uint64_t w = word; w; w &= w - 1) {
              const int key = s.L - s.n + __ffsll(static_cast<long long>(w)) - 1;
              if (key < s.t0 * kKeys || key >= s.t1 * kKeys) continue;
              const int page = p.block_tables[static_cast<int64_t>(s.b) * p.max_pages + key / kPage];
              const uint8_t* src = p.v_cache + ((static_cast<int64_t>(page) * kPage + key % kPage) * p.hkv + s.h) * kHeadDim;
#pragma unroll 1
              for (int d = 128 * half; d < 128 * half + 128; ++d)
                if ((src[d] & 0x7f) == 0x7f) {
                  if (whole) row_out[d] = __float2bfloat16(__int_as_float(0x7fc00000));
                  else row_part[(d / 4) * 4 * kRows + d % 4] = __int_as_float(0x7fc00000);
                }
            }
          }
          if (!whole && valid && half == 0)
            p.lse_part[slot * kRows + r] = bad ? __uint_as_float(kBadLse)
                                               : (l != 0.f ? m + log2f(l) - kShift : -INFINITY);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&bars.o_free));
          mbar_arrive(smem_u32(&bars.seg_free[(e - 1) % kSegRing]));
        }
      }
      if (end) break;
      const int rr = y.m * kRows + r;
      valid = rr < y.n * p.ratio;
      active = __any_sync(0xffffffffu, valid);
      word = valid ? p.mask[y.q0 + rr / p.ratio] : 0ull;
      if (y.n < 64) word &= (1ull << y.n) - 1ull;
      const int tree0 = y.L - y.n;                  // first key of the tree
      const int t0 = y.t0, t1 = y.t1;
      nan_row = sl2_next != sl2_next;
      const float sl2 = nan_row ? 1.f : sl2_next;
      m = -INFINITY;
      l = 0.f;
#pragma unroll 1
      for (int t = t0; t < t1; ++t, ++u) {
        const uint32_t sb = u & 1;
        if (!__all_sync(0xffffffffu, wait_for(smem_u32(&bars.s_full[sb]), (u >> 1) & 1, abort_flag))) {
          alive = false;
          break;
        }
        tc_fence_after();
        // Every phase of pv_done is waited for in its turn, as parities demand; this one is long
        // complete, its products having been issued before the QK that s_full stands for.
        if (t > t0 + 1 &&
            !__all_sync(0xffffffffu, wait_for(smem_u32(&bars.pv_done[u & 1]), ((u - 2) >> 1) & 1, abort_flag))) {
          alive = false;
          break;
        }
        if (active) {
          const uint32_t s_addr = lane_addr + sb * kSCols;
          float x[64];
          {
            uint32_t v0[32], v1[32];
            tmem_ld32(s_addr + 64 * half, v0);
            tmem_ld32(s_addr + 64 * half + 32, v1);
            tmem_ld_wait(v0);
            tmem_ld_wait(v1);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              x[e] = __uint_as_float(v0[e]);
              x[32 + e] = __uint_as_float(v1[e]);
            }
          }
          // the keys of this half tile that the row sees, 32 a word
          const int off = t * kKeys + 64 * half - tree0;
          const bool masked = off + 64 > 0;
          auto seen = [&](int c) -> uint32_t {
            const int st = off + 32 * c;
            if (st <= -32) return 0xffffffffu;
            if (st < 0) return (static_cast<uint32_t>(word) << -st) | ((1u << -st) - 1u);
            return st < 64 ? static_cast<uint32_t>(word >> st) : 0u;
          };
          if (masked) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const uint32_t bits = seen(c);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((bits >> e) & 1u)) x[32 * c + e] = -INFINITY;
            }
          }
          float a = fmaxf(x[0], x[1]), b = fmaxf(x[2], x[3]);
#pragma unroll
          for (int e = 4; e < 64; e += 4) {
            a = max3(a, x[e], x[e + 1]);
            b = max3(b, x[e + 2], x[e + 3]);
          }
          float top = fmaxf(a, b) * sl2;
          if (top != top) top = -INFINITY;           // all NaN
          // the row's maximum over both halves; behind it both warps have read their logits, so
          // P may be written over them
          float* both = xch + (meets & 1) * 2 * kRows;
          both[half * kRows + r] = top;
          if (!meet()) {
            alive = false;
            break;
          }
          top = fmaxf(top, both[(half ^ 1) * kRows + r]);
          float alpha = 1.f;
          bool rescale = false;
          if (top != -INFINITY && (m == -INFINITY || top > m + kTau)) {
            if (m != -INFINITY) {
              alpha = exp2_hw(m - top);
              rescale = true;
            }
            m = top;
          }
          if (t > t0 && __any_sync(0xffffffffu, rescale)) {
            // O may be touched once the previous tile's products are in it
            if (!__all_sync(0xffffffffu, wait_for(smem_u32(&bars.pv_done[(u - 1) & 1]), ((u - 1) >> 1) & 1, abort_flag))) {
              alive = false;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < kHeadDim / 32; ++c) {  // 16 columns at a time: the logits are live
              const uint32_t o_addr = lane_addr + kOCol + 128 * half + 16 * c;
              uint32_t o[16];
              asm volatile(
                  "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
                  "%14,%15}, [%16];\n tcgen05.wait::ld.sync.aligned;\n"
                  : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]), "=r"(o[4]), "=r"(o[5]), "=r"(o[6]),
                    "=r"(o[7]), "=r"(o[8]), "=r"(o[9]), "=r"(o[10]), "=r"(o[11]), "=r"(o[12]), "=r"(o[13]),
                    "=r"(o[14]), "=r"(o[15])
                  : "r"(o_addr)
                  : "memory");
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st16(o_addr, o);
            }
          }
          const float moff = m == -INFINITY ? 0.f : kShift - m;
          float l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int e = 32 * c; e < 32 * c + 32; e += 2) fma_pair(x[e], x[e + 1], sl2, moff);
            uint32_t pw[16];
#pragma unroll
            for (int e = 32 * c; e < 32 * c + 32; e += 4) {
              x[e] = exp2_hw(x[e]);
              x[e + 1] = exp2_hw(x[e + 1]);
              x[e + 2] = exp2_hw(x[e + 2]);
              x[e + 3] = exp2_hw(x[e + 3]);
              add_pair(l0, l1, x[e], x[e + 1]);
              add_pair(l2, l3, x[e + 2], x[e + 3]);
              pw[(e - 32 * c) / 2] = half2_of(x[e], x[e + 1]);
              pw[(e - 32 * c) / 2 + 1] = half2_of(x[e + 2], x[e + 3]);
            }
            tmem_st16(s_addr + 32 * half + 16 * c, pw);
          }
          l = l * alpha + ((l0 + l2) + (l1 + l3));
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars.p_full[sb]));
      }
    }
  }

  // ---- teardown ------------------------------------------------------------------------------
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (*abort_flag && tid == 0) set_status(p.status, MTPATTN_ERR_TIMEOUT);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// The join: out = sum_j w_j o_j / sum_j w_j over a unit's pieces, w_j = 2^(lse_j - max lse).
//
// A CTA takes 32 rows (lane = row) and kDims dims of a unit.  Its warps first share out the pieces
// and leave their weights in shared memory, while the first partials are already on their way;
// then a warp adds kVec blocks of 4 dims of every kGroups-th piece, kAhead pieces in flight.
// Rows leave through shared memory, 2 kDims bytes each side by side: written from the registers,
// 8 bytes a row, the stores were most of the time.  The kernel reads what the main kernel has
// just written, out of L2.
constexpr int kReduceThreads = 256, kReduceWarps = kReduceThreads / 32;
constexpr int kMaxPieces = 160;                      // of a unit: no more than there are CTAs
template <int kDims, int kVec>
constexpr int reduce_groups() {
  return kReduceWarps / (kDims / 4 / kVec);
}
constexpr float kNoKey = -1.f;                       // in a weight's place: the row sees no key of the piece
__device__ __forceinline__ float nan_of(float x) { return x != x ? x : 0.f; }
constexpr int reduce_ctas(int dims) { return (kRows / 32) * (kHeadDim / dims); }   // a unit

template <int kDims, int kVec, int kAhead>
__global__ void __launch_bounds__(kReduceThreads)
tree_reduce_kernel(const __grid_constant__ TreeAttnParams p) {
  constexpr int kDimWarps = kDims / 4 / kVec, kGroups = reduce_groups<kDims, kVec>();
  static_assert(kDimWarps * kGroups == kReduceWarps);
  constexpr int kPitch = 2 * kDims + 16;             // bytes a row in shared memory
  __shared__ float s_w[kMaxPieces][32];
  __shared__ float s_top[kReduceWarps][32], s_sum[kReduceWarps][32];
  __shared__ float4 s_acc[kGroups > 1 ? kGroups - 1 : 1][kGroups > 1 ? kDimWarps * kVec : 1][32];
  __shared__ alignas(16) unsigned char s_out[32 * kPitch];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int dw = warp % kDimWarps, g = warp / kDimWarps;
  const int quad = blockIdx.y / (kHeadDim / kDims), d0 = kDims * (blockIdx.y % (kHeadDim / kDims));
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  asm volatile("griddepcontrol.wait;\n" ::: "memory");   // every partial is written and visible
  const int units = __ldcg(p.units);
  const int4 n0 = __ldcg(reinterpret_cast<const int4*>(p.notes + blockIdx.x));
  const int4 n1 = __ldcg(reinterpret_cast<const int4*>(p.notes + blockIdx.x) + 1);
  if (static_cast<int>(blockIdx.x) >= units || n0.x <= 1) return;
  const int n = n0.x, q0 = n0.w, h = n1.x, m = n1.y;
  // A CTA whose wait ran out may have left no note: what stands there then is not followed.
  if (n > p.ctas || n0.y < 0 || n0.y > p.ctas - n || (n0.z & ~1) || q0 < 0 || h < 0 || h >= p.hkv || m < 0 ||
      m >= MTP_TREE_MAX_NODES * MTP_TREE_MAX_RATIO / kRows || n1.z <= 0 || n1.z > kRows ||
      q0 > p.total_q - 1 - (m * kRows + n1.z - 1) / p.ratio)
    return;
  const int r0 = 32 * quad, rows = min(32, n1.z - r0);   // rows of the unit's, of this quarter
  if (rows <= 0) return;
  const bool mine = lane < rows;
  auto slot_of = [&](int i) -> int64_t { return 2 * (n0.y + i) + (i == 0 ? n0.z : 0); };
  const float* src = p.o_part + (static_cast<int64_t>(d0 / 4 + dw * kVec) * kRows + r0 + lane) * 4;
  constexpr int64_t kSlot = static_cast<int64_t>(kHeadDim) * kRows;
  float4 a[kAhead][kVec];
  auto load = [&](int i0) {                          // pieces i0, i0 + kGroups, ...
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (mine && i0 + j * kGroups < n)
#pragma unroll
        for (int k = 0; k < kVec; ++k)
          a[j][k] = __ldcg(reinterpret_cast<const float4*>(src + slot_of(i0 + j * kGroups) * kSlot + k * 4 * kRows));
  };
  load(g);
  float top = -INFINITY;
  bool bad = false;
  constexpr int kLse = 8;                            // a warp's in flight
#pragma unroll 1
  for (int i0 = warp; i0 < n; i0 += kLse * kReduceWarps) {
    float l[kLse];
#pragma unroll
    for (int j = 0; j < kLse; ++j) {
      const int i = i0 + j * kReduceWarps;
      l[j] = mine && i < n ? __ldcg(p.lse_part + slot_of(i) * kRows + r0 + lane) : -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < kLse; ++j) {
      const int i = i0 + j * kReduceWarps;
      bad |= __float_as_uint(l[j]) == kBadLse;
      if (i < n) s_w[i][lane] = l[j];
      top = fmaxf(top, l[j]);                        // (NaN is passed over)
    }
  }
  s_top[warp][lane] = top;
  bad = __syncthreads_or(bad);                       // (all rows of a sequence with a bad page are)
#pragma unroll
  for (int i = 0; i < kReduceWarps; ++i) top = fmaxf(top, s_top[i][lane]);
  float sum = 0.f;
#pragma unroll 1
  for (int i = warp; i < n; i += kReduceWarps) {
    const float l = s_w[i][lane];
    const float w = l == -INFINITY ? 0.f : exp2_hw(l - top);         // NaN makes the row NaN
    s_w[i][lane] = l == -INFINITY ? kNoKey : w;
    sum += w;
  }
  s_sum[warp][lane] = sum;
  __syncthreads();
  float4 acc[kVec];
#pragma unroll
  for (int k = 0; k < kVec; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int i0 = g; i0 < n; i0 += kAhead * kGroups) {
    if (i0 > g) load(i0);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const float w = i0 + j * kGroups < n ? s_w[i0 + j * kGroups][lane] : kNoKey;
      if (w == kNoKey) continue;                     // (a piece without keys for the row holds anything)
      if (w == 0.f) {                                // far below the others: what is NaN there stays NaN
#pragma unroll
        for (int k = 0; k < kVec; ++k) {
          acc[k].x += nan_of(a[j][k].x);
          acc[k].y += nan_of(a[j][k].y);
          acc[k].z += nan_of(a[j][k].z);
          acc[k].w += nan_of(a[j][k].w);
        }
        continue;
      }
#pragma unroll
      for (int k = 0; k < kVec; ++k) {
        acc[k].x = fmaf(w, a[j][k].x, acc[k].x);
        acc[k].y = fmaf(w, a[j][k].y, acc[k].y);
        acc[k].z = fmaf(w, a[j][k].z, acc[k].z);
        acc[k].w = fmaf(w, a[j][k].w, acc[k].w);
      }
    }
  }
  if (kGroups > 1) {
    if (g > 0)
#pragma unroll
      for (int k = 0; k < kVec; ++k) s_acc[g - 1][dw * kVec + k][lane] = acc[k];
    __syncthreads();
    if (g == 0)
#pragma unroll 1
      for (int o = 0; o < kGroups - 1; ++o)
#pragma unroll
        for (int k = 0; k < kVec; ++k) {
          const float4 x = s_acc[o][dw * kVec + k][lane];
          acc[k].x += x.x;
          acc[k].y += x.y;
          acc[k].z += x.z;
          acc[k].w += x.w;
        }
  }
  if (g == 0) {
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < kReduceWarps; ++i) sum += s_sum[i][lane];
    const float inv = sum == 0.f || bad ? 0.f : 1.f / sum;   // no key, or a bad page: zeros
#pragma unroll
    for (int k = 0; k < kVec; ++k) {
      if (inv == 0.f) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      const __nv_bfloat162 x = __floats2bfloat162_rn(acc[k].x * inv, acc[k].y * inv);
      const __nv_bfloat162 y = __floats2bfloat162_rn(acc[k].z * inv, acc[k].w * inv);
      *reinterpret_cast<uint2*>(s_out + lane * kPitch + (dw * kVec + k) * 8) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
    }
  }
  __syncthreads();
  constexpr int kBlocks = kDims / 8;                 // of 16 bytes a row
  for (int i = t; i < rows * kBlocks; i += kReduceThreads) {
    const int row = i / kBlocks, b = i % kBlocks, rr = m * kRows + r0 + row, node = rr / p.ratio;
    __nv_bfloat16* out = p.out + static_cast<int64_t>(q0 + node) * p.out_stride_tok +
                         static_cast<int64_t>(h * p.ratio + rr - node * p.ratio) * p.out_stride_head + d0 + 8 * b;
    *reinterpret_cast<uint4*>(out) = *reinterpret_cast<const uint4*>(s_out + row * kPitch + 16 * b);
  }
}

__global__ void __launch_bounds__(MTP_TREE_MAX_NODES)
tree_mask_kernel(const int32_t* parents, const int32_t* cu_q, int32_t total_q, uint64_t* mask,
                 int32_t* status) {
  __shared__ int32_t par[MTP_TREE_MAX_NODES];
  const int b = blockIdx.x, i = threadIdx.x;
  const int q0 = cu_q[b], q1 = cu_q[b + 1], n = q1 - q0;
  if (q0 < 0 || q1 <= q0 || q1 > total_q || n > MTP_TREE_MAX_NODES) {
    if (i == 0) set_status(status, MTPATTN_ERR_QLEN);
    return;
  }
  if (i < n) par[i] = i == 0 ? -1 : parents[q0 + i];
  __syncthreads();
  if (i >= n) return;
  // up the path; a node's parent has a smaller number, so at most n steps
  uint64_t word = 0;
  int at = i;
  while (true) {
    word |= 1ull << at;
    if (at == 0) break;
    const int up = par[at];
    if (up < 0 || up >= at) {
      set_status(status, MTP_TREE_ERR_PARENT);
      break;
    }
    at = up;
  }
  mask[q0 + i] = word;
}

// ---- host side -----------------------------------------------------------------------------------

// CTAs of a call: one per SM, but no more than the line can have key tiles.
int64_t units_bound(int32_t num_seqs, int32_t total_q, int32_t hkv, int32_t ratio) {
  return (static_cast<int64_t>(total_q) * ratio / kRows + num_seqs) * hkv;
}
int64_t line_bound(int32_t num_seqs, int32_t total_q, int32_t hkv, int32_t ratio, int32_t max_pages) {
  return units_bound(num_seqs, total_q, hkv, ratio) * ((max_pages + kTilePages - 1) / kTilePages + kUnitTiles);
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

cudaError_t launch_pdl(const void* kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream,
                       TreeAttnParams& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[] = {&p};
  cudaError_t e = cudaLaunchKernelExC(&cfg, kernel, args);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return e;
  }
  return cudaGetLastError();
}

}  // namespace
}  // namespace mtpattn

using namespace mtpattn;

extern "C" int mtp_tree_mask(const int32_t* parents, const int32_t* cu_seqlens_q, int32_t num_seqs,
                             int32_t total_q, uint64_t* mask, int32_t* status, void* stream) {
  if (num_seqs < 0 || total_q < 0) return MTPATTN_E_ARG;
  if (num_seqs == 0) return total_q == 0 ? MTPATTN_OK : MTPATTN_E_ARG;
  if (total_q < num_seqs || !parents || !cu_seqlens_q || !mask) return MTPATTN_E_ARG;
  if (!ptr_aligned(parents, 4) || !ptr_aligned(cu_seqlens_q, 4) || !ptr_aligned(mask, 8) ||
      !ptr_aligned(status, 4))
    return MTPATTN_E_ARG;
  if (total_q > static_cast<int64_t>(num_seqs) * MTP_TREE_MAX_NODES) return MTPATTN_E_UNSUPPORTED;
  const int device = current_device();
  if (device < 0) return MTPATTN_E_DEVICE;
  const void* const ptrs[] = {parents, cu_seqlens_q, mask};
  if (!all_on_device(ptrs, device) || (status && !ptr_on_device(status, device)))
    return MTPATTN_E_DEVICE;
  tree_mask_kernel<<<num_seqs, MTP_TREE_MAX_NODES, 0, static_cast<cudaStream_t>(stream)>>>(
      parents, cu_seqlens_q, total_q, mask, status);
  return cudaGetLastError() == cudaSuccess ? MTPATTN_OK : MTPATTN_E_LAUNCH;
}

extern "C" size_t mtp_tree_attn_workspace_size(int32_t num_seqs, int32_t total_q,
                                               int32_t num_q_heads, int32_t num_kv_heads,
                                               int32_t max_pages_per_seq) {
  if (num_seqs < 0 || total_q < 0 || num_q_heads <= 0 || num_kv_heads <= 0 ||
      max_pages_per_seq < 0 || num_q_heads % num_kv_heads)
    return 0;
  const int sms = std::min(device_sm_count(-1), kMaxPieces);
  if (sms <= 0) return 0;
  const int64_t ctas = std::min<int64_t>(
      sms, line_bound(num_seqs, total_q, num_kv_heads, num_q_heads / num_kv_heads, max_pages_per_seq));
  // partial outputs, then their log-sum-exps, two slots of 128 rows a CTA; the units' notes; their
  // number
  const int64_t units = units_bound(num_seqs, total_q, num_kv_heads, num_q_heads / num_kv_heads);
  return align256(static_cast<size_t>(ctas) * 2 * kRows * (kHeadDim + 1) * sizeof(float)) +
         align256(static_cast<size_t>(units) * sizeof(JoinNote)) + 256;
}

extern "C" int mtp_tree_attn_fwd(const void* q, int64_t q_stride_tok, int64_t q_stride_head,
                                 const void* k_cache, const void* v_cache, int64_t num_pages,
                                 const int32_t* block_tables, int32_t max_pages_per_seq,
                                 const int32_t* seq_lens, const int32_t* cu_seqlens_q,
                                 const uint64_t* tree_mask, int32_t num_seqs, int32_t total_q,
                                 int32_t num_q_heads, int32_t num_kv_heads,
                                 const float* k_descale, const float* v_descale,
                                 float softmax_scale, void* workspace, size_t workspace_bytes,
                                 void* out, int64_t out_stride_tok, int64_t out_stride_head,
                                 int32_t* status, void* stream) {
  // 1. plain argument checks
  if (num_seqs < 0 || total_q < 0 || num_pages < 0 || max_pages_per_seq < 0 || num_q_heads <= 0 ||
      num_kv_heads <= 0)
    return MTPATTN_E_ARG;
  if (num_seqs == 0) return total_q == 0 ? MTPATTN_OK : MTPATTN_E_ARG;
  if (total_q < num_seqs) return MTPATTN_E_ARG;          // every sequence has its root
  if (!q || !k_cache || !v_cache || !block_tables || !seq_lens || !cu_seqlens_q || !tree_mask ||
      !k_descale || !v_descale || !out || num_pages == 0 || max_pages_per_seq == 0)
    return MTPATTN_E_ARG;
  if (!isfinite(softmax_scale)) return MTPATTN_E_ARG;
  if (q_stride_tok <= 0 || q_stride_head <= 0 || out_stride_tok <= 0 || out_stride_head <= 0 ||
      (q_stride_tok | q_stride_head | out_stride_tok | out_stride_head) % 8 != 0)
    return MTPATTN_E_ARG;
  if (!ptr_aligned(q, 16) || !ptr_aligned(out, 16) || !ptr_aligned(k_cache, 16) ||
      !ptr_aligned(v_cache, 16) || !ptr_aligned(block_tables, 4) || !ptr_aligned(seq_lens, 4) ||
      !ptr_aligned(cu_seqlens_q, 4) || !ptr_aligned(tree_mask, 8) || !ptr_aligned(k_descale, 4) ||
      !ptr_aligned(v_descale, 4) || !ptr_aligned(status, 4))
    return MTPATTN_E_ARG;
  // 2. the supported envelope
  if (num_q_heads % num_kv_heads) return MTPATTN_E_UNSUPPORTED;
  const int ratio = num_q_heads / num_kv_heads;
  if (ratio > MTP_TREE_MAX_RATIO) return MTPATTN_E_UNSUPPORTED;
  if (total_q > static_cast<int64_t>(num_seqs) * MTP_TREE_MAX_NODES) return MTPATTN_E_UNSUPPORTED;
  if (num_pages > INT32_MAX || max_pages_per_seq > INT32_MAX / kPage - kTilePages ||
      line_bound(num_seqs, total_q, num_kv_heads, ratio, max_pages_per_seq) > INT32_MAX)
    return MTPATTN_E_UNSUPPORTED;
  // 3. the workspace
  const int device = current_device();
  if (device < 0) return MTPATTN_E_DEVICE;
  const size_t need = mtp_tree_attn_workspace_size(num_seqs, total_q, num_q_heads, num_kv_heads,
                                                   max_pages_per_seq);
  if (!workspace || !ptr_aligned(workspace, 256) || workspace_bytes < need)
    return MTPATTN_E_WORKSPACE;
  // 4. every pointer must be memory the kernels can read on the current device
  const void* const ptrs[] = {q, k_cache, v_cache, block_tables, seq_lens, cu_seqlens_q, tree_mask,
                              k_descale, v_descale, workspace, out};
  if (!all_on_device(ptrs, device) || (status && !ptr_on_device(status, device)))
    return MTPATTN_E_DEVICE;

  TreeAttnParams p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_stride_tok = q_stride_tok;
  p.q_stride_head = q_stride_head;
  p.v_cache = static_cast<const uint8_t*>(v_cache);
  p.num_pages = num_pages;
  p.block_tables = block_tables;
  p.max_pages = max_pages_per_seq;
  p.seq_lens = seq_lens;
  p.cu_q = cu_seqlens_q;
  p.mask = tree_mask;
  p.num_seqs = num_seqs;
  p.total_q = total_q;
  p.hq = num_q_heads;
  p.hkv = num_kv_heads;
  p.ratio = ratio;
  p.k_descale = k_descale;
  p.v_descale = v_descale;
  p.scale_log2 = softmax_scale * kLog2e;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.out_stride_tok = out_stride_tok;
  p.out_stride_head = out_stride_head;
  p.status = status;
  p.ctas = static_cast<int32_t>(std::min<int64_t>(
      std::min(device_sm_count(device), kMaxPieces), line_bound(num_seqs, total_q, num_kv_heads, ratio, max_pages_per_seq)));
  p.o_part = static_cast<float*>(workspace);
  p.lse_part = p.o_part + static_cast<int64_t>(p.ctas) * 2 * kRows * kHeadDim;
  p.unit_bound = static_cast<int32_t>(units_bound(num_seqs, total_q, num_kv_heads, ratio));
  p.units = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + need - 256);
  p.notes = reinterpret_cast<JoinNote*>(static_cast<char*>(workspace) + need - 256 -
                                        align256(static_cast<size_t>(p.unit_bound) * sizeof(JoinNote)));
  AttnParams cache{};                                // what the tensor map goes by
  cache.k_cache = static_cast<const uint8_t*>(k_cache);
  cache.v_cache = p.v_cache;
  cache.num_pages = num_pages;
  cache.num_kv_heads = num_kv_heads;
  if (!kv_tensor_maps(cache, device, &p.tmap_k, &p.tmap_v)) return MTPATTN_E_LAUNCH;
  static std::atomic<bool> attr_set[64];             // per device; setting it twice is harmless
  if (device >= 64) return MTPATTN_E_DEVICE;
  if (!attr_set[device].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(tree_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemTree) !=
        cudaSuccess) {
      cudaGetLastError();
      return MTPATTN_E_LAUNCH;
    }
    attr_set[device].store(true, std::memory_order_release);
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (launch_pdl(reinterpret_cast<const void*>(tree_attn_kernel), dim3(p.ctas), kTreeThreads, kSmemTree,
                 st, p) != cudaSuccess)
    return MTPATTN_E_LAUNCH;
  // units of one key tile are never cut
  if (max_pages_per_seq <= kTilePages) return MTPATTN_OK;
  // Few units are cut into many pieces each: many CTAs of few dims, with four groups of pieces, then;
  // many units into few pieces: few CTAs, whose grid costs less where it has nothing to do.  A whole
  // call, the one and the other: unit_bound 8, 37000 tokens 22.6 and 37.1 us; 32, 16 x 35000 65.5 and
  // 70.8; 60, 30 x 9000 41.3 and 42.4; 100, 50 x 9000 58.7 and 56.1; 128, 32 x 5000 51.1 and 46.2.
  const bool few = p.unit_bound <= 64;
  const void* kernel = few ? reinterpret_cast<const void*>(tree_reduce_kernel<32, 4, 2>)
                           : reinterpret_cast<const void*>(tree_reduce_kernel<128, 4, 1>);
  return launch_pdl(kernel, dim3(p.unit_bound, reduce_ctas(few ? 32 : 128)), kReduceThreads, 0, st, p) == cudaSuccess
             ? MTPATTN_OK : MTPATTN_E_LAUNCH;
}
