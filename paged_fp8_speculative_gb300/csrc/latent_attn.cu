// Latent attention over the paged cache (mtp_latent.h) on the sm_100-family tensor cores (tcgen05, TMA,
// TMEM).
//
// The products are the other way round than usual: keys (and the values' dims) are the rows M = 128 of
// a tcgen05.mma and the queries its columns,
//   S^T [128 keys x rows] = C [128 x 576] Q^T,      O^T [512 dims x rows] = C[:, :512]^T P^T,
// so that few query rows cost few columns, and all 512 dims of the output of up to 64 rows fit into half of
// TMEM (the usual way 128 rows would take all of it, and P none).  A tile of 128 keys is read once, into
// shared memory as TMA puts it, and is an operand of both products as it lies there: K-major for the first,
// M-major (transposed) for the second.  Nothing is widened or copied.
//
// Work.  A sequence's query rows are its new tokens times the heads, row r being token r / heads, head
// r % heads; a unit is up to N of them (16, 32 or 64) over all of the sequence's keys.  All units stand in a
// line, a place for each tile of 128 keys and kUnitTiles ahead of them for the unit's Q and output; the line
// is cut into equal pieces, one per CTA (worked out from seq_lens and cu_seqlens_q on the device, so a
// captured call follows its buffers).  A unit that lies in one piece is written out at once; one that is cut
// leaves its sums, references and outputs in the workspace (two slots a CTA: its first and its last unit),
// and latent_join_kernel joins them, going by the notes that the CTAs with first tiles leave.  Units stay whole
// where cutting them would cost more, and CTAs go over a sequence's keys together where they have its row tiles
// (Walker::start).
//
// Roles (384 threads, one CTA an SM): warp 0 walks over the CTA's piece and issues S's products, warp 1 O's;
// warps 2 and 3 fetch tiles, each two blocks of 32 keys, by TMA: half a page a lane, a box of 9 slices of 64
// bytes of 8 keys, so that one instruction brings 4608 bytes.  Warps 4-11 do the softmax: a warp has 32 keys
// (TMEM lanes) of half of the rows, makes Q's operand, and writes the output.  They get 200 registers a thread,
// the others 104.
//
// Precision.  Codes enter as they are, Q as two e4m3 terms of x = q 2^a (a per row, max |x| in [128,
// 256)): hi = e4m3(x), lo = e4m3(x - hi), as 2 N columns of one product, added in float32.  A bf16 value
// has 8 significant bits and the terms keep 4 each, so x = hi + lo, but for what is below lo's smallest step: at most
// 2^-10, 2^-17 of the row's largest.
// The weights p = 2^(s - ref), at most 2^8.75, are an e4m3 term and an e5m2 one of what it leaves, of 4 and 3
// significant bits: within 2^-8 of p, as a bf16 weight is.  e4m3's smallest step is 2^-9, e5m2's 2^-16: of a weight
// below 2^-6 the second term is what counts, and of one below 2^-10 it is all.  There rounding to nearest would
// bend the sum of many equal weights behind a large one (30000 at 2^-19 are 5% of all).  So a second term below 2^-10
// is rounded up or down in the proportion of the bits that go, by a number of the key's own (its dither): it is off by
// less than 2^-13, and sums are not.  The numbers of a tile's keys are 128 evenly spread ones, the place's bits
// reversed, and each tile has them in another order, so that keys whose values repeat with any period have evenly spread
// ones too; the same bits come every time.  (Two e4m3 terms with one order for all tiles lost the weights below 2^-9
// of whole classes of keys: with a first key 9.5 nats above 8190 others and values of period 2 the output was 0.4 off, in
// 2-norm, where it is now 0.0017.)  The sums of weights, in float32, are of what the terms stand for: a weight that is
// nearly all of its row's comes out whole, where its rounding of up to 2^-8 would be the output's.
//
// Online softmax in the log2 domain with a lazy reference: raised, and O rescaled in TMEM, only when a logit
// exceeds it by more than kTau.  So a tile's maxima over keys (across lanes and warps, which this orientation
// makes dear) are only needed where that happens.  A reference that is raised with tiles to come goes kRoom
// above what it has to, so that it is raised less often; the largest weight is then 2^3 or more instead of
// 2^7, and what the dither leaves below 2^-16 of it.  kRoom's sides, measured (error of the output against 64 bits, of
// which its rounding is 0.00166, over 8191 keys of 64-node trees; time of those trees, and of 16 x 35000 keys with
// 128 heads): 0: 0.00178, 158 and 159 us; 2.5: 0.00181, 147 and 147; 4: 0.00185, 137 and 138; 5: 0.00187, 135 and
// 135, but 0.0030 instead of 0.0018 where 30000 keys of unlike values are 8.5 nats below one.
//
// Masks.  A tile that reaches into the new tokens takes each row's word.  Places that no row sees in full
// are kept out of the second product by value too, since 0 * NaN is NaN: rows behind the sequence are
// stored as zeros, NaN codes of new tokens too (a row that sees one has a NaN logit, and its sum tells).  A
// key's logit is NaN, whatever the row, exactly where a code of it is: so only such keys are gone over.
//
// Shared memory (N = 64): two stages of a tile (147456), Q's terms (73728), the second terms of P (8192;
// the first ones take the place of the tile's 64-byte slice of rotated dims, which only the first product reads).
// TMEM: S double buffer at columns 0 and 128, O at 256, N columns for each 128 dims.
//
// What bounds it.  Shared memory's 128 bytes a clock: for 64 rows a tile's S reads the codes and Q (147 KB; 18
// instructions of 64 clocks, measured alone), O the codes for each of P's two terms and those for each 128 dims
// (192 KB; 16 pairs of 96 clocks), the tile itself is written (74 KB), and P (16 KB): about 3350 clocks.  A
// tile takes 3830 where the cache is in L2 and 4570 where all CTAs have their own from memory (5.1 TB/s; sequences of 4096
// and 12288 tokens, 64 rows each, compared); what is lost is the chain S, softmax, P, O, of which two tiles, all that
// fits, overlap.  Measured, in graphs: 16 x 35000 keys with 4 tokens of 16 heads 84 us (memory's floor 48.8,
// the products' 41.4 at the bf16 rate), with one token 63; 128 heads 138 (82.8 at the bf16 rate); 64-node trees
// over 8191 keys 137 (77.0); 300 keys 10.2.  A call begins with 7 to 9 us (launch, lengths, Q's terms, first
// tiles of all CTAs at once) and ends with 2.5 of output and 4 to 7 of the join; a unit costs 6 to 10 more
// (sums, Q, output), which short sequences pay one by one.
#include "common.cuh"
#include "host_checks.cuh"
#include "sm100.cuh"

#include "../../include/mtp_latent.h"

#include <cuda_fp16.h>
#include <math.h>

#include <algorithm>
#include <atomic>

namespace mtpattn {
namespace {

using namespace sm100;

constexpr int kRow = MTP_LATENT_ROW, kDim = MTP_LATENT_DIM;
constexpr int kLatentThreads = 384;
constexpr int kKeys = 128, kTilePages = kKeys / kPage;
constexpr int kColumns = 4;                          // of 128 dims of the output
constexpr int kSlices = kRow / 64;                   // of 64 dims of a key, the last the rotated ones
constexpr int kAtom = 8 * 64;                        // 8 keys of a slice, 64-byte swizzled
constexpr int kGroup = kSlices * kAtom;              // 8 keys
constexpr int kBlocks = 4, kBlockKeys = kKeys / kBlocks;   // what is fetched and given back at a time
constexpr int kRopeAt = (kSlices - 1) * kAtom;       // in a group
constexpr int kPLow = kKeys * 64;                    // P's second terms
constexpr int kStage = kKeys / 8 * kGroup;
static_assert(kStage % 1024 == 0, "Q's operand behind the stages");
constexpr int kBlockPages = kBlockKeys / kPage;
constexpr int kWarpBlocks = kBlocks / 2, kWarpPages = kWarpBlocks * kBlockPages;   // of a tile, a fetching warp's
constexpr int kStages = 2;
constexpr int kWarpSoft = 4, kSoftWarps = 8;
constexpr int kLaunchRegisters = 168;                // a thread, as the block is launched (checked by the host)
constexpr int kFewRegisters = 104, kManyRegisters = 200;   // ... and as the roles share them out
constexpr int kSBuf = 128, kOCol = 256, kTmemCols = 512;
constexpr int kSegRing = 4;
constexpr int kPrefetch = 1;                         // tiles ahead, into L2
constexpr float kShift = 7.f, kTau = 1.75f;          // a weight is 2^kShift at the reference, and at most
                                                     // 2^(kShift + kTau) = 430 < 448
constexpr float kRoom = 4.f;                        // a raised reference is so far above the row's maximum
constexpr float kNoRef = -INFINITY;                  // no key seen yet (a reference is finite)
constexpr int kUnitTiles = 6, kCutTiles = 7, kCutPieces = 40;   // what a unit's ends, and cutting units, cost, in
                                                     // tiles (kUnitTiles 5, 6 and 7: 8 x 1000 keys, 4 tokens of 16
                                                     // heads, 16.1, 16.0 and 17.0 us; 20 x 2000, 1 token of 128, 29.7,
                                                     // 29.0 and 30.8; the others: Walker::start)
constexpr int kFewTiles = 8;
constexpr int kWholeTiles = 4;                       // tables no longer: units stay whole, and no join is launched
                                                     // (with cuts and without: 64 x 300 keys, 1 token of 128 heads,
                                                     // 22.7 and 19.3 us; 256 x 500 90.9 and 81.8; 16 x 500, 4 tokens of
                                                     // 16, 13.4 and 12.2; but one such 10.3 and 11.3, and 1 x 700 would
                                                     // take 10.4 and 13.8)
constexpr int kMaxCtas = 160;
constexpr uint32_t kBadSum = 0x7fd0bad1u;            // a sum of a sequence with a bad page (a NaN that no
                                                     // arithmetic makes)

template <int N>
constexpr int q_column() { return 2 * N * 128; }     // 128 elements of all rows' two terms
template <int N>
constexpr int off_q() { return kStages * kStage; }
template <int N>
constexpr int off_p() { return off_q<N>() + 2 * N * kRow; }
template <int N>
constexpr int off_bars() { return (off_p<N>() + kPLow + 15) / 16 * 16; }

// What the join goes by: a unit's note, written by the CTA that has its first tile.
struct JoinNote {
  int pieces;                // it lies in; 1: written out whole
  int first, first_slot;     // the first of them, and the unit's slot there (in the others, 0)
  int q0, m, rows;           // its sequence's first row of tokens, row tile, valid rows
  int stride;                // from a piece's CTA to the next one's
  int pad;
};

struct LatentParams {
  CUtensorMap tmap;
  const uint8_t* cache;
  const __nv_bfloat16* q;
  int64_t q_stride_tok, q_stride_head;
  int64_t num_pages;
  const int32_t* block_tables;
  int32_t max_pages;
  const int32_t* seq_lens;
  const int32_t* cu_q;
  const uint64_t* mask;
  int32_t num_seqs, total_q, heads;
  const float* descale;
  float scale_log2;
  __nv_bfloat16* out;
  int64_t out_stride_tok, out_stride_head;
  int32_t* status;
  int32_t ctas;
  float* o_part;             // [ctas][2][N][512]
  float2* sum_part;          // [ctas][2][N]: reference, sum
  int32_t* units;            // for the join: their number
  JoinNote* notes;
  int32_t unit_bound;
  int32_t whole;             // no unit is cut, nothing is joined: tables are that short
};

struct Segment {             // part of one unit: tiles t0 .. t1 - 1 of nt
  int q0, n, L, b;
  int m, t0, t1, nt;
  int slot;                  // 0: the first of the CTA's piece
  int end, bad;
};

struct Bars {
  uint64_t full[kStages][kBlocks], empty[kStages][kBlocks];
  uint64_t s_full[2], s_free[2];
  uint64_t p_full[kBlocks], pv_done, q_full, final_mma[2];
  uint64_t meet[3];          // the softmax warps of a row half, of both
  uint64_t seg_full[kSegRing], seg_free[kSegRing];
  Segment seg[kSegRing];
  uint32_t tmem_base;
  int32_t abort;
};
template <int N>
struct Shared {
  Bars bars;
  alignas(16) float factor[N];         // of the row's logits (log2 domain)
  alignas(16) float ref[N];            // reference - kShift
  alignas(16) float step[N];           // what it was raised by, negative
  alignas(16) float f[N];              // 2^step; the output's factor
  uint64_t word[N];                    // new tokens that the row sees
  alignas(16) float xch[2][4][N / 2];  // row half, key quarter
};
template <int N>
constexpr int smem_bytes() { return off_bars<N>() + static_cast<int>(sizeof(Shared<N>)); }
static_assert(kBlockKeys == 32, "a softmax warp's keys");
static_assert(smem_bytes<64>() <= 232448, "more than a block may have");

// ---- the line of tiles ---------------------------------------------------------------------------

// One sequence on the line: T units of nt tiles.  Rows whose place is not known (cu_seqlens_q out of order)
// take no part; other errors cost one tile a unit.
struct Seq {
  int q0, n, L, T, nt, w, err;
};
struct RawSeq {
  int q0, q1, L;
};
__device__ __forceinline__ RawSeq raw_at(const LatentParams& p, int b) {
  if (b >= p.num_seqs) return RawSeq{0, 0, 0};       // (no rows)
  return RawSeq{p.cu_q[b], p.cu_q[b + 1], p.seq_lens[b]};
}
template <int N>
__device__ __forceinline__ Seq seq_of(const LatentParams& p, const RawSeq& raw) {
  Seq s;
  s.n = s.T = s.nt = s.w = s.err = 0;
  const int q0 = s.q0 = raw.q0, q1 = raw.q1;
  s.L = raw.L;
  if (q0 < 0 || q1 <= q0 || q1 > p.total_q) {
    s.err = MTPATTN_ERR_QLEN;
    return s;
  }
  s.n = q1 - q0;
  if (s.n > MTP_LATENT_MAX_NODES) s.err = MTPATTN_ERR_QLEN;
  else if (s.n > s.L) s.err = MTPATTN_ERR_QLEN_GT_SEQ;
  else if (s.L > p.max_pages * kPage) s.err = MTPATTN_ERR_SEQ_TOO_LONG;
  s.T = static_cast<int>((static_cast<int64_t>(s.n) * p.heads + N - 1) / N);
  s.nt = s.err ? 1 : (s.L + kKeys - 1) / kKeys;
  s.w = s.T * (s.nt + kUnitTiles);
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
// Sum over the warp of numbers from 0 to 2^31 - 1.
__device__ __forceinline__ int64_t warp_total(int v) {
  return (static_cast<int64_t>(__reduce_add_sync(0xffffffffu, v >> 16)) << 16) + __reduce_add_sync(0xffffffffu, v & 0xffff);
}
__device__ __forceinline__ int add_up_to_max(int a, int b) {
  return static_cast<int>(min(static_cast<uint32_t>(a) + static_cast<uint32_t>(b), static_cast<uint32_t>(INT32_MAX)));
}

// A CTA's walk over the units of its piece, by one warp; 32 sequences are held, one a lane.
template <int N>
struct Walker {
  int pos, hi, lo, length, units;
  int C, V;                            // places of a piece; of a unit where none is cut (C is a multiple), else 0
  int G;                               // CTAs that take a piece together, a row tile each: 1, or all T of a sequence
  int b0, before, units_before;        // the held sequences; the line and the units before them
  Seq mine;
  int upto, units_upto;                // running sums of the held sequences' weights and units
  int unit, unit0, unit_places;        // the last segment's unit: its number, and place on the line

  __device__ __forceinline__ void start(const LatentParams& p, int lane) {
    b0 = before = units_before = unit = unit0 = unit_places = 0;
    mine = seq_of<N>(p, raw_at(p, lane));
    int w = mine.w, n = mine.n, T = mine.T, longest = mine.nt, tall = mine.T;
    int low = mine.T ? mine.T : INT32_MAX;           // the fewest row tiles of a sequence, and (tall) the most
    uint32_t group_w = 0, group_T = 0;               // of the 32 sequences from 32 * lane on
    if (p.num_seqs > 32) {
      group_w = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(w));   // (lane 0's)
      group_T = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(T));
      constexpr int kFlight = 4;                     // groups on their way at a time
#pragma unroll 1
      for (int b = 32; b < p.num_seqs; b += 32 * kFlight) {
        RawSeq raw[kFlight];
#pragma unroll
        for (int g = 0; g < kFlight; ++g) raw[g] = raw_at(p, b + 32 * g + lane);
#pragma unroll
        for (int g = 0; g < kFlight; ++g) {
          if (b + 32 * g >= p.num_seqs) break;
          const Seq x = seq_of<N>(p, raw[g]);
          w = add_up_to_max(w, x.w);
          n = add_up_to_max(n, x.n);
          T = add_up_to_max(T, x.T);
          longest = max(longest, x.nt);
          tall = max(tall, x.T);
          low = min(low, x.T ? x.T : INT32_MAX);
          const uint32_t all_w = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(x.w));
          const uint32_t all_T = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(x.T));
          if (lane == b / 32 + g) {
            group_w = all_w;
            group_T = all_T;
          }
        }
      }
    }
    int64_t W = warp_total(w), U = warp_total(T);
    const int64_t rows = warp_total(n);
    // Sequences that claim the same rows again and again (cu_seqlens_q far out of order) could make the line
    // longer than any call's is: then nothing is computed.
    longest = __reduce_max_sync(0xffffffffu, longest) + kUnitTiles;
    if (W > INT32_MAX || rows > 2ll * p.total_q || (p.whole && U * longest > INT32_MAX)) {
      if (blockIdx.x == 0 && lane == 0) set_status(p.status, MTPATTN_ERR_QLEN);
      W = U = 0;
    }
    length = static_cast<int>(W);
    units = static_cast<int>(U);
    C = max(1, static_cast<int>((static_cast<uint32_t>(W) + p.ctas - 1) / static_cast<uint32_t>(p.ctas)));
    V = 0;
    // Units stay whole where so many of the longest take no longer than equal pieces and what cutting costs
    // (in tiles): the join, and its bytes, fewer for units that are not full.  Both sides, of tables above kWholeTiles;
    // 4 tokens of 16 heads where no heads are given.  kCutTiles 4, 7 and 10: 16 x 700 keys 16.2, 15.7 and 15.7 us; 8 x 1000
    // 16.0, 16.0 and 18.4; in tables of 8192 pages 1 x 500 15.7, 19.8 and 19.8, 1 x 1000 15.9, 15.9 and 28.5.  kCutPieces
    // 20, 40 and 80: 64-node trees over 8 x 8191 keys 136.7, 136.6 and 140.1; 20 x 2000, 1 token of 128 heads, 44.2, 29.0
    // and 29.0; in tables of 8192 pages 1 x 500 19.8, 19.8 and 15.7, 1 x 1000 28.4, 15.9 and 15.9.
    const float full = fminf(1.f, static_cast<float>(p.total_q) * static_cast<float>(p.heads) / static_cast<float>(N * max(units, 1)));
    const int join = kCutTiles + static_cast<int>(static_cast<float>(units + p.ctas) * full * (N / 64.f / kCutPieces));
    const int each = max(1, static_cast<int>((static_cast<uint32_t>(units) + p.ctas - 1) / static_cast<uint32_t>(p.ctas)));
    if (static_cast<int64_t>(units) * longest <= INT32_MAX &&
        (p.whole || static_cast<int64_t>(each) * longest <= C + static_cast<int>(static_cast<uint32_t>(join) / each))) {
      V = longest;
      C = each * longest;
      length = units * longest;
    }
    // Where all sequences have the same row tiles, the CTAs that have one piece of a sequence's keys between them
    // go over it at the same time: it comes from memory once.  (On a line of row tiles one after the other, 16 x
    // 35000 tokens with 2 row tiles were read twice, 654 MB.)
    G = 1;
    tall = __reduce_max_sync(0xffffffffu, tall);
    low = __reduce_min_sync(0xffffffffu, low);
    if (!V && tall == low && tall > 1 && p.ctas % tall * 10 <= p.ctas) {
      G = tall;
      const uint32_t groups = static_cast<uint32_t>(p.ctas) / G;
      length = static_cast<int>(static_cast<uint32_t>(length) / G);
      C = static_cast<int>((length + groups - 1) / groups);
    }
    lo = pos = static_cast<int>(min(static_cast<int64_t>(length), static_cast<int64_t>(blockIdx.x / G) * C));
    hi = static_cast<int>(min(static_cast<int64_t>(length), static_cast<int64_t>(lo) + C));
    if (p.num_seqs > 32) {                           // the first sequences of the piece, or the last whose sums are known
      const int gw = V ? group_T * V : group_w / G;
      const int w_upto = warp_scan(gw, lane), T_upto = warp_scan(group_T, lane);
      const int k = min(31, __popc(__ballot_sync(0xffffffffu, w_upto <= lo)));
      before = __shfl_sync(0xffffffffu, w_upto - gw, k);
      units_before = __shfl_sync(0xffffffffu, T_upto - static_cast<int>(group_T), k);
      b0 = 32 * k;
      mine = seq_of<N>(p, raw_at(p, b0 + lane));
    }
    upto = warp_scan(weight(), lane);
    units_upto = warp_scan(mine.T, lane);
  }
  __device__ __forceinline__ int weight() const {    // of the held sequence
    return V ? mine.T * V : G > 1 ? (mine.T ? mine.nt + kUnitTiles : 0) : mine.w;
  }
  // The next segment; s.end if there is none.  Returns the sequence's error bits.
  __device__ __forceinline__ int next(const LatentParams& p, int lane, Segment& s) {
    s.end = 1;
#pragma unroll 1
    while (pos < hi) {
      const int all = __shfl_sync(0xffffffffu, upto, 31);
      if (pos >= before + all) {
        before += all;
        units_before += __shfl_sync(0xffffffffu, units_upto, 31);
        b0 += 32;
        if (b0 >= p.num_seqs) return 0;             // lengths changed under the call
        mine = seq_of<N>(p, raw_at(p, b0 + lane));
        upto = warp_scan(weight(), lane);
        units_upto = warp_scan(mine.T, lane);
        continue;
      }
      const int at = pos - before;
      const int f = __ffs(__ballot_sync(0xffffffffu, upto > at)) - 1;
      const int nt = __shfl_sync(0xffffffffu, mine.nt, f);
      const int places = V ? V : nt + kUnitTiles;
      const int in = at - (f ? __shfl_sync(0xffffffffu, upto, f - 1) : 0);
      const int nth = G > 1 ? blockIdx.x % G : in / places, in_unit = G > 1 ? in : in - nth * places;
      unit = units_before + nth + (f ? __shfl_sync(0xffffffffu, units_upto, f - 1) : 0);
      unit0 = pos - in_unit;
      unit_places = places;
      const int to = min(places, in_unit + hi - pos);                // of the unit, in this piece
      s.t0 = max(0, in_unit - kUnitTiles);
      s.t1 = min(nt, to - kUnitTiles);
      pos += to - in_unit;
      if (s.t0 >= s.t1) continue;                   // none of its tiles
      s.b = b0 + f;
      s.q0 = __shfl_sync(0xffffffffu, mine.q0, f);
      s.n = __shfl_sync(0xffffffffu, mine.n, f);
      s.L = __shfl_sync(0xffffffffu, mine.L, f);
      s.m = nth;
      s.nt = nt;
      s.slot = unit0 <= lo ? 0 : 1;
      s.end = s.bad = 0;
      return __shfl_sync(0xffffffffu, mine.err, f);
    }
    return 0;
  }
  // What the join has to know of the last segment's unit.
  __device__ __forceinline__ JoinNote note(const LatentParams& p, const Segment& s) const {
    JoinNote n;
    // (its first tile is at place kUnitTiles: the pieces are those of its tiles)
    n.first = blockIdx.x;
    n.pieces = V ? 1 : (unit0 + unit_places - 1) / C - n.first / G + 1;
    n.first_slot = s.slot;
    n.q0 = s.q0;
    n.m = s.m;
    n.rows = min(N, s.n * p.heads - s.m * N);
    n.stride = G;
    n.pad = 0;
    return n;
  }
};

// ---- arithmetic and operands ---------------------------------------------------------------------

__device__ __forceinline__ float exp2_hw(float x) {   // 2^x, hardware approximation
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
// The largest of the warp's 32 numbers; NaN is passed over.
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;\n" : "=f"(y) : "f"(x));
  return y;
}
// Two f16x2 words (four values, lowest first) as e4m3 codes hi, and what they leave, as f16x2 words.
__device__ __forceinline__ uint32_t first_term(uint32_t x0, uint32_t x1, uint32_t& y0, uint32_t& y1) {
  uint32_t hi;
  asm("{\n"
      " .reg .b16 h0, h1;\n"
      " .reg .b32 g0, g1;\n"
      " cvt.rn.satfinite.e4m3x2.f16x2 h0, %3;\n"
      " cvt.rn.satfinite.e4m3x2.f16x2 h1, %4;\n"
      " cvt.rn.f16x2.e4m3x2 g0, h0;\n"
      " cvt.rn.f16x2.e4m3x2 g1, h1;\n"
      " sub.rn.f16x2 %1, %3, g0;\n"
      " sub.rn.f16x2 %2, %4, g1;\n"
      " mov.b32 %0, {h0, h1};\n"
      "}\n"
      : "=r"(hi), "=r"(y0), "=r"(y1)
      : "r"(x0), "r"(x1));
  return hi;
}
// Q's: e4m3 codes hi + lo.
__device__ __forceinline__ void two_terms(uint32_t x0, uint32_t x1, uint32_t& hi, uint32_t& lo) {
  uint32_t y0, y1;
  hi = first_term(x0, x1, y0, y1);
  asm("{\n"
      " .reg .b16 l0, l1;\n"
      " cvt.rn.satfinite.e4m3x2.f16x2 l0, %1;\n"
      " cvt.rn.satfinite.e4m3x2.f16x2 l1, %2;\n"
      " mov.b32 %0, {l0, l1};\n"
      "}\n"
      : "=r"(lo)
      : "r"(y0), "r"(y1));
}
// A weight's: hi is an e4m3 code, lo an e5m2 one, which is the upper byte of an f16.  What is added to the lower byte
// first rounds it: half a step to the nearest, where lo is 2^-10 or more; below, the key's dither, 0 to 255 in both
// halves, up or down in the proportion of the bits that go.  (No weight stays none.  A NaN's lo is lost, but not its hi,
// and no carry leaves its half.)
__device__ __forceinline__ uint32_t round_e5m2(uint32_t y, uint32_t dither) {
  const __half2 v = *reinterpret_cast<const __half2*>(&y);
  const uint32_t large = __hgeu2_mask(__habs2(v), __half2half2(__ushort_as_half(0x1400)));   // 2^-10
  return y + ((dither & ~large) | (0x00800080u & large));
}
__device__ __forceinline__ void weight_terms(uint32_t x0, uint32_t x1, uint32_t dither, uint32_t& hi, uint32_t& lo) {
  uint32_t y0, y1;
  hi = first_term(x0, x1, y0, y1);
  lo = __byte_perm(round_e5m2(y0, dither), round_e5m2(y1, dither), 0x7531);
}
// What four weights' terms stand for together, added to l.
__device__ __forceinline__ void add_weights(float* l, uint32_t hi, uint32_t lo) {
  uint32_t x[2];
  asm("{\n"
      " .reg .b16 h0, h1;\n"
      " mov.b32 {h0, h1}, %2;\n"
      " cvt.rn.f16x2.e4m3x2 %0, h0;\n"
      " cvt.rn.f16x2.e4m3x2 %1, h1;\n"
      "}\n"
      : "=r"(x[0]), "=r"(x[1])
      : "r"(hi));
#pragma unroll
  for (int i = 0; i < 2; ++i)
    asm("{\n"
        " .reg .b16 a, b;\n"
        " .reg .b32 both;\n"
        " add.rn.f16x2 both, %2, %3;\n"
        " mov.b32 {a, b}, both;\n"
        " add.rn.f32.f16 %0, a, %0;\n"
        " add.rn.f32.f16 %1, b, %1;\n"
        "}\n"
        : "+f"(l[2 * i]), "+f"(l[2 * i + 1])
        : "r"(x[i]), "r"(__byte_perm(lo, 0u, i ? 0x3424 : 0x1404)));
}
__device__ __forceinline__ uint32_t half2_of(float a, float b) {   // a in the low half
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(d) : "f"(b), "f"(a));
  return d;
}
// A bf16 pair scaled by f (a power of two, twice), as an f16 pair: exact down to 2^-17 of a scaled value.
__device__ __forceinline__ uint32_t scaled_half2(uint32_t w, uint32_t f) {
  asm("mul.rn.bf16x2 %0, %0, %1;\n" : "+r"(w) : "r"(f));
  return half2_of(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// n columns of a lane each, n 8, 16 or 32.
template <int n>
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&v)[n]) {
  if constexpr (n == 32) {
    tmem_ld32(addr, v);
  } else if constexpr (n == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(addr));
  } else {
    static_assert(n == 8);
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(addr));
  }
}
// Waits for the loads above; the registers go through it, so that none is used before.
template <int n>
__device__ __forceinline__ void tmem_wait(uint32_t (&v)[n]) {
  if constexpr (n == 32) {
    tmem_ld_wait(v);
  } else if constexpr (n == 16) {
    asm volatile("tcgen05.wait::ld.sync.aligned;\n"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
                 :
                 : "memory");
  } else {
    asm volatile("tcgen05.wait::ld.sync.aligned;\n"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7])
                 :
                 : "memory");
  }
}
template <int n>
__device__ __forceinline__ void tmem_st(uint32_t addr, const uint32_t (&v)[n]) {
  if constexpr (n == 32) {
    tmem_st32(addr, v);
  } else if constexpr (n == 16) {
    tmem_st16(addr, v);
  } else {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(addr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  }
}

// Descriptors of a 64-byte-swizzled operand (as sdesc_sw128, layout 4): 8-row groups `sbo` apart.
__device__ __forceinline__ uint64_t sdesc_sw64(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFF) | (static_cast<uint64_t>((lbo >> 4) & 0x3FFF) << 16) |
         (static_cast<uint64_t>((sbo >> 4) & 0x3FFF) << 32) | (1ull << 46) | (4ull << 61);
}
constexpr uint32_t kAMajorM = 1u << 15;              // instruction descriptor: A is M-major
constexpr uint32_t kBE5m2 = 1u << 10;                // ... B is of e5m2

// Descriptors (sdesc_sw128 of sm100.cuh, sdesc_sw64) in two words: operands differ in the first one only, by
// constants.  A thread that issues products shares its scheduler with two softmax warps, and a tile's 50
// products have to go out in less than 2500 clocks.
struct Desc {
  uint32_t lo, hi;
};
__device__ __forceinline__ Desc desc_of(uint64_t d) { return {static_cast<uint32_t>(d), static_cast<uint32_t>(d >> 32)}; }

// D (+)= A B
template <bool kAccumulate>
__device__ __forceinline__ void mma_one(uint32_t d_tmem, uint32_t a, uint32_t a_hi, uint32_t b, uint32_t b_hi, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 x, y;\n mov.b64 x, {%1, %2};\n mov.b64 y, {%3, %4};\n setp.ne.b32 p, %6, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %5, p;\n}\n" ::"r"(d_tmem),
      "r"(a), "r"(a_hi), "r"(b), "r"(b_hi), "r"(idesc), "n"(kAccumulate ? 1 : 0)
      : "memory");
}
// D (+)= A B0, D += A B1, B0 and B1 of two formats.  (Measured, M 128, N 64: 96 clocks the pair; shared memory gives 128
// bytes a clock, and A is 4 KB, B 2 KB.  Kept in the collector for the second product, A would come once, in 78, but
// then both products take B in the first one's format, as measured.)
__device__ __forceinline__ void mma_two(uint32_t d_tmem, uint32_t a, uint32_t a_hi, uint32_t b0, uint32_t b0_hi, uint32_t b1,
                                        uint32_t b1_hi, uint32_t idesc0, uint32_t idesc1, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 x, y, z;\n mov.b64 x, {%1, %2};\n mov.b64 y, {%3, %4};\n mov.b64 z, {%5, %6};\n"
      " setp.ne.b32 p, %9, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %7, p;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, z, %8, 1;\n}\n" ::"r"(d_tmem),
      "r"(a), "r"(a_hi), "r"(b0), "r"(b0_hi), "r"(b1), "r"(b1_hi), "r"(idesc0), "r"(idesc1), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void prefetch_line(const void* p) {
  asm volatile("prefetch.global.L2 [%0];\n" ::"l"(reinterpret_cast<uint64_t>(p)) : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;\n" ::"l"(reinterpret_cast<uint64_t>(p)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void st_shared8(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.u32 [%0], {%1,%2};\n" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};\n" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
// Codes with the NaN ones (0x7f, 0xff) as zeros.
__device__ __forceinline__ uint32_t without_nan(uint32_t w) {
  return w & ~__vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu);
}

// What n numbers of every lane come to over the warp, by sums or by the largest (NaN is passed over): lane r
// gets that of v[r % n].
template <int n, typename Join>
__device__ __forceinline__ float over_lanes(float (&v)[n], int lane, Join join) {
#pragma unroll
  for (int o = n / 2; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const bool up = lane & o;
      const float send = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
      v[i] = join(keep, __shfl_xor_sync(0xffffffffu, send, o));
    }
#pragma unroll
  for (int o = n; o < 32; o <<= 1) v[0] = join(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
  return v[0];
}
template <int n>
__device__ __forceinline__ float row_sums(float (&v)[n], int lane) {
  return over_lanes(v, lane, [](float a, float b) { return a + b; });
}
template <int n>
__device__ __forceinline__ float row_maxima(float (&v)[n], int lane) {
  return over_lanes(v, lane, [](float a, float b) { return fmaxf(a, b); });
}

// What shared memory holds of n rows, 16 bytes at a time; from a 16-byte boundary.
template <int n>
__device__ __forceinline__ void load_rows(const float* p, float (&x)[n]) {
#pragma unroll
  for (int i = 0; i < n / 4; ++i) {
    const float4 v = reinterpret_cast<const float4*>(p)[i];
    x[4 * i] = v.x;
    x[4 * i + 1] = v.y;
    x[4 * i + 2] = v.z;
    x[4 * i + 3] = v.w;
  }
}

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
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, wait_for(bar, parity, abort));
}

// Warps that meet, with a limit (a named barrier has none): false after an abort.
struct Meeting {
  uint32_t bar;
  uint32_t turns;
  __device__ __forceinline__ void arrive(int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  }
  __device__ __forceinline__ bool wait(volatile int* abort) { return warp_wait(bar, turns++ & 1, abort); }
  __device__ __forceinline__ bool operator()(int lane, volatile int* abort) {
    arrive(lane);
    return wait(abort);
  }
};

// The four warps of a half of the rows meet once a tile, by the hardware's barrier, which has no limit: so none
// of them leaves the tiles alone.  One whose wait ran out says so here, by a vote, and all leave together.
__device__ __forceinline__ bool any_of_half(int half, bool x) {
  uint32_t y;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %2, 0;\n barrier.cta.red.or.pred q, %1, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(y)
      : "r"(1 + half), "r"(static_cast<uint32_t>(x))
      : "memory");
  return y != 0;
}
__device__ __forceinline__ void meet_half(int half) { asm volatile("barrier.cta.sync %0, 128;\n" ::"r"(1 + half) : "memory"); }

// ---- the kernel ----------------------------------------------------------------------------------

template <int N>
__global__ void __launch_bounds__(kLatentThreads, 1) latent_attn_kernel(const __grid_constant__ LatentParams p) {
  extern __shared__ __align__(1024) unsigned char base[];
  if (smem_u32(base) & 1023) {                     // the operands' swizzle needs it; no kernel sets
    if (threadIdx.x == 0) set_status(p.status, MTPATTN_ERR_TIMEOUT);   // other shared memory aside
    return;
  }
  constexpr int kHalf = N / 2;                     // rows of a softmax warp
  Shared<N>& sh = *reinterpret_cast<Shared<N>*>(base + off_bars<N>());
  Bars& bars = sh.bars;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = &bars.abort;
  const uint32_t smem = smem_u32(base);

  // ---- set-up ------------------------------------------------------------------------------
  if (warp == 1) {
    tmem_alloc(smem_u32(&bars.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i)
      for (int c = 0; c < kBlocks; ++c) {
        mbar_init(smem_u32(&bars.full[i][c]), 1);
        mbar_init(smem_u32(&bars.empty[i][c]), 1);
      }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars.s_full[i]), 1);
      mbar_init(smem_u32(&bars.s_free[i]), kSoftWarps);
    }
    for (int i = 0; i < kBlocks; ++i) mbar_init(smem_u32(&bars.p_full[i]), kSoftWarps / kBlocks);
    mbar_init(smem_u32(&bars.pv_done), 1);
    mbar_init(smem_u32(&bars.q_full), kSoftWarps);
    for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&bars.final_mma[i]), 1);
    for (int i = 0; i < 3; ++i) mbar_init(smem_u32(&bars.meet[i]), i < 2 ? kSoftWarps / 2 : kSoftWarps);
    for (int i = 0; i < kSegRing; ++i) {
      mbar_init(smem_u32(&bars.seg_full[i]), 1);
      mbar_init(smem_u32(&bars.seg_free[i]), kSoftWarps + 3);
    }
    bars.abort = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem_base;
  // What every CTA will want first is asked into L2 while the work before this on the stream still runs (the L2
  // is where all writes meet, so nothing can be stale there): a line of the block tables and of Q a thread.
  {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kLatentThreads + tid;
    const int64_t table_lines = (static_cast<int64_t>(p.num_seqs) * p.max_pages * 4 + 127) / 128;
    constexpr int kRowLines = kRow * 2 / 128;
    if (i < table_lines) prefetch_line(reinterpret_cast<const char*>(p.block_tables) + 128 * i);
    if (i < static_cast<int64_t>(p.total_q) * p.heads * kRowLines) {
      const uint32_t row = static_cast<uint32_t>(i) / kRowLines, tok = row / static_cast<uint32_t>(p.heads);
      prefetch_line(p.q + static_cast<int64_t>(tok) * p.q_stride_tok + static_cast<int64_t>(row - tok * p.heads) * p.q_stride_head +
                    (static_cast<uint32_t>(i) - row * kRowLines) * 64);
    }
  }
  // A programmatic dependent of the previous work on the stream: nothing global was read so far; and
  // the join may be scheduled (it waits for this grid before it reads partials).
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");

  static_assert(kWarpSoft * 32 * kFewRegisters + kSoftWarps * 32 * kManyRegisters <= kLatentThreads * kLaunchRegisters,
                "registers of the block: a larger sum would wait forever");
  if (warp < kWarpSoft) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kFewRegisters));
    if (warp == 0) {
      // ============================== the walk, and the scores =====================================
      Walker<N> walk;
      walk.start(p, lane);
      if (blockIdx.x == 0 && lane == 0) *p.units = walk.V ? 0 : min(walk.units, p.unit_bound);
      constexpr uint32_t kIdesc = idesc_e4m3_f32(128, 2 * N, false);
      const Desc q = desc_of(sdesc_sw128(smem + off_q<N>(), 16, 1024));
      const Desc q_rope = desc_of(sdesc_sw64(smem + off_q<N>() + kColumns * q_column<N>(), 16, 512));
      const Desc c0 = desc_of(sdesc_sw64(smem, 16, kGroup));
      uint32_t u = 0;                                // tiles so far
#pragma unroll 1
      for (int e = 0;;) {
        Segment s;
        const int err = walk.next(p, lane, s);
        auto leave_note = [&]() {
          if (lane == 0 && s.t0 == 0 && !walk.V && walk.unit < p.unit_bound) p.notes[walk.unit] = walk.note(p, s);
        };
        if (!s.end && err) {
          leave_note();
          // zeros for the rows of a sequence that cannot be computed, here: it has no tiles
          if (lane == 0) set_status(p.status, err);
          const int rows = min(N, s.n * p.heads - s.m * N);
#pragma unroll 1
          for (int i = 0; i < rows; ++i) {
            const int rr = s.m * N + i, t = rr / p.heads;
            uint4* out = reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(s.q0 + t) * p.out_stride_tok +
                                                  static_cast<int64_t>(rr - t * p.heads) * p.out_stride_head);
            out[lane] = out[lane + 32] = make_uint4(0u, 0u, 0u, 0u);
          }
          continue;
        }
        if (!warp_wait(smem_u32(&bars.seg_free[e % kSegRing]), ((e / kSegRing) & 1) ^ 1, abort_flag)) break;
        if (lane == 0) {
          bars.seg[e % kSegRing] = s;
          mbar_arrive(smem_u32(&bars.seg_full[e % kSegRing]));
        }
        if (s.end) break;
        leave_note();
        // Its Q is asked into L2 while the softmax warps are with the one before (the first ones are there already).
        if (e > 0) {
          constexpr int kRowLines = kRow * 2 / 128;
          const int lines = min(N, s.n * p.heads - s.m * N) * kRowLines;
#pragma unroll 1
          for (int i = lane; i < lines; i += 32) {
            const int r = i / kRowLines, rr = s.m * N + r, t = rr / p.heads;
            prefetch_line(p.q + static_cast<int64_t>(s.q0 + t) * p.q_stride_tok +
                          static_cast<int64_t>(rr - t * p.heads) * p.q_stride_head + (i - r * kRowLines) * 64);
          }
        }
        if (!warp_wait(smem_u32(&bars.q_full), e & 1, abort_flag)) break;
        const uint32_t end = u + (s.t1 - s.t0);
        if (elect_one()) {
          tc_fence_after();
#pragma unroll 1
          for (; u < end; ++u) {                     // S(u) = C Q^T
            const uint32_t st = u % kStages, parity = (u / kStages) & 1, d = tmem + (u & 1) * kSBuf;
            bool ok = wait_for(smem_u32(&bars.s_free[u & 1]), ((u >> 1) & 1) ^ 1, abort_flag);
#pragma unroll
            for (int c = 0; c < kBlocks; ++c) ok = ok && wait_for(smem_u32(&bars.full[st][c]), parity, abort_flag);
            if (!ok) break;
            tc_fence_after();
            const uint32_t a = c0.lo + st * (kStage >> 4);
            mma_one<false>(d, a, c0.hi, q.lo, q.hi, kIdesc);
#pragma unroll
            for (int k = 1; k < 4 * kColumns; ++k)   // 32 dims
              mma_one<true>(d, a + (((k >> 1) * kAtom + 32 * (k & 1)) >> 4), c0.hi,
                            q.lo + (((k >> 2) * q_column<N>() + 32 * (k & 3)) >> 4), q.hi, kIdesc);
#pragma unroll
            for (int k = 0; k < 2; ++k) mma_one<true>(d, a + ((kRopeAt + 32 * k) >> 4), c0.hi, q_rope.lo + (32 * k >> 4), q_rope.hi, kIdesc);
            mma_commit(smem_u32(&bars.s_full[u & 1]));
          }
        }
        __syncwarp();
        if (*abort_flag) break;
        u = end;
        ++e;
      }
      if (blockIdx.x == 0)                           // tell of sequences whose rows are not known
        for (int b = lane; b < p.num_seqs; b += 32) {
          const int q0 = p.cu_q[b], q1 = p.cu_q[b + 1];
          if (q0 < 0 || q1 <= q0 || q1 > p.total_q) set_status(p.status, MTPATTN_ERR_QLEN);
        }
      __syncwarp();
      if (elect_one()) {                             // no product may run on when the CTA ends
        mma_commit(smem_u32(&bars.final_mma[0]));
        volatile int no_abort = 0;
        wait_for(smem_u32(&bars.final_mma[0]), 0, &no_abort);
      }
      __syncwarp();
    } else if (warp >= 2) {
      // ============================== the tiles by TMA, two blocks a warp ===========================
      const int first = (warp - 2) * kWarpBlocks;
      if (lane == 0) prefetch_tmap(&p.tmap);
      const uint64_t once = l2_policy_evict_first();
      uint64_t again;
      asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;\n" : "=l"(again));
      uint32_t u = 0;                                // tiles so far
      int asked = 0;                                 // blocks of the last one asked for
      bool ok = true;
#pragma unroll 1
      for (int e = 0; ok; ++e) {
        ok = warp_wait(smem_u32(&bars.seg_full[e % kSegRing]), (e / kSegRing) & 1, abort_flag);
        if (!ok) break;
        Segment& s = bars.seg[e % kSegRing];
        if (s.end) break;
        const int t0 = s.t0, t1 = s.t1, pages = (s.L + kPage - 1) / kPage;
        const int32_t* bt = p.block_tables + static_cast<int64_t>(s.b) * p.max_pages;
        const uint64_t policy = static_cast<int64_t>(s.n) * p.heads <= N ? once : again;
        // table entries, a lane one of eight tiles' 4 that are this warp's, with the next 32 on the way
        auto entries = [&](int t) -> int {
          const int64_t pg = static_cast<int64_t>(t + lane / kWarpPages) * kTilePages + first * kBlockPages + lane % kWarpPages;
          return pg < pages ? bt[pg] : 0;
        };
        int now = entries(t0), ahead = entries(t0 + 32 / kWarpPages);
#pragma unroll 1
        for (int t = t0; t < t1; ++t, ++u) {
          const int k = (t - t0) % (32 / kWarpPages);
          if (k == 0 && t > t0) {
            now = ahead;
            ahead = entries(t + 32 / kWarpPages);
          }
          // a lane half a page
          const int np = min(kTilePages, pages - t * kTilePages) - first * kBlockPages;   // this warp's, if above 0
          const int mine = __shfl_sync(0xffffffffu, now, k * kWarpPages + lane % kWarpPages);
          const bool bad = __any_sync(0xffffffffu, lane < min(np, kWarpPages) && (mine < 0 || mine >= p.num_pages));
          if (bad && lane == 0) {
            *const_cast<volatile int*>(&s.bad) = 1;
            set_status(p.status, MTPATTN_ERR_PAGE);
          }
          // A stage is free late, and a fetch from memory would be the longest part of its turn: pages are brought
          // into L2 some tiles ahead.
          {
            const int k2 = k + kPrefetch;
            const int far = __shfl_sync(0xffffffffu, k2 < 32 / kWarpPages ? now : ahead, (k2 % (32 / kWarpPages)) * kWarpPages + lane % kWarpPages);
            if (lane < kWarpPages && t + kPrefetch < t1 &&
                (t + kPrefetch) * kTilePages + first * kBlockPages + lane < pages && far >= 0 && far < p.num_pages)
              prefetch_l2(p.cache + static_cast<int64_t>(far) * (kPage * kRow), kPage * kRow);
          }
          // At first all CTAs ask at once: the first tile, then Q, which the first product wants too, then more.  (In the
          // first segment only: its Q's phase is still the last one there.)
          if (e == 0 && t == t0 + 1 && !(ok = warp_wait(smem_u32(&bars.q_full), 0, abort_flag))) break;
          const int st = u % kStages;
          const uint32_t stage = smem + st * kStage;
#pragma unroll 1
          for (int c = 0; c < kWarpBlocks; ++c) {
            ok = warp_wait(smem_u32(&bars.empty[st][first + c]), ((u / kStages) & 1) ^ 1, abort_flag);
            if (!ok) break;
#ifdef MTPATTN_TEST_STALL
            if (s.b == 0 && s.m == 0 && t == 0 && first + c == 0) continue;   // test builds: the wait for it runs out
#endif
            asked = c + 1;
            const uint32_t bar = smem_u32(&bars.full[st][first + c]);
            const int here = bad ? 0 : max(0, min(kBlockPages, np - c * kBlockPages));   // pages to fetch
            if (lane == 0) {
              if (here == 0) mbar_arrive(bar);       // (of a bad page nothing: the segment's rows become zeros)
              else mbar_arrive_expect_tx(bar, here * kPage * kRow);
            }
            const int pg = __shfl_sync(0xffffffffu, mine, (c * kBlockPages + (lane >> 1)) % kWarpPages);
            if (lane < 2 * here)
              tma_load_4d(stage + (2 * (first + c) * kBlockPages + lane) * kGroup, &p.tmap, bar, 0, (lane & 1) * 8, 0, pg, policy);
            __syncwarp();
          }
          if (!ok) break;
        }
        if (ok && lane == 0) mbar_arrive(smem_u32(&bars.seg_free[e % kSegRing]));
      }
      // What was asked for has to arrive before the CTA may end: u tiles whole, and blocks of one more after
      // an abort.
      if (*abort_flag) {
        volatile int no_abort = 0;
        if (!ok && asked < kWarpBlocks)
          for (int c = 0; c < asked; ++c) wait_for(smem_u32(&bars.full[u % kStages][first + c]), (u / kStages) & 1, &no_abort);
        for (uint32_t k = 1; k <= kStages && k <= u; ++k)
          for (int c = 0; c < kWarpBlocks; ++c)
            wait_for(smem_u32(&bars.full[(u - k) % kStages][first + c]), ((u - k) / kStages) & 1, &no_abort);
      }
    } else if (warp == 1) {
      // ============================== the outputs ===================================================
      // (Issued apart from the scores, so that neither waits for what the other lacks.)
      if (elect_one()) {
        auto wait = [&](uint64_t& bar, uint32_t parity) -> bool { return wait_for(smem_u32(&bar), parity, abort_flag); };
        constexpr uint32_t kIdesc = idesc_e4m3_f32(128, N, true) | kAMajorM;
        const Desc lo = desc_of(sdesc_sw64(smem + off_p<N>(), 512, 512)), hi = desc_of(sdesc_sw64(smem + kRopeAt, 512, kGroup));
        const Desc v0 = desc_of(sdesc_sw64(smem, kAtom, kGroup));
        uint32_t u = 0;
        bool alive = true;
#pragma unroll 1
        for (int e = 0; alive; ++e) {
          if (!(alive = wait(bars.seg_full[e % kSegRing], (e / kSegRing) & 1))) break;
          const volatile Segment& s = bars.seg[e % kSegRing];
          const bool last = s.end;
          const uint32_t end = u + (s.t1 - s.t0);
          mbar_arrive(smem_u32(&bars.seg_free[e % kSegRing]));
          if (last) break;
#pragma unroll 1
          for (uint32_t more = 0; u < end && alive; ++u, more = 1) {   // O (+)= C^T P^T
            const uint32_t st = u % kStages, at = st * (kStage >> 4);
#pragma unroll
            for (int k = 0; k < kBlocks; ++k) {
              if (!(alive = wait(bars.p_full[k], u & 1))) break;
              tc_fence_after();
              // Both terms of P one after the other, the e5m2 one first.
#pragma unroll
              for (int c = 0; c < kColumns; ++c)
                mma_two(tmem + kOCol + c * N, v0.lo + at + ((k * (kBlockKeys / 8) * kGroup + 2 * c * kAtom) >> 4), v0.hi,
                        lo.lo + (k * kBlockKeys * 64 >> 4), lo.hi, hi.lo + at + (k * (kBlockKeys / 8) * kGroup >> 4), hi.hi,
                        kIdesc | kBE5m2, kIdesc, k ? 1u : more);
              mma_commit(smem_u32(&bars.empty[st][k]));    // (with the rows of both of P's terms)
            }
            if (!alive) break;
            mma_commit(smem_u32(&bars.pv_done));
          }
        }
        mma_commit(smem_u32(&bars.final_mma[1]));
        volatile int no_abort = 0;
        wait_for(smem_u32(&bars.final_mma[1]), 0, &no_abort);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kManyRegisters));
    // ============================== softmax, Q's operand, the output ==============================
    const int w = warp - kWarpSoft, quarter = warp & 3, half = w >> 2;
    const int key = quarter * 32 + lane;             // of the tile
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const float descale = *p.descale, factor = p.scale_log2 * descale;
    const int row0 = half * kHalf;
    Meeting meet{smem_u32(&bars.meet[half]), 0}, meet_all{smem_u32(&bars.meet[2]), 0};
    uint32_t u = 0;
    bool alive = true;
    // Q's two terms of a segment, kSide lanes a row, and what there is of each row.  Asks that the last product that
    // reads the previous ones is done: that all S of their segment has been read.
    auto prepare = [&](const Segment& of) {
      const int q0 = of.q0, n = of.n, m = of.m, rows = min(N, n * p.heads - m * N);
      constexpr int kSide = N == 16 ? 16 : 8, kParts = (kRow / 8 + kSide - 1) / kSide;   // blocks of 8 a lane
      constexpr int kStep = kSoftWarps * 32 / kSide;   // rows at a time; a multiple of 8
      const int side = lane % kSide, first = (w * 32 + lane) / kSide;
      constexpr int kTurns = N / kStep;
      uint4 x[kTurns][kParts];                       // all on their way at once
      uint64_t word[kTurns];
      auto fetch = [&](int r, int go) {
        const int rr = m * N + r, tok = r < rows ? rr / p.heads : 0;
        const uint4* src = reinterpret_cast<const uint4*>(p.q + static_cast<int64_t>(q0 + tok) * p.q_stride_tok +
                                                          static_cast<int64_t>(rr - tok * p.heads) * p.q_stride_head) + side;
#pragma unroll
        for (int i = 0; i < kParts; ++i)
          x[go][i] = r < rows && (kParts * kSide == kRow / 8 || side + i * kSide < kRow / 8) ? src[i * kSide]
                                                                                       : make_uint4(0u, 0u, 0u, 0u);
        word[go] = r < rows ? (p.mask ? p.mask[q0 + tok] : (2ull << tok) - 1ull) : 0;
      };
      // Where a row's blocks go.  Block j of the 64 of the latent part is half of a 16-byte place, column j / 16,
      // swizzled by the row's lowest bits, which are the same in all of a lane's rows.
      const uint32_t q = smem + off_q<N>();
      uint32_t place[16 / kSide];
#pragma unroll
      for (int i = 0; i < 16 / kSide; ++i) {
        const uint32_t j = side + i * kSide;
        place[i] = q + first * 128 + (((j >> 1) ^ (first & 7)) << 4) + (j & 1) * 8;
      }
      const uint32_t rope_place = q + kColumns * q_column<N>() + first * 64 + (((side >> 1) ^ ((first >> 1) & 3)) << 4) + (side & 1) * 8;
#pragma unroll
      for (int go = 0; go < kTurns; ++go) fetch(first + go * kStep, go);
#pragma unroll 1
      for (int r = first, go = 0; go < kTurns; ++go, r += kStep) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kParts; ++i)
          top = __vmaxu2(top, __vmaxu2(__vmaxu2(x[0][i].x & 0x7fff7fffu, x[0][i].y & 0x7fff7fffu),
                                       __vmaxu2(x[0][i].z & 0x7fff7fffu, x[0][i].w & 0x7fff7fffu)));
#pragma unroll
        for (int o = 1; o < kSide; o <<= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
        const int exponent = max(top & 0xffffu, top >> 16) >> 7;   // biased; 255: not finite
        const int a = min(134 - exponent, 126);
        uint32_t up = static_cast<uint32_t>(127 + a) << 7;
        if (exponent == 255) up = 0x7fc0u;           // NaN, and so all of the row's codes
        up |= up << 16;
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
          uint32_t h0, h1, l0, l1;
          two_terms(scaled_half2(x[0][i].x, up), scaled_half2(x[0][i].y, up), h0, l0);
          two_terms(scaled_half2(x[0][i].z, up), scaled_half2(x[0][i].w, up), h1, l1);
          if (i * kSide < kDim / 8) {
            const uint32_t at = place[i % (16 / kSide)] + i * kSide / 16 * q_column<N>() + go * kStep * 128;
            st_shared8(at, h0, h1);
            st_shared8(at + N * 128, l0, l1);
          } else if (side < 8) {
            const uint32_t at = rope_place + go * kStep * 64;
            st_shared8(at, h0, h1);
            st_shared8(at + N * 64, l0, l1);
          }
        }
        if (side == 0) {
          sh.factor[r] = r < rows ? factor * __uint_as_float(static_cast<uint32_t>(127 - a) << 23) : 0.f;
          sh.ref[r] = kNoRef;
          sh.word[r] = n < 64 ? word[0] & ((1ull << n) - 1ull) : word[0];
        }
#pragma unroll
        for (int k = 1; k < kTurns; ++k) {
#pragma unroll
          for (int i = 0; i < kParts; ++i) x[k - 1][i] = x[k][i];
          word[k - 1] = word[k];
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars.q_full));
    };
    // Turn e: segment e, and between its products and its output the next one's Q (turn -1: the first one's).
#pragma unroll 1
    for (int e = -1; alive; ++e) {
      Segment s;
      int rows = 0;
      bool whole = false;
      if (e >= 0) {
        s = bars.seg[e % kSegRing];
        rows = min(N, s.n * p.heads - s.m * N);
        // of the rows of this warp, in every lane: a load from shared memory waits for the products' reads
        float l[kHalf], fac[kHalf], ref[kHalf];
        load_rows(sh.factor + row0, fac);
#pragma unroll
        for (int r = 0; r < kHalf; ++r) l[r] = ref[r] = 0.f;
        // A row's products are below 2^26 (256 x 448 x 576): only past this factor can a logit leave float32's range.
        const bool wild = __any_sync(0xffffffffu, lane < kHalf && !(fabsf(sh.factor[row0 + lane % kHalf]) < 0x1p101f));
        const int start = s.L - s.n;                   // first new token
        const bool late = (s.t0 + 1) * kKeys > start;  // a row may see nothing of the first tile
#pragma unroll 1
        for (int t = s.t0; t < s.t1; ++t, ++u) {
          alive &= warp_wait(smem_u32(&bars.s_full[u & 1]), (u >> 1) & 1, abort_flag);
          tc_fence_after();
          const int j = t * kKeys + key;
          const bool ragged = (t + 1) * kKeys > start;  // new tokens, or places behind the sequence
          uint32_t seen = ~0u;                         // the rows of this warp that see the key
          bool nan = false;                            // the key may hold a NaN code
          if (ragged) {
            if (j >= start) seen = 0u;
            const uint64_t word = lane < kHalf ? sh.word[row0 + lane] : 0;
            const int first = t * kKeys + quarter * 32 - start;   // new token that lane 0's key is
#pragma unroll 1
            for (int k = max(0, -first); k < min(32, s.n - first); ++k) {
              const uint32_t rows_of = __ballot_sync(0xffffffffu, (word >> (first + k)) & 1);
              if (lane == k) seen = rows_of;
            }
          }
          float y[kHalf];                              // logits above the reference, then weights
          auto logits = [&]() {
            uint32_t h[kHalf], lo[kHalf];
            const uint32_t at = tmem + lanes + (u & 1) * kSBuf + row0;
            tmem_ld<kHalf>(at, h);
            tmem_ld<kHalf>(at + N, lo);
            tmem_wait<kHalf>(h);
            tmem_wait<kHalf>(lo);
#pragma unroll
            for (int r = 0; r < kHalf; ++r) y[r] = fmaf(__uint_as_float(h[r]) + __uint_as_float(lo[r]), fac[r], -ref[r]);
            if (wild) {                                // a logit that does makes its row NaN, at either end
#pragma unroll
              for (int r = 0; r < kHalf; ++r)
                if (isinf((__uint_as_float(h[r]) + __uint_as_float(lo[r])) * fac[r])) y[r] = NAN;
            }
            if (ragged) {
              nan = !(y[0] == y[0]);
#pragma unroll
              for (int r = 0; r < kHalf; ++r)
                if (!((seen >> r) & 1u)) y[r] = -INFINITY;
            }
          };
          // The dither: a tile's 128 keys have evenly spread numbers, and other ones in every tile of the sequence.
          const uint32_t dither = ((__brev(key) ^ static_cast<uint32_t>(t) * 0x9E3779B1u) >> 24) * 0x00010001u;
          uint32_t hi[kHalf / 4], lo[kHalf / 4];
          auto weights = [&]() {
#pragma unroll
            for (int r = 0; r < kHalf; r += 4) {
#pragma unroll
              for (int i = 0; i < 4; ++i) y[r + i] = exp2_hw(y[r + i]);
              weight_terms(half2_of(y[r], y[r + 1]), half2_of(y[r + 2], y[r + 3]), dither, hi[r / 4], lo[r / 4]);
            }
          };
          logits();
          // A reference is raised where a logit is too far above it, and at first.
          const bool forced = t == s.t0 || (ragged && late);
          bool over = forced;
          if (!forced) {
            float a = y[0], b = y[1];
#pragma unroll
            for (int r = 2; r < kHalf; r += 2) {
              a = fmaxf(a, y[r]);
              b = fmaxf(b, y[r + 1]);
            }
            over = fmaxf(a, b) > kShift + kTau;
          }
          over = any_of_half(half, over || !alive);
          if (over) {
            if (!(alive = !any_of_half(half, !alive || *abort_flag))) break;
            if (!forced) logits();
            float tops[kHalf];
#pragma unroll
            for (int r = 0; r < kHalf; ++r) tops[r] = y[r];
            const float mine = row_maxima<kHalf>(tops, lane);
            if (lane < kHalf) sh.xch[half][quarter][lane] = mine;
            meet_half(half);
            if (quarter == 0 && lane < kHalf) {
              const float (&x)[4][kHalf] = sh.xch[half];
              const float top = fmaxf(fmaxf(x[0][lane], x[1][lane]), fmaxf(x[2][lane], x[3][lane]));
              const float old = sh.ref[row0 + lane];   // kNoRef: the row has seen nothing, y is above 0
              float step = 0.f, f = 1.f;
              if (top > (old == kNoRef ? -INFINITY : kShift + kTau)) {
                step = kShift - top - (s.t1 - t > 2 ? kRoom : 0.f);   // (the last tiles will not raise it much)
                f = old == kNoRef ? 0.f : exp2_hw(step);
                sh.ref[row0 + lane] = (old == kNoRef ? 0.f : old) - step;
              }
              sh.step[row0 + lane] = step;
              sh.f[row0 + lane] = f;
            }
            meet_half(half);
#pragma unroll
            for (int r = 0; r < kHalf; r += 4) {
              float step[4];
              load_rows(sh.step + row0 + r, step);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                y[r + i] += step[i];
                ref[r + i] -= step[i];
              }
            }
            if (t > s.t0) {
              // (O may be touched once the previous tile's products are in it)
              alive &= warp_wait(smem_u32(&bars.pv_done), (u - 1) & 1, abort_flag);
              tc_fence_after();
#pragma unroll
              for (int r = 0; r < kHalf; r += 4) {
                float f[4];
                load_rows(sh.f + row0 + r, f);
#pragma unroll
                for (int i = 0; i < 4; ++i) l[r + i] *= f[i];
              }
#pragma unroll 1
              for (int c = 0; c < kColumns; ++c) {
                const uint32_t at = tmem + lanes + kOCol + c * N + row0;
                uint32_t o[kHalf];
                tmem_ld<kHalf>(at, o);
                tmem_wait<kHalf>(o);
#pragma unroll
                for (int r = 0; r < kHalf; r += 4) {
                  float f[4];
                  load_rows(sh.f + row0 + r, f);
#pragma unroll
                  for (int i = 0; i < 4; ++i) o[r + i] = __float_as_uint(__uint_as_float(o[r + i]) * f[i]);
                }
                tmem_st<kHalf>(at, o);
              }
              tmem_st_wait();
            }
          }
          weights();
          const uint32_t stage = smem + (u % kStages) * kStage;
          const uint32_t swz = (key >> 1) & 3;
          auto write = [&](uint32_t at, const uint32_t (&x)[kHalf / 4]) {
            at += (key & 7) * 64;
            if constexpr (kHalf == 8) {
              st_shared8(at + (swz << 4) + half * 8, x[0], x[1]);
            } else {
#pragma unroll
              for (int i = 0; i < kHalf / 16; ++i)
                st_shared16(at + (((half * (kHalf / 16) + i) ^ swz) << 4), x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
            }
          };
          write(stage + (key >> 3) * kGroup + kRopeAt, hi);
          // the previous tile's second terms of these keys have been read: a quarter is a block
          if (u > 0) alive &= warp_wait(smem_u32(&bars.empty[(u - 1) % kStages][quarter]), ((u - 1) / kStages) & 1, abort_flag);
          write(smem + off_p<N>() + (key >> 3) * kAtom, lo);
          if (ragged && j >= start && nan) {
            // this half's 256 of the key's values, without its NaN; none at all behind the sequence
#pragma unroll 4
            for (int i = 0; i < 16; ++i) {             // (in any order; this one meets all banks)
              const uint32_t at = stage + (key >> 3) * kGroup + (4 * half + (i >> 2)) * kAtom + (key & 7) * 64 +
                                  (((i + (key >> 1)) & 3) << 4);
              uint4 x = make_uint4(0u, 0u, 0u, 0u);
              if (j < s.L) {
                x = ld_shared16(at);
                x.x = without_nan(x.x);
                x.y = without_nan(x.y);
                x.z = without_nan(x.z);
                x.w = without_nan(x.w);
              }
              st_shared16(at, x.x, x.y, x.z, x.w);
            }
          }
          fence_proxy_async_smem();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(smem_u32(&bars.p_full[quarter]));
            mbar_arrive(smem_u32(&bars.s_free[u & 1]));
          }
#pragma unroll
          for (int r = 0; r < kHalf; r += 4) add_weights(l + r, hi[r / 4], lo[r / 4]);
        }
        if (!alive) break;
        // ---- the sums, and the next segment's Q while the last products run
        const bool bad = *const_cast<volatile int*>(&bars.seg[e % kSegRing].bad);
        whole = s.t0 == 0 && s.t1 == s.nt;
        {
          const float sum = row_sums<kHalf>(l, lane);
          if (lane < kHalf) sh.xch[half][quarter][lane] = sum;
        }
        if (!(alive = meet(lane, abort_flag))) break;
        if (quarter == 0) {
          const float (&x)[4][kHalf] = sh.xch[half];
          const int r = lane % kHalf, rr = s.m * N + row0 + r, tok = rr / p.heads;
          const float sum = (x[0][r] + x[1][r]) + (x[2][r] + x[3][r]);
          __syncwarp();
          if (lane < kHalf) {
            sh.f[row0 + r] = bad || sum == 0.f ? 0.f : descale / sum;   // (NaN: the row sees one, or holds one)
            // where the row goes, over the sums
            reinterpret_cast<int64_t*>(sh.xch[half])[r] = static_cast<int64_t>(s.q0 + tok) * p.out_stride_tok +
                                                          static_cast<int64_t>(rr - tok * p.heads) * p.out_stride_head;
            if (!whole)
              p.sum_part[(2 * static_cast<int64_t>(blockIdx.x) + s.slot) * N + row0 + r] = make_float2(sh.ref[row0 + r], bad ? __uint_as_float(kBadSum) : sum);
          }
        }
        if (!(alive = meet_all(lane, abort_flag))) break;
      }
      if (!(alive = warp_wait(smem_u32(&bars.seg_full[(e + 1) % kSegRing]), ((e + 1) / kSegRing) & 1, abort_flag))) break;
      const bool last = bars.seg[(e + 1) % kSegRing].end;
      if (!last) prepare(bars.seg[(e + 1) % kSegRing]);
      if (e >= 0) {
        // ---- the output
        if (!(alive = warp_wait(smem_u32(&bars.pv_done), (u - 1) & 1, abort_flag))) break;
        tc_fence_after();
        const int valid = min(kHalf, rows - row0);     // of this half's
        // A lane has one dim of all rows; exchanged between lanes (a butterfly on their lower bits), it stores 16
        // bytes of a row at a time, 4 dims of partial outputs or 8 of the output.  (4 or 2 bytes at a time took
        // 4100 clocks.)
        const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + s.slot;
        constexpr int kTurn = 4;         // 8 rows of 128 dims at a time, so many beside one another
#pragma unroll 1
        for (int at = 0; at < kColumns * kHalf / 8; at += kTurn) {
          uint32_t o[kTurn][8];
#pragma unroll
          for (int q = 0; q < kTurn; ++q) {
            const int c = (at + q) / (kHalf / 8), r0 = (at + q) % (kHalf / 8) * 8;
            tmem_ld<8>(tmem + lanes + kOCol + c * N + row0 + r0, o[q]);
          }
#pragma unroll
          for (int q = 0; q < kTurn; ++q) tmem_wait<8>(o[q]);
          if (whole) {
#pragma unroll
            for (int q = 0; q < kTurn; ++q) {
              const int c = (at + q) / (kHalf / 8), r0 = (at + q) % (kHalf / 8) * 8;
              const int d0 = c * 128 + quarter * 32;   // (a TMEM lane is a dim here)
              uint32_t x[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {            // rows 2i + bit 0, dims of the pair of lanes
                const float f0 = sh.f[row0 + r0 + 2 * i], f1 = sh.f[row0 + r0 + 2 * i + 1];
                const float v0 = f0 == 0.f ? 0.f : __uint_as_float(o[q][2 * i]) * f0;
                const float v1 = f1 == 0.f ? 0.f : __uint_as_float(o[q][2 * i + 1]) * f1;
                const float keep = lane & 1 ? v1 : v0, got = __shfl_xor_sync(0xffffffffu, lane & 1 ? v0 : v1, 1);
                const __nv_bfloat162 pair = lane & 1 ? __floats2bfloat162_rn(got, keep) : __floats2bfloat162_rn(keep, got);
                x[i] = *reinterpret_cast<const uint32_t*>(&pair);
              }
              uint32_t y[2][2], z[4];
#pragma unroll
              for (int h = 0; h < 2; ++h) {            // rows 4h + bits 0 and 1, dims of 4 lanes
                const uint32_t keep = lane & 2 ? x[2 * h + 1] : x[2 * h];
                const uint32_t got = __shfl_xor_sync(0xffffffffu, lane & 2 ? x[2 * h] : x[2 * h + 1], 2);
                y[h][0] = lane & 2 ? got : keep;
                y[h][1] = lane & 2 ? keep : got;
              }
#pragma unroll
              for (int h = 0; h < 2; ++h) {            // rows bits 0 .. 2, dims of 8 lanes
                const uint32_t keep = lane & 4 ? y[1][h] : y[0][h], got = __shfl_xor_sync(0xffffffffu, lane & 4 ? y[0][h] : y[1][h], 4);
                z[h] = lane & 4 ? got : keep;
                z[2 + h] = lane & 4 ? keep : got;
              }
              const int r = r0 + (lane & 7);
              if (r < valid)
                *reinterpret_cast<uint4*>(p.out + reinterpret_cast<const int64_t*>(sh.xch[half])[r] + d0 + (lane & 24)) =
                    make_uint4(z[0], z[1], z[2], z[3]);
            }
          } else {
#pragma unroll
            for (int q = 0; q < kTurn; ++q) {
              const int c = (at + q) / (kHalf / 8), r0 = (at + q) % (kHalf / 8) * 8;
              const int d0 = c * 128 + quarter * 32;
#pragma unroll
              for (int i = 0; i < 2; ++i) {            // rows 4i + bits 0 and 1, dims of 4 lanes
                uint32_t x[2][2], z[4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const uint32_t w0 = o[q][4 * i + 2 * h], w1 = o[q][4 * i + 2 * h + 1];
                  const uint32_t keep = lane & 1 ? w1 : w0, got = __shfl_xor_sync(0xffffffffu, lane & 1 ? w0 : w1, 1);
                  x[h][0] = lane & 1 ? got : keep;
                  x[h][1] = lane & 1 ? keep : got;
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const uint32_t keep = lane & 2 ? x[1][h] : x[0][h], got = __shfl_xor_sync(0xffffffffu, lane & 2 ? x[0][h] : x[1][h], 2);
                  z[h] = lane & 2 ? got : keep;
                  z[2 + h] = lane & 2 ? keep : got;
                }
                const int r = r0 + 4 * i + (lane & 3);
                if (r < valid)
                  *reinterpret_cast<uint4*>(p.o_part + (slot * N + row0 + r) * kDim + d0 + (lane & 28)) = make_uint4(z[0], z[1], z[2], z[3]);
              }
            }
          }
        }
        tc_fence_before();
      }
      if (last) break;
      // every softmax warp is done with this segment's data, and has written its part of the next one's
      if (!(alive = meet_all(lane, abort_flag))) break;
      if (e >= 0 && lane == 0) mbar_arrive(smem_u32(&bars.seg_free[e % kSegRing]));
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

// The join: out = descale sum_j w_j O_j / sum_j w_j l_j over a unit's pieces, w_j = 2^(ref_j - max ref).  128
// threads take four dims each of kRows rows, kGroups such groups of threads either a part of the pieces
// (kSplit: few units in many pieces) or more rows.  Reads what the main kernel has just written, out of L2;
// bound by its chain of notes, sums and partial outputs.
template <int N, int kRows, int kDims, int kGroups, bool kSplit, int kAhead>
__global__ void __launch_bounds__(kDims / 4 * kGroups) latent_join_kernel(const __grid_constant__ LatentParams p) {
  constexpr int kSide = kDims / 4, kThreads = kSide * kGroups, kCtaRows = kSplit ? kRows : kRows * kGroups;
  __shared__ float s_w[kCtaRows][kMaxCtas];
  __shared__ float s_inv[kCtaRows];
  __shared__ float4 s_acc[kSplit ? kGroups - 1 : 1][kRows][kSide];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  asm volatile("griddepcontrol.wait;\n" ::: "memory");   // every partial is written and visible
  const int units = __ldcg(p.units);
  const int4 a = __ldcg(reinterpret_cast<const int4*>(p.notes + blockIdx.x));
  const int4 b = __ldcg(reinterpret_cast<const int4*>(p.notes + blockIdx.x) + 1);
  if (static_cast<int>(blockIdx.x) >= units || a.x <= 1) return;
  const int n = a.x, first = a.y, q0 = a.w, m = b.x, stride = b.z;
  const int r0 = blockIdx.y * kCtaRows, rows = min(kCtaRows, b.y - r0);
  // A CTA whose wait ran out may have left no note: what stands there then is not followed.
  if (n > p.ctas || stride < 1 || stride > p.ctas || first < 0 || first + static_cast<int64_t>(n - 1) * stride >= p.ctas ||
      (a.z & ~1) || q0 < 0 || m < 0 ||
      m >= MTP_LATENT_MAX_NODES * MTP_LATENT_MAX_HEADS / N || b.y <= 0 || b.y > N ||
      q0 > p.total_q - 1 - (m * N + b.y - 1) / p.heads)
    return;
  if (rows <= 0) return;
  auto slot_of = [&](int i) -> int64_t { return 2 * (first + i * stride) + (i == 0 ? a.z : 0); };
  const int in = tid % kSide, d4 = blockIdx.z * kSide + in, g = tid / kSide;
  const int mine = kSplit ? 0 : g * kRows;             // first row of this thread's
  const float4* src = reinterpret_cast<const float4*>(p.o_part) + (r0 + mine) * (kDim / 4) + d4;
  const int step = kSplit ? kGroups : 1;
  float4 x[kAhead][kRows];
  auto load = [&](int i0) {                            // pieces i0, i0 + step, ...
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
#pragma unroll
      for (int r = 0; r < kRows; ++r)
        if (i0 + j * step < n && mine + r < rows)
          x[j][r] = __ldcg(src + slot_of(i0 + j * step) * (N * kDim / 4) + r * (kDim / 4));
  };
  load(kSplit ? g : 0);                                // (on their way while the weights are worked out)
  // ---- the pieces' weights: a warp a row
#pragma unroll 1
  for (int r = warp; r < rows; r += kThreads / 32) {
    float ref[kMaxCtas / 32], sum[kMaxCtas / 32], top = -INFINITY;
    bool bad = false;
#pragma unroll
    for (int k = 0; k < kMaxCtas / 32; ++k) {
      const int i = lane + 32 * k;
      float2 y = make_float2(kNoRef, 0.f);
      if (i < n) y = __ldcg(p.sum_part + slot_of(i) * N + r0 + r);
      ref[k] = y.x;
      sum[k] = y.y;
      bad |= __float_as_uint(y.y) == kBadSum;
      top = fmaxf(top, y.x);
    }
    top = warp_max(top);
    bad = __any_sync(0xffffffffu, bad);
    float total = 0.f;
#pragma unroll
    for (int k = 0; k < kMaxCtas / 32; ++k) {
      const int i = lane + 32 * k;
      if (i >= n) continue;
      const float w = ref[k] == kNoRef ? 0.f : exp2_hw(ref[k] - top);   // (nothing seen: sum 0, or NaN)
      s_w[r][i] = w;
      total += w * sum[k];
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (lane == 0) s_inv[r] = bad || total == 0.f ? 0.f : *p.descale / total;
  }
  __syncthreads();
  // ---- their sum
  float4 acc[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) acc[r] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int i0 = kSplit ? g : 0; i0 < n;) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
#pragma unroll
      for (int r = 0; r < kRows; ++r)
        if (i0 + j * step < n && mine + r < rows) {
          const float w = s_w[mine + r][i0 + j * step];
          acc[r].x = fmaf(w, x[j][r].x, acc[r].x);
          acc[r].y = fmaf(w, x[j][r].y, acc[r].y);
          acc[r].z = fmaf(w, x[j][r].z, acc[r].z);
          acc[r].w = fmaf(w, x[j][r].w, acc[r].w);
        }
    i0 += kAhead * step;
    if (i0 < n) load(i0);
  }
  if constexpr (kSplit) {
    if (g > 0)
#pragma unroll
      for (int r = 0; r < kRows; ++r) s_acc[g - 1][r][in] = acc[r];
    __syncthreads();
    if (g > 0) return;
#pragma unroll
    for (int o = 0; o < kGroups - 1; ++o)
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const float4 y = s_acc[o][r][in];
        acc[r].x += y.x;
        acc[r].y += y.y;
        acc[r].z += y.z;
        acc[r].w += y.w;
      }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (mine + r >= rows) continue;
    const float inv = s_inv[mine + r];
    if (inv == 0.f) acc[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    const __nv_bfloat162 u = __floats2bfloat162_rn(acc[r].x * inv, acc[r].y * inv);
    const __nv_bfloat162 v = __floats2bfloat162_rn(acc[r].z * inv, acc[r].w * inv);
    const int rr = m * N + r0 + mine + r, tok = rr / p.heads;
    reinterpret_cast<uint2*>(p.out + static_cast<int64_t>(q0 + tok) * p.out_stride_tok +
                             static_cast<int64_t>(rr - tok * p.heads) * p.out_stride_head)[d4] =
        make_uint2(*reinterpret_cast<const uint32_t*>(&u), *reinterpret_cast<const uint32_t*>(&v));
  }
}

// ---- host side -----------------------------------------------------------------------------------

int64_t units_bound(int32_t num_seqs, int32_t total_q, int32_t heads, int rows) {
  return static_cast<int64_t>(total_q) * heads / rows + num_seqs;
}
int64_t line_bound(int64_t units, int32_t max_pages) {
  return units * ((max_pages + kTilePages - 1) / kTilePages + kUnitTiles);
}
// Rows of a unit: as many columns of the products as an average sequence fills.  But 16, whose Q, sums and output
// take 6 us less than those of 64, while then no CTA has more than kFewTiles tiles of a table's length (4 tokens of
// 16 heads over 300 keys 17.3 -> 10.3 us, over 20000 21.3 -> 18.2; above it, over 50000, 16 rows would take 27.2
// instead of 24.4, and 20 x 2000 keys with 1 token of 128 heads 39.8 instead of 29.0).  A table's length, not the
// sequences', which the host does not know: in one of 8192 pages 300 keys take 18.7.
int unit_rows(int32_t num_seqs, int32_t total_q, int32_t heads, int32_t max_pages, int64_t ctas) {
  const int64_t rows = (static_cast<int64_t>(total_q) * heads + num_seqs - 1) / std::max(num_seqs, 1);
  const int64_t tiles = (max_pages + kTilePages - 1) / kTilePages;
  if (rows <= 16 || units_bound(num_seqs, total_q, heads, 16) * tiles <= kFewTiles * ctas) return 16;
  return rows <= 32 ? 32 : 64;
}
size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// The workspace's parts.
struct Parts {
  int rows;
  int64_t units, ctas;
  size_t o, sums, notes, total;        // bytes of partial outputs, sums, notes; of all and the units' number
};
bool parts_of(int32_t num_seqs, int32_t total_q, int32_t heads, int32_t max_pages, int sms, Parts* w) {
  w->rows = unit_rows(num_seqs, total_q, heads, max_pages, std::min(sms, kMaxCtas));
  w->units = units_bound(num_seqs, total_q, heads, w->rows);
  const int64_t line = line_bound(w->units, max_pages);
  if (line > INT32_MAX) return false;
  w->ctas = std::min<int64_t>(std::min(sms, kMaxCtas), line);
  w->o = align256(static_cast<size_t>(w->ctas) * 2 * w->rows * kDim * sizeof(float));
  w->sums = align256(static_cast<size_t>(w->ctas) * 2 * w->rows * sizeof(float2));
  w->notes = align256(static_cast<size_t>(w->units) * sizeof(JoinNote));
  // What a call asks for grows with its arguments, whatever its units' rows are: a workspace made for the largest
  // batch does for the smaller ones.
  const size_t slots = static_cast<size_t>(std::min(sms, kMaxCtas)) * 2 * 64;
  w->total = align256(slots * kDim * sizeof(float)) + align256(slots * sizeof(float2)) +
             align256(static_cast<size_t>(units_bound(num_seqs, total_q, heads, 16)) * sizeof(JoinNote)) + 256;
  return true;
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      return static_cast<EncodeFn>(nullptr);
    }
    return reinterpret_cast<EncodeFn>(f);
  }();
  return fn;
}
// A page as slices of 64 dims of its keys; a box is all slices of 8 keys.
bool encode_map(CUtensorMap* map, const void* cache, int64_t num_pages) {
  const EncodeFn encode = encode_fn();
  if (!encode) return false;
  const cuuint64_t dims[4] = {64, kPage, kSlices, static_cast<cuuint64_t>(num_pages)}, strides[3] = {kRow, 64, kRow * kPage};
  const cuuint32_t box[4] = {64, 8, kSlices, 1}, step[4] = {1, 1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(cache), dims, strides, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_pdl(const void* kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, LatentParams& p) {
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
  const cudaError_t e = cudaLaunchKernelExC(&cfg, kernel, args);
  if (e != cudaSuccess) cudaGetLastError();
  return e;
}

template <int N>
int launch_latent(LatentParams& p, int device, cudaStream_t stream) {
  static std::atomic<bool> allowed[64];              // per device; setting it twice is harmless
  const void* kernel = reinterpret_cast<const void*>(latent_attn_kernel<N>);
  if (!allowed[device].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<N>()) != cudaSuccess) {
      cudaGetLastError();
      return MTPATTN_E_LAUNCH;
    }
    cudaFuncAttributes attr;
    if (cudaFuncGetAttributes(&attr, kernel) != cudaSuccess || attr.numRegs != kLaunchRegisters) {
      cudaGetLastError();
      return MTPATTN_E_LAUNCH;
    }
    allowed[device].store(true, std::memory_order_release);
  }
  if (launch_pdl(kernel, dim3(p.ctas), kLatentThreads, smem_bytes<N>(), stream, p) != cudaSuccess) return MTPATTN_E_LAUNCH;
  if (p.whole) return MTPATTN_OK;
  // Few rows in many pieces are joined by 4 CTAs for each 2 rows (4 tokens of 16 heads over 50000 keys 41.0 -> 24.4 us, 1
  // token over 105000 29.4 -> 21.5), where at most 16 pieces cost 0.1 to 0.4 us more so (1 x 700 10.4 against 10.8).
  const bool one = p.unit_bound * N <= 320 && p.max_pages > 16 * kTilePages, few = p.unit_bound <= 32;
  const void* join = one   ? reinterpret_cast<const void*>(latent_join_kernel<N, 2, 128, 8, true, 8>)
                     : few ? reinterpret_cast<const void*>(latent_join_kernel<N, 2, 512, 2, true, 4>)
                           : reinterpret_cast<const void*>(latent_join_kernel<N, 4, 512, 2, false, 2>);
  return launch_pdl(join, dim3(p.unit_bound, N / (few ? 2 : 8), one ? 4 : 1), 256, 0, stream, p) == cudaSuccess
             ? MTPATTN_OK
             : MTPATTN_E_LAUNCH;
}

}  // namespace
}  // namespace mtpattn

using namespace mtpattn;

extern "C" size_t mtp_latent_attn_workspace_size(int32_t num_seqs, int32_t total_q, int32_t num_heads,
                                                 int32_t max_pages_per_seq) {
  if (num_seqs < 0 || total_q < 0 || num_heads <= 0 || num_heads > MTP_LATENT_MAX_HEADS || max_pages_per_seq < 0)
    return 0;
  const int sms = device_sm_count(-1);
  Parts w;
  return sms > 0 && parts_of(num_seqs, total_q, num_heads, max_pages_per_seq, sms, &w) ? w.total : 0;
}

extern "C" int mtp_latent_attn_fwd(const void* q, int64_t q_stride_tok, int64_t q_stride_head,
                                   const void* cache, int64_t num_pages, const int32_t* block_tables,
                                   int32_t max_pages_per_seq, const int32_t* seq_lens,
                                   const int32_t* cu_seqlens_q, const uint64_t* tree_mask, int32_t num_seqs,
                                   int32_t total_q, int32_t num_heads, const float* descale,
                                   float softmax_scale, void* workspace, size_t workspace_bytes, void* out,
                                   int64_t out_stride_tok, int64_t out_stride_head, int32_t* status,
                                   void* stream) {
  // 1. plain argument checks
  if (num_seqs < 0 || total_q < 0 || num_pages < 0 || max_pages_per_seq < 0 || num_heads <= 0)
    return MTPATTN_E_ARG;
  if (num_seqs == 0) return total_q == 0 ? MTPATTN_OK : MTPATTN_E_ARG;
  if (total_q < num_seqs) return MTPATTN_E_ARG;          // every sequence has a new token
  if (!q || !cache || !block_tables || !seq_lens || !cu_seqlens_q || !descale || !out || num_pages == 0 ||
      max_pages_per_seq == 0)
    return MTPATTN_E_ARG;
  if (!isfinite(softmax_scale)) return MTPATTN_E_ARG;
  if (q_stride_tok <= 0 || q_stride_head <= 0 || out_stride_tok <= 0 || out_stride_head <= 0 ||
      (q_stride_tok | q_stride_head | out_stride_tok | out_stride_head) % 8 != 0)
    return MTPATTN_E_ARG;
  if (!ptr_aligned(q, 16) || !ptr_aligned(out, 16) || !ptr_aligned(cache, 16) || !ptr_aligned(block_tables, 4) ||
      !ptr_aligned(seq_lens, 4) || !ptr_aligned(cu_seqlens_q, 4) || !ptr_aligned(tree_mask, 8) ||
      !ptr_aligned(descale, 4) || !ptr_aligned(status, 4))
    return MTPATTN_E_ARG;
  // 2. the supported envelope
  if (num_heads > MTP_LATENT_MAX_HEADS || total_q > static_cast<int64_t>(num_seqs) * MTP_LATENT_MAX_NODES ||
      num_pages > INT32_MAX || max_pages_per_seq > INT32_MAX / kPage - kTilePages)
    return MTPATTN_E_UNSUPPORTED;
  // 3. the workspace
  const int device = current_device();
  if (device < 0 || device >= 64) return MTPATTN_E_DEVICE;
  const int sms = device_sm_count(device);
  if (sms <= 0) return MTPATTN_E_DEVICE;
  Parts w;
  if (!parts_of(num_seqs, total_q, num_heads, max_pages_per_seq, sms, &w)) return MTPATTN_E_UNSUPPORTED;
  if (!workspace || !ptr_aligned(workspace, 256) || workspace_bytes < w.total) return MTPATTN_E_WORKSPACE;
  // 4. every pointer must be memory the kernels can read on the current device
  const void* const ptrs[] = {q, cache, block_tables, seq_lens, cu_seqlens_q, descale, workspace, out};
  if (!all_on_device(ptrs, device) || (tree_mask && !ptr_on_device(tree_mask, device)) ||
      (status && !ptr_on_device(status, device)))
    return MTPATTN_E_DEVICE;
  LatentParams p{};
  if (!encode_map(&p.tmap, cache, num_pages)) return MTPATTN_E_LAUNCH;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_stride_tok = q_stride_tok;
  p.q_stride_head = q_stride_head;
  p.cache = static_cast<const uint8_t*>(cache);
  p.num_pages = num_pages;
  p.block_tables = block_tables;
  p.max_pages = max_pages_per_seq;
  p.seq_lens = seq_lens;
  p.cu_q = cu_seqlens_q;
  p.mask = tree_mask;
  p.num_seqs = num_seqs;
  p.total_q = total_q;
  p.heads = num_heads;
  p.descale = descale;
  p.scale_log2 = softmax_scale * kLog2e;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.out_stride_tok = out_stride_tok;
  p.out_stride_head = out_stride_head;
  p.status = status;
  p.ctas = static_cast<int32_t>(w.ctas);
  char* ws = static_cast<char*>(workspace);
  p.o_part = reinterpret_cast<float*>(ws);
  p.sum_part = reinterpret_cast<float2*>(ws + w.o);
  p.notes = reinterpret_cast<JoinNote*>(ws + w.o + w.sums);
  p.units = reinterpret_cast<int32_t*>(ws + w.o + w.sums + w.notes);
  p.unit_bound = static_cast<int32_t>(w.units);
  p.whole = max_pages_per_seq <= kWholeTiles * kTilePages;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return w.rows == 16 ? launch_latent<16>(p, device, st)
         : w.rows == 32 ? launch_latent<32>(p, device, st)
                        : launch_latent<64>(p, device, st);
}
