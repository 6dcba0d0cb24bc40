// prefill_paged.cu -- attention of the last `rows` tokens of every sequence over
// a paged cache of 16 or 4 bits that holds them and all tokens before: a prompt's next
// chunk, or drafted tokens to check, for sequences of different lengths in one call.
//
//   o_i = sum_j exp(scale q_i.k_j - lse_i) v_j,  lse_i = log sum_j exp(scale q_i.k_j)
//
// over the keys j <= position of i (causal), or all of the sequence's keys.  One pass
// over the keys with the running maximum (moved only when it rises by more than 2^8, as
// in the forward over contiguous tensors) and sum in fp32.
//
// Work.  A unit is a block of query tokens of one sequence and KV head: NT tiles
// ("H", "L") of 128 rows, whose rows are tokens and, for each, the query heads of
// the KV head (up to hb of them), so that a key tile serves all of them and a
// short chunk still fills rows.  Its key axis has tiles of 128 keys.
//
// Division.  (a) The list of all units' key tiles (order: sequence, head, block of
// tokens, tile) is cut into equal runs, one for each CTA (one an SM), whatever the
// lengths are.  A run covers whole units, which the CTA finishes itself, and at its two
// ends parts of units, whose states (m, l, o) it leaves in the workspace; a second
// kernel folds those and writes the zeros of padding rows.  Every CTA finds its run from
// the lengths, so the host knows none, and results repeat bitwise.  (b) Where equal
// numbers of whole units take hardly longer than equal runs (kSplitCost), CTAs get
// those.  (c) Where the page table has room for few key tiles (launch_t), a cluster of 1
// to 8 CTAs takes each unit and folds its states through shared memory: no division, no
// workspace, no second kernel.
//
// A CTA works through its run without a stop between units: the loaders, the MMA
// issuers, the softmax warps and the guard walk the same list of segments each at
// its own pace.
//
// Warp roles: warps 0-3 (4-7) softmax, correction and epilogue of tile H (L),
// thread = row; lane 0 of two warps issues MMAs (two tiles: one each; one tile: one the
// products with K, the other those with V); over 16 bits a warp that loads (lane = one
// box of a page) and one that guards V; over 4 bits two warps that load (K, V) and four
// or eight that convert codes and factors into fp16 tiles, exactly.
//
// Tensor memory (512 columns): two tiles: S_H, S_L, O_H, O_L and, at d = 64, P_H, P_L
// (at d = 128 P goes through shared memory).  One tile: two places each of S and P,
// and O.
//
// The guard (16 bits; codes of 4 bits and their factors are finite).  A key that a row
// does not see has weight 0, but 0 times a NaN or an infinity in its row of V would be
// NaN.  Tiles with keys that some row does not see (the diagonal's, and the sequence's
// last) therefore pass through a warp which zeroes the rows of V behind the sequence,
// zeroes what is not finite in the rows that some query token sees and others do not,
// and notes for each column the first such key; rows that see it get NaN there at the
// end.  The score of a key that a row does not see becomes -inf, whatever it was.
//
// Fewer bits than fp32: the weights are rounded to the cache's 16-bit type for P.V (as in
// the forward over contiguous tensors; tensor cores take both operands in 16 bits, and a
// second term, which the decode keeps, would be a second product with V), over 4 bits to
// fp16, which 2^-11 keeps below the codes' own spacing (in fp16 a weight below 2^-14 is off
// by up to 2^-25); bf16 queries over 4 bits become fp16 behind a power of two a row.  The sum
// of weights, the maximum, O and what is folded stay fp32.
//
// Measured (us among other calls, and in brackets the floor at the same lengths, from the
// copy rate and the dense bf16 rate; 32 query heads on 8, d = 128, pages of 64):
//   bound by the tensor pipe and the softmax's chain: 4096 tokens of 32768 1346 to 1394
//   (1065; 1479 to 1531 TFLOP/s), 1500 to 2048 tokens of 4 sequences of 4096 to 16384 672
//   (478), over 4 bits 794; d = 64, 2048 of 4 sequences of 12000 728 (380), over 4 bits 859;
//   by the ends and starts of units: 4 x 4096 tokens from their start 491 (284), 500 of each
//   of 16 sequences of 1000 159 (51);
//   by HBM: 5 tokens of 64 sequences of 1024 to 32768 598 (604: reads alone go a little
//   faster than a copy, 6.85 TB/s); over 4 bits 443 (170) by the chains of products
//   into one accumulator, about 100 cycles each whatever their size, 16 a key tile;
//   by latency: 16 tokens of one sequence of 1000 10.5 (0.6), 9.5 of them on the device.
#include <cuda_runtime.h>

#include <cfloat>
#include <cstring>
#include <type_traits>

#include "gbattn_internal.h"
#include "gbattn_parts.h"
#include "gbattn_ptx.cuh"

namespace gbattn {
namespace {

constexpr int kBM = 128;          // rows of a tile (= TMEM lanes)
constexpr int kBN = 128;          // keys of a tile
constexpr int kMaxCtas = 160;     // bound of the grid, for the workspace's size
constexpr float kRescaleThreshold = 8.f;  // base-2 units
constexpr int kPBlock = 64;        // keys whose weights are stored together
constexpr int kBarBytes = 3 << 10;  // of Barriers
// A scale of scores is at least this, so that -inf times it stays -inf: fp32's smallest
// number, 2^-149.  (Rounding a scale to a multiple of it moves no score by more than 2^-150
// times fp32's largest, 2.4e-7.)
constexpr float kLeastScale = 1.4012985e-45f;
// Segments whose notes of the guard are kept: it is at most 3 ahead of every softmax
// warp.  It follows V, which is loaded behind Q; Q's places are loaded when every row tile
// has released the Q before: with its last product with K, at most two key tiles ahead of
// its softmax, or, a tile that visits no key, when each of its softmax warps gets there.
constexpr int kSegRing = 4;
// Key tiles that the states of split units cost (writing, and a second kernel that has
// to fold them) for units of one and two row tiles.  Whole units and runs, us in a
// captured graph: 3 tokens of 40 sequences of 2000 80, 70, over 4 bits 70, 64; 5 of 64 of
// 1024 to 32768 1042, 722, over 4 bits 830, 482.  The estimate takes every unit for as long
// as the longest, so prompts from their start and short ragged batches get runs where whole
// units would win: 2000 tokens of one prompt 67, 75; 3 of 40 of 400 to 1000, 4 bits, 53, 57.
template <int NT>
constexpr int kSplitCost = NT == 2 ? 6 : 4;
constexpr int kTileRing = 16;     // key tiles whose missing pages are kept

// COPIES: with one tile and few rows, the tile holds the rows two or four times, and
// each copy's warps take another part of the keys (the other weights of their rows
// stay 0): the softmax of a tile, which otherwise waits for one or two of the four
// warps, takes a half or a quarter of the time.  The copies are folded at a segment's
// end.  5 tokens of 64 sequences (20 rows), with and without: 4 bits 481, 757 us, 16 bits
// at d = 64 378, 494; at d = 128 in 16 bits HBM bounds both.
template <int D, int NT, bool FP4, int COPIES>
struct Cfg {
  static_assert(NT == 1 || COPIES == 1, "copies are of one tile");
  static constexpr int kDim = D;
  static constexpr int kRows = kBM / COPIES;  // of a copy
  static constexpr int kCols = kBN / COPIES;  // keys of a copy
  // Tensor memory has room for P unless there are two tiles of d = 128.
  static constexpr bool kPInTmem = D == 64 || NT == 1;
  // With one tile S and P have two places each in turn, and one thread issues the
  // products with K, another those with V.  A chain of products into one place takes
  // about 100 cycles each whatever their size is, and a softmax that had to wait for
  // the end of one before it could hand over the next P would wait most of its time
  // (two tiles do each other's waiting).
  static constexpr int kSBufs = NT == 1 ? 2 : 1;
  static constexpr int kSCol = 0, kOCol = 2 * kBN, kPCol = kOCol + NT * D;
  // Where tile x's S number d goes, and its barriers.
  __device__ static __forceinline__ int s_bar(int x, int d) { return NT == 1 ? d & 1 : x; }
  static constexpr int kColBlocks = D / 64;
  static constexpr int kTileBytes = kBM * D * 2;
  static constexpr int kBlockBytes = kBM * 128;
  // Where an output waits for its store: P's place, or one of its own.  One tile over 4
  // bits has none, threads store their rows: shared memory holds more key tiles instead.
  // Copies are folded there, 32 columns at a time, by threads that store the sums.
  static constexpr bool kDirectO = NT == 1 && (FP4 || COPIES > 1);
  static constexpr int kStageBytes = COPIES > 1 ? kBM * 32 * 4 : kDirectO ? 0 : kPInTmem ? kTileBytes : kBM * kBN * 2;
  static constexpr int kQBytes = kTileBytes;
  // 16-bit key and value tiles; of a 4-bit cache's rows, what comes from memory and
  // what the conversion makes of it.
  static constexpr int kStages = FP4 ? (NT == 2 ? (D == 128 ? 2 : 6) : (D == 128 ? 4 : 8))
                                     : (NT == 2 ? (D == 128 ? 3 : 8) : (D == 128 ? 5 : 12));
  static constexpr int kRawStages = !FP4 ? 0 : NT == 2 ? (D == 128 ? 3 : 8) : (D == 128 ? 5 : 12);
  // With two tiles over 16 bits everyone takes every key and value tile in the order of
  // their loads, so all places form one ring.  Otherwise keys and values have issuers
  // or converting warps of their own, each at its own pace, and a ring each: a wait
  // tells only even from odd rounds of a place, so whoever waits has to follow all of
  // its rounds.
  static constexpr bool kOneRing = NT == 2 && !FP4;
  static constexpr int kKStages = kOneRing ? kStages : kStages / 2;   // K's places, [0, kKStages)
  static constexpr int kRawKStages = FP4 ? (kRawStages + 1) / 2 : 0;  // the same of codes and factors
  static_assert(kRawKStages <= 12 && kRawStages <= 12 && kStages <= 12, "barriers");
  static constexpr int kRawBytes = kBN * (D / 2 + D / 16);  // codes, then factors
  static constexpr int kQOff = 0;
  static constexpr int kPOff = NT * kQBytes;
  static constexpr int kRingOff = kPOff + NT * kStageBytes;
  static constexpr int kRawOff = kRingOff + kStages * kTileBytes;
  static constexpr int kBarOff = kRawOff + kRawStages * kRawBytes;
  static constexpr int kSmemBytes = kBarOff + kBarBytes;
  static constexpr int kMmaWarp = 4 * NT;  // tile x's issuer is warp kMmaWarp + x
  static constexpr int kLoadWarp = 4 * NT + 2;
  static constexpr int kGuardWarp = 4 * NT + 3;
  static constexpr int kConvertWarp = 4 * NT + 4;  // the first of kConvertWarps
  static constexpr int kConvertWarps = FP4 ? (NT == 2 ? 4 : 8) : 0;
  static constexpr int kThreads = 128 * (NT + 1) + 32 * kConvertWarps;
  // Registers a thread: at launch, and after the warpgroups have divided them (not
  // with one tile over 16 bits, where there are enough).  One tile over 4 bits, softmax /
  // control / conversion: 240/64/104 423 us (5 tokens of 64 sequences), 208/64/120 431,
  // 160/96/128 and 224/64/112 more.
  static constexpr bool kSplit = FP4 || NT == 2;
  static constexpr int kLaunchRegs = FP4 ? 128 : 168;
  static constexpr int kSoftmaxRegs = FP4 ? (NT == 2 ? 192 : 240) : 216;
  static constexpr int kControlRegs = FP4 ? 64 : 72;
  static constexpr int kConvertRegs = NT == 2 ? 64 : 104;
  static_assert(!kSplit || NT * 128 * kSoftmaxRegs + 128 * kControlRegs + 32 * kConvertWarps * kConvertRegs <=
                               kThreads * kLaunchRegs,
                "register split");
  static_assert(!kSplit || (kSoftmaxRegs >= kLaunchRegs && kControlRegs <= kLaunchRegs && kConvertRegs <= kLaunchRegs),
                "the softmax's registers rise, the others' fall");
};

struct Params {
  CUtensorMap tq, to, tk, tv;   // (no tk, tv for a 4-bit cache)
  const uint8_t* codes[2];
  const uint8_t* factors[2];
  const float* descale[2];
  const int* page_table;
  const int* seqlens;
  const int* new_lens;
  void* o;
  float* lse;
  float* part_o;   // [ctas][2][D / 4][NT * 128][4]
  float2* part_ml; // [ctas][2][NT * 128]: m in base-2 units, l
  int2* parts;     // [B][heads][blocks]: first CTA, number of parts (1: finished)
  int B, H, Hkv, S, g;
  int hb_inverse;  // 65536 / hb rounded up: row / hb = row * hb_inverse >> 16 for the 128 rows of a tile
  int hb, tq_tokens, nblk, heads, blocks;  // heads a tile; tokens a tile; head blocks; Hkv * nblk; token blocks of S
  int page_shift, n_pages, max_pages, box_rows;
  int causal;
  int out_bf16;
  float scale_log2;  // |scale| log2 e, at least kLeastScale
  double scale64;    // the same, where fp32's normal numbers do not have it in 64 bits
  float sign;        // -1 or 0 where scale is negative or 0, and scores are taken times it
  int ctas;
  int wide;          // whether tiles may count past 2^31
  int cluster;       // CTAs of each unit, which fold their states themselves; 0: runs of the list
  int* status;
};

// A sequence: cached tokens, position of query row 0 (negative: the first -p0 rows
// are padding), query rows.
struct Seq {
  int n, p0, rows;
};

struct __align__(8) Barriers {
  uint64_t q_full, q_empty;
  uint64_t q_ready[2];     // queries converted to fp16 (bf16 over 4 bits)
  uint64_t raw_empty[12];  // 4 bits: codes and factors converted (raw: copied)
  uint64_t kv_full[12], kv_empty[12], raw[12];
  uint64_t s_full[2], s_free[2], p_full[2], p_free[2], o_full[2], mma_done[2];
  uint64_t group[2];       // the four warps of a softmax warpgroup
  uint64_t stagger;
  long long per;           // tiles of a run
  long long start_left;    // tiles of this run, or (per = 0) its units
  int start[4];            // its first unit (sequence, head, block) and tile
  Seq start_seq;
  long long scan[16];      // of the warps: tiles,
  long long scan_units[16];  // units that have any,
  int scan_most[16];         // and the most tiles of a unit
  float state[kBM];        // of the rows, with clusters: log2 of the sum of weights
  uint32_t tmem_base;
  int abort_flag;
  uint32_t walk[8][24];    // each softmax warp's cursor and segment while it goes over the keys
  uint8_t bad[2][kTileRing];       // 16-key blocks of a tile (of K, of V) that have no page
  uint8_t nan_any[kSegRing];
  uint8_t nan_from[kSegRing][128]; // column's first non-finite key behind the first row's last key, - 1
};
static_assert(sizeof(Barriers) <= kBarBytes, "barriers fit");

__device__ __forceinline__ Seq load_seq(const Params& p, int b) {
  Seq s;
  const int len = max(p.seqlens[b], 0);
  s.rows = p.new_lens != nullptr ? min(max(p.new_lens[b], 0), p.S) : p.S;
  s.p0 = len - s.rows;
  s.n = min(len, p.max_pages << p.page_shift);
  return s;
}
// Last key that query token t sees (t >= -p0).
__device__ __forceinline__ int limit(const Params& p, const Seq& s, int t) {
  return p.causal ? min(s.p0 + t, s.n - 1) : s.n - 1;
}
// Key tiles that the query tokens [t0, t1) visit.
__device__ __forceinline__ int tiles_of(const Params& p, const Seq& s, int t0, int t1) {
  const int last = min(t1, s.rows) - 1;
  if (last < t0 || s.p0 + last < 0) return 0;
  return limit(p, s, last) / kBN + 1;
}
// Units of a head with any tile, and the most tiles of one: the last one's.
template <int NT>
__device__ __forceinline__ int seq_units(const Params& p, const Seq& s) {
  const int tu = NT * p.tq_tokens;
  return s.rows > 0 && s.p0 + s.rows > 0 ? (s.rows + tu - 1) / tu - max(-s.p0, 0) / tu : 0;
}
__device__ __forceinline__ int most_tiles(const Params& p, const Seq& s) {
  return s.rows > 0 && s.p0 + s.rows > 0 ? limit(p, s, s.rows - 1) / kBN + 1 : 0;
}
template <int NT>
__device__ __forceinline__ long long seq_tiles(const Params& p, const Seq& s) {
  const int tu = NT * p.tq_tokens;
  if (!p.causal) {  // all blocks but those of padding alone
    const int first = max(-s.p0, 0) / tu, end = (s.rows + tu - 1) / tu;
    return s.n > 0 && end > first ? static_cast<long long>(end - first) * ((s.n + kBN - 1) / kBN) : 0;
  }
  long long sum = 0;
  for (int t = 0; t < s.rows; t += tu) sum += tiles_of(p, s, t, t + tu);
  return sum;
}

// A run of key tiles of one unit.
struct Seg {
  Seq s;
  int b, u, k;
  int nt;      // tiles of the unit
  int j0, j1;  // the segment's
  __device__ __forceinline__ bool whole() const { return j0 == 0 && j1 == nt; }
};

// Walks over the segments of a CTA's run.
template <int NT>
struct Cursor {
  Seq s;
  int b, u, k, y;
  bool units;      // `left` counts units, which are whole
  long long left;
  __device__ __forceinline__ void start(const Params& p, const Barriers* bars) {
    b = bars->start[0], u = bars->start[1], k = bars->start[2], y = bars->start[3];
    left = bars->start_left;
    units = bars->per == 0;
    s = bars->start_seq;
  }
  // The tiles [j0, j1) of one unit.
  __device__ __forceinline__ void start(const Seg& seg) {
    s = seg.s, b = seg.b, u = seg.u, k = seg.k, y = seg.j0;
    units = false;
    left = seg.j1 - seg.j0;
  }
  __device__ __forceinline__ bool next(const Params& p, Seg& seg) {
    if (left <= 0) return false;
    const int tu = NT * p.tq_tokens;
    int nt = tiles_of(p, s, k * tu, (k + 1) * tu);
    while (nt == 0) {
      if (!advance(p, tu)) return false;
      nt = tiles_of(p, s, k * tu, (k + 1) * tu);
    }
    seg.s = s;
    seg.b = b, seg.u = u, seg.k = k, seg.nt = nt, seg.j0 = y;
    seg.j1 = units ? nt : static_cast<int>(min(static_cast<long long>(nt), y + left));
    left -= units ? 1 : seg.j1 - seg.j0;
    y = 0;
    if (left > 0) advance(p, tu);
    return true;
  }
  __device__ __forceinline__ bool advance(const Params& p, int tu) {
    if ((++k) * tu < s.rows) return true;
    k = 0;
    if (s.rows > 0 && ++u < p.heads) return true;
    u = 0;
    if (++b >= p.B) return false;
    s = load_seq(p, b);
    return true;
  }
};

// The query token and head of a tile's row.
__device__ __forceinline__ int token_of(const Params& p, int row) { return row * p.hb_inverse >> 16; }

// KV head and first query head (of the KV head's) of a unit.
__device__ __forceinline__ int kv_head(const Params& p, int u) { return p.nblk == 1 ? u : u / p.nblk; }
__device__ __forceinline__ int first_head(const Params& p, int u) { return p.nblk == 1 ? 0 : u % p.nblk * p.hb; }

// What tile x of a segment's unit is.
struct TileRows {
  int t0;       // first token
  int j1;       // visits the segment's tiles [seg.j0, j1)
  int lim_min;  // last key that all of its real rows see
  __device__ __forceinline__ TileRows(const Params& p, const Seg& seg, int x, int nt_tiles) {
    t0 = (seg.k * nt_tiles + x) * p.tq_tokens;
    const int nt = tiles_of(p, seg.s, t0, t0 + p.tq_tokens);
    j1 = max(seg.j0, min(seg.j1, nt));
    lim_min = nt > 0 ? limit(p, seg.s, max(t0, -seg.s.p0)) : 0;
  }
};

// The first tile of the unit with keys that some real row does not see.
template <int NT>
__device__ __forceinline__ int first_masked(const Params& p, const Seg& seg, int& lim0) {
  lim0 = limit(p, seg.s, max(seg.k * NT * p.tq_tokens, -seg.s.p0));
  return (lim0 + 1) / kBN;
}

// The places [FIRST, END) of a ring in turn: the current one and its round.  A place is
// filled in its round for the (round)th time; in round 0 there is nothing to wait for.
template <int FIRST, int END>
struct Ring {
  int st = FIRST;
  uint32_t round = 0;
  __device__ __forceinline__ uint32_t phase() const { return round & 1u; }
  __device__ __forceinline__ void next() {
    if (END - FIRST == 1 || ++st == END) {
      st = FIRST;
      ++round;
    }
  }
};

// Position of V_j among a segment's loads K_0, K_1, V_0, K_2, V_1, .., K_{n-1},
// V_{n-2}, V_{n-1}.
__device__ __forceinline__ int item_of_v(int j, int n) { return j <= n - 2 ? 2 * j + 2 : 2 * n - 1; }

// Divides the list: every CTA sums all sequences' tiles (plan_sum, then a barrier),
// then the thread whose share of the sequences holds the CTA's first tile finds it
// (plan_find, and another barrier).
template <typename T>  // int, or long long where tiles may count past 2^31
struct Plan {
  Seq s;            // the thread's first sequence
  int b0, b1;       // its share
  T tiles, tiles_to;  // of the share; of all up to its end within the warp
  T units, units_to;
};
template <typename C, int NT, typename T>
__device__ __forceinline__ void plan_sum(const Params& p, Barriers* bars, Plan<T>& plan) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int each = (p.B + C::kThreads - 1) / C::kThreads;
  plan.b0 = min(p.B, static_cast<int>(threadIdx.x) * each), plan.b1 = min(p.B, plan.b0 + each);
  plan.tiles = plan.units = 0;
  int most = 0;
  for (int b = plan.b0; b < plan.b1; ++b) {
    const Seq s = load_seq(p, b);
    if (b == plan.b0) plan.s = s;
    plan.tiles += static_cast<T>(seq_tiles<NT>(p, s));
    plan.units += seq_units<NT>(p, s);
    most = max(most, most_tiles(p, s));
  }
  plan.tiles *= p.heads;
  plan.units *= p.heads;
  plan.tiles_to = plan.tiles;
  plan.units_to = plan.units;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T v = __shfl_up_sync(0xffffffffu, plan.tiles_to, o);
    const T u = __shfl_up_sync(0xffffffffu, plan.units_to, o);
    if (lane >= o) plan.tiles_to += v, plan.units_to += u;
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 31) {
    bars->scan[warp] = plan.tiles_to;
    bars->scan_units[warp] = plan.units_to;
    bars->scan_most[warp] = most;
  }
}
template <typename C, int NT, typename T>
__device__ __forceinline__ bool plan_find(const Params& p, Barriers* bars, const Plan<T>& plan) {
  const int warp = threadIdx.x / 32;
  T tiles_before = plan.tiles_to - plan.tiles, units_before = plan.units_to - plan.units;
  T tiles = 0, units = 0;
  int most = 0;
#pragma unroll
  for (int w = 0; w < C::kThreads / 32; ++w) {
    if (w < warp) tiles_before += static_cast<T>(bars->scan[w]), units_before += static_cast<T>(bars->scan_units[w]);
    tiles += static_cast<T>(bars->scan[w]);
    units += static_cast<T>(bars->scan_units[w]);
    most = max(most, bars->scan_most[w]);
  }
  const T run = (tiles + p.ctas - 1) / p.ctas, run_units = (units + p.ctas - 1) / p.ctas;
  const bool whole = run_units * most <= run + kSplitCost<NT>;
  const T step = whole ? run_units : run, all = whole ? units : tiles;
  const T x0 = blockIdx.x * step;
  const T left = all > x0 ? min(step, all - x0) : 0;
  if (threadIdx.x == 0) {
    bars->per = whole ? 0 : run;
    bars->start_left = left;
  }
  const T before = whole ? units_before : tiles_before;
  if (left > 0 && x0 >= before && x0 < before + (whole ? plan.units : plan.tiles)) {
    T x = x0 - before;
    Seq s = plan.s;
    int b = plan.b0;
    T head = static_cast<T>(whole ? seq_units<NT>(p, s) : seq_tiles<NT>(p, s));
    while (x >= head * p.heads) {
      x -= head * p.heads;
      s = load_seq(p, ++b);
      head = static_cast<T>(whole ? seq_units<NT>(p, s) : seq_tiles<NT>(p, s));
    }
    const int u = static_cast<int>(x / head);
    x -= u * head;
    const int tu = NT * p.tq_tokens;
    int k = max(-s.p0, 0) / tu;  // the first block with a real row
    if (whole) {
      k += static_cast<int>(x);
      x = 0;
    } else {
      for (;; ++k) {
        const int nt = tiles_of(p, s, k * tu, (k + 1) * tu);
        if (x < nt) break;
        x -= nt;
      }
    }
    bars->start[0] = b, bars->start[1] = u, bars->start[2] = k, bars->start[3] = static_cast<int>(x);
    bars->start_seq = s;
  }
  return left > 0;
}

// The four pairs of E2M1 codes of a word as fp16 pairs, times a factor's fp16 pair:
// exact, 2 by 4 significant bits of at most 2688.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t f, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t.reg .b32 t0, t1, t2, t3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 t0, b0;\n\tcvt.rn.f16x2.e2m1x2 t1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 t2, b2;\n\tcvt.rn.f16x2.e2m1x2 t3, b3;\n\t"
      "mul.rn.f16x2 %0, t0, %5;\n\tmul.rn.f16x2 %1, t1, %5;\n\t"
      "mul.rn.f16x2 %2, t2, %5;\n\tmul.rn.f16x2 %3, t3, %5;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w), "r"(f));
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}

// Whether rows [r0, 128) of a V tile hold a NaN or an infinity, which 0 times it tells:
// one instruction for two elements.
template <bool BF16, int COL_BLOCKS>
__device__ __forceinline__ bool any_not_finite(const uint8_t* tile, int r0, int lane) {
  uint32_t acc = 0u;
  auto add = [&](uint32_t w) {
    if constexpr (BF16) asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(w), "r"(0u));
    else asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(w), "r"(0u));
  };
#pragma unroll
  for (int cb = 0; cb < COL_BLOCKS; ++cb) {
    const uint8_t* block = tile + cb * (kBM * 128);
#pragma unroll 8
    for (int at = r0 * 128 + lane * 16; at < kBM * 128; at += 512) {
      const uint4 v = *reinterpret_cast<const uint4*>(block + at);
      add(v.x), add(v.y), add(v.z), add(v.w);
    }
  }
  constexpr uint32_t kInf = BF16 ? 0x7F80u : 0x7C00u;
  return __any_sync(0xffffffffu, (acc & 0x7FFFu) > kInf || (acc >> 16 & 0x7FFFu) > kInf);
}

// Where the first 16-byte piece of a row's state's half with columns 4 c4, .. is: in the
// place of Q or in the one for outputs (4 bits: behind Q all the same, where the first
// keys were).
template <typename C>
__device__ __forceinline__ uint8_t* state_row(uint8_t* smem, int row, int c4) {
  constexpr int kHalf = C::kDim / 8;  // pieces of half a row
  return smem + (c4 < kHalf ? C::kQOff : C::kPOff) + row * (kHalf * 16);
}

// Two outputs from a row's sums and 1 / l: the products, but NaN where a sum is infinite.
// A value of V that is not finite makes its elements NaN, as in the decode, not an
// infinity or NaN by what its weight rounds to, whether the guard has noted it, or which
// copy or part of the row met it.
template <bool BF16>
__device__ __forceinline__ uint32_t normalised(float x, float y, float inv) {
  const float2 o = make_float2(x, y), r = ffma2(o, make_float2(inv, inv), fmul2(o, make_float2(0.f, 0.f)));
  return pack2<BF16>(r.x, r.y);
}

__device__ __forceinline__ float ld_cluster(uint32_t a) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

// The cluster's CTAs fold their states, a share of the unit's rows each, and write
// them; rows that count no key become zeros.  By the softmax threads, lanes along
// a row.
template <typename C, int D, bool BF16, int CTAS>
__device__ __forceinline__ void fold_cluster(const Params& p, const Seg& seg, uint8_t* smem, Barriers* bars) {
  constexpr int kItems = kBM / CTAS * (D / 4);  // pieces of four columns
  // Of a thread, requested together: one at a time waited for each trip to another SM.
  constexpr int kAtOnce = CTAS == 8 ? 2 : CTAS == 4 ? 4 : 8;
  const int rank = blockIdx.x % CTAS;
  const int kvh = kv_head(p, seg.u), head0 = first_head(p, seg.u);
  for (int i0 = threadIdx.x; i0 < kItems; i0 += kAtOnce * kBM) {
    float m[kAtOnce][CTAS];
    float4 o[kAtOnce][CTAS];
    long long hrow[kAtOnce];
#pragma unroll
    for (int v = 0; v < kAtOnce; ++v) {
      // (threads without a piece of their own read some)
      const int i = i0 + v * kBM;
      const int row = (i < kItems ? i / (D / 4) : 0) * CTAS + rank, c4 = i % (D / 4);  // every CTAS-th row
      const int row_token = token_of(p, row), head = head0 + row - row_token * p.hb;
      const int t = seg.k * p.tq_tokens + row_token;
      hrow[v] = i < kItems && row_token < p.tq_tokens && head < p.g && t < p.S
                    ? (static_cast<long long>(seg.b) * p.H + kvh * p.g + head) * p.S + t
                    : -1;
      const uint8_t* piece = state_row<C>(smem, row, c4) + ((c4 % (D / 8) ^ (row & 7)) << 4);
#pragma unroll
      for (int r = 0; r < CTAS; ++r) {
        m[v][r] = ld_cluster(mapa_shared(&bars->state[row], r));
        o[v][r] = ld_cluster4(mapa_shared(piece, r));
      }
    }
#pragma unroll
    for (int v = 0; v < kAtOnce; ++v) {
      if (hrow[v] < 0) continue;
      const int c4 = (i0 + v * kBM) % (D / 4);
      float M = -INFINITY, sum = 0.f;
#pragma unroll
      for (int r = 0; r < CTAS; ++r) M = fmaxf(M, m[v][r]);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int r = 0; r < CTAS; ++r) {
        if (m[v][r] == -INFINITY) continue;  // no key counts (and its O is not set)
        const float f = m[v][r] == M ? 1.f : ex2_approx(m[v][r] - M);
        sum += f;
        acc.x = fmaf(f, o[v][r].x, acc.x), acc.y = fmaf(f, o[v][r].y, acc.y);
        acc.z = fmaf(f, o[v][r].z, acc.z), acc.w = fmaf(f, o[v][r].w, acc.w);
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + hrow[v] * D + c4 * 4) =
          make_uint2(normalised<BF16>(acc.x, acc.y, inv), normalised<BF16>(acc.z, acc.w, inv));
      if (c4 == 0 && p.lse != nullptr)
        p.lse[hrow[v]] = sum == 0.f ? -INFINITY : (M + __log2f(sum)) * 0.69314718055994531f;
    }
  }
}

template <int D, bool BF16, int NT, bool FP4, int COPIES>
__global__ void __launch_bounds__(Cfg<D, NT, FP4, COPIES>::kThreads, 1)
    prefill_paged_kernel(const __grid_constant__ Params p) {
  using C = Cfg<D, NT, FP4, COPIES>;
  constexpr bool kMmaBf16 = BF16 && !FP4;  // over 4 bits all operands are fp16
  constexpr bool kReadyQ = BF16 && FP4;  // queries pass through the softmax warps
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem + C::kQOff;
  uint8_t* sP = smem + C::kPOff;
  uint8_t* sRing = smem + C::kRingOff;
  Barriers* bars = reinterpret_cast<Barriers*>(smem + C::kBarOff);
  volatile int* abort_flag = &bars->abort_flag;
  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;

  let_next_kernel_start();
  if ((smem_u32(smem) & 1023u) != 0) {  // the swizzle needs it; the same for all threads
    if (threadIdx.x == 0) atomicCAS(p.status, 0, kStatusSmemAlign);
    return;
  }
  if (threadIdx.x == 0) {
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->q_empty, NT == 1 ? 1 : 5 * NT);  // (of two tiles each: the issuer, and four for what has read Q)
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&bars->kv_full[s], FP4 ? 4 : 1);  // (the converting warps of a tile)
      mbar_init(&bars->kv_empty[s], NT);
      if (!FP4) mbar_init(&bars->raw[s], 1);
    }
    for (int s = 0; s < C::kRawStages; ++s) {
      mbar_init(&bars->raw[s], 1);
      mbar_init(&bars->raw_empty[s], 4);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bars->q_ready[x], kBM);
      mbar_init(&bars->s_full[x], 1);
      mbar_init(&bars->s_free[x], kBM);
      mbar_init(&bars->p_full[x], kBM);
      mbar_init(&bars->p_free[x], 1);
      mbar_init(&bars->o_full[x], 1);
      mbar_init(&bars->mma_done[x], 1);
      mbar_init(&bars->group[x], kBM);
    }
    mbar_init(&bars->stagger, kBM);
    bars->abort_flag = 0;
    fence_mbar_init();
    prefetch_tensormap(&p.tq);
    prefetch_tensormap(&p.to);
    if (!FP4) {
      prefetch_tensormap(&p.tk);
      prefetch_tensormap(&p.tv);
    }
  }
  wait_for_previous_kernel();
  Seg seg{};
  if (COPIES == 1 && p.cluster > 0) {
    // Grid (clusters of the token blocks, heads, sequences); sizes are powers of two.
    const int shift = 31 - __clz(p.cluster), rank = blockIdx.x & (p.cluster - 1);
    seg.k = blockIdx.x >> shift;
    seg.u = blockIdx.y;
    seg.b = blockIdx.z;
    seg.s = load_seq(p, seg.b);
    seg.nt = tiles_of(p, seg.s, seg.k * NT * p.tq_tokens, (seg.k + 1) * NT * p.tq_tokens);
    seg.j0 = seg.nt * rank >> shift;
    seg.j1 = seg.nt * (rank + 1) >> shift;
  } else {
    bool any;
    if (!p.wide) {
      Plan<int> plan;
      plan_sum<C, NT>(p, bars, plan);
      __syncthreads();
      any = plan_find<C, NT>(p, bars, plan);
    } else {
      Plan<long long> plan;
      plan_sum<C, NT>(p, bars, plan);
      __syncthreads();
      any = plan_find<C, NT>(p, bars, plan);
    }
    if (!any) return;  // fewer tiles than CTAs
  }
  if (warp == C::kMmaWarp) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  Cursor<NT> cur;
  if (COPIES == 1 && p.cluster > 0) cur.start(seg);
  else cur.start(p, bars);

  if (FP4 && warp >= C::kConvertWarp) {
    // ================================================================ conversion of 4 bits
    // A thread takes whole rows, 16 bytes of codes at a time: 32 elements, 4 pieces of
    // 16 bytes of the tile.  At d = 128 lanes of one eighth of a warp take their row's
    // pieces in different orders, so that neither reads (rows 64 bytes apart) nor writes
    // meet in a bank.  With one tile one half of the warps takes K, the other V, so that
    // two conversions are under way at once; with two tiles all four warps take both, in
    // the order of the loads: K's and V's one place each come free at different times.
    if constexpr (FP4) {
      regs_dec<C::kConvertRegs>();
      constexpr int kPieces = D / 32;
      const int team = NT == 2 ? 0 : (warp - C::kConvertWarp) / 4;  // NT = 1: V's warps
      const int row = threadIdx.x % kBN;
      // Within a row: where its pieces' first and further 16 bytes go.
      const uint32_t half = (row & 4) << 4, in0 = (row & 3) << 4;
      // (of the two pairs of rings, with one tile each half of the warps moves one)
      Ring<0, C::kRawKStages> raw_k;
      Ring<C::kRawKStages, C::kRawStages> raw_v;
      Ring<0, C::kKStages> at_k;
      Ring<C::kKStages, C::kStages> at_v;
      int tile0 = 0;
      bool ok = true;
      while (ok && cur.next(p, seg)) {
        const int n = seg.j1 - seg.j0;
        for (int i = 0; i < NT * n; ++i) {
          const bool is_v = NT == 2 ? i == 2 * n - 1 || (i > 0 && i % 2 == 0) : team == 1;
          const int j = NT == 1 ? i : i == 0 ? 0 : i == 2 * n - 1 ? n - 1 : (i & 1) ? (i + 1) / 2 : i / 2 - 1;
          const int raw = is_v ? raw_v.st : raw_k.st, at = is_v ? at_v.st : at_k.st;
          ok = bounded_wait(&bars->raw[raw], is_v ? raw_v.phase() : raw_k.phase(), abort_flag, p.status,
                            kStatusTimeoutLoad);
          const uint32_t round = is_v ? at_v.round : at_k.round;
          if (ok && round > 0)
            ok = bounded_wait(&bars->kv_empty[at], (round & 1u) ^ 1u, abort_flag, p.status, kStatusTimeoutLoad);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const uint8_t* src = smem + C::kRawOff + raw * C::kRawBytes;
          // Rows that are not there are zeros.
          const bool there = (seg.j0 + j) * kBN + row < seg.s.n &&
                             !(bars->bad[is_v][(tile0 + j) % kTileRing] >> (row / 16) & 1u);
          uint32_t f[D / 64];
          if constexpr (D == 128) {
            const uint2 v = *reinterpret_cast<const uint2*>(src + kBN * (D / 2) + row * (D / 16));
            f[0] = there ? v.x : 0u, f[1] = there ? v.y : 0u;
          } else {
            const uint32_t v = *reinterpret_cast<const uint32_t*>(src + kBN * (D / 2) + row * (D / 16));
            f[0] = there ? v : 0u;
          }
          uint8_t* dst = sRing + at * C::kTileBytes + row * 128;
#pragma unroll
          for (int q = 0; q < kPieces; ++q) {
            const uint32_t piece = D == 128 ? ((row >> 1) + q) % kPieces : q;
            const uint32_t fw = D == 128 && piece >= 2 ? f[D / 64 - 1] : f[0];
            const uint32_t two = e4m3x2_to_f16(piece & 1 ? fw >> 16 : fw);
            const uint32_t f0 = __byte_perm(two, two, 0x1010), f1 = __byte_perm(two, two, 0x3232);
            const uint4 codes = *reinterpret_cast<const uint4*>(src + row * (D / 2) + piece * 16);
            const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
            uint8_t* to = dst + (piece >> 1) * C::kBlockBytes + ((piece & 1) * 64 ^ half);
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k) {
              uint32_t h[4];
              e2m1x8_to_f16(w[k], k < 2 ? f0 : f1, h);
              *reinterpret_cast<uint4*>(to + (k * 16 ^ in0)) = make_uint4(h[0], h[1], h[2], h[3]);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&bars->raw_empty[raw]);
            mbar_arrive(&bars->kv_full[at]);
          }
          if (is_v) raw_v.next(), at_v.next();
          else raw_k.next(), at_k.next();
        }
        tile0 += n;
      }
    }
  } else if (warp >= C::kMmaWarp) {
    if constexpr (C::kSplit) regs_dec<C::kControlRegs>();
    if (warp == C::kLoadWarp || (FP4 && warp == C::kGuardWarp)) {
      // ================================================================ loader
      // Lane = (box, column block) of a key tile: its page's rows.  Over 4 bits one warp
      // loads keys (and queries), another values; lanes of the first half copy codes,
      // those of the second factors (a page's rows of one head lie one behind another).
      const bool loads_v = FP4 && warp == C::kGuardWarp;
      const int box_shift = min(p.page_shift, 7), boxes_shift = 7 - box_shift;
      const int boxes = 1 << boxes_shift;
      const int box = lane & (boxes - 1), cb = lane >> boxes_shift;
      const uint64_t keep = policy_evict_last(), once = policy_evict_first();
      const int missing = p.n_pages * p.Hkv;  // a coordinate outside: zeros
      const int in_page = (1 << p.page_shift) - 1;
      int segs = 0, tile = 0;
      bool ok = true;
      // Pages are looked up for 32 boxes at a time, a window ahead of their use: lane l
      // has box l % boxes of the window's tile l / boxes (-1 behind the segment or the
      // sequence; a key there may be past what an int counts).
      const int per_window = 32 >> boxes_shift;
      auto lookup = [&](int w) {
        const int j = seg.j0 + w * per_window + cb;
        const uint32_t key = static_cast<uint32_t>(j) * kBN + (box << box_shift);
        return j < seg.j1 && key < static_cast<uint32_t>(seg.s.n)
                   ? p.page_table[static_cast<long long>(seg.b) * p.max_pages + (key >> p.page_shift)]
                   : -1;
      };
      // Notes the 16-key blocks without a page of tile number `at`: they are left out.
      auto note_missing = [&](bool is_v, int at, uint32_t absent) {
        uint32_t bad = 0;
        if (absent != 0) {
          if (lane == 0) report_index(p.status);
          for (int i = 0; i < 8; ++i) bad |= ((absent >> (i * 16 >> box_shift)) & 1u) << i;
        }
        if (lane == 0) bars->bad[is_v][at % kTileRing] = static_cast<uint8_t>(bad);
      };
      auto load_q = [&]() {
        if (lane == 0) {
          ok = segs == 0 || bounded_wait(&bars->q_empty, (segs - 1) & 1, abort_flag, p.status, kStatusTimeoutLoad);
          if (ok) {
            const int t0 = seg.k * NT * p.tq_tokens;
            int real = 0;
            for (int x = 0; x < NT; ++x) real += t0 + x * p.tq_tokens < seg.s.rows;
            constexpr int kLoads = COPIES;
            mbar_arrive_expect_tx(&bars->q_full, real * kLoads * C::kColBlocks * p.hb * p.tq_tokens * 128);
            for (int x = 0; x < real; ++x)
              for (int c = 0; c < C::kColBlocks; ++c)
                for (int i = 0; i < kLoads; ++i)
                  tma_load_5d(sQ + x * C::kQBytes + c * kBM * 128 + i * C::kRows * 128, &p.tq, &bars->q_full,
                              c * 64, first_head(p, seg.u), kv_head(p, seg.u), t0 + x * p.tq_tokens, seg.b, once);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        ++segs;
      };
      if constexpr (FP4) {
        const int row_bytes = cb == 0 ? D / 2 : D / 16;
        const uint32_t bytes = static_cast<uint32_t>(row_bytes << box_shift);
        const uint8_t* const pool = cb == 0 ? p.codes[loads_v] : p.factors[loads_v];
        uint8_t* const dst = smem + C::kRawOff + (cb == 0 ? 0 : kBN * (D / 2)) + box * bytes;
        const int first = loads_v ? C::kRawKStages : 0;
        const int places = loads_v ? C::kRawStages - C::kRawKStages : C::kRawKStages;
        int st = first, round = 0, filled = 0;
        while (ok && cur.next(p, seg)) {
          const int kvh = kv_head(p, seg.u);
          int now = lookup(0), next = lookup(1), in = 0, window = 1;
          if (!loads_v) {
            load_q();
            if (!ok) break;
          }
          int key = seg.j0 * kBN + (box << box_shift);
          for (int j = seg.j0; j < seg.j1; ++j, ++tile, key += kBN) {
            const int page = __shfl_sync(0xffffffffu, now, in * boxes + box);
            if (++in == per_window) {
              in = 0;
              now = next;
              next = lookup(++window);
            }
            const bool inside = key < seg.s.n;
            const bool found = inside && page >= 0 && page < p.n_pages;
            const uint32_t copied = __ballot_sync(0xffffffffu, cb == 0 && found);
            note_missing(loads_v, tile, __ballot_sync(0xffffffffu, cb == 0 && inside && !found));
            const uint8_t* src =
                pool + (((static_cast<long long>(page) * p.Hkv + kvh) << p.page_shift) + (key & in_page)) * row_bytes;
            if (round > 0)
              ok = bounded_wait(&bars->raw_empty[st], (round & 1) ^ 1, abort_flag, p.status, kStatusTimeoutLoad);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(&bars->raw[st], (__popc(copied) << box_shift) * (D / 2 + D / 16));
            __syncwarp();
            if (found && cb < 2) bulk_load(dst + st * C::kRawBytes, src, bytes, &bars->raw[st], keep);
            ++filled;
            if (++st == first + places) st = first, ++round;
          }
        }
        // Every copy must have landed before the CTA ends.
        if (lane == 0) {
          int dummy = 0;
          volatile int* ignore = reinterpret_cast<volatile int*>(&dummy);
          if (segs > 0) bounded_wait(&bars->q_full, (segs - 1) & 1, ignore, p.status, kStatusTimeoutDrain);
          for (int i = max(0, filled - places); i < filled; ++i)
            bounded_wait(&bars->raw[first + i % places], (i / places) & 1, ignore, p.status, kStatusTimeoutDrain);
        }
      } else {
        const bool loads = cb < C::kColBlocks;
        // One ring in the order of the loads, or one for K and one for V.
        Ring<0, C::kKStages> ring_k;
        Ring<C::kOneRing ? 0 : C::kKStages, C::kStages> ring_v;
        int filled[2] = {0, 0};
        while (ok && cur.next(p, seg)) {
          int now = lookup(0), next = lookup(1), window = 1;  // windows of V's tile and the one behind it
          const int kvh = kv_head(p, seg.u);
          int lim0;
          const int jm = first_masked<NT>(p, seg, lim0);
          load_q();
          if (!ok) break;
          auto issue = [&](bool is_v, int j, int page) {
            const bool by_v = is_v && !C::kOneRing;
            const int st = by_v ? ring_v.st : ring_k.st;
            const uint32_t round = by_v ? ring_v.round : ring_k.round;
            const int key = j * kBN + (box << box_shift);
            const bool inside = key < seg.s.n;
            const bool found = inside && page >= 0 && page < p.n_pages;
            if (!is_v) note_missing(false, tile++, __ballot_sync(0xffffffffu, cb == 0 && inside && !found));
            if (round > 0)
              ok = bounded_wait(&bars->kv_empty[st], (round & 1u) ^ 1u, abort_flag, p.status, kStatusTimeoutLoad);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) return;
            uint64_t* bar = is_v && j >= jm ? &bars->raw[st] : &bars->kv_full[st];
            if (lane == 0) mbar_arrive_expect_tx(bar, C::kTileBytes);
            __syncwarp();
            if (loads)
              tma_load_3d(sRing + st * C::kTileBytes + cb * C::kBlockBytes + (box << box_shift) * 128,
                          is_v ? &p.tv : &p.tk, bar, cb * 64, found ? key & in_page : 0,
                          found ? page * p.Hkv + kvh : missing, keep);
            if (by_v) ring_v.next();
            else ring_k.next();
            ++filled[by_v];
          };
          const int n = seg.j1 - seg.j0;
          issue(false, seg.j0, __shfl_sync(0xffffffffu, now, box));
          for (int t = 0, in = 0; ok && t < n; ++t) {  // `in`: V's tile in its window
            const int page_v = __shfl_sync(0xffffffffu, now, in * boxes + box);
            if (++in == per_window) {
              in = 0;
              now = next;
              next = lookup(++window);
            }
            if (t + 1 < n) issue(false, seg.j0 + t + 1, __shfl_sync(0xffffffffu, now, in * boxes + box));
            if (ok) issue(true, seg.j0 + t, page_v);
          }
        }
        // Every copy must have landed before the CTA ends.
        if (lane == 0) {
          int dummy = 0;
          volatile int* ignore = reinterpret_cast<volatile int*>(&dummy);
          if (segs > 0) bounded_wait(&bars->q_full, (segs - 1) & 1, ignore, p.status, kStatusTimeoutDrain);
          for (int r = 0; r < (C::kOneRing ? 1 : 2); ++r) {
            const int first = r ? C::kKStages : 0, places = (r ? C::kStages : C::kKStages) - first;
            for (int i = max(0, filled[r] - places); i < filled[r]; ++i)
              bounded_wait(&bars->kv_full[first + i % places], (i / places) & 1, ignore, p.status, kStatusTimeoutDrain);
          }
        }
      }
      __syncwarp();
    } else if (!FP4 && warp == C::kGuardWarp) {
      // ================================================================ guard of V
      constexpr int kCols = D / 32;  // of a lane, in one 16-byte piece
      const int cbyte = lane * kCols * 2;
      const int cb = cbyte / 128, chunk = (cbyte % 128) / 16, in_chunk = cbyte % 16;
      constexpr uint32_t kExp = BF16 ? 0x7F80u : 0x7C00u;
      int items = 0, segs = 0;
      uint32_t raw_phase = 0;
      bool ok = true;
      while (ok && cur.next(p, seg)) {
        const int n = seg.j1 - seg.j0;
        int lim0;
        const int jm = max(seg.j0, first_masked<NT>(p, seg, lim0));
        uint32_t first[kCols];
#pragma unroll
        for (int c = 0; c < kCols; ++c) first[c] = 255u;
        for (int j = jm; j < seg.j1; ++j) {
          const int st = C::kOneRing
                             ? (items + item_of_v(j - seg.j0, n)) % C::kStages
                             : C::kKStages + (items / 2 + j - seg.j0) % (C::kOneRing ? 1 : C::kStages - C::kKStages);
          ok = bounded_wait(&bars->raw[st], (raw_phase >> st) & 1, abort_flag, p.status, kStatusTimeoutMma);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          raw_phase ^= 1u << st;
          uint8_t* base = sRing + st * C::kTileBytes + cb * C::kBlockBytes;
          const int r0 = max(0, lim0 + 1 - j * kBN);
          if (!any_not_finite<BF16, C::kColBlocks>(sRing + st * C::kTileBytes, r0, lane)) {
            if (j == jm) {  // (later tiles add to what has been noted)
              if (lane == 0) bars->nan_any[segs % kSegRing] = 0;
              __syncwarp();
            }
            if (lane == 0) mbar_arrive(&bars->kv_full[st]);
            continue;
          }
          for (int r = r0; r < kBN; ++r) {
            uint32_t* w = reinterpret_cast<uint32_t*>(base + r * 128 + ((chunk ^ (r & 7)) << 4) + in_chunk);
            const int key = j * kBN + r;
            if (key >= seg.s.n) {
#pragma unroll
              for (int i = 0; i < kCols / 2; ++i) w[i] = 0u;
              continue;
            }
#pragma unroll
            for (int i = 0; i < kCols / 2; ++i) {
              uint32_t v = w[i];
              const bool lo = (v & kExp) == kExp, hi = (v >> 16 & kExp) == kExp;
              if (lo || hi) {
                // below 255 where a row of the unit sees the key
                const uint32_t e = min(static_cast<uint32_t>(key - lim0 - 1), 255u);
                if (lo) first[2 * i] = min(first[2 * i], e), v &= 0xFFFF0000u;
                if (hi) first[2 * i + 1] = min(first[2 * i + 1], e), v &= 0xFFFFu;
                w[i] = v;
              }
            }
          }
          // Noted after each tile: a row tile may end before the unit's last one, and
          // keys noted later are none of its rows'.
          bool any = false;
#pragma unroll
          for (int c = 0; c < kCols; ++c) {
            any |= first[c] != 255u;
            bars->nan_from[segs % kSegRing][lane * kCols + c] = static_cast<uint8_t>(first[c]);
          }
          any = __any_sync(0xffffffffu, any);
          if (lane == 0) bars->nan_any[segs % kSegRing] = any;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->kv_full[st]);
        }
        items += 2 * n;
        ++segs;
      }
    } else if (warp - C::kMmaWarp < 2) {
      // ================================================================ MMA issuers
      // One issuing thread per tile.  Each releases every K/V slot; key tiles that
      // its rows do not visit are released once landed.  (One tile: one for K, one for V.)
      if (lane == 0) {
        const int x = NT == 1 ? 0 : warp - C::kMmaWarp;
        const bool does_qk = NT == 2 || warp == C::kMmaWarp;
        constexpr uint32_t kIdescQK = idesc_f16(kMmaBf16, false, false, kBM, kBN);
        constexpr uint32_t kIdescPV = idesc_f16(kMmaBf16, false, true, kBM, D);
        const uint32_t ring_addr = smem_u32(sRing);
        const uint32_t o_col = tmem + C::kOCol + x * D;
        const uint64_t q_desc = smem_desc_sw128(smem_u32(sQ + x * C::kQBytes), 16, 1024);
        const uint64_t p_desc = smem_desc_sw128(smem_u32(sP + x * C::kStageBytes), 16, 1024);
        auto issue_qk = [&](int st, int d) {
          const uint32_t s_col = tmem + C::kSCol + C::s_bar(x, d) * kBN;
          const uint64_t kd = smem_desc_sw128(ring_addr + st * C::kTileBytes, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t off = ((kk / 4) * C::kBlockBytes + (kk % 4) * 32) >> 4;
            mma_f16_ss(s_col, q_desc + off, kd + off, kIdescQK, kk > 0 ? 1u : 0u);
          }
        };
        auto issue_pv = [&](int st, int d, bool accumulate) {
          const uint32_t p_tcol = tmem + C::kPCol + C::s_bar(x, d) * (kBN / 2);
          const uint64_t vd = smem_desc_sw128(ring_addr + st * C::kTileBytes, C::kBlockBytes, 1024);
#pragma unroll
          for (int kk = 0; kk < kBN / 16; ++kk) {
            const uint32_t acc = (accumulate || kk > 0) ? 1u : 0u;
            if constexpr (C::kPInTmem) {
              mma_f16_ts(o_col, p_tcol + kk * 8, vd + ((kk * 2048) >> 4), kIdescPV, acc);
            } else {
              const uint64_t poff = ((kk / 4) * C::kBlockBytes + (kk % 4) * 32) >> 4;
              mma_f16_ss(o_col, p_desc + poff, vd + ((kk * 2048) >> 4), kIdescPV, acc);
            }
          }
        };
        int segs = 0;
        int done = 0;  // key tiles of this row tile so far
        bool ok = true;
        int st = 0;  // place of the last item waited for
        Ring<0, C::kKStages> ring_k;
        Ring<C::kOneRing ? 0 : C::kKStages, C::kStages> ring_v;
        // The next K or V, all in the order of their loads.
        auto wait_next = [&](auto& ring) {
          st = ring.st;
          const uint32_t phase = ring.phase();
          ring.next();
          return bounded_wait(&bars->kv_full[st], phase, abort_flag, p.status, kStatusTimeoutMma);
        };
        auto wait_item = [&](bool is_v) { return is_v && !C::kOneRing ? wait_next(ring_v) : wait_next(ring_k); };
        // S of the tile that is number `d` of this row tile's.
        auto qk = [&](int d) {
          if (!(ok = wait_item(false))) return;
          // The S before it in this place is in registers.
          if (d >= C::kSBufs &&
              !(ok = bounded_wait(&bars->s_free[C::s_bar(x, d)], (d / C::kSBufs - 1) & 1, abort_flag, p.status,
                                  kStatusTimeoutMma)))
            return;
          tc_fence_after();
          issue_qk(st, d);
          mma_commit(&bars->s_full[C::s_bar(x, d)]);
          mma_commit(&bars->kv_empty[st]);
        };
        auto pv = [&](int d, bool first, bool last) {
          if (!(ok = wait_item(true))) return;
          if (!(ok = bounded_wait(&bars->p_full[C::s_bar(x, d)], (d / C::kSBufs) & 1, abort_flag, p.status,
                                  kStatusTimeoutMma)))
            return;
          tc_fence_after();
          issue_pv(st, d, !first);
          mma_commit(&bars->p_free[C::s_bar(x, d)]);
          if (last) mma_commit(&bars->o_full[x]);
          mma_commit(&bars->kv_empty[st]);
        };
        while (ok && cur.next(p, seg)) {
          const TileRows tile(p, seg, x, NT);
          const int n = seg.j1 - seg.j0, nx = tile.j1 - seg.j0;
          if (NT == 2 || does_qk)
            ok = bounded_wait(kReadyQ ? &bars->q_ready[x] : &bars->q_full, segs & 1, abort_flag, p.status,
                              kStatusTimeoutMma);
          // Tile L starts when tile H has read its first S: the two softmax chains
          // then run staggered.
          if (NT == 2 && ok && x == 1 && segs == 0 && nx > 0) {
            const TileRows other(p, seg, 0, NT);
            if (other.j1 > seg.j0) ok = bounded_wait(&bars->stagger, 0, abort_flag, p.status, kStatusTimeoutMma);
          }
          if (!ok) break;
          if constexpr (NT == 1) {
            // (one row tile: it visits all of the segment's key tiles)
            for (int j = 0; ok && j < n; ++j, ++done) {
              if (does_qk) qk(done);
              else pv(done, j == 0, j == n - 1);
            }
            if (ok && does_qk) mma_commit(&bars->q_empty);
          } else {
            // K_0, then K_{j+1} and V_j in turn; what this tile's rows do not visit is
            // released once landed.
            auto skip = [&](bool is_v) {
              if ((ok = wait_item(is_v))) mbar_arrive(&bars->kv_empty[st]);
            };
            mbar_arrive(&bars->q_empty, nx > 0 ? 4 : 1);  // (the rest: below, or the softmax warps)
            for (int j = -1; ok && j < n; ++j) {
              if (j + 1 < nx) {
                qk(done + j + 1);
                if (ok && j + 2 == nx) mma_commit(&bars->q_empty);
              } else if (j + 1 < n) {
                skip(false);
              }
              if (!ok || j < 0) continue;
              if (j < nx) pv(done + j, j == 0, j == nx - 1);
              else skip(true);
            }
            done += nx;
          }
          ++segs;
        }
        // Every MMA this thread issued must complete before TMEM is released.
        mma_commit(&bars->mma_done[warp - C::kMmaWarp]);
        int dummy = 0;
        bounded_wait(&bars->mma_done[warp - C::kMmaWarp], 0, reinterpret_cast<volatile int*>(&dummy), p.status,
                     kStatusTimeoutDrain);
      }
      __syncwarp();
    }
  } else {
    // ================================================================ softmax
    if constexpr (C::kSplit) regs_inc<C::kSoftmaxRegs>();
    const int x = warp / 4;
    const int wq = warp % 4;
    const int row = wq * 32 + lane;
    const int copy = row / C::kRows, crow = row % C::kRows;  // (a warp's lanes are of one copy)
    const int col0 = copy * C::kCols;                        // its first key of a tile
    const int row_token = token_of(p, crow), row_head = crow - row_token * p.hb;
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t o_tmem = tmem + lane_off + C::kOCol + x * D;
    bool ok = true;
    const uint32_t p_place = tmem + lane_off + C::kPCol;
    // P.V of the tile that is number d of this row tile's is through.
    auto wait_pv = [&](int d) {
      ok = bounded_wait(&bars->p_free[C::s_bar(x, d)], (d / C::kSBufs) & 1, abort_flag, p.status,
                        kStatusTimeoutSoftmax);
      ok = __all_sync(0xffffffffu, ok);
    };
    uint8_t* p_row = sP + x * C::kStageBytes + row * 128;
    float lam = p.scale_log2;  // of this row
    float vd = 1.f;
    int done = 0, segs_x = 0, segs = 0, tiles = 0;
    bool staged = false;  // an output's store may still read the staging buffer
    uint32_t group_phase = 0;
    // Barrier of the tile's four warps; like every wait it ends when another role gave up.
    auto group_sync = [&]() {
      mbar_arrive(&bars->group[x]);
      ok = bounded_wait(&bars->group[x], group_phase, abort_flag, p.status, kStatusTimeoutSoftmax);
      ok = __all_sync(0xffffffffu, ok);
      group_phase ^= 1u;
    };
    auto stage_free = [&]() {
      if (!staged) return;
      if (wq < C::kColBlocks && lane == 0) bulk_wait_group_read0();
      group_sync();
      staged = false;
    };
    if constexpr (COPIES > 1) {  // the weights of the other copies' keys
      uint32_t zero[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) zero[i] = 0u;
#pragma unroll
      for (int i = 0; i < C::kSBufs * kBN / 64; ++i) tmem_st32(p_place + i * 32, zero);
      tmem_wait_st();
    }
    // The walk's state waits in shared memory: the softmax of 128 keys wants its registers
    // (chunks of 4 sequences over 4 bits 858 -> 835 us, 16 bits 727 -> 724; with copies, of
    // fewer keys a thread, it stays in registers: 5 tokens of 64 sequences 423, not 432).
    constexpr bool kParked = COPIES == 1;
    static_assert(sizeof(Cursor<NT>) <= 48 && sizeof(Seg) <= 48, "walk");
    volatile uint32_t* const walk = bars->walk[warp];
    auto put = [&](int at, const auto& v) {
      uint32_t w[sizeof(v) / 4];
      memcpy(w, &v, sizeof(v));
      __syncwarp();
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(v) / 4); ++i) walk[at + i] = w[i];
      __syncwarp();
    };
    auto get = [&](int at, auto& v) {
      uint32_t w[sizeof(v) / 4];
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(v) / 4); ++i) w[i] = walk[at + i];
      memcpy(&v, w, sizeof(v));
    };
    if constexpr (kParked) put(0, cur);
    while (ok) {
      if constexpr (!kParked) {
        if (!cur.next(p, seg)) break;
      } else {
        Cursor<NT> at;
        get(0, at);
        if (!at.next(p, seg)) break;
        put(0, at);
        put(12, seg);
      }
      float r = -INFINITY;  // retained reference, raw score units
      float l = 0.f;
      bool real;
      int lim;
      {
        const TileRows tile(p, seg, x, NT);
        const int t = tile.t0 + row_token;
        const int head = first_head(p, seg.u) + row_head;  // of the KV head's query heads
        const bool in_tile = row_token < p.tq_tokens && head < p.g;
        real = in_tile && t < seg.s.rows && seg.s.p0 + t >= 0;
        lim = real ? limit(p, seg.s, t) : -1;
        [[maybe_unused]] float kd = 1.f, up = 1.f;
        if constexpr (FP4) {
          const int kvh = kv_head(p, seg.u);
          if (p.descale[0] != nullptr) kd = p.descale[0][kvh];
          vd = p.descale[1] != nullptr ? p.descale[1][kvh] : 1.f;
        }
        if constexpr (kReadyQ) {
          // The row of Q, in place, to fp16 behind a power of two that brings its largest
          // element to [1, 2): exact but for elements below 2^-14 of that one.
          ok = bounded_wait(&bars->q_full, segs & 1, abort_flag, p.status, kStatusTimeoutSoftmax);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          uint8_t* q_row = sQ + x * C::kQBytes + row * 128;
          auto piece = [&](int i) {
            return reinterpret_cast<uint4*>(q_row + (i / 8) * C::kBlockBytes + ((i ^ row) & 7) * 16);
          };
          uint32_t top = 0;
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            const uint4 v = *piece(i);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) top = max(top, max(w[k] & 0x7F80u, w[k] >> 16 & 0x7F80u));
          }
          const uint32_t e = min(max(top >> 7, 1u), 253u);
          const float down = __uint_as_float((254u - e) << 23);
          up = __uint_as_float(e << 23);
#pragma unroll 4
          for (int i = 0; i < D / 8; ++i) {
            const uint4 v = *piece(i);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              h[k] = pack2<false>(__uint_as_float(w[k] << 16) * down, __uint_as_float(w[k] & 0xFFFF0000u) * down);
            *piece(i) = make_uint4(h[0], h[1], h[2], h[3]);
          }
          fence_proxy_async_smem();
          mbar_arrive(&bars->q_ready[x]);
        }
        if constexpr (FP4) {
          // The three factors' product may be an fp32 number where that of two is none: in
          // 64 bits then (always, 3 tokens of 40 sequences of 200 took 32.6 us, not 32.3).
          lam = p.scale_log2 * kd;
          if (p.scale_log2 >= FLT_MIN && lam >= FLT_MIN && lam <= FLT_MAX) lam *= up;
          else lam = static_cast<float>(p.scale64 * kd * up);
          if (lam < kLeastScale) lam = kLeastScale;
        }
        const int nx = tile.j1 - seg.j0;
        const bool active = __any_sync(0xffffffffu, real);
        for (int j = 0; j < nx; ++j, ++done) {
          if (!active) {  // no row of this warp counts: P stays as it is
            ok = bounded_wait(&bars->s_full[C::s_bar(x, done)], (done / C::kSBufs) & 1, abort_flag, p.status,
                              kStatusTimeoutSoftmax);
            if (!__all_sync(0xffffffffu, ok)) {
              ok = false;
              break;
            }
            mbar_arrive(&bars->s_free[C::s_bar(x, done)]);
            if (NT == 2 && x == 0 && segs == 0 && j == 0) mbar_arrive(&bars->stagger);
            if (j >= C::kSBufs) {
              wait_pv(done - C::kSBufs);
            } else if constexpr (!C::kPInTmem) {
              stage_free();
            }
            if (!ok) break;
            mbar_arrive(&bars->p_full[C::s_bar(x, done)]);
            continue;
          }
          const uint32_t s_tmem = tmem + lane_off + C::kSCol + C::s_bar(x, done) * kBN + col0;
          ok = bounded_wait(&bars->s_full[C::s_bar(x, done)], (done / C::kSBufs) & 1, abort_flag, p.status,
                            kStatusTimeoutSoftmax);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          tc_fence_after();
          constexpr int kCols = C::kCols;
          constexpr int kBlk = kCols < kPBlock ? kCols : kPBlock;  // keys whose weights are stored together
          const int k0 = (seg.j0 + j) * kBN + col0;
          const uint32_t bad = bars->bad[0][(tiles + j) % kTileRing] >> (col0 / 16);
          const bool masked = k0 + kCols - 1 > tile.lim_min || bad != 0 || p.sign != 1.f;
          if (masked) {
            // A pass of its own, in a loop: as a second form of what follows, unrolled for
            // all keys, it took 7000 cycles of each CTA's first such tile, most of them on
            // instructions' way into their cache, and the other warps with it.
            // 32 keys that all rows of the warp see stay as they are: all four blocks take
            // 2500 cycles, where a key tile takes 2900.
            const int all_see = __reduce_min_sync(0xffffffffu, real ? lim : 0x7FFFFFFF);
#pragma unroll 1
            for (int c = 0; c < kCols / 32; ++c) {
              if (all_see >= k0 + c * 32 + 31 && (bad >> (2 * c) & 3u) == 0 && p.sign == 1.f) continue;
              uint32_t w[32];
              tmem_ld32(s_tmem + c * 32, w);
              tmem_wait_ld();
              reg_fence32(w);
              const int last = lim - (k0 + c * 32);
              const uint32_t gone = bad >> (2 * c);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                w[i] = i <= last && !(gone >> (i / 16) & 1u) ? __float_as_uint(__uint_as_float(w[i]) * p.sign)
                                                             : 0xFF800000u;
              tmem_st32(s_tmem + c * 32, w);
            }
            tmem_wait_st();
          }
          uint32_t u[kCols];
          float mq[kCols / 32];
#pragma unroll
          for (int c = 0; c < kCols / 32; ++c)
            tmem_ld32_max(s_tmem + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&u[c * 32]), mq[c]);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < kCols / 32; ++c) reg_fence32(*reinterpret_cast<uint32_t(*)[32]>(&u[c * 32]));
          tc_fence_before();
          mbar_arrive(&bars->s_free[C::s_bar(x, done)]);
          if (NT == 2 && x == 0 && segs == 0 && j == 0) mbar_arrive(&bars->stagger);
          float* s = reinterpret_cast<float*>(u);
          float mx = mq[0];
#pragma unroll
          for (int c = 1; c < kCols / 32; ++c) mx = fmaxf(mx, mq[c]);
          float gamma = 1.f;
          if (j == 0) {
            r = mx;
          } else {
            const float cand = fmaxf(r, mx);
            if ((cand - r) * lam > kRescaleThreshold) {  // false when both are -inf
              gamma = ex2_approx((r - cand) * lam);
              r = cand;
            }
          }
          l *= gamma;
          const float rs = (r == -INFINITY) ? 0.f : r * lam;
          const float2 lam2 = make_float2(lam, lam);
          const float2 nrs2 = make_float2(-rs, -rs);
          float2 sum4[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int blk = 0; blk < kCols / kBlk; ++blk) {
            uint32_t pk[kBlk / 2];
#pragma unroll
            for (int c8 = 0; c8 < kBlk / 8; ++c8) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int c = blk * kBlk + c8 * 8 + 2 * i;
                const float2 e = ex2_pair(ffma2(make_float2(s[c], s[c + 1]), lam2, nrs2), c / 2);
                sum4[i] = fadd2(sum4[i], e);
                pk[c8 * 4 + i] = pack2<kMmaBf16>(e.x, e.y);
              }
            }
            if (blk == 0) {
              // The last tile that had P in this place, or, before O can be corrected, the
              // tile before this one is through.
              const bool correct = j > 0 && __any_sync(0xffffffffu, gamma != 1.f);
              if (j >= C::kSBufs || correct) {
                if (j >= C::kSBufs) wait_pv(done - C::kSBufs);
                if (C::kSBufs > 1 && ok && correct) wait_pv(done - 1);
                if (!ok) break;
                tc_fence_after();
                if (correct) {
#pragma unroll 1
                  for (int c = 0; c < D / 32; ++c) {
                    uint32_t w32[32];
                    tmem_ld32(o_tmem + c * 32, w32);
                    tmem_wait_ld();
                    reg_fence32(w32);
#pragma unroll
                    for (int i = 0; i < 32; ++i) w32[i] = __float_as_uint(__uint_as_float(w32[i]) * gamma);
                    tmem_st32(o_tmem + c * 32, w32);
                  }
                  tmem_wait_st();
                }
              }
              if constexpr (!C::kPInTmem) {
                if (j == 0) stage_free();
                if (!ok) break;
              }
            }
            if constexpr (!C::kPInTmem) {
#pragma unroll
              for (int c8 = 0; c8 < kBlk / 8; ++c8) {
                const int chunk = (blk * kBlk / 8 + c8) % 8;
                *reinterpret_cast<uint4*>(p_row + blk * kBlk / 64 * C::kBlockBytes + ((chunk ^ (row & 7)) << 4)) =
                    make_uint4(pk[c8 * 4], pk[c8 * 4 + 1], pk[c8 * 4 + 2], pk[c8 * 4 + 3]);
              }
            } else if constexpr (kBlk == 32) {
              tmem_st16(p_place + C::s_bar(x, done) * (kBN / 2) + col0 / 2 + blk * 16, pk);
            } else {
              tmem_st32(p_place + C::s_bar(x, done) * (kBN / 2) + col0 / 2 + blk * 32, pk);
            }
          }
          if (!ok) break;
          const float2 s01 = fadd2(fadd2(sum4[0], sum4[1]), fadd2(sum4[2], sum4[3]));
          l += s01.x + s01.y;
          if constexpr (C::kPInTmem) {
            tmem_wait_st();
          } else {
            fence_proxy_async_smem();
          }
          tc_fence_before();
          mbar_arrive(&bars->p_full[C::s_bar(x, done)]);
        }
        if (!ok) break;
      }
      if (!ok) break;
      if constexpr (kParked) get(12, seg);
      const TileRows tile(p, seg, x, NT);
      const int t = tile.t0 + row_token;
      const int head = first_head(p, seg.u) + row_head;
      const bool in_tile = row_token < p.tq_tokens && head < p.g;
      const int nx = tile.j1 - seg.j0;
      // ---- the segment's end
      if (nx > 0) {
        ok = bounded_wait(&bars->o_full[x], segs_x & 1, abort_flag, p.status, kStatusTimeoutSoftmax);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        ++segs_x;
      } else if constexpr (NT == 2) {  // this warp has read all notes so far
        ok = bounded_wait(&bars->q_full, segs & 1, abort_flag, p.status, kStatusTimeoutSoftmax);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        if (lane == 0) mbar_arrive(&bars->q_empty);
      }
      // Columns whose guarded rows of V are not finite for this row.
      int lim0;
      const bool guarded = !FP4 && tile.j1 > max(seg.j0, first_masked<NT>(p, seg, lim0));
      const bool nan_any = guarded && bars->nan_any[segs % kSegRing] != 0;
      if (nan_any) {
        const uint8_t* nan_from = bars->nan_from[segs % kSegRing];
        const int seen = real ? lim - lim0 : 0;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t w[32];
          tmem_ld32(o_tmem + c * 32, w);
          tmem_wait_ld();
          reg_fence32(w);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (seen > nan_from[c * 32 + i]) w[i] = 0x7FFFFFFFu;
          tmem_st32(o_tmem + c * 32, w);
        }
        tmem_wait_st();
      }
      if constexpr (COPIES > 1) {
        // Fold the copies: their references and sums, then O, 32 columns at a time; a
        // thread sums its row's part of the columns.
        constexpr int kPer = 32 / COPIES;
        const bool whole = seg.whole();
        const bool counts = real && l != 0.f;
        const float m = r * lam;
        float2* ml = reinterpret_cast<float2*>(sP);
        ml[row] = counts ? make_float2(m, l) : make_float2(-INFINITY, 0.f);
        group_sync();
        if (!ok) break;
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int c = 0; c < COPIES; ++c) M = fmaxf(M, ml[crow + c * C::kRows].x);
#pragma unroll
        for (int c = 0; c < COPIES; ++c) {
          const float2 v = ml[crow + c * C::kRows];
          if (v.y != 0.f) L = fmaf(v.x == M ? 1.f : ex2_approx(v.x - M), v.y, L);
        }
        const float weight = !counts ? 0.f : m == M ? vd : vd * ex2_approx(m - M);
        const bool writes = in_tile && t < p.S;
        const long long hrow = (static_cast<long long>(seg.b) * p.H + kv_head(p, seg.u) * p.g + head) * p.S + t;
        const long long part = blockIdx.x * 2LL + (seg.j0 > 0 ? 0 : 1);
        const float inv = L == 0.f ? 0.f : 1.f / L;
        float4* fold = reinterpret_cast<float4*>(sP);  // [8][kBM]
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t u[32];
          tmem_ld32(o_tmem + c * 32, u);
          tmem_wait_ld();
          reg_fence32(u);
          group_sync();  // what was there has been read
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = counts ? __uint_as_float(u[4 * i + k]) * weight : 0.f;
            fold[i * kBM + row] = make_float4(v[0], v[1], v[2], v[3]);
          }
          group_sync();
          if (!ok) break;
          float acc[kPer];
#pragma unroll
          for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
#pragma unroll
          for (int k = 0; k < COPIES; ++k)
#pragma unroll
            for (int i = 0; i < kPer / 4; ++i) {
              const float4 v = fold[(copy * (kPer / 4) + i) * kBM + crow + k * C::kRows];
              acc[4 * i] += v.x, acc[4 * i + 1] += v.y, acc[4 * i + 2] += v.z, acc[4 * i + 3] += v.w;
            }
          if (!writes) continue;
          if (whole) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + hrow * D + c * 32 + copy * kPer);
#pragma unroll
            for (int i = 0; i < kPer / 8; ++i)
              dst[i] = make_uint4(normalised<BF16>(acc[8 * i], acc[8 * i + 1], inv),
                                  normalised<BF16>(acc[8 * i + 2], acc[8 * i + 3], inv),
                                  normalised<BF16>(acc[8 * i + 4], acc[8 * i + 5], inv),
                                  normalised<BF16>(acc[8 * i + 6], acc[8 * i + 7], inv));
          } else {
            float4* dst =
                reinterpret_cast<float4*>(p.part_o) + (part * (D / 4) + c * 8 + copy * (kPer / 4)) * kBM + crow;
#pragma unroll
            for (int i = 0; i < kPer / 4; ++i)
              dst[i * kBM] = make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
          }
        }
        if (!ok) break;
        tc_fence_before();  // O has been read before P's arrival lets it be overwritten
        group_sync();       // the last columns too
        if (!ok) break;
        if (writes && copy == 0) {
          if (!whole) p.part_ml[part * kBM + crow] = make_float2(M, L);
          else if (p.lse != nullptr) p.lse[hrow] = L == 0.f ? -INFINITY : (M + __log2f(L)) * 0.69314718055994531f;
        }
      } else if (NT == 1 && p.cluster > 1) {
        // The row's state: O normalised, and log2 of the sum of its weights.  O lies in
        // two places that are through, half a row each; 16-byte pieces are permuted
        // against bank conflicts.
        const bool counts = real && nx > 0 && l != 0.f;
        bars->state[row] = counts ? r * lam + __log2f(l) : -INFINITY;
        if (__any_sync(0xffffffffu, counts)) {
          const float inv = vd / l;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t u[32];
            tmem_ld32(o_tmem + c * 32, u);
            tmem_wait_ld();
            reg_fence32(u);
            uint8_t* dst = state_row<C>(smem, row, c * 8);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<float4*>(dst + (((c * 8 + i) % (D / 8) ^ (row & 7)) << 4)) =
                  make_float4(__uint_as_float(u[4 * i]) * inv, __uint_as_float(u[4 * i + 1]) * inv,
                              __uint_as_float(u[4 * i + 2]) * inv, __uint_as_float(u[4 * i + 3]) * inv);
          }
        }
      } else if (seg.whole()) {
        [[maybe_unused]] long long store_row = -1;
        if constexpr (C::kDirectO) {
          if (in_tile && t < p.S)
            store_row = (static_cast<long long>(seg.b) * p.H + kv_head(p, seg.u) * p.g + head) * p.S + t;
        }
        if (tile.t0 < p.S) {
          const float inv = (!real || l == 0.f) ? 0.f : vd / l;
          stage_free();
          if (!ok) break;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t u[32];
            if (nx > 0) {
              tmem_ld32(o_tmem + c * 32, u);
              tmem_wait_ld();
              reg_fence32(u);
            }
            if (nx == 0 || !real || l == 0.f) {
#pragma unroll
              for (int i = 0; i < 32; ++i) u[i] = 0u;
            }
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
              pk[i] = normalised<BF16>(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]), inv);
            if constexpr (C::kDirectO) {
              if (store_row >= 0) {
                uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + store_row * D + c * 32);
#pragma unroll
                for (int k = 0; k < 4; ++k) dst[k] = make_uint4(pk[4 * k], pk[4 * k + 1], pk[4 * k + 2], pk[4 * k + 3]);
              }
            } else {
              uint8_t* blk = p_row + (c / 2) * C::kBlockBytes;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int ch = (c % 2) * 4 + k;
                *reinterpret_cast<uint4*>(blk + ((ch ^ (row & 7)) << 4)) =
                    make_uint4(pk[4 * k], pk[4 * k + 1], pk[4 * k + 2], pk[4 * k + 3]);
              }
            }
          }
          tc_fence_before();  // O_X has been read before P's arrival lets it be overwritten
          if constexpr (!C::kDirectO) {
            fence_proxy_async_smem();
            group_sync();
            if (!ok) break;
            // (issuing one takes some 700 cycles: a warp each)
            if (wq < C::kColBlocks && lane == 0) {
              tma_store_5d(&p.to, sP + x * C::kStageBytes + wq * C::kBlockBytes, wq * 64, first_head(p, seg.u),
                           kv_head(p, seg.u), tile.t0, seg.b);
              bulk_commit_group();
            }
            staged = true;
          }
          if (p.lse != nullptr && in_tile && t < p.S) {
            const float lse = !real || l == 0.f ? -INFINITY : (r * lam + __log2f(l)) * 0.69314718055994531f;
            p.lse[(static_cast<long long>(seg.b) * p.H + kv_head(p, seg.u) * p.g + head) * p.S + t] = lse;
          }
        }
      } else {
        const long long part = blockIdx.x * 2LL + (seg.j0 > 0 ? 0 : 1);
        const long long prow = part * (NT * kBM) + x * kBM + row;
        const bool counts = real && nx > 0 && l != 0.f;
        p.part_ml[prow] = counts ? make_float2(r * lam, l) : make_float2(-INFINITY, 0.f);
        if (__any_sync(0xffffffffu, counts)) {
          float4* dst = reinterpret_cast<float4*>(p.part_o) + part * (D / 4) * (NT * kBM) + x * kBM + row;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t u[32];
            tmem_ld32(o_tmem + c * 32, u);
            tmem_wait_ld();
            reg_fence32(u);
            if (counts) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                dst[(c * 8 + i) * (NT * kBM)] =
                    make_float4(__uint_as_float(u[4 * i]) * vd, __uint_as_float(u[4 * i + 1]) * vd,
                                __uint_as_float(u[4 * i + 2]) * vd, __uint_as_float(u[4 * i + 3]) * vd);
            }
          }
          tc_fence_before();
        }
      }
      // The CTA that has the unit's first tile says where its parts are.
      if (seg.j0 == 0 && threadIdx.x == 0 && p.cluster == 0) {
        const int behind = seg.nt - (seg.j1 - seg.j0);  // the unit's tiles in the runs after this one
        const int per = static_cast<int>(min(bars->per, 0x7FFFFFFFLL));
        p.parts[(static_cast<long long>(seg.b) * p.heads + seg.u) * p.blocks + seg.k] =
            make_int2(blockIdx.x, behind == 0 ? 1 : 2 + (behind - 1) / per);
      }
      tiles += seg.j1 - seg.j0;
      ++segs;
    }
    if (staged && wq < C::kColBlocks && lane == 0) bulk_wait_group_read0();
    if (COPIES == 1 && p.cluster > 0) {
      if (segs == 0) {  // no tile for this CTA
        if (NT == 1) bars->state[row] = -INFINITY;
        const int head = first_head(p, seg.u) + row_head, t = (seg.k * NT + x) * p.tq_tokens + row_token;
        if (p.cluster == 1 && row_token < p.tq_tokens && head < p.g && t < p.S) {  // the unit has no key: zeros
          const long long hrow = (static_cast<long long>(seg.b) * p.H + kv_head(p, seg.u) * p.g + head) * p.S + t;
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + hrow * D);
#pragma unroll 1
          for (int i = 0; i < D / 8; ++i) dst[i] = make_uint4(0u, 0u, 0u, 0u);
          if (p.lse != nullptr) p.lse[hrow] = -INFINITY;
        }
      }
      if (NT == 1 && p.cluster > 1) {
        __syncwarp();  // (the cluster's barrier takes whole warps)
        cluster_sync_all();
        if (ok) {
          if (p.cluster == 8) fold_cluster<C, D, BF16, 8>(p, seg, smem, bars);
          else if (p.cluster == 4) fold_cluster<C, D, BF16, 4>(p, seg, smem, bars);
          else fold_cluster<C, D, BF16, 2>(p, seg, smem, bars);
        }
      }
    }
  }
  // The others' arrivals at the first barrier, and the second: no CTA ends while its
  // states are read.
  if (NT == 1 && COPIES == 1 && p.cluster > 1) {
    __syncwarp();
    if (warp >= C::kMmaWarp) cluster_sync_all();
    cluster_sync_all();
  }

  // ---- teardown: all TMEM traffic done before the allocator warp frees it
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == C::kMmaWarp) tmem_dealloc(tmem, 512);
}

// Folds the parts of units that were split, in the order of the parts, and writes
// the zeros of units without a real row; launched while the first kernel runs, it
// waits for its end.  A warp takes 32 rows of a unit, lane = row (the parts' layout),
// D / kSlices elements each.
constexpr int kMergeThreads = 128;

template <int D, int NT>
__global__ void __launch_bounds__(kMergeThreads) prefill_paged_merge_kernel(const __grid_constant__ Params p) {
  constexpr int kSlice = 16;                 // elements of a warp's row
  constexpr int kSlices = D / kSlice, kRowBlocks = NT * kBM / 32;
  const int lane = threadIdx.x % 32;
  const int rows_used = p.hb * p.tq_tokens;
  wait_for_previous_kernel();
  const long long units = static_cast<long long>(p.B) * p.heads * p.blocks;
  const long long work = units * kRowBlocks * kSlices;
  for (long long w = blockIdx.x * (kMergeThreads / 32LL) + threadIdx.x / 32; w < work;
       w += gridDim.x * (kMergeThreads / 32LL)) {
    const int slice = static_cast<int>(w % kSlices), rb = static_cast<int>(w / kSlices % kRowBlocks);
    const long long unit = w / (kSlices * kRowBlocks);
    const int k = static_cast<int>(unit % p.blocks);
    const int u = static_cast<int>(unit / p.blocks % p.heads), b = static_cast<int>(unit / p.blocks / p.heads);
    const int x = rb / (kBM / 32), row = rb % (kBM / 32) * 32 + lane;
    const int tu = NT * p.tq_tokens;
    // Everything is requested before it is known to be needed: the unit's parts with its
    // lengths, the first parts' states and values before their weights.
    const int2 said = p.parts[unit];
    const Seq s = load_seq(p, b);
    int2 part = make_int2(0, 0);
    if (tiles_of(p, s, k * tu, (k + 1) * tu) > 0) {
      part = said;
      if (!split_parts(part.x, part.y, p.ctas)) continue;  // finished by one CTA, or by none
    }
    const int row_token = token_of(p, row);
    const int t = k * tu + x * p.tq_tokens + row_token, head = first_head(p, u) + row - row_token * p.hb;
    if (row >= rows_used || head >= p.g || t >= p.S) continue;
    auto state = [&](int i) { return (part.x + i) * 2LL + (i == 0 ? 1 : 0); };
    auto load_ml = [&](int i) { return p.part_ml[state(i) * (NT * kBM) + x * kBM + row]; };
    auto load_o = [&](int i, float4 (&v)[kSlice / 4]) {
      const float4* src = reinterpret_cast<const float4*>(p.part_o) +
                          (state(i) * (D / 4) + slice * (kSlice / 4)) * (NT * kBM) + x * kBM + row;
#pragma unroll
      for (int e = 0; e < kSlice / 4; ++e) v[e] = src[e * (NT * kBM)];
    };
    constexpr int kAhead = 4;
    float2 ml[kAhead];
    float4 v[kAhead][kSlice / 4];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      ml[i] = make_float2(-INFINITY, 0.f);
      if (i < part.y) {
        ml[i] = load_ml(i);
        load_o(i, v[i]);
      }
    }
    float M = fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x));
#pragma unroll 8
    for (int i = kAhead; i < part.y; ++i) M = fmaxf(M, load_ml(i).x);
    float l = 0.f;
    float acc[kSlice];
#pragma unroll
    for (int e = 0; e < kSlice; ++e) acc[e] = 0.f;
    // (a part without a key that counts has no values)
    auto add = [&](float2 m, const float4 (&o)[kSlice / 4]) {
      if (m.y == 0.f) return;
      const float f = m.x == M ? 1.f : ex2_approx(m.x - M);
      l = fmaf(f, m.y, l);
#pragma unroll
      for (int e = 0; e < kSlice / 4; ++e) {
        acc[4 * e] = fmaf(f, o[e].x, acc[4 * e]);
        acc[4 * e + 1] = fmaf(f, o[e].y, acc[4 * e + 1]);
        acc[4 * e + 2] = fmaf(f, o[e].z, acc[4 * e + 2]);
        acc[4 * e + 3] = fmaf(f, o[e].w, acc[4 * e + 3]);
      }
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (i < part.y) add(ml[i], v[i]);
    for (int base = kAhead; base < part.y; base += kAhead) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (base + i < part.y) {
          ml[i] = load_ml(base + i);
          load_o(base + i, v[i]);
        }
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (base + i < part.y) add(ml[i], v[i]);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint32_t out[kSlice / 2];
#pragma unroll
    for (int e = 0; e < kSlice; e += 2)
      out[e / 2] = p.out_bf16 ? normalised<true>(acc[e], acc[e + 1], inv) : normalised<false>(acc[e], acc[e + 1], inv);
    const long long hrow = (static_cast<long long>(b) * p.H + kv_head(p, u) * p.g + head) * p.S + t;
    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + hrow * D + slice * kSlice);
    dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
    dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
    if (slice == 0 && p.lse != nullptr)
      p.lse[hrow] = l == 0.f ? -INFINITY : (M + __log2f(l)) * 0.69314718055994531f;
  }
}

// How a problem is cut into units.
struct Shape {
  int hb, tokens, nblk, heads, nt, blocks;
  long long units;
};
Shape shape_of(int B, int H, int Hkv, int S, int nt) {
  Shape s;
  const int g = H / Hkv;
  s.nblk = (g + kBM - 1) / kBM;
  s.hb = (g + s.nblk - 1) / s.nblk;
  s.tokens = kBM / s.hb;
  s.heads = Hkv * s.nblk;
  if (S < s.tokens) s.tokens = S;
  s.nt = S == s.tokens ? 1 : nt;
  s.blocks = (S + s.nt * s.tokens - 1) / (s.nt * s.tokens);
  s.units = static_cast<long long>(B) * s.heads * s.blocks;
  return s;
}

// One tile where units of one find an SM each and two tiles would have at most
// kOneTileRun key tiles a CTA: more CTAs then share the work, and a tile alone starts and
// ends sooner.  Elsewhere two tiles share each key tile.  Measured with 8 KV heads of 4
// query heads (us in a captured graph by one tile, by two, and in brackets over 4 bits).
// d = 128: one sequence, 500 tokens of 1000 18.5, 20.6 (22.6, 28.2), 100 of 4000 22.6, 30.6
// (26.7, 41.0), 200 of 4000 30.8, 32.8 (41.0, 45.1); 4 sequences, 100 of 4000 41.0, 43.2 (51.3,
// 58.7).  Beyond the bounds: 4 sequences, 500 of 1000 71, 52; 100 of 16000 168, 113.  The rule
// does not ask for d: at 64 one tile wins for 500 of 1000 16.5, 18.5 and 100 of 4000 18.5,
// 24.7, and loses for 500 of 4000 39.0, 34.9 (43.1, 41.7) and 100 of 16000 41.0, 36.9 (45.1, 44.8).
constexpr long long kOneTileRun = 16;
Shape shape_of(int B, int H, int Hkv, int S, long long max_len, int num_sms) {
  const Shape one = shape_of(B, H, Hkv, S, 1), two = shape_of(B, H, Hkv, S, 2);
  return one.units <= num_sms && two.units * ((max_len + kBN - 1) / kBN) <= kOneTileRun * num_sms ? one : two;
}

// CTAs that can have work: one for each key tile at most.
int max_ctas(const Shape& s, int max_len) {
  const long long per_unit = (static_cast<long long>(max_len) + kBN - 1) / kBN;
  return s.units >= kMaxCtas || s.units * per_unit >= kMaxCtas ? kMaxCtas : static_cast<int>(s.units * per_unit);
}

// Clusters of n CTAs that run at once; the same on every GPU this library runs on.
template <typename Kernel>
int clusters_at_once(Kernel kern, int threads, int smem, int n, std::atomic<int>& known) {
  int most = known.load(std::memory_order_relaxed);
  if (most > 0) return most;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(n));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(n);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&most, kern, &cfg) != cudaSuccess || most < 1) {
    cudaGetLastError();
    return 0;
  }
  known.store(most, std::memory_order_relaxed);
  return most;
}

template <int D, bool BF16, int NT, bool FP4, int COPIES>
int launch_t(Params& p, const PagedPrefillArgs& a, const Shape& s) {
  using C = Cfg<D, NT, FP4, COPIES>;
  static_assert(C::kSmemBytes <= 232448, "shared memory of a CTA");
  auto kern = prefill_paged_kernel<D, BF16, NT, FP4, COPIES>;
  static std::atomic<unsigned long long> attr_done{0};  // per instantiation
  if (!set_smem_limit_once(kern, C::kSmemBytes, attr_done)) return -1;
  if constexpr (COPIES == 1) {
    // CTAs of a cluster that takes a unit, or 0: runs of the list.  The host knows what
    // the pages of a sequence can hold, not the lengths.  Clusters need neither the
    // division of the list nor the second kernel (kScan); one of several CTAs folds its
    // states, the longer the fewer it has (fold); both in key tiles of a unit, fitted to
    // measured times.  Clusters and runs, us in a captured graph, 8 KV heads of 4 query
    // heads, d = 128: 16 tokens of 1000 12.4, 14.4 (4 bits 14.4, 18.5), of 4000 14.4, 21.9; of
    // 16000 the runs are taken.  (With two row tiles the units are too many for several CTAs each, or
    // have so many key tiles that runs win.)
    constexpr float kScan = NT == 2 ? 5.f : 9.f;
    // Few rows have copies in runs: a key tile takes a CTA of a cluster `tile` times as
    // long.  3 tokens of 40 sequences over 4 bits, with and without copies: of 800 51, 64
    // us, of 200 37 both.  5 tokens of 8 sequences over 4 bits, copies and clusters: of 4000
    // 36.2, 38.8, of 1000 21.9, 20.5; over 16 bits with d = 64, of 2000 22.6, 18.5.
    const int rows = s.hb * s.tokens;
    const bool copies = NT == 1 && (FP4 || D == 64) && rows <= kBM / 2;
    const float tile = !copies ? 1.f : FP4 ? 1.6f : 1.3f;
    const float fold = 12.f * static_cast<float>(rows) / kBM;  // of one CTA alone
    static std::atomic<int> at_once[4];  // per instantiation, for clusters of 1, 2, 4 and 8
    const int tiles = ((p.max_pages << p.page_shift) + kBN - 1) / kBN;
    float best = static_cast<float>(s.units) * tiles / p.ctas + kScan;
    for (int i = 0, n = 1; i < (NT == 1 ? 4 : 1); ++i, n *= 2) {
      const float cost = tile * static_cast<float>((tiles + n - 1) / n) + (n > 1 ? fold / n : 0.f);
      if (s.units * n > a.num_sms || n > tiles || cost >= best) continue;
      if (n > 1 && s.units > clusters_at_once(kern, C::kThreads, C::kSmemBytes, n, at_once[i])) continue;
      p.cluster = n;
      best = cost;
    }
    if constexpr (NT == 1 && (FP4 || D == 64)) {
      if (copies && p.cluster == 0)
        return rows <= kBM / 4 ? launch_t<D, BF16, 1, FP4, 4>(p, a, s) : launch_t<D, BF16, 1, FP4, 2>(p, a, s);
    }
  }
  const CacheArgs& c = a.cache;
  const int page = 1 << c.page_shift;
  p.box_rows = page < kBN ? page : kBN;
  if (!make_tmap_heads(&p.tq, a.q, BF16, D, p.g, p.Hkv, a.S, a.B, s.hb, s.tokens) ||
      !make_tmap_heads(&p.to, a.o, BF16, D, p.g, p.Hkv, a.S, a.B, s.hb, s.tokens))
    return -1;
  if (FP4) {
    for (int i = 0; i < 2; ++i) {
      p.codes[i] = static_cast<const uint8_t*>(c.data[i]);
      p.factors[i] = static_cast<const uint8_t*>(c.scale[i]);
      p.descale[i] = c.descale[i];
    }
  } else if (!make_tmap_3d(&p.tk, c.data[0], BF16, D, page, static_cast<long long>(c.n_pages) * c.Hkv, p.box_rows) ||
      !make_tmap_3d(&p.tv, c.data[1], BF16, D, page, static_cast<long long>(c.n_pages) * c.Hkv, p.box_rows))
    return -1;
  if (p.cluster > 0)
    return launch_after(kern, dim3(p.blocks * p.cluster, p.heads, p.B), C::kThreads, a.stream, p, C::kSmemBytes,
                        p.cluster);
  if (launch_after(kern, dim3(static_cast<unsigned>(p.ctas)), C::kThreads, a.stream, p, C::kSmemBytes) != 0) return -1;
  const long long warps = s.units * (NT * kBM / 32) * (D / 16);
  long long ctas = (warps + kMergeThreads / 32 - 1) / (kMergeThreads / 32);
  if (ctas > 8LL * a.num_sms) ctas = 8LL * a.num_sms;
  return launch_after(prefill_paged_merge_kernel<D, NT>, dim3(static_cast<unsigned>(ctas)), kMergeThreads, a.stream, p);
}

template <int D, bool BF16>
int launch_d(Params& p, const PagedPrefillArgs& a, const Shape& s) {
  if (a.cache.fp4()) return s.nt == 2 ? launch_t<D, BF16, 2, true, 1>(p, a, s) : launch_t<D, BF16, 1, true, 1>(p, a, s);
  return s.nt == 2 ? launch_t<D, BF16, 2, false, 1>(p, a, s) : launch_t<D, BF16, 1, false, 1>(p, a, s);
}

}  // namespace

size_t paged_prefill_workspace_bytes(int B, int H, int Hkv, int S, int d, int max_len) {
  size_t most = 0;  // of either shape: the choice depends on the GPU
  for (int nt = 1; nt <= 2; ++nt) {
    const Shape s = shape_of(B, H, Hkv, S, nt);
    const size_t bytes =
        static_cast<size_t>(max_ctas(s, max_len)) * 2 * s.nt * kBM * (static_cast<size_t>(d) + 2) * sizeof(float) +
        static_cast<size_t>(s.units) * sizeof(int2);
    if (bytes > most) most = bytes;
  }
  return most;
}

int launch_prefill_paged(const PagedPrefillArgs& a) {
  const CacheArgs& c = a.cache;
  const Shape s = shape_of(a.B, a.H, c.Hkv, a.S, static_cast<long long>(c.max_pages) << c.page_shift, a.num_sms);
  Params p{};
  p.page_table = c.page_table;
  p.seqlens = c.seqlens;
  p.new_lens = a.new_lens;
  p.o = a.o;
  p.lse = a.lse;
  p.B = a.B;
  p.H = a.H;
  p.Hkv = c.Hkv;
  p.S = a.S;
  p.g = a.H / c.Hkv;
  p.hb = s.hb;
  p.hb_inverse = (65536 + s.hb - 1) / s.hb;
  p.tq_tokens = s.tokens;
  p.nblk = s.nblk;
  p.heads = s.heads;
  p.blocks = s.blocks;
  p.page_shift = c.page_shift;
  p.n_pages = c.n_pages;
  p.max_pages = c.max_pages;
  p.causal = a.causal;
  p.out_bf16 = a.bf16 ? 1 : 0;
  const float scale = a.scale < 0.f ? -a.scale : a.scale;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.scale64 = p.scale_log2 < FLT_MIN ? scale * 1.4426950408889634 : p.scale_log2;
  if (p.scale_log2 < kLeastScale) p.scale_log2 = kLeastScale;
  p.sign = a.scale == 0.f ? 0.f : a.scale < 0.f ? -1.f : 1.f;
  const int most = max_ctas(s, c.max_pages << c.page_shift);
  p.ctas = most < a.num_sms ? most : a.num_sms;
  p.wide = s.units * ((static_cast<long long>(c.max_pages << c.page_shift) + kBN - 1) / kBN) >= (1LL << 31) - kMaxCtas;
  p.status = a.status;
  const size_t states = static_cast<size_t>(most) * 2 * s.nt * kBM;
  float* ws = static_cast<float*>(a.workspace);
  p.part_o = ws;
  p.part_ml = reinterpret_cast<float2*>(ws + states * c.d);
  p.parts = reinterpret_cast<int2*>(ws + states * (c.d + 2));
  if (c.d == 128) return a.bf16 ? launch_d<128, true>(p, a, s) : launch_d<128, false>(p, a, s);
  return a.bf16 ? launch_d<64, true>(p, a, s) : launch_d<64, false>(p, a, s);
}

}  // namespace gbattn
