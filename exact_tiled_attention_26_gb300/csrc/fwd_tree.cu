// Attention of drafted tokens over the paged cache (a single token is a tree of one).
//
// Sequence b has lens[b] keys in the cache, the last n_new[b] of them the drafted
// tokens' own.  Draft token t sees every key of the prefix and, of the drafted ones,
// those whose bit is set in its row of `tree` (without a tree: tokens 0..t).  With
// s_j = q k_j scale over the keys it sees:
//   m = max s_j,  l = sum exp(s_j - m),  O = sum exp(s_j - m) v_j / l,  L = m + ln l.
// A row that sees no key gets O = 0 and L = -inf.
//
// The query rows of one key head (G = H / Hk heads of T tokens, contiguous in Q) are the
// rows of one matrix product, 128 at a time: a key and its value are read, and from e4m3
// converted, once for every 128 of them.
//
// Work.  A unit is (sequence, key head, 128-row tile of its rows); it has one tile of 128
// keys per 128 rows of cache, also where a long chunk's tokens see only some of them.  The
// tiles of all units in a row are cut into equal runs, one per CTA, whatever the lengths are
// (they are only known on the device): every SM reads the same amount of cache, and a single
// long sequence spreads over the whole GPU.  A unit that lies within one CTA is finished there; the others leave partial
// rows (O, m, l) in the workspace, at most two per CTA, which a second kernel joins.
//
// Rows.  The tensor-core tile has 128 rows.  With at most 32 (or 64) query rows they are
// repeated four (two) times in it, and each 32-row group weighs only its own quarter
// (half) of the keys, its weights for the others being zero.  So the four softmax warps
// share a tile's exponentials even for a single query row; the groups' results are
// joined at the end of a unit like the partial rows of different CTAs.
//
// Per CTA: warps 0 and 3 load a ring of K and V tiles (TMA boxes of one page each;
// issuing a tile's boxes takes about as long as its bytes, so K and V each have a warp);
// warp 1 issues S = Q K^T, warp 2 O += P V (tcgen05; Q, P and the accumulators in
// tensor memory); the warpgroup of warps 4..7 puts Q there, runs the softmax and the
// epilogue.  With more than 64 query rows warps 8..11 are a second one, and the two
// share a tile's columns: each takes half of a row's 128 scores, they agree on the row's
// maximum and add their sums at the end (measured when the second was added, 63 drafts x 4 sequences as below: 124 us
// with one, 96 with two).
//
// An e4m3 cache arrives in a ring of its own; the last warps (8..15, or 12..15) turn its
// tiles into f16 tiles (one instruction for two elements, exact) and Q is scaled to f16
// row by row.  The power-of-two scales stay out of the products: a key's multiplies its
// scores, a value's its weights, so that a row's weights are kept in f16's range by the
// largest of score + exponent of the value.
//
// Measured (d = 128, 8 key heads, 32 query heads, pages read once, device time):
//   16 sequences up to 32768, a token each, e4m3: 113 us, 4.7 TB/s (0.69 of a plain copy's rate).  A CTA takes some
//     1700 cycles a tile where its bytes take 1400: the chain load - convert - S - softmax - P V has five hand-overs a
//     tile, and the warp that loads K is busy issuing for most of it.  The same from a bf16 cache, without the
//     conversion and the scales: 6.6 TB/s (0.97).
//   12 drafts x 8 sequences up to 8192, bf16: 36.5 us, 4.1 TB/s; short runs, of which start, unit borders and the join
//     are 10 us.
//   63 drafts x 4 sequences up to 16384, e4m3: 79 us.  252 rows: every tile is loaded, converted and multiplied for two
//     row tiles in turn, and within each the softmax warps (every row weighs every key, 6.7e7 exponentials, scaled and
//     packed) and the products wait for one another; then the join, 10 us.
//   one token over 1000 keys: 9.8 us, two launches and one pass of latencies.
//
// Keys that are not there (behind the end, in no page) are masked; their values are
// replaced by zeros before the product, as 0 * NaN would reach every row.  An infinite or
// NaN value of a drafted token is taken out of the product too and goes only to the
// rows that see the token (`Poison`).  An infinite value of the prefix stays in the product,
// as every row sees it; but where rows are repeated, the groups that weigh its key with zero
// make NaN of it, so the joining kernel looks into rows that hold a NaN (`mend_rows`).
#include <cuda_fp16.h>

#include <cmath>

#include "cache.cuh"
#include "fwd_softmax.cuh"

namespace fa {

namespace {

constexpr int kMaxGrid = 152;  // CTAs at most, one per SM
constexpr int kKeys = 128;     // keys per tile
constexpr int kUnitCost = 6;   // see Walk
constexpr int kConvertRegs = 112;

enum : int { SITE_TREE_PRODUCER = 0x501, SITE_TREE_MMA = 0x502, SITE_TREE_SOFTMAX = 0x503, SITE_TREE_CONVERT = 0x504 };

// Workspace: for every unit the CTAs that hold its first and last tile, then two partial
// slots per CTA: [rows][D] fp32 of O, then [3][rows] of m, l, l of the rounded weights.
struct UnitInfo {
  int first, last;  // first: with kNanUnit where one CTA has all of it and a row holds a NaN that no score explains
};
constexpr int kNanUnit = 1 << 16;

struct TreeArgs {
  CacheView c;
  const __nv_bfloat16* Q;
  __nv_bfloat16* O;
  float* L;
  const unsigned long long* tree;  // [.., T, words], or null
  long long tree_stride;           // words between sequences
  int B, R, M, words;              // R = H / Hk * T rows per key head in M tiles
  int rows;                        // rows of a partial slot: 32, 64 or 128
  float c_log2;
  UnitInfo* info;
  float* part;
  int* status;
};

template <int D, bool FP8, int NS>
struct TCfg {
  static constexpr int SWB = (D * 2 >= 128) ? 128 : D * 2;
  static constexpr int CE = SWB / 2;
  static constexpr int TILE = 128 * D * 2;
  // Softmax warpgroups: two share a tile's columns where every row weighs all 128 keys itself.
  static constexpr int NW = NS == 1 ? 2 : 1;
  static constexpr int NPAIR = NW == 2 ? 1 : 2;            // pairs of converting warps for K, and for V
  static constexpr int NSLOT = D < 128 ? 8 : FP8 ? 4 : 6;  // 16-bit tiles, K and V in turn
  static constexpr int NRAW = FP8 ? NSLOT : 0;             // e4m3 tiles
  // K tiles use the even slots of a ring and V tiles the odd ones, and pairs of warps that take an e4m3 cache's
  // tiles in turn have slots of their own too (2 NPAIR divides NSLOT and NRAW).  So each slot's barriers are waited
  // for by one party that sees every phase of them: with a slot shared, a party that is a tile ahead would take the
  // other's phase for its own.
  static_assert(NSLOT % 2 == 0 && (!FP8 || (NSLOT % (2 * NPAIR) == 0 && NRAW % (2 * NPAIR) == 0)), "slots of their own");
  static constexpr int RAW = 128 * D + 256;     // with the exponent bytes of its keys (K tiles: and of their values)
  static constexpr int NSB = 2;                 // S buffers in tensor memory
  static constexpr int NPB = D == 128 ? 1 : 2;  // P buffers
  static constexpr int NSC = FP8 ? NSLOT / 2 + NSB + 1 : 0;  // tiles whose scales are kept (see the converter)
  static constexpr int OFF_T = 0;
  static constexpr int OFF_X = OFF_T + NSLOT * TILE;      // the epilogue's exchange
  static constexpr int OFF_RAW = OFF_X + (NS > 1 ? 16384 : 0);
  static constexpr int OFF_SCALE = OFF_RAW + NRAW * RAW;  // [NSC][3][128] floats: 2^k of K, 2^k of V, k of V
  static constexpr int OFF_ROWS = OFF_SCALE + NSC * 3 * 128 * 4;  // [3][128] floats
  static constexpr int OFF_TOPS = OFF_ROWS + 3 * 128 * 4;         // NW = 2: [2][2][128] floats
  static constexpr int OFF_BAR = OFF_TOPS + (NW == 2 ? 2560 : 0);  // (and [128] of Q's scales)
  static constexpr int B_QREADY = 0, B_FULL = 1, B_EMPTY = B_FULL + NSLOT,
                       B_RFULL = B_EMPTY + NSLOT, B_REMPTY = B_RFULL + NRAW, B_SFULL = B_REMPTY + NRAW,
                       B_SFREE = B_SFULL + NSB, B_PFULL = B_SFREE + NSB, B_PFREE = B_PFULL + NPB, B_OFULL = B_PFREE + NPB, B_OFREE = B_OFULL + 1,
                       B_MEET = B_OFREE + 1, B_TOP = B_MEET + 1, B_LSUM = B_TOP + (NW == 2 ? 4 : 0),
                       B_SDONE = B_LSUM + (NW == 2 ? 1 : 0), B_PVDONE = B_SDONE + 1, NBAR = B_PVDONE + 1;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;     // 24 words
  static constexpr int SMEM_USED = OFF_MISC + 96;
  static constexpr int SMEM = (SMEM_USED + 1024 > 120 * 1024) ? SMEM_USED + 1024 : 120 * 1024;
  // tensor memory columns: S buffers, P buffers and Q (two elements a column), O.  P has its own columns, so that
  // an S buffer is free again as soon as its scores are in registers: with P written over S the loop
  // softmax - P V - S - softmax bound the kernel (2 buffers: 2040 cycles a tile at d = 128).
  static constexpr int TM_S0 = 0, TM_P0 = NSB * 128, TM_O = TM_P0 + NPB * 64, TM_Q = TM_O + D, TM_COLS = 512;
  static constexpr int NTHREADS = FP8 ? 512 : 128 + 128 * NW;
  // setmaxnreg shares of issue, softmax and converting warps (0: none); their sums over the warpgroups stay within
  // the launch's: 4 x 128 with 512 threads, 3 x 168 with 384
  static constexpr int R_ISSUE = FP8 ? (NW == 2 ? 64 : 80) : 0;
  static constexpr int R_SOFT = FP8 ? (NW == 2 ? 168 : 208) : 0;
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert(TM_Q + D / 2 <= TM_COLS, "tensor memory budget");
};

FA_DEV int tiles_of(const CacheView& c, int b) {
  const int n = (seq_len(c, b) + kKeys - 1) / kKeys;
  return n < 1 ? 1 : n;  // an empty sequence passes through as one masked tile
}

// 64-bit quotients of what nearly always fits in 32 bits (a 64-bit division takes some
// hundred instructions).
FA_DEV long long quotient(long long a, long long b) {
  if (((a | b) >> 31) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// A CTA's run.  The units stand one after the other on a line, each with kUnitCost places
// (what starting and ending a unit costs, in tiles) before its tiles, and the CTAs take
// equal runs of places: those with a unit's border in them get that many tiles less.
// Measured for kUnitCost 0 / 3 / 4 / 6 / 8 / 12: 12 drafts x 8 sequences up to 8192, bf16 46.2 /
// 38.5 / 38.2 / 37.1 / 36.2 / 37.3 us; 63 drafts x 4 sequences up to 16384, e4m3 91.9 / 81.2 / 80.7 /
// 77.0 / 78.9 / 80.6; 24 drafts x 4 at d = 64 18.9 / 17.4 / 17.3 / 17.2 / 17.9 / 19.8; 16 tokens up to
// 32768, e4m3 119.1 / 113.4 / 112.5 / 113.0 / 114.8 / 117.5.
struct Walk {
  int b, hm, t0, nt;  // sequence, key head and row tile (h * M + mt), first tile, tiles of the unit
  int cost;           // places before the first tile
  long long left;     // places of the run from here on
  FA_DEV bool more() const { return left > cost; }
  FA_DEV int n() const { return nt - t0 < left - cost ? nt - t0 : static_cast<int>(left - cost); }
  FA_DEV void next(const CacheView& c, int hms) {
    left -= cost + n();
    t0 = 0;
    cost = kUnitCost;
    if (++hm == hms) {
      hm = 0;
      ++b;
      if (more()) nt = tiles_of(c, b);
    }
  }
};

// A warp's window on a sequence's page table, 32 entries (boxes) at a time, one per lane,
// the next 32 under way: while the SMs stream the cache, a load takes some 2400 cycles,
// more than a tile.
struct TableWindow {
  int now, next, pos, row;  // row: first of the 32 rows' boxes that `next` holds
  FA_DEV void open(const CacheView& c, int b, int first_row, int rb, int lane) {
    now = table_entry(c, b, first_row + lane * rb);
    row = first_row + 32 * rb;
    next = table_entry(c, b, row + lane * rb);
    pos = 0;
  }
  // The entries of the next tile's boxes, in lanes 0 .. boxes - 1.
  FA_DEV int take(const CacheView& c, int b, int boxes, int rb, int lane) {
    const int e = __shfl_sync(0xffffffffu, now, (pos + lane) & 31);
    pos += boxes;
    if (pos == 32) {
      pos = 0;
      now = next;
      row += 32 * rb;
      next = table_entry(c, b, row + lane * rb);
    }
    return e;
  }
};

// The run of one of `ctas` CTAs: its first place `lo`, its places `mine`, the places of
// every full run, and where it begins.  Every warp finds it by itself, each lane with a
// share of the sequences (all call it; the result is the same in every lane).
struct Run {
  long long lo, mine, run;
  Walk w;
};
FA_DEV Run find_run(const CacheView& c, int B, int hms, int cta, int ctas, int lane) {
  const int per = (B + 31) / 32, b0 = min(lane * per, B), b1 = min(b0 + per, B);
  long long sum = 0;
  int first = 0;
  for (int b = b0; b < b1; ++b) {
    const int n = tiles_of(c, b) + kUnitCost;
    if (b == b0) first = n;
    sum += n;
  }
  long long upto = sum;
#pragma unroll 1
  for (int k = 1; k < min(B, 32); k <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, upto, k);
    if (lane >= k) upto += y;
  }
  // (lanes behind the last sequence have their neighbour's sum only after all steps: take the last one's)
  const long long total = __shfl_sync(0xffffffffu, upto, (B - 1) / per) * hms, before = (upto - sum) * hms;
  Run r;
  r.run = quotient(total + ctas - 1, ctas);
  r.lo = r.run * cta;
  r.mine = total - r.lo < r.run ? total - r.lo : r.run;
  r.w = Walk{0, 0, 0, 0, 0, 0};
  if (r.mine <= 0) return r;
  // the lane with the sequence of the run's first place
  const bool here = b0 < b1 && r.lo >= before && r.lo < before + sum * hms;
  int b = b0, hm = 0, place = 0, places = first;
  if (here) {
    long long at = before;
    while (r.lo >= at + static_cast<long long>(places) * hms) {
      at += static_cast<long long>(places) * hms;
      places = tiles_of(c, ++b) + kUnitCost;
    }
    hm = static_cast<int>(quotient(r.lo - at, places));
    place = static_cast<int>(r.lo - at - static_cast<long long>(hm) * places);
  }
  const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
  b = __shfl_sync(0xffffffffu, b, src), hm = __shfl_sync(0xffffffffu, hm, src);
  place = __shfl_sync(0xffffffffu, place, src), places = __shfl_sync(0xffffffffu, places, src);
  r.w = Walk{b, hm, max(place - kUnitCost, 0), places - kUnitCost, max(kUnitCost - place, 0), r.mine};
  return r;
}

// 32 bits of a token's mask from draft index d0 on (bits below index 0 and behind the
// token's words are 0).
FA_DEV uint32_t draft_bits(const unsigned long long* row, int words, int t, int d0) {
  if (d0 <= -32) return 0u;
  if (row == nullptr) {  // tokens 0 .. t
    const int n = t - d0 + 1;  // bits d0 .. t
    uint32_t m = n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
    if (d0 < 0) m &= 0xffffffffu << -d0;
    return m;
  }
  if (d0 < 0) return static_cast<uint32_t>(row[0]) << -d0;
  const int w = d0 >> 6, s = d0 & 63;
  unsigned long long v = w < words ? row[w] >> s : 0ull;
  if (s > 32 && w + 1 < words) v |= row[w + 1] << (64 - s);
  return static_cast<uint32_t>(v);
}
FA_DEV uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

// Signs of infinities and NaNs (both bits) of a value row, and, in a row's thread, of all
// the tokens the row sees.
template <int D>
struct Poison {
  uint32_t pos[D / 32], neg[D / 32];
};

// Four e4m3 numbers as four f16 numbers, exactly.
FA_DEV void e4m3x4_to_f16x4(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
}
FA_DEV uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
FA_DEV uint4 ld_shared_v4(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
FA_DEV void st_shared_v4(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// The e4m3 format's weights are f16 numbers: 2^(score + exponent of the value - reference)
// starts at 2^kF16Start for a row's largest and the reference moves before it passes
// 2^kF16Top.  Whatever is 2^-18 of the largest or more keeps 11 bits.
constexpr float kF16Start = 4.f, kF16Top = 14.f;
// A value's exponent counts as this at least (its scale stays what it is): a weight is then at most 2^(kF16Top + 83) =
// 2^97, and 2^30 of them, the longest sequence, stay below fp32's 2^128.  (Rows of zeros have the least exponent, -100.
// Values below 448 * 2^-83 lose weight bits where none are larger: their largest weights start at 2^-13.)
constexpr int kRangeMin = 127 - 83;
// A sum of weights l taken from reference `from` to `to`.  An e4m3 cache's references follow the values' exponents and
// may lie more than 126 apart, where the factor 2^(from - to) alone would be 0 although l times it is not.
template <bool FP8>
FA_DEV float rescaled(float l, float from, float to) {
  const float f = from == -INFINITY ? 0.f : ex2((FP8 ? 0.5f : 1.f) * (from - to));
  return FP8 ? l * f * f : l * f;
}

// Which 16-byte unit of a row the swizzle puts where: unit ^ swz_row(row).
template <int SWB>
FA_DEV uint32_t swz_row(int row) {
  return SWB == 128 ? row & 7 : (row >> 1) & 3;
}

// Value rows of a tile that is not all prefix, looked after by the four softmax warps
// (which have all met): rows [last, 128), behind the end, become zero, as 0 * NaN would
// reach every row of the product; infinities and NaNs of the drafted tokens, rows
// [first, last), are taken out and noted in the poison of the rows that see the token.
// bad_rows is zero before and after.
template <int D, bool FP8, int NS>
FA_DEV void clean_values(uint32_t tile, int row, int first, int last, bool look, int group, const uint32_t* seen,
                         Poison<D>& poison, uint32_t* bad_rows, volatile uint32_t* bad_stage) {
  using C = TCfg<D, FP8, NS>;
  constexpr int GR = 128 / NS, U = D / 8;  // 16-byte units of a row
  constexpr uint32_t EXP = FP8 ? 0x7c00u : 0x7f80u, MANT = FP8 ? 0x03ffu : 0x007fu;
  auto unit = [&](int r, int u) {
    return tile + (u * 8 / C::CE) * (128 * C::SWB) + r * C::SWB + (((u % (C::CE / 8)) ^ swz_row<C::SWB>(r)) << 4);
  };
#pragma unroll 1
  for (int i = row; i < (128 - last) * U; i += 128) st_shared_v4(unit(last + i / U, i % U), make_uint4(0u, 0u, 0u, 0u));
  if (look) {
#pragma unroll 1
    for (int i = row; i < (last - first) * U; i += 128) {
      const int r = first + i / U;
      const uint4 v = ld_shared_v4(unit(r, i % U));
      const uint32_t x[4] = {v.x, v.y, v.z, v.w};
      bool bad = false;
#pragma unroll
      for (int e = 0; e < 4; ++e) bad |= (x[e] & EXP) == EXP || (x[e] & EXP << 16) == EXP << 16;
      if (bad) atomicOr(bad_rows + (r >> 5), 1u << (r & 31));
    }
  }
  fence_proxy_async_smem();  // the product reads what was written here
  named_bar_sync(1, 128);
  volatile uint32_t* words = bad_rows;
  if ((words[0] | words[1] | words[2] | words[3]) == 0) return;
#pragma unroll 1
  for (int i = 0; i < 128; ++i) {
    if (!((words[i >> 5] >> (i & 31)) & 1u)) continue;
    // row i's infinities and NaNs: out of the tile, into bad_stage, to the rows that see it
    if (row == i) {
#pragma unroll 1
      for (int k = 0; k < D / 32; ++k) {
        uint32_t pos = 0, neg = 0;
#pragma unroll 1
        for (int u = 4 * k; u < 4 * k + 4; ++u) {
          const uint4 v = ld_shared_v4(unit(row, u));
          uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t half = x[e / 2] >> (16 * (e & 1)) & 0xffffu;
            if ((half & EXP) == EXP) {
              const bool nan = (half & MANT) != 0;
              const uint32_t bit = 1u << ((u & 3) * 8 + e);
              if (nan || !(half >> 15)) pos |= bit;
              if (nan || half >> 15) neg |= bit;
              x[e / 2] &= ~(0xffffu << (16 * (e & 1)));
            }
          }
          st_shared_v4(unit(row, u), make_uint4(x[0], x[1], x[2], x[3]));
        }
        bad_stage[k] = pos;
        bad_stage[4 + k] = neg;
      }
      fence_proxy_async_smem();
    }
    named_bar_sync(1, 128);
    const int k = i - group * GR;
    bool sees = false;
#pragma unroll
    for (int e = 0; e < GR / 32; ++e)
      if (k >= 32 * e && k < 32 * e + 32) sees = seen[e] >> (k & 31) & 1u;
    if (sees) {
#pragma unroll
      for (int e = 0; e < D / 32; ++e) {
        poison.pos[e] |= bad_stage[e];
        poison.neg[e] |= bad_stage[4 + e];
      }
    }
    named_bar_sync(1, 128);
  }
  if (row < 4) words[row] = 0u;
}

template <int D, bool FP8, int NS>
__global__ void __launch_bounds__(TCfg<D, FP8, NS>::NTHREADS, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                const __grid_constant__ TreeArgs p) {
  using C = TCfg<D, FP8, NS>;
  constexpr int GR = 128 / NS;  // rows of a group, and keys each group weighs
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  const uint32_t sb = smem_u32(smem);
  auto bar = [&](int i) -> uint32_t { return sb + C::OFF_BAR + 8 * i; };
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  uint32_t* bad_rows = misc + 8;                                    // 4 words
  volatile uint32_t* bad_stage = misc + 12;                         // 8 words
  const Guard guard{p.status, abort_flag};
  const CacheView& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hms = c.Hk * p.M;

  pdl_trigger();  // the joining kernel may be made ready now; it waits for this one's end
  if (threadIdx.x < C::NBAR) {
    const int i = threadIdx.x;
    // one arrival for loads and commits, one for each of four warps elsewhere
    const bool four = i == C::B_QREADY || i == C::B_OFREE || i == C::B_MEET || (C::NW == 2 && i == C::B_LSUM);
    // (of all softmax warps, for the scores read and the weights written)
    const bool all = i >= C::B_SFREE && i < C::B_PFREE;
    // (and of two where the e4m3 tiles are converted, and between two softmax warps of the same rows)
    const bool two = (FP8 && ((i >= C::B_FULL && i < C::B_EMPTY) || (i >= C::B_REMPTY && i < C::B_SFULL))) ||
                     (i >= C::B_TOP && i < C::B_LSUM);
    mbar_init(bar(i), four ? 4 : all ? 4 * C::NW : two ? 2 : 1);
    fence_mbar_init();
  }
  if (threadIdx.x < 4) bad_rows[threadIdx.x] = 0u;
  if (warp == 1) {
    tmem_alloc(smem_u32(misc), C::TM_COLS);
    tmem_relinquish();
  }
  pdl_wait();  // everything from here on may be an earlier kernel's output
  if (threadIdx.x == 64) *abort_flag = (*reinterpret_cast<volatile int*>(p.status) != 0);
  const Run mine = find_run(c, p.B, hms, blockIdx.x, gridDim.x, lane);
  Walk w = mine.w;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  const bool skip = *abort_flag != 0 || !w.more();

  if (warp < 4) {
    if constexpr (C::R_ISSUE > 0) regs_dec<C::R_ISSUE>();
    if ((warp == 0 || warp == 3) && !skip) {
      // ---------------------------------------------------------------- producers: warp 0 K, warp 3 V
      const int kv = warp == 0 ? 0 : 1;
      const int rb = c.page < kKeys ? c.page : kKeys;  // rows of a box: a page, or a tile's share of one
      const int boxes = kKeys / rb;
      const int nowhere = c.pages * c.Hk;              // past the end: TMA fills zeros
      const CUtensorMap* map = kv ? &tmV : &tmK;
      const bool issues = lane < boxes;                // lane i looks up box i
      bool ok = true;
      constexpr int NR = FP8 ? C::NRAW : C::NSLOT, BFULL = FP8 ? C::B_RFULL : C::B_FULL,
                    BEMPTY = FP8 ? C::B_REMPTY : C::B_EMPTY;
      int items = 0, slot = kv;
      uint32_t parity = 1;  // (a fresh barrier's phase of parity 1 counts as complete: the first trips do not wait)
      while (ok && w.more()) {
        TableWindow table;
        table.open(c, w.b, w.t0 * kKeys, rb, lane);
        const int len = seq_len(c, w.b), h = p.M == 1 ? w.hm : w.hm / p.M;
        const int n = w.n();
        for (int j = 0; j < n; ++j) {
          const int tile = w.t0 + j;
          // this lane's box: z coordinate of its page and head
          const int page = table.take(c, w.b, boxes, rb, lane);
          const int z = issues && tile * kKeys + lane * rb < len && page >= 0 && page < c.pages ? page * c.Hk + h : nowhere;
          const int y = (tile * kKeys) & (c.page - 1);  // a tile's place in a page of more than a tile
          if (!(ok = mbar_rest_warp(bar(BEMPTY + slot), parity, guard, SITE_TREE_PRODUCER))) break;
          const uint32_t full = bar(BFULL + slot);
          const uint32_t dst = sb + (FP8 ? C::OFF_RAW + slot * C::RAW : C::OFF_T + slot * C::TILE);
          if constexpr (FP8) {
            const bool there = issues && z != nowhere;
            const int n_there = __popc(__ballot_sync(0xffffffffu, there));
            if (kv == 0 && issues && !there) {  // no page, no exponents: 2^-127
              const uint32_t exps = dst + 128 * D + lane * rb;
              for (int k = 0; k < rb; k += 16) {
                st_shared_v4(exps + k, make_uint4(0u, 0u, 0u, 0u));
                st_shared_v4(exps + 128 + k, make_uint4(0u, 0u, 0u, 0u));
              }
              fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_expect_tx(full, 128 * D + (kv == 0 ? 2 * n_there * rb : 0));
            const unsigned long long at = static_cast<unsigned long long>(z) * c.page + y;
            // Each lane issues its own box.  With lane 0 issuing all of them in turn the loads of K and the exponents
            // bound the kernel: 119.4 us where this takes 113.0 (16 sequences up to 32768, e4m3), 81.3 where 77.0 (63
            // drafts).
            __syncwarp();
            if (issues) {
              tma_load_3d(dst + lane * rb * D, map, full, 0, y, z);
              if (kv == 0 && there) {
                bulk_load(dst + 128 * D + lane * rb, c.Ke + at, rb, full);
                bulk_load(dst + 128 * D + 128 + lane * rb, c.Ve + at, rb, full);
              }
            }
          } else {
            if (lane == 0) mbar_expect_tx(full, C::TILE);
            __syncwarp();
            if (issues) {
#pragma unroll
              for (int ch = 0; ch < D / C::CE; ++ch)
                tma_load_3d(dst + ch * 128 * C::SWB + lane * rb * C::SWB, map, full, ch * C::CE, y, z);
            }
          }
          ++items;
          if ((slot += 2) >= NR) slot -= NR, parity ^= 1;
        }
        if (!ok) break;
        w.next(c, hms);
      }
      if (*abort_flag && lane == 0) {
        // gave up: let every load this warp started land before the CTA exits
        for (int i = items > NR / 2 ? items - NR / 2 : 0; i < items; ++i)
          mbar_drain(bar(BFULL + (2 * i + kv) % NR), ((2 * i + kv) / NR) & 1);
      }
    } else if (warp == 1 && lane == 0 && !skip) {
      // ---------------------------------------------------------------- UMMA issuer: S = Q (tensor memory) x K
      constexpr uint32_t idS = FP8 ? idesc_f16(128, kKeys, false, false) : idesc_bf16(128, kKeys, false, false);
      bool ok = true;
      int seg = 0, b = 0, s = 0;
      uint32_t bpar = 1, spar = 0;
      for (; ok && w.more(); ++seg) {
        const int n = w.n();
        if (!(ok = mbar_rest(bar(C::B_QREADY), seg & 1, guard, SITE_TREE_MMA))) break;
        for (int j = 0; j < n; ++j) {
          // the scores that were in S buffer b have been read
          if (!(ok = mbar_rest(bar(C::B_SFREE + b), bpar, guard, SITE_TREE_MMA))) break;
          if (!(ok = mbar_rest(bar(C::B_FULL + s), spar, guard, SITE_TREE_MMA))) break;
          tc_fence_after();
          const uint32_t kb = sb + C::OFF_T + s * C::TILE;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            mma_ts(tmem + C::TM_S0 + b * 128, tmem + C::TM_Q + ks * 8, sdesc_kmajor<C::SWB, 128>(kb, ks), idS, ks > 0);
          mma_commit(bar(C::B_SFULL + b));
          mma_commit(bar(C::B_EMPTY + s));
          if (++b == C::NSB) b = 0, bpar ^= 1;
          if ((s += 2) >= C::NSLOT) s -= C::NSLOT, spar ^= 1;
        }
        if (!ok) break;
        w.next(c, hms);
      }
      mma_commit(bar(C::B_SDONE));  // drain point for teardown
    } else if (warp == 2 && lane == 0 && !skip) {
      // ---------------------------------------------------------------- UMMA issuer: O += P V
      constexpr uint32_t idO = FP8 ? idesc_f16(128, D, false, true) : idesc_bf16(128, D, false, true);
      bool ok = true;
      int seg = 0, b = 0, s = 1;
      uint32_t bpar = 0, spar = 0;
      for (; ok && w.more(); ++seg) {
        const int n = w.n();
        for (int j = 0; j < n; ++j) {
          if (!(ok = mbar_rest(bar(C::B_PFULL + b), bpar, guard, SITE_TREE_MMA))) break;
          if (!(ok = mbar_rest(bar(C::B_FULL + s), spar, guard, SITE_TREE_MMA))) break;
          // a unit's first product overwrites O: the epilogue before it has read it
          if (j == 0 && seg > 0 && !(ok = mbar_rest(bar(C::B_OFREE), (seg - 1) & 1, guard, SITE_TREE_MMA))) break;
          tc_fence_after();
          const uint32_t vb = sb + C::OFF_T + s * C::TILE, aP = tmem + C::TM_P0 + b * 64;
#pragma unroll
          for (int ks = 0; ks < kKeys / 16; ++ks)
            mma_ts(tmem + C::TM_O, aP + ks * 8, sdesc_mnmajor<C::SWB, 128>(vb, ks), idO, (j > 0 || ks > 0));
          mma_commit(bar(C::B_EMPTY + s));
          mma_commit(bar(C::B_PFREE + b));
          if (++b == C::NPB) b = 0, bpar ^= 1;
          if ((s += 2) >= C::NSLOT) s -= C::NSLOT, spar ^= 1;
        }
        if (!ok) break;
        mma_commit(bar(C::B_OFULL));
        w.next(c, hms);
      }
      mma_commit(bar(C::B_PVDONE));  // every S completed before its P: the end of all UMMAs
    }
  } else if (warp < 4 + 4 * C::NW) {
    if constexpr (C::R_SOFT > 0) regs_inc<C::R_SOFT>();
    if (!skip) {
      // ---------------------------------------------------------------- softmax + epilogue
      // With two warpgroups, warps w and w + 4 have the same rows and each half of the columns.  They agree on a
      // tile's largest score (B_TOP) and so always have the same reference; the first warpgroup (`lead`) also takes
      // Q, cleans values and stores the results.
      const int wq = warp & 3, row = wq * 32 + lane;
      const int wg = C::NW == 2 ? (warp - 4) >> 2 : 0;
      const bool lead = C::NW == 1 || wg == 0;
      constexpr int COLS = GR / C::NW;              // columns of a thread
      const int group = row / GR, r_in = row % GR;  // key group, row of the query tile
      const int col0 = group * GR + wg * COLS;
      const uint32_t tl = tmem + (static_cast<uint32_t>(wq * 32) << 16);
      const int tid = threadIdx.x - 128;
      float* rows = reinterpret_cast<float*>(smem + C::OFF_ROWS);
      float4* xch = reinterpret_cast<float4*>(smem + C::OFF_X);
      const int boxes = c.page < kKeys ? kKeys / c.page : 1;
      const uint32_t all_boxes = boxes == 1 ? 1u : (1u << boxes) - 1u;
      bool ok = true;
      int seg = 0, b = 0, pb = 0, vs_slot = 1, sc = 0;  // S buffer, P buffer, slot of V, scales
      uint32_t bpar = 0, pfree = 1, vpar = 0, meet_parity = 0;
      [[maybe_unused]] uint32_t top_parity = 0;
      // The four softmax warps meet; a wait with a limit.  It does not look at the abort flag, so that
      // either all four pass or none does, and what follows may use plain barriers.
      auto meet = [&]() -> bool {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::B_MEET));
        const uint64_t t0 = gtimer_ns();
        bool all;
        while (!(all = mbar_try_rest(bar(C::B_MEET), meet_parity)) && gtimer_ns() - t0 <= 2 * kWaitLimitNs) {
        }
        meet_parity ^= 1;
        return __all_sync(0xffffffffu, all);
      };
      // This thread's row of a unit's Q into tensor memory; q_scale: what its scores are multiplied by.
      // For an e4m3 cache the row becomes f16, scaled by a power of two to a maximum in [2^14, 2^15): elements
      // of 2^-31 of the maximum and more keep all their bits.
      float q_scale = 0.f;
      [[maybe_unused]] float* q_scales = reinterpret_cast<float*>(smem + C::OFF_TOPS) + 512;
      auto take_q = [&](const Walk& at) {
        if (!lead) return;
        const int h = p.M == 1 ? at.hm : at.hm / p.M, q = (at.hm - h * p.M) * 128 + r_in;
        uint4 x[D / 8];
        const uint4* src =
            reinterpret_cast<const uint4*>(p.Q + ((static_cast<size_t>(at.b) * c.Hk + h) * p.R + (q < p.R ? q : 0)) * D);
#pragma unroll
        for (int u = 0; u < D / 8; ++u) x[u] = src[u];  // (rows that are not there: any row, never stored)
        float mul = 1.f;
        q_scale = p.c_log2;
        if constexpr (FP8) {
          uint32_t m = 0;
#pragma unroll
          for (int u = 0; u < D / 8; ++u) {
            const uint4 v = x[u];
            const uint32_t k = 0x7fff7fffu;
            m = __vmaxu2(m, __vmaxu2(__vmaxu2(v.x & k, v.y & k), __vmaxu2(v.z & k, v.w & k)));
          }
          int e = static_cast<int>(max(m & 0xffffu, m >> 16) >> 7);  // biased exponent of the largest
          e = e < 15 ? 15 : e;
          mul = __int_as_float((268 - e) << 23);                     // 2^(14 - (e - 127))
          q_scale = p.c_log2 * __int_as_float((e - 14) << 23);
        }
        if (C::NW == 2) q_scales[row] = q_scale;
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          uint32_t o[16];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t v[4] = {x[4 * k + i].x, x[4 * k + i].y, x[4 * k + i].z, x[4 * k + i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              o[4 * i + e] = FP8 ? pack_f16x2(__uint_as_float(v[e] << 16) * mul,
                                              __uint_as_float(v[e] & 0xffff0000u) * mul)
                                 : v[e];
          }
          tmem_st16(tl + C::TM_Q + 16 * k, o);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::B_QREADY));
      };
      // The other groups' weights are zero, for good: a tile writes its own group's columns only.
      if constexpr (NS > 1) {
        uint32_t zero[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) zero[k] = 0u;
#pragma unroll
        for (int k = 0; k < C::NPB * 4; ++k) tmem_st16(tl + C::TM_P0 + 16 * k, zero);
      }
      take_q(w);
      // What a unit starts with is loaded before the epilogue of the one before it
      // (as it is in memory, so that the loads are all under way at once).
      auto new_of = [&](int i) { return c.n_new == nullptr ? c.T : c.n_new[i]; };
      int raw_len = c.lens[w.b], raw_new = new_of(w.b);
      TableWindow table;
      table.open(c, w.b, w.t0 * kKeys, kKeys / boxes, lane);
      for (; ok && w.more(); ++seg) {
        const int n = w.n();
        const int h = p.M == 1 ? w.hm : w.hm / p.M, mt = w.hm - h * p.M;
        const int q = mt * 128 + r_in, t = q % c.T;
        const int len = clamp_len(c, raw_len), nn = clamp_new(c, raw_new), prefix = max(raw_len, 0) - nn;
        const int inside = min(prefix, len);  // keys below it are seen by every live row
        const bool live = q < p.R && t < nn;  // rows that are not there see nothing
        const bool warp_live = mt * 128 + (wq * 32) % GR < p.R;
        const unsigned long long* trow =
            p.tree == nullptr ? nullptr : p.tree + w.b * p.tree_stride + static_cast<size_t>(t) * p.words;
        // The scale of its row, from the first warpgroup.  Only a warp with rows may wait here: the first warpgroup
        // meets its partner in every tile (B_TOP), so Q's next phase cannot end before this wait has seen its own.  A
        // warp without rows holds nobody up; it could find that phase passed already and would wait for one that never
        // comes.  (It has no use for the scale, and S of each unit it goes through was made after that unit's Q, so
        // that when it has rows again it is no phase behind either.)
        if (!lead && warp_live) {
          if (!(ok = mbar_rest_warp(bar(C::B_QREADY), seg & 1, guard, SITE_TREE_SOFTMAX))) break;
          q_scale = q_scales[row];
        }
        const float rq = q_scale;
        float ref = -INFINITY, l = 0.f, lr = 0.f;  // reference, sum of weights, sum of weights as rounded
        Poison<D> poison;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) poison.pos[i] = poison.neg[i] = 0u;
        for (int j = 0; j < n; ++j) {
          const int k0 = (w.t0 + j) * kKeys;
          // bit i: box i's page exists
          const int page = table.take(c, w.b, boxes, kKeys / boxes, lane);
          const uint32_t pm =
              __ballot_sync(0xffffffffu, lane < boxes && k0 + lane * (kKeys / boxes) < len && page >= 0 && page < c.pages);
          const bool edge = k0 + kKeys > inside || pm != all_boxes;
          uint32_t seen[GR / 32];  // this row's keys of its group, 32 a word
          if (edge) {
#pragma unroll
            for (int i = 0; i < GR / 32; ++i) {
              const int off = group * GR + 32 * i, j0 = k0 + off;
              uint32_t m = low_bits(inside - j0);
              if (j0 + 32 > prefix) m |= draft_bits(trow, p.words, t, j0 - prefix);
              m &= low_bits(len - j0);
              const int bx = off * boxes / kKeys;
              uint32_t in_page = (pm >> bx) & 1u ? 0xffffffffu : 0u;
              if (boxes == 8) in_page = (in_page & 0xffffu) | ((pm >> (bx + 1)) & 1u ? 0xffff0000u : 0u);  // pages of 16
              seen[i] = live ? m & in_page : 0u;
            }
          }
          if (!(ok = mbar_rest_warp(bar(C::B_SFULL + b), bpar, guard, SITE_TREE_SOFTMAX))) break;
          tc_fence_after();
          if (warp_live) {
            uint32_t r[COLS];
            float s[COLS];
#pragma unroll
            for (int i = 0; i < COLS / 32; ++i) tmem_ld32(tl + C::TM_S0 + b * 128 + col0 + 32 * i, r + 32 * i);
            tmem_ld_wait<COLS>(r);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::B_SFREE + b));
            // scores in base-2 units, and for each row the largest of what decides the weights' range
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            const float* scales = reinterpret_cast<const float*>(smem + C::OFF_SCALE) + sc * 384 + col0;
            if constexpr (FP8) {
#pragma unroll
              for (int k = 0; k < COLS; k += 4) {
                const float4 ks = *reinterpret_cast<const float4*>(scales + k);
                const uint64_t a = fmul2(f2pack(__uint_as_float(r[k]), __uint_as_float(r[k + 1])), f2pack(rq, rq));
                const uint64_t bb = fmul2(f2pack(__uint_as_float(r[k + 2]), __uint_as_float(r[k + 3])), f2pack(rq, rq));
                f2unpack(fmul2(a, f2pack(ks.x, ks.y)), s[k], s[k + 1]);
                f2unpack(fmul2(bb, f2pack(ks.z, ks.w)), s[k + 2], s[k + 3]);
              }
            } else {
#pragma unroll
              for (int k = 0; k < COLS; ++k) s[k] = __uint_as_float(r[k]);
            }
            if (edge) {
#pragma unroll
              for (int k = 0; k < COLS; ++k)
                if (!(((wg == 0 ? seen[k / 32] : seen[(COLS * (C::NW - 1) + k) / 32]) >> (k & 31)) & 1u)) s[k] = -INFINITY;
            }
#pragma unroll
            for (int k = 0; k < COLS; k += 8) {
              float v[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = s[k + e];
              if constexpr (FP8) {
                const float4 a = *reinterpret_cast<const float4*>(scales + 256 + k);
                const float4 bb = *reinterpret_cast<const float4*>(scales + 256 + k + 4);
                f2unpack(fadd2(f2pack(v[0], v[1]), f2pack(a.x, a.y)), v[0], v[1]);
                f2unpack(fadd2(f2pack(v[2], v[3]), f2pack(a.z, a.w)), v[2], v[3]);
                f2unpack(fadd2(f2pack(v[4], v[5]), f2pack(bb.x, bb.y)), v[4], v[5]);
                f2unpack(fadd2(f2pack(v[6], v[7]), f2pack(bb.z, bb.w)), v[6], v[7]);
              }
#pragma unroll
              for (int e = 0; e < 4; ++e) top[e] = fmax3(top[e], v[2 * e], v[2 * e + 1]);
            }
            float tile_top = fmaxf(fmax3(top[0], top[1], top[2]), top[3]);
            if constexpr (C::NW == 2) {  // both halves' largest
              float* tops = reinterpret_cast<float*>(smem + C::OFF_TOPS) + top_parity * 256;
              tops[wg * 128 + row] = tile_top;
              __syncwarp();
              if (lane == 0) mbar_arrive(bar(C::B_TOP + wq));
              if (!(ok = mbar_rest_warp(bar(C::B_TOP + wq), top_parity, guard, SITE_TREE_SOFTMAX))) break;
              tile_top = fmaxf(tile_top, tops[(1 - wg) * 128 + row]);
              top_parity ^= 1;
            }
            if constexpr (!FP8) tile_top *= p.c_log2;
            constexpr float kStart = FP8 ? -kF16Start : kFwdMaxHeadroom, kMove = FP8 ? kF16Top : kFwdRescaleThreshold;
            if (j == 0) {
              ref = tile_top + kStart;
            } else {
              const bool move = tile_top > ref + kMove;
              if (__any_sync(0xffffffffu, move)) {
                const float new_ref = tile_top + kStart;
                const float alpha = move ? ex2(ref - new_ref) : 1.f;
                if (move) {
                  l = rescaled<FP8>(l, ref, new_ref), lr = FP8 ? l : rescaled<FP8>(lr, ref, new_ref);
                  ref = new_ref;
                }
                // the product that last wrote O is done
                const int last = pb == 0 ? C::NPB - 1 : pb - 1;
                if (!(ok = mbar_rest_warp(bar(C::B_PFREE + last), C::NPB == 1 || pb != 0 ? pfree ^ (C::NPB > 1) : pfree, guard,
                                          SITE_TREE_SOFTMAX)))
                  break;
                tc_fence_after();
#pragma unroll 1
                for (int i = wg; i < D / 32; i += C::NW) {
                  uint32_t o[32];
                  tmem_ld32(tl + C::TM_O + 32 * i, o);
                  tmem_ld_wait<32>(o);
#pragma unroll
                  for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                  tmem_st32(tl + C::TM_O + 32 * i, o);
                }
                tmem_st_wait();
              }
            }
            const float neg = ref == -INFINITY ? 0.f : -ref;  // nothing seen so far: every weight is 0
            const uint64_t neg2 = f2pack(neg, neg), cc2 = f2pack(p.c_log2, p.c_log2);
            uint64_t ls[2] = {f2pack(0.f, 0.f), f2pack(0.f, 0.f)};
            float rl[2] = {0.f, 0.f}, rh[2] = {0.f, 0.f};
            // 32 keys at a time: few registers
#pragma unroll
            for (int k0c = 0; k0c < COLS; k0c += 32) {
              uint32_t pk[16];
#pragma unroll
              for (int k = k0c; k < k0c + 32; k += 4) {
                uint64_t vsc[2];
                if constexpr (FP8) {
                  const float4 a = *reinterpret_cast<const float4*>(scales + 128 + k);
                  vsc[0] = f2pack(a.x, a.y), vsc[1] = f2pack(a.z, a.w);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const uint64_t x = f2pack(s[k + 2 * e], s[k + 2 * e + 1]);
                  float t0, t1;
                  f2unpack(FP8 ? fadd2(x, neg2) : ffma2(x, cc2, neg2), t0, t1);
                  const uint64_t w2 = f2pack(ex2(t0), ex2(t1));
                  ls[e] = fadd2(ls[e], w2);
                  const int at = (k - k0c) / 2 + e;
                  float p0, p1;
                  if constexpr (FP8) {
                    f2unpack(fmul2(w2, vsc[e]), p0, p1);
                    pk[at] = pack_f16x2(p0, p1);
                  } else {
                    f2unpack(w2, p0, p1);
                    pk[at] = pack_bf16x2(p0, p1);
                    add_bf16x2_f32(pk[at], rl[e], rh[e]);
                  }
                }
              }
              if (k0c == 0) {  // the product that read this P buffer is done
                if (!(ok = mbar_rest_warp(bar(C::B_PFREE + pb), pfree, guard, SITE_TREE_SOFTMAX))) break;
                tc_fence_after();
              }
              tmem_st16(tl + C::TM_P0 + pb * 64 + (col0 + k0c) / 2, pk);
            }
            if (!ok) break;
            float a0, a1;
            f2unpack(fadd2(ls[0], ls[1]), a0, a1);
            l += a0 + a1;
            // bf16 weights are normalised by their own sum; f16 ones are off by 2^-11 at most
            lr = FP8 ? l : lr + (rl[0] + rl[1]) + (rh[0] + rh[1]);
            tmem_st_wait();
          } else {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::B_SFREE + b));
            // no rows, no weights; but without this wait its arrival below could count for an earlier tile's
            if (!(ok = mbar_rest_warp(bar(C::B_PFREE + pb), pfree, guard, SITE_TREE_SOFTMAX))) break;
          }
          if (lead && k0 + kKeys > inside) {  // the tile holds drafted tokens or rows behind the end
            if (!(ok = mbar_rest_warp(bar(C::B_FULL + vs_slot), vpar, guard, SITE_TREE_SOFTMAX)) || !(ok = meet())) break;
            // (a single token sees itself, or its row sees nothing at all: its values need no look)
            clean_values<D, FP8, NS>(sb + C::OFF_T + vs_slot * C::TILE, row, max(inside - k0, 0),
                                     min(max(len - k0, 0), 128), c.T > 1 || p.tree != nullptr, group, seen, poison,
                                     bad_rows, bad_stage);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::B_PFULL + pb));
          if (++b == C::NSB) b = 0, bpar ^= 1;
          if (++pb == C::NPB) pb = 0, pfree ^= 1;
          if ((vs_slot += 2) >= C::NSLOT) vs_slot -= C::NSLOT, vpar ^= 1;
          if (FP8 && ++sc == C::NSC) sc = 0;
        }
        if (!ok) break;
        // ------------------------------------------------------------ this run's part of the unit is done
        const Walk at = w;
        w.next(c, hms);
        if (w.more()) {
          raw_len = c.lens[w.b], raw_new = new_of(w.b);
          table.open(c, w.b, w.t0 * kKeys, kKeys / boxes, lane);
          take_q(w);  // the next unit's S may be formed meanwhile
        }
        if constexpr (C::NW == 2) {
          // the second warpgroup's sums, for the first; before the next ones it waits until these have been read
          if (!lead) {
            if (seg > 0 && !(ok = mbar_rest_warp(bar(C::B_OFREE), (seg - 1) & 1, guard, SITE_TREE_SOFTMAX))) break;
            rows[128 + row] = l;
            rows[256 + row] = lr;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::B_LSUM));
            continue;
          }
          if (!(ok = mbar_rest_warp(bar(C::B_LSUM), seg & 1, guard, SITE_TREE_SOFTMAX))) break;
          l += rows[128 + row];
          lr += rows[256 + row];
        }
        if (!(ok = mbar_rest_warp(bar(C::B_OFULL), seg & 1, guard, SITE_TREE_SOFTMAX)) || !(ok = meet())) break;
        tc_fence_after();
        const bool whole = at.t0 == 0 && n == at.nt;
        if (at.t0 == 0 && tid == 0) {
          const long long first = mine.lo + mine.mine - at.left + at.cost;  // the place of the unit's first tile
          p.info[static_cast<long long>(at.b) * hms + at.hm] =
              UnitInfo{static_cast<int>(blockIdx.x), static_cast<int>(quotient(first + at.nt - 1, mine.run))};
        }
        // a NaN score does not move the maximum: where nothing else is seen it is still -inf
        if (lr != lr) ref = lr;
        if (!live) ref = -INFINITY, l = lr = 0.f;  // whatever its lane computed
        float* slot = p.part + (2 * static_cast<size_t>(blockIdx.x) + (at.t0 == 0 ? 1 : 0)) * p.rows * (D + 3);
        float* sums = slot + static_cast<size_t>(p.rows) * D;
        const size_t row0 = (static_cast<size_t>(at.b) * c.Hk + h) * p.R + mt * 128;  // the query tile's first row
        // 32 columns of this thread's O at a time.  Loops stay loops: the code runs once per unit, and fetching
        // unrolled code costs more than running it.
        auto load_o = [&](int i, uint32_t (&o)[32]) {
          tmem_ld32(tl + C::TM_O + 32 * i, o);
          tmem_ld_wait<32>(o);
          uint32_t pp = 0, pn = 0;
#pragma unroll
          for (int e = 0; e < D / 32; ++e)
            if (e == i) pp = poison.pos[e], pn = poison.neg[e];
          if (pp | pn) {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const bool a = pp >> e & 1u, d = pn >> e & 1u;
              if (a || d)
                o[e] = __float_as_uint(__uint_as_float(o[e]) +
                                       (a && d ? __int_as_float(0x7fffffff) : a ? INFINITY : -INFINITY));
            }
          }
        };
        if constexpr (NS == 1) {
          const int wrow = wq * 32, nvalid = p.R - mt * 128 - wrow;  // the warp's rows, stored whole rows at a time
          const float inv = lr == 0.f ? 0.f : 1.f / lr;
#pragma unroll 1
          for (int i = 0; i < D / 32; ++i) {
            uint32_t o[32];
            load_o(i, o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = lr == 0.f ? 0u : o[e];
            if (whole) {
              uint32_t pk[16];
#pragma unroll
              for (int e = 0; e < 16; ++e)
                pk[e] = pack_bf16x2(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
              warp_store_rows<4, 0>(pk, reinterpret_cast<uint8_t*>(p.O + (row0 + wrow) * D + 32 * i), D * 2, nvalid, lane);
            } else {
              warp_store_rows<8, 0>(o, reinterpret_cast<uint8_t*>(slot + static_cast<size_t>(wrow) * D + 32 * i), D * 4,
                                    nvalid, lane);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::B_OFREE));
          if (lane < nvalid) {
            if (whole) p.L[row0 + row] = lr == 0.f ? -INFINITY : (ref + lg2(l)) * kFwdLn2;
            else sums[row] = ref, sums[p.rows + row] = l, sums[2 * p.rows + row] = lr;
          }
        } else {
          // The groups' rows are added up through shared memory, XR rows at a time: every thread then has EPT
          // elements of one of them.
          constexpr int XR = 16384 / (NS * D * 4), TPR = 128 / XR, EPT = D / TPR;
          static_assert(EPT % 8 == 0, "whole 16-byte pieces of O");
          rows[row] = ref;
          rows[128 + row] = l;
          rows[256 + row] = lr;
          named_bar_sync(1, 128);
          float mx = -INFINITY;
#pragma unroll
          for (int g = 0; g < NS; ++g) mx = fmaxf(mx, rows[g * GR + r_in]);
          const float f = ref == -INFINITY ? 0.f : ex2(ref - mx);  // this group's share in the row's common reference
          const int n_rows = min(GR, p.R - mt * 128);
#pragma unroll 1
          for (int x0 = 0; x0 < n_rows; x0 += XR) {
            if (x0 > 0) named_bar_sync(1, 128);  // the rows before have been read
            const int xr = r_in - x0;
            const bool mine_now = xr >= 0 && xr < XR;
            if (__any_sync(0xffffffffu, mine_now)) {
              float4* dst = xch + (group * XR + (xr & (XR - 1))) * (D / 4);
#pragma unroll 1
              for (int i = 0; i < D / 32; ++i) {
                uint32_t o[32];
                load_o(i, o);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  float4 v;
                  v.x = f == 0.f ? 0.f : __uint_as_float(o[4 * k]) * f;
                  v.y = f == 0.f ? 0.f : __uint_as_float(o[4 * k + 1]) * f;
                  v.z = f == 0.f ? 0.f : __uint_as_float(o[4 * k + 2]) * f;
                  v.w = f == 0.f ? 0.f : __uint_as_float(o[4 * k + 3]) * f;
                  if (mine_now) dst[8 * i + (k ^ (xr & 7))] = v;
                }
              }
            }
            if (x0 + XR >= n_rows) {  // O has been read
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(bar(C::B_OFREE));
            }
            named_bar_sync(1, 128);
            const int orow = x0 + tid / TPR, part = tid % TPR;
            if (orow < n_rows) {
              float om = -INFINITY, ol = 0.f, olr = 0.f;
#pragma unroll
              for (int g = 0; g < NS; ++g) om = fmaxf(om, rows[g * GR + orow]);
#pragma unroll
              for (int g = 0; g < NS; ++g) {
                const float mg = rows[g * GR + orow];
                ol += rescaled<FP8>(rows[128 + g * GR + orow], mg, om);
                olr += rescaled<FP8>(rows[256 + g * GR + orow], mg, om);
              }
              if (olr != olr) om = olr;  // so that the join keeps the row
              float a[EPT];
#pragma unroll
              for (int k = 0; k < EPT / 4; ++k) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                const int piece = (k / 2 * TPR + part) * 2 + (k & 1);  // eight elements here, eight TPR * 8 on
#pragma unroll
                for (int g = 0; g < NS; ++g) {
                  const float4 y = xch[(g * XR + tid / TPR) * (D / 4) + (piece ^ ((tid / TPR) & 7))];
                  v.x += y.x, v.y += y.y, v.z += y.z, v.w += y.w;
                }
                a[4 * k] = v.x, a[4 * k + 1] = v.y, a[4 * k + 2] = v.z, a[4 * k + 3] = v.w;
              }
              const float inv = olr == 0.f ? 0.f : 1.f / olr;
              if (whole) {
                if constexpr (!FP8) {
                  bool nan = false;
#pragma unroll
                  for (int k = 0; k < EPT; ++k) nan |= a[k] != a[k];
                  // (the unit's own entry has been written before the barriers above)
                  if (nan && olr == olr)
                    p.info[static_cast<long long>(at.b) * hms + at.hm].first = static_cast<int>(blockIdx.x) | kNanUnit;
                }
                uint4* dst = reinterpret_cast<uint4*>(p.O + (row0 + orow) * D) + part;
#pragma unroll
                for (int k = 0; k < EPT / 8; ++k)
                  dst[k * TPR] = make_uint4(pack_bf16x2(a[8 * k] * inv, a[8 * k + 1] * inv),
                                      pack_bf16x2(a[8 * k + 2] * inv, a[8 * k + 3] * inv),
                                      pack_bf16x2(a[8 * k + 4] * inv, a[8 * k + 5] * inv),
                                      pack_bf16x2(a[8 * k + 6] * inv, a[8 * k + 7] * inv));
                if (part == 0) p.L[row0 + orow] = olr == 0.f ? -INFINITY : (om + lg2(ol)) * kFwdLn2;
              } else {
                float4* dst = reinterpret_cast<float4*>(slot + static_cast<size_t>(orow) * D) + 2 * part;
#pragma unroll
                for (int k = 0; k < EPT / 4; ++k)
                  dst[k / 2 * TPR * 2 + (k & 1)] = make_float4(a[4 * k], a[4 * k + 1], a[4 * k + 2], a[4 * k + 3]);
                if (part == 0) sums[orow] = om, sums[p.rows + orow] = ol, sums[2 * p.rows + orow] = olr;
              }
            }
          }
          named_bar_sync(1, 128);  // rows and the exchange are free again
        }
      }
    }
  } else if constexpr (FP8) {
    regs_dec<kConvertRegs>();
    if (!skip) {
      // ---------------------------------------------------------------- e4m3 -> f16 tiles
      // Pairs of warps take a tile each: K and V, and with two pairs for each of them every other one, so that four
      // tiles are under way at once, as most of a tile's time is waits (its barriers, the fence).
      const int cw = warp - 4 - 4 * C::NW, kv = (cw >> 1) & 1, half = cw >> 2, tid = threadIdx.x & 63;
      constexpr int PPR = D / 16, NP = 2 * PPR;  // 16-byte pieces of an e4m3 row; of a thread
      // A loop of a few parts, for short code and few registers: 1 / 2 / 4 parts, 16 sequences of a token each 115.4 /
      // 113.1 / 114.5 us, 63 drafts (one pair of warps) 83.1 / 79.4 / 77.0.
      constexpr int PARTS = C::NPAIR == 1 ? 4 : 2, STEPS = NP / PARTS;
      // Piece `sub` of rows (i * STEPS + k) * ROWS + row.  Eight lanes read 128 bytes of different banks and write 16-byte
      // units of different banks: at d = 128 (two chunks, 8 pieces a row) lanes 4..7 of eight take the upper half of
      // the neighbouring row, whose swizzle differs in the lowest bit.
      constexpr int ROWS = 64 / PPR;
      const int sub = tid % PPR;
      const int row = PPR == 8 ? (tid >> 4) * 2 + (((tid >> 2) ^ (tid >> 3)) & 1) : tid / PPR;
      const uint32_t sw = swz_row<C::SWB>(row);
      const uint32_t u0 = sub * 16 % C::CE / 8;
      const uint32_t to = (sub * 16 / C::CE) * (128 * C::SWB) + row * C::SWB;
      const uint32_t to0 = to + ((u0 ^ sw) << 4), to1 = to + (((u0 + 1) ^ sw) << 4);
      static_assert(ROWS % 8 == 0, "steps keep the swizzle");
      bool ok = true;
      int rs = 2 * half + kv, s = 2 * half + kv, sc = half;  // slots of the rings
      uint32_t rpar = 0, spar = 1;
      int skip_tiles = half;  // the other pair's, before the next of this one's
      for (; ok && w.more(); w.next(c, hms)) {
        const int n = w.n();
        int j = skip_tiles;
        for (; j < n; j += C::NPAIR) {
          if (!(ok = mbar_rest_warp(bar(C::B_RFULL + rs), rpar, guard, SITE_TREE_CONVERT))) break;
          const uint32_t raw = sb + C::OFF_RAW + rs * C::RAW, dst = sb + C::OFF_T + s * C::TILE;
          int ek = 0, ev = 0;
          if (kv == 0) {
            const uint16_t* exps = reinterpret_cast<const uint16_t*>(smem + C::OFF_RAW + rs * C::RAW + 128 * D);
            ek = exps[tid], ev = exps[64 + tid];  // two keys' each
          }
          if (!(ok = mbar_rest_warp(bar(C::B_EMPTY + s), spar, guard, SITE_TREE_CONVERT))) break;
          if (kv == 0) {
            // The tile's scales, for the softmax warps.  This slot held K tile x - NSLOT / 2, whose S is done; so it was
            // begun, and the scores of tile x - NSLOT / 2 - NSB had been taken out of its S buffer.  That tile's weights
            // may still be in the making: it and the NSLOT / 2 + NSB - 1 tiles behind it are not overwritten.
            float2* scale = reinterpret_cast<float2*>(smem + C::OFF_SCALE + sc * 1536) + tid;
            // (a row that holds NaN has NaN elements: its scale is 1)
            // (bytes below kExpMin are of rows never written, a fresh cache's zeros: with an exponent below -100
            // their unscaled weights would pass fp32's range)
            auto power = [](int e) { return e == kExpNaN ? 1.f : __int_as_float(max(e, kExpMin) << 23); };
            auto exponent = [](int e) { return e == kExpNaN ? 0.f : static_cast<float>(max(e, kRangeMin) - 127); };
            scale[0] = make_float2(power(ek & 255), power(ek >> 8));
            scale[64] = make_float2(power(ev & 255), power(ev >> 8));
            scale[128] = make_float2(exponent(ev & 255), exponent(ev >> 8));
            if ((sc += C::NPAIR) >= C::NSC) sc -= C::NSC;
          }
#pragma unroll 1
          for (int i = 0; i < PARTS; ++i) {
            const uint32_t from = raw + (i * STEPS * ROWS + row) * D + sub * 16, part = dst + i * STEPS * ROWS * C::SWB;
            uint4 x[STEPS];
#pragma unroll
            for (int k = 0; k < STEPS; ++k) x[k] = ld_shared_v4(from + k * ROWS * D);
#pragma unroll
            for (int k = 0; k < STEPS; ++k) {
              const uint32_t w4[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
              uint32_t o[8];
#pragma unroll
              for (int q = 0; q < 4; ++q) e4m3x4_to_f16x4(w4[q], o[2 * q], o[2 * q + 1]);
              st_shared_v4(part + to0 + k * ROWS * C::SWB, make_uint4(o[0], o[1], o[2], o[3]));
              st_shared_v4(part + to1 + k * ROWS * C::SWB, make_uint4(o[4], o[5], o[6], o[7]));
            }
          }
          // Only now that every loaded value has been used may the next e4m3 tile come.  Its TMA writes are of the
          // async proxy, which an arrival does not hold back behind loads that are still in flight: with the arrival
          // straight after the loads, 125 of 2500 calls of 1400 short tiles each had rows taken from a later tile.
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::B_REMPTY + rs));
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::B_FULL + s));
          if ((rs += 2 * C::NPAIR) >= C::NRAW) rs -= C::NRAW, rpar ^= 1;
          if ((s += 2 * C::NPAIR) >= C::NSLOT) s -= C::NSLOT, spar ^= 1;
        }
        if (!ok) break;
        skip_tiles = j - n;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    if (!skip && *abort_flag) {
      if (lane == 0) {
        mbar_drain(bar(C::B_SDONE), 0);
        mbar_drain(bar(C::B_PVDONE), 0);
      }
      __syncwarp();
    }
    tc_fence_after();
    tmem_dealloc(tmem, C::TM_COLS);
  }
}

// Signs of 8 bf16 values: bit e for +inf in element e, bit 8 + e for -inf (a NaN counts as both).
FA_DEV uint32_t infinities(uint4 v) {
  const uint32_t x[4] = {v.x, v.y, v.z, v.w};
  uint32_t signs = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t half = x[e / 2] >> (16 * (e & 1)) & 0xffffu;
    const bool nan = (half & 0x7fffu) > 0x7f80u;
    if (nan || half == 0x7f80u) signs |= 1u << e;
    if (nan || half == 0xff80u) signs |= 256u << e;
  }
  return signs;
}
// A block's rows of a unit, of which some hold a NaN though their sums of weights do not: a NaN element that only
// infinities of one sign went into becomes infinite, where it has been stored.  All threads of the block call it.  The
// values are read again, 8 keys a thread under way at once; those of the prefix, which all rows see, once for the
// block's rows.  Measured: 1.04 ms for 32 rows over 32768 keys
// (the whole call without an infinite value: 28 us).
template <int D>
__noinline__ __device__ void mend_rows(const TreeArgs& p, long long head, int q0, int n) {
  constexpr int E = D / 32, U = D / 8, STEP = 128 / U;
  __shared__ uint32_t prefix_signs[2][4];  // bit per element
  const CacheView& c = p.c;
  const int tid = threadIdx.x, lane = tid & 31;
  const int b = static_cast<int>(head / c.Hk), h = static_cast<int>(head - static_cast<long long>(b) * c.Hk);
  const int len = seq_len(c, b), nn = seq_new(c, b), prefix = max(c.lens[b], 0) - nn, inside = min(prefix, len);
  auto row_of = [&](int page, int j) {
    return c.V + ((static_cast<size_t>(page) * c.Hk + h) * c.page + (j & (c.page - 1))) * (D * 2);
  };
  if (tid < 8) prefix_signs[tid >> 2][tid & 3] = 0u;
  __syncthreads();
  uint32_t signs = 0;
#pragma unroll 1
  for (long long j0 = tid / U; j0 < inside; j0 += 8 * STEP) {
    int page[8];
    uint4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) page[i] = j0 + i * STEP < inside ? page_of(c, b, static_cast<int>(j0) + i * STEP) : -1;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = page[i] < 0 ? make_uint4(0, 0, 0, 0)
                         : *reinterpret_cast<const uint4*>(row_of(page[i], static_cast<int>(j0) + i * STEP) + tid % U * 16);
#pragma unroll
    for (int i = 0; i < 8; ++i) signs |= infinities(v[i]);
  }
  const int unit = tid % U;
  if (signs & 0xffu) atomicOr(&prefix_signs[0][unit >> 2], (signs & 0xffu) << (8 * (unit & 3)));
  if (signs >> 8) atomicOr(&prefix_signs[1][unit >> 2], (signs >> 8) << (8 * (unit & 3)));
  __syncthreads();
#pragma unroll 1
  for (int r = blockIdx.y * 4 + (tid >> 5); r < n; r += gridDim.y * 4) {
    const size_t row = head * p.R + q0 + r;
    __nv_bfloat16* at = p.O + row * D + lane * E;
    float o[E];
    bool nan = false;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = __bfloat162float(at[e]), nan |= o[e] != o[e];
    // (a NaN score makes all of the row NaN for good)
    const float L = __shfl_sync(0xffffffffu, lane == 0 ? p.L[row] : 0.f, 0);
    if (L != L || !__any_sync(0xffffffffu, nan)) continue;
    const int t = (q0 + r) % c.T, col = lane * E;
    const unsigned long long* trow =
        p.tree == nullptr ? nullptr : p.tree + b * p.tree_stride + static_cast<size_t>(t) * p.words;
    uint32_t plus = prefix_signs[0][col >> 5] >> (col & 31), minus = prefix_signs[1][col >> 5] >> (col & 31);
#pragma unroll 1
    for (int j = max(prefix, 0); j < len; ++j) {  // the drafted tokens that the row sees
      const int page = page_of(c, b, j);
      if (page < 0 || !(draft_bits(trow, p.words, t, j - prefix) & 1u)) continue;
      const uint4 v = *reinterpret_cast<const uint4*>(row_of(page, j) + col / 8 * 16);
      const uint32_t s = infinities(v);
      plus |= (s & 0xffu) >> (col & 7), minus |= s >> 8 >> (col & 7);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const bool up = plus >> e & 1u, down = minus >> e & 1u;
      if (o[e] != o[e] && up != down) at[e] = __float2bfloat16_rn(up ? INFINITY : -INFINITY);
    }
  }
}

// Joins the partial rows of the units that several CTAs share, one warp per row, and puts right the NaNs that
// infinite values of a bf16 cache left (an e4m3 cache has no infinities).  Lane k
// looks after piece k's sums; the rows of O then come eight pieces at a time.
template <int D, bool FP8>
__global__ void __launch_bounds__(128) tree_join_kernel(const __grid_constant__ TreeArgs p, int grid) {
  constexpr int E = D / 32;  // neighbouring elements of a lane
  pdl_wait();
  const long long unit = blockIdx.x;
  UnitInfo u = p.info[unit];
  if (*reinterpret_cast<volatile int*>(p.status) != 0) return;  // the kernel before gave up
  [[maybe_unused]] bool look = false;  // a row may hold a NaN that an infinite value explains
  if constexpr (!FP8) look = u.first >= 0 && (u.first & kNanUnit) != 0, u.first &= ~kNanUnit;
  if (u.first < 0 || u.last >= grid || (u.last <= u.first && !look)) return;  // finished where it was computed
  const int lane = threadIdx.x & 31;
  const int mt = p.M == 1 ? 0 : static_cast<int>(unit % p.M);
  const int n = min(128, p.R - mt * 128);
  const size_t slot_size = static_cast<size_t>(p.rows) * (D + 3), sums = static_cast<size_t>(p.rows) * D;
  auto slot = [&](int k) { return p.part + (2 * static_cast<size_t>(k) + (k == u.first ? 1 : 0)) * slot_size; };
  const long long head = p.M == 1 ? unit : unit / p.M;
  for (int r = blockIdx.y * 4 + (threadIdx.x >> 5); r < n; r += gridDim.y * 4) {
    if (u.last <= u.first) break;  // (all of it computed by one CTA)
    float mx = -INFINITY, l = 0.f, lr = 0.f, o[E] = {};
    for (int k0 = u.first; k0 <= u.last; k0 += 32) {
      const int k = k0 + lane;
      float m = -INFINITY, pl = 0.f, plr = 0.f;
      if (k <= u.last) {
        const float* at = slot(k) + sums + r;
        m = at[0], pl = at[p.rows], plr = at[2 * p.rows];
      }
      float top = fmaxf(m, mx);
#pragma unroll
      for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
      const float old = mx == -INFINITY ? 0.f : ex2(mx - top);  // what the pieces so far are worth now
      const float f = m == -INFINITY ? 0.f : ex2(m - top);
      if constexpr (FP8)
        pl = rescaled<FP8>(pl, m, top), plr = rescaled<FP8>(plr, m, top);
      else
        pl = f == 0.f ? 0.f : pl * f, plr = f == 0.f ? 0.f : plr * f;
#pragma unroll
      for (int i = 16; i > 0; i >>= 1) {
        pl += __shfl_xor_sync(0xffffffffu, pl, i);
        plr += __shfl_xor_sync(0xffffffffu, plr, i);
      }
      if constexpr (FP8)
        l = rescaled<FP8>(l, mx, top) + pl, lr = rescaled<FP8>(lr, mx, top) + plr, mx = top;
      else
        l = l * old + pl, lr = lr * old + plr, mx = top;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] *= old;
      const int cnt = min(32, u.last - k0 + 1);
      for (int i0 = 0; i0 < cnt; i0 += 8) {
        float v[8][E];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (i0 + i >= cnt) break;
          const float* at = slot(k0 + i0 + i) + static_cast<size_t>(r) * D + lane * E;
          if constexpr (E == 4) {
            const float4 x = *reinterpret_cast<const float4*>(at);
            v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
          } else if constexpr (E == 2) {
            const float2 x = *reinterpret_cast<const float2*>(at);
            v[i][0] = x.x, v[i][1] = x.y;
          } else {
            v[i][0] = at[0];
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float fi = __shfl_sync(0xffffffffu, f, (i0 + i) & 31);
          if (i0 + i >= cnt) break;
          if (fi != 0.f) {
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = fmaf(fi, v[i][e], o[e]);
          }
        }
      }
    }
    if constexpr (!FP8) {
#pragma unroll
      for (int e = 0; e < E; ++e) look |= o[e] != o[e] && lr == lr;
    }
    const size_t grow = head * p.R + mt * 128 + r;
    const float inv = lr == 0.f ? 0.f : 1.f / lr;
    __nv_bfloat16* dst = p.O + grow * D + lane * E;
    if constexpr (E == 4)
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
    else if constexpr (E == 2)
      *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(o[0] * inv, o[1] * inv);
    else
      *dst = __float2bfloat16_rn(o[0] * inv);
    if (lane == 0) p.L[grow] = lr == 0.f ? -INFINITY : (mx + lg2(l)) * kFwdLn2;
  }
  if constexpr (!FP8) {
    if (__syncthreads_or(look)) mend_rows<D>(p, head, mt * 128, n);
  }
}

// A cache without a page: no row sees a key.
__global__ void __launch_bounds__(256) tree_empty_kernel(uint4* O, float* L, long long n16, long long rows) {
  const long long at = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x, step = static_cast<long long>(gridDim.x) * 256;
  for (long long i = at; i < n16; i += step) O[i] = make_uint4(0u, 0u, 0u, 0u);
  for (long long i = at; i < rows; i += step) L[i] = -INFINITY;
}

int row_tiles(int R) { return (R + 127) / 128; }
int slot_rows(int R) { return R <= 32 ? 32 : R <= 64 ? 64 : 128; }
size_t info_bytes(long long units) { return (static_cast<size_t>(units) * sizeof(UnitInfo) + 255) / 256 * 256; }

template <int D, bool FP8, int NS>
fa_status launch_tree(const TreeArgs& p, int grid, cudaStream_t stream) {
  using C = TCfg<D, FP8, NS>;
  const CacheView& c = p.c;
  CUtensorMap mK, mV;
  const int rb = c.page < kKeys ? c.page : kKeys, heads = c.pages * c.Hk;
  if (FP8) {
    if (!encode_u8_3d(&mK, c.K, D, c.page, heads, D, rb) || !encode_u8_3d(&mV, c.V, D, c.page, heads, D, rb))
      return FA_ERR_CUDA;
  } else {
    if (!encode_bf16_3d(&mK, c.K, D, c.page, heads, C::CE, rb) || !encode_bf16_3d(&mV, c.V, D, c.page, heads, C::CE, rb))
      return FA_ERR_CUDA;
  }
  auto kern = tree_kernel<D, FP8, NS>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
    return FA_ERR_CUDA;
  if (launch_pdl(kern, dim3(grid), dim3(C::NTHREADS), C::SMEM, stream, mK, mV, p) != cudaSuccess)
    return FA_ERR_CUDA;
  const unsigned units = static_cast<unsigned>(p.B) * c.Hk * p.M;
  const int n = p.R < 128 ? p.R : 128;
  const cudaError_t e = launch_pdl(tree_join_kernel<D, FP8>, dim3(units, (n + 3) / 4), dim3(128), 0, stream, p, grid);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

template <int D, bool FP8>
fa_status launch_tree_rows(const TreeArgs& p, int grid, cudaStream_t s) {
  return p.R <= 32   ? launch_tree<D, FP8, 4>(p, grid, s)
         : p.R <= 64 ? launch_tree<D, FP8, 2>(p, grid, s)
                     : launch_tree<D, FP8, 1>(p, grid, s);
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_fwd_tree_workspace_size(int B, int H, int Hk, int T, int d) {
  if (B < 0 || H < 0 || Hk < 0 || T < 0 || (d != 32 && d != 64 && d != 128) || (H > 0 && (Hk == 0 || H % Hk != 0)))
    return static_cast<size_t>(-1);
  if (B == 0 || H == 0 || T == 0) return 0;
  const long long R = static_cast<long long>(H / Hk) * T;
  if (static_cast<long long>(B) * H > 65535 || R > (1LL << 30)) return static_cast<size_t>(-1);
  const long long units = static_cast<long long>(B) * Hk * row_tiles(static_cast<int>(R));
  return info_bytes(units) + 2 * static_cast<size_t>(kMaxGrid) * slot_rows(static_cast<int>(R)) * (d + 3) * sizeof(float);
}

fa_status fa_fwd_tree(const void* Q, const fa_cache* cache, void* O, float* L, int B, int H, int T, const int* table,
                      int table_cols, long long table_stride, const int* lens, const int* n_new,
                      const unsigned long long* tree, long long tree_stride, float scale, void* workspace,
                      size_t workspace_bytes, fa_stream_t stream) {
  TreeArgs p{};
  if (H < 0) return FA_ERR_INVALID_ARG;
  const fa_status st = make_cache_view(cache, table, table_cols, table_stride, lens, n_new, B, T, &p.c);
  if (st != FA_OK) return st;
  if (!check_scale(scale)) return FA_ERR_INVALID_ARG;
  if (H > 0 && (cache->Hk == 0 || H % cache->Hk != 0)) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * H > 65535) return FA_ERR_UNSUPPORTED;
  if (tree != nullptr && (!aligned(tree, 8) || tree_stride < 0)) return FA_ERR_INVALID_ARG;
  if (B == 0 || H == 0 || T == 0) return FA_OK;
  const long long R = static_cast<long long>(H / cache->Hk) * T;
  if (R > (1LL << 30)) return FA_ERR_UNSUPPORTED;
  if (!Q || !O || !L || !aligned(Q, 16) || !aligned(O, 16) || !aligned(L, 4)) return FA_ERR_INVALID_ARG;
  const size_t need = fa_fwd_tree_workspace_size(B, H, cache->Hk, T, cache->d);
  if (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 16)) return FA_ERR_WORKSPACE;
  p.status = device_status_word();
  if (p.status == nullptr) return FA_ERR_CUDA;
  p.Q = static_cast<const __nv_bfloat16*>(Q);
  p.O = static_cast<__nv_bfloat16*>(O);
  p.L = L;
  p.tree = tree;
  p.tree_stride = B > 1 ? tree_stride : 0;
  p.B = B, p.R = static_cast<int>(R), p.M = row_tiles(p.R), p.words = (T + 63) / 64;
  p.rows = slot_rows(p.R);
  p.c_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  const long long units = static_cast<long long>(B) * cache->Hk * p.M;
  if (units > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  p.info = static_cast<UnitInfo*>(workspace);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + info_bytes(units));
  if (cache->pages == 0 || table_cols == 0) {
    const long long rows = static_cast<long long>(B) * H * T;
    tree_empty_kernel<<<kMaxGrid, 256, 0, stream>>>(static_cast<uint4*>(O), L, rows * cache->d / 8, rows);
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
  }
  int grid = 0, dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&grid, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return FA_ERR_CUDA;
  // no more CTAs than there can be places
  const long long most =
      units * ((static_cast<long long>(table_cols) * cache->page_size + kKeys - 1) / kKeys + kUnitCost);
  if (grid > kMaxGrid) grid = kMaxGrid;
  if (most < grid) grid = static_cast<int>(most);
  const bool fp8 = cache->format == FA_CACHE_E4M3;
  switch (cache->d) {
    case 32: return fp8 ? launch_tree_rows<32, true>(p, grid, stream) : launch_tree_rows<32, false>(p, grid, stream);
    case 64: return fp8 ? launch_tree_rows<64, true>(p, grid, stream) : launch_tree_rows<64, false>(p, grid, stream);
    default:
      return fp8 ? launch_tree_rows<128, true>(p, grid, stream) : launch_tree_rows<128, false>(p, grid, stream);
  }
}

}  // extern "C"
