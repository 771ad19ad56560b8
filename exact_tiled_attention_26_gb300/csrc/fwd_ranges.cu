// Attention over ranges of keys, forward: O = softmax(s) V over the keys first_i <= j < last_i of each query row, with
//   s = scale q k;  s = cap tanh(s / cap);  s = s - slope |pos_i - j|.
//
// One pass over the keys with the running reference and sums of fwd_softmax.cuh, on tcgen05.  A unit is a 128-row query
// tile of a head; it walks the key tiles that the mask's table lists for its rows.  Persistent: one CTA per SM, whose
// units the order of the mask and UnitWalk decide, the next unit's loads and first S under the last tiles and the
// epilogue of the one before.
//
// Per CTA: warp 0 loads Q (two buffers) and K, warp 3 V tiles (two stages each); warp 1 issues S = Q K^T into three
// 128-column buffers of tensor memory, warp 2 O += P V; warps 4..11 form the weights, P over S: a row's 128 scores of a
// tile are shared by two threads, 64 each; warps 12..15 take O out and store it.
//
// An infinite or NaN value that a row does not see reaches it all the same, through the product's 0 * NaN.  It makes a
// NaN of O where the row's sum of weights is none, so the epilogue notes such units, and the CTA takes them once more
// when it is done with all: now warp 3 takes such values out of the tiles that some row does not see whole and notes
// their keys, and the epilogue adds them to the rows that see the key.  (Looking at every such tile the first time cost
// 11 of 71 us on short packed documents.)
//
// What bounds it.  Long rows (16384 tokens with a prefix, 32 + 8 heads, d = 128: 1.51 ms, 1475 TFLOP/s, 0.77 of a library
// product's burst; 0.86 us a tile pair): issue of the two softmax warps of a scheduler, and shared memory's port, which
// the products' operands and the loads share.  With one warp for a row's 128 scores the same took 1.71 ms.  With a cap the
// special-function unit (ranges_score.cuh), with a bias the issue slots again (2.07 ms).  Short documents (2 x 4096 tokens,
// 7 documents each, 16 + 4 heads: 42.0 us, 25 of them the tile pairs at that rate): the units' borders, and instruction
// fetches.  The roles of a CTA run code of their own all the time, and what does not fit the instruction caches comes from
// one that several SMs share: with 130 KB of code its request rate was at 0.77 of its peak and the same call took 62 us
// (now 70 KB).  So masked and whole tiles run the same code, and what runs once a unit, and the issue of the products, is a
// loop.
#include <type_traits>

#include "fwd_softmax.cuh"
#include "ranges.cuh"

namespace fa {
namespace {

// Long rows (LONG, with more than kLongKeys keys).  The tensor cores cut what they add below 2^-25 of the sum, so a sum of
// n like terms is off by up to n 2^-26: with equal weights 0.5 % at 2^20 keys, 33 % at 2^26.  There O is added to a sum of
// its own in fp32 every kSegment key tiles, as are the weights' sums; its columns were the third S buffer's.  2048 rows of
// some 2^18 keys, 8 + 2 heads, d = 128: 1.98 ms, with three buffers 1.75; d = 64 1.87 and 1.76; capped 2.90 and 2.78.
constexpr int kLongKeys = 1 << 18, kSegment = 512;
struct SegmentSums {
  float l = 0.f, lr = 0.f;  // of the segments before this one, as SoftmaxRow's
};

constexpr int kAgain = 1024;
constexpr uint64_t kTileLimitNs = 8000;  // what a tile pair may take at most, see the epilogue
// A unit as the producer hands it to the other roles.  n: key tiles; kPassEnd: all units have been handed out once; kEnd:
// no more.
constexpr int kRing = 4, kPassEnd = -1, kEnd = -2;
struct __align__(16) Unit {
  int lo, n, full_first, full_last;  // as QueryTile
  int b, qt, h, at;                  // at: its place in the CTA's walk modulo kAgain
  int pass;
  float slope;  // times log2 e
  int pad[2];
  int first[kRangeTile], last[kRangeTile];  // the rows' keys
};

template <int D, bool LONG = false>
struct RCfg {
  static constexpr int BM = kRangeTile, BN = kRangeTile;
  static constexpr int SWB = (D * 2 >= 128) ? 128 : D * 2;
  static constexpr int CE = SWB / 2;
  static constexpr int NCH = D / CE;
  static constexpr int TILE = BM * D * 2;
  static constexpr int OFF_Q = 0;         // two Q buffers
  static constexpr int OFF_K = 2 * TILE;  // two stages
  static constexpr int OFF_V = OFF_K + 2 * TILE;
  static constexpr int OFF_BAR = OFF_V + 2 * TILE;
  static constexpr int NSB = LONG ? 2 : 3;  // S buffers
  static constexpr int B_QFULL = 0, B_QEMPTY = 2, B_KFULL = 4, B_KEMPTY = 6, B_VFULL = 8, B_VEMPTY = 10, B_VCLEAN = 12,
                       B_SFULL = 14, B_PFULL = 17, B_PFREE = 20, B_OFULL = 23, B_OFREE = 24, B_SDONE = 25, B_PVDONE = 26,
                       B_EREADY = 27,  // [unit parity] row state of the unit written by the softmax warps
                       B_EFREE = 29,   // [unit parity] read, like the unit's list of values, by the epilogue warps
                       B_TOP = 31,     // [lane quarter] both column halves' largest scores are written
                       B_PASS = 35,    // all units have been stored once
                       B_UFULL = 36, B_UEMPTY = 36 + kRing, NBAR = 36 + 2 * kRing;
  static constexpr int NTHREADS = 512;
  static constexpr int REG_ISSUE = 64, REG_SOFT = 152, REG_EPI = 144;
  static_assert(REG_ISSUE + 2 * REG_SOFT + REG_EPI == 4 * 128, "register split");
  static_assert(REG_ISSUE <= 128 && REG_SOFT >= 128 && REG_EPI >= 128, "dec and inc from the launch's 128");
  static constexpr int UEMPTY_COUNT = 1 + 1 + 1 + 8 + 4;  // S and P V issuers, V, softmax and epilogue warps
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;     // tensor-memory base, abort flag, whether a unit is taken again
  static constexpr int OFF_RING = OFF_MISC + 32;          // [kRing] units
  static constexpr int OFF_BAD = OFF_RING + kRing * static_cast<int>(sizeof(Unit));  // see BadKeys
  static constexpr int OFF_AGAIN = OFF_BAD + 512;             // a bit per unit of the walk, modulo kAgain
  static constexpr int OFF_ROWS = OFF_AGAIN + kAgain / 8;     // [2][5][128] floats: m, l, l of the bf16 weights (both halves')
  static constexpr int OFF_TOPS = OFF_ROWS + 2 * 5 * BM * 4;  // [tile parity][half][128] floats
  static constexpr int SMEM_USED = OFF_TOPS + 2 * 2 * BM * 4;
  static constexpr int SMEM = (SMEM_USED + 1024 > 120 * 1024) ? SMEM_USED + 1024 : 120 * 1024;
  static constexpr int TM_S0 = 0, TM_O = NSB * 128, TM_SUM = TM_O + 128, TM_COLS = 512;
  static_assert((LONG ? TM_SUM : TM_O) + D <= TM_COLS, "tensor memory budget");
  static_assert(SMEM <= 232448, "shared memory budget");
};

// A unit's keys whose values were taken out: bit r of a tile's words for its key r.  More tiles than kBadTiles: the
// epilogue looks at every key that one of its rows sees.
constexpr int kBadTiles = 8;
struct BadKeys {
  int count;
  int tile[kBadTiles];
  uint32_t words[kBadTiles][4];
};
static_assert(2 * sizeof(BadKeys) <= 512, "shared memory of the lists");

enum : int { SITE_R_PRODUCER = 0x601, SITE_R_MMA = 0x602, SITE_R_SOFTMAX = 0x603, SITE_R_CLEAN = 0x604 };

struct FwdRangesArgs {
  MaskView m;
  ScoreMod mod;
  __nv_bfloat16* O;
  float* L;
  const __nv_bfloat16* V;  // for values that are not finite
  RowStrides sv;
  int H, G, group, qh, qb, kh, kb, vh, vb;  // (…h, …b: 0 where the tensor's heads, batches have stride 0)
  int* status;
};

// Whether all of a key tile is seen by all rows of the query tile.
FA_DEV bool whole_tile(const volatile Unit& t, int k0) {
  return k0 >= t.full_first && k0 + kRangeTile <= t.full_last;
}

// Bits lo .. hi - 1 of 32.
FA_DEV uint32_t key_bits(int lo, int hi) {
  const uint32_t below_hi = hi >= 32 ? 0xffffffffu : hi <= 0 ? 0u : (1u << hi) - 1u;
  return lo >= 32 ? 0u : lo <= 0 ? below_hi : below_hi & (0xffffffffu << lo);
}

FA_DEV void load_scores(float (&s)[64], uint32_t tS) {
  uint32_t r[64];
  tmem_ld32(tS, r);
  tmem_ld32(tS + 32, r + 32);
  tmem_ld_wait<64>(r);
#pragma unroll
  for (int k = 0; k < 64; ++k) s[k] = __uint_as_float(r[k]);
}

// The same scores in tensor memory, 0 where the bit is not set: a loop, as there is little room in the instruction cache.
FA_DEV void zero_masked(uint32_t tS, const uint32_t (&see)[2]) {
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    const uint32_t bits = (c < 2 ? see[0] : see[1]) >> (16 * (c & 1));
    uint32_t r[16];
    tmem_ld16(tS + 16 * c, r);
    tmem_ld_wait<16>(r);
#pragma unroll
    for (int k = 0; k < 16; ++k) r[k] = bits >> k & 1u ? r[k] : 0u;
    tmem_st16(tS + 16 * c, r);
  }
  tmem_st_wait();
}

// Capped scores in tensor memory, each by itself but in rows that are `fast` (whose bits are not to depend on the other
// rows of the warp).  From the scores again: a warp that kept its fast ones meanwhile took 6 % longer in all tiles.
FA_DEV void cap_in_place(uint32_t tS, const CapArgs& cap, bool fast) {
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t r[16];
    float s[16], t[16];
    tmem_ld16(tS + 16 * c, r);
    tmem_ld_wait<16>(r);
#pragma unroll
    for (int k = 0; k < 16; ++k) s[k] = t[k] = __uint_as_float(r[k]);
    cap_scores(s, cap);
    cap_scores_fast(t, cap);
#pragma unroll
    for (int k = 0; k < 16; ++k) r[k] = __float_as_uint(fast ? t[k] : s[k]);
    tmem_st16(tS + 16 * c, r);
  }
  tmem_st_wait();
}

// Scores whose bit of `see` is not set become -inf.
FA_DEV void keep_seen64(float (&s)[64], const uint32_t (&see)[2]) {
#pragma unroll
  for (int k = 0; k < 64; ++k)
    if (!(see[k >> 5] >> (k & 31) & 1u)) s[k] = -INFINITY;
}

// Moves the row's reference for a tile whose largest score is m_tile, where that has to be.  j: the unit's tile.
template <int D, bool LONG, class WaitO>
FA_DEV bool move_reference(SoftmaxRow& st, SegmentSums& sums, float m_tile, int j, uint32_t tO, int half, WaitO&& wait_o) {
  if (j == 0) {
    st.m_run = m_tile + kFwdMaxHeadroom;  // -inf stays -inf (no key seen so far)
    return true;
  }
  const bool move = m_tile > st.m_run + kFwdRescaleThreshold, take = LONG && j % kSegment == 0;
  if (!take && !__any_sync(0xffffffffu, move)) return true;
  const float m_new = m_tile + kFwdMaxHeadroom;
  const float alpha = move ? ex2(st.m_run - m_new) : 1.f;
  if (move) {
    st.l_run *= alpha;
    st.lr_run *= alpha;
    if (LONG) sums.l *= alpha, sums.lr *= alpha;
    st.m_run = m_new;
  }
  if (!wait_o()) return false;
  tc_fence_after();
#pragma unroll 1
  for (int c = half; c < D / 16; c += 2) {
    uint32_t o[16];
    tmem_ld16(tO + 16 * c, o);
    tmem_ld_wait<16>(o);
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
    if (LONG && j > kSegment) {  // there are segments before this one
      uint32_t x[16];
      const uint32_t tX = tO + (RCfg<D, LONG>::TM_SUM - RCfg<D, LONG>::TM_O) + 16 * c;
      tmem_ld16(tX, x);
      tmem_ld_wait<16>(x);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        x[i] = __float_as_uint(fmaf(__uint_as_float(x[i]), alpha, take ? __uint_as_float(o[i]) : 0.f));
      tmem_st16(tX, x);
    } else if (take) {
      tmem_st16(tO + (RCfg<D, LONG>::TM_SUM - RCfg<D, LONG>::TM_O) + 16 * c, o);
    }
    if (!take) tmem_st16(tO + 16 * c, o);  // (else the next product overwrites it)
  }
  tmem_st_wait();
  if (take) sums.l += st.l_run, sums.lr += st.lr_run, st.l_run = 0.f, st.lr_run = 0.f;
  return true;
}

// Half a key tile (64 keys) for the calling thread's query row: S at tS becomes P = 2^(score - reference) in bf16 over its
// first 32 columns.  The reference is moved lazily as in fwd_softmax.cuh; both halves of a row have the same, as they
// exchange their largest score of every tile (`top`: from this half's to the row's, false: gave up) and each rescales its
// own columns of O.  lo, hi: the row's keys, relative to the half (masked tiles only); dist0: the row's position minus the
// half's first key; side: +1 where all keys of the tile are at or before all its rows, -1 behind them, 0 on both sides.
template <int D, int MOD, bool LONG, class Top, class WaitO>
FA_DEV bool ranges_half(SoftmaxRow& st, SegmentSums& sums, uint32_t tS, uint32_t tO, int half, int j, bool masked, int lo,
                        int hi, int dist0, int side, const ScoreMod& mod, float slope, Top&& top, WaitO&& wait_o) {
  if (masked && !__any_sync(0xffffffffu, lo < hi && hi > 0 && lo < 64)) {  // the warp has no pair here
    float m_tile = -INFINITY;
    if (!top(&m_tile) || !move_reference<D, LONG>(st, sums, m_tile, j, tO, half, wait_o)) return false;
    uint32_t p[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) p[k] = 0u;
    tmem_st16(tS, p);
    tmem_st16(tS + 16, p);
    tmem_st_wait();
    return true;
  }
  float s[64];
  float base = 0.f;  // of the half's scores, left out of them
  const uint32_t see[2] = {key_bits(lo, hi), key_bits(lo - 32, hi - 32)};  // the row's keys
  // (capped scores share reciprocals: what is masked must not show in a row's last bits)
  if ((MOD & kModCap) && masked) zero_masked(tS, see);
  load_scores(s, tS);
  if constexpr (MOD != kModNone) {
    if constexpr ((MOD & kModCap) != 0) {
      const bool fast = cap_scores_fast(s, mod.cap);
      if (!__all_sync(0xffffffffu, fast)) {
        cap_in_place(tS, mod.cap, fast);
        load_scores(s, tS);
      }
    }
    const float c = (MOD & kModCap) ? 1.f : mod.c_log2;
    if constexpr ((MOD & kModBias) != 0) {
      const uint64_t c2 = f2pack(c, c);
      const float dist = static_cast<float>(dist0);
      if (side != 0) {  // side * slope * (k - dist0): its constant part stays out
        const float ss = side > 0 ? slope : -slope;
        base = -ss * dist;
        const uint64_t step = f2pack(2.f * ss, 2.f * ss);
#pragma unroll
        for (int k0 = 0; k0 < 64; k0 += 8) {  // (the steps' roundings do not add up beyond 8 columns)
          uint64_t b2 = f2pack(ss * static_cast<float>(k0), ss * static_cast<float>(k0 + 1));
#pragma unroll
          for (int k = k0; k < k0 + 8; k += 2) {
            const uint64_t x = f2pack(s[k], s[k + 1]);
            f2unpack((MOD & kModCap) ? fadd2(x, b2) : ffma2(x, c2, b2), s[k], s[k + 1]);
            b2 = fadd2(b2, step);
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < 64; ++k) s[k] = fmaf(s[k], c, -slope * fabsf(dist - static_cast<float>(k)));
      }
    }
  }
  if (masked) keep_seen64(s, see);
  float m4[4];
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    m4[a] = fmax3(s[16 * a], s[16 * a + 1], s[16 * a + 2]);
#pragma unroll
    for (int b = 3; b < 15; b += 2) m4[a] = fmax3(m4[a], s[16 * a + b], s[16 * a + b + 1]);
    m4[a] = fmaxf(m4[a], s[16 * a + 15]);
  }
  const float mx = fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]);
  float m_tile = MOD == kModNone ? mx * mod.c_log2 : mx + base;
  if (!top(&m_tile) || !move_reference<D, LONG>(st, sums, m_tile, j, tO, half, wait_o)) return false;
  const float neg_m = st.m_run == -INFINITY ? 0.f : base - st.m_run;
  const uint64_t cc2 = f2pack(mod.c_log2, mod.c_log2), nm2 = f2pack(neg_m, neg_m);
  uint64_t ls[2] = {f2pack(0.f, 0.f), f2pack(0.f, 0.f)};
  float rl[2] = {0.f, 0.f}, rh[2] = {0.f, 0.f};
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint32_t p[16];
#pragma unroll
    for (int k = 32 * c; k < 32 * c + 32; k += 2) {
      float t0, t1;
      const uint64_t x = f2pack(s[k], s[k + 1]);
      f2unpack(MOD == kModNone ? ffma2(x, cc2, nm2) : fadd2(x, nm2), t0, t1);
      const float p0 = ex2(t0), p1 = ex2(t1);
      ls[(k >> 1) & 1] = fadd2(ls[(k >> 1) & 1], f2pack(p0, p1));
      const uint32_t pk = pack_bf16x2(p0, p1);
      p[(k - 32 * c) >> 1] = pk;
      add_bf16x2_f32(pk, rl[(k >> 1) & 1], rh[(k >> 1) & 1]);
    }
    tmem_st16(tS + 16 * c, p);
  }
  float a0, a1;
  f2unpack(fadd2(ls[0], ls[1]), a0, a1);
  st.l_run += a0 + a1;
  st.lr_run += (rl[0] + rl[1]) + (rh[0] + rh[1]);
  tmem_st_wait();
  return true;
}

// A value tile with masked places (one warp): its infinities and NaNs become zeros, their keys go into `bad`.
template <int D>
FA_DEV void clean_tile(uint8_t* tile, int tile_index, BadKeys* bad, int lane) {
  using C = RCfg<D>;
  constexpr int UNITS = C::TILE / 16;
  uint4* at = reinterpret_cast<uint4*>(tile);
  uint32_t top = 0;
#pragma unroll 4
  for (int i = lane; i < UNITS; i += 32) {
    const uint4 v = at[i];
    top |= not_finite(v.x) | not_finite(v.y) | not_finite(v.z) | not_finite(v.w);
  }
  if (!__any_sync(0xffffffffu, top != 0)) return;
  int n = 0;
  if (lane == 0) {
    n = bad->count;
    bad->count = n + 1;
    if (n < kBadTiles) {
      bad->tile[n] = tile_index;
      for (int w = 0; w < 4; ++w) bad->words[n][w] = 0u;
    }
  }
  n = __shfl_sync(0xffffffffu, n, 0);
  __syncwarp();
#pragma unroll 1
  for (int i = lane; i < UNITS; i += 32) {
    uint4 v = at[i];
    uint32_t x[4] = {v.x, v.y, v.z, v.w}, any = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t f = not_finite(x[e]);
      any |= f;
      x[e] &= ~((f >> 15) * 0xffffu);  // (bit 15: the lower half, bit 31: the upper)
    }
    if (any) {
      at[i] = make_uint4(x[0], x[1], x[2], x[3]);
      const int row = i / (C::SWB / 16) % C::BN;
      if (n < kBadTiles) atomicOr(&bad->words[n][row >> 5], 1u << (row & 31));
    }
  }
  fence_proxy_async_smem();  // the product reads what was written here
}

// What a row sees that is not finite, a bit an element: +infinity or NaN in pos, -infinity or NaN in neg.
template <int D>
struct NotFinite {
  uint32_t pos[D / 32], neg[D / 32];
};

// A key's values (the whole warp), noted for the lanes whose row sees it.
template <int D>
FA_DEV void note_key(NotFinite<D>& nf, const __nv_bfloat16* v, bool sees, int lane) {
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const uint32_t x = reinterpret_cast<const uint16_t*>(v)[32 * i + lane];
    const bool f = (x & 0x7f80u) == 0x7f80u, nan = (x & 0x7fu) != 0, minus = x >> 15 != 0;
    const uint32_t p = __ballot_sync(0xffffffffu, f && (nan || !minus)), n = __ballot_sync(0xffffffffu, f && (nan || minus));
    if (sees) nf.pos[i] |= p, nf.neg[i] |= n;
  }
}

// Which of eight keys hold a value that is not finite (the whole warp, D / 32 elements a lane; keys behind hi do not).
template <int D>
FA_DEV uint32_t look_at_8(const __nv_bfloat16* v, long long stride, int j0, int hi, int lane) {
  constexpr int W = D == 128 ? 2 : 1;
  uint32_t x[8][W], keys = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const __nv_bfloat16* at = v + min(j0 + e, hi - 1) * stride + D / 32 * lane;
#pragma unroll
    for (int w = 0; w < W; ++w)
      x[e][w] = D == 32 ? *reinterpret_cast<const uint16_t*>(at) : reinterpret_cast<const uint32_t*>(at)[w];
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (__any_sync(0xffffffffu, (not_finite(x[e][0]) | not_finite(x[e][W - 1])) != 0)) keys |= 1u << e;
  return j0 + 8 <= hi ? keys : keys & ((1u << (hi - j0)) - 1u);
}

// Adds what was noted to a stored row of O.
template <int D>
FA_DEV void add_not_finite(const NotFinite<D>& nf, __nv_bfloat16* o) {
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll 1
    for (uint32_t any = nf.pos[i] | nf.neg[i]; any != 0; any &= any - 1) {
      const int e = __ffs(any) - 1;
      const bool p = nf.pos[i] >> e & 1u, n = nf.neg[i] >> e & 1u;
      __nv_bfloat16* at = o + 32 * i + e;
      if (p && n) *reinterpret_cast<uint16_t*>(at) = 0x7fff;
      else *at = __float2bfloat16(__bfloat162float(*at) + (p ? INFINITY : -INFINITY));
    }
}

// What a warp's rows see that is not finite, from a unit taken a second time: of the listed keys, or of all that one of the
// rows sees, eight at a time.  (Each lane by itself, key by key and into memory took 15 us a key of the longest row: 122 ms
// where it sees 8192.)  o: the lane's stored row, or null.  A function of its own: inlined, these rare lines made 16384
// tokens take 1.54 ms instead of 1.51.
template <int D>
__device__ __noinline__ void take_not_finite(const BadKeys& bad, int n_bad, const __nv_bfloat16* v, long long stride,
                                             int first, int last, __nv_bfloat16* o, int lane) {
  NotFinite<D> nf{};
  const bool listed = n_bad <= kBadTiles;
  const int hi = listed ? 4 * n_bad : __reduce_max_sync(0xffffffffu, last), step = listed ? 1 : 8;
#pragma unroll 1
  for (int i = listed ? 0 : __reduce_min_sync(0xffffffffu, first < last ? first : INT_MAX); i < hi; i += step) {
    uint32_t keys = listed ? bad.words[i >> 2][i & 3] : look_at_8<D>(v, stride, i, hi, lane);
    const int j0 = listed ? bad.tile[i >> 2] * kRangeTile + 32 * (i & 3) : i;
#pragma unroll 1
    for (; keys != 0; keys &= keys - 1) {
      const int j = j0 + __ffs(keys) - 1;
      note_key<D>(nf, v + j * stride, j >= first && j < last, lane);
    }
  }
  if (o != nullptr) add_not_finite<D>(nf, o);
}

template <int D, int MOD, bool LONG>
__global__ void __launch_bounds__(RCfg<D, LONG>::NTHREADS, 1)
    fwd_ranges_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ FwdRangesArgs a) {
  using C = RCfg<D, LONG>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  const uint32_t sb = smem_u32(smem);
  auto bar = [&](int i) -> uint32_t { return sb + C::OFF_BAR + 8 * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  volatile int* again_any = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 8);
  uint32_t* again = reinterpret_cast<uint32_t*>(smem + C::OFF_AGAIN);
  Unit* ring = reinterpret_cast<Unit*>(smem + C::OFF_RING);
  BadKeys* bad_keys = reinterpret_cast<BadKeys*>(smem + C::OFF_BAD);
  float* rows = reinterpret_cast<float*>(smem + C::OFF_ROWS);
  const Guard guard{a.status, abort_flag};
  const MaskView& m = a.m;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NBAR; ++i) {
      const bool softmax = (i >= C::B_PFULL && i < C::B_PFREE) || (i >= C::B_EREADY && i < C::B_EFREE);
      const bool epilogue = i == C::B_OFREE || (i >= C::B_EFREE && i < C::B_TOP) || i == C::B_PASS;
      const bool pair = i >= C::B_TOP && i < C::B_PASS;
      mbar_init(bar(i), softmax ? 256 : epilogue ? 128 : pair ? 2 : i >= C::B_UEMPTY ? C::UEMPTY_COUNT : 1);
    }
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), C::TM_COLS);
    tmem_relinquish();
  }
  if (threadIdx.x == 96) *again_any = 0;
  if (threadIdx.x < kAgain / 32) again[threadIdx.x] = 0u;
  pdl_wait();  // everything from here on may be an earlier kernel's output, O and L its input
  if (threadIdx.x == 64) *abort_flag = (*reinterpret_cast<volatile int*>(a.status) != 0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const bool skip = *abort_flag != 0;

  // A role's next unit: waits for entry i of the ring; null: no more, or gave up.  release() when it has no more use for
  // it.  Roles but the epilogue pass over units without keys and the pass's end; k counts the units they take.
  struct Taker {
    int i;  // entries taken
  };
  auto take = [&](Taker& t, bool whole_warp, bool all, int site) -> const volatile Unit* {
    for (;; ++t.i) {
      const int slot = t.i % kRing;
      const uint32_t par = (t.i / kRing) & 1;
      if (!(whole_warp ? mbar_wait_warp(bar(C::B_UFULL + slot), par, guard, site)
                       : mbar_wait(bar(C::B_UFULL + slot), par, guard, site)))
        return nullptr;
      const volatile Unit* u = ring + slot;
      const int n = u->n;
      if (n == kEnd) return nullptr;
      if (n > 0 || all) return u;
      if (whole_warp) __syncwarp();
      if (!whole_warp || lane == 0) mbar_arrive(bar(C::B_UEMPTY + slot));
    }
  };
  auto release = [&](Taker& t, bool whole_warp) {
    if (whole_warp) __syncwarp();
    if (!whole_warp || lane == 0) mbar_arrive(bar(C::B_UEMPTY + t.i % kRing));
    ++t.i;
  };

  if (warp < 4) {
    regs_dec<C::REG_ISSUE>();
    if (warp == 0 && !skip) {
      // ---------------------------------------------------------------- producer of units, Q and K (whole warp)
      int kv = 0, jk = -1, kq = -1, k = 0, i = 0;  // K tiles issued; last K, Q load issued; units with keys; ring entries
      bool ok = true;
      auto slot_free = [&] {
        return i < kRing || mbar_wait_warp(bar(C::B_UEMPTY + i % kRing), ((i / kRing) & 1) ^ 1, guard, SITE_R_PRODUCER);
      };
      for (int pass = 0; ok; pass = 1) {
        UnitWalk w{0, -1, 0};
        QueryTile ahead{0, 0, 0, 0};
        auto look = [&] {  // the next unit's tables are under way while this one's tiles are loaded
          w.look(m.q_order, m.B * m.Tq, a.H, a.group);
          if (w.entry >= 0) ahead = m.qt[w.entry];
        };
        for (look(); ok && w.entry >= 0;) {
          const QueryTile t = ahead;
          const int b = w.entry / m.Tq, qt = w.entry - b * m.Tq, h = w.head, at = w.k % kAgain;
          ++w.k;
          look();
          if (pass > 0 && !(reinterpret_cast<volatile uint32_t*>(again)[at >> 5] >> (at & 31) & 1u)) continue;
          int first[4], last[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int q = qt * C::BM + lane + 32 * e;
            first[e] = last[e] = 0;
            if (q < m.Nq) first[e] = m.first[static_cast<size_t>(b) * m.Nq + q], last[e] = m.last[static_cast<size_t>(b) * m.Nq + q];
          }
          float slope = 0.f;
          if (MOD & kModBias) slope = a.mod.slopes[h] * 1.4426950408889634f;
          if (!(ok = slot_free())) break;
          Unit* u = ring + i % kRing;
#pragma unroll
          for (int e = 0; e < 4; ++e) u->first[lane + 32 * e] = first[e], u->last[lane + 32 * e] = last[e];
          if (lane == 0) {
            u->lo = t.lo, u->n = t.n, u->full_first = t.full_first, u->full_last = t.full_last;
            u->b = b, u->qt = qt, u->h = h, u->at = at, u->pass = pass, u->slope = slope;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::B_UFULL + i % kRing));
          ++i;
          if (t.n == 0) continue;
          const int slot = k & 1, hk = h / a.G;
          // Q buffer k % 2 last held unit k-2's Q: its last S product is done
          if (k >= 2 && !(ok = mbar_wait_warp(bar(C::B_QEMPTY + slot), ((k >> 1) & 1) ^ 1, guard, SITE_R_PRODUCER))) break;
          if (lane == 0) {
            mbar_expect_tx(bar(C::B_QFULL + slot), C::TILE);
            for (int c = 0; c < C::NCH; ++c)
              tma_load_4d(sb + C::OFF_Q + slot * C::TILE + c * C::BM * C::SWB, &tmQ, bar(C::B_QFULL + slot), c * C::CE,
                          qt * C::BM, h * a.qh, b * a.qb);
          }
          kq = k;
          for (int j = 0; j < t.n; ++j, ++kv) {
            const int s = kv & 1;
            if (!(ok = mbar_wait_warp(bar(C::B_KEMPTY + s), ((kv >> 1) & 1) ^ 1, guard, SITE_R_PRODUCER))) break;
            if (lane == 0) {
              mbar_expect_tx(bar(C::B_KFULL + s), C::TILE);
              for (int c = 0; c < C::NCH; ++c)
                tma_load_4d(sb + C::OFF_K + s * C::TILE + c * C::BN * C::SWB, &tmK, bar(C::B_KFULL + s), c * C::CE,
                            (t.lo + j) * C::BN, hk * a.kh, b * a.kb);
            }
            jk = kv;
          }
          ++k;
        }
        if (!ok || !(ok = slot_free())) break;
        if (lane == 0) {
          ring[i % kRing].n = pass == 0 ? kPassEnd : kEnd;
          mbar_arrive(bar(C::B_UFULL + i % kRing));
        }
        ++i;
        if (pass > 0) break;
        if (!(ok = mbar_wait_warp(bar(C::B_PASS), 0, guard, SITE_R_PRODUCER))) break;
        if (*again_any == 0) {
          if (!(ok = slot_free())) break;
          if (lane == 0) {
            ring[i % kRing].n = kEnd;
            mbar_arrive(bar(C::B_UFULL + i % kRing));
          }
          break;
        }
      }
      if (*abort_flag && lane == 0) {
        // gave up: let every load this warp started land before the CTA exits
        for (int k = (kq > 0 ? kq - 1 : 0); k <= kq; ++k) mbar_drain(bar(C::B_QFULL + (k & 1)), (k >> 1) & 1);
        for (int j = (jk > 0 ? jk - 1 : 0); j <= jk; ++j) mbar_drain(bar(C::B_KFULL + (j & 1)), (j >> 1) & 1);
      }
    } else if (warp == 1 && lane == 0 && !skip) {
      // ---------------------------------------------------------------- UMMA issuer: S
      constexpr uint32_t idS = idesc_bf16(128, C::BN, false, false);
      bool ok = true;
      int kv = 0, k = 0;  // K tiles and S buffers used so far, across units
      for (Taker t{0}; ok; ++k) {
        const volatile Unit* u = take(t, false, false, SITE_R_MMA);
        if (u == nullptr) break;
        const int n = u->n, slot = k & 1;
        release(t, false);
        if (!(ok = mbar_wait(bar(C::B_QFULL + slot), (k >> 1) & 1, guard, SITE_R_MMA))) break;
        const uint32_t qb = sb + C::OFF_Q + slot * C::TILE;
        for (int j = 0; j < n; ++j, ++kv) {
          const int s = kv & 1, b = kv % C::NSB;
          // S buffer b last held P of S-tile kv-3: the product that read it is done
          if (kv >= C::NSB && !(ok = mbar_wait(bar(C::B_PFREE + b), ((kv / C::NSB) & 1) ^ 1, guard, SITE_R_MMA))) break;
          if (!(ok = mbar_wait(bar(C::B_KFULL + s), (kv >> 1) & 1, guard, SITE_R_MMA))) break;
          tc_fence_after();
          const uint32_t kb = sb + C::OFF_K + s * C::TILE;
          uint64_t qd = sdesc_kmajor_base<C::SWB, C::BM>(qb), kd = sdesc_kmajor_base<C::SWB, C::BN>(kb);
#pragma unroll 1
          for (int c = 0; c < (D + 63) / 64; ++c) {  // (loops, here and for P V: 4096 tokens of documents 43.1 to 42.1 us)
#pragma unroll
            for (int ks = 0; ks < (D < 64 ? D / 16 : 4); ++ks)
              mma_ss(tmem + C::TM_S0 + b * 128, desc_at(qd, kmajor_off<C::SWB, C::BM>(ks)),
                     desc_at(kd, kmajor_off<C::SWB, C::BN>(ks)), idS, c > 0 || ks > 0);
            qd = desc_at(qd, kmajor_off<C::SWB, C::BM>(4)), kd = desc_at(kd, kmajor_off<C::SWB, C::BN>(4));
          }
          mma_commit(bar(C::B_SFULL + b));
          mma_commit(bar(C::B_KEMPTY + s));
        }
        if (!ok) break;
        mma_commit(bar(C::B_QEMPTY + slot));  // this unit's Q has no later reader
      }
      mma_commit(bar(C::B_SDONE));  // drain point for teardown
    } else if (warp == 2 && lane == 0 && !skip) {
      // ---------------------------------------------------------------- UMMA issuer: P V
      constexpr uint32_t idO = idesc_bf16(128, D, false, true);
      bool ok = true;
      int kv = 0, k = 0;
      uint32_t clean_parity = 0;  // bit s: of stage s's next tile of the second pass
      for (Taker t{0}; ok; ++k) {
        const volatile Unit* u = take(t, false, false, SITE_R_MMA);
        if (u == nullptr) break;
        const int n = u->n, pass = u->pass;
        release(t, false);
        for (int j = 0; j < n; ++j, ++kv) {
          const int s = kv & 1, b = kv % C::NSB;
          if (!(ok = mbar_wait(bar(C::B_PFULL + b), (kv / C::NSB) & 1, guard, SITE_R_MMA))) break;
          if (pass == 0) {
            if (!(ok = mbar_wait(bar(C::B_VFULL + s), (kv >> 1) & 1, guard, SITE_R_MMA))) break;
          } else {
            if (!(ok = mbar_wait(bar(C::B_VCLEAN + s), clean_parity >> s & 1u, guard, SITE_R_MMA))) break;
            clean_parity ^= 1u << s;
          }
          // the first product of a unit overwrites O: the previous unit's epilogue has read it
          if (j == 0 && k > 0 && !(ok = mbar_wait(bar(C::B_OFREE), (k - 1) & 1, guard, SITE_R_MMA))) break;
          tc_fence_after();
          const uint32_t vb = sb + C::OFF_V + s * C::TILE;
          const uint32_t aP = tmem + C::TM_S0 + b * 128;
          uint64_t vd = sdesc_mnmajor_base<C::SWB, C::BN>(vb);
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma_ts(tmem + C::TM_O, aP + 64 * c + 8 * ks, desc_at(vd, mnmajor_off<C::SWB>(ks)), idO,
                     (LONG ? j % kSegment != 0 : j > 0) || c > 0 || ks > 0);
            vd = desc_at(vd, mnmajor_off<C::SWB>(4));
          }
          mma_commit(bar(C::B_VEMPTY + s));
          mma_commit(bar(C::B_PFREE + b));
        }
        if (!ok) break;
        mma_commit(bar(C::B_OFULL));  // O of this unit is complete
      }
      mma_commit(bar(C::B_PVDONE));  // every S completed before its P existed: the end of all UMMAs
    } else if (warp == 3 && !skip) {
      // ---------------------------------------------------------------- producer of V; cleaner in the second pass
      bool ok = true;
      int kv = 0, jv = -1, k = 0;  // V tiles issued, last load issued
      for (Taker t{0}; ok; ++k) {
        const volatile Unit* u = take(t, true, false, SITE_R_CLEAN);
        if (u == nullptr) break;
        const int slot = k & 1, n = u->n, lo = u->lo, b = u->b, hk = u->h / a.G, pass = u->pass;
        if (pass > 0) {  // the list last held unit k-2's keys: its epilogue has read them
          if (k >= 2 && !(ok = mbar_wait_warp(bar(C::B_EFREE + slot), ((k >> 1) & 1) ^ 1, guard, SITE_R_CLEAN))) break;
          if (lane == 0) bad_keys[slot].count = 0;
          __syncwarp();
        }
        for (int j = 0; j < n; ++j, ++kv) {
          const int s = kv & 1, y = (lo + j) * C::BN;
          if (!(ok = mbar_wait_warp(bar(C::B_VEMPTY + s), ((kv >> 1) & 1) ^ 1, guard, SITE_R_CLEAN))) break;
          if (lane == 0) {
            mbar_expect_tx(bar(C::B_VFULL + s), C::TILE);
            for (int c = 0; c < C::NCH; ++c)
              tma_load_4d(sb + C::OFF_V + s * C::TILE + c * C::BN * C::SWB, &tmV, bar(C::B_VFULL + s), c * C::CE, y,
                          hk * a.vh, b * a.vb);
          }
          __syncwarp();
          jv = kv;
          if (pass > 0) {
            if (!(ok = mbar_wait_warp(bar(C::B_VFULL + s), (kv >> 1) & 1, guard, SITE_R_CLEAN))) break;
            if (!whole_tile(*u, y)) clean_tile<D>(smem + C::OFF_V + s * C::TILE, lo + j, bad_keys + slot, lane);
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::B_VCLEAN + s));
          }
        }
        if (!ok) break;
        release(t, true);
      }
      if (*abort_flag && lane == 0)
        for (int j = (jv > 0 ? jv - 1 : 0); j <= jv; ++j) mbar_drain(bar(C::B_VFULL + (j & 1)), (j >> 1) & 1);
    }
  } else if (warp < 12) {
    regs_inc<C::REG_SOFT>();
    if (!skip) {
      // ---------------------------------------------------------------- softmax
      const int wq = warp & 3, row = wq * 32 + lane, half = (warp - 4) >> 2;
      float* tops = reinterpret_cast<float*>(smem + C::OFF_TOPS);
      const uint32_t tl = tmem + (static_cast<uint32_t>(wq * 32) << 16);
      bool ok = true;
      int kv = 0, k = 0;
      for (Taker t{0}; ok; ++k) {
        const volatile Unit* u = take(t, true, false, SITE_R_SOFTMAX);
        if (u == nullptr) break;
        const int n = u->n, slot = k & 1;
        SoftmaxRow st;
        SegmentSums sums;
        for (int j = 0; j < n; ++j, ++kv) {
          const int b = kv % C::NSB, k0 = (u->lo + j) * C::BN, p0 = u->qt * C::BM + m.Nk - m.Nq;
          if (!(ok = mbar_wait_warp(bar(C::B_SFULL + b), (kv / C::NSB) & 1, guard, SITE_R_SOFTMAX))) break;
          tc_fence_after();
          // before a rescale: the last product into O (S-tile kv-1, same unit) is done
          auto wait_o = [&] {
            const int pb = (kv - 1) % C::NSB;
            return mbar_wait_warp(bar(C::B_PFREE + pb), ((kv - 1) / C::NSB) & 1, guard, SITE_R_SOFTMAX);
          };
          // the row's largest score of the tile, from both halves (the slot's last reader, two tiles ago, has arrived for
          // the tile before this one since)
          auto top = [&](float* mine) {
            float* at = tops + (kv & 1) * 2 * C::BM;
            at[half * C::BM + row] = *mine;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::B_TOP + wq));
            if (!mbar_wait_warp(bar(C::B_TOP + wq), kv & 1, guard, SITE_R_SOFTMAX)) return false;
            *mine = fmaxf(*mine, at[(1 - half) * C::BM + row]);
            return true;
          };
          const int side = p0 >= k0 + C::BN - 1 ? 1 : p0 + C::BM - 1 <= k0 ? -1 : 0, c0 = k0 + 64 * half;
          const float slope = (MOD & kModBias) ? u->slope : 0.f;
          const uint32_t tS = tl + C::TM_S0 + b * 128 + 64 * half, tO = tl + C::TM_O;
          bool masked = !whole_tile(*u, k0);
          int lo = 0, hi = 64;
          if (masked) {
            lo = u->first[row] - c0, hi = u->last[row] - c0;
            masked = !__all_sync(0xffffffffu, lo <= 0 && hi >= 64);
          }
          ok = ranges_half<D, MOD, LONG>(st, sums, tS, tO, half, j, masked, lo, hi, p0 + row - c0, side, a.mod, slope, top,
                                         wait_o);
          if (!ok) break;
          tc_fence_before();
          mbar_arrive(bar(C::B_PFULL + b));
        }
        if (!ok) break;
        release(t, true);
        // the row state for the epilogue warps (slot k % 2 last held unit k-2's, which they have read)
        if (k >= 2 && !(ok = mbar_wait_warp(bar(C::B_EFREE + slot), ((k >> 1) & 1) ^ 1, guard, SITE_R_SOFTMAX))) break;
        float* rs = rows + slot * 5 * C::BM;
        if (half == 0) rs[row] = st.m_run;
        rs[(1 + 2 * half) * C::BM + row] = LONG ? sums.l + st.l_run : st.l_run;
        rs[(2 + 2 * half) * C::BM + row] = LONG ? sums.lr + st.lr_run : st.lr_run;
        mbar_arrive(bar(C::B_EREADY + slot));
      }
    }
  } else {
    regs_inc<C::REG_EPI>();
    if (!skip) {
      // ---------------------------------------------------------------- epilogue
      const int wq = warp & 3, row = wq * 32 + lane;
      const uint32_t tl = tmem + (static_cast<uint32_t>(wq * 32) << 16);
      bool ok = true;
      int k = 0;
      for (Taker t{0}; ok;) {
        const volatile Unit* u = take(t, true, true, SITE_R_SOFTMAX);
        if (u == nullptr) break;
        const int n = u->n, b = u->b, h = u->h, at = u->at, pass = u->pass;
        const int q = u->qt * C::BM + row, first = u->first[row], last = u->last[row];
        release(t, true);
        if (n == kPassEnd) {
          mbar_arrive(bar(C::B_PASS));
          continue;
        }
        const int w0 = q - lane;  // the warp's first row
        const size_t row0 = (static_cast<size_t>(b) * a.H + h) * m.Nq;
        uint8_t* out = reinterpret_cast<uint8_t*>(a.O + (row0 + w0) * D);
        const int slot = k & 1;
        float L = -INFINITY, l = 0.f, lr = 0.f, m_run = 0.f;
        if (n > 0) {
          // the one wait that a whole unit's tiles are computed under (0.8 us each: 2^29 keys take 3.4 s)
          const uint64_t limit = kWaitLimitNs + static_cast<uint64_t>(n) * kTileLimitNs;
          if (!(ok = mbar_wait_warp(bar(C::B_EREADY + slot), (k >> 1) & 1, guard, SITE_R_SOFTMAX, limit))) break;
          const float* rs = rows + slot * 5 * C::BM;
          m_run = rs[row], l = rs[C::BM + row] + rs[3 * C::BM + row], lr = rs[2 * C::BM + row] + rs[4 * C::BM + row];
          if (!(ok = mbar_wait_warp(bar(C::B_OFULL), k & 1, guard, SITE_R_SOFTMAX))) break;
          tc_fence_after();
          if (lr != 0.f) L = (m_run + lg2(l)) * kFwdLn2;
        }
        const float inv = 1.f / lr;
        uint64_t nan = f2pack(0.f, 0.f);
        // 32 columns at a time: a loop, as the code of all roles does not fit the instruction cache (see above)
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t pk[16];
          if (n > 0) {
            uint32_t o[32];
            tmem_ld32(tl + C::TM_O + 32 * c, o);
            tmem_ld_wait<32>(o);
            if (LONG && n > kSegment) {
              uint32_t x[32];
              tmem_ld32(tl + C::TM_SUM + 32 * c, x);
              tmem_ld_wait<32>(x);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) + __uint_as_float(x[i]));
            }
            if (c == D / 32 - 1) {
              tc_fence_before();
              mbar_arrive(bar(C::B_OFREE));  // the next unit's first P V may overwrite O
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float x = __uint_as_float(o[2 * i]), y = __uint_as_float(o[2 * i + 1]);
              nan = ffma2(f2pack(x, y), f2pack(0.f, 0.f), nan);  // NaN where an element is not finite
              pk[i] = lr == 0.f ? 0u : pack_bf16x2(x * inv, y * inv);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) pk[i] = 0u;
          }
          warp_store_rows<4, 0>(pk, out + 64 * c, D * 2, m.Nq - w0, lane);
        }
        if (q < m.Nq) a.L[row0 + q] = L;
        if (n == 0) continue;
        if (pass == 0) {
          float n0, n1;
          f2unpack(nan, n0, n1);
          if (__any_sync(0xffffffffu, n0 + n1 != 0.f && lr - lr == 0.f && lr != 0.f) && lane == 0) {
            atomicOr(&again[at >> 5], 1u << (at & 31));
            *again_any = 1;
          }
        } else {
          __syncwarp();  // (the rows have been stored by other lanes)
          const BadKeys& bad = bad_keys[slot];
          const int n_bad = bad.count;
          const __nv_bfloat16* v = a.V + b * a.sv.b + h / a.G * a.sv.h;
          take_not_finite<D>(bad, n_bad, v, a.sv.n, first, last, q < m.Nq ? a.O + (row0 + q) * D : nullptr, lane);
        }
        mbar_arrive(bar(C::B_EFREE + slot));
        ++k;
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

// Heads whose K and V are streamed at the same time: whole groups of query heads that share theirs, as many as keep
// about 64 MiB of K and V in L2.
int heads_at_once(const RangesLaunch& a) {
  const int G = a.H / a.Hk;
  const long long per = 4LL * a.B * a.Nk * a.d;  // K and V of a key head
  const long long n = per > 0 ? (64LL << 20) / per : a.Hk;
  return G * static_cast<int>(n < 1 ? 1 : n > a.Hk ? a.Hk : n);
}

template <int D, int MOD, bool LONG = false>
fa_status launch(const RangesLaunch& a) {
  if (!LONG && a.Nk > kLongKeys) return launch<D, MOD, true>(a);
  using C = RCfg<D, LONG>;
  int dev = 0, nsm = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return FA_ERR_CUDA;
  CUtensorMap mQ, mK, mV;
  // (without a key there is no tile to load)
  if (!encode_bf16_rows(&mQ, a.Q, D, a.Nq, a.H, a.B, a.sq, C::CE, C::BM) ||
      (a.Nk > 0 && (!encode_bf16_rows(&mK, a.K, D, a.Nk, a.Hk, a.B, a.sk, C::CE, C::BN) ||
                    !encode_bf16_rows(&mV, a.V, D, a.Nk, a.Hk, a.B, a.sv, C::CE, C::BN))))
    return FA_ERR_CUDA;
  if (a.Nk == 0) mK = mV = mQ;
  auto kern = fwd_ranges_kernel<D, MOD, LONG>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
    return FA_ERR_CUDA;
  const long long units = static_cast<long long>(a.B) * a.mask.Tq * a.H;
  if (units > INT_MAX / 2) return FA_ERR_UNSUPPORTED;
  const int grid = static_cast<int>(units < nsm ? units : nsm);
  FwdRangesArgs args{a.mask, a.mod, static_cast<__nv_bfloat16*>(a.out), a.L, static_cast<const __nv_bfloat16*>(a.V), a.sv,
                     a.H, a.H / a.Hk, heads_at_once(a), a.sq.h != 0, a.sq.b != 0, a.sk.h != 0, a.sk.b != 0, a.sv.h != 0,
                     a.sv.b != 0, a.status};
  return launch_pdl(kern, dim3(grid), dim3(C::NTHREADS), C::SMEM, a.stream, mQ, mK, mV, args) == cudaSuccess
             ? FA_OK : FA_ERR_CUDA;
}

template <int D>
fa_status launch_mod(const RangesLaunch& a) {
  const bool cap = a.mod.cap.cap_log2 > 0.f, bias = a.mod.slopes != nullptr;
  return cap ? (bias ? launch<D, kModCap | kModBias>(a) : launch<D, kModCap>(a))
             : (bias ? launch<D, kModBias>(a) : launch<D, kModNone>(a));
}

}  // namespace

fa_status launch_fwd_ranges(const RangesLaunch& a) {
  return a.d == 32 ? launch_mod<32>(a) : a.d == 64 ? launch_mod<64>(a) : launch_mod<128>(a);
}

}  // namespace fa
