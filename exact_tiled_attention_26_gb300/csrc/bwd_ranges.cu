// Attention over ranges of keys, gradients (the scores of fwd_ranges.cu):
//   P = exp(s - L), dV = P^T dO, dP = dO V^T, D = rowsum(dO * O), dS = P (dP - D) r, with the cap's derivative
//   r = 1 - tanh^2, dQ = dS K scale, dK = dS^T Q scale; dK and dV are sums over the query heads of a key head.
//
// A unit is a 128-key tile of a key head: K and V stay in shared memory while the CTA walks the query tiles of the
// mask's table, for one query head of the key head after the other, and dK, dV add up in tensor memory over all of
// them (over a part of the steps where a unit is split).  Roles, tensor-memory regions and the per-step barriers are those
// of bwd_steps.cuh; what is new is in the element-wise step (row ranges, cap, bias) and in what its producer stages.
// Persistent: one CTA per SM, units by the mask's order, long ones in parts (split_places).  d = 32 runs with d = 64's
// tiles, whose second half the loads fill with zeros (2 x 4096 tokens of documents, 16 + 4 heads: 108 us, d = 64 123).
//
// What no pair uses may hold anything: a query row that sees no key is zeroed in its tiles before the products with
// dO and Q (their weights 0 would make NaN of a NaN), an infinite or NaN key is zeroed before dQ^T = K^T dS^T, and a
// masked pair's dS is zero whatever dP is.  Pairs that see such a key get NaN for P and dS: L need not be NaN there (a
// score of -infinity has weight 0, a capped one is the cap), and the formula has 0 times infinity.
//
// Three launches: D and the cleared dQ sums; the products; dQ rounded to bf16, and split units' parts added.
//
// What bounds it.  Long rows (8192 tokens with a prefix, 32 + 8 heads, d = 128: 1.35 ms, 1035 TFLOP/s; 2.9 us a step): the
// chain of a step, as in bwd_steps.cuh, and the reductions of dQ in L2.  The cap adds two operations of the
// special-function unit an element (1.49 ms), the bias issue slots (1.37).  Short documents (2 x 4096 tokens, 16 + 4
// heads: 167 us, capped 185): the fullest SM has 41 steps, with 29 on the average; 33 us are the first and the last
// launch, which write and read the fp32 sums of dQ; and instruction fetches, as in fwd_ranges.cu (86 to 99 KB of code, of
// which some 31 run in every step: 16 more there made the 1.39 ms of an earlier form 1.71).
#include <cmath>

#include "bwd_steps.cuh"
#include "ranges.cuh"

namespace fa {
namespace {

using namespace bsteps;

// Barriers of this kernel beyond the per-step ones (bwd_steps.cuh).
enum : int {
  B_KVFULL = 0, B_FINAL = 17, B_ADONE = 18,
  B_KVFREE = 20,   // the unit's last readers of K and V are done (one commit from each issuer, the element-wise warps)
  B_DKVFULL = 21,  // the unit's dK, dV are complete in tensor memory
  B_DKVFREE = 22,  // the element-wise warps have taken them out
  B_KVFULL1 = 23, B_KVFREE1 = 24,  // the second K, V buffer's (d <= 64)
  B_UFULL = 25, B_UEMPTY = 29,     // unit ring
  NBAR = 33
};
// What the producer hands to the other roles: key tile kt of key head h, against query tiles lo .. lo + n - 1 of each of
// its query heads, one head after the other.  n 0: no row sees these keys; n < 0: no more.  slot: where the sums of a
// part of a split unit go, or kWhole.
constexpr int kRing = 4, kWhole = -1;
struct Unit {
  int lo, n, b, kt, h, slot;
};
constexpr int UEMPTY_COUNT = 1 + 1 + 8 + 4;  // issuers A and B, 8 element-wise and 4 drain warps
FA_DEV int kvfull(int b) { return b == 0 ? B_KVFULL : B_KVFULL1; }
FA_DEV int kvfree(int b) { return b == 0 ? B_KVFREE : B_KVFREE1; }
constexpr int ROFF_MISC = NBAR * 8;  // tensor-memory base, abort flag
constexpr int NTHREADS = 512;
// A stage of what goes with a query tile: -L log2 e, D, the rows' ranges, the step's flags and slope.
struct Stage {
  float L[BM], D[BM];
  uint32_t ranges[BM / 2];  // two rows a word, each 128 - first and last relative to the key tile, cut to 0 .. 128
  int masked, dead;         // some pair is not seen; some row sees nothing at all
  float slope;              // times log2 e
  int pad;
};
constexpr int ROFF_RING = ROFF_MISC + 8;
constexpr int ROFF_BAD = ROFF_RING + kRing * static_cast<int>(sizeof(Unit));  // [unit parity][4]: see clean_key
constexpr int ROFF_STAGE = (ROFF_BAD + 2 * 4 * 4 + 15) / 16 * 16, RSMALL = ROFF_STAGE + 2 * static_cast<int>(sizeof(Stage));
static_assert(RSMALL <= 3 * 1024 && sizeof(Stage) % 16 == 0, "small region");

enum : int { SITE_RB_PRODUCER = 0x611, SITE_RB_MMA = 0x612, SITE_RB_COMPUTE = 0x613, SITE_RB_LAYOUT = 0x615 };

struct BwdRangesArgs {
  MaskView m;
  ScoreMod mod;
  const float *L, *D;
  float* dQacc;
  __nv_bfloat16 *dK, *dV;
  float* part;  // [split units][kParts][2][128][D]: dK and dV of a unit's parts
  int H, Hk, G, qh, qb, kh, kb, vh, vb, gh, gb;  // (…h, …b: 0 where the tensor's heads, batches have stride 0)
  float scale;  // of dQ's and dK's sums (with a cap, dS is over kRateScale)
  int* status;
};

// Sums times their scale.  (0 stays +0 with a negative one.)
FA_DEV uint32_t scaled_bf16x2(float x, float y, float scale) {
  return pack_bf16x2(fmaf(x, scale, 0.f), fmaf(y, scale, 0.f));
}

FA_DEV Stage* stage_of(const Ctx& x, int g) { return reinterpret_cast<Stage*>(x.small + ROFF_STAGE) + (g & 1); }

// Producer (whole warp): Q, dO of query tile i of head h into stage g % 2, and the tile's Stage.
template <class LY, int MOD>
FA_DEV bool produce(const Ctx& x, const CUtensorMap* tmQ, const CUtensorMap* tmdO, const BwdRangesArgs& a, int b, int h,
                    int i, int kt, int g, int lane) {
  const int s = g & 1, q0 = i * BM;
  const MaskView& m = a.m;
  const size_t row0 = (static_cast<size_t>(b) * a.H + h) * m.Nq, at0 = static_cast<size_t>(b) * m.Nq;
  // read before waiting for the stage
  const QueryTile t = m.qt[static_cast<size_t>(b) * m.Tq + i];
  float lv[4], dv[4];
  uint32_t rg[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int q = q0 + lane + 32 * u;
    float L = -INFINITY;
    int lo = 0, hi = 0;
    lv[u] = -INFINITY, dv[u] = 0.f;
    if (q < m.Nq) L = a.L[row0 + q], dv[u] = a.D[row0 + q], lo = m.first[at0 + q], hi = m.last[at0 + q];
    if (L != -INFINITY) lv[u] = -L * kLog2e;
    lo = min(max(lo - kt * BN, 0), BN), hi = min(max(hi - kt * BN, 0), BN);
    rg[u] = static_cast<uint32_t>(BN - lo) | static_cast<uint32_t>(hi) << 8;
  }
  float slope = 0.f;
  if (MOD & kModBias) slope = a.mod.slopes[h] * kLog2e;
  if (!mbar_wait_warp(x.bar(B_QEMPTY + s), ((g >> 1) & 1) ^ 1, x.guard, SITE_RB_PRODUCER)) return false;
  if (lane == 0) {
    mbar_expect_tx(x.bar(B_QFULL + s), 2 * LY::TQ);
    for (int c = 0; c < LY::TQ / CHUNK; ++c) {
      tma_load_4d(LY::q(x.tb, s) + c * CHUNK, tmQ, x.bar(B_QFULL + s), c * 64, q0, h * a.qh, b * a.qb);
      tma_load_4d(LY::dO(x.tb, s) + c * CHUNK, tmdO, x.bar(B_QFULL + s), c * 64, q0, h * a.gh, b * a.gb);
    }
  }
  Stage* st = stage_of(x, g);
  uint16_t* ranges = reinterpret_cast<uint16_t*>(st->ranges);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    st->L[lane + 32 * u] = lv[u];
    st->D[lane + 32 * u] = dv[u];
    ranges[lane + 32 * u] = static_cast<uint16_t>(rg[u]);
  }
  if (lane == 0) {
    st->masked = !(kt * BN >= t.full_first && kt * BN + BN <= t.full_last);
    st->dead = t.full_first == kNoFull;
    st->slope = slope;
  }
  mbar_arrive(x.bar(B_QFULL + s));
  return true;
}

// UMMA issuers (one thread each): bwd_steps.cuh's issue_s_dp and issue_dv_dk_dq as loops, for the instruction caches (see
// above): 8192 tokens with a cap 1.72 to 1.48 ms, 4096 tokens of documents with one 207 to 184 us, d = 64 40.6 to 37.2 us.
// (Issuer B unrolled over its sub-chunks: 1.35 ms uncapped where this takes 1.36, 1.57 capped where this takes 1.48.)
template <class LY>
FA_DEV bool issue_a(const Ctx& x, int g, int kvb) {
  constexpr uint32_t idKK = idesc_bf16(128, 128, false, false);
  constexpr int KS = LY::TQ / (128 * 32);
  const int s = g & 1;
  if (!mbar_wait(x.bar(B_QFULL + s), (g >> 1) & 1, x.guard, SITE_RB_MMA)) return false;
#pragma unroll 1
  for (int p = 0; p < 2; ++p) {  // S^T into region s, dP^T into the other
    // what the regions held: dP^T of the step before, read by the element-wise threads, and its dQ^T, by the drain
    if (g > 0 && !mbar_wait(x.bar(p == 0 ? B_DPCONS : B_DQCONS), (g - 1) & 1, x.guard, SITE_RB_MMA)) return false;
    tc_fence_after();
    uint64_t ad = sdesc_kmajor_base<128, 128>(p == 0 ? LY::k(x.tb, kvb) : LY::v(x.tb, kvb));
    uint64_t bd = sdesc_kmajor_base<128, 128>(p == 0 ? LY::q(x.tb, s) : LY::dO(x.tb, s));
    const uint32_t d = x.tmem + TM_R + 128 * (s ^ p);
#pragma unroll 1
    for (int c = 0; c < KS / 4; ++c) {
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
        mma_ss(d, desc_at(ad, kmajor_off<128, 128>(ks)), desc_at(bd, kmajor_off<128, 128>(ks)), idKK, c > 0 || ks > 0);
      ad = desc_at(ad, CHUNK), bd = desc_at(bd, CHUNK);
    }
    mma_commit(x.bar(p == 0 ? B_SFULL : B_DPFULL));
  }
  return true;
}
template <class LY>
FA_DEV bool issue_b(const Ctx& x, int g, int kvb, bool first) {
  constexpr uint32_t idTN = idesc_bf16(128, LY::TQ / 256, false, true), idMN = idesc_bf16(128, 128, true, true);
  const int s = g & 1;
  const uint32_t rs = x.tmem + TM_R + 128 * s;
  // dV += P^T dO, then dK += dS^T Q, each in two sub-chunks of queries
#pragma unroll 1
  for (int j = 0; j < 4; ++j) {
    const int p = j >> 1, c = j & 1;
    if (!mbar_wait(x.bar(p == 0 ? B_PREADY + 2 * s + c : B_DSREADY + c), p == 0 ? (g >> 1) & 1 : g & 1, x.guard, SITE_RB_MMA))
      return false;
    tc_fence_after();
    const uint64_t bd = desc_at(sdesc_mnmajor_base<128, 128>(p == 0 ? LY::dO(x.tb, s) : LY::q(x.tb, s)), mnmajor_off<128>(2 * c));
    const uint32_t d = x.tmem + (p == 0 ? TM_DV : TM_DK), a0 = rs + 32 * p + 16 * c;
#pragma unroll
    for (int u = 0; u < 4; ++u)
      mma_ts(d, a0 + 64 * (u >> 1) + 8 * (u & 1), desc_at(bd, mnmajor_off<128>(4 * (u >> 1) + (u & 1))), idTN,
             !first || c > 0 || u > 0);
  }
  mma_commit(x.bar(B_DKDONE));
  mma_commit(x.bar(B_QEMPTY + s));  // Q, dO of this stage have no later reader
  if (!mbar_wait(x.bar(B_DKDONE), g & 1, x.guard, SITE_RB_MMA)) return false;
  if (!mbar_wait(x.bar(B_DSSMEM), g & 1, x.guard, SITE_RB_MMA)) return false;
  tc_fence_after();
  uint64_t ad = sdesc_mnmajor_base<128, 128>(LY::k(x.tb, kvb)), bd = sdesc_mnmajor_base<128, 128>(x.tb + LY::T_DS);
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
      mma_ss(rs, desc_at(ad, mnmajor_off<128>(ks)), desc_at(bd, mnmajor_off<128>(ks)), idMN, c > 0 || ks > 0);
    ad = desc_at(ad, mnmajor_off<128>(4)), bd = desc_at(bd, mnmajor_off<128>(4));
  }
  mma_commit(x.bar(B_DQFULL));
  return true;
}

// dQ drain (bwd_steps.cuh's drain_step, for DR <= D elements of a row).
template <int D, int DR>
FA_DEV bool drain(const Ctx& x, int g, float* tile, int nq, int qw, int lane) {
  constexpr int NQ = D == 128 ? 128 : 64;
  const int qb = D == 128 ? 0 : 64 * (qw >> 1), col = (D == 128 ? qw : (qw & 1)) * 32 + lane;
  float* dst = tile + static_cast<size_t>(qb) * DR + col;
  const int nv = nq - qb;
  const uint32_t tl = x.tmem + (static_cast<uint32_t>(qw * 32) << 16);
  if (!mbar_wait_warp(x.bar(B_DQFULL), g & 1, x.guard, SITE_RB_COMPUTE)) return false;
  tc_fence_after();
  uint32_t r[NQ];
#pragma unroll
  for (int c = 0; c < NQ / 32; ++c) tmem_ld32(tl + TM_R + 128 * (g & 1) + qb + 32 * c, r + 32 * c);
  tmem_ld_wait<NQ>(r);
  tc_fence_before();
  mbar_arrive(x.bar(B_DQCONS));
  if (DR < D && (qw & 1)) return true;  // columns that are padding
  if (nv >= NQ) {
#pragma unroll
    for (int q = 0; q < NQ; ++q) atomicAdd(dst + static_cast<size_t>(q) * DR, __uint_as_float(r[q]));
  } else {
#pragma unroll
    for (int q = 0; q < NQ; ++q)
      if (q < nv) atomicAdd(dst + static_cast<size_t>(q) * DR, __uint_as_float(r[q]));
  }
  return true;
}

// A unit's K tile, looked through by the element-wise threads, each the row of its key: infinities and NaNs become zeros,
// for the keys' part in dQ^T of rows that do not see them.  Returns what makes bf16 pairs NaN if the key is not finite,
// else 0: the scores of such a key are not its own any more (S^T may have been made before or after), and the pairs that
// see it are made NaN from this.  Half h clears chunk h only.  At d = 128 a chunk is half the row and the other half of the
// threads may have cleared its own already: it has set the key's bit in `bad` (which the thread's warp and its partner
// share) before that.
template <class LY>
FA_DEV uint32_t clean_key(const Ctx& x, int kvb, uint32_t* bad, int h, int kr, int lane) {
  constexpr bool HALVES = LY::TQ == LY::TK;  // (else the second chunk is a copy of the first)
  uint8_t* row = x.tiles + kvb * LY::KVB + kr * 128;
  auto look = [&](int c) {
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < 8; ++u) {  // (from another place in each lane: a row is 128 bytes, all banks)
      const uint4 v = *reinterpret_cast<const uint4*>(row + c * CHUNK + 16 * ((u + lane) & 7));
      top |= not_finite(v.x) | not_finite(v.y) | not_finite(v.z) | not_finite(v.w);
    }
    return top;
  };
  const uint32_t mine = look(h);
  uint32_t any = mine;
  if (HALVES) any |= look(1 - h);
  if (mine != 0) {
    if (HALVES) {
      atomicOr(bad, 1u << lane);
      __threadfence_block();
    }
#pragma unroll 1
    for (int u = 0; u < 8; ++u) {
      uint4* at = reinterpret_cast<uint4*>(row + h * CHUNK + 16 * u);
      const uint4 v = *at;
      uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] &= ~((not_finite(w[e]) >> 15) * 0xffffu);
      *at = make_uint4(w[0], w[1], w[2], w[3]);
    }
    fence_proxy_async_smem();
  }
  if (HALVES) {
    __threadfence_block();
    any |= *reinterpret_cast<volatile uint32_t*>(bad) >> lane & 1u;
  }
  return any != 0 ? 0x7fff7fffu : 0u;
}

// Masks of the pairs of a key with 32 queries: 16 bits of ones for each query that sees it.  R4: the queries' ranges (see
// Stage), eight rows each; here: the key's position in its tile, as added to a row's bytes.
FA_DEV void seen_pairs(const uint4* R4, uint32_t here, uint32_t (&see)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 r = R4[i];
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t t = w[e] + here;  // bits 7 and 15, 23 and 31: at or behind the first key, before the last
      see[4 * i + e] = (((t & (t >> 8)) >> 7) & 0x00010001u) * 0xffffu;
    }
  }
}

// A unit of more than 1.5 times the steps that an SM has on the average (and of 8 at least) is taken in kParts parts, each
// with its share of the query tiles for all heads, whose sums the last kernel adds up.  There are fewer such units than
// SMs.  (4096 tokens of packed documents, 4 key heads of 4 query heads each, 2 sequences: 41 steps on the fullest SM, 49
// with whole units, 29 on the average.)  Pieces are dealt out to and fro as in UnitWalk, in the order of the key tiles'
// work, so that the CTAs stay at the same query heads at a time: all of Q, dO and the sums of dQ may be more than L2.
// Measured and not kept, main kernel: equal runs of steps per CTA whatever the units (8192 tokens, 32 + 8 heads: 1.76 ms where whole units take 1.39); a queue, with long units split by query heads (4096
// tokens in one document: 475 us, 349).
constexpr int kParts = 2;
// How many key tiles of the mask's order are split.
FA_DEV int split_places(const MaskView& m, int heads, int G, int ctas) {
  const long long least = max(m.k_work->tiles * heads * 3 / (2 * ctas) + 1, (8LL + G - 1) / G);
  if (least > m.Tq || least < kParts) return 0;
  // those with at least that many query tiles
  return min(m.k_work->before[work_class(static_cast<int>(least), m.Tq) + (m.Tq < kWorkClasses - 1 ? 1 : 0)], ctas / heads);
}

// Element-wise warps (warp w of 4..11: lane quarter qw = w % 4, query half h = (w-4)/4; one key row per thread): P^T and
// dS^T of step g.  k_first: first key of the tile; q_first: position of the query tile's first row.  poison: the key's, of
// clean_key; any_poison: some key of the warp has one.
template <class LY, int MOD>
FA_DEV bool ew_ranges(const Ctx& x, const ScoreMod& mod, int g, int k_first, int q_first, int qw, int h, int lane,
                      uint32_t poison, bool any_poison) {
  constexpr bool CAP = (MOD & kModCap) != 0, BIAS = (MOD & kModBias) != 0;
  // (as ew_step: at d = 128 the weights go to the dV product once dP^T is out of tensor memory; with a cap the registers
  // hold half of dP^T at a time)
  constexpr bool DP_FIRST = LY::TQ == 128 * 128 * 2 && !CAP;
  const int s = g & 1;
  const int kr = qw * 32 + lane;  // key row (tensor-memory lane)
  const uint32_t tl = x.tmem + (static_cast<uint32_t>(qw * 32) << 16);
  if (!mbar_wait_warp(x.bar(B_QFULL + s), (g >> 1) & 1, x.guard, SITE_RB_COMPUTE)) return false;
  if (!mbar_wait_warp(x.bar(B_SFULL), g & 1, x.guard, SITE_RB_COMPUTE)) return false;
  tc_fence_after();
  const uint32_t rs = tl + TM_R + 128 * s, rd = tl + TM_R + 128 * (s ^ 1);
  const Stage* st = stage_of(x, g);
  const float4* L4 = reinterpret_cast<const float4*>(st->L) + 16 * h;
  const float4* D4 = reinterpret_cast<const float4*>(st->D) + 16 * h;
  const uint4* R4 = reinterpret_cast<const uint4*>(st->ranges) + 8 * h;  // eight rows each
  const bool masked = st->masked != 0 || any_poison;
  // a row's bytes plus these have bit 7 and bit 15 set where the row sees this key (see Stage)
  const uint32_t here = (static_cast<uint32_t>(kr) | static_cast<uint32_t>(127 - kr) << 8) * 0x10001u;
  if (st->dead) {  // (all products that read Q and dO so far are done)
    if (!mbar_wait_warp(x.bar(B_DPFULL), g & 1, x.guard, SITE_RB_COMPUTE)) return false;
    const uint32_t r = reinterpret_cast<const uint16_t*>(st->ranges)[kr];
    if (static_cast<int>(r >> 8) <= BN - static_cast<int>(r & 255u)) {  // row kr sees no key of this tile
      uint8_t* row = x.tiles + LY::T_Q + s * 2 * LY::TQ + h * LY::TQ + kr * 128;  // of Q, or of dO
#pragma unroll 1
      for (int c = 0; c < LY::TQ / CHUNK; ++c)
#pragma unroll
        for (int u = 0; u < 8; ++u) *reinterpret_cast<uint4*>(row + c * CHUNK + 16 * u) = make_uint4(0u, 0u, 0u, 0u);
      fence_proxy_async_smem();
    }
  }
  const uint64_t cc = f2pack(mod.c_log2, mod.c_log2);
  const float slope = BIAS ? st->slope : 0.f;
  const int d0 = q_first + 64 * h - (k_first + kr);  // position of the half's first query less this key's
  const int side = q_first + 64 * h >= k_first + BN - 1 ? 1 : q_first + 64 * h + 63 <= k_first ? -1 : 0;
  const float ss = side >= 0 ? slope : -slope;
  // ---- P^T = 2^(score - L log2 e), two sub-chunks of 32 queries
  uint32_t pk[32];
  [[maybe_unused]] uint32_t pr[CAP ? 32 : 1];  // P r
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint32_t r[32];
    tmem_ld32(rs + 64 * h + 32 * c, r);
    tmem_ld_wait<32>(r);
    float sc[32];
#pragma unroll
    for (int v = 0; v < 32; ++v) sc[v] = __uint_as_float(r[v]);
    [[maybe_unused]] float rate[CAP ? 32 : 1];  // 1 - tanh^2, over kRateScale
    if constexpr (CAP) cap_scores_rate(sc, rate, mod.cap);
    if constexpr (BIAS) {
      const float dist = static_cast<float>(d0 + 32 * c);
      if (side != 0) {
        const float at = -ss * dist;
        const uint64_t step = f2pack(-2.f * ss, -2.f * ss);
#pragma unroll
        for (int v0 = 0; v0 < 32; v0 += 8) {  // (the steps' roundings do not add up beyond 8 queries)
          uint64_t b2 = f2pack(fmaf(-ss, static_cast<float>(v0), at), fmaf(-ss, static_cast<float>(v0 + 1), at));
#pragma unroll
          for (int v = v0; v < v0 + 8; v += 2) {
            const uint64_t x = f2pack(sc[v], sc[v + 1]);
            f2unpack(CAP ? fadd2(x, b2) : ffma2(x, cc, b2), sc[v], sc[v + 1]);
            b2 = fadd2(b2, step);
          }
        }
      } else {
#pragma unroll
        for (int v = 0; v < 32; ++v)
          sc[v] = fmaf(sc[v], CAP ? 1.f : mod.c_log2, -slope * fabsf(dist + static_cast<float>(v)));
      }
    }
    {
#pragma unroll
      for (int v = 0; v < 8; ++v) {
        const float4 l = L4[8 * c + v];
#pragma unroll
        for (int y = 0; y < 4; y += 2) {
          const int xx = 4 * v + y;  // within the sub-chunk
          const uint64_t x2 = f2pack(sc[xx], sc[xx + 1]);
          const uint64_t add = y == 0 ? f2pack(l.x, l.y) : f2pack(l.z, l.w);
          float t0, t1;
          f2unpack(CAP || BIAS ? fadd2(x2, add) : ffma2(x2, cc, add), t0, t1);
          float p0 = ex2(t0), p1 = ex2(t1);
          pk[16 * c + (xx >> 1)] = pack_bf16x2(p0, p1);
          if constexpr (CAP) {
            float q0, q1;
            f2unpack(fmul2(f2pack(p0, p1), f2pack(rate[xx], rate[xx + 1])), q0, q1);
            pr[16 * c + (xx >> 1)] = pack_bf16x2(q0, q1);
          }
        }
      }
    }
    if (masked) {
      uint32_t see[16];
      seen_pairs(R4 + 4 * c, here, see);
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        pk[16 * c + v] = (pk[16 * c + v] | poison) & see[v];
        if constexpr (CAP) pr[16 * c + v] = (pr[16 * c + v] | poison) & see[v];
      }
    }
    tmem_st16(rs + 64 * h + 16 * c, pk + 16 * c);
    if (!DP_FIRST) {
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(x.bar(B_PREADY + 2 * s + c));
    }
  }
  if (DP_FIRST) tmem_st_wait();
  // ---- dS^T = P^T r (dP^T - D)
  if (!mbar_wait_warp(x.bar(B_DPFULL), g & 1, x.guard, SITE_RB_COMPUTE)) return false;
  tc_fence_after();
  uint8_t* row = x.tiles + LY::T_DS + h * CHUNK + kr * 128;
  constexpr int NDP = CAP ? 32 : 64;  // dP^T columns in registers at a time
  uint32_t rdp[NDP];
  if constexpr (!CAP) {
    // all of this thread's dP^T out of tensor memory first, so that S^T of the next step can be formed in its region
    tmem_ld32(rd + 64 * h, rdp);
    tmem_ld32(rd + 64 * h + 32, rdp + 32);
    tmem_ld_wait<64>(rdp);
    tc_fence_before();
    if (DP_FIRST) {
      mbar_arrive(x.bar(B_PREADY + 2 * s));
      mbar_arrive(x.bar(B_PREADY + 2 * s + 1));
    }
    mbar_arrive(x.bar(B_DPCONS));
  }
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    if constexpr (CAP) {
      tmem_ld32(rd + 64 * h + 32 * c, rdp);
      tmem_ld_wait<32>(rdp);
      if (c == 1) {
        tc_fence_before();
        mbar_arrive(x.bar(B_DPCONS));
      }
    }
    const uint32_t* r = rdp + (CAP ? 0 : 32 * c);
    uint32_t dk[16];
    {
#pragma unroll
      for (int v = 0; v < 8; ++v) {
        const float4 dd = D4[8 * c + v];
#pragma unroll
        for (int y = 0; y < 4; y += 2) {
          const int xx = 4 * v + y;
          const uint32_t w = CAP ? pr[16 * c + (xx >> 1)] : pk[16 * c + (xx >> 1)];
          const float p0 = __uint_as_float(w << 16), p1 = __uint_as_float(w & 0xffff0000u);
          const uint64_t t = fadd2(f2pack(__uint_as_float(r[xx]), __uint_as_float(r[xx + 1])),
                                   y == 0 ? f2pack(-dd.x, -dd.y) : f2pack(-dd.z, -dd.w));
          float e0, e1;
          f2unpack(fmul2(f2pack(p0, p1), t), e0, e1);
          dk[xx >> 1] = pack_bf16x2(e0, e1);
        }
      }
    }
    if (masked) {  // (dP of a masked pair may be NaN)
      uint32_t see[16];
      seen_pairs(R4 + 4 * c, here, see);
#pragma unroll
      for (int v = 0; v < 16; ++v) dk[v] &= see[v];
    }
    tmem_st16(rs + 64 * h + 32 + 16 * c, dk);
    // dS^T row kr, queries 64h + 32c .. +31: four 16-byte units of the swizzled row
#pragma unroll
    for (int u = 0; u < 4; ++u)
      *reinterpret_cast<uint4*>(row + (((4 * c + u) ^ (kr & 7)) << 4)) =
          make_uint4(dk[4 * u], dk[4 * u + 1], dk[4 * u + 2], dk[4 * u + 3]);
    tmem_st_wait();
    tc_fence_before();
    mbar_arrive(x.bar(B_DSREADY + c));  // dK reads dS^T from tensor memory
  }
  // dQ^T reads dS^T from shared memory: one proxy fence for both sub-chunks
  fence_proxy_async_smem();
  mbar_arrive(x.bar(B_DSSMEM));
  return true;
}

// D: the tiles' head size (64, 128); DR: the tensors' (32 runs in D = 64).
template <int D, int DR, int MOD>
__global__ void __launch_bounds__(NTHREADS, 1)
    bwd_ranges_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmdO,
                      const __grid_constant__ BwdRangesArgs a) {
  using LY = LayFor<D>;
  constexpr int NKV = LY::NKV;  // K, V buffers
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* tiles = align1024(smem_raw + RSMALL);
  if (tiles + LY::TILES > smem_raw + LY::SMEM) {
    if (threadIdx.x == 0) atomicCAS(a.status, 0, SITE_RB_LAYOUT);
    return;
  }
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem_raw + ROFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem_raw + ROFF_MISC + 4);
  Ctx x{smem_u32(smem_raw), smem_u32(tiles), smem_raw, tiles, 0u, Guard{a.status, abort_flag}};
  auto bar = [&](int i) -> uint32_t { return x.bar(i); };
  const MaskView& m = a.m;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int b = 0; b < NKV; ++b) {
      mbar_init(bar(kvfull(b)), 1);
      mbar_init(bar(kvfree(b)), 2);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(B_QFULL + s), 1 + 32);  // TMA bytes + the producer's 32 lanes (Stage)
      mbar_init(bar(B_QEMPTY + s), 1);
    }
    for (int s = 0; s < kRing; ++s) {
      mbar_init(bar(B_UFULL + s), 1);
      mbar_init(bar(B_UEMPTY + s), UEMPTY_COUNT);
    }
    mbar_init(bar(B_SFULL), 1);
    mbar_init(bar(B_DPFULL), 1);
    for (int c = 0; c < 2; ++c) {
      mbar_init(bar(B_PREADY + c), NCOMP);
      mbar_init(bar(B_PREADY + 2 + c), NCOMP);
      mbar_init(bar(B_DSREADY + c), NCOMP);
    }
    mbar_init(bar(B_DPCONS), NCOMP);
    mbar_init(bar(B_DSSMEM), NCOMP);
    mbar_init(bar(B_DKDONE), 1);
    mbar_init(bar(B_DQFULL), 1);
    mbar_init(bar(B_DQCONS), NDQ);
    mbar_init(bar(B_FINAL), 1);
    mbar_init(bar(B_ADONE), 1);
    mbar_init(bar(B_DKVFULL), 1);
    mbar_init(bar(B_DKVFREE), NCOMP);
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmdO);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), TM_COLS);
    tmem_relinquish();
  }
  uint32_t* bad_keys = reinterpret_cast<uint32_t*>(smem_raw + ROFF_BAD);
  if (threadIdx.x < 8) bad_keys[threadIdx.x] = 0u;
  // (pdl_wait: before D is read and before the first sums of dQ)
  if (threadIdx.x == 64) *abort_flag = (*reinterpret_cast<volatile int*>(a.status) != 0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  x.tmem = *tmem_slot;
  const bool skip = *abort_flag != 0;

  // A role's unit: entry i of the ring, copied and released at once; false: no more, or gave up.
  Unit* ring = reinterpret_cast<Unit*>(smem_raw + ROFF_RING);
  auto take = [&](int* i, Unit* u, bool whole_warp, int site) {
    const int slot = *i % kRing;
    const uint32_t par = (*i / kRing) & 1;
    if (!(whole_warp ? mbar_wait_warp(bar(B_UFULL + slot), par, x.guard, site) : mbar_wait(bar(B_UFULL + slot), par, x.guard, site)))
      return false;
    const volatile Unit* at = ring + slot;
    u->lo = at->lo, u->n = at->n, u->b = at->b, u->kt = at->kt, u->h = at->h;
    u->slot = at->slot;
    if (whole_warp) __syncwarp();
    if (!whole_warp || lane == 0) mbar_arrive(bar(B_UEMPTY + slot));
    ++*i;
    return u->n >= 0;
  };

  if (warp < 4) {
    regs_dec<72>();
    if (warp == 0 && !skip) {
      // ---------------------------------------------------------------- producer (whole warp)
      int g = 0, last = -1, kvk = -1, i = 0;  // steps so far; last step and unit whose loads were issued; ring entries
      bool ok = true;
      auto hand_out = [&](const Unit& u) {
        const int slot = i % kRing;
        if (i >= kRing && !mbar_wait_warp(bar(B_UEMPTY + slot), ((i / kRing) & 1) ^ 1, x.guard, SITE_RB_PRODUCER)) return false;
        if (lane == 0) {
          ring[slot] = u;
          mbar_arrive(bar(B_UFULL + slot));
        }
        __syncwarp();
        ++i;
        return true;
      };
      int k = 0;  // units with steps
      // the first piece if no unit is split: its tables come while that is found out
      int next_entry = m.k_order[min(static_cast<int>(blockIdx.x) / a.Hk, m.B * m.Tk - 1)];
      KeyTile next = m.kt[next_entry];
      const int some = m.k_work->some, split = some > 0 ? split_places(m, a.Hk, a.G, gridDim.x) : 0;
      const int pieces = split * a.Hk * kParts, total = pieces + (some - split) * a.Hk;
      // CTA c takes pieces c, 2 grid - 1 - c, 2 grid + c, ...; the next one is looked up while this one's steps are loaded
      const int grid = gridDim.x, cta = blockIdx.x;
      int round = 0, v = cta;
      auto look = [&] {
        if (v >= total) return;
        next_entry = m.k_order[v < pieces ? v / (a.Hk * kParts) : split + (v - pieces) / a.Hk];
        next = m.kt[next_entry];
      };
      if (split > 0) look();
      while (ok && v < total) {
        const int entry = next_entry, e = v < pieces ? v / kParts : v - pieces;
        Unit u{next.lo, next.n, entry / m.Tk, 0, e % a.Hk, kWhole};
        u.kt = entry - u.b * m.Tk;
        if (v < pieces) {  // its share of the query tiles
          const int part = v % kParts, from = next.n * part / kParts;
          u.lo += from, u.n = next.n * (part + 1) / kParts - from, u.slot = v;
        }
        ++round;
        v = round * grid + ((round & 1) ? grid - 1 - cta : cta);
        look();
        if (!(ok = hand_out(u))) break;
        // K and V of this unit into buffer k % NKV, once the last readers of unit k - NKV are done
        const int b = k % NKV;
        if (k >= NKV && !(ok = mbar_wait_warp(bar(kvfree(b)), (k / NKV - 1) & 1, x.guard, SITE_RB_PRODUCER))) break;
        if (lane == 0) {
          mbar_expect_tx(bar(kvfull(b)), LY::KVB);
          for (int c = 0; c < 2; ++c)  // at D = 64 the second K chunk is a copy of the first
            tma_load_4d(LY::k(x.tb, b) + c * CHUNK, &tmK, bar(kvfull(b)), D == 128 ? c * 64 : 0, u.kt * BN, u.h * a.kh,
                        u.b * a.kb);
          for (int c = 0; c < LY::TQ / CHUNK; ++c)
            tma_load_4d(LY::v(x.tb, b) + c * CHUNK, &tmV, bar(kvfull(b)), c * 64, u.kt * BN, u.h * a.vh, u.b * a.vb);
        }
        kvk = k;
        if (k == 0) pdl_wait();  // D is the kernel before's
        for (int hq = u.h * a.G; ok && hq < u.h * a.G + a.G; ++hq)
          for (int it = 0; it < u.n; ++it, ++g) {
            if (!(ok = produce<LY, MOD>(x, &tmQ, &tmdO, a, u.b, hq, u.lo + it, u.kt, g, lane))) break;
            last = g;
          }
        if (!ok) break;
        ++k;
      }
      // key tiles that no row sees, behind all others in the order
      const int places = m.B * m.Tk;
      for (int u0 = blockIdx.x; ok && u0 < (places - some) * a.Hk; u0 += gridDim.x) {
        const int entry = m.k_order[some + u0 / a.Hk], b = entry / m.Tk;
        ok = hand_out(Unit{0, 0, b, entry - b * m.Tk, u0 % a.Hk, kWhole});
      }
      if (ok) hand_out(Unit{0, -1, 0, 0, 0, kWhole});
      if (lane == 0 && *abort_flag) {
        for (int kk = (kvk >= NKV ? kvk - NKV + 1 : 0); kk <= kvk; ++kk)  // the K, V loads in flight
          mbar_drain(bar(kvfull(kk % NKV)), (kk / NKV) & 1);
        for (int it = (last > 0 ? last - 1 : 0); it <= last; ++it) mbar_drain(bar(B_QFULL + (it & 1)), (it >> 1) & 1);
      }
    } else if (warp == 1 && lane == 0 && !skip) {
      // ---------------------------------------------------------------- UMMA issuer A: S^T, dP^T
      bool ok = true;
      int g = 0, i = 0;
      Unit u;
      for (int k = 0; ok && take(&i, &u, false, SITE_RB_MMA);) {
        if (u.n == 0) continue;
        const int b = k % NKV;
        if (!(ok = mbar_wait(bar(kvfull(b)), (k / NKV) & 1, x.guard, SITE_RB_MMA))) break;
        for (int it = 0; ok && it < u.n * a.G; ++it, ++g) ok = issue_a<LY>(x, g, b);
        if (!ok) break;
        mma_commit(bar(kvfree(b)));  // this unit's S^T, dP^T products (the readers of K, V here) are done
        ++k;
      }
      mma_commit(bar(B_ADONE));
    } else if (warp == 2 && lane == 0 && !skip) {
      // ---------------------------------------------------------------- UMMA issuer B: dV, dK, dQ^T
      bool ok = true;
      int g = 0, i = 0;
      Unit u;
      for (int k = 0; ok && take(&i, &u, false, SITE_RB_MMA);) {
        if (u.n == 0) continue;
        // dK, dV of the previous unit are out of tensor memory
        if (k > 0 && !(ok = mbar_wait(bar(B_DKVFREE), (k - 1) & 1, x.guard, SITE_RB_MMA))) break;
        const int b = k % NKV;
        if (!(ok = mbar_wait(bar(kvfull(b)), (k / NKV) & 1, x.guard, SITE_RB_MMA))) break;
        for (int it = 0; ok && it < u.n * a.G; ++it, ++g) ok = issue_b<LY>(x, g, b, it == 0);
        if (!ok) break;
        mma_commit(bar(B_DKVFULL));  // this unit's dK, dV are complete
        mma_commit(bar(kvfree(b)));  // and its dQ^T products (the last readers of K) are done
        ++k;
      }
      mma_commit(bar(B_FINAL));
    }
  } else if (warp >= 12) {
    regs_inc<144>();
    if (!skip) {
      // ---------------------------------------------------------------- dQ drain
      pdl_wait();  // the sums are cleared by the kernel before
      const int qw = warp & 3;
      bool ok = true;
      int g = 0, i = 0;
      Unit u;
      while (ok && take(&i, &u, true, SITE_RB_COMPUTE)) {
        for (int hq = u.h * a.G; ok && hq < u.h * a.G + a.G; ++hq) {
          const size_t row0 = (static_cast<size_t>(u.b) * a.H + hq) * m.Nq;
          for (int it = 0; ok && it < u.n; ++it, ++g) {
            const int q0 = (u.lo + it) * BM;
            ok = drain<D, DR>(x, g, a.dQacc + (row0 + q0) * DR, min(BM, m.Nq - q0), qw, lane);
          }
        }
      }
    }
  } else {
    regs_inc<144>();
    if (!skip) {
      // ---------------------------------------------------------------- element-wise warps
      const int qw = warp & 3;
      const int h = (warp - 4) >> 2;
      bool ok = true;
      int g = 0, i = 0;
      for (int k = 0; ok;) {
        Unit u;
        if (!take(&i, &u, true, SITE_RB_COMPUTE)) break;
        const int row0 = u.kt * BN + qw * 32;  // the warp's first key
        const size_t krow0 = (static_cast<size_t>(u.b) * a.Hk + u.h) * m.Nk + row0;
        if (u.n == 0) {  // no row sees these keys
          if (lane < m.Nk - row0 && h == 0) {
#pragma unroll 1
            for (int e = 0; e < DR / 8; ++e) {
              reinterpret_cast<uint4*>(a.dK + (krow0 + lane) * DR)[e] = make_uint4(0u, 0u, 0u, 0u);
              reinterpret_cast<uint4*>(a.dV + (krow0 + lane) * DR)[e] = make_uint4(0u, 0u, 0u, 0u);
            }
          }
          continue;
        }
        const int b = k % NKV;
        if (!(ok = mbar_wait_warp(bar(kvfull(b)), (k / NKV) & 1, x.guard, SITE_RB_COMPUTE))) break;
        // before this unit's first dQ^T, which waits for these warps.  The other unit's bits were last read before the steps
        // of the unit before this one, and are next set after this one's.
        if (threadIdx.x == 128)
          for (int e = 0; e < 4; ++e) bad_keys[4 * ((k + 1) & 1) + e] = 0u;
        const uint32_t poison = clean_key<LY>(x, b, bad_keys + 4 * (k & 1) + qw, h, qw * 32 + lane, lane);
        const bool any_poison = __any_sync(0xffffffffu, poison != 0);
        const int q_lo = u.lo * BM + m.Nk - m.Nq;
        for (int hq = 0, it = 0; hq < a.G; ++g) {
          if (!(ok = ew_ranges<LY, MOD>(x, a.mod, g, u.kt * BN, q_lo + it * BM, qw, h, lane, poison,
                                        any_poison)))
            break;
          if (++it == u.n) it = 0, ++hq;
        }
        if (!ok) break;
        if (!(ok = mbar_wait_warp(bar(B_DKVFULL), k & 1, x.guard, SITE_RB_COMPUTE))) break;
        tc_fence_after();
        // dK (times scale) and dV, 32 columns at a time (a loop: the code of all roles has to fit the instruction cache)
        constexpr int CHUNKS = D / 64;  // of this half's columns of dK, and of dV
#pragma unroll 1
        for (int c = 0; c < 2 * CHUNKS; ++c) {
          const bool is_k = c < CHUNKS;
          const int col = D / 2 * h + 32 * (is_k ? c : c - CHUNKS);
          uint32_t r[32], o[16];
          tmem_ld32(x.tmem + (static_cast<uint32_t>(qw * 32) << 16) + (is_k ? TM_DK : TM_DV) + col, r);
          tmem_ld_wait<32>(r);
          if (c == 2 * CHUNKS - 1) {
            tc_fence_before();
            mbar_arrive(bar(B_DKVFREE));
          }
          if (u.slot != kWhole) {  // sums of some of the unit's steps
            float* to = a.part + ((static_cast<size_t>(u.slot) * 2 + (is_k ? 0 : 1)) * BN + qw * 32) * D + col;
            uint4* row = reinterpret_cast<uint4*>(to + static_cast<size_t>(lane) * D);
#pragma unroll
            for (int e = 0; e < 8; ++e) row[e] = make_uint4(r[4 * e], r[4 * e + 1], r[4 * e + 2], r[4 * e + 3]);
            continue;
          }
          const float f = is_k ? a.scale : 1.f;
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = scaled_bf16x2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]), f);
          if (DR == D || h == 0)  // (d = 32: the other half is padding)
            warp_store_rows<4, 0>(o, reinterpret_cast<uint8_t*>((is_k ? a.dK : a.dV) + krow0 * DR + (DR == D ? col : 0)),
                                  DR * 2, m.Nk - row0, lane);
        }
        ++k;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    if (!skip && *abort_flag) {
      if (lane == 0) {
        mbar_drain(bar(B_ADONE), 0);
        mbar_drain(bar(B_FINAL), 0);
      }
      __syncwarp();
    }
    tc_fence_after();
    tmem_dealloc(x.tmem, TM_COLS);
  }
  pdl_wait();  // a CTA that skipped its work has not waited: what follows may rely on the kernel before having ended
}

// D = rowsum(dO * O) of every row (0 where the row sees no key: its dO may be anything), and the row's dQ sums cleared.
template <int D>
__global__ void __launch_bounds__(256) bwd_ranges_prepare(const __nv_bfloat16* __restrict__ O,
                                                          const __nv_bfloat16* __restrict__ dO, RowStrides sd,
                                                          const float* __restrict__ L, float* __restrict__ Dout,
                                                          float* __restrict__ dQacc, int H, int N, long long rows) {
  constexpr int LPR = D / 8;
  pdl_wait();
  pdl_trigger();  // what is before this kernel is done: the next one may load all but D, and sets up meanwhile
  const int part = threadIdx.x % LPR;
  const long long step = static_cast<long long>(gridDim.x) * (256 / LPR);
  for (long long r0 = static_cast<long long>(blockIdx.x) * (256 / LPR); r0 < rows; r0 += step) {
    const long long r = r0 + threadIdx.x / LPR;
    float acc = 0.f;
    if (r < rows) {
      const long long bh = r / N, n = r - bh * N, b = bh / H, h = bh - b * H;
      const uint4 x = *reinterpret_cast<const uint4*>(O + r * D + part * 8);
      const uint4 y = *reinterpret_cast<const uint4*>(dO + b * sd.b + h * sd.h + n * sd.n + part * 8);
      float4* z = reinterpret_cast<float4*>(dQacc + r * D + part * 8);
      z[0] = z[1] = make_float4(0.f, 0.f, 0.f, 0.f);
      const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc = fmaf(__uint_as_float(xs[e] << 16), __uint_as_float(ys[e] << 16), acc);
        acc = fmaf(__uint_as_float(xs[e] & 0xffff0000u), __uint_as_float(ys[e] & 0xffff0000u), acc);
      }
    }
#pragma unroll
    for (int k = LPR / 2; k > 0; k >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, k);
    if (r < rows && part == 0) Dout[r] = L[r] == -INFINITY ? 0.f : acc;
  }
}

// The last launch: dQ = scale times its sums, rounded; and dK, dV of the split units, the parts added up in order
// (kJoin blocks a unit, behind the others).
constexpr int kJoin = 4;
template <int D, int DR>
__global__ void __launch_bounds__(256) bwd_ranges_finish(const __grid_constant__ BwdRangesArgs a, __nv_bfloat16* dQ,
                                                         long long n8, int ctas) {
  pdl_wait();
  if (*reinterpret_cast<volatile int*>(a.status) != 0) return;  // the kernel before gave up
  const int converts = gridDim.x - ctas * kJoin, join = static_cast<int>(blockIdx.x) - converts;
  if (join >= 0) {
    const MaskView& m = a.m;
    const int unit = join / kJoin;
    if (m.k_work->some == 0 || unit >= split_places(m, a.Hk, a.G, ctas) * a.Hk) return;
    const int entry = m.k_order[unit / a.Hk], h = unit % a.Hk, b = entry / m.Tk, row0 = (entry - b * m.Tk) * BN;
    constexpr int V = DR / 4, TILE = BN * D;  // float4 pieces of a row; floats of a tensor's part
    const size_t out0 = (static_cast<size_t>(b) * a.Hk + h) * m.Nk + row0;
    const float* parts = a.part + static_cast<size_t>(unit) * kParts * 2 * TILE;
    for (int i = join % kJoin * 256 + threadIdx.x; i < 2 * BN * V; i += kJoin * 256) {
      const int t = i / (BN * V), row = i / V % BN, col = i % V * 4;
      if (row >= m.Nk - row0) continue;
      float4 x[kParts];
#pragma unroll
      for (int k = 0; k < kParts; ++k)
        x[k] = *reinterpret_cast<const float4*>(parts + static_cast<size_t>(2 * k + t) * TILE + row * D + col);
#pragma unroll
      for (int k = 1; k < kParts; ++k) x[0].x += x[k].x, x[0].y += x[k].y, x[0].z += x[k].z, x[0].w += x[k].w;
      const float f = t == 0 ? a.scale : 1.f;
      *reinterpret_cast<uint2*>((t == 0 ? a.dK : a.dV) + (out0 + row) * DR + col) =
          make_uint2(scaled_bf16x2(x[0].x, x[0].y, f), scaled_bf16x2(x[0].z, x[0].w, f));
    }
    return;
  }
  const long long step = static_cast<long long>(converts) * 256;
  for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < n8; i += step) {
    const float4 x = __ldcs(reinterpret_cast<const float4*>(a.dQacc + 8 * i)), y = __ldcs(reinterpret_cast<const float4*>(a.dQacc + 8 * i + 4));
    *reinterpret_cast<uint4*>(dQ + 8 * i) =
        make_uint4(scaled_bf16x2(x.x, x.y, a.scale), scaled_bf16x2(x.z, x.w, a.scale),
                   scaled_bf16x2(y.x, y.y, a.scale), scaled_bf16x2(y.z, y.w, a.scale));
  }
}

constexpr int kMaxGrid = 152;  // CTAs at most, one per SM
size_t round16(size_t n) { return (n + 15) / 16 * 16; }

// CTAs at most: no more than there can be pieces.
int most_ctas(int B, int Hk, int Nk) {
  const long long pieces = static_cast<long long>(B) * Hk * ((Nk + BN - 1LL) / BN) * kParts;
  return static_cast<int>(pieces < kMaxGrid ? pieces : kMaxGrid);
}

// Where what is in the workspace.
struct Work {
  size_t acc, part, bytes;
};
Work work_of(int B, int H, int Hk, int Nq, int Nk, int d) {
  const size_t rows = static_cast<size_t>(B) * H * Nq, ctas = most_ctas(B, Hk, Nk);
  Work w;
  w.acc = round16(rows * 4);
  w.part = w.acc + rows * d * 4;
  w.bytes = w.part + ctas * kParts * 2 * BN * (d == 128 ? 128 : 64) * 4;  // no more split units than CTAs
  return w;
}

template <int D, int DR, int MOD>
fa_status launch(const RangesLaunch& a) {
  using LY = LayFor<D>;
  const long long rows = static_cast<long long>(a.B) * a.H * a.Nq;
  const Work w = work_of(a.B, a.H, a.Hk, a.Nq, a.Nk, a.d);
  float* Dbuf = reinterpret_cast<float*>(a.workspace);
  float* acc = reinterpret_cast<float*>(a.workspace + w.acc);
  int dev = 0, nsm = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return FA_ERR_CUDA;
  const long long row_blocks = (rows + 256 / (DR / 8) - 1) / (256 / (DR / 8)), most_blocks = 8LL * nsm;
  if (launch_pdl(bwd_ranges_prepare<DR>, dim3(static_cast<unsigned>(row_blocks < most_blocks ? row_blocks : most_blocks)),
                 dim3(256), 0, a.stream, static_cast<const __nv_bfloat16*>(a.O), static_cast<const __nv_bfloat16*>(a.dO),
                 a.sdo, a.Lin, Dbuf, acc, a.H, a.Nq, rows) != cudaSuccess)
    return FA_ERR_CUDA;
  const long long units = static_cast<long long>(a.B) * a.mask.Tk * a.Hk;
  if (units > INT_MAX / 2) return FA_ERR_UNSUPPORTED;
  const int most = most_ctas(a.B, a.Hk, a.Nk), grid = most < nsm ? most : nsm;
  const BwdRangesArgs args{a.mask, a.mod, a.Lin, Dbuf, acc, static_cast<__nv_bfloat16*>(a.dK),
                           static_cast<__nv_bfloat16*>(a.dV), reinterpret_cast<float*>(a.workspace + w.part), a.H, a.Hk, a.H / a.Hk,
                           a.sq.h != 0, a.sq.b != 0, a.sk.h != 0, a.sk.b != 0, a.sv.h != 0, a.sv.b != 0, a.sdo.h != 0,
                           a.sdo.b != 0, a.scale * (MOD & kModCap ? kRateScale : 1.f), a.status};
  if (units > 0) {
    CUtensorMap mQ, mK, mV, mdO;
    if (!encode_bf16_rows(&mK, a.K, DR, a.Nk, a.Hk, a.B, a.sk, 64, BN) ||
        !encode_bf16_rows(&mV, a.V, DR, a.Nk, a.Hk, a.B, a.sv, 64, BN) ||
        !encode_bf16_rows(&mQ, a.Q, DR, a.Nq, a.H, a.B, a.sq, 64, BM) ||
        !encode_bf16_rows(&mdO, a.dO, DR, a.Nq, a.H, a.B, a.sdo, 64, BM))
      return FA_ERR_CUDA;
    auto kern = bwd_ranges_kernel<D, DR, MOD>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, LY::SMEM) != cudaSuccess)
      return FA_ERR_CUDA;
    if (launch_pdl(kern, dim3(grid), dim3(NTHREADS), LY::SMEM, a.stream, mQ, mK, mV, mdO, args) != cudaSuccess)
      return FA_ERR_CUDA;
  }
  const long long n8 = rows * DR / 8, blocks = (n8 + 255) / 256;
  const int ctas = units > 0 ? grid : 0, converts = static_cast<int>(blocks < 16LL * nsm ? blocks : 16LL * nsm);
  return launch_pdl(bwd_ranges_finish<D, DR>, dim3(ctas * kJoin + converts), dim3(256), 0, a.stream, args,
                    static_cast<__nv_bfloat16*>(a.dQ), n8, ctas) == cudaSuccess
             ? FA_OK : FA_ERR_CUDA;
}

template <int D, int DR>
fa_status launch_mod(const RangesLaunch& a) {
  const bool cap = a.mod.cap.cap_log2 > 0.f, bias = a.mod.slopes != nullptr;
  return cap ? (bias ? launch<D, DR, kModCap | kModBias>(a) : launch<D, DR, kModCap>(a))
             : (bias ? launch<D, DR, kModBias>(a) : launch<D, DR, kModNone>(a));
}

}  // namespace

size_t bwd_ranges_workspace(int B, int H, int Hk, int Nq, int Nk, int d) { return work_of(B, H, Hk, Nq, Nk, d).bytes; }

fa_status launch_bwd_ranges(const RangesLaunch& a) {
  if (a.Nq == 0 || a.H == 0) {  // no row, whatever the mask lists (B, Hk and Nk are not 0: fa_bwd_ranges)
    const size_t bytes = static_cast<size_t>(a.B) * a.Hk * a.Nk * a.d * 2;
    const fa_status st = launch_zero(a.dK, bytes, a.stream);
    return st != FA_OK ? st : launch_zero(a.dV, bytes, a.stream);
  }
  return a.d == 32 ? launch_mod<64, 32>(a) : a.d == 64 ? launch_mod<64, 64>(a) : launch_mod<128, 128>(a);
}

}  // namespace fa
