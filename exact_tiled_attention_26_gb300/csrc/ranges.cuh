// The mask of attention over ranges (a range of keys for each query row) as its kernels see it, and the scores'
// modifications.
#pragma once

#include <limits.h>

#include "internal.h"
#include "ptx.cuh"
#include "ranges_score.cuh"

namespace fa {

constexpr int kRangeTile = 128;  // rows of a query tile and keys of a key tile
constexpr int kNoFull = INT_MAX;

// A query tile: the key tiles lo .. lo + n - 1 hold every key that one of its rows sees (n = 0: none); a key tile
// whose keys all lie in [full_first, full_last) is seen whole by every row (full_first = kNoFull: a row sees nothing).
struct __align__(16) QueryTile {
  int lo, n, full_first, full_last;
};
// A key tile: query tiles lo .. lo + n - 1 hold every row that sees one of its keys.
struct __align__(8) KeyTile {
  int lo, n;
};

// Classes of the orders: class 0 for tiles with `most` tiles of work, the last for those without any.
constexpr int kWorkClasses = 2048;
__host__ __device__ inline int work_class(int n, int most) {
  if (n == 0) return kWorkClasses - 1;
  return most < kWorkClasses - 1 ? most - n
                                 : static_cast<int>(static_cast<long long>(most - n) * (kWorkClasses - 2) / most);
}
// The key tiles' work: their query tiles together (a class counted as its largest), how many have any, and how many come
// before each class.
struct KeyWork {
  long long tiles;
  int some, pad;
  int before[kWorkClasses];
};

// The mask buffer (fa.h): row ranges, tile tables, the tiles of all sequences from the longest work down (as
// b * tiles + tile; those without work last), and the key tiles' work.  Each part on 16 bytes.  Row i of sequence b sees
// keys first[b * Nq + i] <= j < last[b * Nq + i] (both 0 for none).
struct MaskView {
  int *first, *last;
  QueryTile* qt;  // [B, Tq]
  KeyTile* kt;    // [B, Tk]
  int *q_order, *k_order;
  KeyWork* k_work;
  int B, Nq, Nk, Tq, Tk;
};

// Fills the view (base may be null: only the size is wanted); false for sizes that do not fit.
inline bool mask_view(void* base, int B, int Nq, int Nk, MaskView* v, size_t* bytes) {
  if (B < 0 || Nq < 0 || Nk < 0) return false;
  v->B = B, v->Nq = Nq, v->Nk = Nk;
  v->Tq = Nq / kRangeTile + (Nq % kRangeTile != 0), v->Tk = Nk / kRangeTile + (Nk % kRangeTile != 0);
  const long long rows = static_cast<long long>(B) * Nq, qts = static_cast<long long>(B) * v->Tq,
                  kts = static_cast<long long>(B) * v->Tk;
  if (rows > INT_MAX || static_cast<long long>(B) * Nk > INT_MAX || Nq > (1 << 30) || Nk > (1 << 30)) return false;
  size_t at = 0;
  auto part = [&](size_t n) {
    uint8_t* p = static_cast<uint8_t*>(base) + at;
    at += (n + 15) / 16 * 16;
    return base == nullptr ? nullptr : p;
  };
  v->first = reinterpret_cast<int*>(part(rows * 4));
  v->last = reinterpret_cast<int*>(part(rows * 4));
  v->qt = reinterpret_cast<QueryTile*>(part(qts * sizeof(QueryTile)));
  v->kt = reinterpret_cast<KeyTile*>(part(kts * sizeof(KeyTile)));
  v->q_order = reinterpret_cast<int*>(part(qts * 4));
  v->k_order = reinterpret_cast<int*>(part(kts * 4));
  v->k_work = reinterpret_cast<KeyWork*>(part(kts > 0 ? sizeof(KeyWork) : 0));
  *bytes = at;
  return true;
}

// A role's walk over its CTA's units, the longest first: (query or key tile of some sequence, head).  Unit u of the grid
// is (place u / heads of the order, head u % heads) within groups of `group` heads; CTA c takes units c, 2 G - 1 - c,
// 2 G + c, ... of G CTAs, so that neighbours in the order, which have about the same work, are spread evenly and each
// CTA's sum comes out alike without a queue (whose counter two launches might come to share).
// The next unit's tables are read one unit ahead.
struct UnitWalk {
  int k, entry, head;  // entry < 0: no more
  FA_DEV void look(const int* order, int tiles, int heads, int group) {
    const int g = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
    const int u = k * g + ((k & 1) ? g - 1 - c : c);
    entry = -1;
    if (u >= tiles * heads) return;  // (and so are all later ones)
    const int per = group * tiles, gi = u / per, r = u - gi * per, gs = min(heads - gi * group, group), place = r / gs;
    head = gi * group + r - place * gs;
    entry = order[place];
  }
};

// What a kernel does to the scores: bits of its MOD.
enum : int { kModNone = 0, kModCap = 1, kModBias = 2 };

// Bits of the halves of x that are infinite or NaN: bit 15 and bit 31.
FA_DEV uint32_t not_finite(uint32_t x) { return ((x & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }

// Caps that are taken: a score's error is the cap's times some 2^-22 (ranges_score.cuh).
constexpr float kCapMin = 1e-3f, kCapMax = 1e3f;

// What is done to the scaled scores s = scale q k: s = cap tanh(s / cap), then s -= slope |pos_i - j|.  In base 2.
struct ScoreMod {
  float c_log2;  // scale log2 e
  CapArgs cap;
  const float* slopes;  // [H] or null
};
inline ScoreMod score_mod(float scale, float cap, const float* slopes) {
  return ScoreMod{static_cast<float>(scale * 1.4426950408889634), cap_args(cap, scale), slopes};
}

struct RangesLaunch {
  const void *Q, *K, *V, *O, *dO;
  RowStrides sq, sk, sv, sdo;
  void *out, *dQ, *dK, *dV;
  float* L;
  const float* Lin;
  MaskView mask;
  int B, H, Hk, Nq, Nk, d;
  float scale;
  ScoreMod mod;
  uint8_t* workspace;
  cudaStream_t stream;
  int* status;
};
fa_status launch_fwd_ranges(const RangesLaunch& a);
fa_status launch_bwd_ranges(const RangesLaunch& a);
size_t bwd_ranges_workspace(int B, int H, int Hk, int Nq, int Nk, int d);

}  // namespace fa
