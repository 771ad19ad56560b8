// The ranges of keys that query rows see, from document borders, prefixes, a causal mask and a window, or from the
// caller's own, and the tables by which the attention over ranges walks its tiles.
//
// Row i of a sequence sits at position p = i + Nk - Nq.  With its document at positions [s, e):
//   first = s, last = e; causal: last = p + 1; window w: first = max(s, p + 1 - w);
//   prefix n: last = max(last, min(s + n, e)), as a row also sees all of its document's first n positions.
// Every mask of this kind is one range per row, so the attention needs two integers of a row, whatever made them.
//
// Three launches, one for few tiles: the rows with their tile's table, the key tiles (from the sequence's query tiles), and
// the tiles in the order of their work (a counting sort).  A mask is made once a step, for all layers and their gradients.
#include <cooperative_groups.h>

#include "ranges.cuh"

namespace fa {
namespace {

struct RowRules {
  const int *documents, *prefix;  // [B, docs + 1], [B, docs]; or both null: one document of Nk positions
  const int *first, *last;        // or the ranges themselves
  int docs, causal, window;
};

// The last of n ascending borders at or before p: how many are.
FA_DEV int borders_before(const int* d, int n, int p) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (d[mid] <= p) lo = mid + 1; else hi = mid;
  }
  return lo;
}
// The range of the row at position p of a sequence; d: its borders, pre: its prefixes (or null); c: its document.
FA_DEV int2 row_range(const RowRules& r, const MaskView& m, const int* d, const int* pre, int p, int c) {
  int first = 0, last = m.Nk, n = 0;
  if (d != nullptr) {
    if (c < 0 || c >= r.docs) return make_int2(0, 0);
    first = max(d[c], 0), last = min(d[c + 1], m.Nk);
    if (pre != nullptr) n = pre[c];
  } else if (pre != nullptr) {
    n = pre[0];
  }
  const int end = last;
  if (r.causal) last = min(last, p + 1);
  if (n > 0) last = max(last, static_cast<int>(min(static_cast<long long>(first) + n, static_cast<long long>(end))));
  if (r.window > 0) first = max(first, p + 1 - r.window);
  return first < last ? make_int2(first, last) : make_int2(0, 0);
}

// A query tile's ranges and its table (a warp, four neighbouring rows a lane); d, pre: the sequence's borders and prefixes.
FA_DEV void rows_of_tile(const MaskView& m, const RowRules& r, const int* d, const int* pre, int b, int tile, int lane) {
  const int i0 = tile * kRangeTile + 4 * lane;
  const size_t at = static_cast<size_t>(b) * m.Nq + i0;
  int lo = INT_MAX, hi = 0, full_first = 0, full_last = INT_MAX, first[4], last[4];
  const int p0 = i0 + m.Nk - m.Nq;
  int c = d != nullptr ? borders_before(d, r.docs + 1, p0) - 1 : 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    first[e] = last[e] = 0;
    if (i0 + e >= m.Nq) continue;
    int2 x;
    if (r.first != nullptr) {
      x = make_int2(max(r.first[at + e], 0), min(r.last[at + e], m.Nk));
      if (x.x >= x.y) x = make_int2(0, 0);
    } else {
      if (d != nullptr)
        while (c < r.docs && d[c + 1] <= p0 + e) ++c;
      x = row_range(r, m, d, pre, p0 + e, c);
    }
    first[e] = x.x, last[e] = x.y;
    if (x.y > 0) lo = min(lo, x.x), hi = max(hi, x.y), full_first = max(full_first, x.x), full_last = min(full_last, x.y);
    else full_first = kNoFull;
  }
  if (i0 + 3 < m.Nq && (at & 3) == 0) {
    *reinterpret_cast<int4*>(m.first + at) = make_int4(first[0], first[1], first[2], first[3]);
    *reinterpret_cast<int4*>(m.last + at) = make_int4(last[0], last[1], last[2], last[3]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i0 + e < m.Nq) m.first[at + e] = first[e], m.last[at + e] = last[e];
  }
  lo = __reduce_min_sync(0xffffffffu, lo), hi = __reduce_max_sync(0xffffffffu, hi);
  full_first = __reduce_max_sync(0xffffffffu, full_first), full_last = __reduce_min_sync(0xffffffffu, full_last);
  if (lane == 0) {
    QueryTile t{0, 0, full_first, full_last};
    if (hi > 0) t.lo = lo / kRangeTile, t.n = (hi - 1) / kRangeTile - t.lo + 1;
    m.qt[static_cast<size_t>(b) * m.Tq + tile] = t;
  }
}

// A sequence's borders and prefixes; null where there are none.
FA_DEV const int* borders_of(const RowRules& r, int b) {
  return r.documents == nullptr ? nullptr : r.documents + static_cast<size_t>(b) * (r.docs + 1);
}
FA_DEV const int* prefixes_of(const RowRules& r, int b) {
  return r.prefix == nullptr ? nullptr : r.prefix + static_cast<size_t>(b) * (r.documents == nullptr ? 1 : r.docs);
}

// A warp per query tile, four neighbouring rows a lane, one search for the first's document; the borders of the block's
// sequence in shared memory where they fit.  16 rows of 131072 in 64 documents each, with prefixes: 11.7 us (16.8 MB
// written); a thread per row with the borders in global memory took 19.5.
constexpr int kRowWarps = 8, kStaged = 1024;
__global__ void __launch_bounds__(32 * kRowWarps) mask_rows_kernel(const __grid_constant__ MaskView m,
                                                                   const __grid_constant__ RowRules r) {
  __shared__ int staged[2 * kStaged];
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.y, tile = blockIdx.x * kRowWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int *d = borders_of(r, b), *pre = prefixes_of(r, b);
  if (d != nullptr && r.docs < kStaged) {
    for (int i = threadIdx.x; i <= r.docs; i += 32 * kRowWarps) {
      staged[i] = d[i];
      if (pre != nullptr && i < r.docs) staged[kStaged + i] = pre[i];
    }
    __syncthreads();
    d = staged, pre = pre == nullptr ? nullptr : staged + kStaged;
  }
  if (tile < m.Tq) rows_of_tile(m, r, d, pre, b, tile, lane);
}

// Four threads per key tile, each with every fourth of the sequence's query tiles, 1024 of them at a time in shared
// memory.  The same masks: 7.5 us; a warp per key tile reading the tables from global memory took 11.8.
constexpr int kKeyChunk = 1024;
__global__ void __launch_bounds__(256) mask_keys_kernel(const __grid_constant__ MaskView m) {
  __shared__ int2 tiles[kKeyChunk];
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.y, k = blockIdx.x * 64 + (threadIdx.x >> 2), sub = threadIdx.x & 3;
  const QueryTile* qt = m.qt + static_cast<size_t>(b) * m.Tq;
  int lo = INT_MAX, hi = -1;
  for (int t0 = 0; t0 < m.Tq; t0 += kKeyChunk) {
    const int n = min(kKeyChunk, m.Tq - t0);
    if (t0 > 0) __syncthreads();
    for (int i = threadIdx.x; i < n; i += 256) tiles[i] = *reinterpret_cast<const int2*>(qt + t0 + i);
    __syncthreads();
#pragma unroll 8
    for (int i = sub; i < n; i += 4) {
      const int2 t = tiles[i];
      if (static_cast<unsigned>(k - t.x) < static_cast<unsigned>(t.y)) lo = min(lo, t0 + i), hi = t0 + i;
    }
  }
#pragma unroll
  for (int e = 1; e < 4; e <<= 1) {
    lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, e));
    hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, e));
  }
  if (sub == 0 && k < m.Tk) m.kt[static_cast<size_t>(b) * m.Tk + k] = hi < 0 ? KeyTile{0, 0} : KeyTile{lo, hi - lo + 1};
}

// Tiles by their work, the longest first: a histogram of the work in kBins classes (the last for tiles without any), its
// prefix sums, and every tile to the next place of its class.  A cluster of CTAS CTAs for query tiles and one for key
// tiles, each CTA with its share of the tiles and a histogram of its own, which the others read.  Lanes of one class
// count as one, as most tiles of a mask have the same work; four tiles a thread at a time, as the block's reads are waits.
// 16384 tiles of each kind: 10.4 us with clusters of 8, 29.5 with a CTA each.
constexpr int kBins = kWorkClasses, kPer = 4, kSortCtas = 8;
template <int CTAS>
__global__ void __cluster_dims__(CTAS, 1, 1) __launch_bounds__(1024)
    mask_order_kernel(const __grid_constant__ MaskView m) {
  __shared__ int bins[kBins];   // this CTA's histogram
  __shared__ int start[kBins];  // the next place of a class
  __shared__ int sums[32];
  __shared__ long long work_sums[32];
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  pdl_wait();
  const bool keys = blockIdx.x >= CTAS;
  const int rank = static_cast<int>(cluster.block_rank()), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int most = keys ? m.Tq : m.Tk, all = m.B * (keys ? m.Tk : m.Tq);  // (at most 2^31 / 128 and more)
  const int share = (all + CTAS - 1) / CTAS, from = min(rank * share, all), to = min(from + share, all);
  int* order = keys ? m.k_order : m.q_order;
  const bool exact = most < kBins - 1;
  // the largest work of a class
  auto work_of = [&](int x) {
    if (x == kBins - 1) return 0;
    if (exact) return max(most - x, 0);
    return most - static_cast<int>((static_cast<long long>(x) * most + kBins - 3) / (kBins - 2));
  };
  for (int i = tid; i < kBins; i += 1024) bins[i] = 0;
  __syncthreads();
  auto pass = [&](bool place) {
    int* count = place ? start : bins;
#pragma unroll 1
    for (int t0 = from; t0 < to; t0 += kPer * 1024) {
      int x[kPer];
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const int t = t0 + e * 1024 + tid;
        x[e] = t < to ? (keys ? m.kt[t].n : m.qt[t].n) : -1;
      }
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const int t = t0 + e * 1024 + tid, bin = x[e] < 0 ? -1 : work_class(x[e], most);
        if (t0 + e * 1024 >= to) break;
        const unsigned same = __match_any_sync(0xffffffffu, bin);
        const int leader = __ffs(same) - 1;
        int at = 0;
        if (lane == leader && bin >= 0) at = atomicAdd(&count[bin], __popc(same));
        at = __shfl_sync(0xffffffffu, at, leader) + __popc(same & ((1u << lane) - 1u));
        if (place && bin >= 0) order[at] = t;
      }
    }
  };
  pass(false);
  cluster.sync();
  // classes 2 tid and 2 tid + 1: their tiles in the CTAs before this one, and in all
  int2 mine = make_int2(0, 0), total = make_int2(0, 0);
#pragma unroll
  for (int c = 0; c < CTAS; ++c) {
    const int2 x = reinterpret_cast<const int2*>(cluster.map_shared_rank(bins, c))[tid];
    if (c < rank) mine.x += x.x, mine.y += x.y;
    total.x += x.x, total.y += x.y;
  }
  int up = total.x + total.y;
  long long work = static_cast<long long>(total.x) * work_of(2 * tid) + static_cast<long long>(total.y) * work_of(2 * tid + 1);
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, up, k);
    const long long z = __shfl_up_sync(0xffffffffu, work, k);
    if (lane >= k) up += y, work += z;
  }
  if (lane == 31) sums[warp] = up, work_sums[warp] = work;
  __syncthreads();
  for (int w = 0; w < warp; ++w) up += sums[w], work += work_sums[w];
  const int before0 = up - total.x - total.y, before1 = up - total.y;  // the tiles before the two classes
  start[2 * tid] = before0 + mine.x, start[2 * tid + 1] = before1 + mine.y;
  if (keys && rank == 0 && all > 0) {
    reinterpret_cast<int2*>(m.k_work->before)[tid] = make_int2(before0, before1);
    if (tid == 1023) m.k_work->tiles = work, m.k_work->some = before1;
  }
  __syncthreads();
  pass(true);
  cluster.sync();  // no CTA ends while another reads its histogram
}

// All of it in one launch and one CTA, for few tiles: a tile's place in the order is how many have more work (or as much,
// and come before it).  4 rows of 1024 tokens: 9.9 us a call, host included (5.5 on the device); in three launches 16.5
// (7.1).  With 64 tiles the device takes 8.3, with 128 13.1 against 7.4.
constexpr int kFewTiles = 64;
__global__ void __launch_bounds__(1024) mask_few_kernel(const __grid_constant__ MaskView m,
                                                        const __grid_constant__ RowRules r) {
  __shared__ int2 tiles[kFewTiles];  // first tile and tiles, of query tiles
  __shared__ int work[2][kFewTiles], sorted[kFewTiles];
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nq = m.B * m.Tq, nk = m.B * m.Tk;
  for (int t = warp; t < nq; t += 32) {
    const int b = t / m.Tq;
    rows_of_tile(m, r, borders_of(r, b), prefixes_of(r, b), b, t - b * m.Tq, lane);
  }
  __syncthreads();
  for (int t = threadIdx.x; t < nq; t += 1024) tiles[t] = *reinterpret_cast<const int2*>(m.qt + t), work[0][t] = tiles[t].y;
  __syncthreads();
  for (int t = threadIdx.x; t < nk; t += 1024) {
    const int b = t / m.Tk, k = t - b * m.Tk;
    int lo = INT_MAX, hi = -1;
    for (int i = 0; i < m.Tq; ++i) {
      const int2 q = tiles[b * m.Tq + i];
      if (static_cast<unsigned>(k - q.x) < static_cast<unsigned>(q.y)) lo = min(lo, i), hi = i;
    }
    work[1][t] = hi < 0 ? 0 : hi - lo + 1;
    m.kt[t] = KeyTile{hi < 0 ? 0 : lo, work[1][t]};
  }
  __syncthreads();
  const int half = threadIdx.x >> 9, count = half ? nk : nq;
  for (int t = threadIdx.x & 511; t < count; t += 512) {
    const int mine = work[half][t];
    int place = 0;
    for (int i = 0; i < count; ++i) place += work[half][i] > mine || (work[half][i] == mine && i < t);
    (half ? m.k_order : m.q_order)[place] = t;
    if (half) sorted[place] = mine;
  }
  __syncthreads();
  if (nk > 0) {
    for (int c = threadIdx.x; c < kWorkClasses; c += 1024) {
      int lo = 0, hi = nk;  // the first of a class at or behind c
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (work_class(sorted[mid], m.Tq) < c) lo = mid + 1; else hi = mid;
      }
      m.k_work->before[c] = lo;
    }
    if (warp == 0) {
      int all = 0, some = 0;
      for (int i = lane; i < nk; i += 32) all += work[1][i], some += work[1][i] > 0;
      all = __reduce_add_sync(0xffffffffu, all), some = __reduce_add_sync(0xffffffffu, some);
      if (lane == 0) m.k_work->tiles = all, m.k_work->some = some;
    }
  }
}

constexpr int kMostDocs = 1 << 29;  // sums of two places among the borders fit 32 bits

fa_status launch_mask(const MaskView& m, const RowRules& r, cudaStream_t s) {
  if (m.B == 0 || (m.Tq == 0 && m.Tk == 0)) return FA_OK;
  if (static_cast<long long>(m.B) * m.Tq <= kFewTiles && static_cast<long long>(m.B) * m.Tk <= kFewTiles)
    return launch_pdl(mask_few_kernel, dim3(1), dim3(1024), 0, s, m, r) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
  if (m.Tq > 0 && launch_pdl(mask_rows_kernel, dim3((m.Tq + kRowWarps - 1) / kRowWarps, m.B), dim3(32 * kRowWarps), 0, s,
                             m, r) != cudaSuccess)
    return FA_ERR_CUDA;
  if (m.Tk > 0 && launch_pdl(mask_keys_kernel, dim3((m.Tk + 63) / 64, m.B), dim3(256), 0, s, m) != cudaSuccess)
    return FA_ERR_CUDA;
  // (up to kPer tiles a thread one CTA is faster: 32 tiles take 6.1 us in all, with clusters 8.9)
  const long long most = static_cast<long long>(m.B) * (m.Tq > m.Tk ? m.Tq : m.Tk);
  const cudaError_t e = most <= kPer * 1024 ? launch_pdl(mask_order_kernel<1>, dim3(2), dim3(1024), 0, s, m)
                                            : launch_pdl(mask_order_kernel<kSortCtas>, dim3(2 * kSortCtas), dim3(1024), 0, s, m);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status mask_args(void* mask, size_t mask_bytes, int B, int Nq, int Nk, MaskView* m) {
  size_t need = 0;
  if (!mask_view(mask, B, Nq, Nk, m, &need)) return B < 0 || Nq < 0 || Nk < 0 ? FA_ERR_INVALID_ARG : FA_ERR_UNSUPPORTED;
  if (B > 65535) return FA_ERR_UNSUPPORTED;
  if (need > 0 && (mask == nullptr || mask_bytes < need || !aligned(mask, 16))) return FA_ERR_WORKSPACE;
  return FA_OK;
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_mask_size(int B, int Nq, int Nk) {
  MaskView m;
  size_t bytes = 0;
  return B <= 65535 && mask_view(nullptr, B, Nq, Nk, &m, &bytes) ? bytes : static_cast<size_t>(-1);
}

fa_status fa_mask_ranges(void* mask, size_t mask_bytes, int B, int Nq, int Nk, int causal, int window,
                         const int* documents, int docs, const int* prefix, fa_stream_t stream) {
  if (documents == nullptr) docs = 0;
  if (window < 0 || docs < 0 || (window > 0 && !causal) || (prefix != nullptr && (!causal || window > 0)) ||
      (documents != nullptr && docs == 0) || !aligned(documents, 4) || !aligned(prefix, 4))
    return FA_ERR_INVALID_ARG;
  MaskView m;
  const fa_status st = mask_args(mask, mask_bytes, B, Nq, Nk, &m);
  if (st != FA_OK) return st;
  if (Nq > Nk || docs > kMostDocs) return FA_ERR_UNSUPPORTED;
  return launch_mask(m, RowRules{documents, prefix, nullptr, nullptr, docs, causal != 0, window}, stream);
}

fa_status fa_mask_from_ranges(void* mask, size_t mask_bytes, int B, int Nq, int Nk, const int* first, const int* last,
                              fa_stream_t stream) {
  MaskView m;
  const fa_status st = mask_args(mask, mask_bytes, B, Nq, Nk, &m);
  if (st != FA_OK) return st;
  if (static_cast<long long>(B) * Nq > 0 && (!first || !last || !aligned(first, 4) || !aligned(last, 4)))
    return FA_ERR_INVALID_ARG;
  return launch_mask(m, RowRules{nullptr, nullptr, first, last, 0, 0, 0}, stream);
}

}  // extern "C"
