// Norm of queries and keys for each head and rotation by position, forward and
// gradients: what a model runs between its projections and the attention.
//
// For every (batch, head, row) vector x of d elements, with weight w and the
// position's angles:
//   r = 1 / sqrt(mean(x^2) + eps),  y = x r w,  z = R y                       (forward)
//   dy = R^T dz,  g = dy w,  dx = r (g - x r^2 mean(g x)),  dw = sum of dy x r (gradients)
// R turns pairs of the first `rope` elements: elements i and i + rope/2, or 2i and
// 2i + 1.  The gradients recompute r from x, which they read anyway, so the forward
// saves nothing.  All arithmetic is in fp32, rounded to bf16 once at the store.
//
// Both are bound by memory: the forward moves 4 d bytes per row, the gradients 6 d.
// d/8 lanes hold one row, 16 bytes each; a lane group takes kHeads heads of one
// (batch, row) at a time, so that it reads that position's cos and sin once for all of
// them and has kHeads independent loads in flight.  A block works on one of the two
// tensors (blocks below grid_q on q, the others on k), so that the weight gradients
// are 8 running sums per lane; they are joined in the block, written to the workspace
// and summed over the blocks in a fixed order by a second small kernel.
#include <cmath>

#include "internal.h"
#include "ptx.cuh"

namespace fa {

namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 4;  // heads per lane group and step
// Blocks resident on an SM: the grid is that many blocks (shared out between q and k by
// their work), each of which runs to the end.  Measured at 1 x 32 x 8192 x 128, q and k
// (heads per step, blocks): forward 49.8 us at (4, 4), 58.8 at (2, 4), 74 at (8, 2);
// gradients 76.7 us at (4, 3), 85.7 at (2, 3), 108 at (4, 2); loading the next step's rows
// ahead 52.7 and 83 at best; twice the blocks 50.1 and 80.1.
template <bool GRAD>
constexpr int kBlocks = GRAD ? 3 : 4;

struct NormTensor {
  const __nv_bfloat16* x;
  const __nv_bfloat16* dz;  // gradients only
  __nv_bfloat16* out;       // z, or dx
  const void* w;            // fp32 or bf16 [d], or null
  float* dw_part;           // gradients: [blocks][d] partial sums, or null
  RowStrides sx, sdz, so;
  int H;
  unsigned items;           // B * N * ceil(H / kHeads)
};

struct NormArgs {
  NormTensor t[2];
  const float *cos, *sin;   // [rows][rope / 2], or null
  const int* pos;           // [B, N], or null (row n is at position n)
  int N, rope, table_rows, interleaved, w_bf16, grid_q;
  float eps;
};

FA_DEV uint4 ld_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
FA_DEV void unpack8(uint4 v, float* f) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
FA_DEV uint4 pack8(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}
FA_DEV void load_weight(const void* w, int bf16, int at, float* f) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 1.f;
  } else if (bf16) {
    unpack8(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(w) + at), f);
  } else {
    const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(w) + at);
    const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(w) + at + 4);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
}
template <int LPR>
FA_DEV float row_sum(float v) {
#pragma unroll
  for (int m = LPR / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// Where r = 1 / sqrt(mean(x^2) + eps) lies outside [2^-60, 2^50], a square or their sum may have passed fp32's range.
// A warp that meets such a row computes it again after its loop, times a power of two (`root_of`, `far_rows`).  The loop
// pays one subtraction and one maximum a row, on r's bits: at 1 x 32 x 8192 x 128 forward 49.5 to 49.6 us, gradients
// 75.9 to 76.5; with a branch per row 56.6 and 83.4, with two comparisons 50.6 and 78.8.
constexpr unsigned kRootMin = 0x21800000u, kRootSpan = 0x58800000u - kRootMin;
FA_DEV unsigned root_offset(float r) { return static_cast<unsigned>(__float_as_int(r)) - kRootMin; }
// Scales a row's elements (8 in a lane) by s = 2^-k, for the larger k of its largest element and of sqrt(eps), and
// returns 1 / sqrt(mean((x s)^2) + eps s^2).  A row of zeros, or with an infinity, is not scaled.
template <int D>
FA_DEV float root_of(float (&f)[8], float eps, float* s) {
  constexpr int LPR = D / 8;
  float m = 0.f, sq = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(f[e]));
#pragma unroll
  for (int i = LPR / 2; i > 0; i >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, i));
  const int kx = (__float_as_int(m) >> 23) - 127, ke = eps > 0.f ? ((__float_as_int(eps) >> 23) - 127) >> 1 : -127;
  *s = m == 0.f || kx == 128 ? 1.f : __int_as_float((127 - min(max(max(kx, ke), -126), 126)) << 23);
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] *= *s, sq = fmaf(f[e], f[e], sq);
  return rsqrtf(row_sum<LPR>(sq) * (1.f / D) + eps * *s * *s);
}

// The angles of one lane's 8 elements: out = c * own + s * other, where `other` is the
// element each is paired with and s carries the sign of the forward rotation.
// Elements behind `rope` get c = 1, s = 0.
struct Angles {
  float c[8], s[8];
};
FA_DEV void load_angles(Angles& a, const NormArgs& p, int position, int col) {
#pragma unroll
  for (int i = 0; i < 8; ++i) a.c[i] = 1.f, a.s[i] = 0.f;
  if (col >= p.rope) return;
  if (position >= p.table_rows) {  // no such angle: the row's rotated part becomes NaN
#pragma unroll
    for (int i = 0; i < 8; ++i) a.c[i] = a.s[i] = __int_as_float(0x7fffffff);
    return;
  }
  const int half = p.rope / 2;
  const float* ct = p.cos + static_cast<size_t>(position) * half;
  const float* st = p.sin + static_cast<size_t>(position) * half;
  if (p.interleaved) {
    const float4 c = *reinterpret_cast<const float4*>(ct + col / 2);
    const float4 s = *reinterpret_cast<const float4*>(st + col / 2);
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a.c[2 * i] = a.c[2 * i + 1] = cc[i];
      a.s[2 * i] = -ss[i];
      a.s[2 * i + 1] = ss[i];
    }
  } else {
    const int at = col < half ? col : col - half;
    const float sign = col < half ? -1.f : 1.f;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const float4 c = *reinterpret_cast<const float4*>(ct + at + 4 * q);
      const float4 s = *reinterpret_cast<const float4*>(st + at + 4 * q);
      a.c[4 * q] = c.x, a.c[4 * q + 1] = c.y, a.c[4 * q + 2] = c.z, a.c[4 * q + 3] = c.w;
      a.s[4 * q] = sign * s.x, a.s[4 * q + 1] = sign * s.y, a.s[4 * q + 2] = sign * s.z, a.s[4 * q + 3] = sign * s.w;
    }
  }
}

// The rows out of range among those of one warp again, in range, and with GRAD the sums of all its rows for the weight
// gradients of its columns.  Not inlined: what it needs is found again, so that the loop keeps its registers.
struct Columns {
  float v[8];
};
template <int D, bool GRAD>
__noinline__ __device__ Columns far_rows(const NormArgs& p) {
  constexpr int LPR = D / 8, GPW = 32 / LPR;  // lane groups per warp
  const bool is_k = blockIdx.x >= static_cast<unsigned>(p.grid_q);
  const NormTensor& t = p.t[is_k ? 1 : 0];
  const unsigned block = is_k ? blockIdx.x - p.grid_q : blockIdx.x;
  const unsigned nblocks = is_k ? gridDim.x - p.grid_q : p.grid_q;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = lane % LPR, col = part * 8;
  const unsigned group = (block * (kThreads / 32) + warp) * GPW + lane / LPR;
  const unsigned ngroups = nblocks * (kThreads / 32) * GPW;
  const unsigned hblocks = (t.H + kHeads - 1) / kHeads;
  const unsigned trips = (t.items + ngroups - 1) / ngroups;
  const int hchunks = p.rope / 16;
  const int other_part = p.interleaved || part >= 2 * hchunks ? part : part < hchunks ? part + hchunks : part - hchunks;
  const int other_lane = lane - part + other_part;
  float w[8], dw[8] = {};
  load_weight(t.w, p.w_bf16, col, w);
#pragma unroll 1
  for (unsigned trip = 0; trip < trips; ++trip) {
    const unsigned item = group + trip * ngroups;
    const bool live = item < t.items;
    const unsigned bn = live ? item / hblocks : 0, hb = live ? item - bn * hblocks : 0;
    const unsigned b = bn / p.N, n = bn - b * p.N;
    const int position = p.pos != nullptr && live ? p.pos[bn] : static_cast<int>(n);
    Angles a;
    load_angles(a, p, live ? position : 0, position < 0 ? D : col);
#pragma unroll 1
    for (int h = hb * kHeads; h < static_cast<int>(hb * kHeads) + kHeads; ++h) {
      const bool there = live && h < t.H;
      float f[8], u[8], o[8], s, sq = 0.f;
      unpack8(there ? ld_stream(t.x + b * t.sx.b + n * t.sx.n + h * t.sx.h + col) : make_uint4(0, 0, 0, 0), f);
#pragma unroll
      for (int e = 0; e < 8; ++e) sq = fmaf(f[e], f[e], sq);
      const bool mine = root_offset(rsqrtf(row_sum<LPR>(sq) * (1.f / D) + p.eps)) > kRootSpan && there;
      if (!GRAD && !__any_sync(0xffffffffu, mine)) continue;
      const float r = root_of<D>(f, p.eps, &s);
      if constexpr (GRAD) {
        unpack8(there ? ld_stream(t.dz + b * t.sdz.b + n * t.sdz.n + h * t.sdz.h + col) : make_uint4(0, 0, 0, 0), u);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = f[e] * w[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float across = __shfl_sync(0xffffffffu, u[e], other_lane);
        o[e] = p.interleaved ? u[e ^ 1] : across;
      }
      float res[8], dot = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if constexpr (!GRAD) {
          res[e] = r * fmaf(u[e], a.c[e], o[e] * a.s[e]);
        } else {
          const float dy = fmaf(u[e], a.c[e], -o[e] * a.s[e]);
          f[e] *= r;
          if (there && position >= 0) dw[e] = fmaf(dy, f[e], dw[e]);
          res[e] = dy * w[e];
          dot = fmaf(res[e], f[e], dot);
        }
      }
      if constexpr (GRAD) {
        const float along = row_sum<LPR>(dot) * (1.f / D);
#pragma unroll
        for (int e = 0; e < 8; ++e) res[e] = r * (res[e] - f[e] * along) * s;
      }
      if (position < 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) res[e] = 0.f;
      }
      if (mine) *reinterpret_cast<uint4*>(t.out + b * t.so.b + n * t.so.n + h * t.so.h + col) = pack8(res);
    }
  }
  Columns sums;
#pragma unroll
  for (int e = 0; e < 8; ++e) sums.v[e] = dw[e];
  return sums;
}

// GRAD: gradients.  LPR = D / 8 lanes per row.
template <int D, bool GRAD>
__global__ void __launch_bounds__(kThreads, kBlocks<GRAD>) norm_rope_kernel(const __grid_constant__ NormArgs p) {
  constexpr int LPR = D / 8, GPW = 32 / LPR;  // lane groups per warp
  const bool is_k = blockIdx.x >= static_cast<unsigned>(p.grid_q);
  const NormTensor& t = p.t[is_k ? 1 : 0];
  const unsigned block = is_k ? blockIdx.x - p.grid_q : blockIdx.x;
  const unsigned nblocks = is_k ? gridDim.x - p.grid_q : p.grid_q;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = lane % LPR, col = part * 8;
  const unsigned group = (block * (kThreads / 32) + warp) * GPW + lane / LPR;
  const unsigned ngroups = nblocks * (kThreads / 32) * GPW;
  const unsigned hblocks = (t.H + kHeads - 1) / kHeads;

  pdl_wait();
  float w[8], wo[8];  // weights of this lane's elements and of the ones they pair with
  load_weight(t.w, p.w_bf16, col, w);
  // half-split pairs: the lane of the same row that holds the other half's elements
  const int hchunks = p.rope / 16;
  const int other_part = p.interleaved || part >= 2 * hchunks ? part : part < hchunks ? part + hchunks : part - hchunks;
  const int other_lane = lane - part + other_part;
  load_weight(t.w, p.w_bf16, other_part * 8, wo);

  float dw[8] = {};
  unsigned far = 0;  // above kRootSpan: a row out of range
  // every lane of a warp makes the same number of trips (shuffles below)
  const unsigned trips = (t.items + ngroups - 1) / ngroups;
  for (unsigned trip = 0; trip < trips; ++trip) {
    const unsigned item = group + trip * ngroups;
    const bool live = item < t.items;
    const unsigned bn = live ? item / hblocks : 0, hb = live ? item - bn * hblocks : 0;
    const unsigned b = bn / p.N, n = bn - b * p.N;
    const int h0 = hb * kHeads;
    const int nh = live ? min(kHeads, t.H - h0) : 0;
    const __nv_bfloat16* x = t.x + b * t.sx.b + n * t.sx.n + h0 * t.sx.h + col;
    uint4 xv[kHeads], gv[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
      xv[i] = i < nh ? ld_stream(x + i * t.sx.h) : make_uint4(0, 0, 0, 0);
    if constexpr (GRAD) {
      const __nv_bfloat16* dz = t.dz + b * t.sdz.b + n * t.sdz.n + h0 * t.sdz.h + col;
#pragma unroll
      for (int i = 0; i < kHeads; ++i)
        gv[i] = i < nh ? ld_stream(dz + i * t.sdz.h) : make_uint4(0, 0, 0, 0);
    }
    const int position = p.pos != nullptr && live ? p.pos[bn] : static_cast<int>(n);
    Angles a;
    load_angles(a, p, live ? position : 0, position < 0 ? D : col);
    if constexpr (!GRAD) {  // the weights are the same for all heads of the step
#pragma unroll
      for (int e = 0; e < 8; ++e) a.c[e] *= w[e], a.s[e] *= p.interleaved ? w[e ^ 1] : wo[e];
    }
    __nv_bfloat16* out = t.out + b * t.so.b + n * t.so.n + h0 * t.so.h + col;
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      float f[8], o[8];
      unpack8(xv[i], f);
      float sq = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sq = fmaf(f[e], f[e], sq);
      const float r = rsqrtf(row_sum<LPR>(sq) * (1.f / D) + p.eps);
      far = max(far, root_offset(r));
      const uint4 src = GRAD ? gv[i] : xv[i];
      uint4 ov;
      ov.x = __shfl_sync(0xffffffffu, src.x, other_lane);
      ov.y = __shfl_sync(0xffffffffu, src.y, other_lane);
      ov.z = __shfl_sync(0xffffffffu, src.z, other_lane);
      ov.w = __shfl_sync(0xffffffffu, src.w, other_lane);
      float u[8], res[8];
      unpack8(src, u);
      unpack8(ov, o);
      if constexpr (!GRAD) {
        if (p.interleaved) {
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = u[e ^ 1];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) res[e] = r * fmaf(u[e], a.c[e], o[e] * a.s[e]);
      } else {
        if (p.interleaved) {
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = u[e ^ 1];
        }
        float g[8], dot = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float dy = fmaf(u[e], a.c[e], -o[e] * a.s[e]);  // the inverse rotation
          const float xh = f[e] * r;
          if (i < nh && position >= 0) dw[e] = fmaf(dy, xh, dw[e]);
          g[e] = dy * w[e];
          dot = fmaf(g[e], xh, dot);
          f[e] = xh;
        }
        const float mean = row_sum<LPR>(dot) * (1.f / D);
#pragma unroll
        for (int e = 0; e < 8; ++e) res[e] = r * (g[e] - f[e] * mean);
      }
      if (position < 0) {  // a padding row
#pragma unroll
        for (int e = 0; e < 8; ++e) res[e] = 0.f;
      }
      if (i < nh) *reinterpret_cast<uint4*>(out + i * t.so.h) = pack8(res);
    }
  }
  if (__any_sync(0xffffffffu, far > kRootSpan)) {
    const Columns all = far_rows<D, GRAD>(p);
    if constexpr (GRAD) {
#pragma unroll
      for (int e = 0; e < 8; ++e) dw[e] = all.v[e];
    }
  }
  if constexpr (GRAD) {
    if (t.dw_part == nullptr) return;
    // lanes of the same part hold sums of the same columns
    __shared__ float red[kThreads / 32][D];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
      for (int m = LPR; m < 32; m <<= 1) dw[e] += __shfl_xor_sync(0xffffffffu, dw[e], m);
      if (lane < LPR) red[warp][col + e] = dw[e];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += kThreads) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < kThreads / 32; ++k) s += red[k][c];
      t.dw_part[static_cast<size_t>(block) * D + c] = s;
    }
  }
}

// dw[c] = sum over the blocks' partial sums, in block order within each of 8 strands
// and then strand by strand: the same order on every run.
struct DwArgs {
  const float* part[2];
  void* dw[2];
  int blocks[2], w_bf16;
};
template <int D>
__global__ void __launch_bounds__(256) dw_sum_kernel(const __grid_constant__ DwArgs p) {
  __shared__ float red[8][32];
  const int which = blockIdx.y, c = blockIdx.x * 32 + (threadIdx.x & 31), strand = threadIdx.x >> 5;
  if (p.dw[which] == nullptr) return;
  pdl_wait();
  float s = 0.f;
  for (int b = strand; b < p.blocks[which]; b += 8) s += p.part[which][static_cast<size_t>(b) * D + c];
  red[strand][threadIdx.x & 31] = s;
  __syncthreads();
  if (strand == 0) {
#pragma unroll
    for (int k = 1; k < 8; ++k) s += red[k][threadIdx.x];
    if (p.w_bf16)
      static_cast<__nv_bfloat16*>(p.dw[which])[c] = __float2bfloat16_rn(s);
    else
      static_cast<float*>(p.dw[which])[c] = s;
  }
}

long long item_count(int B, int H, int N) {
  return static_cast<long long>(B) * N * ((H + kHeads - 1) / kHeads);
}
// Blocks for q (blocks[0]) and k: what the items need, or all that are resident, shared
// out by items.
template <bool GRAD>
void grid_for(int B, int Hq, int Hk, int N, int d, int blocks[2]) {
  const long long per_block = (kThreads / 32) * (32 / (d / 8)), most = 152 * kBlocks<GRAD>;
  const long long iq = item_count(B, Hq, N), ik = item_count(B, Hk, N);
  long long nq = (iq + per_block - 1) / per_block, nk = (ik + per_block - 1) / per_block;
  if (nq + nk > most) {
    const long long all = nq + nk, wq = nq;
    nq = nq * most / all;
    if (nq == 0 && wq > 0) nq = 1;
    if (nq == most && nk > 0) nq = most - 1;
    nk = nk > 0 ? most - nq : 0;
  }
  blocks[0] = static_cast<int>(nq), blocks[1] = static_cast<int>(nk);
}

// Checks shared by both directions; *empty: nothing to do.
fa_status check_norm(int B, int Hq, int Hk, int N, int d, float eps, const float* cos, const float* sin, int rope,
                     int table_rows, const int* positions, bool* empty) {
  if (B < 0 || Hq < 0 || Hk < 0 || N < 0 || rope < 0 || table_rows < 0) return FA_ERR_INVALID_ARG;
  if (d != 32 && d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (!(std::isfinite(eps) && eps >= 0.f)) return FA_ERR_INVALID_ARG;
  if ((cos == nullptr) != (sin == nullptr)) return FA_ERR_INVALID_ARG;
  if (cos == nullptr && (rope != 0 || positions != nullptr)) return FA_ERR_INVALID_ARG;
  if (cos != nullptr && (rope < 16 || rope > d || rope % 16 != 0)) return FA_ERR_UNSUPPORTED;
  if (!aligned(cos, 16) || !aligned(sin, 16) || !aligned(positions, 4)) return FA_ERR_INVALID_ARG;
  if (cos != nullptr && positions == nullptr && N > table_rows) return FA_ERR_INVALID_ARG;
  if (N > (1 << 30) || static_cast<long long>(B) * Hq > 65535 || static_cast<long long>(B) * Hk > 65535)
    return FA_ERR_UNSUPPORTED;
  *empty = B == 0 || N == 0 || (Hq == 0 && Hk == 0);
  if (item_count(B, Hq, N) > 0x7fffffffLL || item_count(B, Hk, N) > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

template <bool GRAD>
cudaError_t launch_norm(const NormArgs& p, int grid, int d, cudaStream_t s) {
  const dim3 g(grid), t(kThreads);
  switch (d) {
    case 32: return launch_pdl(norm_rope_kernel<32, GRAD>, g, t, 0, s, p);
    case 64: return launch_pdl(norm_rope_kernel<64, GRAD>, g, t, 0, s, p);
    default: return launch_pdl(norm_rope_kernel<128, GRAD>, g, t, 0, s, p);
  }
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

fa_status fa_qk_norm_rope(const void* Q, const void* K, void* Qout, void* Kout, const long long* q_strides,
                          const long long* k_strides, const void* q_weight, const void* k_weight, int weight_bf16,
                          const float* cos, const float* sin, int rope, int table_rows, int interleaved,
                          const int* positions, int B, int Hq, int Hk, int N, int d, float eps, fa_stream_t stream) {
  bool empty = false;
  const fa_status st = check_norm(B, Hq, Hk, N, d, eps, cos, sin, rope, table_rows, positions, &empty);
  if (st != FA_OK) return st;
  NormArgs p{};
  if (!read_strides(q_strides, B, Hq, N, d, &p.t[0].sx) || !read_strides(k_strides, B, Hk, N, d, &p.t[1].sx))
    return FA_ERR_INVALID_ARG;
  if (empty) return FA_OK;
  if ((Hq > 0 && (!Q || !Qout)) || (Hk > 0 && (!K || !Kout))) return FA_ERR_INVALID_ARG;
  for (const void* ptr : {Q, K, static_cast<const void*>(Qout), static_cast<const void*>(Kout), q_weight, k_weight})
    if (!aligned(ptr, 16)) return FA_ERR_INVALID_ARG;
  const void* x[2] = {Q, K};
  void* out[2] = {Qout, Kout};
  const void* w[2] = {q_weight, k_weight};
  const int H[2] = {Hq, Hk};
  int blocks[2];
  for (int i = 0; i < 2; ++i) {
    NormTensor& t = p.t[i];
    t.x = static_cast<const __nv_bfloat16*>(x[i]);
    t.out = static_cast<__nv_bfloat16*>(out[i]);
    t.w = w[i];
    read_strides(nullptr, B, H[i], N, d, &t.so);
    t.H = H[i];
    t.items = static_cast<unsigned>(item_count(B, H[i], N));
  }
  grid_for<false>(B, Hq, Hk, N, d, blocks);
  p.cos = cos, p.sin = sin, p.pos = positions;
  p.N = N, p.rope = rope, p.table_rows = table_rows, p.interleaved = interleaved ? 1 : 0;
  p.w_bf16 = weight_bf16 ? 1 : 0, p.grid_q = blocks[0], p.eps = eps;
  return launch_norm<false>(p, blocks[0] + blocks[1], d, stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_qk_norm_rope_bwd_workspace_size(int B, int Hq, int Hk, int N, int d) {
  if (B < 0 || Hq < 0 || Hk < 0 || N < 0 || (d != 32 && d != 64 && d != 128)) return static_cast<size_t>(-1);
  int blocks[2];
  grid_for<true>(B, Hq, Hk, N, d, blocks);
  return (static_cast<size_t>(blocks[0]) + blocks[1]) * d * sizeof(float);
}

fa_status fa_qk_norm_rope_bwd(const void* Q, const void* K, const void* dQout, const void* dKout, void* dQ, void* dK,
                              const long long* q_strides, const long long* k_strides, const long long* dqout_strides,
                              const long long* dkout_strides, const long long* dq_strides,
                              const long long* dk_strides, const void* q_weight, const void* k_weight,
                              void* dq_weight, void* dk_weight, int weight_bf16, const float* cos, const float* sin,
                              int rope, int table_rows, int interleaved, const int* positions, int B, int Hq, int Hk,
                              int N, int d, float eps, void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  bool empty = false;
  const fa_status st = check_norm(B, Hq, Hk, N, d, eps, cos, sin, rope, table_rows, positions, &empty);
  if (st != FA_OK) return st;
  NormArgs p{};
  if (!read_strides(q_strides, B, Hq, N, d, &p.t[0].sx) || !read_strides(k_strides, B, Hk, N, d, &p.t[1].sx) ||
      !read_strides(dqout_strides, B, Hq, N, d, &p.t[0].sdz) || !read_strides(dkout_strides, B, Hk, N, d, &p.t[1].sdz) ||
      !read_strides(dq_strides, B, Hq, N, d, &p.t[0].so) || !read_strides(dk_strides, B, Hk, N, d, &p.t[1].so))
    return FA_ERR_INVALID_ARG;
  for (const void* ptr : {Q, K, dQout, dKout, static_cast<const void*>(dQ), static_cast<const void*>(dK), q_weight,
                          k_weight})
    if (!aligned(ptr, 16)) return FA_ERR_INVALID_ARG;
  if (!aligned(dq_weight, 4) || !aligned(dk_weight, 4)) return FA_ERR_INVALID_ARG;
  const int H[2] = {Hq, Hk};
  void* dw[2] = {dq_weight, dk_weight};
  for (int i = 0; i < 2; ++i) {  // rows of an output must not share memory
    const RowStrides& so = p.t[i].so;
    if (!empty && H[i] > 0 && ((B > 1 && so.b < d) || (H[i] > 1 && so.h < d) || (N > 1 && so.n < d)))
      return FA_ERR_INVALID_ARG;
  }
  if (!empty && ((Hq > 0 && (!Q || !dQout || !dQ)) || (Hk > 0 && (!K || !dKout || !dK)))) return FA_ERR_INVALID_ARG;
  const bool any_dw = dw[0] != nullptr || dw[1] != nullptr;
  const size_t need = empty ? 0 : fa_qk_norm_rope_bwd_workspace_size(B, Hq, Hk, N, d);
  if (any_dw && need > 0 && (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 16)))
    return FA_ERR_WORKSPACE;
  DwArgs r{};
  r.w_bf16 = weight_bf16 ? 1 : 0;
  if (!empty) {
    const void* x[2] = {Q, K};
    const void* dz[2] = {dQout, dKout};
    void* dx[2] = {dQ, dK};
    const void* w[2] = {q_weight, k_weight};
    float* part = static_cast<float*>(workspace);
    grid_for<true>(B, Hq, Hk, N, d, r.blocks);
    for (int i = 0; i < 2; ++i) {
      NormTensor& t = p.t[i];
      t.x = static_cast<const __nv_bfloat16*>(x[i]);
      t.dz = static_cast<const __nv_bfloat16*>(dz[i]);
      t.out = static_cast<__nv_bfloat16*>(dx[i]);
      t.w = w[i];
      t.H = H[i];
      t.items = static_cast<unsigned>(item_count(B, H[i], N));
      t.dw_part = dw[i] != nullptr ? part : nullptr;
      r.part[i] = part;
      if (part != nullptr) part += static_cast<size_t>(r.blocks[i]) * d;
    }
    p.cos = cos, p.sin = sin, p.pos = positions;
    p.N = N, p.rope = rope, p.table_rows = table_rows, p.interleaved = interleaved ? 1 : 0;
    p.w_bf16 = weight_bf16 ? 1 : 0, p.grid_q = r.blocks[0], p.eps = eps;
    if (launch_norm<true>(p, r.blocks[0] + r.blocks[1], d, stream) != cudaSuccess) return FA_ERR_CUDA;
  }
  if (!any_dw) return FA_OK;
  r.dw[0] = dw[0], r.dw[1] = dw[1];  // with no rows the sums are zero
  const dim3 grid(d / 32, 2);
  const cudaError_t e = d == 32   ? launch_pdl(dw_sum_kernel<32>, grid, dim3(256), 0, stream, r)
                        : d == 64 ? launch_pdl(dw_sum_kernel<64>, grid, dim3(256), 0, stream, r)
                                  : launch_pdl(dw_sum_kernel<128>, grid, dim3(256), 0, stream, r);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
