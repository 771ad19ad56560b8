// The paged key/value cache: rows written into it (rounded to bf16's own values, or
// quantised to e4m3) and read back out of it.
//
// e4m3 rows carry one power-of-two scale each, 2^k with the least k such that
// max |x| <= 448 2^k, stored as the byte k + 127.  A power of two costs a floating
// point format nothing in relative precision and makes both directions exact but for
// the one rounding to 4 significant bits: x 2^-k and v 2^k are exact in fp32, and every
// value read back is a bf16 number.
//
// Both kernels are bound by memory.  A lane holds 16 bytes of a bf16 row (D / 8 lanes to
// a row); neighbouring lane groups take neighbouring positions of one head, which lie
// next to each other in a page.  Rows are independent, so the order of the work does
// not change what is stored.
#include <cuda_fp8.h>

#include "cache.cuh"

namespace fa {

namespace {

constexpr int kThreads = 256;
constexpr int kRows = 4;      // rows per lane group and step, read and written
// Blocks, at most, for each of K and V: so many that few lane groups take a second step.
// The rows' addresses come from the lengths and the table, and a block that waits for
// those is best overlapped by another.  Measured at 8 heads of 128 (blocks 152 x 4 / x 8 /
// x 64): writing 4 x up to 8192 bf16 rows 34.9 / 33.8 / 31.1 us (6.4 TB/s); 2048 e4m3
// rows each of 4 sequences written and up to 16384 rows read back 78 / 71.9 / 68.2 us.
// Rows at a time when reading back: 1, 2, 4, 8: 107, 68.5, 68.2, 68.5 us.
constexpr int kMaxBlocks = 152 * 64;

struct WriteArgs {
  CacheView c;
  const __nv_bfloat16* x[2];  // new keys, new values
  RowStrides s[2];
  unsigned items;             // B * Hk * ceil(T / kRows); the grid's y picks K or V
};

// The largest of 8 bf16 magnitudes, as the 15 bits of its encoding (NaN above infinity
// above every number).
FA_DEV uint32_t max_abs_bits(uint4 v) {
  const uint32_t m = 0x7fff7fffu;
  const uint32_t a = __vmaxu2(__vmaxu2(v.x & m, v.y & m), __vmaxu2(v.z & m, v.w & m));
  return max(a & 0xffffu, a >> 16);
}
// The exponent byte of a row whose largest magnitude has these bits.
FA_DEV int exponent_byte(uint32_t bits) {
  if (bits >= 0x7f80u) return kExpNaN;
  const int e = static_cast<int>(bits >> 7) - 8 + ((bits & 0x7fu) > 0x60u);  // 448 = 1.75 * 2^8
  return e < kExpMin ? kExpMin : e;
}
FA_DEV float clamp_abs(float x, float lim) {  // NaN stays NaN
  return fabsf(x) > lim ? copysignf(lim, x) : x;
}
FA_DEV uint32_t to_e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const __grid_constant__ WriteArgs p) {
  constexpr int LPR = D / 8, GPW = 32 / LPR;
  const CacheView& c = p.c;
  const int which = blockIdx.y;
  uint8_t* data = which ? c.V : c.K;
  uint8_t* exps = which ? c.Ve : c.Ke;
  const RowStrides s = p.s[which];
  const int lane = threadIdx.x & 31, part = lane % LPR;
  const unsigned group = (blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * GPW + lane / LPR;
  const unsigned ngroups = gridDim.x * (kThreads / 32) * GPW;
  const unsigned tblocks = (c.T + kRows - 1) / kRows;
  pdl_wait();
  const unsigned trips = (p.items + ngroups - 1) / ngroups;
  for (unsigned trip = 0; trip < trips; ++trip) {
    const unsigned item = group + trip * ngroups;
    const bool live = item < p.items;
    const unsigned bh = live ? item / tblocks : 0;
    const int t0 = live ? static_cast<int>(item - bh * tblocks) * kRows : 0;
    const int b = bh / c.Hk, h = bh - b * c.Hk;
    const int nn = live ? seq_new(c, b) : 0;
    const __nv_bfloat16* x = p.x[which] + b * s.b + h * s.h + t0 * s.n + part * 8;
    uint4 v[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      v[i] = t0 + i < nn ? *reinterpret_cast<const uint4*>(x + i * s.n) : make_uint4(0, 0, 0, 0);
    const int first = live ? seq_prefix(c, b) + t0 : 0;  // position of token t0
    const int cap = c.cols << c.page_shift;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int j = first + i;
      const int page = t0 + i < nn && j >= 0 && j < cap ? page_of(c, b, j) : -1;
      const size_t row =
          (static_cast<size_t>(page < 0 ? 0 : page) * c.Hk + h) * c.page + (j & (c.page - 1));
      if constexpr (!FP8) {
        if (page >= 0) *reinterpret_cast<uint4*>(data + row * (D * 2) + part * 16) = v[i];
      } else {
        uint32_t m = max_abs_bits(v[i]);
#pragma unroll
        for (int k = LPR / 2; k > 0; k >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, k));
        const int e = exponent_byte(m);
        // 2^(127 - e); a row with an infinity or a NaN stores NaN in every element
        const float inv = e == kExpNaN ? __int_as_float(0x7fffffff) : __int_as_float((254 - e) << 23);
        // at the largest scale, 2^120, a value may not round up to 256 2^120 = 2^128
        const float lim = e == kExpMax ? 240.f : 448.f;
        const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        float f[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          f[2 * k] = clamp_abs(__uint_as_float(u[k] << 16) * inv, lim);
          f[2 * k + 1] = clamp_abs(__uint_as_float(u[k] & 0xffff0000u) * inv, lim);
        }
        if (page >= 0) {
          *reinterpret_cast<uint2*>(data + row * D + part * 8) =
              make_uint2(to_e4m3x4(f[0], f[1], f[2], f[3]), to_e4m3x4(f[4], f[5], f[6], f[7]));
          if (part == 0) exps[row] = static_cast<uint8_t>(e);
        }
      }
    }
  }
}

struct ReadArgs {
  CacheView c;
  __nv_bfloat16* out[2];
  unsigned items;  // B * Hk * ceil(N / kRows)
  int N;
};

template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const __grid_constant__ ReadArgs p) {
  constexpr int LPR = D / 8, GPW = 32 / LPR;  // 8 elements in a lane
  const CacheView& c = p.c;
  const int which = blockIdx.y;
  const uint8_t* data = which ? c.V : c.K;
  const uint8_t* exps = which ? c.Ve : c.Ke;
  const int lane = threadIdx.x & 31, part = lane % LPR;
  const unsigned group = (blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * GPW + lane / LPR;
  const unsigned ngroups = gridDim.x * (kThreads / 32) * GPW;
  const unsigned nblocks = (p.N + kRows - 1) / kRows;
  pdl_wait();
  for (unsigned item = group; item < p.items; item += ngroups) {
    const unsigned bh = item / nblocks;
    const int j0 = static_cast<int>(item - bh * nblocks) * kRows;
    const int b = bh / c.Hk, h = bh - b * c.Hk;
    const int len = seq_len(c, b);
    // a page holds a multiple of kRows rows: one entry for the item
    const int entry = c.cols > 0 ? table_entry(c, b, j0) : -1;
    const int page = entry >= 0 && entry < c.pages ? entry : -1;
    const size_t row = (static_cast<size_t>(page < 0 ? 0 : page) * c.Hk + h) * c.page + (j0 & (c.page - 1));
    uint4 v[kRows];
    uint8_t e[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      v[i] = make_uint4(0, 0, 0, 0);
      e[i] = 0;
      if (page >= 0 && j0 + i < len) {
        if constexpr (FP8) {
          const uint2 q = *reinterpret_cast<const uint2*>(data + (row + i) * D + part * 8);
          v[i].x = q.x, v[i].y = q.y;
          e[i] = exps[row + i];
        } else {
          v[i] = *reinterpret_cast<const uint4*>(data + (row + i) * (2 * D) + part * 16);
        }
      }
    }
    uint4* out = reinterpret_cast<uint4*>(p.out[which] + (static_cast<size_t>(bh) * p.N + j0) * D + part * 8);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (j0 + i >= p.N) break;
      if constexpr (FP8) {
        const float scale = __int_as_float(static_cast<int>(e[i]) << 23);
        const uint32_t q[4] = {v[i].x & 0xffffu, v[i].x >> 16, v[i].y & 0xffffu, v[i].y >> 16};
        uint32_t r[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(q[k]), __NV_E4M3);
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hr));
          r[k] = pack_bf16x2(f.x * scale, f.y * scale);
        }
        out[static_cast<size_t>(i) * D / 8] = make_uint4(r[0], r[1], r[2], r[3]);
      } else {
        out[static_cast<size_t>(i) * D / 8] = v[i];
      }
    }
  }
}

int blocks_for(long long items, int lanes, int most) {  // lanes: of a row
  const long long per_block = (kThreads / 32) * (32 / lanes);
  const long long n = (items + per_block - 1) / per_block;
  return static_cast<int>(n < most ? n : most);
}

}  // namespace

fa_status make_cache_view(const fa_cache* c, const int* table, int cols, long long table_stride, const int* lens,
                          const int* n_new, int B, int T, CacheView* out) {
  if (c == nullptr || B < 0 || T < 0 || cols < 0) return FA_ERR_INVALID_ARG;
  if (c->pages < 0 || c->Hk < 0 || c->page_size < 0) return FA_ERR_INVALID_ARG;
  if (c->d != 32 && c->d != 64 && c->d != 128) return FA_ERR_UNSUPPORTED;
  if (c->format != FA_CACHE_BF16 && c->format != FA_CACHE_E4M3) return FA_ERR_UNSUPPORTED;
  if (c->page_size < 16 || (c->page_size & (c->page_size - 1)) != 0 || c->page_size > (1 << 20))
    return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * c->Hk > 65535 || T > (1 << 30)) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(c->pages) * c->Hk > 0x7fffffffLL - 1) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(cols) * c->page_size > (1LL << 30)) return FA_ERR_UNSUPPORTED;
  if (B > 1 && table_stride < 0) return FA_ERR_INVALID_ARG;
  const bool some = c->pages > 0 && c->Hk > 0;
  if (some && (!c->K || !c->V || !aligned(c->K, 16) || !aligned(c->V, 16))) return FA_ERR_INVALID_ARG;
  if (some && c->format == FA_CACHE_E4M3 &&
      (!c->K_exp || !c->V_exp || !aligned(c->K_exp, 16) || !aligned(c->V_exp, 16)))
    return FA_ERR_INVALID_ARG;
  if (B > 0 && (!lens || (!table && cols > 0))) return FA_ERR_INVALID_ARG;
  if (!aligned(table, 4) || !aligned(lens, 4) || !aligned(n_new, 4)) return FA_ERR_INVALID_ARG;
  int shift = 0;
  while ((1 << shift) < c->page_size) ++shift;
  *out = CacheView{static_cast<uint8_t*>(c->K), static_cast<uint8_t*>(c->V), c->K_exp, c->V_exp, table,
                   B > 1 ? table_stride : 0, lens, n_new, cols, c->pages, c->Hk, c->page_size, shift, T};
  return FA_OK;
}

}  // namespace fa

using namespace fa;

extern "C" {

fa_status fa_cache_write(const fa_cache* cache, const void* K, const void* V, const long long* k_strides,
                         const long long* v_strides, int B, int T, const int* table, int table_cols,
                         long long table_stride, const int* lens, const int* n_new, fa_stream_t stream) {
  WriteArgs p{};
  const fa_status st = make_cache_view(cache, table, table_cols, table_stride, lens, n_new, B, T, &p.c);
  if (st != FA_OK) return st;
  const int d = cache->d;
  if (!read_strides(k_strides, B, cache->Hk, T, d, &p.s[0]) || !read_strides(v_strides, B, cache->Hk, T, d, &p.s[1]))
    return FA_ERR_INVALID_ARG;
  const long long items = static_cast<long long>(B) * cache->Hk * ((static_cast<long long>(T) + kRows - 1) / kRows);
  if (items > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  if (items == 0 || cache->pages == 0 || table_cols == 0) return FA_OK;
  if (!K || !V || !aligned(K, 16) || !aligned(V, 16)) return FA_ERR_INVALID_ARG;
  p.x[0] = static_cast<const __nv_bfloat16*>(K);
  p.x[1] = static_cast<const __nv_bfloat16*>(V);
  p.items = static_cast<unsigned>(items);
  const dim3 grid(blocks_for(items, d / 8, kMaxBlocks), 2);
  const bool fp8 = cache->format == FA_CACHE_E4M3;
  cudaError_t e = cudaSuccess;
#define FA_WRITE(D)  \
  case D:  \
    if (fp8) e = launch_pdl(cache_write_kernel<D, true>, grid, dim3(kThreads), 0, stream, p);  \
    else e = launch_pdl(cache_write_kernel<D, false>, grid, dim3(kThreads), 0, stream, p);  \
    break;
  switch (d) {
    FA_WRITE(32)
    FA_WRITE(64)
    FA_WRITE(128)
  }
#undef FA_WRITE
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_cache_read(const fa_cache* cache, void* K, void* V, int B, int N, const int* table, int table_cols,
                        long long table_stride, const int* lens, fa_stream_t stream) {
  ReadArgs p{};
  if (N < 0) return FA_ERR_INVALID_ARG;
  const fa_status st = make_cache_view(cache, table, table_cols, table_stride, lens, nullptr, B, 0, &p.c);
  if (st != FA_OK) return st;
  if (N > (1 << 30)) return FA_ERR_UNSUPPORTED;
  const int d = cache->d;
  const long long items = static_cast<long long>(B) * cache->Hk * ((static_cast<long long>(N) + kRows - 1) / kRows);
  if (items > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  if (items == 0) return FA_OK;
  if (!K || !V || !aligned(K, 16) || !aligned(V, 16)) return FA_ERR_INVALID_ARG;
  p.out[0] = static_cast<__nv_bfloat16*>(K);
  p.out[1] = static_cast<__nv_bfloat16*>(V);
  p.items = static_cast<unsigned>(items);
  p.N = N;
  const bool fp8 = cache->format == FA_CACHE_E4M3;
  const dim3 grid(blocks_for(items, d / 8, kMaxBlocks), 2);
  cudaError_t e = cudaSuccess;
#define FA_READ(D)  \
  case D:  \
    if (fp8) e = launch_pdl(cache_read_kernel<D, true>, grid, dim3(kThreads), 0, stream, p);  \
    else e = launch_pdl(cache_read_kernel<D, false>, grid, dim3(kThreads), 0, stream, p);  \
    break;
  switch (d) {
    FA_READ(32)
    FA_READ(64)
    FA_READ(128)
  }
#undef FA_READ
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
