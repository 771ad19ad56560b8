// Attention of drafted tokens over the paged cache (a single token is a tree of one).
//
// Sequence b has lens[b] keys in the cache, the last n_new[b] of them the drafted
// tokens' own.  Draft token t sees every key of the prefix and, of the drafted ones,
// those whose bit is set in its row of `tree` (without a tree: tokens 0..t).  With
// s_j = q k_j scale over the keys it sees:
//   m = max s_j,  l = sum exp(s_j - m),  O = sum exp(s_j - m) v_j / l,  L = m + ln l.
// A row that sees no key gets O = 0 and L = -inf.
//
// One block per query row, one key per warp at a time, online softmax in each warp and
// one merge at the end.
#include <cuda_fp8.h>

#include <cmath>

#include "cache.cuh"

namespace fa {

namespace {

struct TreeArgs {
  CacheView c;
  const __nv_bfloat16* Q;
  __nv_bfloat16* O;
  float* L;
  const unsigned long long* tree;  // [.., T, words], or null
  long long tree_stride;           // words between sequences
  int B, H, words;
  float c_log2;
};

template <int D, bool FP8>
__global__ void __launch_bounds__(128) tree_rows_kernel(const __grid_constant__ TreeArgs p) {
  constexpr int EPL = D / 32;
  const CacheView& c = p.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x, bh = blockIdx.y, b = bh / p.H, h = bh - b * p.H, hk = h / (p.H / c.Hk);
  const size_t row = static_cast<size_t>(bh) * c.T + t;
  const int len = t < seq_new(c, b) ? seq_len(c, b) : 0, prefix = seq_prefix(c, b);
  float q[EPL], o[EPL] = {}, m = -INFINITY, l = 0.f;
  for (int e = 0; e < EPL; ++e) q[e] = __bfloat162float(p.Q[row * D + e * 32 + lane]) * p.c_log2;
  for (int j = warp; j < len; j += 4) {
    const int dj = j - prefix;
    if (dj >= 0) {
      const bool seen = p.tree == nullptr
                            ? dj <= t
                            : p.tree[b * p.tree_stride + static_cast<size_t>(t) * p.words + dj / 64] >> (dj % 64) & 1;
      if (!seen) continue;
    }
    const int page = page_of(c, b, j);
    if (page < 0) continue;
    const size_t kr = (static_cast<size_t>(page) * c.Hk + hk) * c.page + (j & (c.page - 1));
    auto load = [&](const uint8_t* data, const uint8_t* exps, int e) -> float {
      if constexpr (FP8) {
        const __half_raw hr = __nv_cvt_fp8_to_halfraw(data[kr * D + e * 32 + lane], __NV_E4M3);
        return __half2float(__half(hr)) * __int_as_float(static_cast<int>(exps[kr]) << 23);
      } else {
        return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(data)[kr * D + e * 32 + lane]);
      }
    };
    float s = 0.f;
    for (int e = 0; e < EPL; ++e) s = fmaf(q[e], load(c.K, c.Ke, e), s);
    for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    const float mn = fmaxf(m, s);
    const float a = m == -INFINITY ? 0.f : exp2f(m - mn), w = exp2f(s - mn);
    l = l * a + w;
    for (int e = 0; e < EPL; ++e) o[e] = fmaf(w, load(c.V, c.Ve, e), o[e] * a);
    m = mn;
  }
  __shared__ float sm[4], sl[4], so[4][D];
  if (lane == 0) sm[warp] = m, sl[warp] = l;
  for (int e = 0; e < EPL; ++e) so[warp][e * 32 + lane] = o[e];
  __syncthreads();
  if (warp != 0) return;
  const float mx = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  float f[4], lt = 0.f;
  for (int w = 0; w < 4; ++w) {
    f[w] = sm[w] == -INFINITY ? 0.f : exp2f(sm[w] - mx);
    lt += f[w] * sl[w];
  }
  for (int e = 0; e < EPL; ++e) {
    float v = 0.f;
    for (int w = 0; w < 4; ++w)
      if (f[w] != 0.f) v += f[w] * so[w][e * 32 + lane];
    p.O[row * D + e * 32 + lane] = __float2bfloat16_rn(lt == 0.f ? 0.f : v / lt);
  }
  if (lane == 0) p.L[row] = lt == 0.f ? -INFINITY : (mx + log2f(lt)) * 0.6931471805599453f;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_fwd_tree_workspace_size(int B, int H, int Hk, int T, int d) {
  if (B < 0 || H < 0 || Hk < 0 || T < 0 || (d != 32 && d != 64 && d != 128) || (H > 0 && (Hk == 0 || H % Hk != 0)))
    return static_cast<size_t>(-1);
  return 0;
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
  if (static_cast<long long>(H / cache->Hk) * T > (1LL << 30)) return FA_ERR_UNSUPPORTED;
  if (!Q || !O || !L || !aligned(Q, 16) || !aligned(O, 16) || !aligned(L, 4)) return FA_ERR_INVALID_ARG;
  (void)workspace, (void)workspace_bytes;
  p.Q = static_cast<const __nv_bfloat16*>(Q);
  p.O = static_cast<__nv_bfloat16*>(O);
  p.L = L;
  p.tree = tree;
  p.tree_stride = B > 1 ? tree_stride : 0;
  p.B = B, p.H = H, p.words = (T + 63) / 64;
  p.c_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  const dim3 grid(T, B * H);
  const bool fp8 = cache->format == FA_CACHE_E4M3;
#define FA_TREE(D)                                                       \
  case D:                                                                \
    if (fp8) tree_rows_kernel<D, true><<<grid, 128, 0, stream>>>(p);     \
    else tree_rows_kernel<D, false><<<grid, 128, 0, stream>>>(p);        \
    break;
  switch (cache->d) {
    FA_TREE(32)
    FA_TREE(64)
    FA_TREE(128)
  }
#undef FA_TREE
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
