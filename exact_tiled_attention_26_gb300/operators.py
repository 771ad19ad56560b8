"""Tensor calls of the operators around the attention: per-head norm and rotation of queries and keys, the paged
key/value cache, attention of drafted tokens over it (the C entry points are in include/fa.h).

They check their tensors, allocate outputs and workspace with PyTorch and launch on the current stream of the tensors'
device, like the helpers of the package's main module.  A decoding step calls them once per layer and its kernels take a
few microseconds, so that work is native (csrc/tensor_calls.cpp).  A refused tensor raises ValueError, a status of the
library FAError.  Rows of strided tensors start on 16 bytes: their strides are multiples of 8 elements.
"""
from __future__ import annotations

import torch

try:
    from . import tensor_calls as _native
except ImportError as e:
    raise ImportError("tensor_calls.so is missing or does not load: build it with `python "
                      "exact_tiled_attention_26_gb300/build.py` (or __graft_entry__.build())") from e

_BF16, _I64, _U8, _E4M3 = torch.bfloat16, torch.int64, torch.uint8, torch.float8_e4m3fn


def qk_norm_rope(q, k, q_weight=None, k_weight=None, cos=None, sin=None, positions=None, eps=1e-6, interleaved=False):
    """RMS norm of each head of bf16 q [B,H,N,d] and k [B,Hk,N,d] (any strides with contiguous rows, e.g. the
    transposed view of a projection's output), then rotation by position; contiguous bf16 [B,H,N,d], [B,Hk,N,d].

    cos, sin: fp32 [positions, rope/2]; positions: int32 [B,N], default 0..N-1 (a negative one marks a padding row,
    which comes back zero); interleaved: pairs (2i, 2i+1) instead of (i, i + rope/2).  See fa_qk_norm_rope."""
    return _native.qk_norm_rope(q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved)


def qk_norm_rope_backward(q, k, dq_out, dk_out, q_weight=None, k_weight=None, cos=None, sin=None, positions=None,
                          eps=1e-6, interleaved=False, workspace=None):
    """dq, dk (in the layout of q and k) and the weights' gradients (None without a weight) of qk_norm_rope, from its
    inputs and the gradients of its outputs."""
    return _native.qk_norm_rope_backward(q, k, dq_out, dk_out, q_weight, k_weight, cos, sin, positions, eps,
                                         interleaved, workspace)


class KVCache:
    """A paged cache: k, v [pages, Hk, page_size, d], bf16, or float8_e4m3fn with one exponent byte per row in k_exp,
    v_exp (uint8 [pages, Hk, page_size]; a row's scale is 2^(byte - 127)).  The calls that use it check its tensors."""

    __slots__ = ("k", "v", "k_exp", "v_exp")

    def __init__(self, k, v, k_exp=None, v_exp=None):
        self.k, self.v, self.k_exp, self.v_exp = k, v, k_exp, v_exp

    def __iter__(self):
        return iter((self.k, self.v, self.k_exp, self.v_exp))


def new_cache(pages, heads, page_size, d, dtype=None, device=None):
    """A KVCache of zeros; dtype: torch.bfloat16 (the default) or torch.float8_e4m3fn."""
    dtype = _BF16 if dtype is None else dtype
    if dtype not in (_BF16, _E4M3):
        raise ValueError("a cache is bf16 or float8_e4m3fn")
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    shape = (pages, heads, page_size, d)
    if dtype == _BF16:
        return KVCache(*(torch.zeros(shape, dtype=dtype, device=device) for _ in range(2)))
    return KVCache(*(torch.zeros(shape, dtype=_U8, device=device).view(dtype) for _ in range(2)),
                   *(torch.zeros(shape[:3], dtype=_U8, device=device) for _ in range(2)))


def cache_write(cache, k, v, table, lens, n_new=None):
    """Writes bf16 k, v [B,Hk,T,d] (any strides with contiguous rows) into the cache: token t < n_new[b] (default T) of
    sequence b goes to row lens[b] - n_new[b] + t of its pages table[b].  lens counts the new tokens."""
    _native.cache_write(cache.k, cache.v, cache.k_exp, cache.v_exp, k, v, table, lens, n_new)


def cache_read(cache, table, lens, length):
    """k, v: rows 0 .. length-1 of every sequence as contiguous bf16 [B,Hk,length,d], zero behind lens[b]."""
    return _native.cache_read(cache.k, cache.v, cache.k_exp, cache.v_exp, table, lens, length)


def tree_words(parents):
    """The `tree` of attention_tree from draft trees: parents is a CPU integer tensor or nested list [T] or [B,T] with
    the index of the token that each token follows (smaller than its own), or -1 at a root.  Returns int64 words
    [T, W] or [B, T, W] on the CPU: bit j of a token's words is set for itself and its ancestors."""
    p = torch.as_tensor(parents)
    rows = (p if p.dim() == 2 else p[None]).tolist()
    T = p.shape[-1]
    W = (T + 63) // 64
    out = []
    for row in rows:
        seen = []
        for t, at in enumerate(row):
            if not -1 <= at < t:
                raise ValueError("a token's parent must come before it (-1: none)")
            seen.append((seen[at] if at >= 0 else 0) | 1 << t)
        words = [[(s >> (64 * w)) & (2 ** 64 - 1) for w in range(W)] for s in seen]
        out.append([[u - 2 ** 64 if u >= 2 ** 63 else u for u in ws] for ws in words])
    res = torch.tensor(out, dtype=_I64).reshape(len(rows), T, W)
    return res if p.dim() == 2 else res[0]


def attention_tree(q, cache, table, lens, tree=None, n_new=None, scale=None, workspace=None):
    """O [B,H,T,d], L [B,H,T] of T drafted tokens per sequence (T = 1: a decoded token) over the cache that holds their
    own keys and values too: q bf16 contiguous [B,H,T,d], H a multiple of the cache's heads.  tree: int64 words [B,T,W]
    or, for one tree, [T,W], W = ceil(T/64) (tree_words); None: token t sees tokens 0..t.  See fa_fwd_tree."""
    return _native.attention_tree(q, cache.k, cache.v, cache.k_exp, cache.v_exp, table, lens, tree, n_new, scale,
                                  workspace)
