"""Tensor helpers of the operators around the attention: per-head norm and rotation of queries and keys, the paged
key/value cache, attention of drafted tokens over it (the C entry points are in include/fa.h).

They check their tensors, allocate outputs and workspace with PyTorch and launch on the current stream of the tensors'
device, like the helpers of the package's main module.  A decoding step calls them once per layer and its kernels take a
few microseconds, so the checks are few attribute reads each and a cache's are made once.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import FA_CACHE_BF16, FA_CACHE_E4M3, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, check, fa_cache, lib

_BF16, _F32, _I32, _I64, _U8, _E4M3 = (torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8,
                                       torch.float8_e4m3fn)
_BAD_SIZE = ctypes.c_size_t(-1).value
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def _call(fn, what, device, *args):
    """Launches on the current stream of `device` (an index), which is current for the call."""
    if _current_device() == device:
        status = fn(*args, _raw_stream(device))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _raw_stream(device))
    if status:
        check(status, what)


_Longs6, _Longs18 = ctypes.c_longlong * 6, ctypes.c_longlong * 18
_address = ctypes.addressof


def _ptr(t):
    """Address of a tensor's elements; None for no tensor and for an empty one."""
    return None if t is None else t.data_ptr() or None


def _check_rows(name, t):
    """bf16 CUDA tensor [B,H,N,d] with contiguous rows; its strides between batches, heads and rows."""
    if t.dtype is not _BF16 or t.dim() != 4 or not t.is_cuda:
        raise ValueError(f"{name}: expected a bf16 CUDA tensor of shape [B, H, N, d]")
    st = t.stride()
    if st[3] != 1 and t.numel() and t.shape[3] > 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    return st[:3]


def _check_ints(name, t, shape, device):
    if t.dtype is not _I32 or t.shape != shape or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous int32 tensor of shape {tuple(shape)} on cuda:{device}")


def _norm_args(q, k, q_weight, k_weight, cos, sin, positions):
    """Checks of qk_norm_rope and its gradients; (device, strides of q, of k, bf16 weights, rope, rows of the tables)."""
    sq, sk = _check_rows("q", q), _check_rows("k", k)
    B, _, N, d = q.shape
    device = q.get_device()
    ks = k.shape
    if ks[0] != B or ks[2] != N or ks[3] != d or k.get_device() != device:
        raise ValueError("k must be [B, Hk, N, d] with the B, N and d of q, on its device")
    for w in (q_weight, k_weight):
        if w is not None and (w.shape != (d,) or (w.dtype is not _F32 and w.dtype is not _BF16)
                              or w.get_device() != device or not w.is_contiguous()):
            raise ValueError("weights must be contiguous fp32 or bf16 tensors [d] on q's device")
    if q_weight is not None and k_weight is not None and q_weight.dtype is not k_weight.dtype:
        raise ValueError("both weights must have one type")
    one = k_weight if q_weight is None else q_weight
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin come together")
    rope = rows = 0
    if cos is not None:
        for t in (cos, sin):
            if t.dtype is not _F32 or t.dim() != 2 or t.shape != cos.shape or t.get_device() != device or \
                    not t.is_contiguous():
                raise ValueError("cos and sin must be contiguous fp32 tensors [positions, rope / 2] on q's device")
        rows, rope = cos.shape[0], 2 * cos.shape[1]
    if positions is not None:
        if cos is None:
            raise ValueError("positions need the cos and sin tables")
        _check_ints("positions", positions, (B, N), device)
    return device, sq, sk, int(one is not None and one.dtype is _BF16), rope, rows


def qk_norm_rope(q, k, q_weight=None, k_weight=None, cos=None, sin=None, positions=None, eps=1e-6, interleaved=False):
    """RMS norm of each head of bf16 q [B,H,N,d] and k [B,Hk,N,d] (any strides with contiguous rows, e.g. the
    transposed view of a projection's output), then rotation by position; contiguous bf16 [B,H,N,d], [B,Hk,N,d].

    cos, sin: fp32 [positions, rope/2]; positions: int32 [B,N], default 0..N-1 (a negative one marks a padding row,
    which comes back zero); interleaved: pairs (2i, 2i+1) instead of (i, i + rope/2).  See fa_qk_norm_rope."""
    device, sq, sk, bf16, rope, rows = _norm_args(q, k, q_weight, k_weight, cos, sin, positions)
    B, H, N, d = q.shape
    Hk = k.shape[1]
    qo = torch.empty((B, H, N, d), dtype=_BF16, device=q.device)
    ko = torch.empty((B, Hk, N, d), dtype=_BF16, device=q.device)
    strides = _Longs6(*sq, *sk)
    at = _address(strides)
    _call(lib.fa_qk_norm_rope, "fa_qk_norm_rope", device, _ptr(q), _ptr(k), _ptr(qo), _ptr(ko), at, at + 24, _ptr(q_weight), _ptr(k_weight), bf16, _ptr(cos), _ptr(sin), rope, rows, 1 if interleaved else 0,
          _ptr(positions), B, H, Hk, N, d, eps)
    return qo, ko


def qk_norm_rope_backward(q, k, dq_out, dk_out, q_weight=None, k_weight=None, cos=None, sin=None, positions=None,
                          eps=1e-6, interleaved=False, workspace=None):
    """dq, dk (in the layout of q and k) and the weights' gradients (None without a weight) of qk_norm_rope, from its
    inputs and the gradients of its outputs."""
    device, sq, sk, bf16, rope, rows = _norm_args(q, k, q_weight, k_weight, cos, sin, positions)
    sdq, sdk = _check_rows("dq_out", dq_out), _check_rows("dk_out", dk_out)
    for name, g, t in (("dq_out", dq_out, q), ("dk_out", dk_out, k)):
        if g.shape != t.shape or g.get_device() != device:
            raise ValueError(f"{name}: expected shape {tuple(t.shape)} on {t.device}")
    B, H, N, d = q.shape
    Hk = k.shape[1]
    dq, dk = torch.empty_like(q), torch.empty_like(k)
    dqw = None if q_weight is None else torch.empty_like(q_weight)
    dkw = None if k_weight is None else torch.empty_like(k_weight)
    n = 0
    if dqw is not None or dkw is not None:
        need = lib.fa_qk_norm_rope_bwd_workspace_size(B, H, Hk, N, d)
        if need == _BAD_SIZE:
            check(FA_ERR_UNSUPPORTED, "fa_qk_norm_rope_bwd_workspace_size")
        workspace, n = _workspace(workspace, need, q.device)
    else:
        workspace = None
    strides = _Longs18(*sq, *sk, *sdq, *sdk, *dq.stride()[:3], *dk.stride()[:3])
    at = _address(strides)
    _call(lib.fa_qk_norm_rope_bwd, "fa_qk_norm_rope_bwd", device, _ptr(q), _ptr(k), _ptr(dq_out), _ptr(dk_out), _ptr(dq),
          _ptr(dk), at, at + 24, at + 48, at + 72, at + 96, at + 120, _ptr(q_weight), _ptr(k_weight), _ptr(dqw), _ptr(dkw), bf16, _ptr(cos), _ptr(sin), rope, rows, 1 if interleaved else 0,
          _ptr(positions), B, H, Hk, N, d, eps, _ptr(workspace), n)
    return dq, dk, dqw, dkw


def _workspace(workspace, need, device):
    """The caller's workspace if it is large enough, else a new one, and its bytes."""
    if workspace is not None:
        n = workspace.numel() * workspace.element_size()
        if n >= need and workspace.device == device:
            return workspace, n
    return torch.empty(need or 16, dtype=_U8, device=device), need or 16


class KVCache:
    """A paged cache: k, v [pages, Hk, page_size, d], bf16, or float8_e4m3fn with one exponent byte per row in k_exp,
    v_exp (uint8 [pages, Hk, page_size]; a row's scale is 2^(byte - 127)).  The tensors are checked when the cache is
    first used."""

    __slots__ = ("k", "v", "k_exp", "v_exp", "_args")

    def __init__(self, k, v, k_exp=None, v_exp=None):
        self.k, self.v, self.k_exp, self.v_exp, self._args = k, v, k_exp, v_exp, None

    def __iter__(self):
        return iter((self.k, self.v, self.k_exp, self.v_exp))

    def args(self):
        """(device index, fa_cache)."""
        a = self._args
        if a is None or a[2] is not self.k or a[3] is not self.v or a[1].K != (self.k.data_ptr() or None) or \
                a[1].V != (self.v.data_ptr() or None):
            a = self._args = self._check()
        return a

    def _check(self):
        k, v = self.k, self.v
        for t in (k, v):
            if t.dim() != 4 or t.dtype not in (_BF16, _E4M3) or not t.is_cuda or not t.is_contiguous() or \
                    t.shape != k.shape or t.dtype != k.dtype or t.device != k.device:
                raise ValueError("a cache's k and v must be contiguous bf16 or float8_e4m3fn CUDA tensors "
                                 "[pages, Hk, page_size, d] of one type and device")
        fp8 = k.dtype == _E4M3
        for t in (self.k_exp, self.v_exp):
            if (t is not None) != fp8:
                raise ValueError("an e4m3 cache has exponent bytes k_exp and v_exp, a bf16 cache has none")
            if fp8 and (t.dtype != _U8 or t.shape != k.shape[:3] or t.device != k.device or not t.is_contiguous()):
                raise ValueError(
                    "exponent bytes must be contiguous uint8 tensors [pages, Hk, page_size] on the cache's device")
        pages, hk, page_size, d = k.shape
        c = fa_cache(_ptr(k), _ptr(v), _ptr(self.k_exp), _ptr(self.v_exp), FA_CACHE_E4M3 if fp8 else FA_CACHE_BF16,
                     pages, hk, page_size, d)
        return k.get_device(), c, k, v


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


def _cache_args(cache, table, lens, n_new):
    """Checks of a cache and its table; (fa_cache, (table, columns, stride, lens)), device index, B."""
    device, c = cache.args()[:2]
    if table.dim() != 2 or table.dtype is not _I32 or table.get_device() != device or \
            (table.shape[1] > 1 and table.stride(1) != 1):
        raise ValueError("the page table must be an int32 tensor [B, columns] on the cache's device, rows contiguous")
    B, cols = table.shape
    _check_ints("lens", lens, (B,), device)
    if n_new is not None:
        _check_ints("n_new", n_new, (B,), device)
    return c, (_ptr(table), cols, table.stride(0), _ptr(lens))


def cache_write(cache, k, v, table, lens, n_new=None):
    """Writes bf16 k, v [B,Hk,T,d] (any strides with contiguous rows) into the cache: token t < n_new[b] (default T) of
    sequence b goes to row lens[b] - n_new[b] + t of its pages table[b].  lens counts the new tokens."""
    sk, sv = _check_rows("k", k), _check_rows("v", v)
    c, tab = _cache_args(cache, table, lens, n_new)
    B, hk, T, d = k.shape
    device = k.get_device()
    if v.shape != k.shape or v.get_device() != device or B != table.shape[0] or hk != c.Hk or d != c.d or \
            device != cache.k.get_device():
        raise ValueError("k and v must be [B, Hk, T, d] with the table's B and the cache's Hk and d, on its device")
    strides = _Longs6(*sk, *sv)
    at = _address(strides)
    _call(lib.fa_cache_write, "fa_cache_write", device, c, _ptr(k), _ptr(v), at, at + 24, B, T, *tab, _ptr(n_new))


def cache_read(cache, table, lens, length):
    """k, v: rows 0 .. length-1 of every sequence as contiguous bf16 [B,Hk,length,d], zero behind lens[b]."""
    c, tab = _cache_args(cache, table, lens, None)
    B = table.shape[0]
    dev = table.device
    k = torch.empty((B, c.Hk, length, c.d), dtype=_BF16, device=dev)
    v = torch.empty((B, c.Hk, length, c.d), dtype=_BF16, device=dev)
    _call(lib.fa_cache_read, "fa_cache_read", cache.k.get_device(), c, _ptr(k), _ptr(v), B, length, *tab)
    return k, v


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
    if q.dtype is not _BF16 or q.dim() != 4 or not q.is_cuda or not q.is_contiguous():
        raise ValueError("q: expected a contiguous bf16 CUDA tensor of shape [B, H, T, d]")
    c, tab = _cache_args(cache, table, lens, n_new)
    B, H, T, d = q.shape
    device = q.get_device()
    if B != table.shape[0] or d != c.d or device != cache.k.get_device():
        raise ValueError("q must be [B, H, T, d] with the table's B and the cache's d, on its device")
    if H and (c.Hk == 0 or H % c.Hk):
        raise ValueError("the heads of q must be a multiple of the cache's")
    stride = 0
    if tree is not None:
        W = (T + 63) // 64
        if tree.dtype is not _I64 or tree.get_device() != device or not tree.is_contiguous() or \
                (tree.shape != (B, T, W) and tree.shape != (T, W)):
            raise ValueError(f"tree must be a contiguous int64 tensor [{B}, {T}, {W}] or [{T}, {W}] on q's device")
        stride = T * W if tree.dim() == 3 else 0
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = torch.empty_like(q)
    lse = torch.empty((B, H, T), dtype=_F32, device=q.device)
    need = lib.fa_fwd_tree_workspace_size(B, H, c.Hk, T, d)
    if need == _BAD_SIZE:
        check(FA_ERR_INVALID_ARG, "fa_fwd_tree_workspace_size")
    workspace, n = _workspace(workspace, need, q.device)
    _call(lib.fa_fwd_tree, "fa_fwd_tree", device, _ptr(q), c, _ptr(o), _ptr(lse), B, H, T, *tab, _ptr(n_new), _ptr(tree),
          stride, scale, workspace.data_ptr(), n)
    return o, lse
