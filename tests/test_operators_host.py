"""The operators around the attention, without a GPU: refusals of the C entry points and of the Python helpers, the
draft-tree words, and the oracle's own definitions against differences and brute force."""
import ctypes
import math

import pytest
import torch

from oracle import operators as orc

P = 4096  # a 16-byte aligned fake address: never dereferenced, validation fails first
BAD, NO, WS = 1, 2, 5  # FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_WORKSPACE


def norm(fa, **kw):
    a = dict(Q=P, K=P, Qo=P, Ko=P, qs=None, ks=None, qw=None, kw=None, wb=0, cos=P, sin=P, rope=64, rows=64, inter=0,
             pos=None, B=1, Hq=4, Hk=2, N=8, d=64, eps=1e-6, s=None)
    a.update(kw)
    return fa.fa_qk_norm_rope(*a.values())


@pytest.mark.parametrize("change, status", [
    (dict(d=48), NO), (dict(B=-1), BAD), (dict(Hq=-2), BAD), (dict(N=-1), BAD), (dict(B=70000), NO),
    (dict(N=(1 << 30) + 1, rows=2 ** 31 - 1), NO), (dict(eps=-1.0), BAD), (dict(eps=math.nan), BAD),
    (dict(eps=math.inf), BAD), (dict(sin=None), BAD), (dict(cos=None), BAD), (dict(cos=None, sin=None), BAD),
    (dict(cos=None, sin=None, rope=0, pos=P), BAD), (dict(rope=8), NO), (dict(rope=24), NO), (dict(rope=80), NO),
    (dict(rope=-16), BAD), (dict(N=65), BAD), (dict(cos=P + 4), BAD), (dict(pos=P + 2), BAD), (dict(Q=None), BAD),
    (dict(Ko=None), BAD), (dict(Q=P + 8), BAD), (dict(qw=P + 4), BAD), (dict(qs=(512, 64, 4), Hq=2), BAD),
    (dict(ks=(-8, 64, 64), B=2), BAD), (dict(rows=-1), BAD),
])
def test_norm_rope_refusals(fa_lib, change, status):
    assert norm(fa_lib, **change) == status


def test_norm_rope_empty_is_a_no_op(fa_lib):
    none = dict(Q=None, K=None, Qo=None, Ko=None)
    assert norm(fa_lib, B=0, **none) == 0
    assert norm(fa_lib, N=0, **none) == 0
    assert norm(fa_lib, Hq=0, Hk=0, **none) == 0


def grad(fa, **kw):
    a = dict(Q=P, K=P, dQo=P, dKo=P, dQ=P, dK=P, s1=None, s2=None, s3=None, s4=None, s5=None, s6=None, qw=P, kw=P,
             dqw=P, dkw=P, wb=0, cos=P, sin=P, rope=64, rows=64, inter=0, pos=None, B=2, Hq=4, Hk=2, N=8, d=64,
             eps=1e-6, ws=P, n=1 << 20, s=None)
    a.update(kw)
    return fa.fa_qk_norm_rope_bwd(*a.values())


@pytest.mark.parametrize("change, status", [
    (dict(d=96), NO), (dict(dQo=None), BAD), (dict(dK=None), BAD), (dict(ws=None), WS), (dict(n=16), WS),
    (dict(ws=P + 8), WS), (dict(s5=(0, 512, 64)), BAD), (dict(s5=(2048, 512, 0)), BAD), (dict(s6=(1024, 8, 64)), BAD),
    (dict(s3=(2048, 512, 60)), BAD), (dict(dqw=P + 2), BAD), (dict(dQ=P + 2), BAD), (dict(eps=-0.5), BAD),
])
def test_norm_rope_backward_refusals(fa_lib, change, status):
    assert grad(fa_lib, **change) == status


def test_norm_rope_backward_workspace_size(fa_lib):
    fa, bad = fa_lib, ctypes.c_size_t(-1).value
    assert fa.fa_qk_norm_rope_bwd_workspace_size(1, 4, 2, 8, 96) == bad
    assert fa.fa_qk_norm_rope_bwd_workspace_size(-1, 4, 2, 8, 64) == bad
    assert fa.fa_qk_norm_rope_bwd_workspace_size(0, 4, 2, 8, 64) == 0
    big = fa.fa_qk_norm_rope_bwd_workspace_size(8, 16, 16, 1 << 20, 128)
    assert 0 < fa.fa_qk_norm_rope_bwd_workspace_size(1, 1, 1, 1, 128) <= big <= 16 << 20  # bounded by the grid


def cache(fa, **kw):
    a = dict(K=P, V=P, K_exp=P, V_exp=P, format=fa.FA_CACHE_E4M3, pages=4, Hk=2, page_size=16, d=64)
    a.update(kw)
    return fa.fa_cache(*a.values())


BAD_CACHES = [
    (dict(d=48), NO), (dict(format=2), NO), (dict(page_size=8), NO), (dict(page_size=24), NO), (dict(page_size=0), NO),
    (dict(page_size=-16), BAD), (dict(pages=-1), BAD), (dict(Hk=-1), BAD), (dict(K=None), BAD), (dict(V=P + 8), BAD),
    (dict(K_exp=None), BAD), (dict(pages=1 << 30, Hk=2), NO), (dict(page_size=1 << 21), NO),
]


def write(fa, c, **kw):
    a = dict(K=P, V=P, ks=None, vs=None, B=2, T=3, table=P, cols=4, stride=4, lens=P, n_new=None, s=None)
    a.update(kw)
    return fa.fa_cache_write(c, *a.values())


def read(fa, c, **kw):
    a = dict(K=P, V=P, B=2, N=64, table=P, cols=4, stride=4, lens=P, s=None)
    a.update(kw)
    return fa.fa_cache_read(c, *a.values())


def tree(fa, c, **kw):
    a = dict(Q=P, O=P, L=P, B=2, H=4, T=3, table=P, cols=4, stride=4, lens=P, n_new=None, tree=None, ts=0, scale=0.1,
             ws=P, n=1 << 40, s=None)
    a.update(kw)
    q = a.pop("Q")
    return fa.fa_fwd_tree(q, c, *a.values())


@pytest.mark.parametrize("call", [write, read, tree])
@pytest.mark.parametrize("change, status", BAD_CACHES)
def test_bad_caches(fa_lib, call, change, status):
    assert call(fa_lib, cache(fa_lib, **change)) == status


TABLES = [(dict(B=-1), BAD), (dict(cols=-1), BAD), (dict(cols=1 << 27), NO), (dict(table=None), BAD),
          (dict(lens=None), BAD), (dict(stride=-4), BAD), (dict(B=40000), NO), (dict(table=P + 2), BAD),
          (dict(lens=P + 1), BAD)]


@pytest.mark.parametrize("call, change, status", [(c, *t) for c in (write, read, tree) for t in TABLES] + [
    (write, dict(T=-1), BAD), (write, dict(K=None), BAD), (write, dict(V=P + 8), BAD), (write, dict(n_new=P + 2), BAD),
    (write, dict(ks=(384, 192, 60)), BAD), (write, dict(vs=(-8, 192, 64)), BAD), (write, dict(T=2 ** 31 - 1), NO),
    (read, dict(N=-1), BAD), (read, dict(K=P + 8), BAD), (read, dict(V=None), BAD), (read, dict(N=2 ** 31 - 1), NO),
    (tree, dict(T=-1), BAD), (tree, dict(H=3), BAD), (tree, dict(H=-2), BAD), (tree, dict(H=40000), NO),
    (tree, dict(scale=0.0), BAD), (tree, dict(scale=math.nan), BAD), (tree, dict(Q=None), BAD), (tree, dict(O=P + 8), BAD),
    (tree, dict(L=P + 2), BAD), (tree, dict(tree=P + 4), BAD), (tree, dict(tree=P, ts=-1), BAD),
    (tree, dict(T=1 << 30), NO),
])
def test_cache_call_refusals(fa_lib, call, change, status):
    assert call(fa_lib, cache(fa_lib), **change) == status


def test_cache_calls_empty(fa_lib):
    fa, none = fa_lib, dict(K=None, V=None)
    assert write(fa, cache(fa), T=0, **none) == 0
    assert write(fa, cache(fa), B=0, table=None, lens=None, **none) == 0
    assert write(fa, cache(fa, pages=0, K=None, V=None, K_exp=None, V_exp=None)) == 0
    assert read(fa, cache(fa), N=0, **none) == 0
    assert tree(fa, cache(fa), T=0, Q=None, O=None, L=None) == 0
    assert tree(fa, cache(fa), H=0, Q=None, O=None, L=None) == 0


def test_tree_workspace_size(fa_lib):
    fa, bad = fa_lib, ctypes.c_size_t(-1).value
    assert fa.fa_fwd_tree_workspace_size(2, 4, 3, 1, 64) == bad
    assert fa.fa_fwd_tree_workspace_size(2, 4, 2, 1, 48) == bad
    assert fa.fa_fwd_tree_workspace_size(-2, 4, 2, 1, 64) == bad
    assert fa.fa_fwd_tree_workspace_size(0, 4, 2, 1, 64) == 0


def test_helpers_refuse_cpu_tensors(fa_lib):
    fa = fa_lib
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.qk_norm_rope(x, x)
    with pytest.raises(ValueError):
        fa.qk_norm_rope_backward(x, x, x, x)
    c = fa.KVCache(x, x)
    i = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.cache_write(c, x, x, i, i[0])
    with pytest.raises(ValueError):
        fa.cache_read(c, i, i[0], 4)
    with pytest.raises(ValueError):
        fa.attention_tree(x, c, i, i[0])
    with pytest.raises(ValueError):
        fa.new_cache(1, 1, 16, 64, dtype=torch.float16, device="cpu")


def test_helpers_refuse_what_is_no_tensor(fa_lib):
    fa = fa_lib
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, 1, dtype=torch.int32)
    for bad in (lambda: fa.qk_norm_rope(x, None), lambda: fa.qk_norm_rope([1.0], x), lambda: fa.qk_norm_rope(x, x, 1.0),
                lambda: fa.cache_write(fa.KVCache(None, x), x, x, i, i[0]),
                lambda: fa.attention_tree(7, fa.KVCache(x, x), i, i[0])):
        with pytest.raises((TypeError, ValueError)):
            bad()


def test_tree_words(fa_lib):
    fa = fa_lib
    w = fa.tree_words([-1, 0, 0, 1, -1])
    assert w.shape == (5, 1) and w[:, 0].tolist() == [0b1, 0b11, 0b101, 0b1011, 0b10000]
    chain = fa.tree_words(torch.arange(130)[None].expand(2, 130) - 1)
    assert chain.shape == (2, 130, 3)
    for t in (0, 62, 63, 64, 127, 129):
        bits = sum((int(v) % 2 ** 64) << (64 * i) for i, v in enumerate(chain[1, t]))
        assert bits == 2 ** (t + 1) - 1
    assert fa.tree_words([]).shape == (0, 0)
    for bad in ([0], [-1, 1], [-2]):
        with pytest.raises(ValueError):
            fa.tree_words(bad)


# ------------------------------------------------------------------ the oracle itself

@pytest.mark.parametrize("d, rope, interleaved", [(32, 32, False), (64, 32, True), (32, 0, False)])
def test_oracle_norm_rope_gradients_against_differences(d, rope, interleaved):
    g = torch.Generator().manual_seed(d + rope)
    x, dz = (torch.randn(1, 2, 3, d, generator=g, dtype=torch.float64) for _ in range(2))
    w = torch.randn(d, generator=g, dtype=torch.float64)
    ang = torch.rand(8, rope // 2, generator=g, dtype=torch.float64) * 6
    cos, sin = (ang.cos(), ang.sin()) if rope else (None, None)
    pos = torch.tensor([[5, -1, 2]], dtype=torch.int32) if rope else None

    def loss(x, w):
        return (orc.norm_rope(x, w, cos, sin, pos, 1e-3, interleaved)[0] * dz).sum()

    dx, dw, _, _ = orc.norm_rope_grad(x, dz, w, cos, sin, pos, 1e-3, interleaved)
    step = 1e-6
    for at in [(0, 0, 0, 0), (0, 1, 2, d - 1), (0, 1, 0, d // 2), (0, 0, 1, 3)]:
        e = torch.zeros_like(x)
        e[at] = step
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * step) - dx[at]) < 1e-7
    for c in (0, d // 2, d - 1):
        e = torch.zeros_like(w)
        e[c] = step
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * step) - dw[c]) < 1e-7


def test_oracle_e4m3_is_the_nearest_value_of_the_format():
    grid = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).to(torch.float64)  # 0 .. 448, NaN left out
    g = torch.Generator().manual_seed(3)
    for mult in (1.0, 1e-3, 3e4, 448.0, 1e-30):
        x = (torch.randn(64, generator=g) * mult).to(torch.bfloat16)
        val, byte = orc.e4m3_row(x)
        scale = 2.0 ** (byte - 127)
        assert float(x.abs().max()) <= 448 * scale and (byte == 27 or float(x.abs().max()) > 224 * scale)
        err = (val - x.to(torch.float64)).abs()
        best = ((x.to(torch.float64).abs() / scale)[:, None] - grid).abs().amin(1) * scale
        assert torch.equal(err, best)
    assert orc.e4m3_row(torch.tensor([1.0, math.inf]))[1] == 255


def test_oracle_tree_is_attention_when_the_tree_is_a_chain():
    import oracle
    g = torch.Generator().manual_seed(9)
    q = torch.randn(1, 2, 3, 32, generator=g, dtype=torch.float64)
    k, v = (torch.randn(1, 2, 16, 32, generator=g, dtype=torch.float64) for _ in range(2))  # one page, two heads
    table, lens = torch.zeros(1, 1, dtype=torch.int32), torch.tensor([11], dtype=torch.int32)
    o, lse, _, _ = orc.tree_attention(q, k, v, table, lens, None, None, 32 ** -0.5)
    # rows at the end of an 11-key sequence: the last 3 rows of full causal attention
    full_q = torch.cat([torch.zeros(1, 2, 8, 32, dtype=torch.float64), q], 2).numpy()
    O, L = oracle.standard_attention_fwd(full_q, k[:, :, :11].numpy(), v[:, :, :11].numpy(), True)
    assert abs(o.numpy() - O[:, :, 8:]).max() < 1e-12 and abs(lse.numpy() - L[:, :, 8:]).max() < 1e-12
