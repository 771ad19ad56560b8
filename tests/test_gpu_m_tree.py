"""Attention of drafted tokens over the paged cache, against the float64 oracle.

Tolerances, per element.  A score adds d products in fp32: off by at most 2 d 2^-24 of sum |q k| scale =: e, which
changes each weight by a factor within 1 +- 2 e.  Weights enter the second product rounded to bf16 (2^-8 each) and are
normalised by their own sum (2^-8 again at worst), sums in fp32 and the exponential's few ulp are below 2^-14.  So
|O - ref| <= 2^-8 |ref| + (2^-7 + 2 e + 2^-14) sum p |v|, and |L - ref| <= e + 2^-18 (1 + |ref|).
"""
import math

import pytest
import torch

from oracle import operators as orc

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4M3 = torch.float8_e4m3fn


def cache_values(cache):
    out = []
    for data, exps in ((cache.k, cache.k_exp), (cache.v, cache.v_exp)):
        vals = data.cpu().double()
        if exps is not None:
            e = exps.cpu().double()
            vals = vals * torch.where(e == 255, math.nan, 2.0 ** (e - 127))[..., None]
        out.append(vals)
    return out


def random_tree(B, T, g):
    """Tree words [B,T,W] and the bits of every token as Python integers."""
    W = (T + 63) // 64
    bits = [[0] * T for _ in range(B)]
    for b in range(B):
        for t in range(T):
            p = int(torch.randint(max(-1, t - 5), max(t, 0), (1,), generator=g)) if t else -1
            bits[b][t] = (bits[b][p] if p >= 0 else 0) | 1 << t
    words = [[[(s >> 64 * w) & (2 ** 64 - 1) for w in range(W)] for s in row] for row in bits]
    words = [[[u - 2 ** 64 if u >= 2 ** 63 else u for u in ws] for ws in row] for row in words]
    return torch.tensor(words, dtype=torch.int64), bits


def make(fa, B, H, Hk, T, d, page, cols, fp8, seed, mult=1.0, garbage=True):
    """q, a cache whose every row is written, a shuffled table.  Pages no table names are NaN."""
    g = torch.Generator().manual_seed(seed)
    pages = B * cols + 2
    table = torch.randperm(pages, generator=g)[:B * cols].reshape(B, cols).to(torch.int32)
    q = (torch.randn(B, H, T, d, generator=g) * mult).to(torch.bfloat16)
    cache = fa.new_cache(pages, Hk, page, d, E4M3 if fp8 else torch.bfloat16)
    if garbage:
        for t in cache:
            if t is not None:
                t.view(torch.uint8).fill_(0x7f if t.dtype == E4M3 else 0xff)
    return q, cache, table, g


def put(fa, cache, table, lens, g, mult=1.0):
    """Random rows for every sequence; rows behind lens keep the garbage."""
    pages, Hk, page, d = cache.k.shape
    B, cols = table.shape
    k, v = ((torch.randn(B, Hk, cols * page, d, generator=g) * mult).to(torch.bfloat16).to(DEV) for _ in range(2))
    full = torch.tensor([min(max(int(n), 0), cols * page) for n in lens], dtype=torch.int32, device=DEV)
    fa.cache_write(cache, k, v, table.to(DEV), full, full)


def compare(got_o, got_l, q, cache, table, lens, n_new, bits, scale):
    kv, vv = cache_values(cache)
    o, lse, mag, dot = orc.tree_attention(q, kv, vv, table, lens, n_new, bits, scale)
    d = q.shape[-1]
    e = 2 * d * 2.0 ** -24 * dot
    go, gl = got_o.cpu().double(), got_l.cpu().double()
    assert torch.equal(torch.isneginf(gl), torch.isneginf(lse))
    seen = ~torch.isneginf(lse)
    assert (go[~seen] == 0).all()
    assert torch.equal(go.isnan(), o.isnan())
    fine = seen & ~o.isnan().any(-1)
    tol = 2.0 ** -8 * o.abs() + (2.0 ** -7 + 2 * e[..., None] + 2.0 ** -14) * mag + 1e-30
    ratio = ((go - o).abs() / tol)[fine]
    assert ratio.numel() == 0 or float(ratio.max()) <= 1.0, f"O: {float(ratio.max()):.3f} of the bound"
    tol_l = e + 2.0 ** -18 * (1 + lse.abs())
    ratio = ((gl - lse).abs() / tol_l)[fine]
    assert ratio.numel() == 0 or float(ratio.max()) <= 1.0, f"L: {float(ratio.max()):.3f} of the bound"


CASES = [
    # B, H, Hk, T, d, page, cols, lens, n_new, tree, fp8, mult
    (1, 1, 1, 1, 128, 16, 1, [1], None, False, False, 1.0),
    (1, 4, 1, 1, 64, 16, 9, [129], None, False, False, 1.0),
    (2, 8, 2, 1, 128, 64, 5, [257, 320], None, False, True, 1.0),
    (3, 6, 2, 3, 32, 32, 8, [3, 128, 250], [3, 2, 0], True, False, 1.0),
    (3, 6, 2, 3, 32, 32, 8, [3, 128, 250], [3, 2, 0], True, True, 1.0),
    (2, 4, 4, 24, 64, 16, 24, [24, 383], [24, 17], True, False, 3.0),
    (2, 8, 1, 12, 128, 128, 4, [500, 140], None, True, True, 2.0),
    (1, 8, 1, 17, 128, 16, 20, [300], None, True, False, 1.0),          # 136 rows: more than one row tile
    (2, 12, 4, 65, 64, 32, 7, [224, 65], [65, 64], True, True, 1.0),    # two words a row
    (1, 2, 1, 130, 32, 64, 5, [310], None, False, False, 1.0),          # a chunk: tokens see 0 .. t
    (4, 2, 2, 5, 128, 256, 2, [0, -5, 3, 700], [5, 5, 5, 5], True, False, 1.0),  # none, negative, too short, too long
    (4, 2, 2, 5, 64, 16, 3, [0, 2, 48, 48], [5, 5, 9, -1], False, True, 1.0),
    (9, 3, 3, 1, 64, 16, 17, [1, 16, 17, 128, 129, 127, 255, 256, 257], None, False, False, 1.0),
    (1, 32, 8, 1, 128, 16, 150, [2391], None, False, False, 1.0),
    (1, 8, 8, 2, 128, 128, 21, [2600], None, True, True, 4.0),
]


@pytest.mark.parametrize("B, H, Hk, T, d, page, cols, lens, n_new, tree, fp8, mult", CASES)
def test_against_the_oracle(fa_lib, B, H, Hk, T, d, page, cols, lens, n_new, tree, fp8, mult):
    fa = fa_lib
    q, cache, table, g = make(fa, B, H, Hk, T, d, page, cols, fp8, T * 31 + d + sum(lens), mult)
    put(fa, cache, table, lens, g)
    lens = torch.tensor(lens, dtype=torch.int32)
    n_new = None if n_new is None else torch.tensor(n_new, dtype=torch.int32)
    words, bits = random_tree(B, T, g) if tree else (None, None)
    args = (q.to(DEV), cache, table.to(DEV), lens.to(DEV), None if words is None else words.to(DEV),
            None if n_new is None else n_new.to(DEV))
    o, lse = fa.attention_tree(*args)
    compare(o, lse, q, cache, table, lens, n_new, bits, 1 / math.sqrt(d))
    again = fa.attention_tree(*args)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    st, _ = fa.fa_poll_device_error(torch.cuda.current_stream().cuda_stream)
    assert st == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_any_mask_words(fa_lib, fp8, d):
    """Words that are no tree: rows that see nothing of the drafts, rows that see only later ones, bits past T."""
    fa = fa_lib
    B, H, Hk, T, page, cols = 2, 4, 2, 7, 16, 10
    q, cache, table, g = make(fa, B, H, Hk, T, d, page, cols, fp8, 77 + d)
    lens = torch.tensor([7, 150], dtype=torch.int32)  # no prefix at all; a prefix
    put(fa, cache, table, lens, g)
    rows = [[0, 0b1000000, 0b1111111, 0b0010010, -1, 1 << 5, 0], [0b11, 0, -1, 0b1010101, 1, 0b1000000, -128]]
    words = torch.tensor(rows, dtype=torch.int64)[..., None]
    bits = [[w % 2 ** 64 for w in r] for r in rows]
    o, lse = fa.attention_tree(q.to(DEV), cache, table.to(DEV), lens.to(DEV), words.to(DEV))
    compare(o, lse, q, cache, table, lens, None, bits, 1 / math.sqrt(d))
    one, lone = fa.attention_tree(q.to(DEV), cache, table.to(DEV), lens.to(DEV), words[1].to(DEV))  # one for all
    compare(one, lone, q, cache, table, lens, None, [bits[1], bits[1]], 1 / math.sqrt(d))


@pytest.mark.parametrize("fp8", [False, True])
def test_pages_that_are_not_there(fa_lib, fp8):
    """Entries outside the cache hide their keys, wherever they lie, and every key of a sequence may be hidden."""
    fa = fa_lib
    B, H, Hk, T, d, page, cols = 4, 4, 2, 3, 64, 16, 12
    q, cache, table, g = make(fa, B, H, Hk, T, d, page, cols, fp8, 5)
    lens = torch.tensor([180, 192, 40, 100], dtype=torch.int32)
    put(fa, cache, table, lens, g)
    table[0, 0] = table[0, 5] = -1
    table[1, 11] = 2147483647
    table[2, :] = -2147483648
    table[3, 0:6] = cache.k.shape[0]
    o, lse = fa.attention_tree(q.to(DEV), cache, table.to(DEV), lens.to(DEV))
    compare(o, lse, q, cache, table, lens, None, None, 1 / math.sqrt(d))
    assert torch.isneginf(lse[2]).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
def test_values_that_are_not_seen_do_not_reach_a_row(fa_lib, fp8, what):
    """A drafted token whose key and value are infinite or NaN changes only the rows that see it."""
    fa = fa_lib
    B, H, Hk, T, d, page, cols = 1, 4, 2, 6, 64, 16, 10
    q, cache, table, g = make(fa, B, H, Hk, T, d, page, cols, fp8, 11)
    lens = torch.tensor([131], dtype=torch.int32)  # the drafts lie across two key tiles
    put(fa, cache, table, lens, g)
    words = fa.tree_words([-1, 0, 0, 1, 2, -1])
    args = (table.to(DEV), lens.to(DEV), words.to(DEV))
    clean, clean_l = fa.attention_tree(q.to(DEV), cache, *args)
    for bad in (1, 5):  # rows 1 and 3 see token 1; only row 5 sees token 5
        k, v = (torch.randn(1, Hk, T, d, generator=g).to(torch.bfloat16) for _ in range(2))
        old_k, old_v = (x[:, :, 125:131] for x in fa.cache_read(cache, table.to(DEV), lens.to(DEV), 131))
        k, v = old_k.clone(), old_v.clone()
        k[0, :, bad, 3], v[0, :, bad, 7] = what, what
        fa.cache_write(cache, k, v, table.to(DEV), lens.to(DEV))
        o, lse = fa.attention_tree(q.to(DEV), cache, *args)
        for t in range(T):
            if (words[t, 0] >> bad) & 1:
                assert o[0, :, t].isnan().any() or o[0, :, t].isinf().any()
            else:
                assert torch.equal(o[0, :, t], clean[0, :, t]) and torch.equal(lse[0, :, t], clean_l[0, :, t])
        fa.cache_write(cache, old_k.contiguous(), old_v.contiguous(), table.to(DEV), lens.to(DEV))
    o, lse = fa.attention_tree(q.to(DEV), cache, *args)
    assert torch.equal(o, clean) and torch.equal(lse, clean_l)


def test_an_infinite_value_alone(fa_lib):
    """Only the value's one element is infinite: the rows that see it are infinite there and right elsewhere."""
    fa = fa_lib
    q, cache, table, g = make(fa, 1, 2, 1, 4, 64, 16, 3, False, 12)
    lens = torch.tensor([40], dtype=torch.int32)
    put(fa, cache, table, lens, g)
    args = (table.to(DEV), lens.to(DEV), fa.tree_words([-1, 0, -1, 2]).to(DEV))
    clean, clean_l = fa.attention_tree(q.to(DEV), cache, *args)
    page, slot = int(table[0, 37 // 16]), 37 % 16  # draft token 1
    cache.v[page, 0, slot, 9] = math.inf
    o, lse = fa.attention_tree(q.to(DEV), cache, *args)
    assert (o[0, :, 1, 9] == math.inf).all()
    o[0, :, 1, 9] = clean[0, :, 1, 9]
    # element 9 of row 1 apart, the same numbers
    assert torch.equal(o, clean) and torch.equal(lse, clean_l)


def test_large_scores_and_a_long_ragged_batch(fa_lib):
    """Scores of a standard deviation near 30 over lengths from 1 to 5000, against fp64 on the GPU."""
    fa = fa_lib
    B, H, Hk, d, page, cols = 24, 8, 2, 128, 64, 79
    q, cache, table, g = make(fa, B, H, Hk, 1, d, page, cols, False, 13, mult=30.0)
    lens = torch.tensor([1 + (b * b * 9) % 5000 for b in range(B)], dtype=torch.int32)
    lens[3], lens[7] = 5000, 5056
    put(fa, cache, table, lens, g)
    o, lse = fa.attention_tree(q.to(DEV), cache, table.to(DEV), lens.to(DEV))
    k, v = fa.cache_read(cache, table.to(DEV), lens.to(DEV), cols * page)
    for b in range(B):
        n = int(lens[b])
        for h in range(H):
            kk, vv = k[b, h // 4, :n].double(), v[b, h // 4, :n].double()
            prod = q[b, h, 0].to(DEV).double() * kk
            s = prod.sum(-1) / math.sqrt(d)
            e = 2 * d * 2.0 ** -24 * float(prod.abs().sum(-1).max()) / math.sqrt(d)
            w = torch.softmax(s, 0)
            ref, mag = w @ vv, w @ vv.abs()
            tol = 2.0 ** -8 * ref.abs() + (2.0 ** -7 + 2 * e + 2.0 ** -14) * mag
            assert ((o[b, h, 0].double() - ref).abs() <= tol).all(), (b, h)
            L = float(torch.logsumexp(s, 0))
            assert abs(float(lse[b, h, 0]) - L) <= e + 2.0 ** -18 * (1 + abs(L))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d, G, T", [(128, 4, 1), (128, 5, 12), (128, 4, 63), (64, 1, 24), (64, 8, 9), (32, 3, 33)])
def test_long_caches_again_and_again(fa_lib, fp8, d, G, T):
    """Sequences long enough to run every ring round many times, each call the same bits, and right against fp64."""
    fa = fa_lib
    B, Hk, page, cols = 3, 8, 64, 150
    q, cache, table, g = make(fa, B, Hk * G, Hk, T, d, page, cols, fp8, 16 + d + T)
    lens = torch.tensor([9600, 5001, 7300], dtype=torch.int32)
    put(fa, cache, table, lens, g)
    words, bits = random_tree(B, T, g)
    args = (q.to(DEV), cache, table.to(DEV), lens.to(DEV), words.to(DEV))
    o, lse = fa.attention_tree(*args)
    for _ in range(30):
        again = fa.attention_tree(*args)
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    k, v = fa.cache_read(cache, table.to(DEV), lens.to(DEV), cols * page)
    for b in range(B):
        n = int(lens[b])
        see = torch.ones(T, n, dtype=torch.bool)
        see[:, n - T:] = torch.tensor([[bool(bits[b][t] >> j & 1) for j in range(T)] for t in range(T)])
        see = see.to(DEV).repeat(G, 1)
        for hk in range(Hk):
            kk, vv = k[b, hk, :n].double(), v[b, hk, :n].double()
            rows = args[0][b, hk * G:(hk + 1) * G].reshape(G * T, d).double()
            s = (rows @ kk.T / math.sqrt(d)).masked_fill(~see, -math.inf)
            e = 2 * d * 2.0 ** -24 * (rows.abs() @ kk.abs().T).amax(-1, keepdim=True) / math.sqrt(d)
            w = torch.softmax(s, -1)
            ref, mag = w @ vv, w @ vv.abs()
            got = o[b, hk * G:(hk + 1) * G].reshape(G * T, d).double()
            assert ((got - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -7 + 2 * e + 2.0 ** -14) * mag).all(), (b, hk)
            L = torch.logsumexp(s, -1)
            assert ((lse[b, hk * G:(hk + 1) * G].reshape(-1).double() - L).abs() <= e[:, 0] + 2.0 ** -18 * (1 + L.abs())).all()


def test_guard_bands_and_a_dirty_workspace(fa_lib):
    fa = fa_lib
    B, H, Hk, T, d, page, cols = 3, 4, 2, 5, 64, 16, 30
    q, cache, table, g = make(fa, B, H, Hk, T, d, page, cols, False, 14)
    lens = torch.tensor([480, 5, 300], dtype=torch.int32)
    put(fa, cache, table, lens, g)
    ref_o, ref_l = fa.attention_tree(q.to(DEV), cache, table.to(DEV), lens.to(DEV))
    n_ws = fa.fa_fwd_tree_workspace_size(B, H, Hk, T, d)
    sizes = [q.numel() * 2, B * H * T * 4, n_ws]
    bufs = [torch.full((n + 512,), 0xA5, dtype=torch.uint8, device=DEV) for n in sizes]
    bufs[2][256:256 + n_ws] = 0xFF
    qd, td, ld = q.to(DEV), table.to(DEV), lens.to(DEV)
    c = fa.fa_cache(cache.k.data_ptr(), cache.v.data_ptr(), None, None, fa.FA_CACHE_BF16, *cache.k.shape)
    for _ in range(2):  # the second call on what the first left
        st = fa.fa_fwd_tree(qd.data_ptr(), c, bufs[0].data_ptr() + 256, bufs[1].data_ptr() + 256, B, H, T, td.data_ptr(),
                            cols, cols, ld.data_ptr(), None, None, 0, 1 / math.sqrt(d), bufs[2].data_ptr() + 256, n_ws,
                            torch.cuda.current_stream().cuda_stream)
        assert st == 0
        for b in bufs:
            assert (b[:256] == 0xA5).all() and (b[-256:] == 0xA5).all()
        assert torch.equal(bufs[0][256:-256].view(torch.bfloat16).view(ref_o.shape), ref_o)
        assert torch.equal(bufs[1][256:-256].view(torch.float32).view(ref_l.shape), ref_l)


def test_two_streams_and_a_captured_call(fa_lib):
    """Calls on two streams at once with a workspace each; a captured call sees the lengths of the moment."""
    fa = fa_lib
    B, H, Hk, T, d, page, cols = 4, 8, 2, 2, 128, 64, 16
    q, cache, table, g = make(fa, B, H, Hk, T, d, page, cols, True, 15)
    put(fa, cache, table, [1024] * B, g)
    qd, td = q.to(DEV), table.to(DEV)
    lens = [torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([1024, 3, 700, 129], [50, 1000, 2, 640])]
    want = [fa.attention_tree(qd, cache, td, n) for n in lens]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = fa.attention_tree(qd, cache, td, lens[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(got[i][0], want[i][0]) and torch.equal(got[i][1], want[i][1])
    n = lens[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fa.attention_tree(qd, cache, td, n)
    for i in (0, 1, 0):
        n.copy_(lens[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[i][0]) and torch.equal(out[1], want[i][1])


def test_refusals_of_the_helper(fa_lib):
    fa = fa_lib
    q = torch.zeros(2, 4, 3, 64, dtype=torch.bfloat16, device=DEV)
    c = fa.new_cache(4, 2, 16, 64)
    t, n = torch.zeros(2, 1, dtype=torch.int32, device=DEV), torch.ones(2, dtype=torch.int32, device=DEV)
    for bad in (
        lambda: fa.attention_tree(q.transpose(1, 2), c, t, n), lambda: fa.attention_tree(q[:, :3], c, t, n),
        lambda: fa.attention_tree(q[:, :3].contiguous(), c, t, n), lambda: fa.attention_tree(q[:1], c, t, n),
        lambda: fa.attention_tree(q, c, t, n, torch.zeros(2, 3, 2, dtype=torch.int64, device=DEV)),
        lambda: fa.attention_tree(q, c, t, n, torch.zeros(2, 3, 1, dtype=torch.int32, device=DEV)),
        lambda: fa.attention_tree(q, c, t, n, torch.zeros(3, 1, dtype=torch.int64)),
        lambda: fa.attention_tree(q.half(), c, t, n), lambda: fa.attention_tree(q[..., :32].contiguous(), c, t, n),
    ):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(fa.FAError):
        fa.attention_tree(q, c, t, n, scale=-1.0)


@pytest.mark.parametrize("fp8", [False, True])
def test_pages_past_32_bit_offsets(fa_lib, fp8):
    """A cache of more than 2^32 bytes and elements: rows written, read and attended to at its far end."""
    fa = fa_lib
    Hk, page, d = 4, 128, 128
    pages = 2 ** 32 // (Hk * page * d) + 40
    cache = fa.new_cache(pages, Hk, page, d, E4M3 if fp8 else torch.bfloat16)
    assert cache.k.numel() > 2 ** 32
    g = torch.Generator().manual_seed(31)
    table = torch.tensor([[pages - 1, 3, pages - 2], [pages // 2 + 1, pages - 7, 0]], dtype=torch.int32)
    lens = torch.tensor([300, 384], dtype=torch.int32)
    k, v = (torch.randn(2, Hk, 384, d, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    k, v = k[:, :, :300].contiguous(), v[:, :, :300].contiguous()
    fa.cache_write(cache, k, v, table.to(DEV), torch.tensor([300, 384], dtype=torch.int32, device=DEV))
    rk, rv = fa.cache_read(cache, table.to(DEV), lens.to(DEV), 384)
    if not fp8:
        assert torch.equal(rk[0, :, :300], k[0]) and torch.equal(rv[1, :, 84:], v[1])
    assert not rk[0, :, 300:].any() and not rv[1, :, :84].any()
    q = torch.randn(2, 8, 2, d, generator=g).to(torch.bfloat16).to(DEV)
    o, lse = fa.attention_tree(q, cache, table.to(DEV), lens.to(DEV))
    for b in range(2):
        n = int(lens[b])
        for h in range(8):
            for t in range(2):
                see = slice(0, n - 1 + t)
                kk, vv = rk[b, h // 2, see].double(), rv[b, h // 2, see].double()
                prod = q[b, h, t].double() * kk
                s = prod.sum(-1) / math.sqrt(d)
                e = 2 * d * 2.0 ** -24 * float(prod.abs().sum(-1).max()) / math.sqrt(d)
                w = torch.softmax(s, 0)
                ref, mag = w @ vv, w @ vv.abs()
                assert ((o[b, h, t].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -7 + 2 * e + 2.0 ** -14) * mag).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_many_sequences_of_few_keys(fa_lib, fp8):
    """More sequences than a warp has lanes, many more units than CTAs, lengths 0 to 40, against the oracle at some."""
    fa = fa_lib
    B, H, Hk, d, page, cols = 700, 4, 2, 64, 16, 3
    q, cache, table, g = make(fa, B, H, Hk, 1, d, page, cols, fp8, 41)
    lens = torch.randint(0, 41, (B,), generator=g, dtype=torch.int32)
    put(fa, cache, table, lens, g)
    o, lse = fa.attention_tree(q.to(DEV), cache, table.to(DEV), lens.to(DEV))
    assert torch.equal(torch.isneginf(lse).all(-1).all(-1).cpu(), lens == 0)
    some = torch.arange(0, B, 9)
    compare(o[some], lse[some], q[some], cache, table[some], lens[some], None, None, 1 / math.sqrt(d))


def test_a_long_chunk_over_the_cache(fa_lib):
    """300 new tokens for each of 4 heads of a key head (10 row tiles): the causal attention of the same tensors."""
    fa = fa_lib
    B, H, Hk, T, d, page, cols = 1, 4, 1, 300, 128, 64, 16
    q, cache, table, g = make(fa, B, H, Hk, T, d, page, cols, False, 51)
    lens = torch.tensor([900], dtype=torch.int32)
    put(fa, cache, table, lens, g)
    o, lse = fa.attention_tree(q.to(DEV), cache, table.to(DEV), lens.to(DEV))
    k, v = fa.cache_read(cache, table.to(DEV), lens.to(DEV), 900)
    ro, rl = fa.attention_forward(q.to(DEV), k.expand(B, H, 900, d).contiguous(), v.expand(B, H, 900, d).contiguous(), True)
    # both round their weights and results to bf16 against the same exact value: twice the bound above, |v| < 5
    assert (o.float() - ro.float()).abs().max() <= 2 * (2.0 ** -8 + 2.0 ** -7 + 2.0 ** -13) * 5
    assert (lse - rl).abs().max() <= 2.0 ** -14


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_never_written(fa_lib, fp8):
    """A fresh cache reads as zeros: every key weighs the same and every value is zero."""
    fa = fa_lib
    cache = fa.new_cache(4, 2, 64, 128, E4M3 if fp8 else torch.bfloat16)
    table = torch.arange(4, dtype=torch.int32, device=DEV).view(2, 2)
    n = torch.tensor([128, 77], dtype=torch.int32, device=DEV)
    q = torch.randn(2, 4, 1, 128, device=DEV).to(torch.bfloat16)
    o, lse = fa.attention_tree(q, cache, table, n)
    assert not o.any()
    assert (lse - n.float().log()[:, None, None]).abs().max() <= 2.0 ** -18 * 6


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("G, T", [(1, 1), (8, 6), (8, 11)])
def test_values_of_very_different_scales(fa_lib, fp8, G, T):
    """Keys and values whose rows differ by up to 2^120 in size, zeros among them; query rows too."""
    fa = fa_lib
    B, Hk, d, page, cols = 2, 2, 64, 16, 40
    q, cache, table, g = make(fa, B, Hk * G, Hk, T, d, page, cols, fp8, 61 + T)
    lens = torch.tensor([640, 333], dtype=torch.int32)
    n = cols * page
    k = torch.randn(B, Hk, n, d, generator=g)
    v = torch.randn(B, Hk, n, d, generator=g) * 2.0 ** torch.randint(-60, 61, (B, Hk, n, 1), generator=g)
    v[:, :, ::7] = 0
    k = k * 2.0 ** torch.randint(-20, 1, (B, Hk, n, 1), generator=g)
    q = (q.float() * 2.0 ** torch.randint(-12, 3, (B, Hk * G, T, 1), generator=g)).to(torch.bfloat16)
    full = torch.full((B,), n, dtype=torch.int32, device=DEV)
    fa.cache_write(cache, k.to(torch.bfloat16).to(DEV), v.to(torch.bfloat16).to(DEV), table.to(DEV), full)
    o, lse = fa.attention_tree(q.to(DEV), cache, table.to(DEV), lens.to(DEV))
    compare(o, lse, q, cache, table, lens, None, None, 1 / math.sqrt(d))


def test_no_pages_and_no_columns(fa_lib):
    fa = fa_lib
    q = torch.randn(2, 4, 3, 64, device=DEV).to(torch.bfloat16)
    n = torch.tensor([5, 0], dtype=torch.int32, device=DEV)
    x = torch.randn(2, 2, 3, 64, device=DEV).to(torch.bfloat16)
    for cache, table in ((fa.new_cache(0, 2, 16, 64), torch.zeros(2, 3, dtype=torch.int32, device=DEV)),
                         (fa.new_cache(4, 2, 16, 64), torch.zeros(2, 0, dtype=torch.int32, device=DEV))):
        fa.cache_write(cache, x, x, table, n)
        o, lse = fa.attention_tree(q, cache, table, n)
        assert not o.any() and torch.isneginf(lse).all()
        k, v = fa.cache_read(cache, table, n, 7)
        assert k.shape == (2, 2, 7, 64) and not k.any() and not v.any()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("G, T", [(8, 5), (8, 9), (8, 17), (4, 63)])  # 40, 72, 136 and 252 rows on a key head
def test_many_units_on_a_cta(fa_lib, G, T, d, fp8):
    """Each CTA goes through five units of one to three tiles or more, row tiles with and without rows for all of its
    warps in turn: every barrier of a unit comes back to each of its phases.  Each call gives the same bits."""
    fa = fa_lib
    tiles = (G * T + 127) // 128
    Hk, page, cols = 2 // tiles, 128, 3
    B = 420
    assert B * Hk * tiles >= 5 * 152
    q, cache, table, g = make(fa, B, Hk * G, Hk, T, d, page, cols, fp8, 71 + d + T)
    lens = torch.randint(0, 301, (B,), generator=g, dtype=torch.int32)
    lens[::2] = lens[::2] % 129
    n_new = torch.randint(0, T + 1, (B,), generator=g, dtype=torch.int32)
    n_new[::3] = T
    put(fa, cache, table, lens, g)
    words, bits = random_tree(B, T, g)
    args = (q.to(DEV), cache, table.to(DEV), lens.to(DEV), words.to(DEV), n_new.to(DEV))
    o, lse = fa.attention_tree(*args)
    st, site = fa.fa_poll_device_error(torch.cuda.current_stream().cuda_stream)
    assert st == 0, hex(site)
    for _ in range(20):
        again = fa.attention_tree(*args)
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    some = torch.arange(0, B, 37)
    compare(o[some], lse[some], q[some], cache, table[some], lens[some], n_new[some], [bits[b] for b in some],
            1 / math.sqrt(d))


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("G, T", [(4, 1), (8, 5), (8, 9), (4, 63)])
def test_short_e4m3_sequences_hundreds_of_times(fa_lib, G, T, d):
    """Many short units over pages that are NaN behind their sequence's end: a tile that is overwritten before all of it
    has been read shows as NaN rows or other bits in some call."""
    fa = fa_lib
    tiles = (G * T + 127) // 128
    B, Hk, page, cols = 420, 2 // tiles, 128, 3
    q, cache, table, g = make(fa, B, Hk * G, Hk, T, d, page, cols, True, 91 + d + T)
    lens = torch.randint(0, 301, (B,), generator=g, dtype=torch.int32)
    lens[::2] = lens[::2] % 129
    put(fa, cache, table, lens, g)
    args = (q.to(DEV), cache, table.to(DEV), lens.to(DEV))
    o, lse = fa.attention_tree(*args)
    assert not o.isnan().any() and not lse.isnan().any()
    differ = torch.zeros((), dtype=torch.int64, device=DEV)
    for _ in range(500):
        again = fa.attention_tree(*args)
        differ += (o != again[0]).any().long() + (lse != again[1]).any()
    assert int(differ) == 0
    some = torch.arange(0, B, 53)
    compare(o[some], lse[some], q[some], cache, table[some], lens[some], None, None, 1 / math.sqrt(d))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("G, T", [(1, 1), (4, 1), (33, 1), (66, 1), (2, 3), (8, 5), (8, 9)])
def test_infinite_values_that_are_seen(fa_lib, G, T, d, fp8):
    """Infinite values of the prefix, of a single token itself and of drafted tokens, in units of one CTA and of several:
    infinite of that sign in the rows that see them, NaN where both signs or a NaN meet, and right everywhere else.  (An
    e4m3 row that holds one is NaN.)"""
    fa = fa_lib
    B, Hk, page, cols = 4, 2, 32, 80
    q, cache, table, g = make(fa, B, Hk * G, Hk, T, d, page, cols, fp8, 81 + d + T + G)
    lens = torch.tensor([2500, T, 300, 140], dtype=torch.int32)
    n_new = torch.tensor([T, T, (T + 1) // 2, T], dtype=torch.int32)
    n = cols * page
    k, v = (torch.randn(B, Hk, n, d, generator=g).to(torch.bfloat16) for _ in range(2))
    inf = math.inf
    v[0, 0, 5, 3], v[0, 0, 1700, 4], v[0, 0, 130, d - 1] = inf, -inf, inf
    v[0, 0, 900, 9], v[0, 0, 2000, 9], v[0, 0, 2499 - T, 11] = inf, -inf, math.nan
    v[0, 1, 77, 1] = -inf
    v[1, 0, 0, 7] = inf                       # the only key, or the first draft
    v[2, 1, 300 - int(n_new[2]), 6] = -inf    # a token's own value, every live row sees it
    v[2, 1, 3, 6], v[2, 1, 4, 8] = inf, inf   # the other sign in the prefix
    v[3, 0, 139, 2], v[3, 1, 139, 2], v[3, 1, 0, 2] = inf, -inf, -inf  # seen by the last draft alone; and a prefix's
    full = torch.full((B,), n, dtype=torch.int32, device=DEV)
    fa.cache_write(cache, k.to(DEV), v.to(DEV), table.to(DEV), full)
    words, bits = random_tree(B, T, g) if T > 1 and d != 32 else (None, None)
    args = (q.to(DEV), cache, table.to(DEV), lens.to(DEV), None if words is None else words.to(DEV), n_new.to(DEV))
    o, lse = fa.attention_tree(*args)
    kv, vv = cache_values(cache)
    want, want_l, _, dot = orc.tree_attention(q, kv, vv, table, lens, n_new, bits, 1 / math.sqrt(d))
    got = o.cpu().double()
    for kind in (torch.isposinf, torch.isneginf, torch.isnan):
        assert torch.equal(kind(got), kind(want)), kind.__name__
    # elsewhere the bound of the file's head, with the magnitudes of the finite values
    vf = torch.where(torch.isfinite(vv), vv, 0.0)
    _, _, mag, _ = orc.tree_attention(q, kv, vf, table, lens, n_new, bits, 1 / math.sqrt(d))
    e = 2 * d * 2.0 ** -24 * dot
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -7 + 2 * e[..., None] + 2.0 ** -14) * mag + 1e-30
    fine = torch.isfinite(want)
    assert ((got - want).abs() <= tol)[fine].all()
    live = ~torch.isneginf(want_l) & ~torch.isnan(want_l)
    assert ((lse.cpu().double() - want_l).abs() <= e + 2.0 ** -18 * (1 + want_l.abs()))[live].all()
    again = fa.attention_tree(*args)
    assert torch.equal(o.nan_to_num(), again[0].nan_to_num()) and torch.equal(lse.nan_to_num(), again[1].nan_to_num())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G, T", [(2, 1), (8, 5), (8, 9)])
def test_scales_that_change_along_the_sequence(fa_lib, G, T, d):
    """e4m3 values of size zero first, then of 2^40, 2^-90 and 1, in stretches of 32 keys, of tiles and of many tiles: what
    the first ones add to the sum of weights counts however small their values are."""
    fa = fa_lib
    B, Hk, page, cols = 3, 2, 64, 45
    q, cache, table, g = make(fa, B, Hk * G, Hk, T, d, page, cols, True, 101 + d + T)
    lens = torch.tensor([128, 512 + T, 2800], dtype=torch.int32)  # groups of a tile; a CTA's tiles; several CTAs
    n = cols * page
    k = torch.randn(B, Hk, n, d, generator=g) * 0.25
    v = torch.randn(B, Hk, n, d, generator=g)
    for b, step in enumerate((32, 128, 700)):
        size = torch.tensor([0.0, 2.0 ** 40, 2.0 ** -90, 1.0])[torch.arange(n) // step % 4]
        v[b] *= size[:, None]
    full = torch.full((B,), n, dtype=torch.int32, device=DEV)
    fa.cache_write(cache, k.to(torch.bfloat16).to(DEV), v.to(torch.bfloat16).to(DEV), table.to(DEV), full)
    o, lse = fa.attention_tree(q.to(DEV), cache, table.to(DEV), lens.to(DEV))
    compare(o, lse, q, cache, table, lens, None, None, 1 / math.sqrt(d))


@pytest.mark.parametrize("G", [1, 40, 66])
def test_sums_of_many_weights_stay_finite(fa_lib, G):
    """65536 keys with values of zero (the least exponent), of which the first 128 score 0 and all others 6.5: their sum
    of weights is a long way above the first ones'.  As many sequences as SMs, so that a CTA has one to itself."""
    fa = fa_lib
    d, page, n, B = 64, 1024, 65536, 152
    cache = fa.new_cache(n // page, 1, page, d, E4M3)
    table = torch.arange(n // page, dtype=torch.int32, device=DEV)[None].expand(B, -1)
    k = torch.full((1, 1, n, d), 0.8125, dtype=torch.bfloat16, device=DEV)
    k[:, :, :128] = 0
    lens = torch.full((B,), n, dtype=torch.int32, device=DEV)
    fa.cache_write(cache, k, torch.zeros_like(k), table[:1], lens[:1])
    o, lse = fa.attention_tree(torch.ones(B, G, 1, d, dtype=torch.bfloat16, device=DEV), cache, table, lens)
    want = math.log(128 + (n - 128) * math.exp(6.5))
    assert not o.any()
    # exact scores; the sum and its logarithm as in the file's head
    assert (lse.double() - want).abs().max() <= 2.0 ** -18 * (1 + want)


def test_refused_sizes_carry_the_entry_points_status(fa_lib):
    """What fa_fwd_tree calls unsupported is unsupported from Python too."""
    fa = fa_lib
    t, n = torch.zeros(2, 1, dtype=torch.int32, device=DEV), torch.ones(2, dtype=torch.int32, device=DEV)

    def call(H, d, page=16):
        q = torch.zeros(2, H, 1, d, dtype=torch.bfloat16, device=DEV)
        return fa.attention_tree(q, fa.new_cache(1, 2, page, d), t, n)
    for args in ((4, 48), (40000, 32), (4, 64, 24), (4, 96, 16)):
        with pytest.raises(fa.FAError) as e:
            call(*args)
        assert e.value.status == fa.FA_ERR_UNSUPPORTED, args
    call(4, 64)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H, Hk, T, d, n", [(4, 1, 300, 128, 900), (6, 2, 129, 64, 1500), (2, 2, 1000, 32, 1003)])
def test_a_chunk_over_the_cache_element_by_element(fa_lib, fp8, H, Hk, T, d, n):
    """Hundreds of new tokens on several row tiles against fp64, with the bound of the file's head."""
    fa = fa_lib
    page = 64
    cols = (n + page - 1) // page
    q, cache, table, g = make(fa, 1, H, Hk, T, d, page, cols, fp8, 111 + d)
    lens = torch.tensor([n], dtype=torch.int32)
    put(fa, cache, table, lens, g)
    o, lse = fa.attention_tree(q.to(DEV), cache, table.to(DEV), lens.to(DEV))
    k, v = (x[0].double() for x in fa.cache_read(cache, table.to(DEV), lens.to(DEV), n))
    at = torch.arange(n, device=DEV)[None]
    hidden = at > n - T + torch.arange(T, device=DEV)[:, None]
    for h in range(H):
        kk, vv = k[h // (H // Hk)], v[h // (H // Hk)]
        rows = q[0, h].to(DEV).double()
        s = (rows @ kk.T / math.sqrt(d)).masked_fill(hidden, -math.inf)
        e = 2 * d * 2.0 ** -24 * (rows.abs() @ kk.abs().T).amax(-1, keepdim=True) / math.sqrt(d)
        w = torch.softmax(s, -1)
        ref, mag = w @ vv, w @ vv.abs()
        assert ((o[0, h].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -7 + 2 * e + 2.0 ** -14) * mag).all(), h
        L = torch.logsumexp(s, -1)
        assert ((lse[0, h].double() - L).abs() <= e[:, 0] + 2.0 ** -18 * (1 + L.abs())).all(), h
