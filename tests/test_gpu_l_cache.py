"""The paged cache: written and read back, against the format's definition.  Nothing here is rounded twice, so every
comparison is exact."""
import math

import pytest
import torch

from oracle import operators as orc

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4M3 = torch.float8_e4m3fn


def page_table(B, cols, pages, g, holes=()):
    ids = torch.randperm(pages, generator=g)[:B * cols].reshape(B, cols).to(torch.int32)
    for b, c, value in holes:
        ids[b, c] = value
    return ids


def fill(cache, byte):
    for t in cache:
        if t is not None:
            t.view(torch.uint8).fill_(byte)


def layout(t, kind):
    """The values of t [B,H,T,d] on the GPU, contiguous or as the transposed view of [B,T,H,d]."""
    return t.to(DEV) if kind == "bhtd" else t.transpose(1, 2).contiguous().to(DEV).transpose(1, 2)


CASES = [
    # B, Hk, T, d, page, cols, lens, n_new, fp8, layout, holes
    (1, 1, 1, 128, 16, 2, [17], None, False, "bhtd", ()),
    (1, 1, 1, 32, 16, 1, [1], None, True, "bhtd", ()),
    (3, 2, 5, 64, 16, 4, [5, 33, 64], [5, 2, 0], True, "bthd", ()),
    (3, 3, 7, 128, 32, 3, [7, 96, 20], [3, 7, 6], False, "bthd", ((1, 2, -1),)),
    (2, 4, 70, 128, 64, 3, [70, 192], None, True, "bhtd", ((0, 1, 1 << 30),)),
    (4, 1, 9, 32, 128, 1, [0, 4, 200, -3], [9, 9, 4, 9], False, "bhtd", ()),  # too short, too long, negative
    (2, 8, 33, 64, 256, 1, [256, 40], [33, 31], True, "bthd", ()),
    (2, 2, 4, 128, 16, 5, [80, 81], [100, -7], True, "bhtd", ()),  # more new tokens than T, and a negative count
]


@pytest.mark.parametrize("B, Hk, T, d, page, cols, lens, n_new, fp8, kind, holes", CASES)
def test_write_and_read(fa_lib, B, Hk, T, d, page, cols, lens, n_new, fp8, kind, holes):
    fa = fa_lib
    g = torch.Generator().manual_seed(T * 100 + d + page)
    pages = B * cols + 2
    table = page_table(B, cols, pages, g, holes)
    lens = torch.tensor(lens, dtype=torch.int32)
    n_new = None if n_new is None else torch.tensor(n_new, dtype=torch.int32)
    k, v = (torch.randn(B, Hk, T, d, generator=g).to(torch.bfloat16) * 3 for _ in range(2))
    k[0, 0, 0] = 0
    v[-1, -1, -1, 0] = 3e38
    if T > 3:
        k[0, 0, 1, 3], v[0, 0, 2, 5] = math.inf, math.nan
        k[0, 0, 3] = 1e-38
    cache = fa.new_cache(pages, Hk, page, d, E4M3 if fp8 else torch.bfloat16)
    fill(cache, 0x35)
    before = [None if t is None else t.clone() for t in cache]
    on = table.to(DEV), lens.to(DEV)
    fa.cache_write(cache, layout(k, kind), layout(v, kind), *on, None if n_new is None else n_new.to(DEV))
    touched = torch.zeros(pages, page, dtype=torch.bool)
    for b in range(B):
        for t in range(T):
            at = orc.row_place(table, lens, n_new, T, page, pages, b, t)
            if at is None:
                continue
            touched[at] = True
            for h in range(Hk):
                for data, exps, x in ((cache.k, cache.k_exp, k), (cache.v, cache.v_exp, v)):
                    row = data[at[0], h, at[1]].cpu()
                    if not fp8:
                        assert torch.equal(row.view(torch.int16), x[b, h, t].view(torch.int16))
                        continue
                    want, byte = orc.e4m3_row(x[b, h, t])
                    assert int(exps[at[0], h, at[1]]) == byte
                    got = row.double() * (math.nan if byte == 255 else 2.0 ** (byte - 127))
                    assert torch.equal(got.nan_to_num(7.5), want.nan_to_num(7.5))
    # every other row is as it was
    for t, old in zip(cache, before):
        if t is not None:
            same = (t.view(torch.uint8) == old.view(torch.uint8)).reshape(pages, Hk, page, -1).all(-1).all(1).cpu()
            assert (same | touched).all()
    length = cols * page + 3
    ko, vo = (x.cpu() for x in fa.cache_read(cache, *on, length))
    for data, exps, out in ((cache.k, cache.k_exp, ko), (cache.v, cache.v_exp, vo)):
        vals = data.cpu().double()
        if fp8:
            e = exps.cpu().double()
            vals = vals * torch.where(e == 255, math.nan, 2.0 ** (e - 127))[..., None]
        for b in range(B):
            n = min(max(int(lens[b]), 0), cols * page)
            want = torch.zeros(Hk, length, d, dtype=torch.float64)
            rows, there = orc.sequence(vals, table, n, page, b)
            want[:, :n] = torch.where(there[None, :, None], rows, 0.0)
            assert torch.equal(out[b].double().nan_to_num(7.5), want.to(torch.bfloat16).double().nan_to_num(7.5))


def test_every_bf16_magnitude_quantises_as_defined(fa_lib):
    """Rows whose largest element runs over every exponent and the borders of its scale."""
    fa = fa_lib
    bits = torch.arange(0, 0x7f80, 7, dtype=torch.int32).to(torch.int16)
    top = bits.view(torch.bfloat16)
    T = len(top)
    g = torch.Generator().manual_seed(1)
    x = (torch.rand(1, 1, T, 32, generator=g) * 2 - 1).to(torch.bfloat16) * top[None, None, :, None]
    x[0, 0, :, 5] = -top
    cols = (T + 63) // 64
    cache = fa.new_cache(cols, 1, 64, 32, E4M3)
    table = torch.arange(cols, dtype=torch.int32, device=DEV)[None]
    lens = torch.tensor([T], dtype=torch.int32, device=DEV)
    fa.cache_write(cache, x.to(DEV), x.to(DEV), table, lens)
    k, v = fa.cache_read(cache, table, lens, T)
    assert torch.equal(k, v)
    for i in range(0, T, 3):
        want, byte = orc.e4m3_row(x[0, 0, i])
        assert int(cache.k_exp.view(-1)[i]) == byte
        assert torch.equal(k[0, 0, i].cpu().double(), want), i


def test_a_table_that_is_a_slice(fa_lib):
    """Rows of the table further apart than its columns."""
    fa = fa_lib
    wide = torch.full((2, 9), -1, dtype=torch.int32, device=DEV)
    wide[:, 3:5] = torch.tensor([[3, 1], [0, 2]], dtype=torch.int32)
    cache = fa.new_cache(4, 1, 16, 64)
    x = torch.randn(2, 1, 20, 64, device=DEV).to(torch.bfloat16)
    lens = torch.full((2,), 20, dtype=torch.int32, device=DEV)
    fa.cache_write(cache, x, x, wide[:, 3:5], lens)
    k, v = fa.cache_read(cache, wide[:, 3:5], lens, 20)
    assert torch.equal(k, x) and torch.equal(v, x)


def test_refusals_of_the_helpers(fa_lib):
    fa = fa_lib
    x = torch.zeros(2, 1, 3, 64, dtype=torch.bfloat16, device=DEV)
    c = fa.new_cache(4, 1, 16, 64)
    t, n = torch.zeros(2, 1, dtype=torch.int32, device=DEV), torch.ones(2, dtype=torch.int32, device=DEV)
    for bad in (
        lambda: fa.cache_write(c, x.float(), x, t, n), lambda: fa.cache_write(c, x, x[:, :, :2], t, n),
        lambda: fa.cache_write(c, x, x, t.long(), n), lambda: fa.cache_write(c, x, x, t, n.long()),
        lambda: fa.cache_write(c, x, x, t[:1], n), lambda: fa.cache_write(c, x, x, t, n, n[:1]),
        lambda: fa.cache_write(c, x[..., :32], x[..., :32], t, n), lambda: fa.cache_read(c, t.cpu(), n, 3),
        lambda: fa.cache_read(fa.KVCache(c.k, c.v, n, n), t, n, 3), lambda: fa.cache_read(c, t, n[:1], 3),
        lambda: fa.cache_read(fa.KVCache(c.k.view(torch.uint8).view(E4M3), c.v), t, n, 3),
        lambda: fa.cache_write(c, x.transpose(2, 3), x.transpose(2, 3), t, n),
    ):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(fa.FAError):
        fa.cache_read(fa.KVCache(c.k.view(4, 1, 8, 128), c.v.view(4, 1, 8, 128)), t, n, 3)  # pages of 8 rows
