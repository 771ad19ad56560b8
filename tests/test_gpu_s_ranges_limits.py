"""Attention over ranges of keys at the limits of what it takes: keys that are not finite in the gradients, no
query heads, scores far beyond the cap, masks far from their rows, many
values that are not finite, rows of very many keys, a device error pending.

Bounds as in test_gpu_o_ranges.py and oracle/ranges.py.
"""
import math

import pytest
import torch

from oracle import ranges as orc
from test_gpu_o_ranges import check, check_forward, close, rand, slopes_of
from test_gpu_q_ranges_edges import INF, NAN, clean_status, i32

pytestmark = pytest.mark.gpu
DEV = "cuda"


# ------------------------------------------------------------------ keys that are not finite, gradients

@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("value", [-INF, INF, NAN])
def test_gradients_of_a_key_that_is_not_finite(fa_lib, d, cap, value):
    """NaN for the key's gradients and dQ of the rows that see it; where L is finite (a score of -infinity, or a cap) all
    others are those of the scores as they are.  For these a finite element stands in that makes the same ones: -infinity
    by a weight below 2^-1074, the cap to 2 cap e^-20 (below 2^-27 of it)."""
    fa = fa_lib
    B, H, Hk, N = 1, 4, 2, 450
    g = torch.Generator().manual_seed(d)
    q, k, v, do = (rand(g, B, h, N, d) for h in (H, Hk, Hk, H))
    spots = [(0, 130, 3), (1, 200, d - 1), (1, 390, d // 2)]  # key head, key, element
    for _, _, e in spots:
        q[..., e] = 1.0
    q = q.contiguous()
    bad, stand_in = k.clone(), k.clone()
    size = (250.0 if cap else 1000.0) * math.sqrt(d)  # the score of such a pair but for the other elements' 15 or so
    for h, j, e in spots:
        bad[0, h, j, e] = value
        stand_in[0, h, j, e] = size if value == INF else -size
    m = fa.mask_ranges(B, N, causal=True, documents=i32([[0, 150, 450]]))
    sees = torch.zeros(H, N, dtype=torch.bool, device=DEV)
    for h, j, _ in spots:
        sees[2 * h:2 * h + 2, j:150 if j < 150 else N] = True
    o, lse = fa.attention_ranges(q, bad, v, m, softcap=cap)
    finite = value == -INF or (cap and value == INF)
    assert torch.equal(torch.isnan(lse[0]), torch.zeros_like(sees) if finite else sees)
    dq, dk, dv = fa.attention_ranges_backward(q, bad, v, o, lse, do, m, softcap=cap)
    assert torch.isnan(dq[0][sees]).all()
    for h, j, _ in spots:
        assert torch.isnan(dk[0, h, j]).all() and torch.isnan(dv[0, h, j]).all()
    refs = orc.backward(q, stand_in, v, do, m.first, m.last, d ** -0.5, cap)
    (ref, tol) = refs[0]
    close(dq[0][~sees], ref[0][~sees], tol[0][~sees], "dQ")
    if finite:
        others = torch.ones(Hk, N, dtype=torch.bool, device=DEV)
        for h, j, _ in spots:
            others[h, j] = False
        for got, (ref, tol), name in zip((dk, dv), refs[1:], ("dK", "dV")):
            close(got[0][others], ref[0][others], tol[0][others], name)
    for _ in range(20):
        _, dk2, dv2 = fa.attention_ranges_backward(q, bad, v, o, lse, do, m, softcap=cap)
        assert torch.equal(dk.isnan(), dk2.isnan()) and torch.equal(dk.nan_to_num(), dk2.nan_to_num())
        assert torch.equal(dv.isnan(), dv2.isnan()) and torch.equal(dv.nan_to_num(), dv2.nan_to_num())
    clean_status(fa)


# ------------------------------------------------------------------ no rows

@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("B,H,Hk,Nq,Nk", [(2, 0, 2, 5, 5), (2, 0, 2, 300, 1000), (1, 4, 2, 0, 129), (3, 0, 1, 0, 1)])
def test_no_query_rows_give_keys_no_gradients(fa_lib, B, H, Hk, Nq, Nk, d):
    fa = fa_lib
    q = torch.ones(B, H, Nq, d, dtype=torch.bfloat16, device=DEV)
    k, v = (torch.ones(B, Hk, Nk, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    lse = torch.zeros(B, H, Nq, device=DEV)
    m = fa.mask_ranges(B, Nq, Nk)
    ws = torch.empty(fa.fa_bwd_ranges_workspace_size(B, H, Hk, Nq, Nk, d), dtype=torch.uint8, device=DEV)
    dk, dv = (torch.full_like(k, 7.0) for _ in range(2))
    stream = torch.cuda.current_stream().cuda_stream
    status = fa.fa_bwd_ranges(0, k.data_ptr(), v.data_ptr(), 0, 0, 0, 0, dk.data_ptr(), dv.data_ptr(), None, None, None,
                              None, m.buffer.data_ptr(), m.buffer.nbytes, B, H, Hk, Nq, Nk, d, 0.0, None, 1.0,
                              ws.data_ptr(), ws.nbytes, stream)
    assert status == 0 and not dk.any() and not dv.any()
    dq, dk, dv = fa.attention_ranges_backward(q, k, v, q, lse, q, m)
    assert dq.shape == q.shape and not dk.any() and not dv.any()
    clean_status(fa)


@pytest.mark.parametrize("d,cap", [(128, 0.0), (128, 20.0), (64, 20.0), (32, 20.0)])
def test_zero_gradients_are_positive_zeros(fa_lib, d, cap):
    """Padding (rows without keys, keys that no row sees), in tiles with others and in tiles of its own."""
    fa = fa_lib
    g = torch.Generator().manual_seed(3)
    q, k, v, do = (rand(g, 2, h, 700, d) for h in (4, 2, 2, 4))
    m = fa.mask_ranges(2, 700, causal=True, documents=i32([[0, 700], [0, 300]]))
    o, lse = fa.attention_ranges(q, k, v, m, softcap=cap)
    for x in fa.attention_ranges_backward(q, k, v, o, lse, do, m, softcap=cap):
        assert not x[1, :, 300:].contiguous().view(torch.int16).any()


# ------------------------------------------------------------------ scores far beyond the cap

@pytest.mark.parametrize("d,bias", [(32, False), (64, True), (128, False)])
def test_large_scores_of_other_rows_do_not_show(fa_lib, d, bias):
    """Rows 0 .. 39 and 40 .. 299 are documents of their own, and some of the second have scores of hundreds of caps, or
    see a key that is not finite: the others' bits stay.  (Rows 32 .. 63 share a warp.)"""
    fa = fa_lib
    H, Hk, N = 4, 2, 300
    g = torch.Generator().manual_seed(17)
    q, k, v = rand(g, 1, H, N, d, mult=2.0), rand(g, 1, Hk, N, d), rand(g, 1, Hk, N, d)
    slopes = torch.rand(H, generator=g).to(DEV) * 0.01 if bias else None
    m = fa.mask_ranges(1, N, causal=True, documents=i32([[0, 40, 300]]))
    want, wl = fa.attention_ranges(q, k, v, m, softcap=0.5, slopes=slopes)
    big = q.clone()
    loud = torch.zeros(N, dtype=torch.bool, device=DEV)
    loud[41::3] = True
    big[:, :, loud] *= 512.0
    o, lse = fa.attention_ranges(big, k, v, m, softcap=0.5, slopes=slopes)
    assert torch.equal(o[:, :, ~loud], want[:, :, ~loud]) and torch.equal(lse[:, :, ~loud], wl[:, :, ~loud])
    bad = k.clone()
    bad[:, :, 60] = NAN
    o, lse = fa.attention_ranges(q, bad, v, m, softcap=0.5, slopes=slopes)
    assert torch.equal(o[:, :, :60], want[:, :, :60]) and torch.equal(lse[:, :, :60], wl[:, :, :60])
    clean_status(fa)


def capped_reference(q, k, v, do, m, scale, cap, slopes):
    """O, L, dQ, dK, dV in 64 bits, each with its bound.

    A score before the cap is off by its products' and sums' roundings, d 2^-24 of size = sum |q k| scale; after it by that
    times the derivative (times 1.25: it is up to a tenth of the cap here, and e^0.2 < 1.25), 2^-19 cap, and 2^-22 of the
    bias.  With 2^-18 of the exponentials this is eps.  The derivative 4 w (1 - w) is off by rr of it: twice the score's error
    over the cap, the rounding of 2 log2 e s / cap (4 2^-24 of it), 2^-19 of the exponential and the reciprocal.  A weight
    (times the derivative), dS, O and the results are rounded to bf16, 2^-8 each; sums of fp32 are off by 2^-14.  What is
    below 2^-126 on the way may become 0: less than 2^-100 in a result, whose other factors are below 2^10 in sums of 300."""
    H, Hk, d, N = q.shape[1], k.shape[1], q.shape[-1], q.shape[2]
    tiny = 2.0 ** -100
    s, _, size = orc._scores(q, k, m.first, m.last, scale, cap, slopes)
    raw = (q.double().view(*k.shape[:2], H // Hk, N, d) @ k.double()[:, :, None].transpose(-1, -2)).view_as(s) * scale
    u = torch.exp(-2 * raw.abs() / cap)
    rate = 4 * u / (1 + u) ** 2  # (1 - tanh^2 is 0 in 64 bits from 19 caps on)
    p, lse = orc._softmax(s)
    bias = 0.0 if slopes is None else float(slopes.abs().max()) * N
    eps = (d * 2.0 ** -24 * 1.25 * size * rate).amax(-1, keepdim=True) + 2.0 ** -19 * cap + 2.0 ** -22 * bias + 2.0 ** -18
    rr = 2 * (d + 4) * 2.0 ** -24 * size / cap + 2.0 ** -19
    qf, kf, vf, g = q.double(), orc._heads(k, H), orc._heads(v, H), do.double()
    o, mag = p @ vf, p @ vf.abs()
    off_o = 2.0 ** -8 * o.abs() + (2.0 ** -7 + 2 * eps) * mag + tiny
    dp, D = g @ vf.transpose(-1, -2), (g * o).sum(-1, keepdim=True)
    off_d = (g.abs() * (off_o + 2.0 ** -14 * o.abs())).sum(-1, keepdim=True) + 2.0 ** -14 * (g.abs() @ vf.abs().transpose(-1, -2))
    ds = p * rate * (dp - D)
    off = p * rate * ((2 * 2.0 ** -8 + 2 * eps + rr) * (dp.abs() + D.abs()) + off_d)

    def shared(x):
        return x.view(x.shape[0], Hk, H // Hk, *x.shape[2:]).sum(2)

    def up(ref, err, terms):
        err = err + 2.0 ** -14 * terms
        return ref, err + 2.0 ** -8 * (ref.abs() + err) + tiny

    dst, offt, pt = (x.transpose(-1, -2) for x in (ds, off, p))
    dq = up(ds @ kf * scale, off @ kf.abs() * scale, ds.abs() @ kf.abs() * scale)
    dk = up(shared(dst @ qf) * scale, shared(offt @ qf.abs()) * scale, shared(dst.abs() @ qf.abs()) * scale)
    dv = up(shared(pt @ g), shared((2.0 ** -8 + 2 * eps.transpose(-1, -2)) * pt @ g.abs()), shared(pt @ g.abs()))
    return (o, off_o), (lse, eps[..., 0] + 2.0 ** -20 * lse.abs()), dq, dk, dv


@pytest.mark.parametrize("cap,mult", [(1e-3, 1.0), (0.25, 3.0), (1.0, 30.0), (30.0, 300.0), (1000.0, 3.0), (1000.0, 3000.0)])
@pytest.mark.parametrize("d,bias", [(32, True), (64, False), (128, False), (128, True)])
def test_scores_beyond_the_cap(fa_lib, d, bias, cap, mult):
    """Caps at both ends, scores from a small part of the cap to thousands of it, signs of both kinds.  Where all scores of a
    row are far beyond it, its gradients are as small as the cap's derivative."""
    fa = fa_lib
    B, H, Hk, N = 2, 4, 2, 300
    g = torch.Generator().manual_seed(23)
    q, k, v, do = (rand(g, B, h, N, d, mult=x) for h, x in ((H, mult), (Hk, 1.0), (Hk, 1.0), (H, 1.0)))
    slopes = torch.rand(H, generator=g).to(DEV) * 0.1 if bias else None
    m = fa.mask_ranges(B, N, causal=True, documents=i32([[0, 100, 300], [0, 250, 290]]))
    o, lse = fa.attention_ranges(q, k, v, m, softcap=cap, slopes=slopes)
    got = (o, lse, *fa.attention_ranges_backward(q, k, v, o, lse, do, m, softcap=cap, slopes=slopes))
    for x, (ref, tol), name in zip(got, capped_reference(q, k, v, do, m, d ** -0.5, cap, slopes), ("O", "L", "dQ", "dK", "dV")):
        close(x, ref, tol, name)
    clean_status(fa)


# ------------------------------------------------------------------ masks

@pytest.mark.parametrize("d,cap,mult", [(64, 0.0, 4.0), (128, 300.0, 3.0)])
@pytest.mark.parametrize("Nq,Nk", [(2500, 1100), (1200, 3000)])
def test_ranges_far_from_their_rows(fa_lib, d, cap, mult, Nq, Nk):
    """Ranges that run against the rows' order, more rows than keys, with slopes either way: biases of hundreds, on either
    side of the row's position, in tiles that one row of many sees.  A bias is off by 2^-22 of it, which is less than what
    the products' bound of 2^-16 size leaves beyond the error of a sum of 128 (2^-17 size)."""
    fa = fa_lib
    H, Hk = 4, 2
    g = torch.Generator().manual_seed(29)
    q, k, v, do = (rand(g, 1, h, n, d, mult=x) for h, n, x in ((H, Nq, mult), (Hk, Nk, mult), (Hk, Nk, 1.0), (H, Nq, 1.0)))
    i = torch.arange(Nq)
    first = (Nk - 1 - i * Nk // Nq - torch.randint(0, 200, (Nq,), generator=g)).clamp_min(0)
    last = (first + torch.randint(0, 300, (Nq,), generator=g)).clamp_max(Nk)
    last[::97] = Nk
    m = fa.range_mask(first[None].int().to(DEV), last[None].int().to(DEV), Nk)
    slopes = torch.tensor([0.2, 0.05, -0.0125, -0.2], device=DEV)
    size = orc.forward(q, k, v, m.first, m.last, d ** -0.5, cap, slopes)[3]
    assert 32 * size[:, :, (first < last).to(DEV)].min() >= 0.2 * 3000
    check(fa, q, k, v, m, cap, slopes, do=do)


# ------------------------------------------------------------------ many values that are not finite

@pytest.mark.parametrize("d,H,Nq,Nk,every", [(32, 2, 200, 3000, 7), (64, 2, 300, 2999, 1), (128, 2, 129, 3001, 31),
                                              (128, 512, 128, 160000, 300), (64, 512, 128, 160000, 1),
                                              (128, 3, 100, 300000, 300), (32, 3, 200, 270000, 77)])
def test_many_values_that_are_not_finite(fa_lib, d, H, Nq, Nk, every):
    """In every tile that a unit takes with masked places, for several units of a CTA: each row's elements are infinite or NaN
    by the keys it sees, the others as if those values were zeros, and no wait runs out."""
    fa = fa_lib
    g = torch.Generator().manual_seed(37)
    q, k, v = rand(g, 1, H, Nq, d), rand(g, 1, 1, Nk, d), rand(g, 1, 1, Nk, d)
    first = torch.randint(0, Nk // 2, (1, Nq), generator=g, dtype=torch.int32)
    last = first + torch.randint(0, Nk // 2, (1, Nq), generator=g, dtype=torch.int32)
    first[0, 0], last[0, 0] = 0, Nk
    last[0, 1::64] = 0  # rows without keys: no tile is seen whole
    m = fa.range_mask(first.to(DEV), last.to(DEV), Nk)
    values = torch.tensor([INF, -INF, NAN], dtype=torch.bfloat16)
    at = torch.arange(3, Nk, every)
    what, e = torch.randint(0, 3, at.shape, generator=g), torch.randint(0, d // 2, at.shape, generator=g)
    bad, zero = v.clone(), v.clone()
    bad[0, 0, at.to(DEV), e.to(DEV)] = values[what].to(DEV)
    zero[0, 0, at.to(DEV), e.to(DEV)] = 0.0
    want, wl = fa.attention_ranges(q, k, zero, m)
    o, lse = fa.attention_ranges(q, k, bad, m)
    clean_status(fa)
    assert torch.equal(lse, wl)

    def sees(some):  # [Nq, d]: whether the row sees a key with such an element
        n = torch.cat([torch.zeros(1, d), (some.float().cumsum(0))]).double()
        return n[m.last[0].cpu().long()] - n[m.first[0].cpu().long()] > 0

    x = bad[0, 0].cpu()
    up, down = sees((x == INF) | torch.isnan(x)), sees((x == -INF) | torch.isnan(x))
    add = torch.where(up & down, NAN, torch.where(up, INF, torch.where(down, -INF, 0.0))).to(DEV)
    ref = want.double() + add
    close(o, ref, torch.zeros_like(ref), "O")


# ------------------------------------------------------------------ rows of very many keys

@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("n", [1 << 18, (1 << 22) + 1000])
def test_sums_of_very_many_like_terms(fa_lib, d, n):
    """Equal weights, values in 1 .. 2.  The tensor cores cut each term by up to 2^-25 of the sum; over 2^18 keys at most (2^16
    where there are more) that is 2^-7 (2^-9) of it, and half of that on the average; the result's rounding 2^-8."""
    fa = fa_lib
    g = torch.Generator(device=DEV).manual_seed(41)
    q = torch.zeros(1, 1, 100, d, dtype=torch.bfloat16, device=DEV)
    v = (1 + torch.rand(1, 1, n, d, generator=g, device=DEV)).to(torch.bfloat16)
    o, lse = fa.attention_ranges(q, v, v, fa.mask_ranges(1, 100, n))
    ref = v.double().mean(2, keepdim=True)
    close(o, ref.expand_as(o), ((2.0 ** -8 + (2.0 ** -8 if n == 1 << 18 else 2.0 ** -9)) * ref).expand_as(o), "O")
    assert (lse - math.log(n)).abs().max() <= 2.0 ** -18 + 2.0 ** -20 * 16
    clean_status(fa)


@pytest.mark.parametrize("d,cap,bias", [(128, 0.0, False), (128, 20.0, True), (64, 0.0, True), (32, 20.0, False)])
def test_long_rows(fa_lib, d, cap, bias):
    """Rows of 2^18 keys and more: ranges that begin and end anywhere, rows without keys, scores that grow along the row
    (references move, before and after a segment's end) or fall.  Slopes of 2^-10 at most: biases of 300, of which 2^-22 is
    less than the products' bound leaves (2^-17 size, and size is 2.5 or more for d >= 32)."""
    fa = fa_lib
    H, Hk, Nq, Nk = 2, 1, 140, (1 << 18) + 70001
    g = torch.Generator().manual_seed(43)
    q, k, v = rand(g, 1, H, Nq, d, mult=1.5), rand(g, 1, Hk, Nk, d, mult=1.5), rand(g, 1, Hk, Nk, d)
    k *= torch.linspace(0.3, 3.0, Nk, device=DEV)[:, None].to(torch.bfloat16)
    first = torch.randint(0, Nk // 3, (1, Nq), generator=g, dtype=torch.int32)
    last = Nk - torch.randint(0, Nk // 3, (1, Nq), generator=g, dtype=torch.int32)
    first[0, 5:9], last[0, 5:9] = 0, Nk
    last[0, 10::50] = 0
    last[0, 11::50] = first[0, 11::50] + 70
    m = fa.range_mask(first.to(DEV), last.to(DEV), Nk)
    slopes = slopes_of(H) * 2.0 ** -6 if bias else None
    o, lse = fa.attention_ranges(q, k, v, m, softcap=cap, slopes=slopes)
    check_forward(o, lse, q, k, v, m, d ** -0.5, cap, slopes)
    o2, lse2 = fa.attention_ranges(q, k, v, m, softcap=cap, slopes=slopes)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    clean_status(fa)


def test_a_row_of_very_many_keys(fa_lib):
    """One unit of 2^22 tiles and one more takes longer than any single wait may.  All scores are 0 and all values 1 (keys and
    values are one tensor): weights are a power of two, and the sums, below 2^6 in steps of 2^-17, exact but for the last
    tile's 77 weights of 2^-24."""
    fa = fa_lib
    n = (1 << 29) + 77
    if torch.cuda.mem_get_info()[0] < 64 * n + (4 << 30):
        pytest.skip("not enough memory free")
    q = torch.zeros(1, 1, 1, 32, dtype=torch.bfloat16, device=DEV)
    k = torch.ones(1, 1, n, 32, dtype=torch.bfloat16, device=DEV)
    m = fa.mask_ranges(1, 1, n)
    o, lse = fa.attention_ranges(q, k, k, m)
    clean_status(fa)
    assert (o == 1).all() and abs(lse.item() - math.log(n)) <= 2.0 ** -18 + 2.0 ** -20 * 21


# ------------------------------------------------------------------ a device error pending

def test_calls_while_a_device_error_is_pending(fa_lib):
    """A wait that ran out sets the status word: calls behind it skip their work and leave the outputs, the workspace may be
    used again as soon as they have ended, and once the error is taken results are right."""
    fa = fa_lib
    g = torch.Generator().manual_seed(47)
    B, H, Hk, N, d = 2, 4, 2, 3000, 128
    q, k, v, do = (rand(g, B, h, N, d) for h in (H, Hk, Hk, H))
    m = fa.mask_ranges(B, N, causal=True)
    o, lse = fa.attention_ranges(q, k, v, m)
    want = fa.attention_ranges_backward(q, k, v, o, lse, do, m)
    ws = torch.empty(fa.fa_bwd_ranges_workspace_size(B, H, Hk, N, N, d), dtype=torch.uint8, device=DEV)
    outs = [torch.full_like(x, 7.0) for x in (q, k, v)]
    stream = torch.cuda.current_stream().cuda_stream
    fa.check(fa.fa_debug_timeout_probe(1000, stream))
    for _ in range(20):
        status = fa.fa_bwd_ranges(*(x.data_ptr() for x in (q, k, v, o, do, lse, *outs)), None, None, None, None,
                                  m.buffer.data_ptr(), m.buffer.nbytes, B, H, Hk, N, N, d, 0.0, None, d ** -0.5,
                                  ws.data_ptr(), ws.nbytes, stream)
        assert status == 0
        ws.fill_(0x5a)
        assert (ws == 0x5a).all()
    assert fa.fa_poll_device_error(stream)[0] == fa.FA_ERR_TIMEOUT
    assert all((x == 7.0).all() for x in outs)
    o2, lse2 = fa.attention_ranges(q, k, v, m)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    got = fa.attention_ranges_backward(q, k, v, o, lse, do, m, workspace=ws)
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    clean_status(fa)
