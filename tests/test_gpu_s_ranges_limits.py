"""Attention over ranges of keys at the limits of what it takes: keys that are not finite in the gradients, no
query heads, scores far beyond the cap.

Bounds as in test_gpu_o_ranges.py and oracle/ranges.py.
"""
import math

import pytest
import torch

from oracle import ranges as orc
from test_gpu_o_ranges import close, rand
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
