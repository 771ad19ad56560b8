"""The operators together, as a model uses them: a prompt prefilled, a chunk prefilled on the cached prefix, drafted
tokens decoded, against one causal attention over the whole sequence."""
import math

import pytest
import torch

from oracle import operators as orc

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("fp8", [False, True])
def test_prompt_chunk_and_drafts(fa_lib, fp8):
    fa = fa_lib
    B, H, d, page = 2, 4, 64, 32
    prompt, chunk, drafts = 70, 50, 5
    total = prompt + chunk + drafts
    g = torch.Generator().manual_seed(21)
    # the projections' outputs for the whole sequence; the last tokens are a tree: 0 - 1 - 2, 0 - 3, 4
    parents = [-1, 0, 1, 0, -1]
    depth = torch.tensor([0, 1, 2, 1, 0])
    qp, kp, vp = (torch.randn(B, total, H, d, generator=g).to(torch.bfloat16).to(DEV) for _ in range(3))
    w = (1 + 0.2 * torch.randn(2, d, generator=g)).to(DEV)
    ang = torch.arange(200, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    cos, sin = ang.cos().float().to(DEV), ang.sin().float().to(DEV)
    pos = torch.cat([torch.arange(prompt + chunk), prompt + chunk + depth]).to(torch.int32)

    def heads(a, b):
        """q, k normed and rotated and v of tokens a .. b-1, [B,H,n,d]."""
        q, k = fa.qk_norm_rope(qp[:, a:b].transpose(1, 2), kp[:, a:b].transpose(1, 2), w[0], w[1], cos, sin,
                               pos[a:b].expand(B, b - a).contiguous().to(DEV))
        return q, k, vp[:, a:b].transpose(1, 2)

    cols = (total + page - 1) // page
    pages = B * cols
    table = torch.randperm(pages, generator=g).reshape(B, cols).to(torch.int32).to(DEV)
    cache = fa.new_cache(pages, H, page, d, torch.float8_e4m3fn if fp8 else torch.bfloat16)
    n = torch.full((B,), prompt, dtype=torch.int32, device=DEV)
    q, k, v = heads(0, prompt)
    fa.cache_write(cache, k, v, table, n)
    n += chunk
    q, k, v = heads(prompt, prompt + chunk)
    fa.cache_write(cache, k, v, table, n)
    kk, vv = fa.cache_read(cache, table, n, prompt + chunk)
    o_chunk, l_chunk = fa.attention_forward(q, kk, vv, causal=True)
    # the chunk's attention straight over the cache: the same keys, the same mask
    o_tree, l_tree = fa.attention_tree(q, cache, table, n)
    n += drafts
    qd, k, v = heads(prompt + chunk, total)
    fa.cache_write(cache, k, v, table, n)
    words = fa.tree_words(parents)
    o_draft, l_draft = fa.attention_tree(qd, cache, table, n, words.to(DEV))

    K, V = (x.cpu().double() for x in fa.cache_read(cache, table, n, total))
    # what is in the cache is what the norm gave, rounded to the cache's format
    _, kall, _ = heads(0, total)
    err = (K - kall.cpu().double()).abs()
    if fp8:  # at most half a step of e4m3 (2^-4 of the value), or of its smallest step, 2^-10 of a scale <= amax / 224
        assert (err <= 2.0 ** -4 * K.abs() + 2.0 ** -10 * K.abs().amax(-1, keepdim=True) / 200).all()
    else:
        assert not err.any()

    def ref(qrow, see, b, h):
        prod = qrow.cpu().double() * K[b, h, see]
        s = prod.sum(-1) / math.sqrt(d)
        wgt = torch.softmax(s, 0)
        e = 2 * d * 2.0 ** -24 * float(prod.abs().sum(-1).max()) / math.sqrt(d)
        mag = wgt @ V[b, h, see].abs()
        o = wgt @ V[b, h, see]
        return o, 2.0 ** -8 * o.abs() + (2.0 ** -7 + 2 * e + 2.0 ** -14) * mag

    for b in range(B):
        for h in range(H):
            for i in (0, 13, chunk - 1):
                o, tol = ref(q[b, h, i], list(range(prompt + i + 1)), b, h)
                for got in (o_chunk, o_tree):
                    assert ((got[b, h, i].cpu().double() - o).abs() <= tol).all()
            for t in range(drafts):
                see = list(range(prompt + chunk)) + [prompt + chunk + j for j in range(drafts) if int(words[t, 0]) >> j & 1]
                o, tol = ref(qd[b, h, t], see, b, h)
                assert ((o_draft[b, h, t].cpu().double() - o).abs() <= tol).all()


def test_training_through_norm_and_attention(fa_lib):
    """Gradients of a loss through norm, rotation and attention reach the projections and the weights, and agree with
    float64 autograd over the same formula."""
    from exact_tiled_attention_26_gb300.autograd import flash_attention, qk_norm_rope
    B, H, N, d = 1, 2, 33, 64
    g = torch.Generator().manual_seed(22)
    x = [torch.randn(B, N, H, d, generator=g).to(torch.bfloat16) for _ in range(3)]
    do = torch.randn(B, H, N, d, generator=g).to(torch.bfloat16)
    w = [1 + 0.2 * torch.randn(d, generator=g) for _ in range(2)]
    ang = torch.rand(N, d // 2, generator=g) * 6
    cos, sin = ang.cos(), ang.sin()
    leaves = [t.to(DEV).requires_grad_() for t in x + w]
    q, k, v = (t.transpose(1, 2) for t in leaves[:3])
    qo, ko = qk_norm_rope(q, k, leaves[3], leaves[4], cos.to(DEV), sin.to(DEV))
    flash_attention(qo, ko, v, causal=True).backward(do.to(DEV))
    ref = [t.double().requires_grad_() for t in x + w]
    rq, rk, rv = (t.transpose(1, 2) for t in ref[:3])

    def normed(t, wt):
        y = t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6) * wt
        a, b = y[..., :d // 2], y[..., d // 2:]
        c, s = cos.double(), sin.double()
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    s = normed(rq, ref[3]) @ normed(rk, ref[4]).transpose(-1, -2) / math.sqrt(d)
    s = s.masked_fill(torch.ones(N, N, dtype=torch.bool).triu(1), -math.inf)
    (torch.softmax(s, -1) @ rv).backward(do.double())
    for got, want in zip(leaves, ref):
        # the chain rounds to bf16 at q, k, P, dS, dO's product and the gradients: a few 2^-8 of the norm
        assert (got.grad.cpu().double() - want.grad).norm() <= 6 * 2.0 ** -8 * want.grad.norm()


def test_the_oracle_agrees_with_the_cache_it_reads(fa_lib):
    """The oracle's own reading of pages is the kernel's (one sequence, one hole)."""
    fa = fa_lib
    cache = fa.new_cache(3, 1, 16, 32)
    table = torch.tensor([[2, -1, 0]], dtype=torch.int32)
    x = torch.randn(1, 1, 40, 32).to(torch.bfloat16)
    n = torch.tensor([40], dtype=torch.int32)
    fa.cache_write(cache, x.to(DEV), x.to(DEV), table.to(DEV), n.to(DEV))
    rows, there = orc.sequence(cache.k.cpu().double(), table, 40, 16, 0)
    assert there.tolist() == [True] * 16 + [False] * 16 + [True] * 8
    assert torch.equal(rows[0, there], x[0, 0, there].double())


def test_calls_keep_no_tensor(fa_lib):
    """Returned and refused calls hold no reference to their tensors: after many calls the memory is what it was."""
    import sys
    fa = fa_lib
    q = torch.randn(2, 4, 3, 64, device=DEV).to(torch.bfloat16)
    k = torch.randn(2, 2, 3, 64, device=DEV).to(torch.bfloat16)
    w = torch.ones(64, device=DEV)
    cache = fa.new_cache(4, 2, 16, 64)
    table = torch.tensor([[0], [1]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([3, 9], dtype=torch.int32, device=DEV)

    def calls():
        fa.cache_write(cache, k, k, table, lens)
        fa.cache_read(cache, table, lens, 9)
        fa.attention_tree(q, cache, table, lens)
        fa.qk_norm_rope(q, k, w, w)
        fa.qk_norm_rope_backward(q, k, q, k, w, w)
        fa.qk_norm_rope_backward(q, k, q, k)
        with pytest.raises(ValueError):
            fa.attention_tree(q.float(), cache, table, lens)
        with pytest.raises(fa.FAError):
            fa.attention_tree(q, cache, table, lens, scale=-1.0)

    calls()
    torch.cuda.synchronize()
    held = (q, k, w, cache.k, cache.v, table, lens)
    before = torch.cuda.memory_allocated(), [sys.getrefcount(t) for t in held], sys.getrefcount(None)
    for _ in range(200):
        calls()
    torch.cuda.synchronize()
    after = torch.cuda.memory_allocated(), [sys.getrefcount(t) for t in held], sys.getrefcount(None)
    assert after[:2] == before[:2] and abs(after[2] - before[2]) < 100


def test_workspaces_of_the_caller(fa_lib):
    """A workspace that is large enough is used as it is, a smaller one is not; a misaligned one is refused."""
    fa = fa_lib
    g = torch.Generator().manual_seed(5)
    q = torch.randn(2, 8, 3, 64, generator=g).to(torch.bfloat16).to(DEV)
    k = torch.randn(2, 2, 3, 64, generator=g).to(torch.bfloat16).to(DEV)
    cache = fa.new_cache(64, 2, 16, 64)
    x = torch.randn(2, 2, 500, 64, generator=g).to(torch.bfloat16).to(DEV)
    table = torch.arange(64, dtype=torch.int32, device=DEV).view(2, 32)
    lens = torch.tensor([500, 333], dtype=torch.int32, device=DEV)
    fa.cache_write(cache, x, x, table, lens, lens)
    want = fa.attention_tree(q, cache, table, lens)
    n = fa.fa_fwd_tree_workspace_size(2, 8, 2, 3, 64)
    ws = torch.full((n + 16,), 0xFF, dtype=torch.uint8, device=DEV)
    for given in (ws[:n], ws[:n], ws[:n - 1], torch.empty(0, dtype=torch.uint8, device=DEV), ws.cpu()):
        got = fa.attention_tree(q, cache, table, lens, workspace=given)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert not (ws[:n] == 0xFF).all() and (ws[n:] == 0xFF).all()
    with pytest.raises(fa.FAError):
        fa.attention_tree(q, cache, table, lens, workspace=ws[1:])
    w = torch.ones(64, device=DEV)
    want = fa.qk_norm_rope_backward(q, k, q, k, w, w)
    n = fa.fa_qk_norm_rope_bwd_workspace_size(2, 8, 2, 3, 64)
    ws = torch.full((n + 16,), 0xFF, dtype=torch.uint8, device=DEV)
    for given in (ws[:n], ws[:n - 1]):
        assert all(torch.equal(a, b) for a, b in zip(fa.qk_norm_rope_backward(q, k, q, k, w, w, workspace=given), want))
    with pytest.raises(fa.FAError):
        fa.qk_norm_rope_backward(q, k, q, k, w, w, workspace=ws[1:])


def test_views_of_one_projection_and_broadcast_gradients(fa_lib):
    """q and k as views of one fused projection, gradients that are one row for all: the same as of copies."""
    fa = fa_lib
    g = torch.Generator().manual_seed(6)
    B, N, H, Hk, d = 2, 7, 4, 2, 64
    qkv = torch.randn(B, N, H + 2 * Hk, d, generator=g).to(torch.bfloat16).to(DEV)
    q, k = qkv[:, :, :H].transpose(1, 2), qkv[:, :, H:H + Hk].transpose(1, 2)
    w = (1 + 0.1 * torch.randn(2, d, generator=g)).to(DEV)
    row = torch.randn(d, generator=g).to(torch.bfloat16).to(DEV)
    dq, dk = row.expand(B, H, N, d), row.expand(B, Hk, N, d)
    for a, b in zip(fa.qk_norm_rope(q, k, w[0], w[1]), fa.qk_norm_rope(q.contiguous(), k.contiguous(), w[0], w[1])):
        assert a.is_contiguous() and torch.equal(a, b)
    got = fa.qk_norm_rope_backward(q, k, dq, dk, w[0], w[1])
    want = fa.qk_norm_rope_backward(q.contiguous(), k.contiguous(), dq.contiguous(), dk.contiguous(), w[0], w[1])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
