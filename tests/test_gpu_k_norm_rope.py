"""Per-head norm and rotation of queries and keys, forward and gradients, against the float64 oracle.

Tolerances, per element, from the arithmetic: a bf16 output is off by at most 2^-8 of its value for the one rounding;
before it, fp32: the mean of squares adds d <= 128 terms in a tree (relative error below 16 * 2^-24), the reciprocal root
2 ulp, a handful of products, so less than 64 * 2^-24 = 2^-18 of the magnitudes that enter (both elements of a pair; for
dx also the mean's tree: 2^-17 of r (|g| + |xh| mean |g xh|)).  A weight gradient is a sum of n rows: each partial sum adds
at most n terms in sequence, so its error is below (n + 64) * 2^-24 of the sum of magnitudes.
"""
import pytest
import torch

from oracle import operators as orc

pytestmark = pytest.mark.gpu
DEV = "cuda"


def tables(rows, rope, seed=0):
    ang = torch.rand(rows, rope // 2, generator=torch.Generator().manual_seed(seed)) * 40 - 20
    return ang.cos(), ang.sin()


def make(B, H, N, d, layout, g, mult=1.0):
    """bf16 [B,H,N,d] on the GPU with the strides of a layout, and its CPU values."""
    if layout == "bhnd":
        t = torch.randn(B, H, N, d, generator=g)
    elif layout == "bnhd":
        t = torch.randn(B, N, H, d, generator=g).transpose(1, 2)
    else:  # a slice of a wider projection: rows apart by more than d
        t = torch.randn(B, N, H + 3, d + 16, generator=g)[:, :, 1:H + 1, 8:d + 8].transpose(1, 2)
    t = (t * mult).to(torch.bfloat16)
    # keep the strides on the device
    base = torch.zeros(int(sum((n - 1) * s for n, s in zip(t.shape, t.stride())) + 1) if t.numel() else 0,
                       dtype=torch.bfloat16, device=DEV)
    dev = base.as_strided(t.shape, t.stride())
    dev.copy_(t)
    return dev, t


def pair_magnitude(y, rope, interleaved):
    m = y.abs()
    out = m.clone()
    if rope:
        a, b = ((slice(0, rope, 2), slice(1, rope, 2)) if interleaved
                else (slice(0, rope // 2), slice(rope // 2, rope)))
        out[..., a] = out[..., b] = m[..., a] + m[..., b]
    return out


def check(got, ref, mag, units, what):
    got = got.detach().cpu().to(torch.float64)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), what
    err, tol = (got - ref).abs(), 2.0 ** -8 * ref.abs() + units * mag + 1e-38
    ok = torch.isnan(ref) | (err <= tol)
    assert ok.all(), f"{what}: {float((err / tol)[~ok].max()):.3f} of the bound"


CASES = [
    # B, H, Hk, N, d, rope, layout, interleaved, weights, positions
    (1, 1, 1, 1, 128, 128, "bhnd", False, "f32", None),
    (3, 4, 1, 7, 64, 64, "bnhd", True, "bf16", "mixed"),
    (2, 5, 3, 33, 32, 32, "slice", False, "f32", "mixed"),
    (2, 8, 2, 65, 128, 96, "slice", False, "f32", "mixed"),
    (1, 6, 6, 130, 128, 64, "bnhd", True, "f32", "far"),
    (4, 9, 1, 1, 64, 16, "bnhd", False, "bf16", "mixed"),
    (2, 3, 2, 19, 128, 0, "bhnd", False, "f32", None),
    (1, 4, 4, 21, 32, 16, "slice", True, None, None),
    (1, 4, 0, 5, 64, 64, "bhnd", False, "f32", None),
    (2, 32, 8, 515, 128, 128, "bnhd", False, "f32", "mixed"),
]


@pytest.mark.parametrize("B, H, Hk, N, d, rope, layout, interleaved, weights, positions", CASES)
def test_forward_and_gradients(fa_lib, B, H, Hk, N, d, rope, layout, interleaved, weights, positions):
    fa = fa_lib
    g = torch.Generator().manual_seed(B * 1000 + N * 10 + d)
    q, qc = make(B, H, N, d, layout, g, 2.0)
    k, kc = make(B, Hk, N, d, layout, g, 0.5)
    if N > 2 and H > 1:
        q[0, 1, 2] = 0  # a row of zeros: r = 1 / sqrt(eps)
        qc[0, 1, 2] = 0
    dz, dzc = make(B, H, N, d, "slice", g)
    dzk, dzkc = make(B, Hk, N, d, "bhnd", g)
    rows = max(N, 70)
    cos, sin = tables(rows, rope) if rope else (None, None)
    pos = None
    if positions:
        pos = torch.randint(0, rows, (B, N), generator=g, dtype=torch.int32)
        if positions == "mixed" and N > 4:
            pos[0, 1], pos[-1, 3] = -1, -2147483648
        if positions == "far":
            pos[0, 2], pos[0, 5] = rows, 2147483647
    wt = {"f32": torch.float32, "bf16": torch.bfloat16, None: None}[weights]
    qw = None if wt is None else (1 + 0.5 * torch.randn(d, generator=g)).to(wt)
    kw = None if wt is None else (1 + 0.5 * torch.randn(d, generator=g)).to(wt)
    on = [None if t is None else t.to(DEV) for t in (qw, kw, cos, sin, pos)]
    eps = 1e-5
    qo, ko = fa.qk_norm_rope(q, k, *on, eps, interleaved)
    dq, dk, dqw, dkw = fa.qk_norm_rope_backward(q, k, dz, dzk, *on, eps, interleaved)
    again = fa.qk_norm_rope_backward(q, k, dz, dzk, *on, eps, interleaved)
    for a, b in zip((dq, dk, dqw, dkw), again):
        assert (a is None and b is None) or torch.equal(a.nan_to_num(), b.nan_to_num())
    assert qo.is_contiguous() and ko.is_contiguous() and qo.shape == q.shape and ko.shape == k.shape
    for what, x, w, z, dx, dw, got in (("q", qc, qw, dzc, dq, dqw, qo), ("k", kc, kw, dzkc, dk, dkw, ko)):
        ref, y = orc.norm_rope(x, w, cos, sin, pos, eps, interleaved)
        check(got, ref, pair_magnitude(y, rope, interleaved), 2.0 ** -18, what + " out")
        rdx, rdw, mag, wmag = orc.norm_rope_grad(x, z, w, cos, sin, pos, eps, interleaved)
        check(dx, rdx, pair_magnitude(mag, rope, interleaved), 2.0 ** -17, "d" + what)
        if dw is None:
            assert weights is None
        else:
            n = x.shape[0] * x.shape[1] * x.shape[2]
            half = 2.0 ** -8 if wt == torch.bfloat16 else 2.0 ** -24
            gotw = dw.cpu().to(torch.float64)
            assert torch.equal(torch.isnan(gotw), torch.isnan(rdw))
            bound = half * rdw.abs() + (n + 64) * 2.0 ** -24 * pair_magnitude(wmag, rope, interleaved) * 2
            assert (torch.isnan(rdw) | ((gotw - rdw).abs() <= bound + 1e-30)).all(), what + " weight"


def test_gradient_against_differences(fa_lib):
    """The GPU's gradients against differences of the float64 forward along random directions."""
    fa = fa_lib
    g = torch.Generator().manual_seed(5)
    B, H, Hk, N, d = 2, 3, 1, 5, 64
    q, qc = make(B, H, N, d, "bnhd", g)
    k, _ = make(B, Hk, N, d, "bhnd", g)
    dz, dzc = make(B, H, N, d, "bhnd", g)
    dzk = torch.zeros_like(k)
    cos, sin = tables(16, d)
    w = 1 + 0.3 * torch.randn(d, generator=g)
    dq, dk, dqw, _ = fa.qk_norm_rope_backward(q, k, dz, dzk, w.to(DEV), w.to(DEV), cos.to(DEV), sin.to(DEV))
    assert not dk.any()

    def loss(x, w):
        return float((orc.norm_rope(x, w, cos, sin, None, 1e-6, False)[0] * dzc.double()).sum())

    x, h = qc.double(), 1e-5
    for _ in range(4):
        u, v = torch.randn(x.shape, generator=g).double(), torch.randn(d, generator=g).double()
        fd = (loss(x + h * u, w.double()) - loss(x - h * u, w.double())) / (2 * h)
        # bf16 gradients: each of the n products u dq is off by at most 2^-8 of itself
        tol = 2.0 ** -8 * float((u * dq.cpu().double()).abs().sum()) + 1e-4
        assert abs(fd - float((u * dq.cpu().double()).sum())) <= tol
        fw = (loss(x, w.double() + h * v) - loss(x, w.double() - h * v)) / (2 * h)
        assert abs(fw - float((v * dqw.cpu().double()).sum())) <= 1e-3


def test_broadcast_inputs_and_gradients(fa_lib):
    """One head expanded to many (stride 0): read as it lies, its gradient the sum over the heads."""
    from exact_tiled_attention_26_gb300.autograd import qk_norm_rope
    g = torch.Generator().manual_seed(6)
    base = torch.randn(2, 1, 9, 64, generator=g).to(torch.bfloat16).to(DEV).requires_grad_()
    one = torch.randn(2, 1, 9, 64, generator=g).to(torch.bfloat16).to(DEV)
    w = torch.ones(64, device=DEV, requires_grad=True)
    cos, sin = (t.to(DEV) for t in tables(9, 64))
    qo, _ = qk_norm_rope(base.expand(2, 4, 9, 64), one, w, None, cos, sin)
    dz = torch.randn(2, 4, 9, 64, generator=g).to(torch.bfloat16).to(DEV)
    qo.backward(dz)
    x = base.detach().cpu().expand(2, 4, 9, 64)
    rdx, rdw, mag, wmag = orc.norm_rope_grad(x, dz.cpu(), torch.ones(64), cos.cpu(), sin.cpu(), None, 1e-6, False)
    err = (base.grad.cpu().double() - rdx.sum(1, keepdim=True)).abs()
    # four bf16 gradients summed in bf16 (torch): each rounding at most 2^-8 of the running magnitude
    assert (err <= 5 * 2.0 ** -8 * rdx.abs().sum(1, keepdim=True) + 2.0 ** -15 * mag.sum(1, keepdim=True)
            + 2.0 ** -7 * 0.01).all()
    bound = 136 * 2.0 ** -23 * pair_magnitude(wmag, 64, False)
    assert ((w.grad.cpu().double() - rdw).abs() <= bound).all()


def test_outputs_stay_inside_and_workspace_is_only_scratch(fa_lib):
    """Guard bands around every output and the workspace, which comes filled with NaN."""
    fa = fa_lib
    g = torch.Generator().manual_seed(7)
    B, H, Hk, N, d = 2, 3, 2, 11, 32
    q, _ = make(B, H, N, d, "bhnd", g)
    k, _ = make(B, Hk, N, d, "bhnd", g)
    w = torch.ones(d, device=DEV)
    cos, sin = (t.to(DEV) for t in tables(N, d))
    ref = fa.qk_norm_rope_backward(q, k, q, k, w, w, cos, sin)
    n_ws = fa.fa_qk_norm_rope_bwd_workspace_size(B, H, Hk, N, d)

    def guarded(nbytes):
        t = torch.full((nbytes + 512,), 0xA5, dtype=torch.uint8, device=DEV)
        return t, t.data_ptr() + 256

    bufs = [guarded(n) for n in (q.numel() * 2, k.numel() * 2, d * 4, d * 4, n_ws, q.numel() * 2, k.numel() * 2)]
    (dq, pdq), (dk, pdk), (dw, pdw), (dv, pdv), (ws, pws), (qo, pqo), (ko, pko) = bufs
    ws[256:256 + n_ws] = 0xFF
    s = torch.cuda.current_stream().cuda_stream
    assert fa.fa_qk_norm_rope(q.data_ptr(), k.data_ptr(), pqo, pko, None, None, w.data_ptr(), w.data_ptr(), 0,
                              cos.data_ptr(), sin.data_ptr(), d, N, 0, None, B, H, Hk, N, d, 1e-6, s) == 0
    assert fa.fa_qk_norm_rope_bwd(q.data_ptr(), k.data_ptr(), q.data_ptr(), k.data_ptr(), pdq, pdk, *[None] * 6,
                                  w.data_ptr(), w.data_ptr(), pdw, pdv, 0, cos.data_ptr(), sin.data_ptr(), d, N, 0, None,
                                  B, H, Hk, N, d, 1e-6, pws, n_ws, s) == 0
    for buf, _ in bufs:
        assert (buf[:256] == 0xA5).all() and (buf[-256:] == 0xA5).all()
    for buf, want in ((dq, ref[0]), (dk, ref[1]), (dw, ref[2]), (dv, ref[3])):
        assert torch.equal(buf[256:-256].view(want.dtype).view(want.shape), want)
    qr, kr = fa.qk_norm_rope(q, k, w, w, cos, sin)
    assert torch.equal(qo[256:-256].view(qr.dtype).view(qr.shape), qr)
    assert torch.equal(ko[256:-256].view(kr.dtype).view(kr.shape), kr)


def test_no_rows_give_zero_weight_gradients(fa_lib):
    q = torch.empty(0, 4, 8, 64, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(64, device=DEV)
    dq, dk, dqw, dkw = fa_lib.qk_norm_rope_backward(q, q, q, q, w, w)
    assert dq.shape == q.shape and not dqw.any() and not dkw.any()


def test_other_stream_and_graph(fa_lib):
    """The call runs on the current stream, and a captured step replays on new inputs."""
    from exact_tiled_attention_26_gb300.autograd import flash_attention, qk_norm_rope
    g = torch.Generator().manual_seed(8)
    q, k, v = (torch.randn(1, 2, 130, 64, generator=g).to(torch.bfloat16).to(DEV) for _ in range(3))
    w = torch.ones(64, device=DEV)
    cos, sin = (t.to(DEV) for t in tables(130, 64))

    def step():
        qq, kk, ww = (t.detach().requires_grad_() for t in (q, k, w))
        qo, ko = qk_norm_rope(qq, kk, ww, ww, cos, sin)
        flash_attention(qo, ko, v, causal=True).backward(v)
        return qq.grad, kk.grad, ww.grad

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        eager = [t.clone() for t in step()]
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, eager):
        assert (a - b).abs().max() <= 2.0 ** -6 * b.abs().max()  # dQ's L2 reductions come in any order
    q.copy_(torch.randn(q.shape, generator=g).to(torch.bfloat16))
    graph.replay()
    fresh = step()
    torch.cuda.synchronize()
    for a, b in zip(out, fresh):
        assert (a - b).abs().max() <= 2.0 ** -6 * b.abs().max()


@pytest.mark.parametrize("d, rope, interleaved", [(32, 32, False), (64, 16, True), (128, 128, False)])
@pytest.mark.parametrize("eps", [0.0, 1e-40, 1e-6, 1e30])
def test_rows_of_any_size(fa_lib, d, rope, interleaved, eps):
    """Rows whose squares pass fp32's range, up to bf16's largest and down to its least numbers, next to ordinary ones, and
    an eps anywhere in it: the tolerances of the file's head."""
    fa = fa_lib
    g = torch.Generator().manual_seed(d + rope)
    B, H, Hk, N = 2, 5, 2, 9
    sizes = [1.0, 1e20, 1e-20, 5e37, 1e-38, 3e-40, 1e10, 1e-30, 0.0]

    def rows(heads):
        t = torch.randn(B, heads, N, d, generator=g).clamp(-4, 4)
        return (t * torch.tensor(sizes)[:, None]).to(torch.bfloat16)

    def grads(heads):  # so that dx, about dz / size, is a number of bf16
        t = torch.randn(B, heads, N, d, generator=g)
        at = torch.tensor([max(s, 1e-38) for s in sizes], dtype=torch.float64).clamp(1e-3, 1e30)
        return (t * at[:, None]).to(torch.bfloat16) if eps == 0 else (t * at.clamp(max=1.0)[:, None]).to(torch.bfloat16)
    q, k, dz, dzk = rows(H), rows(Hk), grads(H), grads(Hk)
    cos, sin = tables(N, rope)
    w = 1 + 0.5 * torch.randn(d, generator=g)
    on = [t.to(DEV) for t in (w, w, cos, sin)]
    qo, ko = fa.qk_norm_rope(q.to(DEV), k.to(DEV), *on, None, eps, interleaved)
    got = fa.qk_norm_rope_backward(q.to(DEV), k.to(DEV), dz.to(DEV), dzk.to(DEV), *on, None, eps, interleaved)
    live = slice(0, N) if eps else slice(0, N - 1)  # a row of zeros has no direction: NaN with eps = 0
    if not eps:
        assert qo[:, :, N - 1].isnan().all() and ko[:, :, N - 1].isnan().all()
    for what, x, z, out, dx, dw in (("q", q, dz, qo, got[0], got[2]), ("k", k, dzk, ko, got[1], got[3])):
        eps32 = float(torch.tensor(eps, dtype=torch.float32))
        ref, y = orc.norm_rope(x, w, cos, sin, None, eps32, interleaved)
        check(out[:, :, live], ref[:, :, live], pair_magnitude(y, rope, interleaved)[:, :, live], 2.0 ** -18, what)
        rdx, _, mag, _ = orc.norm_rope_grad(x, z, w, cos, sin, None, eps32, interleaved)
        rdx, mag = rdx[:, :, live], pair_magnitude(mag, rope, interleaved)[:, :, live]
        top = torch.finfo(torch.bfloat16).max
        fits = (rdx.abs() + 2.0 ** -17 * mag) < top  # what passes bf16's range is infinite
        gotx = dx.cpu().double()[:, :, live]
        err, tol = (gotx - rdx).abs(), 2.0 ** -8 * rdx.abs() + 2.0 ** -17 * mag + 1e-38
        assert (~fits | (err <= tol)).all(), what
        _, rdw, _, wmag = orc.norm_rope_grad(x[:, :, live], z[:, :, live], w, cos[live], sin[live], None, eps32, interleaved)
        if eps:
            n = B * x.shape[1] * N
            assert ((dw.cpu().double() - rdw).abs() <= (n + 64) * 2.0 ** -23 * pair_magnitude(wmag, rope, interleaved)
                    + 2.0 ** -24 * rdw.abs() + 1e-30).all(), what + " weight"


@pytest.mark.parametrize("B, H, Hk, N, d, rope, interleaved", [(2, 32, 8, 515, 128, 128, False), (3, 6, 2, 1021, 64, 32, True),
                                                               (1, 16, 16, 700, 32, 32, False)])
def test_weight_gradients_within_the_bound_of_their_sums(fa_lib, B, H, Hk, N, d, rope, interleaved):
    """The bound of the sum that is made, not of one made row by row.  A term passes through at most `depth` additions: 4 rows
    a step in a lane, the lanes of the warp with the same columns, 8 warps, the blocks in 8 strands, the strands.  Each
    addition is off by at most 2^-24 of the sum of magnitudes, each term by 2^-18 of its own, a result in fp32 by 2^-24 of
    itself.  So narrow a bound sees one block's rows missing."""
    fa = fa_lib
    g = torch.Generator().manual_seed(B * 7 + d)
    q, qc = make(B, H, N, d, "bnhd", g, 2.0)
    k, kc = make(B, Hk, N, d, "bnhd", g, 0.5)
    dz, dzc = make(B, H, N, d, "bhnd", g)
    dzk, dzkc = make(B, Hk, N, d, "bhnd", g)
    cos, sin = tables(N, rope)
    w = 1 + 0.5 * torch.randn(d, generator=g)
    on = [t.to(DEV) for t in (w, w, cos, sin)]
    got = fa.qk_norm_rope_backward(q, k, dz, dzk, *on, None, 1e-6, interleaved)
    blocks = fa.fa_qk_norm_rope_bwd_workspace_size(B, H, Hk, N, d) // (4 * d)
    groups = 8 * 32 // (d // 8)  # lane groups of a block, 4 heads of a (batch, row) each step
    items = [B * N * ((h + 3) // 4) for h in (H, Hk)]
    for which, (x, z, dw) in enumerate(((qc, dzc, got[2]), (kc, dzkc, got[3]))):
        mine = max(1, blocks * items[which] // sum(items) - 1)  # at least so many blocks work on this tensor
        trips = -(-items[which] // (mine * groups))
        depth = 4 * trips + (32 // (d // 8)).bit_length() + 8 + -(-blocks // 8) + 8
        _, ref, _, wmag = orc.norm_rope_grad(x, z, w, cos, sin, None, 1e-6, interleaved)
        bound = (depth * 2.0 ** -24 + 2.0 ** -18) * pair_magnitude(wmag, rope, interleaved) + 2.0 ** -24 * ref.abs()
        assert ((dw.cpu().double() - ref).abs() <= bound).all(), (which, depth)
        # without the rows of one block's first step (its groups' 4 heads each)
        less = z.clone()
        less.view(B, x.shape[1], N, d)[0, :4, :groups] = 0
        _, short, _, _ = orc.norm_rope_grad(x, less, w, cos, sin, None, 1e-6, interleaved)
        assert ((short - ref).abs() > bound).float().mean() > 0.9


def test_no_rows_and_no_positions(fa_lib):
    """An empty batch with tables of no positions: empty outputs, zero weight gradients."""
    fa = fa_lib
    w = torch.ones(64, device=DEV)
    tab = torch.empty(0, 32, device=DEV)
    for shape in ((2, 4, 0, 64), (0, 4, 8, 64)):
        q, k = (torch.empty(shape[0], h, *shape[2:], dtype=torch.bfloat16, device=DEV) for h in (4, 2))
        pos = torch.empty(shape[0], shape[2], dtype=torch.int32, device=DEV)
        for p in (None, pos):
            if shape[2] and p is None:
                continue  # 8 rows, no position for them
            qo, ko = fa.qk_norm_rope(q, k, w, w, tab, tab, p)
            assert qo.shape == q.shape and ko.shape == k.shape
            dq, dk, dqw, dkw = fa.qk_norm_rope_backward(q, k, q, k, w, w, tab, tab, p)
            assert dq.shape == q.shape and not dqw.any() and not dkw.any()
