"""Cases for the operators around exact attention: per-head norm + rotation of queries and keys (forward and
gradients), the paged key/value cache (write, read back) and attention of drafted tokens over that cache.

`run` computes each operator in a plain form (elementary torch operations in fp32) or, with `own` set, through the
framework's entry points.  `exact` computes it from the definition in float64, written separately.
"""
import math
import random

import torch

own = False

DEV = "cuda"
BF16, F32, F64, E4M3 = torch.bfloat16, torch.float32, torch.float64, torch.float8_e4m3fn


def _fa():
    import exact_tiled_attention_26_gb300 as fa
    return fa


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decoding step of 32 sequences: the smallest call, latency counts
        dict(name="norm_rope_step", op="norm_rope", B=32, H=32, Hk=8, N=1, d=128, rope=128, pos=32768,
             interleaved=False, far=True),
        # a whole training or prefill pass over the 8192-token shape, from the projections' [B,N,H,d] layout
        dict(name="norm_rope_long", op="norm_rope", B=1, H=32, Hk=32, N=8192, d=128, rope=128, pos=8192,
             interleaved=False, far=False),
        # gradients of the same shape
        dict(name="norm_rope_grad_long", op="norm_rope_grad", B=1, H=32, Hk=32, N=8192, d=128, rope=128, pos=8192,
             interleaved=False, far=False),
        # gradients at d = 64, an odd length, shared key heads, half of each head rotated in neighbouring pairs
        dict(name="norm_rope_grad_odd", op="norm_rope_grad", B=4, H=8, Hk=2, N=1021, d=64, rope=32, pos=4096,
             interleaved=True, far=True),
        # a prompt written into a bf16 cache, ragged batch
        dict(name="cache_write_prompt", op="cache_write", B=4, Hk=8, T=8192, d=128, page=64, length=8192, fp8=False),
        # one token per sequence quantised into a short e4m3 cache, then the cache read back
        dict(name="cache_append_read", op="cache_write_read", B=8, Hk=8, T=1, d=128, page=16, length=509, fp8=True),
        # a chunk of a prompt quantised as it is written, then prefix and chunk read back for the chunk's attention
        dict(name="cache_chunk_read", op="cache_write_read", B=4, Hk=8, T=2048, d=128, page=64, length=16384,
             fp8=True),
        # a single token of one sequence over a short bf16 cache: latency
        dict(name="tree_single", op="tree", B=1, H=32, Hk=8, T=1, d=128, page=16, length=1000, fp8=False),
        # decoding a ragged batch over long e4m3 caches: bandwidth
        dict(name="tree_decode_ragged", op="tree", B=16, H=32, Hk=8, T=1, d=128, page=64, length=32768, fp8=True),
        # a small draft tree, padded batch, bf16 cache
        dict(name="tree_draft", op="tree", B=8, H=32, Hk=8, T=12, d=128, page=32, length=8192, fp8=False),
        # a wide draft tree over shared heads: 252 query rows on each key head, e4m3 cache
        dict(name="tree_wide", op="tree", B=4, H=32, Hk=8, T=63, d=128, page=128, length=16384, fp8=True),
        # no shared heads, d = 64
        dict(name="tree_mha_64", op="tree", B=4, H=16, Hk=16, T=24, d=64, page=16, length=4091, fp8=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_grad", "cache_write", "cache_write_read", "tree", "tree", "tree"])
    d = rng.choice([32, 64, 128, 128])
    Hk = rng.choice([1, 2, 4, 8, 16])
    G = rng.choice([1, 2, 3, 4, 8]) if Hk <= 8 else 1
    if op in ("norm_rope", "norm_rope_grad"):
        N = _log(rng, 1, 8192)
        rows = 2 * 32 * 8192 * 128 // (d * Hk * (G + 1) * N)  # batches that cost as much as the largest listed case
        B = _log(rng, 1, max(1, min(64, rows)))
        if Hk * (G + 1) * N * d > 2 * 32 * 8192 * 128:
            G = 1
        return dict(op=op, B=B, H=Hk * G, Hk=Hk, N=N, d=d, rope=rng.choice([d, d, d // 2]), pos=max(N, 4096),
                    interleaved=rng.random() < 0.4, far=rng.random() < 0.5)
    page = rng.choice([16, 32, 64, 128])
    if op == "tree":
        T = rng.choice([1, 1, _log(rng, 2, 64)])
        length = _log(rng, max(128, T), 32768)
        # keys read and rows multiplied both stay below the largest listed cases
        cap_bytes = 16 * 8 * 32768 * 128 // (Hk * length * d * 2)
        cap_flops = 4 * 32 * 63 * 16384 * 128 // (Hk * G * T * length * d)
        B = _log(rng, 1, max(1, min(64, cap_bytes, cap_flops)))
        if cap_flops < 1:
            T, B = 1, 1
        return dict(op=op, B=B, H=Hk * G, Hk=Hk, T=T, d=d, page=page, length=length, fp8=rng.random() < 0.5)
    length = _log(rng, 128, 16384)
    B = _log(rng, 1, max(1, min(64, 4 * 8 * 8192 * 128 // (Hk * length * d))))
    T = length if op == "cache_write" else _log(rng, 1, min(length, 2048))
    return dict(op=op, B=B, Hk=Hk, T=T, d=d, page=page, length=length, fp8=op == "cache_write_read")


# ------------------------------------------------------------------ inputs

def _batch(case):
    """Lengths and new tokens of a padded, ragged batch: the first sequence is the longest and brings the most.
    They belong to the case, so that every seed has the same work."""
    B, T, top = case["B"], case["T"], case["length"]
    rng = random.Random("%d %d %d" % (B, T, top))
    new = [T] + [rng.randrange(max(1, T // 2), T + 1) for _ in range(B - 1)]
    if case["op"] == "cache_write":
        return list(new), new
    return [top] + [max(T, _log(rng, max(1, top // 8), top)) for _ in range(B - 1)], new


def _tree_words(B, T, rng):
    """Random draft trees: each token hangs on an earlier one or on the prefix; bit j of word [b,t,j//64] = token t
    sees token j (its ancestors and itself)."""
    W = (T + 63) // 64
    out = []
    for _ in range(B):
        seen = []
        for t in range(T):
            p = rng.randrange(max(-1, t - 6), t) if t else -1
            seen.append((seen[p] if p >= 0 else 0) | (1 << t))
        out.append([[_signed(s >> (64 * w) & (2 ** 64 - 1)) for w in range(W)] for s in seen])
    return torch.tensor(out, dtype=torch.int64)


def _signed(u):
    return u - 2 ** 64 if u >= 2 ** 63 else u


def _scale_of(byte):
    """The power of two an exponent byte stands for."""
    return (byte.to(torch.int32) << 23).view(F32)


def _quantise(x):
    """x [..., d] -> e4m3 values and one exponent byte for each row, scale 2^(byte - 127)."""
    x = x.to(F32)
    m, e = torch.frexp(x.abs().amax(-1))
    k = (e.to(torch.int32) - 9 + (m > 0.875)).clamp_min(-100)
    return (x * _scale_of(127 - k)[..., None]).to(E4M3), (k + 127).to(torch.uint8)


def prepare(case, seed):
    rng = random.Random(seed * 7919 + 17)
    g = torch.Generator(device=DEV).manual_seed(seed)
    op, d = case["op"], case["d"]

    def randn(*shape, mult=1.0):
        return (torch.randn(*shape, generator=g, device=DEV, dtype=F32) * mult).to(BF16)

    if op in ("norm_rope", "norm_rope_grad"):
        B, H, Hk, N, r = case["B"], case["H"], case["Hk"], case["N"], case["rope"]
        st = dict(case=case, eps=1e-6, interleaved=case["interleaved"])
        # the projections write [B,N,H,d]; the operator takes the [B,H,N,d] views
        st["q"] = randn(B, N, H, d, mult=1.5).transpose(1, 2)
        st["k"] = randn(B, N, Hk, d, mult=0.75).transpose(1, 2)
        st["qw"] = 1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)
        st["kw"] = 1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)
        inv = 10000.0 ** (-torch.arange(0, r, 2, dtype=F64, device=DEV) / r)
        ang = torch.arange(case["pos"], dtype=F64, device=DEV)[:, None] * inv
        st["cos"], st["sin"] = ang.cos().to(F32), ang.sin().to(F32)
        st["pos"] = None
        if case["far"]:  # each sequence starts somewhere in the table
            base = [rng.randrange(case["pos"] - N + 1) for _ in range(B)]
            st["pos"] = (torch.tensor(base, dtype=torch.int32, device=DEV)[:, None]
                         + torch.arange(N, dtype=torch.int32, device=DEV)).contiguous()
        if op == "norm_rope_grad":
            st["dq"], st["dk"] = randn(B, H, N, d, mult=0.01), randn(B, Hk, N, d, mult=0.01)
        return st

    B, Hk, T, page = case["B"], case["Hk"], case["T"], case["page"]
    lens, new = _batch(case)
    per_seq = [(n + page - 1) // page for n in lens]
    cols = max(per_seq)
    num = sum(per_seq) + 3
    ids = list(range(num))
    rng.shuffle(ids)
    table = torch.full((B, cols), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(per_seq):
        table[b, :n] = torch.tensor(ids[at:at + n], dtype=torch.int32)
        at += n
    st = dict(case=case, table=table.to(DEV), lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
              new=torch.tensor(new, dtype=torch.int32, device=DEV))
    if op == "cache_write":
        ck = torch.zeros(num, Hk, page, d, dtype=BF16, device=DEV)
        cv = torch.zeros(num, Hk, page, d, dtype=BF16, device=DEV)
    else:  # keys with a few strong channels, as models have them
        chan = 1.0 + 4.0 * (torch.rand(d, generator=g, device=DEV) < 0.05)
        ck = (torch.randn(num, Hk, page, d, generator=g, device=DEV) * chan).to(BF16)
        cv = randn(num, Hk, page, d)
    if case["fp8"]:
        ck, ke = _quantise(ck)
        cv, ve = _quantise(cv)
    else:
        ke = ve = None
    st.update(ck=ck, cv=cv, ke=ke, ve=ve)
    if op == "tree":
        st["q"] = randn(B, case["H"], T, d)
        st["tree"] = _tree_words(B, T, rng).to(DEV) if T > 1 else None
    else:
        st["k"], st["v"] = randn(B, Hk, T, d, mult=2.0), randn(B, T, Hk, d).transpose(1, 2)
    if own:
        st["cache"] = _fa().KVCache(ck, cv, ke, ve)
    return st


# ------------------------------------------------------------------ the framework's calls and the plain forms

def run(st):
    op = st["case"]["op"]
    return (_own if own else _plain)[op](st)


def _own_norm_rope(st):
    return _fa().qk_norm_rope(st["q"], st["k"], st["qw"], st["kw"], st["cos"], st["sin"], st["pos"], st["eps"],
                              st["interleaved"])


def _own_norm_rope_grad(st):
    return _fa().qk_norm_rope_backward(st["q"], st["k"], st["dq"], st["dk"], st["qw"], st["kw"], st["cos"],
                                       st["sin"], st["pos"], st["eps"], st["interleaved"])


def _own_write(st):
    _fa().cache_write(st["cache"], st["k"], st["v"], st["table"], st["lens"], st["new"])
    return st["ck"], st["cv"]


def _own_write_read(st):
    fa = _fa()
    fa.cache_write(st["cache"], st["k"], st["v"], st["table"], st["lens"], st["new"])
    return fa.cache_read(st["cache"], st["table"], st["lens"], st["case"]["length"])


def _own_tree(st):
    return _fa().attention_tree(st["q"], st["cache"], st["table"], st["lens"], st["tree"], st["new"])


def _rows(st, name):
    """cos or sin of every row's position, [B or 1, 1, N, rope/2]."""
    N = st["case"]["N"]
    if st["pos"] is None:
        return st[name][:N][None, None]
    return st[name][st["pos"].long()][:, None]


def _rotate(x, c, s, interleaved):
    r = 2 * c.shape[-1]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
    u, v = a * c - b * s, b * c + a * s
    rot = torch.stack((u, v), -1).flatten(-2) if interleaved else torch.cat((u, v), -1)
    return torch.cat((rot, x[..., r:]), -1)


def _plain_norm_rope(st):
    c, s = _rows(st, "cos"), _rows(st, "sin")
    out = []
    for x, w in ((st["q"], st["qw"]), (st["k"], st["kw"])):
        x = x.to(F32)
        y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + st["eps"]) * w
        out.append(_rotate(y, c, s, st["interleaved"]).to(BF16).contiguous())
    return tuple(out)


def _plain_norm_rope_grad(st):
    c, s = _rows(st, "cos"), _rows(st, "sin")
    dx, dw = [], []
    for x, w, dz in ((st["q"], st["qw"], st["dq"]), (st["k"], st["kw"], st["dk"])):
        x = x.to(F32)
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + st["eps"])
        dy = _rotate(dz.to(F32), c, -s, st["interleaved"])
        xh, gw = x * r, dy * w
        dx.append((r * (gw - xh * (gw * xh).mean(-1, keepdim=True))).to(BF16))
        dw.append((dy * xh).sum((0, 1, 2), dtype=F64).to(F32))
    return dx[0], dx[1], dw[0], dw[1]


def _slots(st):
    """(page, slot, batch, token) of every new token that has a place."""
    T, page = st["case"]["T"], st["case"]["page"]
    t = torch.arange(T, device=DEV)[None]
    pos = (st["lens"] - st["new"])[:, None].long() + t
    b, t = (t < st["new"][:, None]).nonzero(as_tuple=True)
    pos = pos[b, t]
    return st["table"][b, pos // page].long(), pos % page, b, t


def _plain_write(st):
    p, s, b, t = _slots(st)
    for name, new, byte in (("ck", st["k"], "ke"), ("cv", st["v"], "ve")):
        rows = new[b, :, t]
        if st[byte] is None:
            st[name][p, :, s] = rows
        else:
            val, e = _quantise(rows)
            st[name].view(torch.uint8)[p, :, s] = val.view(torch.uint8)
            st[byte][p, :, s] = e
    return st["ck"], st["cv"]


def _gather(st, length):
    """k and v of every sequence in fp32, [B,Hk,length,d]; zeros behind its end."""
    page, table = st["case"]["page"], st["table"]
    there = torch.arange(length, device=DEV)[None] < st["lens"][:, None]
    out = []
    for name, byte in (("ck", "ke"), ("cv", "ve")):
        ids = table[:, :(length + page - 1) // page].clamp_min(0).long()
        if st[byte] is None:
            x = st[name][ids].to(F32)
        else:
            x = st[name].view(torch.uint8)[ids].view(E4M3).to(F32) * _scale_of(st[byte][ids])[..., None]
        x = x.transpose(1, 2).flatten(2, 3)[:, :, :length]
        out.append(x * there[:, None, :, None])
    return out


def _plain_write_read(st):
    _plain_write(st)
    return tuple(x.to(BF16).contiguous() for x in _gather(st, st["case"]["length"]))


def _seen(st, length):
    """[B,T,length]: whether draft token t sees key j."""
    T = st["case"]["T"]
    j = torch.arange(length, device=DEV)[None]
    prefix = (st["lens"] - st["new"])[:, None]
    rel = (j - prefix).clamp(0, T - 1)
    t = torch.arange(T, device=DEV)[None, :, None]
    if st["tree"] is None:
        own_bits = rel[:, None] <= t
    else:
        word = torch.gather(st["tree"], 2, (rel // 64)[:, None].expand(-1, T, -1).long())
        own_bits = (word >> (rel % 64)[:, None]) & 1 != 0
    live = (j < st["lens"][:, None])[:, None] & (t < st["new"][:, None, None])
    return live & ((j < prefix)[:, None] | own_bits)


def _plain_tree(st):
    c = st["case"]
    B, H, Hk, T, d, L = c["B"], c["H"], c["Hk"], c["T"], c["d"], c["length"]
    k, v = _gather(st, L)
    q = st["q"].to(F32).view(B, Hk, H // Hk, T, d)
    s = torch.matmul(q.flatten(2, 3), k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    seen = _seen(st, L)[:, None, None].expand(B, 1, H // Hk, T, L).flatten(2, 3)
    s = torch.where(seen, s, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(l == 0, 1.0, l)
    return o.to(BF16).view(B, H, T, d), (m + torch.log(l)).view(B, H, T)


_own = dict(norm_rope=_own_norm_rope, norm_rope_grad=_own_norm_rope_grad, cache_write=_own_write,
            cache_write_read=_own_write_read, tree=_own_tree)
_plain = dict(norm_rope=_plain_norm_rope, norm_rope_grad=_plain_norm_rope_grad, cache_write=_plain_write,
              cache_write_read=_plain_write_read, tree=_plain_tree)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op, d = case["op"], case["d"]
    if op in ("norm_rope", "norm_rope_grad"):
        rows = case["B"] * (case["H"] + case["Hk"]) * case["N"]
        tables = min(case["B"] * case["N"] if case["far"] else case["N"], case["pos"]) * case["rope"] * 4
        grad = op == "norm_rope_grad"
        return {"bytes": rows * d * (6 if grad else 4) + tables, "flops": rows * d * (14 if grad else 7)}
    B, Hk = case["B"], case["Hk"]
    lens, new = _batch(case)
    row = d + 1 if case["fp8"] else 2 * d
    if op == "tree":
        return {"bytes": 2 * Hk * sum(lens) * row + 4 * case["H"] * sum(new) * d,
                "flops": sum(4 * case["H"] * t * n * d for t, n in zip(new, lens))}
    wrote = 2 * Hk * sum(new) * (2 * d + row)
    if op == "cache_write":
        return {"bytes": wrote, "flops": 0}
    return {"bytes": wrote + 2 * Hk * (sum(lens) * row + B * case["length"] * 2 * d),
            "flops": 2 * Hk * (sum(lens) + sum(new)) * d}


# ------------------------------------------------------------------ from the definitions, in float64

def exact(case, seed):
    st = prepare(case, seed)
    return _exact[case["op"]](case, st)


def _turn(case, st):
    """Rotation of every row as a complex number of modulus one, [B,1,N,rope/2], from the tables."""
    B, N = case["B"], case["N"]
    at = torch.arange(N, device=DEV).expand(B, N) if st["pos"] is None else st["pos"].long()
    return torch.complex(st["cos"].to(F64)[at], st["sin"].to(F64)[at])[:, None]


def _spin(x, turn, interleaved):
    h = turn.shape[-1]
    x = x.clone()
    if interleaved:
        pair = torch.complex(x[..., 0:2 * h:2].clone(), x[..., 1:2 * h:2].clone()) * turn
        x[..., 0:2 * h:2], x[..., 1:2 * h:2] = pair.real, pair.imag
    else:
        pair = torch.complex(x[..., :h].clone(), x[..., h:2 * h].clone()) * turn
        x[..., :h], x[..., h:2 * h] = pair.real, pair.imag
    return x


def _exact_norm_rope(case, st):
    turn = _turn(case, st)
    out = []
    for x, w in ((st["q"], st["qw"]), (st["k"], st["kw"])):
        x = x.to(F64)
        out.append(_spin(x / (x.square().sum(-1, keepdim=True) / case["d"] + st["eps"]).sqrt() * w.to(F64), turn,
                         case["interleaved"]).contiguous())
    return tuple(out)


def _exact_norm_rope_grad(case, st):
    turn = _turn(case, st).conj()
    res = []
    for x, w, dz in ((st["q"], st["qw"], st["dq"]), (st["k"], st["kw"], st["dk"])):
        x, w, d = x.to(F64), w.to(F64), case["d"]
        root = (x.square().sum(-1, keepdim=True) / d + st["eps"]).sqrt()
        dy = _spin(dz.to(F64), turn, case["interleaved"])
        along = (dy * w * x).sum(-1, keepdim=True)
        res.append((dy * w / root - x * along / (d * root ** 3), (dy * x / root).sum((0, 1, 2))))
    return res[0][0], res[1][0], res[0][1], res[1][1]


def _two_to(k):
    """2^k in float64, exactly (a power function may be an ulp off)."""
    return ((k.to(torch.int64) + 1023) << 52).view(F64)


def _exact_e4m3(x):
    """Values that x [rows, d] stands for after quantising, from the format: 3 fraction bits, least exponent -6."""
    top = x.abs().amax(-1, keepdim=True)
    k = torch.frexp(top)[1] - 9  # 448 2^k is 0.875 of the power of two above top
    k = torch.where(top > 448.0 * _two_to(k), k + 1, k).clamp_min(-100)
    y = x / _two_to(k)
    step = _two_to((torch.frexp(y)[1] - 1).clamp_min(-6) - 3)
    return torch.round(y / step) * step * _two_to(k)  # round() takes ties to the even step


def _page_values(st, name, byte):
    x = st[name].to(F32).to(F64)
    return x if st[byte] is None else x * _two_to(st[byte].to(torch.int64) - 127)[..., None]


def _exact_pages(case, st):
    """The cache's values after the write, in float64."""
    page, out = case["page"], []
    table, lens, new = st["table"].tolist(), st["lens"].tolist(), st["new"].tolist()
    for name, byte, src in (("ck", "ke", st["k"]), ("cv", "ve", st["v"])):
        vals = _page_values(st, name, byte)
        for b in range(case["B"]):
            rows = src[b, :, :new[b]].to(F64)
            if case["fp8"]:
                rows = _exact_e4m3(rows)
            at, t = lens[b] - new[b], 0
            while t < new[b]:
                n = min(new[b] - t, page - (at + t) % page)
                vals[table[b][(at + t) // page], :, (at + t) % page:(at + t) % page + n] = rows[:, t:t + n]
                t += n
        out.append(vals)
    return out


def _exact_write(case, st):
    return tuple(_exact_pages(case, st))


def _exact_sequence(case, st, vals, b):
    n = int(st["lens"][b])
    ids = st["table"][b, :(n + case["page"] - 1) // case["page"]].long()
    return vals[ids].permute(1, 0, 2, 3).reshape(case["Hk"], -1, case["d"])[:, :n]


def _exact_write_read(case, st):
    res = []
    for vals in _exact_pages(case, st):
        out = torch.zeros(case["B"], case["Hk"], case["length"], case["d"], dtype=F64, device=DEV)
        for b in range(case["B"]):
            x = _exact_sequence(case, st, vals, b)
            out[b, :, :x.shape[1]] = x
        res.append(out)
    return tuple(res)


def _exact_tree(case, st):
    B, H, Hk, T, d = case["B"], case["H"], case["Hk"], case["T"], case["d"]
    o = torch.zeros(B, H, T, d, dtype=F64, device=DEV)
    lse = torch.full((B, H, T), -math.inf, dtype=F64, device=DEV)
    vk, vv = _page_values(st, "ck", "ke"), _page_values(st, "cv", "ve")
    for b in range(B):
        n, new = int(st["lens"][b]), int(st["new"][b])
        k, v = _exact_sequence(case, st, vk, b), _exact_sequence(case, st, vv, b)
        see = torch.ones(new, n, dtype=torch.bool)
        for t in range(new):
            for j in range(new):
                if st["tree"] is None:
                    see[t, n - new + j] = j <= t
        if st["tree"] is not None:
            words = st["tree"][b].tolist()
            for t in range(new):
                see[t, n - new:] = torch.tensor([words[t][j // 64] >> (j % 64) & 1 for j in range(new)]) != 0
        see = see.to(DEV)
        for h in range(H):
            s = st["q"][b, h, :new].to(F64) @ k[h // (H // Hk)].T / math.sqrt(d)
            s = s.masked_fill(~see, -math.inf)
            lse[b, h, :new] = torch.logsumexp(s, -1)
            o[b, h, :new] = torch.softmax(s, -1) @ v[h // (H // Hk)]
    return o, lse


_exact = dict(norm_rope=_exact_norm_rope, norm_rope_grad=_exact_norm_rope_grad, cache_write=_exact_write,
              cache_write_read=_exact_write_read, tree=_exact_tree)
