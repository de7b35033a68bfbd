"""More operators of this library as they are measured: norms with positions, and attention over shared prefixes.

norm      what stands between a layer's projections and its attention: each head's query and the shared kv row are
          normalised (root mean square, optional weights) and some of their columns rotated by the token's position;
          forward, backward, and the serving form over the packed tokens of a step;
rope      the rotation alone: kv is key and value at once, so each head's output is turned back by its query's position;
shared    heavily compressed attention over the 8-bit cache for requests that begin with the same compressed entries,
          which are attended once for all of them.

``run`` computes them in plain torch, or with ``own`` set through the library's entry points.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
BASE = 10000.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    def norm(name, **k):
        return dict(dict(dict(name=name, op="norm", way="fwd", B=1, H=64, S=1, D=128, rot=64, axes=1, halves=False, weight=True,
                              dtype="bf16"), **k))

    def packed(name, op, **k):
        return dict(dict(dict(name=name, op=op, way="serve", H=64, D=128, rot=64, axes=1, halves=False, weight=True, dtype="bf16",
                              t_lo=1, t_hi=1), **k))

    def shared(name, **k):
        return dict(dict(dict(name=name, op="shared", H=64, D=128, t_lo=1, t_hi=1, m=128, W=128, bs=64, dtype="bf16"), **k))

    return [
        # one layer of a long training sequence, the sizes of this library's headline benchmark: queries as the projection leaves them
        norm("norm-train", S=65536),
        # its gradient
        norm("norm-train-bwd", S=65536, way="bwd"),
        # fp32 training of a small model, all columns rotated in halves, odd length
        norm("norm-bwd-fp32", B=2, H=8, S=4093, D=64, rot=64, halves=True, dtype="fp32", way="bwd"),
        # video tokens: time, height and width each have a third of the frequencies
        norm("norm-axes", B=3, H=16, S=9241, D=64, rot=48, axes=3, weight=False),
        # a decode step of a batch, a token each
        packed("norm-decode", "norm", R=64, len_lo=8000, len_hi=131072),
        # chunks of long prompts
        packed("norm-prefill", "norm", R=3, len_lo=2001, len_hi=50000, t_lo=700, t_hi=1001),
        # the attention's output of a training sequence, turned back and brought into the output projection's order
        norm("rope-train", op="rope", S=16384, way="train"),
        # the same for a decode step
        packed("rope-decode", "rope", R=64, len_lo=8000, len_hi=131072),
        # a decode step at compression ratio 128: two system prompts and some requests without one
        shared("shared-decode", prefix="40x16 8x0 16x9", len_lo=500, len_hi=8000),
        # a decode step of a batch over one long document at ratio 4
        shared("shared-ratio4", prefix="64x390", len_lo=100, len_hi=4000, m=4),
        # chunks of prompts that go on from the same document
        shared("shared-chunk", prefix="3x156", len_lo=0, len_hi=5000, t_lo=700, t_hi=1001, m=4),
        # fp32 arithmetic on a small model's sizes, one or two tokens a request
        shared("shared-fp32", prefix="5x15 3x4", H=4, D=64, len_lo=0, len_hi=700, t_hi=2, m=16, W=64, bs=16, dtype="fp32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm", "rope", "shared", "shared", "shared"])
    top = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        fp32 = rng.random() < 0.3
        c = dict(op=op, dtype="fp32" if fp32 else "bf16")
        if op == "shared":
            c.update(H=rng.choice([1, 3, 4, 8]) if fp32 else rng.choice([1, 5, 8, 16, 24, 32, 64, 64, 128]), D=rng.choice([64, 128]),
                     t_lo=1, t_hi=1 if rng.random() < 0.6 else _log_int(rng, 1, 4 if fp32 else 300), m=rng.choice([4, 16, 128]),
                     W=rng.choice([1, 64, 128, 500]), bs=rng.choice([16, 32, 64, 128]))
            pages = (3000 if fp32 else 30000) // c["bs"]
            c["prefix"] = " ".join("%dx%d" % (_log_int(rng, 1, 8 if fp32 else 90), rng.choice([0, 1, 1, 1]) * _log_int(rng, 1, pages))
                                   for _ in range(rng.choice([1, 1, 2, 4])))
            c["len_hi"] = _log_int(rng, 1, 6000)
            c["len_lo"] = rng.randint(0, c["len_hi"])
            if _scores(c) > 3e9:
                continue
        else:
            D = rng.choice([32, 64, 64, 72, 128, 128, 192, 256, 512])
            c.update(H=_log_int(rng, 1, 128), D=D, rot=16 * rng.randint(1, min(D, 128) // 16), axes=rng.choice([1, 1, 1, 2, 3]),
                     halves=rng.random() < 0.4, weight=rng.random() < 0.7)
            if rng.random() < 0.4:
                c.update(way="serve", R=_log_int(rng, 1, 300), len_hi=_log_int(rng, 1, 1000000), t_lo=1, t_hi=_log_int(rng, 1, 1000))
                c["len_lo"] = rng.randint(0, c["len_hi"])
            else:
                c.update(way="train" if op == "rope" else rng.choice(["fwd", "bwd"]), B=_log_int(rng, 1, 16), S=_log_int(rng, 1, 65536))
        if _cost(c) <= top:
            return c


def _spread(lo, hi, n, salt):
    """n whole numbers in [lo, hi], the same ones for a case every time."""
    return [lo + int((hi - lo + 1) * ((i * 0.6180339887498949 + salt) % 1.0)) for i in range(n)]


def _prefixes(c):
    """(requests, common columns of their compressed tables) of every prefix."""
    return [tuple(int(v) for v in p.split("x")) for p in c["prefix"].split()]


def _requests(c):
    return sum(n for n, _ in _prefixes(c)) if c["op"] == "shared" else c["R"]


def _lengths(c):
    """(tokens held before the step, tokens added by it) of every request; a prefix's tokens are held."""
    held = _spread(c["len_lo"], c["len_hi"], _requests(c), 0.13)
    if c["op"] == "shared":
        tokens = [cols * c["bs"] * c["m"] for n, cols in _prefixes(c) for _ in range(n)]
        held = [h + t for h, t in zip(held, tokens)]
    return held, _spread(c["t_lo"], c["t_hi"], _requests(c), 0.57)


def _tokens(c):
    return sum(_lengths(c)[1]) if c["way"] == "serve" else c["B"] * c["S"]


def _cost(c):
    w = work(c)
    return max(w["bytes"] / 6.8e12, w["flops"] / 1.9e15)


def _scores(c):
    """Elements of the plain form's score matrices."""
    held, add = _lengths(c)
    n, at = 0, 0
    for k, cols in _prefixes(c):
        n += sum(add[at:at + k]) * c["H"] * cols * c["bs"]
        at += k
    return n + len(add) * max(add) * c["H"] * (c["W"] + max(add) + _most_own(c))


def _own_entries(c):
    held, add = _lengths(c)
    skip = [cols * c["bs"] for n, cols in _prefixes(c) for _ in range(n)]
    return [(h + a) // c["m"] - s for h, a, s in zip(held, add, skip)]


def _most_own(c):
    return max(_own_entries(c))


def work(case):
    """What a pass cannot do without: every input it needs read once, every output written once."""
    c = case
    if c["op"] != "shared":
        n, es = _tokens(c), _esize(c)
        heads = c["H"] + (1 if c["op"] == "norm" else 0)
        nbytes = (3 if c["way"] == "bwd" else 2) * n * heads * c["D"] * es
        nbytes += 8 * c["R"] if c["way"] == "serve" else 4 * n * c["axes"]
        if c["op"] == "norm" and c["weight"]:
            nbytes += (16 if c["way"] == "bwd" else 8) * c["D"]
        per = {"fwd": 4, "serve": 4, "bwd": 10, "train": 0}[c["way"]] if c["op"] == "norm" else 0
        return {"bytes": nbytes, "flops": n * heads * (per * c["D"] + 3 * c["rot"])}
    held, add = _lengths(c)
    n, rows, pairs = sum(add), sum(cols * c["bs"] for _, cols in _prefixes(c)), 0
    for h, a, e in zip(held, add, _own_entries(c)):
        rows += min(h, c["W"] - 1) + a + e
        for i in range(h, h + a):
            pairs += min(i + 1, c["W"]) + (i + 1) // c["m"]
    nbytes = rows * c["D"] + 8 * (rows // c["bs"]) + n * c["H"] * (2 * c["D"] * _esize(c) + 4) + 8 * len(add)
    return {"bytes": nbytes, "flops": 4 * c["D"] * c["H"] * pairs}


def _esize(c):
    return 4 if c["dtype"] == "fp32" else 2


def _dtype(c):
    return torch.float32 if c["dtype"] == "fp32" else torch.bfloat16


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _normal(g, *shape, dtype=torch.float32, spread=None):
    x = torch.randn(*shape, generator=g, device="cuda")
    return (x if spread is None else x.mul_(spread)).to(dtype)


def _frequencies(c):
    """[axes, rot/2]: each axis has its own share of the pairs, from fast to slow."""
    n = c["rot"] // 2
    f = torch.zeros(c["axes"], n)
    for a in range(c["axes"]):
        mine = torch.arange(a, n, c["axes"])
        f[a, mine] = BASE ** (-torch.arange(len(mine)) / max(1, len(mine)))
    return f.cuda()


def _coordinates(c):
    """[axes, B, S] positions: documents that begin anew, or frames of a video."""
    B, S = c["B"], c["S"]
    s = torch.arange(S, device="cuda").repeat(B, 1)
    if c["axes"] == 1:
        return (s - torch.where(s >= S // 3, S // 3, 0))[None].int().contiguous()
    w = max(1, math.isqrt(S // 4))
    parts = [s // (w * w), s // w % w, s % w] if c["axes"] == 3 else [s // w, s % w]
    return torch.stack(parts).int().contiguous()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if c["op"] == "shared":
        return _prepare_shared(c, seed, g)
    H, D, dt = c["H"], c["D"], _dtype(c)
    st = dict(op=c["op"], way=c["way"], halves=c["halves"], first=D - c["rot"], freq=_frequencies(c), wq=None, wkv=None)
    loud = torch.exp2(2 * torch.rand(H, 1, generator=g, device="cuda") - 1)  # heads of different magnitudes
    if c["op"] == "norm" and c["weight"]:
        st.update(wq=1 + 0.2 * _normal(g, D), wkv=1 + 0.2 * _normal(g, D))
    if c["way"] == "serve":
        held, add = _lengths(c)
        n = sum(add)
        st.update(held=_int32(held), start=_int32(np.concatenate([[0], np.cumsum(add)]).tolist()), pos=None)
        if c["axes"] > 1:
            st["pos"] = torch.randint(0, c["len_hi"] + 1, (c["axes"], n), generator=g, device="cuda", dtype=torch.int32)
        st["q"] = _normal(g, n, H, D, dtype=dt, spread=loud)
        if c["op"] == "norm":
            st["kv"] = _normal(g, n, D, dtype=dt)
        return st
    B, S = c["B"], c["S"]
    st["pos"] = _coordinates(c)
    if c["op"] == "rope":
        st["q"] = _normal(g, B, H, S, D, dtype=dt, spread=loud[:, None])  # as the attention writes it
        return st
    # as a projection writes them: token by token
    st["q"] = _normal(g, B, S, H, D, dtype=dt, spread=loud).transpose(1, 2)
    st["kv"] = _normal(g, B, S, D, dtype=dt)
    if c["way"] == "bwd":
        st["dq"] = _normal(g, B, H, S, D, dtype=dt, spread=loud[:, None])
        st["dkv"] = _normal(g, B, S, D, dtype=dt)
    return st


def _random_blocks(n, bs, D, g):
    """n cache blocks of N(0, 1) rows with a spread of magnitudes, and their scales: powers of two, as the cache writes them."""
    pool = torch.empty(n, bs, D, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(n, dtype=torch.float32, device="cuda")
    for a in range(0, n, 4096):
        b = min(n, a + 4096)
        x = torch.randn(b - a, bs, D, generator=g, device="cuda")
        x *= torch.exp2(torch.randint(-1, 2, (b - a, 1, 1), generator=g, device="cuda").float())
        s = torch.exp2(torch.ceil(torch.log2(x.abs().amax(dim=(1, 2)) / 448.0)))
        pool[a:b] = (x / s[:, None, None]).to(torch.float8_e4m3fn)
        scale[a:b] = s
    return pool, scale


def _prepare_shared(c, seed, g):
    held, add = _lengths(c)
    rng = np.random.RandomState(seed % (2 ** 31))
    bs, m, R = c["bs"], c["m"], len(held)
    total = [h + a for h, a in zip(held, add)]
    # raw rows in rings behind the windows
    cols = min(-(-max(total) // bs), -(-(c["W"] - 1 + max(add)) // bs) + 1)
    used = [min(-(-t // bs), cols) for t in total]
    perm = rng.permutation(sum(used) + 3)
    raw_table = np.full((R, cols), -1, dtype=np.int32)
    at = 0
    for r, n in enumerate(used):
        raw_table[r, :n] = perm[at:at + n]
        at += n
    raw = (*_random_blocks(len(perm), bs, c["D"], g), torch.from_numpy(raw_table).cuda())
    # compressed entries: a prefix's columns are the same blocks in all its requests
    pages = [-(-(t // m) // bs) for t in total]
    skip = [k for n, k in _prefixes(c) for _ in range(n)]
    nblocks = sum(k for _, k in _prefixes(c)) + sum(p - k for p, k in zip(pages, skip)) + 3
    perm = rng.permutation(nblocks)
    table = np.full((R, max(1, max(pages))), -1, dtype=np.int32)
    at, r = 0, 0
    for n, k in _prefixes(c):
        common = perm[at:at + k]
        at += k
        for _ in range(n):
            table[r, :k] = common
            table[r, k:pages[r]] = perm[at:at + pages[r] - k]
            at += pages[r] - k
            r += 1
    comp = (*_random_blocks(nblocks, bs, c["D"], g), torch.from_numpy(table).cuda())
    first = np.concatenate([[0], np.cumsum([n for n, _ in _prefixes(c)])]).tolist()
    start = np.concatenate([[0], np.cumsum(add)]).tolist()
    q = torch.randn(sum(add), c["H"], c["D"], generator=g, device="cuda")
    q *= torch.exp2(2 * torch.rand(1, c["H"], 1, generator=g, device="cuda") - 0.5)  # flat and peaked heads
    return dict(op="shared", held=_int32(held), start=_int32(start), first=_int32(first), cols=_int32([k for _, k in _prefixes(c)]),
                raw=raw, comp=comp, W=c["W"], m=m, softmax_scale=1.0 / math.sqrt(c["D"]), q=q.to(_dtype(c)),
                groups=[(first[i], first[i + 1], start[first[i]], start[first[i + 1]], k) for i, (_, k) in enumerate(_prefixes(c))],
                max_new=max(add), max_own=_most_own(c))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    if own:
        return _run_own(state)
    return {"norm": _plain_norm, "rope": _plain_rope, "shared": _plain_shared}[state["op"]](state)


def _run_own(st):
    from block_sparse_compressed_gb300 import hca
    if st["op"] == "shared":
        out, lse = hca.hca_cache_attn_shared(st["q"], st["start"], st["held"], st["raw"], st["comp"], st["first"], st["cols"], st["W"],
                                             st["m"], st["softmax_scale"])
        return {"out": out, "lse": lse}
    f, kw = st["freq"], dict(first=st["first"], halves=st["halves"])
    if st["op"] == "rope":
        if st["way"] == "serve":
            return {"y": hca.hca_cache_rope(st["q"], st["start"], st["held"], f, inverse=True, pos=st["pos"], **kw)}
        B, H, S, D = st["q"].shape
        y = torch.empty(B, S, H, D, dtype=st["q"].dtype, device=st["q"].device)
        hca.hca_rope(st["q"], st["pos"], f, inverse=True, y=y.transpose(1, 2), **kw)
        return {"y": y}
    if st["way"] == "serve":
        q, kv = hca.hca_cache_norm_rope(st["q"], st["kv"], st["start"], st["held"], st["wq"], st["wkv"], f, EPS, pos=st["pos"], **kw)
        return {"q": q, "kv": kv}
    if st["way"] == "fwd":
        q, kv = hca.hca_norm_rope_fwd(st["q"], st["kv"], st["wq"], st["wkv"], st["pos"], f, EPS, **kw)
        return {"q": q, "kv": kv}
    dq, dkv, dwq, dwkv = hca.hca_norm_rope_bwd(st["q"], st["kv"], st["wq"], st["wkv"], st["pos"], f, EPS, st["dq"], st["dkv"], **kw)
    return {"dq": dq, "dkv": dkv, "dwq": dwq, "dwkv": dwkv}


def _token_positions(st):
    """Positions of a step's packed tokens, [axes, N]."""
    if st["pos"] is not None:
        return st["pos"]
    n = st["q"].shape[0]
    t = torch.arange(n, device=st["q"].device)
    r = torch.searchsorted(st["start"][1:].long(), t, right=True)
    return (st["held"][r] + t - st["start"][r])[None]


def _turn(st, pos):
    """cos and sin of the angles [..., rot/2] of positions [axes, ...]: the angles in 64 bits."""
    a = torch.einsum("a...,ap->...p", pos.double(), st["freq"].double())
    return torch.cos(a).float(), torch.sin(a).float()


def _pairs(x, st):
    """The columns of x [..., D] in front of the rotated ones, both halves of the pairs, and the columns behind."""
    n, a = st["freq"].shape[1], st["first"]
    z = x[..., a:a + 2 * n]
    u, v = (z[..., :n], z[..., n:]) if st["halves"] else (z[..., 0::2], z[..., 1::2])
    return x[..., :a], u, v, x[..., a + 2 * n:]


def _rotate(x, st, cos, sin):
    a, u, v, b = _pairs(x, st)
    u, v = u * cos - v * sin, u * sin + v * cos
    z = torch.cat([u, v], -1) if st["halves"] else torch.stack([u, v], -1).flatten(-2)
    return torch.cat([a, z, b], -1)


def _norm(x, w):
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return y if w is None else y * w


def _norm_grad(x, w, g):
    """Gradients of _norm for the cotangent g."""
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    dw = None if w is None else (g * x * r).flatten(0, -2).sum(0, dtype=torch.float64).float()
    h = g if w is None else g * w
    return r * (h - x * (r * r * (h * x).mean(-1, keepdim=True))), dw


def _plain_norm(st):
    dt = st["q"].dtype
    if st["way"] == "serve":
        cos, sin = _turn(st, _token_positions(st))
        cq, sq = cos[:, None], sin[:, None]
    else:
        cos, sin = _turn(st, st["pos"])
        cq, sq = cos[:, None], sin[:, None]
    if st["way"] != "bwd":
        q = _rotate(_norm(st["q"].float(), st["wq"]), st, cq, sq).to(dt)
        return {"q": q, "kv": _rotate(_norm(st["kv"].float(), st["wkv"]), st, cos, sin).to(dt)}
    dq, dwq = _norm_grad(st["q"].float(), st["wq"], _rotate(st["dq"].float(), st, cq, -sq))
    dkv, dwkv = _norm_grad(st["kv"].float(), st["wkv"], _rotate(st["dkv"].float(), st, cos, -sin))
    return {"dq": dq.to(dt), "dkv": dkv.to(dt), "dwq": dwq, "dwkv": dwkv}


def _plain_rope(st):
    x = st["q"]
    if st["way"] == "serve":
        cos, sin = _turn(st, _token_positions(st))
        return {"y": _rotate(x.float(), st, cos[:, None], -sin[:, None]).to(x.dtype)}
    cos, sin = _turn(st, st["pos"])
    return {"y": _rotate(x.float(), st, cos[:, None], -sin[:, None]).to(x.dtype).transpose(1, 2).contiguous()}


def _rows(cache, blk, row, ok=None):
    """Rows of cache blocks as fp32, zero where not ok."""
    pool, scale, _ = cache
    nblocks, bs, D = pool.shape
    if ok is not None:
        blk, row = torch.where(ok, blk, torch.zeros_like(blk)), torch.where(ok, row, torch.zeros_like(row))
    x = pool.view(torch.uint8).view(nblocks * bs, D)[blk * bs + row].view(torch.float8_e4m3fn).float() * scale[blk][..., None]
    return x if ok is None else torch.where(ok[..., None], x, torch.zeros_like(x))


def _partial(s, kv):
    """Largest score, sum and weighted rows of scores [..., K] and keys [..., K, D]."""
    top = s.amax(-1, keepdim=True)
    s = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
    return top, s.sum(-1, keepdim=True), torch.matmul(s, kv)


def _plain_shared(st):
    q, start, held, W, m = st["q"], st["start"].long(), st["held"].long(), st["W"], st["m"]
    N, H, D = q.shape
    R, T, dev, bs = held.shape[0], st["max_new"], q.device, st["raw"][0].shape[1]
    scale, table = st["softmax_scale"], st["comp"][2].long()
    # each request's own keys: its window and the entries behind its prefix
    new = start[1:] - start[:-1]
    t = torch.arange(T, device=dev)[None, :]
    there = t < new[:, None]
    tok = torch.where(there, start[:-1, None] + t, torch.zeros_like(start[:-1, None] + t))
    pos = held[:, None] + t
    key = (held - W + 1).clamp(min=0)[:, None] + torch.arange(W - 1 + T, device=dev)[None, :]
    ok = key < (held + new)[:, None]
    raw_table = st["raw"][2].long()
    kv = _rows(st["raw"], torch.gather(raw_table, 1, key // bs % raw_table.shape[1]), key % bs, ok)
    vis = ok[:, None, :] & (key[:, None, :] <= pos[:, :, None]) & (key[:, None, :] > pos[:, :, None] - W)
    if st["max_own"] > 0:
        skip = torch.repeat_interleave(st["cols"].long() * bs, (st["first"][1:] - st["first"][:-1]).long(), output_size=R)
        ent = skip[:, None] + torch.arange(st["max_own"], device=dev)[None, :]
        ok = ent < ((held + new) // m)[:, None]
        blk = torch.gather(table, 1, torch.where(ok, ent // bs, torch.zeros_like(ent)))
        kv = torch.cat([kv, _rows(st["comp"], blk, ent % bs, ok)], 1)
        vis = torch.cat([vis, ok[:, None, :] & ((ent[:, None, :] + 1) * m <= pos[:, :, None] + 1)], 2)
    s = torch.matmul(q.float()[tok].reshape(R, T * H, D), kv.transpose(1, 2)).view(R, T, H, -1) * scale
    s = s.masked_fill(~vis[:, :, None, :], -math.inf).view(R, T * H, -1)
    top, total, o = _partial(s, kv)
    r = torch.searchsorted(start[1:], torch.arange(N, device=dev), right=True)
    k = torch.arange(N, device=dev) - start[r]
    top, total, o = (x.view(R, T, H, -1)[r, k] for x in (top, total, o))
    # the common entries, for all tokens of a prefix's requests at once
    for r0, _, a, b, cols in st["groups"]:
        if cols == 0:
            continue
        kv = _rows(st["comp"], table[r0, :cols, None], torch.arange(bs, device=dev)[None, :]).view(cols * bs, D)
        step = max(1, int(5e8) // (H * cols * bs))
        for i in range(a, b, step):
            j = min(b, i + step)
            s = torch.matmul(q[i:j].float().reshape(-1, D), kv.t()) * scale
            pt, ps, po = (x.view(j - i, H, -1) for x in _partial(s, kv))
            both = torch.maximum(pt, top[i:j])
            wp, wo = torch.exp(pt - both), torch.exp(top[i:j] - both)
            o[i:j] = o[i:j] * wo + po * wp
            total[i:j] = total[i:j] * wo + ps * wp
            top[i:j] = both
    return {"out": (o / total).to(q.dtype), "lse": (top + torch.log(total))[..., 0]}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "shared":
        return _exact_shared(st) if work(case)["flops"] < 6e12 else None
    return _exact_rows(st)


def _phases(st, pos):
    """exp(i theta) of positions [axes, ...]."""
    a = (pos.double()[..., None] * st["freq"].double().view(st["freq"].shape[0], *[1] * (pos.dim() - 1), -1)).sum(0)
    return torch.polar(torch.ones_like(a), a)


def _forward(x, w, e, st):
    """Rows of doubles, normalised where there is a norm, their pairs as complex numbers times e."""
    if st["op"] == "norm":
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
        if w is not None:
            x = x * w
    n, a = e.shape[-1], st["first"]
    z = x[..., a:a + 2 * n].unflatten(-1, (2, n) if st["halves"] else (n, 2))
    z = torch.view_as_complex((z.transpose(-1, -2) if st["halves"] else z).contiguous()) * e
    z = torch.view_as_real(z)
    return torch.cat([x[..., :a], (z.transpose(-1, -2) if st["halves"] else z).flatten(-2), x[..., a + 2 * n:]], -1)


def _exact_rows(st):
    """In slices of tokens; gradients by differentiating the forward."""
    serve, norm, grad = st["way"] == "serve", st["op"] == "norm", st["way"] == "bwd"
    q = st["q"].transpose(0, 1)[None] if serve else st["q"]  # [B, H, S, D]
    kv = None if not norm else st["kv"][None] if serve else st["kv"]
    pos = _token_positions(st)[:, None] if serve else st["pos"]
    out = {}
    step = max(1, int(6e7) // (q.shape[0] * q.shape[1] * q.shape[3]))
    for i in range(0, q.shape[2], step):
        e = _phases(st, pos[:, :, i:i + step])
        for name, x, w in (("q", q[:, :, i:i + step], st["wq"]), ("kv", kv[:, None, i:i + step] if norm else None, st["wkv"])):
            if x is None:
                continue
            x = x.double()
            phase = e[:, None] if norm else e[:, None].conj()
            if not grad:
                out.setdefault(name, []).append(_forward(x, w, phase, st))
                continue
            x.requires_grad_(True)
            wd = None if w is None else w.double().requires_grad_(True)
            g = st["d" + name]
            y = _forward(x, wd, phase, st)
            d = torch.autograd.grad(y, [x] if w is None else [x, wd], (g[:, :, i:i + step] if name == "q" else g[:, None, i:i + step]).double())
            out.setdefault("d" + name, []).append(d[0])
            if w is not None:
                out["dw" + name] = out["dw" + name] + d[1] if "dw" + name in out else d[1]
    res = {k: torch.cat(v, 2) if isinstance(v, list) else v for k, v in out.items()}
    for k in ("kv", "dkv"):
        if k in res:
            res[k] = res[k][:, 0]
    if serve:
        res = {k: v[0].transpose(0, 1) if k == "q" else v[0] for k, v in res.items()}
    if not norm:
        return {"y": res["q"] if serve else res["q"].transpose(1, 2)}
    if grad:
        res.setdefault("dwq", None)
        res.setdefault("dwkv", None)
        return {k: res[k] for k in ("dq", "dkv", "dwq", "dwkv")}
    return res


def _exact_shared(st):
    """Token by token over the table of its own request: nothing is shared here."""
    start, held = st["start"].tolist(), st["held"].tolist()
    q, W, m, bs = st["q"].double(), st["W"], st["m"], st["raw"][0].shape[1]

    def rows(cache, r, e):
        pool, scale, table = cache
        parts = []
        for p in e.split(8192):
            blk = table[r].long()[(p // bs) % table.shape[1]]
            parts.append(pool[blk, p % bs].double() * scale[blk].double()[:, None])
        return torch.cat(parts) if parts else q.new_zeros(0, q.shape[2])

    outs, lses = [], []
    for r in range(len(held)):
        a, b = start[r], start[r + 1]
        last = held[r] + b - a
        raw = torch.arange(max(0, held[r] - W + 1), last, device=q.device)
        ent = torch.arange(last // m, device=q.device)
        kv = torch.cat([rows(st["raw"], r, raw), rows(st["comp"], r, ent)])
        seen_from = torch.cat([raw, (ent + 1) * m - 1])
        seen_to = torch.cat([raw + W - 1, torch.full_like(ent, 1 << 40)])
        step = max(1, int(2e8) // (q.shape[1] * len(kv)))
        for i in range(a, b, step):
            pos = torch.arange(held[r] + i - a, held[r] + min(b, i + step) - a, device=q.device)[:, None, None]
            s = torch.einsum("thd,kd->thk", q[i:min(b, i + step)], kv) * st["softmax_scale"]
            s = torch.where((seen_from <= pos) & (pos <= seen_to), s, torch.full_like(s, -math.inf))
            lse = torch.logsumexp(s, 2)
            outs.append(torch.einsum("thk,kd->thd", torch.exp(s - lse[..., None]), kv))
            lses.append(lse)
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
