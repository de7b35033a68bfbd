"""The serving operators of this library as they are measured: planning, writing and attending over an 8-bit cache.

Three operators, one after the other in a serving step:

plan    block tables and slot maps for the entries that a step adds, from the requests' lengths;
append  rows into the cache: e4m3 with one power-of-two scale per block of tokens;
attn    heavily compressed attention of a step's query tokens over the cache: a sliding window of raw rows and the
        completed compressed entries, one softmax, one shared kv head that is both key and value.

``run`` computes them in plain torch, or with ``own`` set through the library's entry points.
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
MIN_SCALE_EXP = -96  # smallest block scale is 2^-96


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    def plan(name, **k):
        return dict(dict(name=name, op="plan"), **k)

    def append(name, **k):
        return dict(dict(name=name, op="append"), **k)

    def attn(name, **k):
        return dict(dict(dict(name=name, op="attn", t_lo=1, t_hi=1, m=128, W=128, bs=64, dtype="bf16", comp=True), **k))

    return [
        # one decode step of a batch: a token each, raw rows kept in a ring of blocks behind the window
        plan("plan-decode", R=64, len_lo=1000, len_hi=60000, add_lo=1, add_hi=1, bs=64, m=1, cols=4),
        # a mixed step of a large batch: some requests prefill a chunk, compressed entries of ratio 4
        plan("plan-mixed", R=509, len_lo=0, len_hi=30000, add_lo=1, add_hi=777, bs=16, m=4, cols=512),
        # admission of long prompts: about a million raw rows at once
        plan("plan-prompts", R=16, len_lo=0, len_hi=0, add_lo=30001, add_hi=100003, bs=64, m=1, cols=2048),
        # one decode step's rows: one row for each request, in the middle of its block
        append("append-decode", R=64, t_lo=1, t_hi=1, D=128, bs=64, dtype="bf16"),
        # a prefill of packed prompts
        append("append-prefill", R=8, t_lo=4001, t_hi=12345, D=128, bs=64, dtype="bf16"),
        # short ragged requests in fp32, small rows and blocks
        append("append-fp32", R=31, t_lo=1, t_hi=97, D=64, bs=16, dtype="fp32"),
        # one user, short context: latency
        attn("attn-single", R=1, H=64, D=128, len_lo=8191, len_hi=8191),
        # decode of a batch, compression ratio 128
        attn("attn-decode", R=64, H=64, D=128, len_lo=8000, len_hi=131072),
        # decode with compression ratio 4, every entry attended: the longest caches
        attn("attn-ratio4", R=64, H=64, D=128, len_lo=60000, len_hi=131072, m=4),
        # several tokens a request (speculative decoding), head dim 64, ragged
        attn("attn-spec", R=37, H=16, D=64, len_lo=3, len_hi=20000, t_lo=1, t_hi=4, m=16, W=64, bs=32),
        # chunked prefill over a long cache
        attn("attn-chunk", R=3, H=64, D=128, len_lo=2001, len_hi=50000, t_lo=700, t_hi=1001),
        # fp32 arithmetic on a small model's sizes
        attn("attn-fp32", R=8, H=4, D=64, len_lo=50, len_hi=4000, t_lo=1, t_hi=2, m=16, W=64, bs=16, dtype="fp32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "attn", "attn"])
    bs = rng.choice([16, 32, 64, 128])
    if op == "plan":
        m = rng.choice([1, 4, 16, 128])
        R = _log_int(rng, 1, 700)
        add_hi = _log_int(rng, 1, max(2, 900000 // R))
        len_hi = _log_int(rng, 1, 100000)
        full = (len_hi + add_hi) // m // bs + 1
        ring = rng.random() < 0.4
        cols = rng.randint(1, min(full, 8)) if ring else full
        return dict(op="plan", R=R, len_lo=0, len_hi=len_hi, add_lo=rng.randint(0, min(1, add_hi)), add_hi=add_hi, bs=bs, m=m,
                    cols=cols)
    if op == "append":
        R = _log_int(rng, 1, 200)
        t_hi = _log_int(rng, 1, max(2, 60000 // R))
        return dict(op="append", R=R, t_lo=1, t_hi=t_hi, D=rng.choice([64, 128]), bs=bs, dtype=rng.choice(["bf16", "bf16", "fp32"]))
    top = max(_cost(c) for c in listed() if c["op"] == "attn")
    while True:
        fp32 = rng.random() < 0.2
        m = rng.choice([4, 16, 128])
        H = rng.choice([1, 3, 4, 8]) if fp32 else rng.choice([1, 5, 8, 16, 24, 32, 64, 64, 96, 128])
        R = _log_int(rng, 1, 8 if fp32 else 100)
        len_hi = _log_int(rng, 2, 5000 if fp32 else 131072)
        t_hi = 1 if rng.random() < 0.6 else _log_int(rng, 1, 4 if fp32 else 300)
        c = dict(op="attn", R=R, H=H, D=rng.choice([64, 128]), len_lo=rng.randint(0, len_hi), len_hi=len_hi, t_lo=1, t_hi=t_hi, m=m,
                 W=rng.choice([1, 64, 128, 500]), bs=bs, dtype="fp32" if fp32 else "bf16", comp=rng.random() < 0.8)
        if _cost(c) <= top and _scores(c) <= 1.5e9:
            return c


def _spread(lo, hi, n, salt):
    """n whole numbers in [lo, hi], the same ones for a case every time."""
    return [lo + int((hi - lo + 1) * ((i * 0.6180339887498949 + salt) % 1.0)) for i in range(n)]


def _lengths(c):
    """(tokens held before the step, tokens added by it) of every request."""
    held = _spread(c["len_lo"], c["len_hi"], c["R"], 0.13) if c["op"] != "append" else _spread(0, 4 * c["bs"], c["R"], 0.13)
    lo, hi = (c["add_lo"], c["add_hi"]) if c["op"] == "plan" else (c["t_lo"], c["t_hi"])
    return held, _spread(lo, hi, c["R"], 0.57)


def _cost(c):
    w = work(c)
    return max(w["bytes"] / 6.8e12, w["flops"] / 1.9e15)


def _scores(c):
    """Elements of the plain form's score matrix."""
    held, add = _lengths(c)
    t = max(add)
    keys = c["W"] - 1 + t + (max(h + a for h, a in zip(held, add)) // c["m"] if c["comp"] else 0)
    return c["R"] * t * c["H"] * keys


def _entries(held, add, m):
    return [(h + a) // m - h // m for h, a in zip(held, add)]


def work(case):
    """What a pass cannot do without: every input it needs read once, every output written once."""
    c = case
    held, add = _lengths(c)
    if c["op"] == "plan":
        new = _entries(held, add, c["m"])
        blocks = sum(_nblocks((h + a) // c["m"], c) - _nblocks(h // c["m"], c) for h, a in zip(held, add))
        return {"bytes": 8 * c["R"] + 4 * (c["R"] + 1) + 4 * sum(new) + 8 * blocks + 8, "flops": 0}
    if c["op"] == "append":
        n = sum(add)
        blocks = sum((h + a - 1) // c["bs"] - h // c["bs"] + 1 for h, a in zip(held, add) if a)
        return {"bytes": n * c["D"] * (_esize(c) + 1) + 4 * n + 4 * blocks, "flops": 2 * n * c["D"]}
    n, rows, pairs = sum(add), 0, 0
    for h, a in zip(held, add):
        ncomp = (h + a) // c["m"] if c["comp"] else 0
        rows += min(h, c["W"] - 1) + a + ncomp
        for i in range(h, h + a):
            pairs += min(i + 1, c["W"]) + ((i + 1) // c["m"] if c["comp"] else 0)
    nbytes = rows * c["D"] + 8 * (rows // c["bs"]) + n * c["H"] * (2 * c["D"] * _esize(c) + 4) + 8 * c["R"]
    return {"bytes": nbytes, "flops": 4 * c["D"] * c["H"] * pairs}


def _esize(c):
    return 4 if c["dtype"] == "fp32" else 2


def _dtype(c):
    return torch.float32 if c["dtype"] == "fp32" else torch.bfloat16


def _nblocks(entries, c):
    return min(-(-entries // c["bs"]), c["cols"])


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _pow2_scale(amax):
    """Smallest power of two s with amax <= 448 s (fp32 in, fp32 out)."""
    mant, exp = torch.frexp(amax)
    e = torch.where(mant <= 0.875, exp - 9, exp - 8)
    e = torch.where(amax > 0, e, torch.full_like(e, MIN_SCALE_EXP)).clamp(min=MIN_SCALE_EXP)
    return torch.ldexp(torch.ones_like(amax), e)


def _random_blocks(n, bs, D, g):
    """n cache blocks of N(0, 1) rows with a spread of magnitudes, and their scales."""
    pool = torch.empty(n, bs, D, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(n, dtype=torch.float32, device="cuda")
    for a in range(0, n, 4096):
        b = min(n, a + 4096)
        x = torch.randn(b - a, bs, D, generator=g, device="cuda")
        x *= torch.exp2(torch.randint(-1, 2, (b - a, 1, 1), generator=g, device="cuda").float())
        s = _pow2_scale(x.abs().amax(dim=(1, 2)))
        pool[a:b] = (x / s[:, None, None]).to(torch.float8_e4m3fn)
        scale[a:b] = s
    return pool, scale


def _spill(pool, table, entries, cols):
    """Rows of each request's last block behind its last entry: whatever was there, NaN among it."""
    bs = pool.shape[1]
    for r, e in enumerate(entries):
        if e % bs and e <= cols * bs:
            pool.view(torch.uint8)[int(table[r, (e - 1) // bs % cols]), e % bs:] = 0x7F


def _tables(entries, cols, bs, perm):
    """Block tables (host) for requests of so many entries, blocks taken from perm."""
    table = np.full((len(entries), cols), -1, dtype=np.int32)
    at = 0
    for r, e in enumerate(entries):
        n = min(-(-e // bs), cols)
        table[r, :n] = perm[at:at + n]
        at += n
    return table


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    held, add = _lengths(c)
    rng = np.random.RandomState(seed % (2 ** 31))
    st = dict(op=c["op"], bs=c["bs"], held=_int32(held), added=_int32(add), R=c["R"])
    if c["op"] == "plan":
        e0 = [h // c["m"] for h in held]
        new = _entries(held, add, c["m"])
        used = sum(_nblocks(e, c) for e in e0)
        need = sum(_nblocks(e + n, c) - _nblocks(e, c) for e, n in zip(e0, new))
        nblocks = used + need + 100
        perm = rng.permutation(nblocks).astype(np.int32)
        st.update(m=c["m"], cols=c["cols"], nblocks=nblocks, nslots=max(1, sum(new) + 5),
                  table=torch.from_numpy(_tables(e0, c["cols"], c["bs"], perm)).cuda(),
                  free=torch.from_numpy(perm[used:].copy()).cuda(), free_count=_int32([nblocks - used]))
        return st
    if c["op"] == "append":
        # blocks in random order; a request's first new row may sit in the middle of a block that holds earlier rows
        cols = [-(-(h + a) // c["bs"]) for h, a in zip(held, add)]
        nblocks = sum(cols) + 7
        table = _tables([h + a for h, a in zip(held, add)], max(cols), c["bs"], rng.permutation(nblocks))
        slots = np.concatenate([table[r, np.arange(h, h + a) // c["bs"]] * c["bs"] + np.arange(h, h + a) % c["bs"]
                                for r, (h, a) in enumerate(zip(held, add))])
        slots = np.concatenate([slots, np.full(3, -1)]).astype(np.int32)  # the step's rows are padded
        pool, scale = _random_blocks(nblocks, c["bs"], c["D"], g)
        x = torch.randn(len(slots), c["D"], generator=g, device="cuda")
        x *= torch.exp2(torch.randint(-1, 3, (len(slots), 1), generator=g, device="cuda").float())
        st.update(x=x.to(_dtype(c)), slots=torch.from_numpy(slots).cuda(), pool=pool, scale=scale)
        return st
    # attn: the cache already holds the step's own rows
    total = [h + a for h, a in zip(held, add)]
    cols = min(-(-max(total) // c["bs"]), -(-(c["W"] - 1 + max(add)) // c["bs"]) + 1)
    nraw = sum(min(-(-t // c["bs"]), cols) for t in total) + 3
    table = _tables(total, cols, c["bs"], rng.permutation(nraw))
    pool, scale = _random_blocks(nraw, c["bs"], c["D"], g)
    _spill(pool, table, total, cols)
    st.update(raw=(pool, scale, torch.from_numpy(table).cuda()), comp=None, W=c["W"], m=c["m"])
    st["max_comp"] = 0
    if c["comp"]:
        ent = [t // c["m"] for t in total]
        cols = max(1, -(-max(ent) // c["bs"]))
        ncomp = sum(-(-e // c["bs"]) for e in ent) + 3
        table = _tables(ent, cols, c["bs"], rng.permutation(ncomp))
        pool, scale = _random_blocks(ncomp, c["bs"], c["D"], g)
        _spill(pool, table, ent, cols)
        st["comp"] = (pool, scale, torch.from_numpy(table).cuda())
        st["max_comp"] = max(ent)
    q = torch.randn(sum(add), c["H"], c["D"], generator=g, device="cuda")
    q *= torch.exp2(2 * torch.rand(1, c["H"], 1, generator=g, device="cuda") - 0.5)  # flat and peaked heads
    st.update(q=q.to(_dtype(c)), start=_int32(np.concatenate([[0], np.cumsum(add)]).tolist()), max_new=max(add),
              softmax_scale=1.0 / math.sqrt(c["D"]))
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    if own:
        return _run_own(state)
    return {"plan": _plain_plan, "append": _plain_append, "attn": _plain_attn}[state["op"]](state)


def _run_own(st):
    from block_sparse_compressed_gb300 import hca
    if st["op"] == "plan":
        start, slots, left = hca.hca_cache_plan(st["held"], st["added"], st["table"], st["free"], st["free_count"], st["nblocks"],
                                                st["bs"], st["nslots"], m=st["m"])
        return {"start": start, "slots": slots, "free_count": left, "table": st["table"]}
    if st["op"] == "append":
        hca.hca_cache_append(st["x"], st["slots"], st["pool"], st["scale"])
        return {"pool": st["pool"], "scale": st["scale"]}
    out, lse = hca.hca_cache_attn(st["q"], st["start"], st["held"], st["raw"], st["comp"], st["W"], st["m"], st["softmax_scale"])
    return {"out": out, "lse": lse}


def _plain_plan(st):
    bs, cols, m = st["bs"], st["cols"], st["m"]
    e0 = torch.div(st["held"], m, rounding_mode="floor").long()
    e1 = torch.div(st["held"] + st["added"], m, rounding_mode="floor").long()
    zero = torch.zeros(1, dtype=torch.long, device=e0.device)
    start = torch.cat([zero, torch.cumsum(e1 - e0, 0)])
    n0 = ((e0 + bs - 1) // bs).clamp(max=cols)
    n1 = ((e1 + bs - 1) // bs).clamp(max=cols)
    taken = torch.cat([zero, torch.cumsum(n1 - n0, 0)])
    col = torch.arange(cols, device=e0.device)[None, :]
    k = st["free_count"].long() - 1 - (taken[:-1, None] + col - n0[:, None])
    fresh = st["free"][k.clamp(0, st["free"].numel() - 1)]
    table = torch.where((col >= n0[:, None]) & (col < n1[:, None]), fresh, st["table"])
    st["table"].copy_(table)
    i = torch.arange(st["nslots"], device=e0.device)
    r = torch.searchsorted(start[1:], i, right=True)
    live = r < st["R"]
    r = r.clamp(max=st["R"] - 1)
    e = e0[r] + i - start[r]
    live &= (e1[r] - 1) // bs - e // bs < cols  # else a later new entry takes the row
    slot = table[r, (e // bs) % cols].long() * bs + e % bs
    slots = torch.where(live, slot, torch.full_like(slot, -1))
    return {"start": start.int(), "slots": slots.int(), "free_count": (st["free_count"] - taken[-1]).int(), "table": st["table"]}


def _plain_append(st):
    x, slots, pool, scale = st["x"].float(), st["slots"].long(), st["pool"], st["scale"]
    nblocks, bs, D = pool.shape
    live = torch.nonzero(slots >= 0)[:, 0]
    x, slots = x[live], slots[live]
    blk, off = slots // bs, slots % bs
    row = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(1)
    amax = torch.zeros(nblocks, device=x.device).scatter_reduce(0, blk, row, "amax")
    first = torch.full((nblocks,), bs, dtype=torch.long, device=x.device).scatter_reduce(0, blk, off, "amin")
    need = _pow2_scale(amax)
    new = torch.where(first == 0, need, torch.maximum(scale, need))
    new = torch.where(first < bs, new, scale)
    grown = torch.nonzero((first > 0) & (first < bs) & (new > scale))[:, 0]
    old = pool[grown].float() * (scale[grown] / new[grown])[:, None, None]
    keep = torch.arange(bs, device=x.device)[None, :] < first[grown][:, None]
    rows = (grown[:, None] * bs + torch.arange(bs, device=x.device)[None, :])[keep]
    flat = pool.view(torch.uint8).view(nblocks * bs, D)
    flat[rows] = old[keep].to(torch.float8_e4m3fn).view(torch.uint8)
    flat[slots] = (x / new[blk][:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    scale.copy_(new)
    return {"pool": pool, "scale": scale}


def _gather(cache, col, row, ok):
    """Rows of a paged cache as fp32: table column and row in block of every (request, key), zero where not ok."""
    pool, scale, table = cache
    nblocks, bs, D = pool.shape
    blk = torch.gather(table.long(), 1, torch.where(ok, col, torch.zeros_like(col)))
    blk = torch.where(ok, blk, torch.zeros_like(blk))
    idx = blk * bs + torch.where(ok, row, torch.zeros_like(row))
    x = pool.view(torch.uint8).view(nblocks * bs, D)[idx].view(torch.float8_e4m3fn).float()
    return torch.where(ok[..., None], x * scale[blk][..., None], torch.zeros_like(x))


def _plain_attn(st):
    q, start, held, W, m, bs = st["q"], st["start"].long(), st["held"].long(), st["W"], st["m"], st["bs"]
    N, H, D = q.shape
    R, T, dev = st["R"], st["max_new"], q.device
    new = start[1:] - start[:-1]
    t = torch.arange(T, device=dev)[None, :]
    there = t < new[:, None]
    tok = torch.where(there, start[:-1, None] + t, torch.zeros_like(start[:-1, None] + t))
    pos = held[:, None] + t  # [R, T]
    lo = (held - W + 1).clamp(min=0)
    key = lo[:, None] + torch.arange(W - 1 + T, device=dev)[None, :]
    ok = key < (held + new)[:, None]
    kv = _gather(st["raw"], (key // bs) % st["raw"][2].shape[1], key % bs, ok)
    vis = ok[:, None, :] & (key[:, None, :] <= pos[:, :, None]) & (key[:, None, :] > pos[:, :, None] - W)
    if st["comp"] is not None and st["max_comp"]:
        ent = torch.arange(st["max_comp"], device=dev)[None, :].expand(R, -1)
        ok = ent < ((held + new) // m)[:, None]
        kv = torch.cat([kv, _gather(st["comp"], ent // bs, ent % bs, ok)], 1)
        vis = torch.cat([vis, ok[:, None, :] & ((ent[:, None, :] + 1) * m <= pos[:, :, None] + 1)], 2)
    qf = q.float()[tok].reshape(R, T * H, D)
    s = torch.matmul(qf, kv.transpose(1, 2)).view(R, T, H, -1) * st["softmax_scale"]
    s = s.masked_fill(~vis[:, :, None, :], -math.inf)
    top = s.amax(3, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(3, keepdim=True)
    out = torch.matmul(p.view(R, T * H, -1), kv).view(R, T, H, D) / total
    lse = (top + torch.log(total))[..., 0]
    r = torch.searchsorted(start[1:], torch.arange(N, device=dev), right=True)
    k = torch.arange(N, device=dev) - start[r]
    return {"out": out[r, k].to(q.dtype), "lse": lse[r, k]}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    return {"plan": _exact_plan, "append": _exact_append, "attn": _exact_attn}[st["op"]](st)


def _exact_plan(st):
    held, added, table = (st[k].cpu().numpy().astype(np.int64) for k in ("held", "added", "table"))
    free, left = st["free"].cpu().numpy(), int(st["free_count"])
    bs, cols, m = st["bs"], st["cols"], st["m"]
    start, slots = [0], []
    for r in range(st["R"]):
        a, b = held[r] // m, (held[r] + added[r]) // m
        for j in range(min(-(-a // bs), cols), min(-(-b // bs), cols)):
            left -= 1
            table[r, j] = free[left]
        e = np.arange(a, b)
        s = table[r, (e // bs) % cols] * bs + e % bs
        slots.append(np.where((b - 1) // bs - e // bs >= cols, -1, s))
        start.append(start[-1] + b - a)
    slots = np.concatenate(slots)
    slots = np.concatenate([slots, np.full(st["nslots"] - len(slots), -1)])
    return {"start": np.array(start, np.int32), "slots": slots.astype(np.int32), "free_count": np.array([left], np.int32),
            "table": table.astype(np.int32)}


def _e4m3_values(v):
    """Nearest e4m3 value, ties to even, of doubles of magnitude up to 448."""
    a = np.abs(v)
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(a, 1e-300))), -6.0) - 3.0)
    return np.sign(v) * np.rint(a / step) * step


def _exact_append(st):
    x, slots = st["x"].double().cpu().numpy(), st["slots"].cpu().numpy()
    pool, scale = st["pool"].double().cpu().numpy(), st["scale"].double().cpu().numpy()
    bs = pool.shape[1]
    i = 0
    while i < len(slots):
        j = i + 1
        if slots[i] < 0:
            i = j
            continue
        while j < len(slots) and slots[j] == slots[j - 1] + 1 and slots[j] % bs:
            j += 1
        b, o = divmod(int(slots[i]), bs)
        amax = np.abs(x[i:j]).max()
        s = 2.0 ** max(math.ceil(math.log2(amax / E4M3_MAX)) if amax > 0 else MIN_SCALE_EXP, MIN_SCALE_EXP)
        if o and s > scale[b]:
            pool[b, :o] = _e4m3_values(pool[b, :o] * (scale[b] / s))
        scale[b] = max(s, scale[b]) if o else s
        pool[b, o:o + j - i] = _e4m3_values(x[i:j] / scale[b])
        i = j
    return {"pool": pool, "scale": scale}


def _exact_attn(st):
    start, held = st["start"].tolist(), st["held"].tolist()
    q, W, m, bs = st["q"].double(), st["W"], st["m"], st["bs"]
    outs, lses = [], []

    def rows(cache, r, e):
        pool, scale, table = cache
        blk = table[r].long()[(e // bs) % table.shape[1]]
        return pool[blk].double()[torch.arange(len(e), device=e.device), e % bs] * scale[blk].double()[:, None]

    def rows_in_parts(cache, r, e):
        return torch.cat([rows(cache, r, p) for p in e.split(8192)]) if len(e) else q.new_zeros(0, q.shape[2])

    for r in range(st["R"]):
        a, b = start[r], start[r + 1]
        if a == b:
            continue
        last = held[r] + b - a
        pos = torch.arange(held[r], last, device=q.device)[:, None]
        raw = torch.arange(max(0, held[r] - W + 1), last, device=q.device)
        ent = torch.arange(last // m if st["comp"] is not None else 0, device=q.device)
        kv = rows_in_parts(st["raw"], r, raw)
        vis = (raw[None, :] <= pos) & (pos - raw[None, :] < W)
        if len(ent):
            kv = torch.cat([kv, rows_in_parts(st["comp"], r, ent)])
            vis = torch.cat([vis, ent[None, :] * m + m - 1 <= pos], 1)
        s = torch.einsum("thd,kd->thk", q[a:b], kv) * st["softmax_scale"]
        s = torch.where(vis[:, None, :], s, torch.full_like(s, -math.inf))
        lse = torch.logsumexp(s, 2)
        outs.append(torch.einsum("thk,kd->thd", torch.exp(s - lse[..., None]), kv))
        lses.append(lse)
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
