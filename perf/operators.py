"""Work of the 8-bit key/value cache operators: the cases, their plain forms and their 64-bit definition.

The cache holds S sequences.  A page is 64 tokens of one KV head: 8-bit codes (stored plus 128) with one fp32
scale for its keys and one for its values.  The rows of a page that is not complete yet stay in fp32 (`tail`).
`table[s][h]` is a permutation of the pages that (s, h) owns: page p of the sequence lives at table[s][h][p].
Inside a page the codes lie in the order in which one warp reads them (see _tile_keys and _tile_values).
"""
import math

import numpy as np
import torch

own = False

PAGE = 64
DEV = "cuda"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one token for each of 16 sequences of a served batch, some of them completing a page; the page is read back
        dict(name="append-step", op="append", seqs=16, kv_heads=8, group=4, dim=128, n=1, length=4095, ragged=True,
             dtype="fp32"),
        # a long prompt's rows of one layer go into an empty cache and come back out (saving, or handing over, a cache)
        dict(name="append-prompt", op="append", seqs=1, kv_heads=8, group=4, dim=128, n=32768, length=0, ragged=False,
             dtype="bf16"),
        # the smallest call: one token of a small model (14 query heads over 2 KV heads of 64) after 513 tokens
        dict(name="attend-small", op="attend", seqs=1, kv_heads=2, group=7, dim=64, n=1, length=513, ragged=False,
             dtype="fp32", mask="none", mass=False),
        # one greedy step of one layer of a model of 32 heads over 8 KV heads of 128, after 4095 tokens
        dict(name="attend-step", op="attend", seqs=1, kv_heads=8, group=4, dim=128, n=1, length=4095, ragged=False,
             dtype="fp32", mask="none", mass=False),
        # the verification of a draft tree of 16 nodes at the same place
        dict(name="attend-tree", op="attend", seqs=1, kv_heads=8, group=4, dim=128, n=16, length=4096, ragged=False,
             dtype="fp32", mask="tree", mass=False),
        # one token at the far end of a long context
        dict(name="attend-long", op="attend", seqs=1, kv_heads=8, group=4, dim=128, n=1, length=131071, ragged=False,
             dtype="bf16", mask="none", mass=False),
        # a served batch of 64 sequences of many lengths, one token each
        dict(name="attend-batch", op="attend", seqs=64, kv_heads=8, group=4, dim=128, n=1, length=8191, ragged=True,
             dtype="bf16", mask="none", mass=False),
        # a bucket of 64 prompt tokens deep in a prompt, with the weight that lands on each page (for eviction)
        dict(name="attend-bucket-mass", op="attend", seqs=1, kv_heads=8, group=4, dim=128, n=64, length=32000,
             ragged=False, dtype="bf16", mask="none", mass=True),
        # one token at the far end of a long context, reading the 64 pages that score best
        dict(name="sparse-long", op="sparse", seqs=1, kv_heads=8, group=4, dim=128, n=1, length=131071, ragged=False,
             dtype="fp32", top_k=64, first=1, last=2),
        # 16 sequences with four draft nodes each, 32 pages for each node
        dict(name="sparse-batch", op="sparse", seqs=16, kv_heads=8, group=4, dim=128, n=4, length=32767, ragged=True,
             dtype="bf16", top_k=32, first=1, last=1),
        # one sequence thinned to a quarter
        dict(name="evict-one", op="evict", seqs=1, kv_heads=8, dim=64, length=32777, ragged=False, keep=128, first=1,
             last=4),
        # a served batch thinned together
        dict(name="evict-batch", op="evict", seqs=32, kv_heads=8, dim=64, length=131000, ragged=True, keep=512,
             first=1, last=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "sparse", "sparse", "evict"])
    kv_heads, group, dim = rng.choice([(8, 4, 128), (2, 7, 64), (4, 8, 64), (1, 5, 128), (3, 1, 64), (4, 16, 128),
                                       (2, 2, 128)])
    dtype = rng.choice(["fp32", "bf16"])
    seqs = rng.choice([1, 1, 2, 3, _log(rng, 4, 48)])
    room = max(200, 131071 * 8 * 128 // (kv_heads * dim * seqs))  # no more cached values than the largest case has
    length = _log(rng, 1, min(room, 131071))
    c = dict(op=op, seqs=seqs, kv_heads=kv_heads, dim=dim, length=length, ragged=seqs > 1)
    if op == "append":
        step = rng.random() < 0.4
        c.update(group=group, n=1 if step else _log(rng, 1, min(room // 4, 32768)), dtype=dtype)
        c.update(length=length if step else 0, ragged=True)
    elif op == "attend":
        most = max(1, min(64, 2 ** 26 // (seqs * kv_heads * group * max(length, 64))))  # logits of the plain form
        n = min(rng.choice([1, 1, rng.randint(2, 16), rng.randint(17, 64)]), most)
        c.update(group=group, n=n, dtype=dtype, mask=rng.choice(["none", "tree"]) if n > 1 else "none",
                 mass=rng.random() < 0.3)
    elif op == "sparse":
        top_k = _log(rng, 4, 128)
        most = max(1, min(16, 2 ** 28 // (seqs * kv_heads * top_k * PAGE * dim)))  # rows the plain form gathers
        c.update(group=group, n=min(rng.choice([1, rng.randint(1, 16)]), most), dtype=dtype, top_k=top_k,
                 first=rng.randint(0, 2), last=rng.randint(0, 2))
    else:
        keep = _log(rng, 4, 1024)
        c.update(dim=64, length=min(length, 2 ** 27 // (seqs * kv_heads)),keep=keep, first=rng.randint(0, 2), last=rng.randint(0, 2))
    return c


# ------------------------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _lengths(case, g):
    S, L = case["seqs"], case["length"]
    if not case["ragged"]:
        return torch.full((S,), L, dtype=torch.int32, device=DEV)
    lens = torch.randint(0, L + 1, (S,), generator=g, device=DEV, dtype=torch.int32)
    lens[0] = L
    return lens


def _tile_keys(c):
    """[..., 64 tokens, D] -> [..., 64 * D]: 16-token tiles, 32-dim chunks, then token % 8, 8-dim groups, halves of
    four dims, token / 8, dim."""
    b, D = c.shape[:-2], c.shape[-1]
    o, k = len(b), c.reshape(*b, 4, 2, 8, D // 32, 4, 2, 4)
    return k.permute(*range(o), o, o + 3, o + 2, o + 4, o + 5, o + 1, o + 6).reshape(*b, PAGE * D)


def _untile_keys(c, D):
    b = c.shape[:-1]
    o, k = len(b), c.reshape(*b, 4, D // 32, 8, 4, 2, 2, 4)
    return k.permute(*range(o), o, o + 5, o + 2, o + 1, o + 3, o + 4, o + 6).reshape(*b, PAGE, D)


def _tile_values(c):
    """[..., 64 tokens, D] -> [..., 64 * D]: 16-dim tiles, 32-token chunks, then dim % 8, token pairs, 16-token
    halves, dim / 8, 8-token halves, token."""
    b, D = c.shape[:-2], c.shape[-1]
    o, v = len(b), c.reshape(*b, 2, 2, 2, 4, 2, D // 16, 2, 8)
    return v.permute(*range(o), o + 5, o, o + 7, o + 3, o + 1, o + 6, o + 2, o + 4).reshape(*b, PAGE * D)


def _untile_values(c, D):
    b = c.shape[:-1]
    o, v = len(b), c.reshape(*b, D // 16, 2, 8, 4, 2, 2, 2, 2)
    return v.permute(*range(o), o + 1, o + 4, o + 6, o + 3, o + 7, o, o + 5, o + 2).reshape(*b, PAGE, D)


def _cache(case, g, lens, extra, fill=True):
    """The tensors of a cache of the case's lengths: codes, scales, sums, tail, table, len, ctl."""
    S, H, D = case["seqs"], case["kv_heads"], case["dim"]
    P = max(1, (case["length"] + extra + PAGE - 1) // PAGE)
    codes = torch.empty(S, H, P, 2, PAGE * D, dtype=torch.uint8, device=DEV)
    sums = torch.zeros(S, H, P, D, dtype=torch.int16, device=DEV)
    if fill:
        drift = _randn(g, S, H, P, 1, D) * 10  # the keys of a page have something in common
        k = (_randn(g, S, H, P, PAGE, D) * 28 + drift).round_().clamp_(-127, 127)
        sums.copy_(k.sum(dim=3))
        codes[:, :, :, 0] = _tile_keys(k.add_(128).to(torch.uint8))
        k = (_randn(g, S, H, P, PAGE, D) * 32).round_().clamp_(-127, 127)
        codes[:, :, :, 1] = _tile_values(k.add_(128).to(torch.uint8))
        del k
    scales = torch.rand(S, H, P, 2, generator=g, device=DEV) * 0.02 + 0.02
    tail = _randn(g, S, H, 2, PAGE, D)
    table = torch.rand(S, H, P, generator=g, device=DEV).argsort(dim=-1).to(torch.int32)
    ctl = torch.zeros(1, dtype=torch.int32, device=DEV)
    return dict(codes=codes, scales=scales, sums=sums, tail=tail, table=table, len=lens.clone(), ctl=ctl)


def _tree_mask(g, S, n):
    """int64 [S][n]: bit j of entry i is set where node j is node i or one of its ancestors (random trees)."""
    parent = [(torch.rand(S, generator=g, device=DEV) * i).long() for i in range(n)]
    rows = [torch.ones(S, dtype=torch.int64, device=DEV)]
    for i in range(1, n):
        rows.append(torch.gather(torch.stack(rows, 1), 1, parent[i][:, None])[:, 0] | (1 << i if i < 63 else -(1 << 63)))
    return torch.stack(rows, 1)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    S, H, D = case["seqs"], case["kv_heads"], case["dim"]
    lens = _lengths(case, g)
    st = dict(case=dict(case))
    if op == "append":
        n = case["n"]
        st["cache"] = _cache(case, g, lens, n)
        st["k"], st["v"] = ((_randn(g, S, n, H, D) * (1 + i)).to(TYPES[case["dtype"]]) for i in range(2))
        st["counts"] = torch.randint((n + 1) // 2, n + 1, (S,), generator=g, device=DEV, dtype=torch.int32)
        st["len_out"] = torch.zeros_like(lens)
        st["first"] = (lens // PAGE * PAGE).to(torch.int32)
        st["rows"] = n if case["length"] == 0 else n + PAGE - 1
    elif op in ("attend", "sparse"):
        n, Hq, t = case["n"], case["kv_heads"] * case["group"], TYPES[case["dtype"]]
        st["cache"] = _cache(case, g, lens, 0)
        st["q"] = (_randn(g, S, n, Hq, D) * 2).to(t)
        st["k"], st["v"] = (_randn(g, S, n, H, D).to(t) for _ in range(2))
        st["scale"] = D ** -0.5
        if op == "attend":
            st["mask"] = _tree_mask(g, S, n) if case["mask"] == "tree" else None
            st["mass"] = torch.rand(S, H, st["cache"]["table"].shape[2], generator=g, device=DEV) if case["mass"] else None
    else:
        st["cache"] = _cache(case, g, lens, 0, fill=False)  # eviction reads no codes
        P = st["cache"]["table"].shape[2]
        mass = torch.rand(S, H, P, generator=g, device=DEV).pow_(8) * 50
        st["mass"] = torch.where(torch.rand(S, H, P, generator=g, device=DEV) < 0.1, torch.zeros_like(mass), mass)
    if own:
        import w4a8_verify_gb300 as W
        st["handle"] = W.KV8Cache(S, H, st["cache"]["tail"].shape[-1], st["cache"]["table"].shape[2],
                                  tensors=st["cache"])
    return st


# ------------------------------------------------------------------------------------ one pass

def run(st):
    return (_run_own if own else _run_plain)[st["case"]["op"]](st)


# The framework's calls.

def _own_append(st):
    c = st["handle"]
    c.append(st["k"], st["v"], counts=st["counts"], len_out=st["len_out"])
    t = st["cache"]
    k, v = c.read(st["first"], st["rows"], length=st["len_out"])
    return dict(k=k, v=v, len=st["len_out"], scales=t["scales"], sums=t["sums"], tail=t["tail"])


def _own_attend(st):
    if st["mass"] is None:
        return dict(out=st["handle"].attention(st["q"], st["k"], st["v"], scale=st["scale"], mask=st["mask"]))
    mass = torch.empty_like(st["mass"])
    out = st["handle"].attention(st["q"], st["k"], st["v"], scale=st["scale"], mask=st["mask"], mass=st["mass"],
                                 mass_out=mass)
    return dict(out=out, mass=mass)


def _own_sparse(st):
    c, s = st["case"], st["handle"]
    pages = s.select(st["q"], c["top_k"], first_pages=c["first"], last_pages=c["last"])
    out = s.attention(st["q"], st["k"], st["v"], scale=st["scale"], pages=pages)
    return dict(out=out, pages=pages)


def _own_evict(st):
    c = st["case"]
    table, mass, length = st["handle"].evict(st["mass"], c["keep"], first_pages=c["first"], last_pages=c["last"])
    return dict(table=table, mass=mass, len=length)


# The plain forms.

def _gather(x, table):
    """x [S][H][P][...] in the order of table [S][H][...pages]."""
    S, H = table.shape[:2]
    s = torch.arange(S, device=DEV).view(S, 1, *[1] * (table.dim() - 2))
    h = torch.arange(H, device=DEV).view(1, H, *[1] * (table.dim() - 2))
    return x[s, h, table.long()]


def _page_values(cache, table, D):
    """fp32 keys and values [..., 64, D] of the pages that table names."""
    codes, scales = _gather(cache["codes"], table), _gather(cache["scales"], table)
    k = _untile_keys(codes[..., 0, :], D).float().sub_(128).mul_(scales[..., 0, None, None])
    v = _untile_values(codes[..., 1, :], D).float().sub_(128).mul_(scales[..., 1, None, None])
    return k, v


def _quantise(x):
    """x [..., 64, D] -> codes, scales (one scale for the page)."""
    s = x.abs().amax(dim=(-2, -1)) / torch.full((), 127.0, device=DEV)
    safe = torch.where(s > 0, s, torch.ones_like(s))[..., None, None]
    return torch.where((s > 0)[..., None, None], (x / safe).round().clamp(-127, 127), torch.zeros_like(x)), s


def _plain_append(st):
    c, t = st["case"], st["cache"]
    S, H, D, n = c["seqs"], c["kv_heads"], c["dim"], c["n"]
    lens, first = t["len"].long(), st["first"].long()
    end = lens + st["counts"].long()
    W = (n + PAGE - 1 + PAGE - 1) // PAGE  # pages that a call can touch
    at = torch.arange(W * PAGE, device=DEV)
    pos = first[:, None] + at  # position of each row of the window
    new = (pos - lens[:, None]).clamp(0, n - 1)
    fresh = (pos >= lens[:, None])[:, :, None, None]
    s = torch.arange(S, device=DEV)[:, None]
    page = first[:, None] // PAGE + torch.arange(W, device=DEV)  # [S][W]
    whole = (page + 1) * PAGE <= end[:, None]
    sq, wq = whole.nonzero(as_tuple=True)
    phys = t["table"].long()[sq, :, page[sq, wq]]  # [X][H]
    held = []
    for i, x in enumerate((st["k"], st["v"])):  # the keys, then the values
        old = t["tail"][:, :, i].transpose(1, 2)  # [S][64][H][D]
        rows = torch.where(fresh, x.float()[s, new], old[:, at % PAGE])  # [S][W * 64][H][D]
        blocks = rows.view(S, W, PAGE, H, D).transpose(2, 3)  # [S][W][H][64][D]
        codes, scales = _quantise(blocks)
        done = whole[:, :, None, None, None]
        held.append(torch.where(done, codes * scales[..., None, None], blocks))
        hq = torch.arange(H, device=DEV)[None]
        tiled = (_tile_keys if i == 0 else _tile_values)((codes[sq, wq] + 128).to(torch.uint8))
        t["codes"][sq[:, None], hq, phys, i] = tiled
        t["scales"][sq[:, None], hq, phys, i] = scales[sq, wq]
        if i == 0:
            t["sums"][sq[:, None], hq, phys] = codes[sq, wq].sum(dim=-2).to(torch.int16)
        left = (pos >= (end // PAGE * PAGE)[:, None]) & (pos < end[:, None]) & (pos >= lens[:, None])
        sl, rl = left.nonzero(as_tuple=True)
        t["tail"][sl, :, i, pos[sl, rl] % PAGE] = rows[sl, rl]
    st["len_out"].copy_(end)
    m = st["rows"]
    seen = (first[:, None] + torch.arange(m, device=DEV) < end[:, None])[:, :, None, None]
    k, v = (torch.where(seen, x.transpose(2, 3).reshape(S, W * PAGE, H, D)[:, :m], 0.0) for x in held)
    return dict(k=k, v=v, len=st["len_out"], scales=t["scales"], sums=t["sums"], tail=t["tail"])


def _seen_new(st, S, n):
    """[S][n][n]: whether query i sees new row j."""
    if st.get("mask") is None:
        return torch.ones(n, n, dtype=torch.bool, device=DEV).tril().expand(S, n, n)
    return (st["mask"][:, :, None] >> torch.arange(n, device=DEV)) & 1 == 1


def _attend(logits, seen, values):
    """Weights and their sum with the values; logits, seen [..., R, T], values [..., T, D]."""
    top = torch.where(seen, logits, -math.inf).amax(dim=-1, keepdim=True)
    w = torch.where(seen, (logits - torch.where(top > -math.inf, top, 0.0)).exp(), 0.0)
    total = w.sum(dim=-1, keepdim=True)
    w = w / torch.where(total > 0, total, 1.0)
    return w, w @ values


def _plain_attend(st):
    c, t = st["case"], st["cache"]
    S, H, G, D, n = c["seqs"], c["kv_heads"], c["group"], c["dim"], c["n"]
    P = t["table"].shape[2]
    k, v = (x.reshape(S, H, P * PAGE, D) for x in _page_values(t, t["table"], D))
    lens, whole = t["len"].long(), t["len"].long() // PAGE * PAGE
    q = st["q"].float().view(S, n, H, G, D).permute(0, 2, 1, 3, 4).reshape(S, H, n * G, D)
    k = torch.cat([k, t["tail"][:, :, 0], st["k"].float().transpose(1, 2)], dim=2)
    v = torch.cat([v, t["tail"][:, :, 1], st["v"].float().transpose(1, 2)], dim=2)
    seen = torch.cat([(torch.arange(P * PAGE, device=DEV) < whole[:, None])[:, None].expand(S, n, -1),
                      (torch.arange(PAGE, device=DEV) < (lens - whole)[:, None])[:, None].expand(S, n, -1),
                      _seen_new(st, S, n)], dim=2)
    seen = seen[:, None, :, None].expand(S, H, n, G, -1).reshape(S, H, n * G, -1)
    logits = (q @ k.transpose(2, 3)) * st["scale"]
    w, o = _attend(logits, seen, v)
    out = o.view(S, H, n, G, D).permute(0, 2, 1, 3, 4).reshape(S, n, H * G, D).to(st["q"].dtype)
    if st["mass"] is None:
        return dict(out=out)
    mass = w[..., :P * PAGE].reshape(S, H, n * G, P, PAGE).sum(dim=(2, 4))
    return dict(out=out, mass=st["mass"] + mass)


def _order(score, valid, first, last, whole):
    """Places of the pages [..., P] by descending (forced, score), ties to the lowest index; invalid ones last."""
    p = torch.arange(score.shape[-1], device=DEV)
    forced = (p < first) | (p >= whole - last)
    key = torch.where(valid, torch.where(forced, math.inf, score), -math.inf)
    return key.sort(dim=-1, descending=True, stable=True).indices


def _plain_sparse(st):
    c, t = st["case"], st["cache"]
    S, H, G, D, n, K = c["seqs"], c["kv_heads"], c["group"], c["dim"], c["n"], c["top_k"]
    P = t["table"].shape[2]
    lens = t["len"].long()
    whole = lens // PAGE
    q = st["q"].float().view(S, n, H, G, D).transpose(1, 2)  # [S][H][n][G][D]
    a = q.abs().amax(dim=(-2, -1), keepdim=True) / torch.full((), 127.0, device=DEV)
    qc = torch.where(a > 0, (q / torch.where(a > 0, a, 1.0)).round().clamp(-127, 127), 0.0)
    sums, sk = _gather(t["sums"], t["table"]), _gather(t["scales"], t["table"])[..., 0]
    dots = qc.double().view(S, H, n * G, D) @ sums.double().transpose(2, 3)  # whole numbers below 2^53
    score = dots.view(S, H, n, G, P).amax(dim=3).float() * sk[:, :, None]
    valid = torch.arange(P, device=DEV) < whole[:, None, None, None]
    picked = _order(score, valid, c["first"], c["last"], whole[:, None, None, None])[..., :min(K, P)]
    picked = torch.where(picked < whole[:, None, None, None], picked, P).sort(dim=-1).values
    picked = torch.cat([picked, picked.new_full((S, H, n, max(0, K - P)), P)], dim=-1)
    at = picked.clamp(max=P - 1)
    phys = torch.gather(t["table"].long()[:, :, None].expand(S, H, n, P), 3, at)
    k, v = (x.reshape(S, H, n, K * PAGE, D) for x in _page_values(t, phys, D))
    more = [torch.cat([t["tail"][:, :, i], x.float().transpose(1, 2)], dim=2)[:, :, None].expand(S, H, n, -1, D)
            for i, x in enumerate((st["k"], st["v"]))]
    k, v = torch.cat([k, more[0]], dim=3), torch.cat([v, more[1]], dim=3)
    tail = (torch.arange(PAGE, device=DEV) < (lens % PAGE)[:, None])[:, None].expand(S, n, PAGE)
    seen = torch.cat([tail, _seen_new(st, S, n)], dim=2)[:, None].expand(S, H, n, -1)
    seen = torch.cat([(picked < P)[..., None].expand(S, H, n, K, PAGE).reshape(S, H, n, -1), seen], dim=3)
    logits = (q @ k.transpose(3, 4)) * st["scale"]
    _, o = _attend(logits, seen[:, :, :, None], v)
    out = o.transpose(1, 2).reshape(S, n, H * G, D).to(st["q"].dtype)
    return dict(out=out, pages=torch.where(picked < P, picked, -1).transpose(1, 2).to(torch.int32).contiguous())


def _plain_evict(st):
    c, t = st["case"], st["cache"]
    P = t["table"].shape[2]
    whole = (t["len"].long() // PAGE)[:, None, None]
    kept = whole.clamp(max=c["keep"])
    p = torch.arange(P, device=DEV)
    order = _order(st["mass"], p < whole, c["first"], c["last"], whole)
    rank = torch.empty_like(order).scatter_(2, order, p.expand_as(order))
    # kept pages, then dropped ones, then those that were free, each in their order
    place = (torch.where(rank < kept, 0, 1) + (p >= whole)).sort(dim=-1, stable=True).indices
    table = torch.gather(t["table"], 2, place)
    mass = torch.where(p < kept, torch.gather(st["mass"], 2, place), 0.0)
    length = t["len"] - (PAGE * (whole - kept))[:, 0, 0].to(torch.int32)
    return dict(table=table, mass=mass, len=length)


_run_plain = dict(append=_plain_append, attend=_plain_attend, sparse=_plain_sparse, evict=_plain_evict)
_run_own = dict(append=_own_append, attend=_own_attend, sparse=_own_sparse, evict=_own_evict)


# ------------------------------------------------------------------------------------ what a pass cannot do without

def work(case):
    S, H, D, op = case["seqs"], case["kv_heads"], case["dim"], case["op"]
    mean = (case["length"] + (S - 1) * case["length"] / 2) / S if case["ragged"] else case["length"]
    pages = S * H * (mean // PAGE)  # whole pages of all heads
    if op == "evict":
        cut = min(mean // PAGE, case["keep"])
        return dict(bytes=8 * pages + S * H * (4 * (mean // PAGE) + 4 * cut), flops=pages)
    size, n = 4 if case["dtype"] == "fp32" else 2, case["n"]
    if op == "append":
        rows = S * H * n * 0.75  # of one of keys and values
        back = rows if case["length"] == 0 else S * H * (PAGE / 2 + n)
        held = rows * D if case["length"] == 0 else rows * D * 4
        return dict(bytes=2 * (rows * D * size + held + back * D * 4), flops=2 * 3 * rows * D)
    Hq = H * case["group"]
    small = S * n * D * size * (2 * Hq + 2 * H) + S * H * 2 * (mean % PAGE) * D * 4
    if op == "attend":
        more = 8 * pages + (8 * pages if case["mass"] else 0)
        return dict(bytes=2 * pages * PAGE * D + more + small, flops=4 * S * n * Hq * D * (mean + n))
    read = min(mean // PAGE, case["top_k"])
    return dict(bytes=pages * (2 * D + 4) + S * H * min(mean // PAGE, read * n) * (2 * PAGE * D + 8) + small,
                flops=2 * n * case["group"] * pages * D + 4 * S * n * Hq * D * (read * PAGE + PAGE // 2 + n))


# ------------------------------------------------------------------------------------ the definition in 64 bits

def _codes64(x):
    """x fp32 [64][D] (numpy) -> codes (fp64), scale (fp32): the codes are decided in 32 bits, by definition."""
    s = np.float32(np.abs(x).max()) / np.float32(127)
    if not s > 0:
        return np.zeros(x.shape), s
    return np.clip(np.rint((x / s).astype(np.float32)), -127, 127).astype(np.float64), s


def _softmax64(logits):
    e = torch.exp(logits - logits.max(dim=-1, keepdim=True).values)
    return e / e.sum(dim=-1, keepdim=True)


def _rows64(t, s, h, pages, D):
    """fp64 keys and values of some pages of (s, h), then those of the open page."""
    got = [[], []]
    if len(pages):
        phys = t["table"][s, h, pages].long()
        for i, untile in enumerate((_untile_keys, _untile_values)):
            x = untile(t["codes"][s, h, phys, i].double() - 128, D) * t["scales"][s, h, phys, i].double()[:, None, None]
            got[i].append(x.reshape(-1, D))
    open_rows = int(t["len"][s]) % PAGE
    for i in range(2):
        got[i].append(t["tail"][s, h, i, :open_rows].double())
    return torch.cat(got[0]), torch.cat(got[1])


def _exact_append(st):
    c, t = st["case"], st["cache"]
    S, H, D, m = c["seqs"], c["kv_heads"], c["dim"], st["rows"]
    if S * H * m * D > 1 << 26:
        return None
    k, v = np.zeros((S, m, H, D)), np.zeros((S, m, H, D))
    scales, sums = t["scales"].double().cpu().numpy(), t["sums"].cpu().numpy().copy()
    tail, table = t["tail"].double().cpu().numpy(), t["table"].cpu().numpy()
    new = [st["k"].float().cpu().numpy(), st["v"].float().cpu().numpy()]
    for s in range(S):
        L, cnt, first = int(t["len"][s]), int(st["counts"][s]), int(st["first"][s])
        for h in range(H):
            rows = [np.concatenate([tail[s, h, i, :L - first].astype(np.float32), new[i][s, :cnt, h]]) for i in range(2)]
            for a in range(0, len(rows[0]), PAGE):
                for i, out in enumerate((k, v)):
                    x = rows[i][a:a + PAGE]
                    if len(x) < PAGE:
                        old = max(0, L - first - a)
                        tail[s, h, i, old:len(x)] = x[old:]
                        out[s, a:a + len(x), h] = x[:m - a]
                        continue
                    code, scale = _codes64(x)
                    out[s, a:a + PAGE, h] = (code * np.float64(scale))[:m - a]
                    scales[s, h, table[s, h, (first + a) // PAGE], i] = scale
                    if i == 0:
                        sums[s, h, table[s, h, (first + a) // PAGE]] = code.sum(0)
    length = (t["len"] + st["counts"]).cpu().numpy()
    return dict(k=k, v=v, len=length, scales=scales, sums=sums, tail=tail)


def _exact_attend(st):
    c, t = st["case"], st["cache"]
    S, H, G, D, n = c["seqs"], c["kv_heads"], c["group"], c["dim"], c["n"]
    out = torch.zeros(S, n, H * G, D, dtype=torch.float64, device=DEV)
    mass = None if st["mass"] is None else st["mass"].double()
    for s in range(S):
        whole = int(t["len"][s]) // PAGE
        for h in range(H):
            k, v = _rows64(t, s, h, torch.arange(whole, device=DEV), D)
            k, v = torch.cat([k, st["k"][s, :, h].double()]), torch.cat([v, st["v"][s, :, h].double()])
            q = st["q"][s, :, h * G:(h + 1) * G].double()
            logits = torch.einsum("ngd,td->ngt", q, k) * st["scale"]
            for i in range(n):
                sees = (1 << (i + 1)) - 1 if st["mask"] is None else int(st["mask"][s, i])
                blind = [j for j in range(n) if not sees >> j & 1]
                if blind:
                    logits[i, :, [len(k) - n + j for j in blind]] = -math.inf
            w = _softmax64(logits)
            out[s, :, h * G:(h + 1) * G] = torch.einsum("ngt,td->ngd", w, v)
            if mass is not None:
                mass[s, h, :whole] += w[:, :, :whole * PAGE].sum(dim=(0, 1)).view(whole, PAGE).sum(dim=1)
    return dict(out=out) if mass is None else dict(out=out, mass=mass)


def _exact_sparse(st):
    c, t = st["case"], st["cache"]
    S, H, G, D, n, K = c["seqs"], c["kv_heads"], c["group"], c["dim"], c["n"], c["top_k"]
    out = torch.zeros(S, n, H * G, D, dtype=torch.float64, device=DEV)
    listed_pages = np.full((S, n, H, K), -1, np.int32)
    q32 = st["q"].float().cpu().numpy()
    for s in range(S):
        whole = int(t["len"][s]) // PAGE
        for h in range(H):
            phys = t["table"][s, h, :whole].long()
            sums = t["sums"][s, h, phys].cpu().numpy().astype(np.int64)
            scale = t["scales"][s, h, phys, 0].cpu().numpy()
            for i in range(n):
                code, _ = _codes64(q32[s, i, h * G:(h + 1) * G])
                score = scale * (sums @ code.astype(np.int64).T).max(axis=1).astype(np.float32) if whole else scale
                if whole:
                    score[:c["first"]] = math.inf
                    score[max(0, whole - c["last"]):] = math.inf
                best = np.sort(np.argsort(-score, kind="stable")[:K])
                listed_pages[s, i, h, :len(best)] = best
                k, v = _rows64(t, s, h, torch.from_numpy(best).to(DEV), D)
                k = torch.cat([k, st["k"][s, :i + 1, h].double()])
                v = torch.cat([v, st["v"][s, :i + 1, h].double()])
                w = _softmax64(st["q"][s, i, h * G:(h + 1) * G].double() @ k.T * st["scale"])
                out[s, i, h * G:(h + 1) * G] = w @ v
    return dict(out=out, pages=listed_pages)


def _exact_evict(st):
    c, t = st["case"], st["cache"]
    table, mass = t["table"].cpu().numpy().copy(), st["mass"].double().cpu().numpy()
    length = t["len"].cpu().numpy().copy()
    for s in range(table.shape[0]):
        whole = int(length[s]) // PAGE
        kept = min(whole, c["keep"])
        for h in range(table.shape[1]):
            m = mass[s, h, :whole].copy()
            m[:c["first"]] = math.inf
            m[max(0, whole - c["last"]):] = math.inf
            stay = np.sort(np.argsort(-m, kind="stable")[:kept])
            gone = np.setdiff1d(np.arange(whole), stay)
            table[s, h, :whole] = table[s, h, np.concatenate([stay, gone])]
            mass[s, h] = np.concatenate([mass[s, h, stay], np.zeros(mass.shape[2] - kept)])
        length[s] -= PAGE * (whole - kept)
    return dict(table=table, mass=mass, len=length)


def exact(case, seed):
    if case["op"] == "sparse" and case["seqs"] * case["kv_heads"] * case["n"] > 1024:
        return None
    if case["op"] == "attend" and case["seqs"] * case["kv_heads"] * case["n"] > 4096:
        return None
    st = prepare(case, seed)
    return dict(append=_exact_append, attend=_exact_attend, sparse=_exact_sparse, evict=_exact_evict)[case["op"]](st)
