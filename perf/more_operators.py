"""Work of the 4-bit key/value cache and of the norm-and-rotation of queries and keys: the cases, their plain forms and
their 64-bit definition.

The cache holds S sequences in one pool of pages.  A page is 64 tokens of every KV head; `table[s][p]` is the page of the
pool that holds tokens 64 p .. 64 p + 63 of sequence s, and sequences may share pages (a common prefix).  A row of a head is
held in groups of 32 dims: whole numbers -7 .. 7 times a scale of eight bits (five of exponent, bias 15, three of
mantissa): scale = absmax / 7 to the nearest such number, at most 240.

A page of one head is 68 D bytes: codes of the keys (32 D), of the values (32 D), scales of the keys (2 D), of the values
(2 D), in the order in which a warp reads them (see _pack_keys and the functions beside it).
"""
import math

import numpy as np
import torch

own = False

PAGE = 64
MAX_SCALE = 240.0
DEV = "cuda"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one token for each of 16 sequences of a served batch; the open page is read back
        dict(name="append-step", op="append", seqs=16, kv_heads=8, dim=128, n=1, length=4095, ragged=True, dtype="fp32"),
        # a long prompt's rows of one layer go into an empty cache and come back out (saving, or handing over, a cache)
        dict(name="append-prompt", op="append", seqs=1, kv_heads=8, dim=128, n=32768, length=0, ragged=False,
             dtype="bf16"),
        # the smallest call: one token of a small model (14 query heads over 2 KV heads of 64) after 513 tokens
        dict(name="attend-small", op="attend", seqs=1, kv_heads=2, group=7, dim=64, n=1, length=513, ragged=False,
             dtype="fp32", mask="none", shared=0),
        # one greedy step of one layer of a model of 32 heads over 8 KV heads of 128, after 4095 tokens
        dict(name="attend-step", op="attend", seqs=1, kv_heads=8, group=4, dim=128, n=1, length=4095, ragged=False,
             dtype="fp32", mask="none", shared=0),
        # the verification of a draft tree of 16 nodes at the same place
        dict(name="attend-tree", op="attend", seqs=1, kv_heads=8, group=4, dim=128, n=16, length=4096, ragged=False,
             dtype="fp32", mask="tree", shared=0),
        # one token at the far end of a long context
        dict(name="attend-long", op="attend", seqs=1, kv_heads=8, group=4, dim=128, n=1, length=131071, ragged=False,
             dtype="bf16", mask="none", shared=0),
        # a served batch of 64 sequences of many lengths behind one common prefix of 512 tokens, one token each
        dict(name="attend-batch", op="attend", seqs=64, kv_heads=8, group=4, dim=128, n=1, length=8191, ragged=True,
             dtype="bf16", mask="none", shared=8),
        # a bucket of 64 prompt tokens deep in a prompt
        dict(name="attend-bucket", op="attend", seqs=1, kv_heads=8, group=4, dim=128, n=64, length=32000, ragged=False,
             dtype="bf16", mask="none", shared=0),
        # one token of the small model: its rows are part of one projection's output, no norm
        dict(name="rotate-step", op="rotate", seqs=1, kv_heads=2, group=7, dim=64, rot=64, n=1, far=513, ragged=False,
             dtype="fp32", axes=1, split="blocks", pairs="halves", norm=False),
        # draft trees of 16 nodes for a batch of 16 sequences, with norms
        dict(name="rotate-trees", op="rotate", seqs=16, kv_heads=8, group=4, dim=128, rot=128, n=16, far=32000, ragged=True,
             dtype="fp32", axes=1, split="blocks", pairs="halves", norm=True),
        # a long prompt of one layer, with norms
        dict(name="rotate-prompt", op="rotate", seqs=1, kv_heads=8, group=4, dim=128, rot=128, n=32768, far=0, ragged=False,
             dtype="bf16", axes=1, split="blocks", pairs="halves", norm=True),
        # two prompts of video tokens: time, height and width take their shares of the frequencies
        dict(name="rotate-video", op="rotate", seqs=2, kv_heads=8, group=4, dim=128, rot=128, n=5001, far=900, ragged=True,
             dtype="bf16", axes=3, split="blocks", pairs="halves", norm=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "rotate", "rotate"])
    kv_heads, group, dim = rng.choice([(8, 4, 128), (2, 7, 64), (4, 8, 64), (1, 5, 128), (3, 1, 64), (4, 16, 128),
                                       (2, 2, 128)])
    dtype = rng.choice(["fp32", "bf16"])
    seqs = rng.choice([1, 1, 2, 3, _log(rng, 4, 48)])
    room = max(200, 131071 * 8 * 128 // (kv_heads * dim * seqs))  # no more cached values than the largest case has
    length = _log(rng, 1, min(room, 131071))
    c = dict(op=op, seqs=seqs, kv_heads=kv_heads, dim=dim, dtype=dtype)
    if op == "append":
        step = rng.random() < 0.4
        c.update(n=1 if step else _log(rng, 1, min(room // 4, 32768)), length=length if step else 0, ragged=True)
    elif op == "attend":
        most = max(1, min(64, 2 ** 26 // (seqs * kv_heads * group * max(length, 64))))  # logits of the plain form
        n = min(rng.choice([1, 1, rng.randint(2, 16), rng.randint(17, 64)]), most)
        c.update(group=group, n=n, length=length, ragged=seqs > 1, mask=rng.choice(["none", "tree"]) if n > 1 else "none",
                 shared=rng.choice([0, rng.randint(0, length // PAGE)]) if seqs > 1 else 0)
    else:
        n = _log(rng, 1, max(1, min(32768, 2 ** 26 // (seqs * kv_heads * group * dim))))
        c.update(group=group, n=n, rot=rng.choice([dim, dim, dim // 2]), far=_log(rng, 1, 1 << 20), ragged=seqs > 1,
                 axes=rng.choice([1, 1, 2, 3]), split=rng.choice(["blocks", "turns"]),
                 pairs=rng.choice(["halves", "neighbours"]), norm=rng.random() < 0.6)
    return c


# ------------------------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _lengths(case, g, L):
    S = case["seqs"]
    if not case["ragged"]:
        return torch.full((S,), L, dtype=torch.int32, device=DEV)
    lens = torch.randint(0, L + 1, (S,), generator=g, device=DEV, dtype=torch.int32)
    lens[0] = L
    return lens


def _pack(x):
    """[..., halves, 4] whole numbers 0 .. 15 -> [..., bytes]: four to 16 bits, turned two bits to the left."""
    shift = torch.tensor([0, 4, 8, 12], device=x.device)
    w = (x.int() << shift).sum(dim=-1)
    w = ((w << 2) | (w >> 14)) & 0xffff
    return torch.stack([w & 255, w >> 8], dim=-1).to(torch.uint8).flatten(-2)


def _unpack(b):
    """The inverse of _pack, as whole numbers -8 .. 7."""
    w = b.unflatten(-1, (-1, 2)).int()
    w = w[..., 0] | (w[..., 1] << 8)
    w = (w >> 2) | ((w << 14) & 0xffff)
    return ((w[..., None] >> torch.tensor([0, 4, 8, 12], device=b.device)) & 15) - 8


def _pack_keys(c):
    """[..., 64 tokens, D] codes -> [..., 32 D] bytes: 16-token tiles, 64-dim parts, token % 8, 8-dim groups of 32, 32-dim
    halves, 4-dim halves, dim % 2, then the four of a 16-bit word: 2-dim halves, token / 8."""
    o, D = c.dim() - 2, c.shape[-1]
    x = (c + 8).reshape(*c.shape[:-2], 4, 2, 8, D // 64, 2, 4, 2, 2, 2)
    x = x.permute(*range(o), o, o + 3, o + 2, o + 5, o + 4, o + 6, o + 8, o + 7, o + 1)
    return _pack(x.reshape(*c.shape[:-2], 16 * D, 4))


def _unpack_keys(b):
    o, D = b.dim() - 1, b.shape[-1] // 32
    x = _unpack(b).reshape(*b.shape[:-1], 4, D // 64, 8, 4, 2, 2, 2, 2, 2)
    return x.permute(*range(o), o, o + 8, o + 2, o + 1, o + 4, o + 3, o + 5, o + 7, o + 6).reshape(*b.shape[:-1], PAGE, D)


def _pack_values(c):
    """[..., 64 tokens, D] codes -> [..., 32 D] bytes: 16-token tiles, 64-dim parts, dim % 8, token pairs of 8, 16-dim tiles,
    token % 2, then the four of a 16-bit word: 8-dim halves, token / 8."""
    o, D = c.dim() - 2, c.shape[-1]
    x = (c + 8).reshape(*c.shape[:-2], 4, 2, 4, 2, D // 64, 4, 2, 8)
    x = x.permute(*range(o), o, o + 4, o + 7, o + 2, o + 5, o + 3, o + 6, o + 1)
    return _pack(x.reshape(*c.shape[:-2], 16 * D, 4))


def _unpack_values(b):
    o, D = b.dim() - 1, b.shape[-1] // 32
    x = _unpack(b).reshape(*b.shape[:-1], 4, D // 64, 8, 4, 4, 2, 2, 2)
    return x.permute(*range(o), o, o + 7, o + 3, o + 5, o + 1, o + 4, o + 6, o + 2).reshape(*b.shape[:-1], PAGE, D)


def _tile_key_scales(s):
    """[..., 64, D / 32] -> [..., 2 D]: 16-token tiles, token % 8, token / 8, 32-dim groups."""
    o = s.dim() - 2
    return s.reshape(*s.shape[:-2], 4, 2, 8, s.shape[-1]).permute(*range(o), o, o + 2, o + 1, o + 3).flatten(-4)


def _untile_key_scales(b):
    o = b.dim() - 1
    x = b.reshape(*b.shape[:-1], 4, 8, 2, b.shape[-1] // PAGE)
    return x.permute(*range(o), o, o + 2, o + 1, o + 3).reshape(*b.shape[:-1], PAGE, -1)


def _tile_value_scales(s):
    """[..., 64, D / 32] -> [..., 2 D]: 16-token tiles, token pairs of 8, 32-dim groups, token / 8, token % 2."""
    o = s.dim() - 2
    x = s.reshape(*s.shape[:-2], 4, 2, 4, 2, s.shape[-1])
    return x.permute(*range(o), o, o + 2, o + 4, o + 1, o + 3).flatten(-5)


def _untile_value_scales(b):
    o = b.dim() - 1
    x = b.reshape(*b.shape[:-1], 4, 4, b.shape[-1] // PAGE, 2, 2)
    return x.permute(*range(o), o, o + 3, o + 1, o + 4, o + 2).reshape(*b.shape[:-1], PAGE, -1)


def _pages(k, ks, v, vs):
    """Codes [..., 64, D] and scale bytes [..., 64, D / 32] of keys and values -> the bytes of pages."""
    return torch.cat([_pack_keys(k), _pack_values(v), _tile_key_scales(ks), _tile_value_scales(vs)], dim=-1)


def _cache(case, g, lens, extra):
    """The tensors of a cache of the case's lengths: pages, table, len, ctl."""
    S, H, D = case["seqs"], case["kv_heads"], case["dim"]
    P = max(1, (case["length"] + extra + PAGE - 1) // PAGE)
    N = S * P + 3
    pages = torch.empty(N, H, 68 * D, dtype=torch.uint8, device=DEV)
    some = min(N, 1024)  # of this many the pages are made; the others repeat them with other scales
    drift = _randn(g, some, H, 1, D)  # the keys of a page have something in common
    k = ((_randn(g, some, H, PAGE, D) * 2 + drift)).round_().clamp_(-7, 7).int()
    v = (_randn(g, some, H, PAGE, D) * 2.5).round_().clamp_(-7, 7).int()
    pages[:, :, :64 * D] = torch.cat([_pack_keys(k), _pack_values(v)], dim=-1)[torch.arange(N, device=DEV) % some]
    pages[:, :, 64 * D:] = torch.randint(100, 116, (N, H, 4 * D), generator=g, device=DEV, dtype=torch.uint8)
    table = torch.randperm(N, generator=g, device=DEV)[:S * P].view(S, P).to(torch.int32)
    shared = case.get("shared", 0)
    table[:, :shared] = table[0, :shared]
    return dict(pages=pages, table=table.contiguous(), len=lens.clone(), ctl=torch.zeros(1, dtype=torch.int32, device=DEV))


def _tree_mask(g, S, n):
    """int64 [S][n]: bit j of entry i is set where node j is node i or one of its ancestors (random trees)."""
    parent = [(torch.rand(S, generator=g, device=DEV) * i).long() for i in range(n)]
    rows = [torch.ones(S, dtype=torch.int64, device=DEV)]
    for i in range(1, n):
        rows.append(torch.gather(torch.stack(rows, 1), 1, parent[i][:, None])[:, 0] | (1 << i if i < 63 else -(1 << 63)))
    return torch.stack(rows, 1)


def _rotation(case):
    """inv_freq fp64 [rot / 2] and the axis of each frequency."""
    half, axes = case["rot"] // 2, case["axes"]
    inv = 10000.0 ** (-np.arange(half) / half)
    if case["split"] == "turns":
        return inv, np.arange(half) % axes
    return inv, np.minimum((np.arange(half) + half // (2 * axes)) * axes // half, axes - 1)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    S, H, D, n, t = case["seqs"], case["kv_heads"], case["dim"], case["n"], TYPES[case["dtype"]]
    st = dict(case=dict(case))
    if op == "rotate":
        Hq = H * case["group"]
        st["qkv"] = (_randn(g, S, n, Hq + 2 * H, D) * torch.exp(_randn(g, D) * 0.5)).to(t)  # one projection's output
        st["q"], st["k"] = st["qkv"][:, :, :Hq], st["qkv"][:, :, Hq:Hq + H]
        st["start"] = _lengths(case, g, case["far"])
        st["pos"] = None  # position start + row
        if case["axes"] > 1:  # tokens of frames, rows and columns
            st["pos"] = torch.stack([torch.randint(0, 1 + n // (1, 8, 8)[a], (S, n), generator=g, device=DEV, dtype=torch.int32)
                                     for a in range(case["axes"])])
        st["gains"] = [(1 + 0.3 * _randn(g, D)) for _ in range(2)] if case["norm"] else [None, None]
        st["eps"] = 1e-6
        st["inv_freq"], st["axis"] = _rotation(case)
        st["inv"], st["ax"] = torch.from_numpy(st["inv_freq"]).to(DEV), torch.from_numpy(st["axis"]).to(DEV)
    else:
        lens = _lengths(case, g, case["length"])
        if op == "append":
            st["cache"] = _cache(case, g, lens, n)
            gain = torch.exp(_randn(g, H, D) * 0.7)  # some dims of a head are larger than others
            st["k"], st["v"] = ((_randn(g, S, n, H, D) * gain * (1 + i)).to(t) for i in range(2))
            st["counts"] = torch.randint((n + 1) // 2, n + 1, (S,), generator=g, device=DEV, dtype=torch.int32)
            st["len_out"] = torch.zeros_like(lens)
            st["first"] = (lens // PAGE * PAGE).to(torch.int32)
            st["rows"] = n if case["length"] == 0 else n + PAGE - 1
        else:
            st["cache"] = _cache(case, g, lens, 0)
            st["q"] = (_randn(g, S, n, H * case["group"], D) * 2).to(t)
            st["k"], st["v"] = (_randn(g, S, n, H, D).to(t) for _ in range(2))
            st["scale"] = D ** -0.5
            st["mask"] = _tree_mask(g, S, n) if case["mask"] == "tree" else None
    if own:
        import w4a8_verify_gb300 as W
        if op == "rotate":
            st["handle"] = W.Rotary(D, case["rot"], inv_freq=st["inv_freq"], axis=st["axis"],
                                    neighbours=case["pairs"] == "neighbours")
        else:
            c = st["cache"]
            st["handle"] = W.KV4Cache(S, H, D, c["table"].shape[1], c["pages"].shape[0], tensors=c)
    return st


# ------------------------------------------------------------------------------------ one pass

def run(st):
    return (_run_own if own else _run_plain)[st["case"]["op"]](st)


# The framework's calls.

def _own_append(st):
    c = st["handle"]
    c.append(st["k"], st["v"], counts=st["counts"], len_out=st["len_out"])
    k, v = c.read(st["first"], st["rows"], length=st["len_out"], dtype=st["k"].dtype)
    return dict(k=k, v=v, len=st["len_out"])


def _own_attend(st):
    return dict(out=st["handle"].attention(st["q"], st["k"], st["v"], scale=st["scale"], mask=st["mask"]))


def _own_rotate(st):
    q, k = st["handle"].apply(st["q"], st["k"], positions=st["pos"], start=st["start"],
                              eps=st["eps"] if st["case"]["norm"] else None, q_gain=st["gains"][0], k_gain=st["gains"][1])
    return dict(q=q, k=k)


# The plain forms.

def _scale_value(b):
    """fp32 values of scale bytes."""
    return (b.to(torch.int16) << 7).view(torch.float16).float()


def _held(pages, D):
    """fp32 keys and values [..., 64, D] of pages [..., 68 D]."""
    k, v, ks, vs = pages.split([32 * D, 32 * D, 2 * D, 2 * D], dim=-1)
    ks, vs = _scale_value(_untile_key_scales(ks)), _scale_value(_untile_value_scales(vs))
    return (_unpack_keys(k).float() * ks.repeat_interleave(32, dim=-1),
            _unpack_values(v).float() * vs.repeat_interleave(32, dim=-1))


def _quantise(x):
    """x fp32 [..., D] -> codes [..., D], scale bytes and scales [..., D / 32]."""
    x = x.unflatten(-1, (-1, 32))
    s = x.abs().amax(dim=-1) / torch.full((), 7.0, device=DEV)
    step = torch.ldexp(torch.ones_like(s), (torch.frexp(s).exponent - 1).clamp(min=-14) - 3)
    s = ((s / step).round() * step).clamp(max=MAX_SCALE)
    safe = torch.where(s > 0, s, 1.0)[..., None]
    c = torch.where(s[..., None] > 0, (x / safe).round().clamp(-7, 7), 0.0)
    return c.flatten(-2), (s.half().view(torch.int16) >> 7).to(torch.uint8), s


def _plain_append(st):
    c, t = st["case"], st["cache"]
    S, H, D, n = c["seqs"], c["kv_heads"], c["dim"], c["n"]
    lens, first = t["len"].long(), st["first"].long()
    end = lens + st["counts"].long()
    P = t["table"].shape[1]
    W = (n + PAGE - 1 + PAGE - 1) // PAGE  # pages that a call can touch
    page = first[:, None] // PAGE + torch.arange(W, device=DEV)  # [S][W]
    touched = page * PAGE < end[:, None]
    phys = torch.gather(t["table"].long(), 1, page.clamp(max=P - 1))
    pos = first[:, None] + torch.arange(W * PAGE, device=DEV)  # position of each row of the window
    j = (pos - lens[:, None]).clamp(0, n - 1)
    fresh = ((pos >= lens[:, None]) & (pos < end[:, None])).view(S, W, 1, PAGE, 1)
    rows = torch.arange(S, device=DEV)[:, None]
    old = t["pages"][phys]  # [S][W][H][68 D]

    def merged(x, old_codes, old_scales):
        codes, scales, _ = _quantise(x.float()[rows, j].view(S, W, PAGE, H, D).transpose(2, 3))
        return torch.where(fresh, codes.int(), old_codes), torch.where(fresh, scales, old_scales)

    kc, vc, ks, vs = old.split([32 * D, 32 * D, 2 * D, 2 * D], dim=-1)
    k, ks = merged(st["k"], _unpack_keys(kc), _untile_key_scales(ks))
    v, vs = merged(st["v"], _unpack_values(vc), _untile_value_scales(vs))
    t["pages"][phys[touched]] = _pages(k, ks, v, vs)[touched]
    st["len_out"].copy_(end)
    m = st["rows"]
    seen = (pos[:, :m] < end[:, None])[:, :, None, None]

    def back(codes, scales):
        x = (codes.float() * _scale_value(scales).repeat_interleave(32, dim=-1)).transpose(2, 3).reshape(S, W * PAGE, H, D)
        return torch.where(seen, x[:, :m], 0.0).to(st["k"].dtype)

    return dict(k=back(k, ks), v=back(v, vs), len=st["len_out"])


def _seen_new(st, S, n):
    """[S][n][n]: whether query i sees new row j."""
    if st["mask"] is None:
        return torch.ones(n, n, dtype=torch.bool, device=DEV).tril().expand(S, n, n)
    return (st["mask"][:, :, None] >> torch.arange(n, device=DEV)) & 1 == 1


def _plain_attend(st):
    c, t = st["case"], st["cache"]
    S, H, G, D, n = c["seqs"], c["kv_heads"], c["group"], c["dim"], c["n"]
    P = t["table"].shape[1]
    k, v = (x.transpose(1, 2).reshape(S, H, P * PAGE, D) for x in _held(t["pages"][t["table"].long()], D))
    q = st["q"].float().view(S, n, H, G, D).permute(0, 2, 1, 3, 4).reshape(S, H, n * G, D)
    k = torch.cat([k, st["k"].float().transpose(1, 2)], dim=2)
    v = torch.cat([v, st["v"].float().transpose(1, 2)], dim=2)
    seen = torch.cat([(torch.arange(P * PAGE, device=DEV) < t["len"][:, None])[:, None].expand(S, n, -1),
                      _seen_new(st, S, n)], dim=2)
    seen = seen[:, None, :, None].expand(S, H, n, G, -1).reshape(S, H, n * G, -1)
    logits = torch.where(seen, (q @ k.transpose(2, 3)) * st["scale"], -math.inf)
    w = (logits - logits.amax(dim=-1, keepdim=True)).exp()  # a row sees itself at least
    o = (w / w.sum(dim=-1, keepdim=True)) @ v
    return dict(out=o.view(S, H, n, G, D).permute(0, 2, 1, 3, 4).reshape(S, n, H * G, D).to(st["q"].dtype))


def _plain_rotate(st):
    c = st["case"]
    S, n, rot, half = c["seqs"], c["n"], c["rot"], c["rot"] // 2
    pos = torch.arange(n, device=DEV).expand(c["axes"], S, n) if st["pos"] is None else st["pos"].long()
    pos = (pos + st["start"].long()[:, None])[st["ax"]].permute(1, 2, 0)  # [S][n][rot / 2]
    angle = pos.double() * st["inv"]
    cos, sin = angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]

    def one(x, gain):
        dtype, x = x.dtype, x.float()
        if c["norm"]:
            x = x / (x.square().mean(dim=-1, keepdim=True) + st["eps"]).sqrt() * gain
        if c["pairs"] == "halves":
            a, b = x[..., :half], x[..., half:rot]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
        else:
            a, b = x[..., :rot:2], x[..., 1:rot:2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
        return torch.cat([y, x[..., rot:]], dim=-1).to(dtype)

    return dict(q=one(st["q"], st["gains"][0]), k=one(st["k"], st["gains"][1]))


_run_plain = dict(append=_plain_append, attend=_plain_attend, rotate=_plain_rotate)
_run_own = dict(append=_own_append, attend=_own_attend, rotate=_own_rotate)


# ------------------------------------------------------------------------------------ what a pass cannot do without

def work(case):
    S, H, D, op, n = case["seqs"], case["kv_heads"], case["dim"], case["op"], case["n"]
    size = 4 if case["dtype"] == "fp32" else 2
    if op == "rotate":
        values = S * n * H * (case["group"] + 1) * D
        return dict(bytes=2 * values * size, flops=values * (7 if case["norm"] else 3))
    L = case["length"]
    mean = (L + (S - 1) * L / 2) / S if case["ragged"] else L
    token = 2 * H * (D // 2 + D // 32)  # bytes of a cached token's keys and values
    if op == "append":
        rows = S * n * 0.75
        back = rows if L == 0 else S * (PAGE / 2 + n)
        return dict(bytes=rows * (2 * H * D * size + token) + back * (token + 2 * H * D * size), flops=2 * 4 * rows * H * D)
    held = S * mean - (S - 1) * min(case["shared"] * PAGE, mean)  # tokens, each read once
    Hq = H * case["group"]
    return dict(bytes=held * token + S * n * D * size * (2 * Hq + 2 * H), flops=4 * S * n * Hq * D * (mean + n))


# ------------------------------------------------------------------------------------ the definition in 64 bits

def _places(D):
    """Byte and low bit of the code of each (token, dim) in a page, byte of its scale; keys, then values."""
    tok, d = np.meshgrid(np.arange(PAGE), np.arange(D), indexing="ij")
    tile, r = tok // 16, tok % 16
    out = []
    for val in (False, True):
        if not val:
            lane, word = (r % 8) * 4 + d % 32 // 8, d % 64 // 32 * 2 + d % 8 // 4
            high, nibble = d % 2, d % 4 // 2 * 2 + r // 8
            scale = 64 * D + (tile * 8 + r % 8) * (D // 16) + r // 8 * (D // 32) + d // 32
        else:
            lane, word = (d % 8) * 4 + r % 8 // 2, d % 64 // 16
            high, nibble = r % 2, d % 16 // 8 * 2 + r // 8
            scale = 66 * D + ((tile * 4 + r % 8 // 2) * (D // 32) + d // 32) * 4 + r // 8 * 2 + r % 2
        half = 32 * D * val + (((tile * (D // 64) + d // 64) * 32 + lane) * 4 + word) * 4 + 2 * high
        out.append((half, 2 + 4 * nibble, scale))
    return out


def _scale64(b):
    e, m = b >> 3, b & 7
    return np.where(e == 0, m * 2.0 ** -17, (8.0 + m) * 2.0 ** (e.astype(np.float64) - 18))


def _rows64(pages, D):
    """fp64 keys and values [tokens][D] of pages uint8 [P][68 D] (numpy) of one head."""
    got = []
    for half, bit, scale in _places(D):
        w = pages[:, half].astype(np.uint32) | pages[:, half + 1].astype(np.uint32) << 8
        w |= w << 16  # the turned word, twice
        got.append((((w >> bit.astype(np.uint32)) & 15).astype(np.float64) - 8) * _scale64(pages[:, scale]))
    return [x.reshape(-1, D) for x in got]


def _scales32(x):
    """x fp32 [..., 32] (numpy) -> scale (fp64): decided in 32 bits, by definition."""
    s = (np.abs(x).max(axis=-1) / np.float32(7)).astype(np.float64)
    step = 2.0 ** (np.maximum(np.frexp(np.where(s > 0, s, 1.0))[1] - 1, -14) - 3.0)
    return np.minimum(np.rint(s / step) * step, MAX_SCALE)


def _exact_append(st):
    c, t = st["case"], st["cache"]
    S, H, D, m = c["seqs"], c["kv_heads"], c["dim"], st["rows"]
    if S * H * m * D > 1 << 26:
        return None
    out = [np.zeros((S, m, H, D)) for _ in range(2)]
    table = t["table"].cpu().numpy()
    new = [st[x].float().cpu().numpy() for x in "kv"]
    for s in range(S):
        L, cnt, first = int(t["len"][s]), int(st["counts"][s]), int(st["first"][s])
        for i in range(2):
            x = new[i][s, :cnt].reshape(cnt, H, D // 32, 32)
            scale = _scales32(x)[..., None]
            safe = np.where(scale > 0, scale, 1.0).astype(np.float32)
            code = np.clip(np.rint((x / safe).astype(np.float32)), -7, 7).astype(np.float64)
            held = (np.where(scale > 0, code, 0.0) * scale).reshape(cnt, H, D)
            out[i][s, L - first:L - first + cnt] = held[:max(0, m - (L - first))]
        if L > first:
            page = t["pages"][int(table[s, first // PAGE])].cpu().numpy()
            for h in range(H):
                for i, x in enumerate(_rows64(page[None, h], D)):
                    out[i][s, :L - first, h] = x[:min(m, L - first)]
    return dict(k=out[0], v=out[1], len=(t["len"] + st["counts"]).cpu().numpy())


def _exact_attend(st):
    c, t = st["case"], st["cache"]
    S, H, G, D, n = c["seqs"], c["kv_heads"], c["group"], c["dim"], c["n"]
    out = torch.zeros(S, n, H * G, D, dtype=torch.float64, device=DEV)
    table = t["table"].long()
    for s in range(S):
        L = int(t["len"][s])
        pages = t["pages"][table[s, :(L + PAGE - 1) // PAGE]].cpu().numpy()
        for h in range(H):
            k, v = (torch.from_numpy(x[:L]).to(DEV) for x in _rows64(pages[:, h], D))
            k, v = torch.cat([k, st["k"][s, :, h].double()]), torch.cat([v, st["v"][s, :, h].double()])
            logits = torch.einsum("ngd,td->ngt", st["q"][s, :, h * G:(h + 1) * G].double(), k) * st["scale"]
            for i in range(n):
                sees = (1 << (i + 1)) - 1 if st["mask"] is None else int(st["mask"][s, i])
                blind = [j for j in range(n) if not sees >> j & 1]
                if blind:
                    logits[i, :, [L + j for j in blind]] = -math.inf
            e = torch.exp(logits - logits.max(dim=-1, keepdim=True).values)
            out[s, :, h * G:(h + 1) * G] = torch.einsum("ngt,td->ngd", e / e.sum(dim=-1, keepdim=True), v)
    return dict(out=out)


def _exact_rotate(st):
    c = st["case"]
    n, rot = c["n"], c["rot"]
    start = st["start"].cpu().numpy().astype(np.int64)
    pos = np.arange(n) + np.zeros((c["axes"], len(start), 1), np.int64) if st["pos"] is None else st["pos"].cpu().numpy()
    angle = torch.from_numpy(((pos + start[:, None])[st["axis"]] * st["inv_freq"][:, None, None])).to(DEV)
    turn = torch.polar(torch.ones_like(angle), angle).permute(1, 2, 0)[:, :, None]
    out = {}
    for name, gain in zip("qk", st["gains"]):
        x = st[name].double()
        if c["norm"]:
            x = x * torch.rsqrt((x * x).sum(dim=-1, keepdim=True) / x.shape[-1] + st["eps"]) * gain.double()
        r = x[..., :rot]
        z = torch.complex(*(r.unflatten(-1, (2, -1)).unbind(-2) if c["pairs"] == "halves" else r.unflatten(-1, (-1, 2)).unbind(-1)))
        z = torch.view_as_real(z * turn)
        y = x.clone()
        y[..., :rot] = z.transpose(-1, -2).flatten(-2) if c["pairs"] == "halves" else z.flatten(-2)
        out[name] = y
    return out


def exact(case, seed):
    if case["op"] == "attend" and case["seqs"] * case["kv_heads"] * max(case["n"], case["length"] // 4096) > 4096:
        return None
    st = prepare(case, seed)
    return dict(append=_exact_append, attend=_exact_attend, rotate=_exact_rotate)[case["op"]](st)
