"""Attention over the 4-bit cache where a CTA goes through many pages: ranges that begin and end inside sequences and hold the end
of one and the beginning of another, maxima that move on pages behind a range's first, more segments than CTAs.

The reference is the definition in 64 bits over what the cache reads back (exact in fp32); bounds as derived in
tests/test_gpu_kv4.py: |out - ref| <= max|V| (2 d + 2^-16) in fp32, max|V| (2 d + 2^-10) + 2^-8 |ref| in bf16, with
d = 2^-18 |scale| max|q| max_t sum|k_t|.
"""
import pytest

torch = pytest.importorskip("torch")

import w4a8_verify_gb300 as W

pytestmark = pytest.mark.gpu
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    W.lib()


def _randn(g, shape, amp=1.0):
    return torch.randn(shape, generator=g, device="cuda") * amp


def _cache(g, S, H, D, lens, dtype, spikes):
    """A cache of those lengths whose unwritten tokens are NaN.  Its keys are small but for some tokens of each head along one
    direction u [H][D], the later the stronger: their logits pass those in front by 8 to 10 (log2) for a query with 9 u."""
    P = max(1, (int(lens.max()) + 63) // 64)
    cache = W.KV4Cache(S, H, D, P, S * P + 2)
    cache.tensors["pages"].fill_(255)
    cache.tensors["table"].copy_(torch.randperm(S * P + 2, generator=g, device="cuda")[:S * P].view(S, P).to(torch.int32))
    n = max(1, int(lens.max()))
    u = _randn(g, (H, D))
    u /= u.norm(dim=-1, keepdim=True)
    k = _randn(g, (S, n, H, D), 0.3)
    unit = 9.0 / (1.4426950408889634 * 9.0 * D ** -0.5)             # 9 in log2 for a query of 9 u
    for i, at in enumerate(spikes):
        if at < n:
            some = (torch.rand((S, H), generator=g, device="cuda") < 0.7).float()
            k[:, at] += some[..., None] * (1 + i) * unit * u
    cache.append(k.to(TYPES[dtype]), _randn(g, (S, n, H, D), 0.5).to(TYPES[dtype]), counts=lens)
    return cache, u, n


def _check(cache, held, q, k, v, scale, counts, out, gone=()):
    """Every row of out against the definition; causal new rows.  gone: (sequence, page) that are left out."""
    S, H, D = cache.shape[:3]
    n, G = q.shape[1], q.shape[2] // H
    kc, vc = cache.read(torch.zeros(S, dtype=torch.int32, device="cuda"), held)
    rows, tok = torch.arange(n, device="cuda"), torch.arange(held, device="cuda")
    for s in range(S):
        cnt = n if counts is None else int(counts[s])
        if cnt == 0:
            continue
        there = tok < cache.len[s]
        for _, p in (x for x in gone if x[0] == s):
            there &= tok // 64 != p
        for h in range(H):
            K, V, see = kc[s, there, h].double(), vc[s, there, h].double(), torch.ones(cnt, int(there.sum()), device="cuda", dtype=torch.bool)
            if k is not None:
                K, V = torch.cat([K, k[s, :cnt, h].double()]), torch.cat([V, v[s, :cnt, h].double()])
                see = torch.cat([see, rows[:cnt, None] >= rows[:cnt]], 1)
            got = out[s, :cnt, h * G:(h + 1) * G].double()
            if not len(K):
                assert not got.any()
                continue
            qd = q[s, :cnt, h * G:(h + 1) * G].double()
            logits = torch.where(see[:, None], torch.einsum("ngd,td->ngt", qd, K) * scale, -torch.inf)
            ref = torch.softmax(logits, -1) @ V
            d = 2.0 ** -18 * abs(scale) * qd.abs().amax(-1, keepdim=True) * K.abs().sum(-1).max()
            top = V.abs().max()
            bound = top * (2 * d + 2.0 ** -16) if q.dtype is torch.float32 else top * (2 * d + 2.0 ** -10) + 2.0 ** -8 * ref.abs()
            err = (got - ref).abs()
            assert (err <= bound + 1e-30).all(), (s, h, (err / bound).max().item())


# From 10 to 28 pages to a CTA of the tcgen05 kernel, one of them with 192 segments; the last two are the split kernel's.
@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("S,H,G,D,n,lens", [
    (3, 8, 4, 128, 40, [9000, 4000, 130]),
    (3, 4, 8, 64, 40, [9000, 0, 7100]),
    (24, 8, 8, 64, 6, None),
    (24, 8, 4, 128, 7, None),
    (1, 2, 16, 128, 33, [20011]),
    (5, 8, 4, 128, 1, [9000, 40, 6000, 64, 2111]),
    (5, 8, 2, 64, 4, [9000, 40, 6000, 64, 2111]),
])
def test_many_pages_of_a_cta(S, H, G, D, n, lens, dtype, aligned):
    g = torch.Generator(device="cuda")
    g.manual_seed(S * n + D)
    lens = torch.tensor(lens, dtype=torch.int32, device="cuda") if lens else torch.randint(1, 1300, (S,), generator=g, device="cuda", dtype=torch.int32)
    # one maximum behind another, some pages apart; the second half of the batch's rows look the other way
    cache, u, held = _cache(g, S, H, D, lens, dtype, [70, 500, 1000, 3000, 6100])
    q = _randn(g, (S, n, H * G, D)) + 9 * torch.where(torch.rand((S, n, H * G, 1), generator=g, device="cuda") < 0.6, 1.0, -1.0) \
        * u.repeat_interleave(G, dim=0)
    q, k, v = (x.to(TYPES[dtype]) for x in (q, _randn(g, (S, n, H, D)), _randn(g, (S, n, H, D))))
    if not aligned:
        wide = torch.empty(S, n, H * (G + 2), D + 1, dtype=q.dtype, device="cuda")[..., 1:]
        for part, x in zip(wide.split([H * G, H, H], dim=2), (q, k, v)):
            part.copy_(x)
        q, k, v = wide.split([H * G, H, H], dim=2)
    scale = D ** -0.5
    out = cache.attention(q, k, v, scale=scale)
    _check(cache, held, q, k, v, scale, None, out)
    for _ in range(3):
        assert torch.equal(out, cache.attention(q, k, v, scale=scale))
    counts = torch.randint(0, n + 1, (S,), generator=g, device="cuda", dtype=torch.int32)
    counts[0] = n
    given = torch.full((S, n, H * G, D), 7.0, dtype=q.dtype, device="cuda")
    cache.attention(q, k, v, scale=-scale, counts=counts, out=given)
    _check(cache, held, q, k, v, -scale, counts, given)
    assert (given[torch.arange(n, device="cuda") >= counts[:, None]] == 7).all()
    assert cache.check() == 0
    # a table entry out of range on the first page of every head's range, one in the middle, and the last
    gone, table = [], cache.tensors["table"]
    longest = int(lens.argmax())
    for page in (0, (int(lens[longest]) // 64) // 2, (int(lens[longest]) - 1) // 64):
        gone.append((longest, page))
    kept = table.clone()
    for i, (s, p) in enumerate(gone):
        table[s, p] = (-1, cache.shape[4], 1 << 30)[i]
    bad = cache.attention(q, scale=scale)
    assert cache.check() == W.FLAG_ERR_TREE
    table.copy_(kept)
    _check(cache, held, q, None, None, scale, None, bad, gone)
