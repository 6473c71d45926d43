"""More of the 4-bit cache on the GPU: ranges of work that hold many short sequences, largest numbers of sequences, codes of bf16
values at and next to half steps.

The attention reference is the definition in 64 bits over what the cache reads back (exact in fp32); bounds as in
tests/test_gpu_kv4.py: |out - ref| <= max|V| (2 d + 2^-16) in fp32, max|V| (2 d + 2^-10) + 2^-8 |ref| in bf16, with
d = 2^-18 |scale| max|q| max_t sum|k_t|.
"""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import w4a8_verify_gb300 as W
from oracle import kv4 as O

gpu = pytest.mark.gpu
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    W.lib()


def _randn(g, shape, dtype, amp=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * amp).to(TYPES[dtype])


def _cache(g, S, H, D, lens, dtype, shuffle=True):
    """A cache of those lengths whose unwritten tokens are NaN."""
    P = max(1, (int(lens.max()) + 63) // 64)
    cache = W.KV4Cache(S, H, D, P, S * P + 1)
    cache.tensors["pages"].fill_(255)
    if shuffle:
        cache.tensors["table"].copy_(torch.randperm(S * P + 1, generator=g, device="cuda")[:S * P].view(S, P).to(torch.int32))
    n = max(1, int(lens.max()))
    cache.append(_randn(g, (S, n, H, D), dtype), _randn(g, (S, n, H, D), dtype, 0.5), counts=lens)
    return cache, n


def _check(cache, held, q, k, v, scale, counts, out):
    """Every row of out against the definition; causal new rows.  held: rows to read back."""
    S, H, D = cache.shape[:3]
    n, G = q.shape[1], q.shape[2] // H
    kc, vc = (x.double().transpose(1, 2) for x in cache.read(torch.zeros(S, dtype=torch.int32, device="cuda"), held))
    lens, dtype = cache.len.long(), q.dtype
    see = (torch.arange(held, device="cuda") < lens[:, None])[:, None].expand(S, n, held)
    cnt = torch.full_like(lens, n) if counts is None else counts.long()
    rows = torch.arange(n, device="cuda")
    if k is not None:
        here = (rows < cnt[:, None])[:, None]
        live = (rows < cnt[:, None])[:, :, None, None]
        kc = torch.cat([kc, torch.where(live, k.double(), 0).transpose(1, 2)], 2)
        vc = torch.cat([vc, torch.where(live, v.double(), 0).transpose(1, 2)], 2)
        see = torch.cat([see, (rows[:, None] >= rows).expand(S, n, n) & here], 2)
    qd = torch.where((rows < cnt[:, None])[:, :, None, None], q.double(), 0).view(S, n, H, G, D).permute(0, 2, 1, 3, 4)
    see = see[:, None, :, None]
    logits = torch.where(see, torch.einsum("shngd,shtd->shngt", qd, kc) * scale, -torch.inf)
    m = logits.amax(-1, keepdim=True).clamp(min=-1e300)
    e = torch.exp(logits - m)
    total = e.sum(-1, keepdim=True)
    ref = torch.einsum("shngt,shtd->shngd", e / torch.where(total > 0, total, 1), vc)
    B = abs(scale) * qd.abs().amax(-1) * kc.abs().sum(-1).amax(-1)[:, :, None, None]
    d = 2.0 ** -18 * B[..., None]
    top = vc.abs().amax((-1, -2))[:, :, None, None, None]
    bound = top * (2 * d + 2.0 ** -16) if dtype is torch.float32 else top * (2 * d + 2.0 ** -10) + 2.0 ** -8 * ref.abs()
    got = out.double().view(S, n, H, G, D).permute(0, 2, 1, 3, 4)
    live = (rows < cnt[:, None])[:, None, :, None, None].expand_as(got)
    bad = ~((got - ref).abs() <= bound + 1e-30) & live
    assert not bad.any(), (bad.nonzero()[0].tolist(), (got - ref).abs()[live].max().item())


# Ranges of work that hold whole sequences, the end of one and the beginning of another; one row and blocks of rows.
@gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("S,H,G,D,n,longest", [
    (4096, 1, 4, 64, 1, 3),      # lengths beyond those that are kept in shared memory
    (1500, 2, 4, 128, 1, 150),
    (700, 4, 2, 64, 2, 200),
    (300, 4, 8, 128, 2, 300),    # two column tiles
    (600, 8, 1, 128, 3, 70),
    (90, 2, 16, 64, 1, 2500),
])
def test_many_sequences(S, H, G, D, n, longest, dtype):
    _need_gpu()
    g = torch.Generator(device="cuda")
    g.manual_seed(S + n)
    lens = torch.randint(0, longest + 1, (S,), generator=g, device="cuda", dtype=torch.int32)
    lens[0], lens[S // 2:S // 2 + 5] = longest, 0
    cache, held = _cache(g, S, H, D, lens, dtype)
    q, k, v = (_randn(g, (S, n, h, D), dtype, a) for h, a in ((H * G, 2.0), (H, 1.0), (H, 1.0)))
    scale = D ** -0.5
    out = cache.attention(q, k, v, scale=scale)
    _check(cache, held, q, k, v, scale, None, out)
    for _ in range(3):
        assert torch.equal(out, cache.attention(q, k, v, scale=scale))
    # the cache alone: sequences of length zero see nothing
    alone = cache.attention(q, scale=-scale)
    _check(cache, held, q, None, None, -scale, None, alone)
    assert (alone[lens == 0] == 0).all()
    # a padded batch
    counts = torch.randint(0, n + 1, (S,), generator=g, device="cuda", dtype=torch.int32)
    given = torch.full_like(out, 7)
    cache.attention(q, k, v, scale=scale, counts=counts, out=given)
    _check(cache, held, q, k, v, scale, counts, given)
    rest = torch.arange(n, device="cuda") >= counts[:, None]
    assert (given[rest] == 7).all()
    assert cache.check() == 0
    assert all(not t[:W.KV4_TICKETS].any() for _, _, t in cache._kept.values())


@gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_calls_one_behind_the_other_in_one_workspace(dtype):
    """Calls of different sizes and kernels without a wait between them: tickets and parts of one are not another's."""
    _need_gpu()
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    S, H, G, D = 9, 2, 4, 128
    lens = torch.tensor([3000, 0, 64, 1, 700, 63, 65, 128, 5], dtype=torch.int32, device="cuda")
    cache, held = _cache(g, S, H, D, lens, dtype)
    work = []
    for n in (1, 2, 3, 4, 5, 9, 1):
        q, k, v = (_randn(g, (S, n, h, D), dtype) for h in (H * G, H, H))
        work.append((q, k, v, cache.attention(q, k, v, scale=0.1)))
        torch.cuda.synchronize()
        _check(cache, held, q, k, v, 0.1, None, work[-1][3])
    for _ in range(20):
        got = [cache.attention(q, k, v, scale=0.1) for q, k, v, _ in work]
        for a, (_, _, _, b) in zip(got, work):
            assert torch.equal(a, b)
    assert cache.check() == 0


def _bf16_groups(exponent):
    """Groups of 32 whose largest magnitude runs through the 128 mantissas of an exponent, the others through all bf16 numbers
    of the six binades below it, both signs."""
    m = np.arange(128)
    below = (np.arange(6 * 128) + ((exponent + 127 - 5) << 7)).astype(np.uint32)
    below = (below << 16).view(np.float32)
    below = np.concatenate([below, -below, [0.0]])
    per = -(-len(below) // 31)
    rest = np.resize(below, (per, 31)).astype(np.float32)
    top = ((m + ((exponent + 127) << 7)).astype(np.uint32) << 16).view(np.float32)
    x = np.zeros((128, per, 32), np.float32)
    x[:, :, 5] = top[:, None]
    x[:, :, [i for i in range(32) if i != 5]] = np.clip(rest[None], -top[:, None, None], top[:, None, None])
    return x.reshape(-1, 32)


@gpu
@pytest.mark.parametrize("exponent", [-12, -13, -24, 0, 9, 10, 11])
def test_codes_of_every_bf16_value(exponent):
    """Half steps (one bf16 value in a hundred is exactly half way between two codes), the smallest scales, the largest: every bit."""
    _need_gpu()
    D = 128
    x = _bf16_groups(exponent)
    x = np.resize(x, (-(-len(x) // 8) * 8, 32)).reshape(-1, 2, D)       # [rows][heads][D]
    n = len(x)
    codes, scales = O.quantize(x)
    want = O.value(codes, scales).astype(np.float32)
    t = torch.from_numpy(x)[None].cuda()
    for dtype in ("bf16", "fp32"):                                     # the same values either way
        for k, v in ((t, t.flip(1)), (t.flip(1), t)):
            cache = W.KV4Cache(1, 2, D, (n + 63) // 64)
            cache.append(k.to(TYPES[dtype]).contiguous(), v.to(TYPES[dtype]).contiguous())
            got = cache.read(torch.zeros(1, dtype=torch.int32, device="cuda"), n)
            for a, src in zip(got, (k, v)):
                w = want if src is t else want[::-1].copy()
                assert np.array_equal(a[0].cpu().numpy(), w)


@gpu
def test_codes_next_to_half_steps():
    """fp32 values one unit in the last place on either side of a half step, and at it."""
    _need_gpu()
    D, rng = 64, np.random.default_rng(4)
    amax = (rng.uniform(1, 2, 600) * 2.0 ** rng.integers(-13, 10, 600)).astype(np.float32)
    g = np.zeros((600, 32), np.float32)
    g[:, 0] = amax
    _, byte = O.quantize(g)
    s = O.VALUES[byte[:, 0]]
    half = ((np.arange(6) + 0.5) * s[:, None]).astype(np.float32)      # exact: seven bits
    near = np.concatenate([np.nextafter(half, np.float32(0)), half, np.nextafter(half, np.float32(np.inf))], 1)
    near = np.minimum(near, amax[:, None])
    g[:, 1:19] = near
    g[:, 19:31] = -near[:, 3:15]
    x = g.reshape(-1, 1, D)
    codes, scales = O.quantize(x)
    want = O.value(codes, scales).astype(np.float32)
    t = torch.from_numpy(x)[None].cuda()
    cache = W.KV4Cache(1, 1, D, (len(x) + 63) // 64)
    cache.append(t, t)
    for a in cache.read(torch.zeros(1, dtype=torch.int32, device="cuda"), len(x)):
        assert np.array_equal(a[0].cpu().numpy(), want)


@gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_read_of_every_code_and_scale(dtype):
    """Every code under every scale that an append writes, from pages made by hand."""
    _need_gpu()
    D = 128
    page = np.zeros((184 * 16 // (64 * 4) + 1, 68 * D), np.uint8)
    want = np.zeros((2, len(page) * 64, D), np.float32)
    rng = np.random.default_rng(2)
    for val, place in ((0, O.key_place), (1, O.value_place)):
        words = np.zeros((len(page), 32 * D), np.uint16)
        for p in range(len(page)):
            for tok in range(64):
                for gr in range(4):
                    byte = ((p * 64 + tok) * 4 + gr) % 184
                    for d in range(32 * gr, 32 * gr + 32):
                        c = int(rng.integers(-7, 8))
                        w, f, sc = place(D, tok, d)
                        u = (c + 8) << (4 * f)
                        words[p, w] |= (u << 2 | u >> 14) & 0xffff
                        page[p, sc] = byte
                        want[val, p * 64 + tok, d] = c * O.VALUES[byte]
        # words of the values begin behind those of the keys
        half = slice(0, 32 * D) if val == 0 else slice(32 * D, 64 * D)
        src = words[:, :16 * D] if val == 0 else words[:, 16 * D:]
        page[:, half] = np.ascontiguousarray(src).view(np.uint8)
    n = len(page) * 64
    cache = W.KV4Cache(1, 1, D, len(page))
    cache.tensors["pages"].copy_(torch.from_numpy(page)[:, None].cuda())
    cache.len.fill_(n)
    for got, w in zip(cache.read(torch.zeros(1, dtype=torch.int32, device="cuda"), n, dtype=TYPES[dtype]), want):
        assert np.array_equal(got[0, :, 0].float().cpu().numpy(), w)


def test_new_lengths_on_what_the_call_reads_are_refused():
    lib = W.lib()
    c = W.KV4CacheDesc(4, 2, 64, 4, 16, 0x10000, 0x20000, 0x30000, 0x40000)
    r = ctypes.byref(W.Rows(0x100000, 8192, 128, 64))
    call = lambda counts, index, out: lib.w4a8_kv4_append(c, r, r, 0, 64, 64, counts, index, out, None)  # noqa: E731
    for counts, index, out in ((0x50000, None, 0x50000), (0x50000, None, 0x5000c), (None, 0x50000, 0x503fc), (None, None, 0x20010),
                               (None, None, 0x30004), (None, None, 0x40000 - 4), (0x30000, None, 0x30000)):
        assert call(counts, index, out) == 1, (counts, index, out)


@gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
def test_new_rows_in_the_grid_of_the_wide_kernel(D, dtype):
    """A few blocks of new rows are CTAs behind those of the pages: ragged counts, strides that are not of 16 bytes, no new
    rows at all, a cache of length zero, and copies that are withheld from the first CTA."""
    _need_gpu()
    g = torch.Generator(device="cuda")
    g.manual_seed(D)
    S, H, G, n = 3, 2, 4, 13
    lens = torch.tensor([260, 0, 70], dtype=torch.int32, device="cuda")
    cache, held = _cache(g, S, H, D, lens, dtype)
    rows = _randn(g, (S, n, H * (G + 2), D + 1), dtype)[..., 1:]
    q, k, v = rows[:, :, :H * G], rows[:, :, H * G:H * G + H], rows[:, :, H * G + H:]
    counts = torch.tensor([n, n - 1, 5], dtype=torch.int32, device="cuda")
    out = torch.full((S, n, H * G, D), 7.0, dtype=TYPES[dtype], device="cuda")
    cache.attention(q, k, v, scale=0.1, counts=counts, out=out)
    _check(cache, held, q, k, v, 0.1, counts, out)
    assert (out[torch.arange(n, device="cuda") >= counts[:, None]] == 7).all()
    alone = cache.attention(q, scale=0.1)
    _check(cache, held, q, None, None, 0.1, None, alone)
    assert (alone[1] == 0).all() and cache.check() == 0
    real = cache._attention
    want = cache.attention(q, k, v, scale=0.1)
    try:
        cache._attention = lambda c, a, w, b, st: W.lib().w4a8_kv4_attention_inject_timeout(c, a, w, b, 0, st)
        got = cache.attention(q, k, v, scale=0.1)
        assert cache.check() == W.FLAG_ERR_TIMEOUT
    finally:
        cache._attention = real
    bad = torch.isnan(got).any(-1)
    assert bad.any() and not bad.all() and torch.isnan(got[bad]).all() and torch.equal(got[~bad], want[~bad])
    cache.tensors["ctl"].zero_()
    assert torch.equal(cache.attention(q, k, v, scale=0.1), want) and cache.check() == 0


@gpu
def test_two_captured_graphs_with_one_memory_pool():
    """The workspace of a captured call is set up by the call: a second graph that is given the first one's memory, and replays of
    both in turn, do not meet what the other left."""
    _need_gpu()
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    S, H, G, D = 2, 4, 4, 128
    lens = torch.tensor([1500, 333], dtype=torch.int32, device="cuda")
    cache, _ = _cache(g, S, H, D, lens, "fp32")
    work, graphs, pool = [], [], None
    for n in (1, 2, 12):
        q, k, v = (_randn(g, (S, n, h, D), "fp32") for h in (H * G, H, H))
        want = cache.attention(q, k, v, scale=0.1)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        out = torch.empty_like(want)
        with torch.cuda.graph(graph, pool=pool):
            cache.attention(q, k, v, scale=0.1, out=out)
        pool = pool or graph.pool()
        graphs.append(graph)
        work.append((q, k, v, out, want))
    for i in (0, 1, 2, 1, 0, 0, 2, 1):
        work[i][3].fill_(0)
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(work[i][3], work[i][4]), i
    assert cache.check() == 0
