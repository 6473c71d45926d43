"""The 8-bit key/value cache, further calls: many of the same, beside other work, and those that a wait cuts short.

Bounds as in test_gpu_kv8.py.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import w4a8_verify_gb300 as W
from oracle import kv8 as O
from test_gpu_kv8 import _check_state, _filled, _i32, _long_check, _np, _random_cache, _rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    W.lib()


@pytest.mark.parametrize("dtype,S,H,G,D,n,L,calls", [
    ("bf16", 1, 8, 4, 128, 64, 32000, 1800),   # a prompt bucket: 52 pages of at most two segments for a CTA
    ("bf16", 3, 2, 8, 64, 40, 9000, 600),
    ("bf16", 40, 2, 16, 128, 9, 700, 600),     # runs of a few pages, many of them in a CTA
    ("fp32", 1, 8, 4, 128, 64, 16000, 300),
])
def test_wide_calls_again_and_again(dtype, S, H, G, D, n, L, calls):
    """The tcgen05 kernel over three caches in turn, beside another stream's copies that hold its warps up: the same bits
    each time, and no wait runs out."""
    rng = np.random.default_rng(n + D)
    jobs = []
    for i in range(3):
        lens = [L] + [int(x) for x in rng.integers(0, L, S - 1)]
        c = _random_cache(100 + i, lens, H, D)
        q = _rows(rng, S, n, H * G, D, dtype, 2.0)
        k, v = _rows(rng, S, n, H, D, dtype), _rows(rng, S, n, H, D, dtype)
        old, new = torch.rand(S, H, c.shape[3], device="cuda"), torch.empty(S, H, c.shape[3], device="cuda")
        out = c.attention(q, k, v, scale=D ** -0.5, mass=old, mass_out=new)
        _long_check(c, q, k, v, D ** -0.5, out, [0, H - 1], [0, S - 1], old, new)
        assert c.check() == 0
        jobs.append((c, q, k, v, old, out.clone(), new.clone(), torch.empty_like(out), torch.empty_like(new)))
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    side, block = torch.cuda.Stream(), torch.zeros(1 << 24, device="cuda")
    torch.cuda.synchronize()
    for i in range(calls):
        if i % 5 == 0:
            with torch.cuda.stream(side):
                block.add_(1.0)
        c, q, k, v, old, out, new, o, m = jobs[i % 3]
        c.attention(q, k, v, scale=D ** -0.5, mass=old, mass_out=m, out=o)
        wrong += (o != out).any().long() + (m != new).any().long()
    torch.cuda.synchronize()
    assert int(wrong) == 0
    assert [j[0].check() for j in jobs] == [0, 0, 0]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("lens,H,G,D,n,cta", [
    ([3000, 40, 700, 5000], 2, 4, 128, 1, 3),          # a page and a worker a warp
    ([3000, 40, 700, 5000], 2, 4, 64, 12, 150),        # several warps to a page, one of the last CTAs, if it has pages
    ([64, 0, 127], 1, 4, 128, 2, 0),                   # three rows of one page each: one CTA has all or one
    ([20000, 63, 9000], 2, 8, 128, 40, 60),            # tcgen05, runs of several segments
    ([9000, 63, 5000], 2, 16, 64, 9, 0),
])
def test_a_wait_that_runs_out_shows(dtype, lens, H, G, D, n, cta):
    """One CTA's copies are withheld (w4a8_kv8_attention_inject_timeout): the rows that miss its part are NaN, the others
    and the pages' mass as ever, the status word says so, and the next call on the same workspace is right."""
    rng = np.random.default_rng(n)
    S = len(lens)
    c = _random_cache(n, lens, H, D)
    q = _rows(rng, S, n, H * G, D, dtype, 2.0)
    k, v = _rows(rng, S, n, H, D, dtype), _rows(rng, S, n, H, D, dtype)
    old, mass = torch.rand(S, H, c.shape[3], device="cuda"), torch.empty(S, H, c.shape[3], device="cuda")
    want = c.attention(q, k, v, scale=0.1, mass=old, mass_out=mass)
    pages = c.select(q, 6, last_pages=1)
    sparse = c.attention(q, k, v, scale=0.1, pages=pages)
    assert c.check() == 0
    real = c._attention
    f = W.lib().w4a8_kv8_attention_inject_timeout

    def cut_short(ref, a, workspace, size, stream):
        return f(ref, a, workspace, size, cta, stream)
    for lists in (False, True):
        c._attention = cut_short
        m2 = torch.zeros_like(mass)
        if lists:
            got, ref = c.attention(q, k, v, scale=0.1, pages=pages), sparse
        else:
            got, ref = c.attention(q, k, v, scale=0.1, mass=old, mass_out=m2), want
        c._attention = real
        nan = torch.isnan(got)
        rows = nan.all(-1)
        assert torch.equal(nan.any(-1), rows)
        assert torch.equal(got[~rows], ref[~rows])
        if cta == 150 and not rows.any():                              # a call of few pages: none for this CTA
            assert c.check() == 0
            continue
        assert rows.any()
        short = [s for s in range(S) if lens[s] < 64]
        assert not rows[short].any()                                   # no pages: nothing of theirs is missing
        if max(lens) > 1000:
            assert int(rows.sum()) < rows.numel() // 2
        if not lists:
            lost = rows.view(S, n, H, G).any(dim=3).any(dim=1)         # [S][H]
            full = torch.tensor([[x // 64 for _ in range(H)] for x in lens], device="cuda")
            held = torch.arange(c.shape[3], device="cuda") < full[..., None]
            assert torch.equal(torch.isnan(m2), held & lost[..., None])
            assert torch.equal(m2[~lost], mass[~lost])
        assert c.check() == W.FLAG_ERR_TIMEOUT
        c.tensors["ctl"].zero_()
    assert torch.equal(c.attention(q, k, v, scale=0.1, pages=pages), sparse)
    assert torch.equal(c.attention(q, k, v, scale=0.1, mass=old, mass_out=m2), want) and torch.equal(m2, mass)
    assert c.check() == 0


@pytest.mark.parametrize("first,last,k", [(1, 2, 4), (1, 2, 2), (0, 3, 3), (0, 1, 1), (2, 2, 9), (0, 0, 4)])
def test_first_and_last_pages_come_before_infinite_scores(first, last, k):
    """Pages of NaN and of infinite score or mass in front of the last pages: those stay all the same."""
    D, P = 64, 30
    cache, ref = W.KV8Cache(1, 1, D, P), O.Cache(1, 1, D, P)
    x = torch.from_numpy(np.random.default_rng(k).standard_normal((1, 64 * P, 1, D)).astype(np.float32)).cuda()
    x[:, 64 * 2:64 * 6] = float("nan")
    cache.append(x, torch.ones_like(x))
    ref.append(0, x[0].cpu().numpy(), np.ones((64 * P, 1, D), np.float32))
    q = torch.ones(1, 1, 2, D, device="cuda")
    got = cache.select(q, k, first_pages=first, last_pages=last)[0, 0, 0].tolist()
    assert got == O.select(ref, 0, 0, np.ones((2, D), np.float32), k, first, last)
    must = [p for p in range(P) if p < first or p >= P - last]
    assert set(must[:k]) <= set(got)
    mass = torch.rand(1, 1, P, device="cuda")
    mass[0, 0, 3:7], mass[0, 0, 9:12] = float("inf"), float("nan")
    held = cache.tensors["table"][0, 0].tolist()
    kept, gone = O.evict(mass[0, 0].tolist(), k, first, last)
    assert set(must[:k]) <= set(kept)
    table, left, length = cache.evict(mass, k, first_pages=first, last_pages=last)
    assert table[0, 0].tolist() == [held[p] for p in kept + gone] and int(length[0]) == 64 * k
    assert torch.equal(left[0, 0, :k].nan_to_num(nan=-1.0), mass[0, 0, kept].nan_to_num(nan=-1.0))


def test_tensors_of_a_call_on_a_given_stream_may_be_dropped():
    """The caller's last references to the rows, the cache's to its pages, go while the given stream is still busy with
    something else: their memory is not handed out again before the call has read it."""
    lens, H, D = [500, 77], 2, 64

    def case():
        r = np.random.default_rng(92)
        return _random_cache(8, lens, H, D), _rows(r, 2, 3, 4 * H, D, "fp32"), _rows(r, 2, 3, H, D, "fp32")
    c, q, k = case()
    want = c.attention(q, k, k, scale=0.1)
    before = c.tensors["codes"].numel()
    c.append(k, k)
    held = c.read(_i32([480, 60]), 30)
    side = torch.cuda.Stream()
    for what in ("rows", "cache", "append"):
        c, q, k = case()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(100_000_000)                     # tens of milliseconds
        if what == "append":
            c.append(k, k, stream=side)
        else:
            got = c.attention(q, k, k, scale=0.1, stream=side)
        sizes = (q.shape, k.shape) if what != "cache" else [t.shape for t in c.tensors.values() if t.dtype == torch.float32]
        if what == "cache":
            c = None
        q = k = None
        junk = [torch.full(s, float("nan"), device="cuda") for s in sizes for _ in range(3)]
        junk.append(torch.full((before,), 255, dtype=torch.uint8, device="cuda"))
        torch.cuda.synchronize()
        if what == "append":
            assert all(torch.equal(a, b) for a, b in zip(c.read(_i32([480, 60]), 30), held))
        else:
            assert torch.equal(got, want)
        del junk


@pytest.mark.parametrize("seq,row,head", [(64 * 3, 64 * 12, 64 * 2), (64 * 2, 64 * 9, 64 * 36), (64 * 24, 64 * 4 + 1, 64), (65, 65 * 3, 65 * 6)])
def test_outputs_in_any_layout_without_overlap(seq, row, head):
    """Rows of out between one another (strides that do not nest), in any order: each where it belongs, nothing else."""
    rng = np.random.default_rng(seq)
    S, H, G, D, n = 3, 1, 4, 64, 2
    if seq == 64 * 3:
        S = 2                                                  # 0, 3 rows and 0, 2, 4, 6: no two alike
    c = _random_cache(5, [300, 64, 90][:S], H, D)
    q, k = _rows(rng, S, n, H * G, D, "fp32"), _rows(rng, S, n, H, D, "fp32")
    want = c.attention(q, k, k, scale=0.1)
    buf = torch.full((64 * 200,), 5.0, device="cuda")
    out = buf.as_strided((S, n, H * G, D), (seq, row, head, 1))
    c.attention(q, k, k, scale=0.1, out=out)
    assert torch.equal(out, want)
    out.fill_(5.0)
    assert (buf == 5.0).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_what_an_append_with_lengths_apart_leaves(dtype):
    """At the new lengths every sequence is right; at the old ones those that completed no page, and every whole page."""
    rng = np.random.default_rng(17)
    S, H, D = 4, 2, 64
    lens, n = [10, 60, 127, 128], 20
    cache, ref = _filled(rng, S, H, D, lens, dtype)
    k, v = _rows(rng, S, n, H, D, dtype), _rows(rng, S, n, H, D, dtype)
    before = cache.read(_i32([0] * S), 160)
    after = torch.zeros(S, dtype=torch.int32, device="cuda")
    cache.append(k, v, len_out=after)
    assert after.tolist() == [x + n for x in lens] and cache.len.tolist() == lens
    old = cache.read(_i32([0] * S), 160)
    for a, b in zip(before, old):
        assert torch.equal(a[[0, 3]], b[[0, 3]]) and torch.equal(a[2, :64], b[2, :64])
    for a, b in zip(cache.read(_i32([0] * S), 160, length=after), (0, 1)):
        for s in range(S):
            rows = (k, v)[b][s].float()
            whole = (lens[s] + n) // 64 * 64
            assert torch.equal(a[s, whole:lens[s] + n], torch.cat([before[b][s, :lens[s]], rows])[whole:])
    cache.len.copy_(after)
    for s in range(S):
        ref.append(s, _np(k)[s], _np(v)[s])
    _check_state(cache, ref)
    assert cache.check() == 0


@pytest.mark.parametrize("dtype,n,G,room", [("fp32", 5, 4, 0), ("fp32", 11, 4, 0), ("bf16", 10, 4, 0), ("fp32", 7, 4, 300),
                                            ("bf16", 9, 5, 300), ("fp32", 31, 4, 0), ("bf16", 11, 8, 300)])
def test_long_ragged_ranges_of_row_counts_without_divisors(dtype, n, G, room):
    """One warp to a page and many column blocks, a ring of one page a warp, runs over several segments; with room in the
    cache behind the sequences; and where that room takes the call to the tcgen05 kernel."""
    rng = np.random.default_rng(n * G + room)
    S, H, D = 4, 2, 128
    lens = [7000, 333, 4095, 6400]
    c = _random_cache(n, lens, H, D, max_pages=110 + room)
    q = _rows(rng, S, n, H * G, D, dtype, 2.0)
    k, v = _rows(rng, S, n, H, D, dtype), _rows(rng, S, n, H, D, dtype)
    old, new = torch.rand(S, H, c.shape[3], device="cuda"), torch.empty(S, H, c.shape[3], device="cuda")
    out = c.attention(q, k, v, scale=D ** -0.5, mass=old, mass_out=new)
    _long_check(c, q, k, v, D ** -0.5, out, range(H), range(S), old, new)
    assert c.check() == 0


@pytest.mark.parametrize("given", [True, False])
def test_check_waits_for_its_stream(given):
    """The status word of a call that is still queued on a stream of its own."""
    c = _random_cache(8, [500, 77], 2, 64)
    q = _rows(np.random.default_rng(3), 2, 3, 8, 64, "fp32")
    counts = _i32([3, 4])                                      # out of range
    c.attention(q, scale=0.1)
    assert c.check() == 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    if given:
        c.attention(q, scale=0.1, counts=counts, stream=side)
        assert c.check(stream=side) == W.FLAG_ERR_CAPACITY
    else:
        with torch.cuda.stream(side):
            c.attention(q, scale=0.1, counts=counts)
            assert c.check() == W.FLAG_ERR_CAPACITY


@pytest.mark.parametrize("dtype,D,G", [("bf16", 64, 16), ("fp32", 128, 15)])
def test_wide_calls_of_4096_sequences(dtype, D, G):
    """The most sequences of a call in the tcgen05 kernel: a few checked."""
    rng = np.random.default_rng(D)
    S, n, H = 4096, 9, 1
    lens = [int(x) for x in rng.integers(0, 192, S)]
    c = _random_cache(11, lens, H, D, max_pages=3)
    q, k = _rows(rng, S, n, H * G, D, dtype, 2.0), _rows(rng, S, n, H, D, dtype)
    out = c.attention(q, k, k, scale=0.1)
    _long_check(c, q, k, k, 0.1, out, [0], [0, 1, 2, 777, S - 2, S - 1])
    assert c.check() == 0


def test_1024_heads():
    rng = np.random.default_rng(12)
    S, H, D = 2, 1024, 64
    cache, ref = W.KV8Cache(S, H, D, 4), O.Cache(S, H, D, 4)
    k, v = _rows(rng, S, 150, H, D, "fp32"), _rows(rng, S, 150, H, D, "fp32")
    cache.append(k, v, counts=_i32([150, 70]))
    for s, c in enumerate((150, 70)):
        ref.append(s, _np(k)[s, :c], _np(v)[s, :c])
    q = _rows(rng, S, 2, H, D, "fp32")
    old, new = torch.rand(S, H, 4, device="cuda"), torch.empty(S, H, 4, device="cuda")
    out = cache.attention(q, k[:, :2], v[:, :2], scale=0.1, mass=old, mass_out=new)
    _long_check(cache, q, k[:, :2], v[:, :2], 0.1, out, [0, 1, 511, 1023], [0, 1], old, new)
    pages = cache.select(q, 1, last_pages=1)
    assert pages[0].eq(1).all() and pages[1].eq(0).all()
    table, mass, length = cache.evict(old, 1)
    best = old[0, :, :2].argmax(dim=1)
    assert torch.equal(table[0, :, 0], best.int()) and length.tolist() == [86, 70]
    kk, vv = cache.read(_i32([100, 0]), 50)
    assert torch.equal(kk[0, 28:50], k[0, 128:150]) and torch.equal(vv[0, 28:50], v[0, 128:150])
    assert cache.check() == 0


def test_the_longest_lists_and_eviction():
    """16384 pages of one head: read by a list of all of them and without one; eviction to none, some and all."""
    L, D = 64 * 16384 + 5, 64
    rng = np.random.default_rng(1)
    c = _random_cache(12, [L], 1, D, max_pages=16384)
    q, k = _rows(rng, 1, 1, 2, D, "fp32"), _rows(rng, 1, 1, 1, D, "fp32")
    pages = c.select(q, 16384)
    assert torch.equal(pages[0, 0, 0], torch.arange(16384, device="cuda", dtype=torch.int32))
    for lists in (None, pages):
        _long_check(c, q, k, k, 0.2, c.attention(q, k, k, scale=0.2, pages=lists), [0], [0], pages=lists)
    mass = torch.rand(1, 1, 16384, device="cuda")
    order = mass[0, 0].argsort(descending=True, stable=True)
    for keep in (0, 1, 100, 8192, 16383, 16384, 20000):
        table, left, length = c.evict(mass, keep)
        kept = order[:keep].sort().values
        held = c.tensors["table"][0, 0]
        assert torch.equal(table[0, 0, :len(kept)], held[kept]) and torch.equal(left[0, 0, :len(kept)], mass[0, 0, kept])
        assert sorted(table[0, 0].tolist()) == list(range(16384)) and int(length[0]) == 64 * len(kept) + 5
    assert c.check() == 0


@pytest.mark.parametrize("dtype,n", [("fp32", 3), ("bf16", 40)])
def test_rows_written_over_the_queries(dtype, n):
    """out is q itself: every kernel that reads the queries is done before they are written."""
    rng = np.random.default_rng(n)
    c = _random_cache(14, [3000, 100], 2, 128)
    q, k = _rows(rng, 2, n, 8, 128, dtype), _rows(rng, 2, n, 2, 128, dtype)
    pages = c.select(q, 5)
    for lists in (None, pages):
        want = c.attention(q, k, k, scale=0.1, pages=lists)
        mine = q.clone()
        assert c.attention(mine, k, k, scale=0.1, pages=lists, out=mine) is mine and torch.equal(mine, want)
