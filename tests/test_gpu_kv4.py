"""The 4-bit key/value cache and the rotation of queries and keys through the C ABI against their definitions
(oracle/kv4.py, oracle/rotary.py, 64 bits).

Exact: codes, scale bytes, lengths, what is read back (all decided in fp32 or integers on both sides).

Attention bounds, from the operands.  Let B = |scale| max|q_d| max_t sum_d |k_td| of a row, so every logit and every partial
sum of one is at most B.  fp32 calls: q as f16 hi + lo is off by 2^-23 of its row's largest, the group sums and their
additions by less than 2^-21 B, the dot products with new rows (at most 13 additions one after the other) by 2^-20 B, the
scaling by 2^-22 B: a logit is off by less than d = 2^-18 B, a weight by 2 d relative; ex2 (2^-22), the weights' hi + lo
(2^-22, and 2^-32 of the largest weight for each of up to 2^15 tokens: 2^-17) and the value sums add less than 2^-16, so
|out - ref| <= max|V| (2 d + 2^-16).  bf16 calls: one f16 factor of a weight is off by half a step (2^-11), its sum is not;
the output is off by half a step of bf16 (2^-8 of its value): max|V| (2 d + 2^-10) + 2^-8 |ref|.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import w4a8_verify_gb300 as W
from oracle import kv4 as O

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    W.lib()


def _np(t):
    return t.detach().float().cpu().numpy()


def _i32(x):
    return torch.tensor(np.asarray(x).tolist(), dtype=torch.int32, device="cuda")


def _rows(rng, S, n, H, D, dtype, amp=1.0):
    return torch.from_numpy((rng.standard_normal((S, n, H, D)) * amp).astype(np.float32)).cuda().to(TYPES[dtype])


def _empty(S, H, D, P, N=None, rng=None):
    """An empty cache whose pages hold bytes that are NaN as scales, with a shuffled table, and its oracle."""
    cache = W.KV4Cache(S, H, D, P, N)
    cache.tensors["pages"].fill_(255)
    if rng is not None:
        cache.tensors["table"].copy_(_i32(rng.permutation(cache.shape[4])[:S * P].reshape(S, P)))
    return cache, O.Cache(S, H, D)


def _filled(rng, S, H, D, lens, dtype="fp32", P=None, amp=1.0):
    P = P or max(lens) // 64 + 2
    cache, ref = _empty(S, H, D, P, S * P + 3, rng)
    n = max(max(lens), 1)
    k, v = _rows(rng, S, n, H, D, dtype, amp), _rows(rng, S, n, H, D, dtype, amp * 0.5)
    cache.append(k, v, counts=_i32(lens))
    for s in range(S):
        ref.append(s, _np(k)[s, :lens[s]], _np(v)[s, :lens[s]])
    return cache, ref


def _check_state(cache, ref):
    S, H, D, P, _ = cache.shape
    pages, table = cache.tensors["pages"].cpu().numpy(), cache.tensors["table"].cpu().numpy()
    assert cache.len.tolist() == [ref.length(s) for s in range(S)]
    for s in range(S):
        L = ref.length(s)
        for p in range((L + 63) // 64):
            m = min(64, L - 64 * p)
            for h in range(H):
                for place, (codes, scales) in ((O.key_place, ref.rows[s][:2]), (O.value_place, ref.rows[s][2:])):
                    c, b = O.read_page(pages[table[s, p], h], D, place)
                    assert np.array_equal(b[:m], scales[64 * p:64 * p + m, h]), (s, p, h)
                    assert np.array_equal(c[:m], codes[64 * p:64 * p + m, h]), (s, p, h)


# ------------------------------------------------------------------------------- append and read

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_append_in_pieces(D, dtype):
    """Single rows, pieces that end inside tiles and pages, several pages at once, sequences that get nothing: every bit."""
    rng = np.random.default_rng(D + len(dtype))
    S, H, P = 3, 2, 9
    cache, ref = _empty(S, H, D, P, 30, rng)
    for n in (1, 14, 1, 1, 16, 17, 130, 64, 5, 63, 1, 200):
        k, v = _rows(rng, S, n, H, D, dtype, 3.0), _rows(rng, S, n, H, D, dtype)
        counts = [n, int(rng.integers(0, n + 1)), 0 if n % 2 else n]
        cache.append(k, v, counts=_i32(counts))
        for s in range(S):
            ref.append(s, _np(k)[s, :counts[s]], _np(v)[s, :counts[s]])
        _check_state(cache, ref)
    first = [0, 70, 500]
    for out in ("fp32", "bf16"):
        kk, vv = (_np(x) for x in cache.read(_i32(first), 150, dtype=TYPES[out]))
        for s in range(S):
            for h in range(H):
                for got, want in zip((kk, vv), ref.held(s, h)):
                    w = np.zeros((150, D))
                    x = want[first[s]:first[s] + 150]
                    w[:len(x)] = x
                    assert np.array_equal(got[s, :, h], w.astype(np.float32))
    assert cache.check() == 0


@pytest.mark.parametrize("n", [16, 40])
def test_append_strides_index_and_len_out(n):
    """Rows inside a fused tensor, the accepted path of a tree (rows out of order and twice), lengths kept apart: the cache is
    right at the old lengths and at the new ones."""
    rng = np.random.default_rng(5)
    S, H, D = 2, 3, 64
    cache, ref = _filled(rng, S, H, D, [60, 127], P=5)               # room for all of it
    qkv = _rows(rng, S, n, 4 * H, D, "fp32")
    k, v = qkv[:, :, H:2 * H], qkv[:, :, 2 * H:3 * H]
    m = n - 11
    index = rng.integers(0, n, (S, m))
    index[:, :4] = [0, 3, 3, n - 1]
    out = torch.full((S,), -7, dtype=torch.int32, device="cuda")
    cache.append(k, v, counts=_i32([m, m - 1]), index=_i32(index), len_out=out)
    assert out.tolist() == [60 + m, 127 + m - 1] and cache.len.tolist() == [60, 127]
    _check_state(cache, ref)
    cache.len.copy_(out)
    for s, c in enumerate((m, m - 1)):
        ref.append(s, _np(k)[s, index[s][:c]], _np(v)[s, index[s][:c]])
    _check_state(cache, ref)
    # a transposed source, [n_seqs][heads][n][head_dim], and one that is not 16-byte aligned
    x = _rows(rng, S, H, 70, D, "bf16").transpose(1, 2)
    y = _rows(rng, S, 70, H, D + 1, "bf16")[..., 1:]
    cache.append(x, y)
    for s in range(S):
        ref.append(s, _np(x)[s], _np(y)[s])
    _check_state(cache, ref)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_append_special_values(dtype):
    """Zeros, one value, ties of codes and of scales, the smallest scales, values beyond the largest scale, NaN and infinity."""
    rng = np.random.default_rng(6)
    D, H, n = 128, 1, 40
    x = rng.standard_normal((1, n, H, D)).astype(np.float32)
    x[0, 0] = 0
    x[0, 1] = 0
    x[0, 1, 0, 9] = -3.0
    for i, s in enumerate((1.0, 0.125, 1.875, 13 * 2.0 ** -9)):       # halves of a step
        x[0, 2 + i] = (rng.integers(-7, 7, D) + 0.5) * s
        x[0, 2 + i, 0, ::32] = 7 * s
    x[0, 6, 0, ::32] = 7 * np.array([1.0625, 1.1875, 2.125, 15.5])    # halves of a step of the scale
    x[0, 7] *= 2.0 ** -15
    x[0, 8] *= 2.0 ** -17
    x[0, 9] *= 1e-42
    x[0, 10] *= 1e3
    x[0, 11] *= 1e38 * 0.5
    x[0, 12, 0, 77] = np.nan
    x[0, 13, 0, 0] = -np.inf
    x[0, 14, 0, 40:48] = 1.75e3
    t = torch.from_numpy(x).cuda().to(TYPES[dtype])
    cache, ref = _empty(1, H, D, 2)
    cache.append(t, t.flip(1))
    ref.append(0, _np(t)[0], _np(t)[0, ::-1])
    _check_state(cache, ref)
    k, v = (_np(y) for y in cache.read(_i32([0]), n))
    for got, want in zip((k, v), ref.held(0, 0)):
        assert np.array_equal(got[0, :, 0], want.astype(np.float32), equal_nan=True)


def test_append_leaves_what_is_out_of_range():
    rng = np.random.default_rng(7)
    S, H, D, P = 5, 2, 64, 2
    cache, ref = _filled(rng, S, H, D, [128, 110, 10, 20, 30], P=P)
    x = _rows(rng, S, 20, H, D, "fp32")
    keep = cache.tensors["pages"].clone()
    # full; would pass the end; a count out of range; a source row out of range; fine
    cache.append(x, x, counts=_i32([1, 20, 21, 3, 4]), index=_i32([[0] * 20] * 3 + [[0, 20, 1] + [0] * 17] + [[3, 2, 1, 0] + [0] * 16]))
    assert cache.len.tolist() == [128, 110, 10, 20, 34]
    assert cache.check() == W.FLAG_ERR_CAPACITY | W.FLAG_ERR_TOKEN
    ref.append(4, _np(x)[4, [3, 2, 1, 0]], _np(x)[4, [3, 2, 1, 0]])
    _check_state(cache, ref)
    mine = cache.tensors["table"][4, 0].item()
    keep[mine] = cache.tensors["pages"][mine]
    assert torch.equal(cache.tensors["pages"], keep)
    # lengths out of range; a table entry out of range takes no rows and reads as 0
    cache.tensors["ctl"].zero_()
    cache.len[0], cache.len[1], cache.tensors["table"][2, 0] = -1, 129, cache.shape[4]
    cache.append(x[:, :1], x[:, :1])
    assert cache.check() == W.FLAG_ERR_CAPACITY | W.FLAG_ERR_TREE
    keep[mine] = cache.tensors["pages"][mine]
    keep[cache.tensors["table"][3, 0].item()] = cache.tensors["pages"][cache.tensors["table"][3, 0].item()]
    assert torch.equal(cache.tensors["pages"], keep)
    k, _ = cache.read(_i32([0, 0, 0, -1, 0]), 30)
    assert not k[:4].any() and k[4].any()
    with pytest.raises(W.W4A8Error):
        cache.append(_rows(rng, S, 129, H, D, "fp32"), _rows(rng, S, 129, H, D, "fp32"))


# ------------------------------------------------------------------------------- attention

def _masks(rng, S, n, kind):
    if kind == "causal":
        return None, [[(1 << (i + 1)) - 1 for i in range(n)] for _ in range(S)]
    m = [[0] * n for _ in range(S)]
    for s in range(S):
        for i in range(n):
            m[s][i] = (m[s][int(rng.integers(0, i))] if i else 0) | 1 << i
            if kind == "odd":                                       # any bits: rows that see nothing new, or later rows
                m[s][i] = int(rng.integers(0, 1 << 62)) * int(rng.integers(0, 2)) & (1 << n) - 1
    signed = [[b - (1 << 64) if b >> 63 else b for b in row] for row in m]
    return torch.tensor(signed, dtype=torch.int64, device="cuda"), m


def _check_attention(cache, ref, q, k, v, scale, masks, counts=None, mask=None, out=None, rows=None, **kw):
    S, n, Hq, D = q.shape
    H = ref.H
    G = Hq // H
    dtype = "fp32" if q.dtype == torch.float32 else "bf16"
    got = cache.attention(q, k, v, scale=scale, counts=None if counts is None else _i32(counts), mask=mask, out=out, **kw)
    gn, qn = _np(got), _np(q).astype(np.float64)
    kn, vn = (None, None) if k is None else (_np(k).astype(np.float64), _np(v).astype(np.float64))
    none = np.zeros((0, D))
    worst = 0.0
    for s in range(S):
        for h in range(H):
            kh, vh = ref.held(s, h)
            cnt = n if counts is None else counts[s]
            top = max([0.0] + [np.abs(x).max() for x in (vh, none if vn is None else vn[s, :cnt, h]) if x.size])
            for i in range(cnt):
                for hq in range(h * G, (h + 1) * G):
                    if rows is not None and (s, i, hq) not in rows:
                        continue
                    m = masks[s][i] & (1 << cnt) - 1
                    want, B = O.attention(kh, vh, qn[s, i, hq], none if kn is None else kn[s, :, h], none if vn is None else vn[s, :, h], m, scale)
                    d = 2.0 ** -18 * B
                    bound = top * (2 * d + 2.0 ** -16) if dtype == "fp32" else top * (2 * d + 2.0 ** -10) + 2.0 ** -8 * np.abs(want)
                    err = np.abs(gn[s, i, hq] - want)
                    assert (err <= bound + 1e-30).all(), (s, i, hq, err.max(), np.max(bound))
                    worst = max(worst, float(np.linalg.norm(err) / (np.linalg.norm(want) + 1e-30)))
    return got, worst


CASES = [  # S, H, G, D, n, lengths, mask
    (1, 2, 7, 64, 1, [513], "causal"),
    (1, 8, 4, 128, 1, [4095], "causal"),
    (1, 2, 1, 128, 1, [0], "causal"),
    (2, 1, 16, 128, 1, [1, 63], "causal"),
    (5, 3, 2, 64, 2, [0, 1, 64, 65, 1000], "causal"),
    (3, 2, 5, 128, 3, [127, 128, 129], "tree"),
    (2, 2, 4, 128, 16, [700, 31], "tree"),
    (2, 1, 3, 64, 17, [97, 260], "odd"),
    (1, 2, 4, 64, 64, [333], "tree"),
    (1, 1, 16, 128, 64, [100], "causal"),
    (37, 2, 1, 64, 1, list(range(0, 37 * 9, 9)), "causal"),
    (2, 1, 8, 128, 5, [0, 0], "odd"),
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_attention(case, dtype):
    S, H, G, D, n, lens, kind = CASES[case]
    rng = np.random.default_rng(100 + case)
    cache, ref = _filled(rng, S, H, D, lens, dtype)
    q, k, v = _rows(rng, S, n, H * G, D, dtype, 2.0), _rows(rng, S, n, H, D, dtype), _rows(rng, S, n, H, D, dtype)
    mask, bits = _masks(rng, S, n, kind)
    some = None
    if S * n * H * G > 400:
        some = {(int(rng.integers(S)), int(rng.integers(n)), int(rng.integers(H * G))) for _ in range(300)}
        some |= {(s, i, h) for s in (0, S - 1) for i in (0, n - 1) for h in (0, H * G - 1)}
    a, _ = _check_attention(cache, ref, q, k, v, D ** -0.5, bits, mask=mask, rows=some)
    b = cache.attention(q, k, v, scale=D ** -0.5, mask=mask)
    assert torch.equal(a, b)                                         # nothing depends on timing
    assert not cache._kept or all(not t[:W.KV4_TICKETS].any() for _, _, t in cache._kept.values())
    if any(lens):
        _check_attention(cache, ref, q, None, None, -0.3 * D ** -0.5, [[0] * n] * S, rows=some)
    assert cache.check() == 0


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("n", [1, 9, 40])
def test_counts_strides_and_given_output(dtype, n):
    """A padded batch: rows behind a sequence's count stay as they were, in the output as in what is read (NaN there)."""
    rng = np.random.default_rng(11)
    S, H, G, D = 4, 2, 4, 128
    cache, ref = _filled(rng, S, H, D, [300, 64, 0, 77], dtype)
    qkv = _rows(rng, S, n + 3, H * (G + 2), D, dtype)
    counts = [n, 0, max(1, n - 1), n // 2]
    for s in range(S):
        qkv[s, counts[s]:] = float("nan")
    q, k, v = qkv[:, :n, :H * G], qkv[:, :n, H * G:H * G + H], qkv[:, :n, H * G + H:]
    big = torch.full((S, H * G, n, D + 8), 7.0, dtype=TYPES[dtype], device="cuda")
    out = big.transpose(1, 2)[..., :D]                               # heads outside rows
    _check_attention(cache, ref, q, k, v, 0.1, [[(1 << (i + 1)) - 1 for i in range(n)]] * S, counts=counts, out=out)
    for s in range(S):
        assert (out[s, counts[s]:] == 7).all()
    assert (big[..., D:] == 7).all()
    odd = torch.empty(S, n, H * G, D + 1, dtype=TYPES[dtype], device="cuda")[..., 1:]   # no 16-byte access
    odd.copy_(q)
    _check_attention(cache, ref, odd, k, v, 0.1, [[(1 << (i + 1)) - 1 for i in range(n)]] * S, counts=counts)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("n", [3, 33])
def test_new_rows_touch_only_the_rows_that_see_them(dtype, n):
    rng = np.random.default_rng(12)
    S, H, G, D = 1, 2, 4, 64
    cache, ref = _filled(rng, S, H, D, [200], dtype)
    q, k, v = _rows(rng, S, n, H * G, D, dtype), _rows(rng, S, n, H, D, dtype), _rows(rng, S, n, H, D, dtype)
    k[0, 1], v[0, 2] = float("nan"), float("inf")
    mask = torch.tensor([[1] * (n - 1) + [0b111]], dtype=torch.int64, device="cuda")
    bits = [[1] * (n - 1) + [0]]
    out = cache.attention(q, k, v, scale=0.2, mask=mask)
    assert not torch.isfinite(out[0, n - 1]).any() and torch.isfinite(out[0, :n - 1]).all()
    clean_k, clean_v = k.clone(), v.clone()
    clean_k[0, 1:], clean_v[0, 1:] = 0, 0
    _, _ = _check_attention(cache, ref, q[:, :, :], clean_k, clean_v, 0.2, bits, mask=torch.tensor([[1] * (n - 1) + [0]], device="cuda"))
    assert torch.equal(out[0, :n - 1], cache.attention(q, clean_k, clean_v, scale=0.2, mask=mask)[0, :n - 1])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("n", [1, 40])
def test_extreme_logits(dtype, n):
    """Logits of +-1e4 (one token takes all), equal keys, a scale of zero, a query of zeros, of huge and of tiny values."""
    rng = np.random.default_rng(13)
    S, H, G, D = 1, 1, 4, 128
    cache, ref = _filled(rng, S, H, D, [777], dtype, amp=30.0)
    q, k, v = _rows(rng, S, n, G, D, dtype, 3.0), _rows(rng, S, n, H, D, dtype), _rows(rng, S, n, H, D, dtype)
    q[0, 0, 0] = 0
    q[0, 0, 1] *= 1e-30
    bits = [[(1 << (i + 1)) - 1 for i in range(n)]]
    _check_attention(cache, ref, q, k, v, 0.0, bits)
    _check_attention(cache, ref, q, k, v, 1e-3, bits)
    got = cache.attention(q * 1e4, k, v, scale=1.0)                  # the bound says nothing here: finite, and a value of one token
    assert torch.isfinite(got).all()
    lim = max(np.abs(ref.held(0, 0)[1]).max(), _np(v).__abs__().max())
    assert got.float().abs().max().item() <= lim * 1.01
    x = cache.attention(torch.full_like(q, float("nan")), k, v)
    assert torch.isnan(x).all()


def test_shared_pages_and_nan_groups():
    """Two sequences name the same prefix pages; a NaN group of a cached value makes its dims NaN, of a key the whole row."""
    rng = np.random.default_rng(14)
    S, H, G, D = 3, 2, 4, 64
    cache, ref = _filled(rng, S, H, D, [130, 128, 140])
    t = cache.tensors["table"]
    t[1, :2] = t[0, :2]
    ref.rows[1] = tuple(x[:128] for x in ref.rows[0])
    q, k, v = _rows(rng, S, 1, H * G, D, "fp32"), _rows(rng, S, 1, H, D, "fp32"), _rows(rng, S, 1, H, D, "fp32")
    _check_attention(cache, ref, q, k, v, 0.125, [[1]] * S)
    x = _rows(rng, S, 1, H, D, "fp32")
    y = x.clone()
    y[0, 0, 0, 40] = float("nan")
    cache.append(x, y, counts=_i32([1, 0, 0]))
    out = cache.attention(q, k, v, scale=0.125)
    assert torch.isnan(out[0, 0, :G, 32:]).all() and torch.isfinite(out[0, 0, :G, :32]).all()
    assert torch.isfinite(out[0, 0, G:]).all() and torch.isfinite(out[1:]).all()
    cache.append(y, x, counts=_i32([0, 0, 1]))                       # row 0 of y is finite for sequence 2
    y[2, 0, 1, 3] = float("inf")
    cache.append(y, x, counts=_i32([0, 0, 1]))
    out = cache.attention(q, k, v, scale=0.125)
    assert torch.isfinite(out[2, 0, :G]).all() and torch.isnan(out[2, 0, G:]).all()


def test_table_and_lengths_out_of_range():
    rng = np.random.default_rng(15)
    S, H, G, D = 4, 2, 4, 64
    cache, ref = _filled(rng, S, H, D, [300, 300, 300, 300])
    q, k, v = _rows(rng, S, 1, H * G, D, "fp32"), _rows(rng, S, 1, H, D, "fp32"), _rows(rng, S, 1, H, D, "fp32")
    cache.len[1] = 64 * cache.shape[3] + 1
    cache.len[2] = -5
    cache.tensors["table"][0, 1], cache.tensors["table"][3, 4] = -1, cache.shape[4]
    out = torch.full_like(q, 7.0)
    cache.attention(q, k, v, scale=0.125, out=out)
    assert cache.check() == W.FLAG_ERR_CAPACITY | W.FLAG_ERR_TREE
    assert (out[1:3] == 7).all()
    ref.rows[0] = tuple(np.delete(x, np.s_[64:128], axis=0) for x in ref.rows[0])
    ref.rows[3] = tuple(x[:256] for x in ref.rows[3])
    for s in (1, 2):
        ref.rows[s] = tuple(x[:0] for x in ref.rows[s])
    cache.len[1:3] = 0
    _check_attention(cache, ref, q, k, v, 0.125, [[1]] * S)


# ------------------------------------------------------------------------------- streams, graphs, sizes

@pytest.mark.parametrize("n", [1, 40])
def test_captured_calls_follow_lengths_and_tables(n):
    rng = np.random.default_rng(16)
    S, H, G, D = 2, 2, 4, 128
    cache, ref = _filled(rng, S, H, D, [100, 10], P=40)
    q, k, v = _rows(rng, S, n, H * G, D, "fp32"), _rows(rng, S, n, H, D, "fp32"), _rows(rng, S, n, H, D, "fp32")
    out = torch.empty_like(q)
    bits = [[(1 << (i + 1)) - 1 for i in range(n)]] * S
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.attention(q, k, v, scale=0.1, out=out)
        cache.append(k, v)
    assert cache.len.tolist() == [100, 10]
    for step in range(4):
        q.copy_(_rows(rng, S, n, H * G, D, "fp32"))
        k.copy_(_rows(rng, S, n, H, D, "fp32"))
        if step == 2:
            cache.len[1] = 0
            ref.rows[1] = tuple(x[:0] for x in ref.rows[1])
        graph.replay()
        want, _ = out.clone(), torch.cuda.synchronize()
        back = cache.len.clone()
        cache.len.copy_(_i32([ref.length(s) for s in range(S)]))
        eager, _ = _check_attention(cache, ref, q, k, v, 0.1, bits)
        assert torch.equal(eager, want)
        cache.len.copy_(back)
        for s in range(S):
            ref.append(s, _np(k)[s], _np(v)[s])
    _check_state(cache, ref)


def test_calls_at_once_on_several_streams_and_threads():
    import threading
    rng = np.random.default_rng(17)
    S, H, G, D = 3, 4, 4, 128
    cache, _ = _filled(rng, S, H, D, [3000, 1700, 5])
    work = []
    for n in (1, 1, 3, 20, 40, 1):
        q, k, v = _rows(rng, S, n, H * G, D, "fp32"), _rows(rng, S, n, H, D, "fp32"), _rows(rng, S, n, H, D, "fp32")
        work.append((q, k, v, cache.attention(q, k, v, scale=0.1)))
    torch.cuda.synchronize()
    streams, bad = [torch.cuda.Stream() for _ in range(3)], []

    def go(i):
        for _ in range(20):
            q, k, v, want = work[i]
            got = cache.attention(q, k, v, scale=0.1, stream=streams[i % 3])
            streams[i % 3].synchronize()
            if not torch.equal(got, want):
                bad.append(i)

    threads = [threading.Thread(target=go, args=(i,)) for i in range(len(work))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad and cache.check() == 0


def test_workspace_of_the_caller():
    """Any content, and calls of other sizes in the same one: the tickets at its start are set by the call."""
    rng = np.random.default_rng(18)
    cache, ref = _filled(rng, 2, 2, 64, [700, 90])
    ws = torch.full((64 << 20,), 0xab, dtype=torch.uint8, device="cuda")
    for n in (1, 30, 2):
        q, k, v = _rows(rng, 2, n, 8, 64, "fp32"), _rows(rng, 2, n, 2, 64, "fp32"), _rows(rng, 2, n, 2, 64, "fp32")
        got = cache.attention(q, k, v, scale=0.2, workspace=ws)
        assert torch.equal(got, cache.attention(q, k, v, scale=0.2))
        ws[W.KV4_TICKETS:].fill_(0xff)
    with pytest.raises(W.W4A8Error):
        cache.attention(q, k, v, workspace=ws[:W.KV4_TICKETS])
    with pytest.raises(ValueError):
        cache.attention(q, k, v, workspace=ws[::2])


def test_long_context_behind_four_gigabytes_of_pages():
    """A pool of more than 2^32 bytes, 65537 tokens in its last pages."""
    rng = np.random.default_rng(19)
    H, G, D, L = 8, 2, 128, 65537
    P = (L + 63) // 64
    N = (1 << 32) // (H * 68 * D) + P + 10
    cache = W.KV4Cache(1, H, D, P, N)
    cache.tensors["table"].copy_(_i32(N - P + rng.permutation(P)[None]))
    ref = O.Cache(1, H, D)
    k, v = _rows(rng, 1, L, H, D, "bf16"), _rows(rng, 1, L, H, D, "bf16")
    cache.append(k, v)
    ref.append(0, _np(k)[0], _np(v)[0])
    first = L - 100
    kk, _ = cache.read(_i32([first]), 100)
    assert np.array_equal(_np(kk)[0, :, H - 1], ref.held(0, H - 1)[0][first:].astype(np.float32))
    for dtype in ("fp32", "bf16"):
        q, kn, vn = _rows(rng, 1, 1, H * G, D, dtype, 2.0), _rows(rng, 1, 1, H, D, dtype), _rows(rng, 1, 1, H, D, dtype)
        _check_attention(cache, ref, q, kn, vn, D ** -0.5, [[1]], rows={(0, 0, 0), (0, 0, 2 * H - 1)})


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_waits_that_run_out(n, dtype):
    """One CTA's copies are withheld: its rows are NaN, the others are right, the status word says so, and the next call is as ever."""
    import ctypes
    rng = np.random.default_rng(20)
    S, H, G, D = 3, 2, 4, 128
    cache, _ = _filled(rng, S, H, D, [6000, 2000, 40], dtype)
    q, k, v = _rows(rng, S, n, H * G, D, dtype), _rows(rng, S, n, H, D, dtype), _rows(rng, S, n, H, D, dtype)
    want = cache.attention(q, k, v, scale=0.1)
    torch.cuda.synchronize()
    real = cache._attention
    try:
        cache._attention = lambda c, a, w, b, st: W.lib().w4a8_kv4_attention_inject_timeout(c, a, w, b, 3, st)
        got = cache.attention(q, k, v, scale=0.1)
        assert cache.check() == W.FLAG_ERR_TIMEOUT
    finally:
        cache._attention = real
    nan = torch.isnan(got).flatten(2).any(-1)
    assert nan.any() and not nan.all()
    bad = torch.isnan(got).any(-1)
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], want[~bad])
    cache.tensors["ctl"].zero_()
    assert torch.equal(cache.attention(q, k, v, scale=0.1), want) and cache.check() == 0


def test_refusals_in_python():
    rng = np.random.default_rng(21)
    cache, _ = _filled(rng, 2, 2, 64, [10, 20])
    q, k, v = _rows(rng, 2, 1, 4, 64, "fp32"), _rows(rng, 2, 1, 2, 64, "fp32"), _rows(rng, 2, 1, 2, 64, "fp32")
    for args, kw in (((q.half(), k, v), {}), ((q, k, None), {}), ((q, k.bfloat16(), v), {}), ((q, k[:, :, :1], v), {}),
                     ((q.transpose(2, 3), k, v), {}), ((q[:1], k, v), {}), ((q.cpu(), k, v), {}),
                     ((q, k, v), dict(counts=_i32([1]))), ((q, k, v), dict(mask=_i32([[1], [1]]))), ((q, k, v), dict(out=q[:, :, :2]))):
        with pytest.raises(ValueError):
            cache.attention(*args, **kw)
    with pytest.raises(W.W4A8Error):
        cache.attention(q, k, v, out=q)
    with pytest.raises(ValueError):
        cache.read(_i32([0, 0]), 4, dtype=torch.float16)
    with pytest.raises(ValueError):
        W.KV4Cache(2, 2, 64, 1, 2, tensors=cache.tensors)
    with pytest.raises(W.W4A8Error):
        W.KV4Cache(1, 1, 96, 1)
