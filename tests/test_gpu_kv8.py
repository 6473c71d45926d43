"""The 8-bit key/value cache through the C ABI against its definition (oracle/kv8.py, 64 bits).

Exact: codes, scales, code sums, tail rows, lengths, tables, selected pages, evicted pages (all decided in
fp32 or integers on both sides).

Attention bounds, from the operands.  Let A = the largest sum_d |scale q_d k_d| of a row.  fp32 calls split each
operand into f16 hi + lo (2^-21 relative of a product, two operands) and accumulate in fp32 (at most 2^-20 of the
sum of magnitudes): a logit is off by less than d = 2^-19 A, a weight by 2 d relative, and the weights' own
split and the value sums add less than 2^-17, so |out - ref| <= max|V| (2 d + 2^-17).  bf16 calls use one f16
factor: tail rows of fp32 appends 2^-11 relative (d = 2^-10 A with both factors rounded), weights 2^-11
numerator and denominator, and round the output by 2^-8 of its value: max|V| (2 d + 2^-9) + 2^-8 |ref|.
The mass of a page is a sum of weights: 2 d + 2^-17 relative (bf16: 2 d + 2^-9), plus fp32 additions.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import w4a8_verify_gb300 as W
from oracle import kv8 as O

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
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _rows(rng, S, n, H, D, dtype, amp=1.0):
    return torch.from_numpy((rng.standard_normal((S, n, H, D)) * amp).astype(np.float32)).cuda().to(TYPES[dtype])


def _filled(rng, S, H, D, lens, dtype="fp32", max_pages=None, shuffle=True, amp=1.0):
    """A cache and its oracle with the given lengths, tables shuffled."""
    P = max_pages or max(lens) // 64 + 2
    cache, ref = W.KV8Cache(S, H, D, P), O.Cache(S, H, D, P)
    if shuffle:
        for s in range(S):
            for h in range(H):
                cache.tensors["table"][s, h] = _i32(rng.permutation(P).tolist())
    n = max(max(lens), 1)
    k, v = _rows(rng, S, n, H, D, dtype, amp), _rows(rng, S, n, H, D, dtype, amp * 0.5)
    cache.append(k, v, counts=_i32(list(lens)))
    for s in range(S):
        ref.append(s, _np(k)[s, :lens[s]], _np(v)[s, :lens[s]])
    return cache, ref


def _check_state(cache, ref):
    D = cache.shape[2]
    t = {k: v.cpu().numpy() for k, v in cache.tensors.items()}
    kb, vb = O.byte_order(D, O.key_byte), O.byte_order(D, O.value_byte)
    assert t["len"].tolist() == [ref.length(s) for s in range(ref.S)]
    for s in range(ref.S):
        for h in range(ref.H):
            assert sorted(t["table"][s, h]) == list(range(ref.max_pages))
            for p, (ck, sk, cv, sv) in enumerate(ref.pages[s][h]):
                pg = t["table"][s, h, p]
                assert np.array_equal(t["codes"][s, h, pg, 0][kb].astype(int) - 128, ck), (s, h, p)
                assert np.array_equal(t["codes"][s, h, pg, 1][vb].astype(int) - 128, cv), (s, h, p)
                assert np.array_equal(t["scales"][s, h, pg], np.array([sk, sv]), equal_nan=True)
                assert np.array_equal(t["sums"][s, h, pg], ck.sum(axis=0))
            n = len(ref.open[s][0])
            for i in range(2):
                assert np.array_equal(t["tail"][s, h, i, :n], ref.open[s][i][:, h])


# ------------------------------------------------------------------------------- append and read

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_append_in_pieces(D, dtype):
    """Single rows, page-completing pieces, several pages at once, sequences that get nothing: every bit."""
    rng = np.random.default_rng(D + len(dtype))
    S, H, P = 3, 2, 9
    cache, ref = W.KV8Cache(S, H, D, P), O.Cache(S, H, D, P)
    cache.tensors["table"].copy_(_i32(np.stack([[rng.permutation(P) for _ in range(H)] for _ in range(S)]).tolist()))
    for n in (1, 62, 1, 1, 130, 64, 5, 63, 200):
        k, v = _rows(rng, S, n, H, D, dtype, 3.0), _rows(rng, S, n, H, D, dtype)
        counts = [n, int(rng.integers(0, n + 1)), 0 if n % 2 else n]
        cache.append(k, v, counts=_i32(counts))
        for s in range(S):
            ref.append(s, _np(k)[s, :counts[s]], _np(v)[s, :counts[s]])
    _check_state(cache, ref)
    assert cache.check() == 0
    first = [0, 70, 500]
    kk, vv = (_np(x) for x in cache.read(_i32(first), 150))
    for s in range(S):
        for h in range(H):
            k, v = ref.held(s, h)
            for got, want in ((kk, k), (vv, v)):
                w = np.zeros((150, D))
                x = want[first[s]:first[s] + 150]
                w[:len(x)] = x
                assert np.array_equal(got[s, :, h], w.astype(np.float32))


def test_append_strides_index_and_len_out():
    """Rows inside a fused tensor, the accepted path of a tree (rows out of order and twice), lengths kept apart."""
    rng = np.random.default_rng(5)
    S, H, D, n = 2, 3, 64, 16
    cache, ref = _filled(rng, S, H, D, [60, 127])
    qkv = _rows(rng, S, n, 4 * H, D, "fp32")
    k, v = qkv[:, :, H:2 * H], qkv[:, :, 2 * H:3 * H]
    index = [[0, 3, 3, 15, 9], [7, 0, 1, 2, 14]]
    out = torch.full((S,), -7, dtype=torch.int32, device="cuda")
    cache.append(k, v, counts=_i32([5, 4]), index=_i32(index), len_out=out)
    assert out.tolist() == [65, 131] and cache.len.tolist() == [60, 127]
    cache.len.copy_(out)
    for s, c in enumerate((5, 4)):
        ref.append(s, _np(k)[s, index[s][:c]], _np(v)[s, index[s][:c]])
    _check_state(cache, ref)
    # a transposed source: [n_seqs][heads][n][head_dim]
    x = _rows(rng, S, H, 70, D, "bf16").transpose(1, 2)
    cache.append(x, x)
    for s in range(S):
        ref.append(s, _np(x)[s], _np(x)[s])
    _check_state(cache, ref)


def test_append_special_values():
    """Zero pages, one value, subnormals, the largest values, NaN and infinity."""
    rng = np.random.default_rng(6)
    D, H = 64, 1
    x = np.zeros((1, 64 * 7, H, D), np.float32)
    x[0, 64 + 5, 0, 9] = -3.0
    x[0, 128:192] = rng.standard_normal((64, H, D)) * 1e-42
    x[0, 192:256] = rng.standard_normal((64, H, D)) * 1e38 * 0.5
    x[0, 256:320] = rng.standard_normal((64, H, D))
    x[0, 300, 0, 63] = np.nan
    x[0, 320:384] = rng.standard_normal((64, H, D))
    x[0, 321, 0, 0] = -np.inf
    t = torch.from_numpy(x).cuda()
    cache, ref = W.KV8Cache(1, H, D, 8), O.Cache(1, H, D, 8)
    cache.append(t, t.flip(1))
    ref.append(0, x[0], x[0, ::-1])
    _check_state(cache, ref)


def test_append_refuses_on_the_device():
    rng = np.random.default_rng(7)
    cache, ref = _filled(rng, 3, 1, 64, [60, 120, 130], max_pages=2)
    k = _rows(rng, 3, 70, 1, 64, "fp32")
    cache.append(k, k, counts=_i32([70, 70, 1]))               # 60 + 70 <= 191, 120 + 70 <= 191, 131
    for s, c in enumerate((70, 70, 1)):
        ref.append(s, _np(k)[s, :c], _np(k)[s, :c])
    _check_state(cache, ref)
    assert cache.check() == 0
    cache.append(k, k, counts=_i32([61, 2, 71]))               # 130 + 61 = 191 fits, 190 + 2 does not, 71 > n
    ref.append(0, _np(k)[0, :61], _np(k)[0, :61])
    _check_state(cache, ref)
    assert cache.check() == W.FLAG_ERR_CAPACITY
    cache.tensors["ctl"].zero_()
    idx = _i32([[0], [70], [-1]])
    cache.append(k[:, :1], k[:, :1], index=idx, counts=_i32([0, 1, 1]))
    _check_state(cache, ref)
    assert cache.check() == W.FLAG_ERR_TOKEN
    cache.reset()
    assert cache.check() == 0 and cache.len.tolist() == [0, 0, 0]


# ------------------------------------------------------------------------------- attention

def _tree_mask(rng, n):
    rows = [1]
    for i in range(1, n):
        rows.append(rows[int(rng.integers(0, i))] | 1 << i)
    return rows


def _signed(m):
    return m - (1 << 64) if m >> 63 else m


def _attend(cache, ref, q, k, v, scale, counts=None, mask=None, pages=None, mass=None):
    """Runs the attention and checks every row (and the mass) against the oracle."""
    S, n, Hq, D = q.shape
    H = ref.H
    G = Hq // H
    counts = [n] * S if counts is None else counts
    fill = 7.25
    out = torch.full(q.shape, fill, dtype=q.dtype, device="cuda")
    mt = None if mask is None else torch.tensor([[_signed(m) for m in r] for r in mask], dtype=torch.int64, device="cuda")
    mo = None if mass is None else torch.empty_like(mass)
    cache.attention(q, k, v, scale=scale, counts=_i32(counts), mask=mt, out=out, mass=mass, mass_out=mo,
                    pages=None if pages is None else _i32(pages))
    got, qn = _np(out), _np(q).astype(np.float64)
    kn = None if k is None else _np(k)
    vn = None if v is None else _np(v)
    bf = q.dtype == torch.bfloat16
    want_mass = None if mass is None else mass.double().cpu().numpy()
    slack = 0.0
    num = den = 0.0
    for s in range(S):
        assert (got[s, counts[s]:] == fill).all()              # rows behind the last one
        for i in range(counts[s]):
            m = (1 << (i + 1)) - 1 if mask is None else mask[s][i]
            for hq in range(Hq):
                h, c = hq // G, counts[s] if k is not None else 0
                pg = None if pages is None else [p for p in pages[s][i][h] if p >= 0]
                kr = kn[s, :c, h] if c else np.zeros((0, D))
                vr = vn[s, :c, h] if c else np.zeros((0, D))
                o, w, A = O.attention(ref, s, h, qn[s, i, hq], kr, vr, m, scale, pg)
                seen = [j for j in range(c) if m >> j & 1]
                V = max([np.abs(ref.held(s, h, pg)[1]).max(initial=0.0)] + [np.abs(vr[j]).max() for j in seen])
                d = (2.0 ** -10 if bf else 2.0 ** -19) * A
                tol = V * (2 * d + 2.0 ** -9) + 2.0 ** -8 * np.abs(o) if bf else V * (2 * d + 2.0 ** -17)
                assert (np.abs(got[s, i, hq] - o) <= tol).all(), (s, i, hq, np.abs(got[s, i, hq] - o).max(), np.max(tol))
                num, den = num + ((got[s, i, hq] - o) ** 2).sum(), den + (o ** 2).sum()
                if mass is not None:
                    full = len(ref.pages[s][h])
                    want_mass[s, h, :full] += w[:64 * full].reshape(full, 64).sum(axis=1)
                    slack = max(slack, 2 * d + (2.0 ** -9 if bf else 2.0 ** -17))
    if den:                                                    # on the whole the errors are far below their bounds
        assert (num / den) ** 0.5 <= (4e-3 if bf else 5e-6)
    if mass is not None:
        g = mo.cpu().numpy()
        old = mass.cpu().numpy()
        assert (np.abs(g - want_mass) <= slack * (want_mass - old) + 2.0 ** -20 * want_mass + 1e-30).all()
    return out


SHAPES = [(2, 7, 64), (2, 4, 128), (1, 1, 64), (1, 16, 128), (3, 5, 64)]
LENS = [0, 1, 63, 64, 65, 128, 200, 391]


@pytest.mark.parametrize("H,G,D", SHAPES)
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_single_rows_at_many_lengths(H, G, D, dtype):
    rng = np.random.default_rng(H * 100 + G + D)
    cache, ref = _filled(rng, len(LENS), H, D, LENS, dtype)
    q = _rows(rng, len(LENS), 1, H * G, D, dtype, 2.0)
    k, v = _rows(rng, len(LENS), 1, H, D, dtype), _rows(rng, len(LENS), 1, H, D, dtype)
    mass = torch.rand(len(LENS), H, cache.shape[3], device="cuda")
    _attend(cache, ref, q, k, v, D ** -0.5)
    _attend(cache, ref, q, k, v, D ** -0.5, mass=mass)
    _attend(cache, ref, q, None, None, D ** -0.5)              # the cache alone: an empty one gives 0
    assert cache.check() == 0


@pytest.mark.parametrize("n", [2, 3, 5, 8, 9, 16, 17, 31, 64])
@pytest.mark.parametrize("H,G,D,dtype", [(2, 4, 128, "fp32"), (1, 7, 64, "bf16"), (1, 3, 64, "fp32"),
                                         (2, 4, 128, "bf16"), (1, 16, 128, "fp32")])
def test_trees_chains_and_counts(n, H, G, D, dtype):
    rng = np.random.default_rng(n * 10 + G)
    lens = [0, 70, 130]
    cache, ref = _filled(rng, 3, H, D, lens, dtype)
    q = _rows(rng, 3, n, H * G, D, dtype, 2.0)
    k, v = _rows(rng, 3, n, H, D, dtype), _rows(rng, 3, n, H, D, dtype)
    mask = [_tree_mask(rng, n) for _ in range(3)]
    _attend(cache, ref, q, k, v, D ** -0.5, mask=mask, counts=[n, n - 1, 1])
    if n in (3, 16, 64):
        _attend(cache, ref, q, k, v, D ** -0.5, counts=[n - 1, 0, n], mass=torch.rand(3, H, cache.shape[3], device="cuda"))


@pytest.mark.parametrize("n,H,G,D,dtype", [(64, 2, 4, 128, "fp32"), (64, 2, 2, 64, "bf16"), (48, 1, 16, 64, "fp32"),
                                           (20, 3, 5, 128, "bf16")])
def test_padded_batches(n, H, G, D, dtype):
    """Sequences of few rows between full ones: blocks of rows that nobody has take no part."""
    rng = np.random.default_rng(n + D)
    lens = [200, 330, 64, 129, 500]
    cache, ref = _filled(rng, 5, H, D, lens, dtype)
    q = _rows(rng, 5, n, H * G, D, dtype, 2.0)
    k, v = _rows(rng, 5, n, H, D, dtype), _rows(rng, 5, n, H, D, dtype)
    for counts in ([1, n, 3, n, 2], [n, 0, n - 1, 1, n], [0, 1, n // 2 + 1, 0, n // 4 + 1]):
        _attend(cache, ref, q, k, v, D ** -0.5, counts=counts)
        _attend(cache, ref, q, k, v, D ** -0.5, counts=counts, mass=torch.rand(5, H, cache.shape[3], device="cuda"))
    assert cache.check() == 0


@pytest.mark.parametrize("S,n,H,G,D,dtype", [(38, 7, 2, 7, 64, "fp32"), (40, 14, 2, 5, 128, "bf16"), (20, 33, 3, 3, 64, "bf16"),
                                             (21, 16, 4, 4, 128, "fp32")])
def test_many_sequences_of_several_rows(S, n, H, G, D, dtype):
    """Many parts of fp32 rows, with all pages and with lists of them."""
    rng = np.random.default_rng(S + n)
    lens = [int(x) for x in rng.integers(0, 210, S)]
    cache, ref = _filled(rng, S, H, D, lens, dtype)
    q = _rows(rng, S, n, H * G, D, dtype, 2.0)
    k, v = _rows(rng, S, n, H, D, dtype), _rows(rng, S, n, H, D, dtype)
    mask = [_tree_mask(rng, n) for _ in range(S)]
    counts = [int(x) for x in rng.integers(0, n + 1, S)]
    _attend(cache, ref, q, k, v, D ** -0.5, mask=mask, counts=counts)
    pages = cache.select(q, 2, first_pages=1, counts=_i32(counts))
    _attend(cache, ref, q, k, v, D ** -0.5, mask=mask, counts=counts, pages=pages.tolist())
    assert cache.check() == 0


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("n", [4, 16, 40])
def test_masked_rows_with_nan_and_infinities(dtype, n):
    """A new row that a row does not see has no effect on it; rows that see nothing are 0; padded rows are not read."""
    rng = np.random.default_rng(n)
    S, H, G, D = 2, 2, 4, 128
    cache, ref = _filled(rng, S, H, D, [0, 75], dtype)
    q = _rows(rng, S, n, H * G, D, dtype)
    k, v = _rows(rng, S, n, H, D, dtype), _rows(rng, S, n, H, D, dtype)
    k[:, 1], v[:, 1] = float("nan"), float("inf")
    v[:, 2, :, 5] = float("-inf")
    k[:, n - 1], v[:, n - 1] = float("nan"), float("nan")
    q[:, n - 1] = float("nan")
    keep = ((1 << n) - 1) & ~0b110 & ~(1 << (n - 1))
    mask = [[((1 << (i + 1)) - 1) & keep for i in range(n)] for _ in range(S)]
    mask[0][0] = mask[1][0] = 0
    _attend(cache, ref, q, k, v, D ** -0.5, mask=mask, counts=[n - 1, n - 1])
    # seen, they do their work: row 2 takes row 2's infinity, row 0 stays clean
    mask = [[1, 1, 1 | 4] + [1] * (n - 3) for _ in range(S)]
    out = cache.attention(q, k, v, scale=D ** -0.5, mask=torch.tensor(mask, device="cuda"), counts=_i32([n - 1] * S))
    bad = ~torch.isfinite(out[:, :n - 1].float())
    assert bad[:, 2, :, 5].all() and not bad[:, :2].any() and not bad[:, 3:].any()


@pytest.mark.parametrize("dtype,n", [("fp32", 2), ("bf16", 2), ("fp32", 40), ("bf16", 40)])
def test_non_finite_queries_and_pages(dtype, n):
    rng = np.random.default_rng(11)
    H, G, D = 1, 4, 64
    cache, ref = _filled(rng, 2, H, D, [130, 130])
    bad = _rows(rng, 2, 1, H, D, "fp32")
    bad[0] = float("inf")
    cache.append(bad.expand(2, 62, H, D), bad.expand(2, 62, H, D))      # completes page 2 of both, with infinities in 0's
    q = _rows(rng, 2, n, H * G, D, dtype)
    q[1, 0, 2, 7] = float("nan")
    q[1, 1, 0, 0] = float("inf")
    k = _rows(rng, 2, n, H, D, dtype)
    out = cache.attention(q, k, k, scale=0.1)
    assert torch.isnan(out[0]).all()
    nan = torch.isnan(out[1])
    assert nan[0, 2].all() and nan[1, 0].all() and int(nan.sum()) == 2 * D


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_extreme_magnitudes(dtype):
    """Tiny and huge rows, a huge page next to ordinary ones, peaked softmax: scaled splits, no f16 overflow."""
    rng = np.random.default_rng(12)
    H, G, D = 1, 4, 64
    for amp_k, amp_q, scale in ((1e-6, 1e5, 1.0), (3e4, 1e-4, 0.125), (1e8, 1e-9, 1.0), (1.0, 30.0, 1.0)):
        cache, ref = W.KV8Cache(1, H, D, 6), O.Cache(1, H, D, 6)
        x = _rows(rng, 1, 210, H, D, dtype, amp_k)
        v = _rows(rng, 1, 210, H, D, dtype)
        v[:, 64:128] *= 1e4
        cache.append(x, v)
        ref.append(0, _np(x)[0], _np(v)[0])
        q = _rows(rng, 1, 3, H * G, D, dtype, amp_q)
        if amp_q == 30.0 and dtype == "bf16":
            continue                                           # logits of thousands: f16 factors decide nothing
        _attend(cache, ref, q, _rows(rng, 1, 3, H, D, dtype, amp_k), _rows(rng, 1, 3, H, D, dtype), scale)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_strided_and_unaligned_rows(dtype):
    rng = np.random.default_rng(13)
    S, H, G, D, n = 2, 2, 3, 64, 5
    cache, ref = _filled(rng, S, H, D, [100, 64], dtype)
    flat = _rows(rng, 1, 1, 1, S * n * (G + 2) * H * (D + 1) + 1, dtype).reshape(-1)[1:]   # one element off
    qkv = flat.view(S, n, (G + 2) * H, D + 1)[..., :D]
    q, k, v = qkv[:, :, :G * H], qkv[:, :, G * H:(G + 1) * H], qkv[:, :, (G + 1) * H:]
    want = _attend(cache, ref, q, k, v, 0.2)
    buf = torch.zeros(n, S, G * H, 2 * D + 1, dtype=q.dtype, device="cuda")
    out = buf.permute(1, 0, 2, 3)[..., 1:D + 1]
    cache.attention(q, k, v, scale=0.2, out=out)
    assert torch.equal(out, want)
    assert not buf[..., 0].any() and not buf[..., D + 1:].any()


def test_out_of_range_state_is_left_out():
    rng = np.random.default_rng(14)
    H, G, D = 1, 4, 64
    cache, ref = _filled(rng, 3, H, D, [70, 70, 70])
    q = _rows(rng, 3, 1, H * G, D, "fp32")
    k = _rows(rng, 3, 1, H, D, "fp32")
    want = cache.attention(q, k, k, scale=0.1)
    assert cache.check() == 0
    cache.len.copy_(_i32([70, -1, 64 * cache.shape[3] + 64]))
    out = torch.full_like(q, 3.0)
    cache.attention(q, k, k, scale=0.1, out=out)
    assert torch.equal(out[0], want[0]) and (out[1:] == 3.0).all()
    assert cache.check() == W.FLAG_ERR_CAPACITY
    cache.tensors["ctl"].zero_()
    cache.len.copy_(_i32([70, 70, 70]))
    cache.attention(q, k, k, scale=0.1, out=out, counts=_i32([1, 2, -1]))
    assert cache.check() == W.FLAG_ERR_CAPACITY
    cache.tensors["ctl"].zero_()
    old = cache.tensors["table"].clone()
    cache.tensors["table"][0, 0, 0] = cache.shape[3]
    cache.tensors["table"][1, 0, 0] = -1
    cache.attention(q, k, k, scale=0.1, out=out)
    assert torch.equal(out[2], want[2]) and cache.check() == W.FLAG_ERR_TREE
    cache.tensors["ctl"].zero_()
    cache.tensors["table"].copy_(old)
    cache.attention(q, k, k, scale=0.1, out=out)
    assert torch.equal(out, want) and cache.check() == 0


# ------------------------------------------------------------------------------- selection, sparse attention

@pytest.mark.parametrize("H,G,D,n,dtype", [(2, 4, 128, 1, "fp32"), (1, 7, 64, 3, "bf16"), (3, 1, 64, 2, "fp32"),
                                           (1, 16, 128, 5, "bf16")])
@pytest.mark.parametrize("top_k,first,last", [(1, 0, 0), (4, 1, 2), (5, 0, 3), (2, 2, 2), (9, 0, 0), (40, 1, 1)])
def test_select_and_sparse_attention(H, G, D, n, dtype, top_k, first, last):
    rng = np.random.default_rng(G * n + top_k)
    lens = [0, 63, 64 * 5, 64 * 9 + 10]
    cache, ref = _filled(rng, 4, H, D, lens, dtype, max_pages=12)
    q = _rows(rng, 4, n, H * G, D, dtype, 2.0)
    counts = [n, n, max(0, n - 1), n]
    pages = cache.select(q, top_k, first_pages=first, last_pages=last, counts=_i32(counts))
    got = pages.cpu().numpy()
    for s in range(4):
        for i in range(n):
            for h in range(H):
                want = O.select(ref, s, h, _np(q)[s, i, h * G:(h + 1) * G], top_k, first, last) if i < counts[s] else []
                assert got[s, i, h].tolist() == want + [-1] * (top_k - len(want)), (s, i, h)
    k, v = _rows(rng, 4, n, H, D, dtype), _rows(rng, 4, n, H, D, dtype)
    mask = [_tree_mask(rng, n) for _ in range(4)]
    _attend(cache, ref, q, k, v, D ** -0.5, counts=counts, mask=mask, pages=got.tolist())
    assert cache.check() == 0


def test_more_rows_than_a_grid_dimension():
    """4096 sequences (65536 lists and 131072 segments): every limit of the grids that only the first dimension lifts."""
    rng = np.random.default_rng(23)
    S, H, D, n = 4096, 2, 64, 16
    c = _random_cache(2, [130 if s % 7 == 0 else 200 for s in range(S)], H, D, max_pages=3)
    q, k = _rows(rng, S, n, H, D, "bf16"), _rows(rng, S, n, H, D, "bf16")
    pages = c.select(q, 2)
    out = c.attention(q, k, k, scale=0.1, pages=pages)
    at = [0, 1, 7, S - 2, S - 1]
    small = W.KV8Cache(len(at), H, D, 3, tensors={x: (t if x == "ctl" else t[at].contiguous()) for x, t in c.tensors.items()})
    assert torch.equal(pages[at], small.select(q[at].contiguous(), 2))
    _long_check(c, q, k, k, 0.1, out, range(H), at, pages=pages)
    out = c.attention(q[:, :1], k[:, :1], k[:, :1], scale=0.1)
    _long_check(c, q[:, :1], k[:, :1], k[:, :1], 0.1, out, range(H), at)
    assert c.check() == 0


def test_select_ties_zero_queries_and_nan_scales():
    D, H = 64, 1
    cache, ref = W.KV8Cache(1, H, D, 40), O.Cache(1, H, D, 40)
    x = torch.ones(1, 64 * 30, H, D, device="cuda")            # every page scores the same
    x[:, 64 * 20:64 * 21] = float("nan")
    cache.append(x, torch.ones_like(x))
    ref.append(0, _np(x)[0], np.ones_like(_np(x)[0]))
    for q in (torch.ones(1, 1, 2, D, device="cuda"), torch.zeros(1, 1, 2, D, device="cuda"),
              -torch.ones(1, 1, 2, D, device="cuda")):
        got = cache.select(q, 4).cpu().numpy()[0, 0, 0].tolist()
        assert got == O.select(ref, 0, 0, _np(q)[0, 0], 4, 0, 0) == [0, 1, 2, 20]


def test_page_lists_out_of_order_are_left_out():
    rng = np.random.default_rng(21)
    H, G, D = 1, 4, 64
    cache, ref = _filled(rng, 1, H, D, [64 * 6], max_pages=8)
    q = _rows(rng, 1, 1, H * G, D, "fp32")
    k = _rows(rng, 1, 1, H, D, "fp32")
    _attend(cache, ref, q, k, k, 0.2, pages=[[[[-1, -1, -1, -1]]]])
    _attend(cache, ref, q, k, k, 0.2, pages=[[[[1, 4, -1, -1]]]])
    assert cache.check() == 0
    want = cache.attention(q, k, k, scale=0.2, pages=_i32([[[[1, 4, -1, -1]]]]))
    for bad in ([1, 4, 4, -1], [1, 4, 2, -1], [1, 4, 6, -1], [1, 4, -2, -1], [1, 4, -1, 5]):
        out = cache.attention(q, k, k, scale=0.2, pages=_i32([[[bad]]]))
        assert torch.equal(out, want), bad
        assert cache.check() == W.FLAG_ERR_TREE
        cache.tensors["ctl"].zero_()


# ------------------------------------------------------------------------------- eviction

@pytest.mark.parametrize("keep,first,last", [(0, 0, 0), (1, 0, 0), (3, 1, 1), (5, 2, 4), (100, 0, 0), (7, 0, 2)])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict(keep, first, last, in_place):
    rng = np.random.default_rng(keep)
    lens, H, D, P = [0, 63, 64 * 5 + 1, 64 * 37, 64 * 20 + 63], 3, 64, 40
    cache, ref = _filled(rng, len(lens), H, D, lens, max_pages=P)
    mass = torch.from_numpy(rng.integers(0, 6, (len(lens), H, P)).astype(np.float32)).cuda()
    mass[3, 1, 7], mass[3, 1, 20] = float("nan"), float("inf")
    mass[3, 2, 3] = -0.0
    m0, t0 = _np(mass), cache.tensors["table"].cpu().numpy()
    held = [[list(ref.pages[s][h]) for h in range(H)] for s in range(len(lens))]
    table, new, length = cache.evict(mass, keep, first_pages=first, last_pages=last, in_place=in_place)
    table, new = table.cpu().numpy(), _np(new)
    for s, L in enumerate(lens):
        n = L // 64
        for h in range(H):
            kept, gone = O.evict(m0[s, h, :n].tolist(), keep, first, last)
            want = list(t0[s, h, kept]) + list(t0[s, h, gone]) + list(t0[s, h, n:])
            assert table[s, h].tolist() == want
            assert np.array_equal(new[s, h], np.concatenate([m0[s, h, kept], np.zeros(P - len(kept), np.float32)]),
                                  equal_nan=True)
            ref.pages[s][h] = [held[s][h][p] for p in kept]
        assert int(length[s]) == L - 64 * (n - min(n, keep))
    if in_place:                                               # the cache goes on: append into freed pages, attend
        q, k = _rows(rng, len(lens), 2, H * 2, D, "fp32"), _rows(rng, len(lens), 70, H, D, "fp32")
        _attend(cache, ref, q, k[:, :2], k[:, 2:4], 0.2)
        cache.append(k, k)
        for s in range(len(lens)):
            ref.append(s, _np(k)[s], _np(k)[s])
        _check_state(cache, ref)
        _attend(cache, ref, q, k[:, :2], k[:, 2:4], 0.2)


# ------------------------------------------------------------------------------- together

def test_a_served_batch_with_eviction_and_sparse_reads():
    """Decode steps of a batch: attend with mass, append, thin at a limit, then sparse steps; the oracle alongside."""
    rng = np.random.default_rng(31)
    S, H, G, D, P = 3, 2, 4, 64, 8
    cache, ref = _filled(rng, S, H, D, [250, 128, 3], max_pages=P)
    mass = torch.zeros(S, H, P, device="cuda")
    for step in range(6):
        n = 1 + step % 3
        q, k, v = _rows(rng, S, n, H * G, D, "fp32", 2.0), _rows(rng, S, n, H, D, "fp32"), _rows(rng, S, n, H, D, "fp32")
        before = mass.clone()
        _attend(cache, ref, q, k, v, D ** -0.5, mass=mass)
        cache.attention(q, k, v, scale=D ** -0.5, mass=mass, mass_out=mass)     # accumulates in place
        assert (mass >= before).all() and float((mass - before).sum()) > 0
        cache.append(k, v)
        for s in range(S):
            ref.append(s, _np(k)[s], _np(v)[s])
        if step == 3:
            m = _np(mass)
            cache.evict(mass, 2, first_pages=1, in_place=True)
            for s in range(S):
                for h in range(H):
                    kept, _ = O.evict(m[s, h, :len(ref.pages[s][h])].tolist(), 2, 1, 0)
                    ref.pages[s][h] = [ref.pages[s][h][p] for p in kept]
        _check_state(cache, ref)
        pages = cache.select(q, 2, last_pages=1)
        _attend(cache, ref, q, k, v, D ** -0.5, pages=pages.cpu().numpy().tolist())
    assert cache.check() == 0


def test_same_result_as_the_session_attention():
    """The fp32 cache of a session holding exactly the 8-bit cache's values gives the same tree attention."""
    import synth
    import synth.cuda as SC
    from w4a8_verify_gb300 import models as WM
    shape = synth.ModelShape("d64-g7-kv2-1L", 1, 896, 14, 2, 64, 1024, 1024, 1024, False)

    def fill(kind, layer, out):
        out.normal_(0, 0.02)
    SC.lib()
    m = WM.build_model(shape.n_layers, shape.hidden, shape.n_heads, shape.n_kv_heads, shape.head_dim, shape.ffn,
                       shape.vocab, shape.tied, fill, shape.rms_eps, shape.rope_base)
    s = W.Session(m, 512, 576, 16, -1)
    L, n, H, D = 200, 11, 2, 64
    rng = np.random.default_rng(41)
    s.prefill(_i32(rng.integers(0, 1024, L + 1).tolist()), max_new=8)
    tok, parent = synth.random_tree(rng, n, shape.vocab)
    s.set_tree([int(t) for t in tok], [int(p) for p in parent])
    s.tree_verify_step(n)                                      # the nodes' keys and values, slots L .. L + n - 1
    kf, vf = (torch.empty(H, L + n, D, device="cuda") for _ in range(2))
    s.copy_kv(0, 0, L + n, kf, vf)
    cache = W.KV8Cache(1, H, D, 4)
    cache.append(kf[:, :L].transpose(0, 1)[None], vf[:, :L].transpose(0, 1)[None])
    kh, vh = cache.read(_i32([0]), L)                          # what the 8-bit cache holds, under both
    s.load_kv(0, 0, L, kh[0].transpose(0, 1).contiguous(), vh[0].transpose(0, 1).contiguous())
    assert float((kh[0].transpose(0, 1) - kf[:, :L]).abs().max()) <= float(cache.tensors["scales"][0, :, :3].max()) * 0.51
    q = _rows(rng, 1, n, 14, D, "fp32")
    want = torch.empty(n, 14 * D, device="cuda")
    s.attention(0, n, q[0].contiguous(), want)
    mask = []
    for i in range(n):
        mask.append((mask[parent[i]] if i else 0) | 1 << i)
    new = [x[:, L:].transpose(0, 1)[None] for x in (kf, vf)]
    got = cache.attention(q, new[0], new[1], mask=torch.tensor([mask], device="cuda"))
    err = (got[0].reshape(n, -1) - want).abs().max()
    assert float(err) <= 4e-5 * float(vf.abs().max())          # 2e-5 max|V| each, the session kernel's own bound


def test_captured_calls_follow_the_device_state():
    """One graph of attention (with mass) and append, replayed as the lengths grow past a page, equals eager calls;
    a second graph with its own workspace runs beside it."""
    rng = np.random.default_rng(51)
    S, H, G, D, n = 2, 2, 4, 128, 2
    lens = [62, 125]
    a, _ = _filled(rng, S, H, D, lens, max_pages=6, shuffle=False)
    b = W.KV8Cache(S, H, D, 6, tensors={k: t.clone() for k, t in a.tensors.items()})
    q, k, v = _rows(rng, S, n, H * G, D, "fp32"), _rows(rng, S, n, H, D, "fp32"), _rows(rng, S, n, H, D, "fp32")
    out, pages = torch.empty_like(q), torch.empty(S, n, H, 2, dtype=torch.int32, device="cuda")
    sparse = torch.empty_like(q)
    mass = torch.zeros(S, H, 6, device="cuda")

    def step(c, out, sparse, pages, mass):
        c.attention(q, k, v, scale=0.1, out=out, mass=mass, mass_out=mass)
        c.select(q, 2, out=pages)
        c.attention(q, k, v, scale=0.1, pages=pages, out=sparse)
        c.append(k, v)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        warm = W.KV8Cache(S, H, D, 6, tensors={k_: t.clone() for k_, t in a.tensors.items()})
        step(warm, torch.empty_like(q), torch.empty_like(q), torch.empty_like(pages), torch.zeros_like(mass))
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        step(a, out, sparse, pages, mass)
    o2, s2, p2, m2 = torch.empty_like(q), torch.empty_like(q), torch.empty_like(pages), torch.zeros_like(mass)
    for _ in range(40):
        q.normal_(), k.normal_(), v.normal_()
        graph.replay()
        step(b, o2, s2, p2, m2)
        assert torch.equal(out, o2) and torch.equal(sparse, s2) and torch.equal(pages, p2) and torch.equal(mass, m2)
    assert a.len.tolist() == b.len.tolist() == [142, 205]
    assert all(torch.equal(a.tensors[x], b.tensors[x]) for x in ("scales", "sums", "table", "tail"))
    assert a.check() == 0 and b.check() == 0


def test_two_streams_at_once():
    rng = np.random.default_rng(61)
    S, H, G, D = 2, 2, 4, 128
    jobs = []
    for i in range(2):
        cache, _ = _filled(rng, S, H, D, [700 + i, 333], "bf16")
        q, k = _rows(rng, S, 8, H * G, D, "bf16"), _rows(rng, S, 8, H, D, "bf16")
        jobs.append((cache, q, k, cache.attention(q, k, k, scale=0.1)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [[], []]
    for _ in range(10):
        for i, (cache, q, k, _) in enumerate(jobs):
            with torch.cuda.stream(streams[i]):
                got[i].append(cache.attention(q, k, k, scale=0.1))
    torch.cuda.synchronize()
    for i, (_, _, _, want) in enumerate(jobs):
        assert all(torch.equal(x, want) for x in got[i])


def test_binding_refusals():
    cache = W.KV8Cache(2, 2, 64, 4)
    q, k = torch.zeros(2, 1, 4, 64, device="cuda"), torch.zeros(2, 1, 2, 64, device="cuda")
    with pytest.raises(ValueError):
        cache.attention(q.half(), k.half(), k.half())
    with pytest.raises(ValueError):
        cache.attention(q, k.bfloat16(), k.bfloat16())
    with pytest.raises(ValueError):
        cache.attention(q, k)
    with pytest.raises(ValueError):
        cache.attention(q[:1], k[:1], k[:1])
    with pytest.raises(ValueError):
        cache.attention(q.cpu(), k, k)
    with pytest.raises(ValueError):
        cache.attention(q, k, k, counts=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        cache.attention(q.transpose(2, 3).contiguous().transpose(2, 3), k, k)
    with pytest.raises(ValueError):
        cache.evict(torch.zeros(2, 2, 5, device="cuda"), 1)
    with pytest.raises(ValueError):
        W.KV8Cache(2, 2, 64, 4, tensors={n: t[:1] for n, t in cache.tensors.items()})
    with pytest.raises(W.W4A8Error):
        W.KV8Cache(2, 2, 96, 4)
    with pytest.raises(W.W4A8Error):
        cache.attention(torch.zeros(2, 1, 3, 64, device="cuda"), k, k)
    with pytest.raises(W.W4A8Error):
        cache.attention(q, k, k, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda")[:0])
    with pytest.raises(W.W4A8Error):
        cache.select(q, 16385)


# ------------------------------------------------------------------------------- long ranges

def _random_cache(seed, lens, H, D, max_pages=None):
    """A cache of random codes, scales, tail rows and tables (code sums to match)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    S, P = len(lens), max_pages or max(lens) // 64 + 1
    c = W.KV8Cache(S, H, D, P)
    t = c.tensors
    t["codes"].random_(1, 256, generator=g)
    t["scales"].uniform_(0.01, 0.03, generator=g)
    t["tail"].normal_(0, 1, generator=g)
    t["table"].copy_(torch.rand(S, H, P, generator=g, device="cuda").argsort(dim=-1))
    t["len"].copy_(_i32(list(lens)))
    at = torch.from_numpy(O.byte_order(D, O.key_byte)).cuda()
    if P * S * H < 1 << 16:
        for s in range(S):
            t["sums"][s] = (t["codes"][s, :, :, 0][..., at.reshape(-1)].view(H, P, 64, D).int() - 128).sum(2)
    return c


def _held64(c, s, h, pages=None):
    """fp64 keys and values of the whole pages (or of those listed), then of the open page."""
    D, L, t = c.shape[2], int(c.len[s]), c.tensors
    at = [torch.from_numpy(O.byte_order(D, b)).cuda().reshape(-1) for b in (O.key_byte, O.value_byte)]
    phys = t["table"][s, h, :L // 64].long()
    phys = phys if pages is None else phys[pages]
    out = []
    for i in range(2):
        x = (t["codes"][s, h, phys, i][:, at[i]].double() - 128) * t["scales"][s, h, phys, i].double()[:, None]
        out.append(torch.cat([x.view(-1, D), t["tail"][s, h, i, :L % 64].double()]))
    return out


def _long_check(c, q, k, v, scale, out, heads, seqs, mass=None, mass_out=None, pages=None):
    """Rows of some heads and sequences against fp64 on the device (new rows causal), with the bounds of this file."""
    n, G, D = q.shape[1], q.shape[2] // c.shape[1], q.shape[3]
    bf = q.dtype == torch.bfloat16
    num = den = 0.0
    for s in seqs:
        for h in heads:
            for i in (range(n) if pages is not None else (None,)):
                lst = None if pages is None else pages[s, i, h][pages[s, i, h] >= 0].long()
                K, V = _held64(c, s, h, lst)
                held = len(K)
                K, V = torch.cat([K, k[s, :, h].double()]), torch.cat([V, v[s, :, h].double()])
                rows = slice(0, n) if i is None else slice(i, i + 1)
                Q = q[s, rows, h * G:(h + 1) * G].double().reshape(-1, D)
                logits = Q @ K.T * scale
                A = float((Q.abs() @ K.abs().T).max()) * abs(scale)
                node = torch.arange(n, device="cuda")[rows].repeat_interleave(G)
                hide = torch.arange(n, device="cuda")[None] > node[:, None]
                logits[:, held:][hide] = -float("inf")
                w = torch.softmax(logits, -1)
                ref = w @ V
                got = out[s, rows, h * G:(h + 1) * G].double().reshape(-1, D)
                d = (2.0 ** -10 if bf else 2.0 ** -19) * A
                tol = float(V.abs().max()) * (2 * d + (2.0 ** -9 if bf else 2.0 ** -17)) + (2.0 ** -8 * ref.abs() if bf else 0)
                assert ((got - ref).abs() <= tol).all(), (s, h, i, float((got - ref).abs().max()))
                num, den = num + float(((got - ref) ** 2).sum()), den + float((ref ** 2).sum())
                if mass is not None:
                    full = int(c.len[s]) // 64
                    add = w[:, :64 * full].sum(0).view(full, 64).sum(1)
                    have = (mass_out[s, h] - mass[s, h]).double()
                    slack = 2 * d + (2.0 ** -9 if bf else 2.0 ** -17)
                    assert ((have[:full] - add).abs() <= slack * add + 2.0 ** -20 * mass_out[s, h, :full].abs()).all()
                    assert not have[full:].any()
    assert (num / den) ** 0.5 <= (4e-3 if bf else 2e-6)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("S,H,G,D,n,L,mass", [
    (24, 2, 4, 128, 1, 6000, True),       # ragged batch: many segments for a worker
    (48, 4, 7, 64, 1, 9000, False),       # two warps on a page, rings of several pages
    (3, 2, 4, 128, 16, 5000, True),       # a tree's rows on two and four warps a page
    (2, 1, 12, 64, 8, 4000, False),       # twelve warps on a page
    (3, 2, 8, 128, 17, 9000, True),       # tcgen05: runs of several segments in a CTA, the ring of codes in turns
    (2, 3, 16, 64, 9, 12000, False),
])
def test_long_ragged_ranges(dtype, S, H, G, D, n, L, mass):
    rng = np.random.default_rng(S + n)
    lens = [L] + [int(x) for x in rng.integers(0, L, S - 1)]
    c = _random_cache(S * n, lens, H, D)
    q = _rows(rng, S, n, H * G, D, dtype, 2.0)
    k, v = _rows(rng, S, n, H, D, dtype), _rows(rng, S, n, H, D, dtype)
    old = torch.rand(S, H, c.shape[3], device="cuda") if mass else None
    new = torch.empty_like(old) if mass else None
    for scale in (D ** -0.5, -0.05):
        out = c.attention(q, k, v, scale=scale, mass=old, mass_out=new)
        _long_check(c, q, k, v, scale, out, range(H), sorted({0, 1, S - 1}), old, new)
        assert torch.equal(out, c.attention(q, k, v, scale=scale, mass=old, mass_out=new))   # no dependence on timing
    assert c.check() == 0


def test_a_million_tokens_past_four_gigabytes():
    """Twenty heads of 2^20 tokens of 128: page addresses beyond 32 bits, hundreds of pages for a worker, every
    length the format allows; attention, selection and a sparse read of the last head."""
    L = 64 * 16384 + 63
    rng = np.random.default_rng(0)
    H, D = 20, 128
    c = _random_cache(3, [L], H, D, max_pages=16384)
    assert c.tensors["codes"].numel() > 1 << 32
    q, k = _rows(rng, 1, 1, H, D, "fp32", 2.0), _rows(rng, 1, 1, H, D, "fp32")
    out = c.attention(q, k, k, scale=D ** -0.5)
    _long_check(c, q, k, k, D ** -0.5, out, [0, H - 1], [0])
    c.tensors["sums"].random_(-500, 500)
    pages = c.select(q, 50, first_pages=1, last_pages=1)
    h, t = H - 1, c.tensors
    phys = t["table"][0, h].long()
    code, _ = O.quantize_page(_np(q)[0, 0, h:h + 1])
    dot = (t["sums"][0, h, phys].double() @ torch.from_numpy(code).double().cuda().T).amax(1).float()
    score = (t["scales"][0, h, phys, 0] * dot).cpu().numpy()
    score[0] = score[-1] = np.inf
    want = np.sort(np.argsort(-score, kind="stable")[:50])
    assert pages[0, 0, h].tolist() == want.tolist()
    out = c.attention(q, k, k, scale=D ** -0.5, pages=pages)
    _long_check(c, q, k, k, D ** -0.5, out, [0, H - 1], [0], pages=pages)
    assert c.check() == 0


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_long_sparse_reads(dtype):
    rng = np.random.default_rng(5)
    S, H, G, D, n = 6, 2, 4, 128, 5
    c = _random_cache(9, [20000, 0, 64 * 40, 64 * 39 + 5, 12345, 19999], H, D)
    q = _rows(rng, S, n, H * G, D, dtype, 2.0)
    k, v = _rows(rng, S, n, H, D, dtype), _rows(rng, S, n, H, D, dtype)
    pages = c.select(q, 40, last_pages=1)
    out = c.attention(q, k, v, scale=0.1, pages=pages)
    _long_check(c, q, k, v, 0.1, out, range(H), range(S), pages=pages)


def test_wide_calls_in_a_graph_and_with_empty_sequences():
    """tcgen05 calls captured and replayed with other lengths, counts of zero, an empty cache, a page out of range."""
    rng = np.random.default_rng(71)
    S, H, G, D, n = 3, 1, 16, 64, 12                       # 192 query rows
    c = _random_cache(4, [700, 0, 1300], H, D, max_pages=24)
    q, k, v = _rows(rng, S, n, H * G, D, "bf16"), _rows(rng, S, n, H, D, "bf16"), _rows(rng, S, n, H, D, "bf16")
    counts = _i32([n, n, n])
    out, mass = torch.empty_like(q), torch.zeros(S, H, 24, device="cuda")
    zero = torch.zeros_like(mass)
    c.attention(q, k, v, scale=0.1, counts=counts, out=out, mass=zero, mass_out=mass)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.attention(q, k, v, scale=0.1, counts=counts, out=out, mass=zero, mass_out=mass)
    for lens, cnt in (([700, 0, 1300], [n] * 3), ([64, 1000, 63], [n, 0, n]), ([1535, 1, 5], [1, n, 7]), ([0, 0, 0], [n, 1, n])):
        c.len.copy_(_i32(lens))
        counts.copy_(_i32(cnt))
        out.fill_(9.0)
        graph.replay()
        want, m2 = torch.full_like(out, 9.0), torch.empty_like(mass)
        c.attention(q, k, v, scale=0.1, counts=counts, out=want, mass=zero, mass_out=m2)
        assert torch.equal(out, want) and torch.equal(mass, m2)
        for s in range(S):
            assert (out[s, cnt[s]:] == 9.0).all()
            if cnt[s] == n:
                _long_check(c, q, k, v, 0.1, out, [0], [s], zero, mass)
    assert c.check() == 0
    c.len.copy_(_i32([700, 0, 1300]))
    c.tensors["table"][0, 0, 3] = 24
    c.attention(q, k, v, scale=0.1, out=out)
    assert c.check() == W.FLAG_ERR_TREE
    assert torch.equal(out[1:], c.attention(q, k, v, scale=0.1)[1:])


def test_threads_and_a_given_stream():
    """Two threads on one stream share the workspace that the cache keeps; a call on another stream has its own."""
    import threading
    rng = np.random.default_rng(81)
    c = _random_cache(6, [3000, 900], 2, 128)
    jobs = []
    for n in (1, 24):
        q, k = _rows(rng, 2, n, 8, 128, "fp32"), _rows(rng, 2, n, 2, 128, "fp32")
        jobs.append((q, k, c.attention(q, k, k, scale=0.1)))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    bad = []

    def work(j, stream):
        q, k, want = jobs[j]
        outs = [c.attention(q, k, k, scale=0.1, stream=stream) for _ in range(40)]
        torch.cuda.synchronize()
        bad.extend(1 for o in outs if not torch.equal(o, want))
    threads = [threading.Thread(target=work, args=(j % 2, side if j == 3 else None)) for j in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
