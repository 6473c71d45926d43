"""Norm and rotation of queries and keys through the C ABI against the definition (oracle/rotary.py, 64 bits), and a run of
the serving operators together.

Bounds: the angle's cosine and sine are off by less than 2^-22 of 1 (what is left of the angle, at most pi / 4, is rounded to
fp32 and goes through a function of 2 ulp; the tables' frequencies are rounded to 64-bit floating point, so a position p adds
2 pi p 2^-54 f); a turned pair of size m by 2^-22 m for them, 2^-23 m for its two products and their sum.  The norm's sum
of D / LPH = 16 products and at most four exchanges is off by 20 2^-24, half of which reaches its root, plus two products:
2^-20.  So |y - ref| <= 2^-19 m factor in fp32, and half a step (2^-8 of the value) more in bf16.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import w4a8_verify_gb300 as W
from oracle import kv4 as O
from oracle import rotary as R

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


def _check(x, y, position, inv, rot, neighbours=False, factor=1.0, eps=None, gain=None, rows=None, dtype="fp32"):
    """position(s, j) -> one number for each frequency."""
    xn, yn = _np(x).astype(np.float64), _np(y).astype(np.float64)
    S, n, H, D = xn.shape
    for s in range(S):
        for j in range(n if rows is None else rows[s]):
            for h in range(H):
                want = R.turn(xn[s, j, h], position(s, j), inv, neighbours, factor, eps, gain)
                base = xn[s, j, h] if eps is None else R.turn(xn[s, j, h], [], [], False, 1.0, eps, gain)
                size = np.abs(base)
                a, b = (slice(0, rot, 2), slice(1, rot, 2)) if neighbours else (slice(0, rot // 2), slice(rot // 2, rot))
                both = np.hypot(base[a], base[b])
                size[a], size[b] = both, both
                size[:rot] *= abs(factor)
                bound = 2.0 ** -19 * size + (2.0 ** -8 * np.abs(want) if dtype == "bf16" else 0)
                err = np.abs(yn[s, j, h] - want)
                assert (err <= bound + 1e-38).all(), (s, j, h, (err / (bound + 1e-38)).max())


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("D, rot", [(64, 64), (128, 128), (128, 64), (80, 80), (96, 32), (256, 256), (16, 16), (112, 0)])
def test_turn(D, rot, neighbours, dtype):
    rng = np.random.default_rng(D + rot)
    S, n, Hq, Hk = 2, 3, 5, 2
    q, k = _rows(rng, S, n, Hq, D, dtype), _rows(rng, S, n, Hk, D, dtype)
    inv = 10000.0 ** (-np.arange(rot // 2) / max(rot // 2, 1))
    start, pos = [5, 70000], rng.integers(0, 50, (S, n))
    g, eps = (1 + 0.3 * rng.standard_normal(D)).astype(np.float32), 1e-5
    rope = W.Rotary(D, rot, neighbours=neighbours)
    at = lambda s, j: np.full(rot // 2, float(start[s] + pos[s, j]))  # noqa: E731
    a, b = rope.apply(q, k, positions=_i32(pos), start=_i32(start))
    _check(q, a, at, inv, rot, neighbours, dtype=dtype)
    _check(k, b, at, inv, rot, neighbours, dtype=dtype)
    a, b = rope.apply(q, k, positions=_i32(pos), start=_i32(start), eps=eps, k_gain=torch.from_numpy(g).cuda())
    _check(q, a, at, inv, rot, neighbours, eps=eps, dtype=dtype)
    _check(k, b, at, inv, rot, neighbours, eps=eps, gain=g, dtype=dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_axes(dtype):
    """Time, height and width by blocks and by turns; a factor; no keys."""
    rng = np.random.default_rng(1)
    S, n, H, D = 2, 7, 3, 128
    q = _rows(rng, S, n, H, D, dtype)
    pos = rng.integers(0, 500, (3, S, n))
    for axis in (np.repeat([0, 1, 2], [16, 24, 24]), np.arange(64) % 3):
        rope = W.Rotary(D, base=1e6, axis=axis, factor=1.25)
        assert rope.n_axes == 3
        y = rope.apply(q, positions=_i32(pos))
        _check(q, y, lambda s, j: pos[axis, s, j], 1e6 ** (-np.arange(64) / 64), D, factor=1.25, dtype=dtype)
        z = rope.apply(q, start=_i32([3, 4]))                       # text: the row's number on every axis
        assert torch.equal(z, W.Rotary(D, base=1e6, factor=1.25).apply(q, start=_i32([3, 4])))


def test_far_positions_are_exact():
    """Frequencies that are binary fractions of a turn: the angle of any 32-bit position is known, and position p gives bit for bit
    what p modulo the period gives.  Negative positions turn back."""
    D, n = 32, 6
    inv = 2 * np.pi * 2.0 ** -np.arange(1.0, 17.0)
    p = np.array([[0, 3, 40000, 65535, 12345, 1]])
    rng = np.random.default_rng(2)
    q = _rows(rng, 1, n, 2, D, "fp32")
    rope = W.Rotary(D, inv_freq=inv)
    near = rope.apply(q, positions=_i32(p))
    _check(q, near, lambda s, j: np.full(16, float(p[s, j])), inv, D)
    for shift in (1 << 16, (1 << 30) + (1 << 16), -(1 << 31)):
        assert torch.equal(rope.apply(q, positions=_i32(p + shift)), near)
        assert torch.equal(rope.apply(q, positions=_i32(p), start=_i32([shift])), near)
    far = _i32([[2 ** 31 - 1] * n])
    assert torch.equal(rope.apply(q, positions=far, start=_i32([2 ** 31 - 1])), rope.apply(q, positions=_i32([[-2] * n])))
    back = rope.apply(near, positions=_i32(-p))
    assert (back - q).abs().max().item() < 1e-5


def test_ordinary_frequencies_at_far_positions():
    """Base 10000 at positions of a million, against angles in exact whole-number arithmetic on the same 64-bit frequencies."""
    from fractions import Fraction
    D, n = 64, 5
    inv = 10000.0 ** (-np.arange(32) / 32)
    p = [1_000_003, 131071, 7, 2 ** 31 - 1, 1 << 20]
    x = torch.zeros(1, n, 1, D, device="cuda")
    x[..., :32] = 1.0
    y = _np(W.Rotary(D, inv_freq=inv).apply(x, positions=_i32([p])))[0, :, 0]
    pi = Fraction(314159265358979323846264338327950288419716939937510, 10 ** 50)
    for j, pos in enumerate(p):
        for i in range(32):
            a = float((Fraction(float(inv[i])) * pos) % (2 * pi))
            lim = 2.0 ** -20 + pos * inv[i] * 2.0 ** -52
            assert abs(y[j, i] - np.cos(a)) < lim and abs(y[j, 32 + i] - np.sin(a)) < lim, (pos, i)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_in_place_in_one_projection_and_padded_rows(dtype):
    """q and k are parts of one tensor and are turned in place, with rows behind the counts left alone; the same bits as from
    separate tensors, whatever the strides and alignment."""
    rng = np.random.default_rng(3)
    S, n, Hq, Hk, D = 3, 4, 6, 2, 64
    base = _rows(rng, S, n, Hq + 2 * Hk, D, dtype)
    counts = [4, 0, 2]
    rope = W.Rotary(D)
    q, k = rope.apply(base[:, :, :Hq].contiguous(), base[:, :, Hq:Hq + Hk].contiguous(), eps=1e-6, start=_i32([1, 2, 3]))
    for layout in range(4):
        if layout == 0:
            x = base.clone()
        elif layout == 1:                                            # heads outside rows
            x = base.transpose(1, 2).contiguous().transpose(1, 2)
        elif layout == 2:                                            # not 16-byte aligned
            x = torch.zeros(S, n, Hq + 2 * Hk, D + 1, dtype=base.dtype, device="cuda")[..., 1:]
            x.copy_(base)
        else:                                                        # rows outside sequences
            x = base.transpose(0, 1).contiguous().transpose(0, 1)
        a, b = x[:, :, :Hq], x[:, :, Hq:Hq + Hk]
        got = rope.apply(a, b, eps=1e-6, start=_i32([1, 2, 3]), counts=_i32(counts), q_out=a, k_out=b)
        assert got[0] is a and got[1] is b
        for s in range(S):
            c = counts[s]
            assert torch.equal(a[s, :c], q[s, :c]) and torch.equal(b[s, :c], k[s, :c])
            assert torch.equal(x[s, c:], base[s, c:]) and torch.equal(x[s, :, Hq + Hk:], base[s, :, Hq + Hk:])


def test_special_values():
    rope = W.Rotary(64)
    x = torch.zeros(1, 6, 1, 64, device="cuda")
    x[0, 1] = 3e38                                                   # squares overflow: the norm is 0
    x[0, 2] = float("nan")
    x[0, 3, 0, 5] = float("inf")
    x[0, 4] = 1e-30
    y = rope.apply(x, eps=1e-6)
    assert not y[0, 0].any() and torch.isfinite(y[0, 4:]).all() and torch.isnan(y[0, 2]).all()
    assert torch.isnan(y[0, 3, 0, 5]) and not torch.isfinite(y[0, 3]).all()
    assert not rope.apply(x[:, :1], eps=0.0, q_gain=torch.full((64,), float("nan"), device="cuda")).isfinite().any()


def test_refusals():
    rng = np.random.default_rng(4)
    rope = W.Rotary(64, axis=np.arange(32) % 2)
    q, k = _rows(rng, 2, 3, 4, 64, "fp32"), _rows(rng, 2, 3, 2, 64, "fp32")
    pos = _i32(np.zeros((2, 2, 3)))
    rope.apply(q, k, positions=pos)
    for args, kw in (((q.half(), k), {}), ((q, k.bfloat16()), {}), ((q[..., :32], k), {}), ((q, k[:1]), {}), ((q.cpu(), k), {}),
                     ((q, k), dict(positions=pos[0])), ((q, k), dict(positions=pos.long())), ((q, k), dict(start=_i32([1]))),
                     ((q, k), dict(q_gain=torch.ones(64, device="cuda"))), ((q,), dict(k_out=k)),
                     ((q, k), dict(eps=1e-6, q_gain=torch.ones(32, device="cuda"))), ((q, k), dict(q_out=q[:, :, :2])),
                     ((q, k), dict(counts=_i32([[1, 1]]))), ((q, k[0]), {})):
        with pytest.raises(ValueError):
            rope.apply(*args, **kw)
    with pytest.raises(W.W4A8Error):
        rope.apply(q, k, eps=-1.0)
    with pytest.raises(W.W4A8Error):
        rope.apply(q, k, q_out=torch.empty(2, 1, 4, 64, device="cuda").expand(2, 3, 4, 64))
    with pytest.raises(W.W4A8Error):
        rope.apply(q, k, k_out=q[:, :, :2])


def test_stream_and_graph():
    rng = np.random.default_rng(5)
    rope = W.Rotary(128)
    q, k = _rows(rng, 2, 300, 8, 128, "bf16"), _rows(rng, 2, 300, 2, 128, "bf16")
    start = _i32([0, 10])
    want = rope.apply(q, k, start=start, eps=1e-6)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = rope.apply(q, k, start=start, eps=1e-6, stream=stream)
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph, a, b = torch.cuda.CUDAGraph(), torch.empty_like(q), torch.empty_like(k)
    with torch.cuda.graph(graph):
        rope.apply(q, k, start=start, eps=1e-6, q_out=a, k_out=b)
    start.copy_(_i32([700, 3]))
    graph.replay()
    want = rope.apply(q, k, start=start, eps=1e-6)
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])


# ------------------------------------------------------------------------------- together

@pytest.mark.parametrize("captured", [False, True])
def test_serving_steps_together(captured):
    """A layer's attention as a server runs it: a prompt, then draft trees: rotate queries and keys at the cache's
    lengths, attend to the cache and the tree, append the accepted path.  Each step against the oracles."""
    rng = np.random.default_rng(6)
    S, H, G, D, n = 3, 2, 4, 64, 5
    rope = W.Rotary(D, base=1e5)
    inv = 1e5 ** (-np.arange(32) / 32)
    gains = [(1 + 0.2 * rng.standard_normal(D)).astype(np.float32) for _ in range(2)]
    gq, gk = (torch.from_numpy(x).cuda() for x in gains)
    cache, ref = W.KV4Cache(S, H, D, 8), O.Cache(S, H, D)
    prompt = [150, 61, 1]
    qkv = _rows(rng, S, max(prompt), (G + 2) * H, D, "fp32")
    counts = _i32(prompt)
    _, k = rope.apply(qkv[:, :, :G * H], qkv[:, :, G * H:-H], eps=1e-6, q_gain=gq, k_gain=gk, counts=counts)
    cache.append(k, qkv[:, :, -H:], counts=counts)
    for s in range(S):
        ref.append(s, _np(k)[s, :prompt[s]], _np(qkv)[s, :prompt[s], -H:])
    # a tree: node 0 the root, 1 and 2 its children, 3 and 4 children of 1
    depth, mask = [0, 1, 1, 2, 2], [0b1, 0b11, 0b101, 0b1011, 0b10011]
    pos, bits = _i32([depth] * S), torch.tensor([mask] * S, dtype=torch.int64, device="cuda")
    path, taken = _i32([[0, 1, 4, 0, 0], [0, 2, 0, 0, 0], [0, 0, 0, 0, 0]]), _i32([3, 2, 1])
    new = torch.empty(S, n, (G + 2) * H, D, device="cuda")
    out, qr, kr = (torch.empty(S, n, h * H, D, device="cuda") for h in (G, G, 1))

    def step():
        rope.apply(new[:, :, :G * H], new[:, :, G * H:-H], positions=pos, start=cache.len, eps=1e-6, q_gain=gq, k_gain=gk,
                   q_out=qr, k_out=kr)
        cache.attention(qr, kr, new[:, :, -H:], scale=0.125, mask=bits, out=out)
        cache.append(kr, new[:, :, -H:], counts=taken, index=path)

    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    for _ in range(4):
        new.copy_(_rows(rng, S, n, (G + 2) * H, D, "fp32"))
        lens = [ref.length(s) for s in range(S)]
        assert cache.len.tolist() == lens
        graph.replay() if captured else step()
        at = lambda s, j: np.full(32, float(lens[s] + depth[j]))  # noqa: E731
        _check(new[:, :, :G * H], qr, at, inv, D, eps=1e-6, gain=gains[0])
        _check(new[:, :, G * H:-H], kr, at, inv, D, eps=1e-6, gain=gains[1])
        q, k, v, o = _np(qr).astype(np.float64), _np(kr), _np(new)[:, :, -H:], _np(out)
        for s in range(S):
            for h in range(G * H):
                kh, vh = ref.held(s, h // G)
                for i in range(n):
                    want, B = O.attention(kh, vh, q[s, i, h], k[s, :, h // G], v[s, :, h // G], mask[i], 0.125)
                    top = max(np.abs(vh).max(), np.abs(v).max())
                    assert np.abs(o[s, i, h] - want).max() <= top * (2.0 ** -17 * B + 2.0 ** -16)
            p = path[s, :int(taken[s])].tolist()
            ref.append(s, k[s, p], v[s, p])
    kk, vv = cache.read(_i32([0] * S), 64 * 8)
    for s in range(S):
        for h in range(H):
            for got, want in zip((kk, vv), ref.held(s, h)):
                assert np.array_equal(_np(got)[s, :ref.length(s), h], want.astype(np.float32))
    assert cache.check() == 0
