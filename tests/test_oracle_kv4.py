"""The 4-bit cache's and the rotation's oracles against closed forms, and the host-side refusals of their entry points (CPU)."""
import ctypes

import numpy as np
import pytest

import w4a8_verify_gb300 as W
from oracle import kv4 as O
from oracle import rotary as R
from w4a8_verify_gb300 import build as B


@pytest.fixture(scope="module")
def lib():
    B.build()
    return W.lib()


@pytest.mark.parametrize("D", [64, 128])
def test_places_are_a_permutation(D):
    tok, d = np.meshgrid(np.arange(64), np.arange(D), indexing="ij")
    words, scales = [], []
    for place in (O.key_place, O.value_place):
        w, f, s = place(D, tok, d)
        words += (w * 4 + f).reshape(-1).tolist()
        s = s.reshape(64, D // 32, 32)
        assert (s == s[..., :1]).all()
        scales += s[..., 0].reshape(-1).tolist()
    assert sorted(words) == list(range(2 * 64 * D)) and sorted(scales) == list(range(64 * D, 68 * D))


def test_quantiser_closed_forms():
    x = np.zeros((1, 32), np.float32)
    c, b = O.quantize(x)
    assert b == 0 and not c.any()
    x[0, :4] = -7.0, 2.5, 1.5, 0.5                                   # scale 1: halves go to the even code
    c, b = O.quantize(x)
    assert O.scale_value(int(b[0, 0])) == 1 and c[0, :4].tolist() == [-7, 2, 2, 0]
    x[0, 0] = 7 * 1.0625                                             # halfway between 1 and 1.125: the even one, and code 7
    c, b = O.quantize(x)
    assert O.scale_value(int(b[0, 0])) == 1 and c[0, 0] == 7
    x[0, 0] = 1e30
    c, b = O.quantize(x)
    assert O.scale_value(int(b[0, 0])) == 240 and c[0, 0] == 7 and not c[0, 1:].any()
    x[0, 9] = np.inf
    c, b = O.quantize(x)
    assert b == 255 and not c.any()
    x[:] = 0
    x[0, 0] = 7 * 2.0 ** -18                                         # half of the smallest scale: 0, the even one
    assert O.quantize(x)[1] == 0
    x[0, 0] = 7 * 2.0 ** -17 * 1.6
    assert O.quantize(x)[1] == 2


def test_scale_values_are_exact_half_floats():
    bits = (np.arange(184, dtype=np.uint16) << 7).view(np.float16)
    assert np.array_equal(bits.astype(np.float64), O.VALUES) and (np.diff(O.VALUES) > 0).all()
    for s in O.VALUES:                                               # what the kernels rely on: 264 s, 24 s and c s in f16
        for f in (264, 24, *range(8)):
            assert float(np.float16(f * s)) == f * s


def test_codes_without_a_division():
    """The kernels decide a code by x fl(1 / s) and the exact remainder x - f s: the same as rint of the IEEE quotient."""
    rng = np.random.default_rng(0)
    f32 = np.float32
    for s in O.VALUES[[1, 2, 7, 8, 60, 101, 103, 107, 111, 183]].astype(f32):
        k = rng.integers(-7, 7, 4000)
        x = np.concatenate([(rng.standard_normal(4000) * 3 * s).astype(f32), ((k + 0.5) * s).astype(f32)])
        x = np.clip(np.concatenate([x, np.nextafter(x, f32(np.inf)), np.nextafter(x, f32(-np.inf))]), -7 * s, 7 * s).astype(f32)
        want = np.clip(np.rint((x / s).astype(f32)), -7, 7)
        for inv in (np.nextafter(f32(1) / s, f32(0)), f32(1) / s, np.nextafter(f32(1) / s, f32(np.inf))):
            f = np.rint(x.astype(np.float64) * inv)                  # one rounding to a whole number
            d = x.astype(np.float64) - f * s
            over = (np.abs(d) > s / 2) | ((np.abs(d) == s / 2) & (f % 2 != 0))
            assert np.array_equal(f + np.where(over, np.sign(d), 0), want)


def test_attention_special_cases():
    none, q = np.zeros((0, 64)), np.ones(64)
    out, _ = O.attention(none, none, q, none, none, 0, 1.0)
    assert not out.any()                                             # nothing to see
    v = np.arange(128, dtype=np.float64).reshape(2, 64)
    assert np.array_equal(O.attention(none, none, q, np.zeros((2, 64)), v, 0b10, 1.0)[0], v[1])
    assert np.allclose(O.attention(none, none, q, np.zeros((2, 64)), v, 0b11, 1.0)[0], v.mean(axis=0))


def test_turn_closed_forms():
    x = np.arange(1.0, 9.0)
    inv = np.array([np.pi / 2, np.pi])
    assert np.allclose(R.turn(x, [1, 1], inv), [-3, -2, 1, -4, 5, 6, 7, 8])
    assert np.allclose(R.turn(x, [1, 1], inv, neighbours=True), [-2, 1, -3, -4, 5, 6, 7, 8])
    assert np.allclose(R.turn(x, [0, 0], inv, factor=2.0), [2, 4, 6, 8, 5, 6, 7, 8])
    y = R.turn(np.full(4, 3.0), [0], np.array([1.0]), eps=0.0, gain=np.array([1.0, 2, 3, 4]))
    assert np.allclose(y, [1, 2, 3, 4])


# ---------------------------------------------------------------------------------------- refusals

def _desc(S=1, H=2, D=64, P=4, N=4, ptr=0x10000):
    return W.KV4CacheDesc(S, H, D, P, N, ptr, ptr, ptr, ptr)


def _attn(n=1, heads=4, dtype=0, ptr=0x100000, D=64, k=True, H=2):
    q = W.Rows(ptr, n * heads * D, heads * D, D)
    out = W.Rows(ptr + 0x1000000, n * heads * D, heads * D, D)
    kv = W.Rows(ptr + 0x2000000 if k else 0, n * H * D, H * D, D)
    return W.KV4Attn(n, heads, dtype, 1.0, q, out, kv, kv, None, None)


def test_cache_dimensions(lib):
    b = (ctypes.c_size_t * 4)()
    assert lib.w4a8_kv4_bytes(_desc(3, 2, 128, 5, 7), b) == 0
    assert list(b) == [7 * 2 * 68 * 128, 3 * 5 * 4, 3 * 4, 4]
    for bad in (_desc(S=0), _desc(S=4097), _desc(H=0), _desc(H=1025), _desc(D=96), _desc(D=32), _desc(P=0), _desc(P=16385),
                _desc(N=0), _desc(H=1024, N=1 << 21)):
        assert lib.w4a8_kv4_bytes(bad, b) == 2
    assert lib.w4a8_kv4_bytes(None, b) == 1
    assert lib.w4a8_kv4_bytes(_desc(), None) == 1


def test_cache_pointers(lib):
    for bad in (_desc(ptr=0), W.KV4CacheDesc(1, 2, 64, 4, 4, 0x10040, 0x10000, 0x10000, 0x10000),
                W.KV4CacheDesc(1, 2, 64, 4, 4, 0x10000, 0x10002, 0x10000, 0x10000)):
        assert lib.w4a8_kv4_reset(bad, None) == 1
        f = ctypes.c_uint32()
        assert lib.w4a8_kv4_check(bad, ctypes.byref(f)) == 1
    assert lib.w4a8_kv4_check(_desc(), None) == 1


def test_append_and_read_refusals(lib):
    c, r = _desc(), W.Rows(0x100000, 128, 128, 64)
    rb, p = ctypes.byref(r), 0x20000
    append = lambda *x: lib.w4a8_kv4_append(c, *x, None)  # noqa: E731
    assert append(None, rb, 0, 1, 1, None, None, p) == 1
    assert append(rb, rb, 2, 1, 1, None, None, p) == 1              # type
    assert append(rb, rb, 0, 1, 1, None, None, None) == 1           # no len_out
    assert append(rb, rb, 0, 1, 0, None, None, p) == 1
    assert append(rb, rb, 0, 1, 2, None, None, p) == 2              # fewer source rows than rows
    assert append(rb, rb, 0, 1, 1025, None, p, p) == 2              # a list that long
    assert append(rb, rb, 0, 300, 257, None, None, p) == 4          # more than the pages hold
    assert append(rb, rb, 0, 1, 1, p + 2, None, p) == 1             # alignment
    assert append(ctypes.byref(W.Rows(0x100002, 128, 128, 64)), rb, 0, 1, 1, None, None, p) == 1
    read = lambda *x: lib.w4a8_kv4_read(c, *x, None)  # noqa: E731
    assert read(None, None, 1, 0, p, p) == 1
    assert read(p, None, 0, 0, p, p) == 1
    assert read(p, None, 1, 7, p, p) == 1
    assert read(p, None, 1, 0, p + 8, p) == 1
    assert read(p, None, 257, 0, p, p) == 4


def test_attention_refusals(lib):
    c, n = _desc(), ctypes.c_size_t()
    size = lambda a, d=c: lib.w4a8_kv4_attention_workspace_bytes(d, ctypes.byref(a), ctypes.byref(n))  # noqa: E731
    assert size(_attn()) == 0 and n.value >= W.KV4_TICKETS
    for a in (_attn(n=0), _attn(n=65), _attn(heads=3), _attn(heads=0), _attn(heads=34)):
        assert size(a) == 2
    assert size(_attn(dtype=3)) == 1
    a = _attn()
    a.v.data = 0
    assert size(a) == 1                                             # keys without values
    assert size(_attn(n=64, heads=16 * 1024), _desc(S=4096, H=1024, P=16384)) == 2
    call = lambda a, ws=0x4000000, b=1 << 30: lib.w4a8_kv4_attention(c, ctypes.byref(a), ws, b, None)  # noqa: E731
    assert call(_attn(), ws=0) == 1 and call(_attn(), ws=0x4000080) == 1
    assert call(_attn(), b=W.KV4_TICKETS) == 4
    a = _attn(n=2)
    a.out.row = 64                                                  # rows of out on one another
    assert call(a) == 1
    a = _attn(n=2)
    a.out.data = a.q.data                                           # out on q
    assert call(a) == 1
    a.out.data = a.k.data
    assert call(a) == 1
    a = _attn()
    a.mask = 0x10004
    assert call(a) == 1
    assert lib.w4a8_kv4_attention_inject_timeout(c, ctypes.byref(_attn()), 0x4000000, 1 << 30, -1, None) == 1


def _rotary(S=2, n=3, Hq=4, Hk=2, D=64, rot=64, axes=1, dtype=0, base=0x1000000, gap=0x1000000):
    q = W.Rows(base, n * Hq * D, Hq * D, D)
    k = W.Rows(base + 2 * gap, n * Hk * D, Hk * D, D)
    return W.QKRotaryArgs(S, n, Hq, Hk, D, rot, axes, 0, dtype, 1, 1e-6, 1.0, 0x10000, None, None, None, None, None, None, q,
                          W.Rows(base + gap, q.seq, q.row, q.head), k, W.Rows(base + 3 * gap, k.seq, k.row, k.head))


def test_rotary_refusals(lib):
    call = lambda a: lib.w4a8_qk_rotary(ctypes.byref(a), None)  # noqa: E731
    for kw in (dict(S=0), dict(n=0), dict(Hq=0), dict(Hk=-1), dict(D=24), dict(D=272), dict(rot=80), dict(rot=8), dict(axes=0),
               dict(axes=5), dict(S=1 << 20, n=1 << 10)):
        assert call(_rotary(**kw)) == 2, kw
    assert call(_rotary(dtype=2)) == 1 and lib.w4a8_qk_rotary(None, None) == 1
    for field, x in (("turns", None), ("eps", -1.0), ("eps", float("nan")), ("factor", float("inf")), ("pos", 0x10002),
                     ("q_gain", 0x10001), ("turns", 0x10004)):
        a = _rotary()
        setattr(a, field, x)
        assert call(a) == 1, field
    for name, x in (("q", 0), ("k_out", 0), ("q_out", 0x2000002)):
        a = _rotary()
        getattr(a, name).data = x
        assert call(a) == 1, name
    # outputs on inputs or outputs in another way than row by row
    for out, on, off in (("q_out", "q", 64 * 4), ("q_out", "k", 0), ("k_out", "q", 64 * 4), ("k_out", "q_out", 0), ("k_out", "k", 4)):
        a = _rotary()
        getattr(a, out).data = getattr(a, on).data + off
        assert call(a) == 1, (out, on)
    a = _rotary()
    a.q_out.row = 64
    assert call(a) == 1


def test_rotary_turns(lib):
    inv = np.array([0.0, 1.0, 2 * np.pi, np.pi, -np.pi / 2, 1e-300, 1e6])
    out = np.zeros(len(inv), np.uint64)
    assert lib.w4a8_rotary_turns(inv.ctypes.data, len(inv), out.ctypes.data) == 0
    want = [0.0, 1 / (2 * np.pi), 0.0, 0.5, 0.75, 0.0, (1e6 / (2 * np.pi)) % 1.0]
    got = out.astype(np.float64) / 2.0 ** 64
    assert np.all(np.abs((got - want + 0.5) % 1.0 - 0.5) < 1e-10)
    bad = np.array([np.nan])
    assert lib.w4a8_rotary_turns(bad.ctypes.data, 1, out.ctypes.data) == 1
    assert lib.w4a8_rotary_turns(None, 1, out.ctypes.data) == 1


def test_rotary_arguments_in_python():
    for kw in (dict(head_dim=24), dict(head_dim=512), dict(head_dim=64, rot_dim=80), dict(head_dim=64, rot_dim=8),
               dict(head_dim=64, inv_freq=[1.0]), dict(head_dim=64, axis=[0] * 31), dict(head_dim=64, axis=[4] * 32),
               dict(head_dim=64, axis=[-1] * 32)):
        with pytest.raises(ValueError):
            W.Rotary(device="cpu", **kw)
    with pytest.raises(ValueError):
        W.Rotary(64, device="cpu")                                  # no CPU path
