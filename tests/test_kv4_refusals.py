"""Calls on the 4-bit cache, and rotations, whose outputs lie on what they read: refused by the host (CPU)."""
import ctypes
import itertools
import random

import pytest

import w4a8_verify_gb300 as W
from w4a8_verify_gb300 import build as B

ARG = 1


@pytest.fixture(scope="module")
def lib():
    B.build()
    return W.lib()


# pages of 16 x 2 heads of 64 (0x22000 bytes), table, lengths and status word, apart from one another
S, H, D, P, N = 4, 2, 64, 4, 16
PAGES, TABLE, LEN, CTL = 0x1000000, 0x2000000, 0x3000000, 0x4000000
POOL = N * H * 68 * D
DESC = W.KV4CacheDesc(S, H, D, P, N, PAGES, TABLE, LEN, CTL)


@pytest.mark.parametrize("at", [PAGES, PAGES + POOL - 4, PAGES - 4 * S + 4])
def test_new_lengths_on_the_pages(lib, at):
    r = ctypes.byref(W.Rows(0x10000000, 8192, 128, 64))
    for n in (1, 64):
        assert lib.w4a8_kv4_append(DESC, r, r, 0, n, n, None, None, at, None) == ARG


def test_rows_on_what_an_append_writes(lib):
    good, n = W.Rows(0x10000000, 8192, 128, 64), 64
    out = 0x20000000
    last = 4 * ((S - 1) * 8192 + (n - 1) * 128 + 64 + D - 1)        # bytes to the last element
    for data in (PAGES, PAGES + POOL - 4, PAGES - last, out, out + 4 * S - 4, out - last):
        bad = W.Rows(data, 8192, 128, 64)
        for k, v in ((bad, good), (good, bad)):
            assert lib.w4a8_kv4_append(DESC, ctypes.byref(k), ctypes.byref(v), 0, n, n, None, None, out, None) == ARG, hex(data)


def test_only_rows_that_lie_there_are_refused(lib):
    """Random strides, around the pages and the new lengths: exactly the calls one of whose rows lies on them.  (The others are
    refused for another reason, that the rows are more than the pages take: nothing is launched.)"""
    rng = random.Random(1)
    n, out, seen = 64 * P + 1, 0x20000000, [0, 0]
    good = ctypes.byref(W.Rows(0x10000000, n * H * D, H * D, D))
    assert lib.w4a8_kv4_append(DESC, good, good, 0, n, n, None, None, out, None) == 4
    for trial in range(300):
        el, dtype = rng.choice([(4, 0), (2, 1)])
        strides = [rng.choice([0, 1, -1]) * rng.choice([64, 128, 1000, 40000, 1 << 20, rng.randint(1, 1 << 18)]) for _ in range(3)]
        lo, size = rng.choice([(PAGES, POOL), (out, 4 * S)])
        i = [rng.randrange(x) for x in (S, n, H)]                    # a row near one end of what is written
        data = rng.choice([lo - D * el, lo + size]) + el * rng.choice([-1, 0, 0, 1, rng.randint(-300, 300)])
        data -= el * sum(a * b for a, b in zip(i, strides))
        if data <= 0:
            continue
        rows = [data + el * sum(a * b for a, b in zip(x, strides)) for x in itertools.product(range(S), range(n), range(H))]
        touch = any(a < b + c and b < a + D * el for b, c in ((PAGES, POOL), (out, 4 * S)) for a in rows)
        bad = ctypes.byref(W.Rows(data, *strides))
        status = lib.w4a8_kv4_append(DESC, bad, good, dtype, n, n, None, None, out, None)
        assert status == (ARG if touch else 4), (data, strides, touch)
        seen[touch] += 1
    assert min(seen) > 40


def _attn(out, n=2, heads=4, counts=None, mask=None, strides=None):
    at = lambda base, h: W.Rows(base, n * h * D, h * D, D)  # noqa: E731
    q, k, v = at(0x10000000, heads), at(0x18000000, H), at(0x1c000000, H)
    return W.KV4Attn(n, heads, 0, 0.1, q, W.Rows(out, *(strides or (n * heads * D, heads * D, D))), k, v, counts, mask)


def test_attention_output_on_what_it_reads(lib):
    ws, need = 0x40000000, ctypes.c_size_t()
    assert lib.w4a8_kv4_attention_workspace_bytes(DESC, ctypes.byref(_attn(0x20000000)), ctypes.byref(need)) == 0
    counts, mask, n, heads = 0x50000000, 0x60000000, 2, 4
    call = lambda a, b=need.value: lib.w4a8_kv4_attention(DESC, ctypes.byref(a), ws, b, None)  # noqa: E731
    end = 4 * (S * n * heads * D - 1)                                # bytes to the output's last element
    for at, size in ((PAGES, POOL), (TABLE, 4 * S * P), (LEN, 4 * S), (CTL, 4), (counts, 4 * S), (mask, 8 * S * n), (ws, need.value)):
        for out in (at, at + size - 4, at - end):
            assert call(_attn(out, counts=counts, mask=mask)) == ARG, hex(out)
        # one row of many on it, the others around
        assert call(_attn(at + size - 4 - 3 * (1 << 20) * 4, counts=counts, mask=mask, strides=(1 << 20, 1 << 16, 1 << 10))) == ARG


def test_rotation_outputs_on_its_tables(lib):
    S, n, Hq, Hk, D, axes = 2, 3, 4, 2, 64, 3
    names = (("turns", 8 * 32), ("axis", 32), ("pos", 4 * axes * S * n), ("start", 4 * S), ("counts", 4 * S), ("q_gain", 4 * D),
             ("k_gain", 4 * D))
    at = {name: 0x100000 * (i + 1) for i, (name, _) in enumerate(names)}
    rows = lambda base, h: W.Rows(base, n * h * D, h * D, D)  # noqa: E731
    for name, size in names:
        for out, h in (("q_out", Hq), ("k_out", Hk)):
            end = 4 * (S * n * h * D - 1)
            for place in (at[name], at[name] + (size - 1) // 4 * 4, at[name] - end):
                a = W.QKRotaryArgs(S, n, Hq, Hk, D, D, axes, 0, 0, 1, 1e-6, 1.0, *at.values(), rows(0x10000000, Hq),
                                   rows(0x20000000, Hq), rows(0x30000000, Hk), rows(0x40000000, Hk))
                getattr(a, out).data = place
                assert lib.w4a8_qk_rotary(ctypes.byref(a), None) == ARG, (name, out, hex(place))


def test_read_outputs_on_what_it_reads(lib):
    n, far, first, length = 64, 0x70000000, 0x50000000, 0x60000000
    bytes_ = S * n * H * D * 2
    call = lambda k, v: lib.w4a8_kv4_read(DESC, first, length, n, 1, k, v, None)  # noqa: E731
    for at, size in ((PAGES, POOL), (TABLE, 4 * S * P), (LEN, 4 * S), (CTL, 4), (first, 4 * S), (length, 4 * S), (far, bytes_)):
        for out in (at, at + size - 16 if size > 16 else at, at - bytes_ + 16):
            assert call(out, far) == ARG and call(far, out) == ARG, hex(out)
