"""The 8-bit cache's oracle against closed forms, and the host-side refusals of its entry points (CPU)."""
import ctypes

import numpy as np
import pytest

import w4a8_verify_gb300 as W
from oracle import kv8 as O
from w4a8_verify_gb300 import build as B


@pytest.fixture(scope="module")
def lib():
    B.build()
    return W.lib()


@pytest.mark.parametrize("D", [64, 128])
def test_page_bytes_are_a_permutation(D):
    for byte in (O.key_byte, O.value_byte):
        assert sorted(O.byte_order(D, byte).reshape(-1)) == list(range(64 * D))


def test_page_quantiser_closed_forms():
    x = np.zeros((64, 64), np.float32)
    c, s = O.quantize_page(x)
    assert s == 0 and not c.any()
    x[3, 5], x[0, 0], x[1, 1], x[2, 2] = -127.0, 2.5, 1.5, 0.5     # scale 1: halves go to the even code
    c, s = O.quantize_page(x)
    assert s == 1 and (c[3, 5], c[0, 0], c[1, 1], c[2, 2]) == (-127, 2, 2, 0)
    x[9, 9] = np.inf
    c, s = O.quantize_page(x)
    assert np.isnan(s) and not c.any()


def test_attention_special_cases():
    c = O.Cache(1, 1, 64, 4)
    q = np.ones(64)
    out, _, _ = O.attention(c, 0, 0, q, np.zeros((0, 64)), np.zeros((0, 64)), 0, 1.0)
    assert not out.any()                                            # nothing to see
    v = np.arange(128, dtype=np.float64).reshape(2, 64)
    out, _, _ = O.attention(c, 0, 0, q, np.zeros((2, 64)), v, 0b10, 1.0)
    assert np.array_equal(out, v[1])                                # one visible row
    out, _, _ = O.attention(c, 0, 0, q, np.zeros((2, 64)), v, 0b11, 1.0)
    assert np.allclose(out, v.mean(axis=0))                         # equal logits


def test_select_and_evict_tie_rules():
    assert O.evict([1.0, 2.0, 2.0, 0.5], 2, 0, 0) == ([1, 2], [0, 3])
    assert O.evict([1.0, 1.0, 1.0, 1.0], 2, 0, 0) == ([0, 1], [2, 3])
    assert O.evict([0.0, 5.0, 9.0, 0.0], 2, 1, 1) == ([0, 3], [1, 2])
    c = O.Cache(1, 1, 64, 8)
    c.append(0, np.ones((64 * 5, 1, 64)), np.ones((64 * 5, 1, 64)))
    assert O.select(c, 0, 0, np.ones((2, 64), np.float32), 3, 0, 0) == [0, 1, 2]
    assert O.select(c, 0, 0, np.ones((2, 64), np.float32), 3, 0, 2) == [0, 3, 4]


def _desc(S=1, H=2, D=64, P=4, ptr=0x10000):
    return W.KV8CacheDesc(S, H, D, P, ptr, ptr, ptr, ptr, ptr, ptr, ptr)


def test_refusals_without_a_gpu(lib):
    """Every bad argument is refused before any launch (the pointers here are never read)."""
    sz, by = ctypes.c_size_t(), (ctypes.c_size_t * 7)()
    ref = ctypes.byref
    assert lib.w4a8_kv8_bytes(ref(_desc(2, 3, 64, 5)), by) == 0
    assert list(by) == [2 * 3 * 5 * 2 * 4096, 2 * 3 * 5 * 8, 2 * 3 * 5 * 128, 2 * 3 * 2 * 64 * 256, 2 * 3 * 5 * 4, 8, 4]
    for bad in (_desc(S=0), _desc(S=4097), _desc(H=0), _desc(H=1025), _desc(D=96), _desc(P=0), _desc(P=16385),
                _desc(S=4096, H=1024, P=16384)):
        assert lib.w4a8_kv8_bytes(ref(bad), by) == 2
        assert lib.w4a8_kv8_reset(ref(bad), None) == 2
    null = _desc()
    null.tail = None
    assert lib.w4a8_kv8_reset(ref(null), None) == 1
    odd = _desc()
    odd.codes = 0x10010
    assert lib.w4a8_kv8_reset(ref(odd), None) == 1
    c, rows = _desc(), W.Rows(0x10000, 1, 1, 1)
    p = ctypes.c_void_p(0x10000)

    def append(k=rows, v=rows, dtype=0, n_src=4, n=4, index=None, out=p):
        return lib.w4a8_kv8_append(ref(c), ref(k), ref(v), dtype, n_src, n, None, index, out, None)
    assert append(k=W.Rows()) == 1 and append(dtype=2) == 1 and append(n=0) == 1 and append(out=None) == 1
    assert append(k=W.Rows(0x10002, 1, 1, 1)) == 1                  # fp32 rows off their alignment
    assert append(n=5) == 2 and append(n=2000, index=p) == 2
    assert append(n_src=400, n=400) == 4                            # more than the cache holds
    assert lib.w4a8_kv8_read(ref(c), None, None, 1, p, p, None) == 1
    assert lib.w4a8_kv8_read(ref(c), p, None, 0, p, p, None) == 1

    def attn(**kw):
        a = W.KV8Attn(4, 4, 0, 1.0, rows, rows, rows, rows)
        ws = kw.pop("ws", p)
        for k, v in kw.items():
            setattr(a, k, v)
        st = lib.w4a8_kv8_attention_workspace_bytes(ref(c), ref(a), ref(sz))
        return st or lib.w4a8_kv8_attention(ref(c), ref(a), ws, kw.get("bytes", 0), None)
    assert attn(n=0) == 2 and attn(n=65) == 2 and attn(n_heads=3) == 2 and attn(n_heads=34) == 2
    assert attn(dtype=7) == 1 and attn(k=W.Rows()) == 1             # k and v come together
    assert attn(pages=0x10000, top_k=0) == 2 and attn(pages=0x10000, top_k=16385) == 2
    assert attn(pages=0x10000, top_k=2, mass_out=0x10000) == 3
    assert attn(q=W.Rows()) == 1 and attn(ws=None) == 1 and attn(ws=ctypes.c_void_p(0x10010)) == 1
    assert attn(out=W.Rows(0x10000, 1, 0, 1)) == 1                  # rows on one another
    assert attn() == 4                                              # a workspace of no bytes
    a = W.KV8Attn(4, 4, 0, 1.0, rows)

    def select(top_k=2, first=0, last=0, out=p, a=a):
        return lib.w4a8_kv8_select(ref(c), ref(a), top_k, first, last, out, p, 0, None)
    assert select(top_k=0) == 1 and select(first=-1) == 1 and select(last=-1) == 1 and select(out=None) == 1
    assert select(top_k=16385) == 2 and select() == 4 and select(a=W.KV8Attn(0, 4, 0, 1.0, rows)) == 2
    assert lib.w4a8_kv8_evict(ref(c), None, 1, 0, 0, p, p, p, None) == 1
    assert lib.w4a8_kv8_evict(ref(c), p, -1, 0, 0, p, p, p, None) == 1


def test_first_and_last_pages_come_before_infinities():
    inf, nan = float("inf"), float("nan")
    assert O.evict([inf, nan, 1.0, 0.0], 1, 0, 1) == ([3], [0, 1, 2])
    assert O.evict([inf, nan, 1.0, 0.0], 3, 0, 1) == ([0, 1, 3], [2])
    assert O.evict([0.0, inf, inf, 0.0], 2, 2, 1) == ([0, 1], [2, 3])
    c = O.Cache(1, 1, 64, 8)
    x = np.ones((64 * 6, 1, 64))
    x[:64 * 3] = nan
    c.append(0, x, x)
    assert O.select(c, 0, 0, np.ones((2, 64), np.float32), 2, 0, 1) == [0, 5]


def _overlap(seq, row, head, S, n, heads, D):
    """Whether two rows of D elements share one, element by element."""
    at = (np.arange(S)[:, None, None] * seq + np.arange(n)[:, None] * row + np.arange(heads) * head).reshape(-1)
    return len(np.unique(at[:, None] + np.arange(D))) < at.size * D


LAYOUTS = [(64 * 8 - 1, 128, 64), (64 * 6, 64, 65), (64, 64 * 4, 63), (64 * 8, 64 * 4 - 1, 64), (4096, 64, 64 * 2 - 1),
           (64 * 3, 64 * 5, 64 * 4 + 1), (-64 * 7, 64 * 2, 64), (130, 64 * 3, 64 * 6), (1 << 62, 1, 64), (64, -64, 1 << 40)]


@pytest.mark.parametrize("seq,row,head", LAYOUTS, ids=str)
def test_overlapping_output_rows_are_refused(lib, seq, row, head):
    """Rows of out that share elements, by any of their strides (3 sequences, 2 rows, 4 heads of 64)."""
    if pytest.importorskip("torch").cuda.is_available():
        pytest.skip("the pointers of an accepted call would be read")
    assert abs(seq) > 1 << 30 or abs(head) > 1 << 30 or _overlap(seq, row, head, 3, 2, 4, 64)
    rows = W.Rows(0x100000, 4096, 512, 64)
    a = W.KV8Attn(2, 4, 0, 1.0, rows, W.Rows(0x100000, seq, row, head))
    p = ctypes.c_void_p(0x100000)
    assert lib.w4a8_kv8_attention(ctypes.byref(_desc(3, 2, 64, 4)), ctypes.byref(a), p, 1 << 40, None) == 1


@pytest.mark.parametrize("dtype", [0, 1])
def test_size_limit_of_the_header(lib, dtype):
    """n_seqs * n_kv_heads * B < 2^22 with B blocks of at least the header's rows: such calls are accepted, whatever the number
    of rows; so is B * pages of a row up to 2^31."""
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "w4a8.h")).read()
    least = int(re.search(r"at least (\d+) \(fp32\) or (\d+) \(bf16\)\s+(?:\* )?query rows", text).group(1 + dtype))
    rows, sz = W.Rows(0x100000, 4096, 512, 64), ctypes.c_size_t()
    for G in (1, 4, 7, 16):
        for n in range(1, 65):
            B = -(-n * G // least)
            H = min(1024, ((1 << 22) - 1) // (4096 * B))
            a = W.KV8Attn(n, H * G, dtype, 1.0, rows, rows)
            size = lib.w4a8_kv8_attention_workspace_bytes
            for pages in (1, min(511, ((1 << 31) - 1) // (4096 * H * B))):
                assert size(ctypes.byref(_desc(4096, H, 64, pages)), ctypes.byref(a), ctypes.byref(sz)) == 0, (G, n, H, pages)


@pytest.mark.parametrize("dtype,rows", [(0, 4), (1, 8)])
def test_the_kernel_of_a_call_goes_by_its_tiles(lib, dtype, rows):
    """Row counts of the same tiles take the same kernel (seen in the scratch they need), at every length near the crossover
    of 2^21 tile-page-dims: head size 128, one KV head, no new rows."""
    r, sz = W.Rows(0x100000, 4096, 512, 64), ctypes.c_size_t()

    def scratch(n, pages):
        a = W.KV8Attn(n, 1, dtype, 1.0, r, r)
        assert lib.w4a8_kv8_attention_workspace_bytes(ctypes.byref(_desc(1, 1, 128, pages)), ctypes.byref(a), ctypes.byref(sz)) == 0
        return sz.value
    for tiles in range(32 // rows + 1, 64 // rows + 1):
        at = -(-(1 << 21) // (tiles * 128))                     # the first length of the wide kernel
        for pages in (at - 1, at):
            assert len({scratch(n, pages) for n in range((tiles - 1) * rows + 1, tiles * rows + 1)}) == 1, (tiles, pages)
        assert scratch(tiles * rows, at - 1) != scratch(tiles * rows, at)


def test_pointers_off_their_alignment_are_refused(lib):
    """Lengths, counts, lists, masks and masses too: a kernel would fault on them.  (No pointer here is read: every call is
    refused, by a workspace of no bytes at the latest.)"""
    if pytest.importorskip("torch").cuda.is_available():
        pytest.skip("the pointers of an accepted call would be read")
    c, p, odd = ctypes.byref(_desc(1, 2, 64, 4)), ctypes.c_void_p(0x100000), ctypes.c_void_p(0x100002)
    rows = W.Rows(0x100000, 4096, 512, 64)
    r = ctypes.byref(rows)
    assert lib.w4a8_kv8_append(c, r, r, 0, 4, 4, odd, None, p, None) == 1
    assert lib.w4a8_kv8_append(c, r, r, 0, 4, 4, None, odd, p, None) == 1
    assert lib.w4a8_kv8_append(c, r, r, 0, 4, 4, None, None, odd, None) == 1
    assert lib.w4a8_kv8_read(c, odd, None, 4, p, p, None) == 1 and lib.w4a8_kv8_read(c, p, odd, 4, p, p, None) == 1
    for args in ((odd, p, p, p), (p, odd, p, p), (p, p, odd, p), (p, p, p, odd)):
        assert lib.w4a8_kv8_evict(c, args[0], 1, 0, 0, *args[1:], None) == 1
    for name, value in (("counts", 0x100002), ("mask", 0x100004), ("pages", 0x100001), ("mass", 0x100003), ("mass_out", 0x100002)):
        a = W.KV8Attn(4, 4, 0, 1.0, rows, rows, rows, rows, top_k=1)
        assert lib.w4a8_kv8_attention(c, ctypes.byref(a), p, 0, None) == 4
        if name == "mass":
            a.mass_out = 0x100000
        setattr(a, name, value)
        assert lib.w4a8_kv8_attention(c, ctypes.byref(a), p, 0, None) == 1, name
    a = W.KV8Attn(4, 4, 0, 1.0, rows)
    assert lib.w4a8_kv8_select(c, ctypes.byref(a), 1, 0, 0, p, p, 0, None) == 4
    assert lib.w4a8_kv8_select(c, ctypes.byref(a), 1, 0, 0, odd, p, 0, None) == 1
    a.counts = 0x100002
    assert lib.w4a8_kv8_select(c, ctypes.byref(a), 1, 0, 0, p, p, 0, None) == 1
