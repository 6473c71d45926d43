"""The 8-bit key/value cache, further calls: many of the same, beside other work, and those that a wait cuts short.

Bounds as in test_gpu_kv8.py.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import w4a8_verify_gb300 as W
from test_gpu_kv8 import _i32, _long_check, _random_cache, _rows

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
